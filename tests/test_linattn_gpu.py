"""GPU parity of the linear attention with a decay for each head (kda_linattn_*) against the FP64 oracle.

Bounds.  Rows of 128 channels are held in the 2-norm.  A product's bf16 operand (scores, states) is off by at
most 2^-8 of itself, so a row moves by at most about 2^-8 of the root of the sum of its terms' squares
(roundings are independent; a uniform one's rms is below 0.6 of its bound); the output's own rounding adds 2^-8
of the row.  States are fp32 sums: a 128-token chunk adds in some 24 steps of 2^-23 at most, decays are off by a few
2^-24 of their exponent: 32 2^-23 = 4e-6 in the 2-norm.
"""
import numpy as np
import pytest
import torch

from linear_attention_chunked_gb300 import kda
from oracle import linattn

pytestmark = pytest.mark.gpu

ROW, STATE = 2.0 ** -8, 4e-6
D = 128


def _np(t):
    return None if t is None else t.detach().cpu().double().numpy()


def _case(lens, H, Hk, h0=True, seed=0, slopes=None, strided=True):
    gen = torch.Generator("cpu").manual_seed(seed + sum(lens))
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    T, N = sum(lens), len(lens)
    qkv = rn(T, (2 * Hk + H) * D).bfloat16().cuda()
    q, k, v = qkv.split([Hk * D, Hk * D, H * D], 1)
    q, k, v = q.unflatten(1, (Hk, D)), k.unflatten(1, (Hk, D)), v.unflatten(1, (H, D))
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    slope = -torch.exp2(-8.0 * torch.rand(H, generator=gen)) if slopes is None else torch.tensor(slopes)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    st = lambda: rn(N, H, D, D).cuda() if h0 else None  # noqa: E731
    return dict(q=q, k=k, v=v, slope=slope.float().cuda(), cu=cu, h0=st(), dht=st(), dO=rn(T, H, D).bfloat16().cuda(), scale=D ** -0.5)


def _term_size(qn, kn, vn, slope, cu, s0, scale, back, trans):
    """Root of the sum of the squares of a walk's terms, per row: scores times values within 128 tokens and a query's
    channels times states -- taken together as the walk over squares (every token's term, its channels apart)."""
    a = np.exp(2 * np.asarray(slope, np.float64))
    with np.errstate(divide="ignore"):
        s2 = np.log(a)
    sq = lambda x: None if x is None else (np.swapaxes(x, -1, -2) if trans else x) ** 2  # noqa: E731
    if not back:
        o, _ = linattn.linattn_fwd(qn ** 2, kn ** 2, vn ** 2, s2, cu, h0=sq(s0), scale=1.0)
    else:
        g = linattn.linattn_bwd(kn ** 2, qn ** 2, np.zeros_like(vn), s2, cu, vn ** 2, dht=sq(s0), scale=1.0)
        o = g["dv"]
    return scale * np.sqrt(o.sum(-1))


def _rows(name, got, ref, size):
    err = np.linalg.norm(_np(got) - ref, axis=-1)
    tol = ROW * (np.linalg.norm(ref, axis=-1) + size) + 1e-6
    assert (err <= tol).all(), f"{name}: {float((err / tol).max()):.2f} of the bound"


def _state(name, got, ref):
    err, size = np.linalg.norm(_np(got) - ref), np.linalg.norm(ref)
    assert err <= STATE * size + 1e-30, f"{name}: {err / size:.2e}"


def _run(c, save=True):
    a, kw = (c["q"], c["k"], c["v"], c["slope"], c["cu"]), dict(h0=c["h0"], scale=c["scale"])
    o, ht, saved = kda.kda_linattn_fwd(*a, **kw, save=save)
    return dict(kda.kda_linattn_bwd(*a, c["dO"], **kw, dht=c["dht"], saved=saved), o=o, ht=ht)


def _check(c, got):
    n = {k: _np(c[k]) for k in ("q", "k", "v", "slope", "h0", "dht", "dO")}
    cu, scale, H = c["cu"].tolist(), c["scale"], c["v"].shape[1]
    o, ht = linattn.linattn_fwd(n["q"], n["k"], n["v"], n["slope"], cu, n["h0"], scale)
    g = linattn.linattn_bwd(n["q"], n["k"], n["v"], n["slope"], cu, n["dO"], n["h0"], n["dht"], scale)
    _state("ht", got["ht"], ht)
    _state("dh0", got["dh0"], g["dh0"])
    share = H // n["q"].shape[1]
    Q, K, V, G = np.repeat(n["q"], share, 1), np.repeat(n["k"], share, 1), n["v"], n["dO"]
    _rows("o", got["o"], o, _term_size(Q, K, V, n["slope"], cu, n["h0"], scale, False, False))
    sums = lambda x: np.sqrt((x ** 2).reshape(*x.shape[:1], -1, share).sum(-1))  # noqa: E731  (shared heads' terms)
    _rows("dq", got["dq"], g["dq"], sums(_term_size(G, V, K, n["slope"], cu, n["h0"], scale, False, True)))
    # (dht is not scaled: its square over scale^2 stands in)
    dht = None if n["dht"] is None else n["dht"] / scale
    _rows("dv", got["dv"], g["dv"], _term_size(K, Q, G, n["slope"], cu, dht, scale, True, False))
    _rows("dk", got["dk"], g["dk"], sums(_term_size(V, G, Q, n["slope"], cu, dht, scale, True, True)))


CASES = [([1], 1, 1, True), ([37], 2, 2, False), ([1, 0, 777, 127, 128, 129, 300], 6, 2, True), ([255, 256, 257], 3, 1, False),
         ([64, 65, 63, 0, 0, 2], 4, 4, True), ([513, 512, 511], 2, 2, True), ([1100], 4, 2, True), ([2100, 30], 2, 2, False)]


@pytest.mark.parametrize("lens,H,Hk,h0", CASES)
def test_forward_and_backward(lens, H, Hk, h0):
    c = _case(lens, H, Hk, h0)
    got = _run(c)
    _check(c, got)
    again = _run(c)
    assert all(torch.equal(got[k], again[k]) for k in got)
    replay = _run(c, save=False)
    assert all(torch.equal(got[k], replay[k]) for k in got)


def test_decays_of_every_kind():
    # no decay, one that forgets within a token, none kept at all, and growth
    c = _case([300, 140], 5, 5, True, slopes=[0.0, -30.0, float("-inf"), 0.01, -1e-4])
    _check(c, _run(c))


def test_dense_rows_and_shared_heads_are_the_same_numbers():
    c = _case([200, 77], 4, 1, True)
    d = dict(c, q=c["q"].expand(-1, 4, -1).contiguous(), k=c["k"].expand(-1, 4, -1).contiguous(), v=c["v"].contiguous())
    a, b = _run(c), _run(d)
    assert all(torch.equal(a[k], b[k]) for k in ("o", "ht", "dv", "dh0"))
    for k in ("dq", "dk"):  # bf16 parts of four heads added: each off by 2^-8 of itself at most
        _rows(k, a[k], _np(b[k]).sum(1, keepdims=True), np.linalg.norm(_np(b[k]), axis=-1).sum(1, keepdims=True))


@pytest.mark.parametrize("lens", [[700, 5, 1300, 128], [600, 600]])
def test_a_document_alone_and_in_a_pack(lens):
    c = _case(lens, 3, 3, True)
    whole = _run(c)
    for i in range(len(lens)):
        r = slice(sum(lens[:i]), sum(lens[:i + 1]))
        one = dict(c, cu=torch.tensor([0, lens[i]], dtype=torch.int32, device="cuda"), h0=c["h0"][i:i + 1], dht=c["dht"][i:i + 1],
                   **{k: c[k][r] for k in ("q", "k", "v", "dO")})
        got = _run(one)
        for k in ("o", "dq", "dk", "dv"):
            assert torch.equal(got[k], whole[k][r]), (k, i)
        for k in ("ht", "dh0"):
            assert torch.equal(got[k][0], whole[k][i]), (k, i)


def test_non_finite_rows_stay_in_their_document():
    lens = [130, 70, 200]
    c = _case(lens, 2, 2, True)
    want = _run(c)
    for bad in (float("nan"), float("inf")):
        d = {k: (x.clone() if torch.is_tensor(x) else x) for k, x in c.items()}
        for k in ("q", "k", "v", "dO"):
            d[k][130:200] = bad
        d["h0"][1] = bad
        d["dht"][1] = bad
        got = _run(d)
        for k in ("o", "dq", "dk", "dv"):
            assert torch.equal(got[k][:130], want[k][:130]) and torch.equal(got[k][200:], want[k][200:]), k
            assert not torch.isfinite(got[k][130:200].float()).any(), k
        for k in ("ht", "dh0"):
            assert torch.equal(got[k][0], want[k][0]) and torch.equal(got[k][2], want[k][2]), k


def test_causal_within_and_between_chunks():
    # a later token's values change no earlier row
    c = _case([400], 2, 2, False)
    o, _, _ = kda.kda_linattn_fwd(c["q"], c["k"], c["v"], c["slope"], c["cu"])
    for t in (399, 256, 200, 128, 127, 1):
        k, v = c["k"].clone(), c["v"].clone()
        k[t:], v[t:] = 3.0, -2.0
        o2, _, _ = kda.kda_linattn_fwd(c["q"], k, v, c["slope"], c["cu"])
        assert torch.equal(o2[:t], o[:t]) and not torch.equal(o2[t:], o[t:])


def test_no_tokens():
    c = _case([0, 0], 2, 1, True)
    got = _run(c)
    assert torch.equal(got["ht"], c["h0"]) and torch.equal(got["dh0"], c["dht"]) and got["o"].shape == (0, 2, D)
    c = _case([0], 2, 1, False)
    assert not _run(c)["ht"].any()


def test_malformed_offsets_are_reported():
    c = _case([100, 60], 2, 2, False)
    ws = torch.empty(kda.kda_linattn_workspace_size(160, 2, 2, 2, kda.KDA_OP_BWD_REPLAY)[0], dtype=torch.uint8, device="cuda")
    a = (c["q"], c["k"], c["v"], c["slope"])
    for cu in ([0, 200, 160], [0, 100, 159], [1, 100, 160], [0, 120, 100], [0, -5, 160], [0, 2 ** 31 - 1, 160]):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        kda.kda_linattn_fwd(*a, cu, save=False, ws=ws)
        assert kda.kda_read_device_status(ws) == kda.KDA_ERR_DEVICE_CHECK
        kda.kda_linattn_bwd(*a, cu, c["dO"], ws=ws)
        assert kda.kda_read_device_status(ws) == kda.KDA_ERR_DEVICE_CHECK
    kda.kda_linattn_fwd(*a, c["cu"], save=False, ws=ws)
    assert kda.kda_read_device_status(ws) == kda.KDA_OK


def test_gradient_against_differences():
    # o is linear in q, k, v and h0 apart: central differences are exact but for the outputs' roundings, each row's
    # 2^-8 of its terms and independent, weighted by dO
    c = _case([150, 20], 2, 1, True)
    g = _run(c)
    size = float(_run(c)["o"].float().norm())
    gen = torch.Generator("cuda").manual_seed(5)
    for name, got in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("h0", "dh0")):
        d = torch.randn(c[name].shape, generator=gen, device="cuda")
        out = []
        for s in (1.0, -1.0):
            x = (c[name].float() + s * d).to(c[name].dtype)
            o, ht, _ = kda.kda_linattn_fwd(*(x if n == name else c[n] for n in ("q", "k", "v")), c["slope"], c["cu"],
                                           h0=x if name == "h0" else c["h0"], scale=c["scale"])
            out.append((x.double(), o, ht))
        step = (out[0][0] - out[1][0])
        num = float(((out[0][1].double() - out[1][1].double()) * c["dO"].double()).sum()
                    + ((out[0][2].double() - out[1][2].double()) * c["dht"].double()).sum())
        want = float((g[got].double() * step).sum())
        noise = 2.0 ** -8 * (4 * size * float(c["dO"].float().abs().max()) + float(g[got].float().norm()) * float(step.abs().max()))
        assert abs(num - want) <= noise, (name, num, want, noise)


def test_on_another_stream_and_in_a_graph():
    c = _case([300, 40, 700], 4, 2, True)
    want = _run(c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _run(c)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(got[k], want[k]) for k in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _run(c)
    for t in out.values():
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], want[k]) for k in want)
    # replayed with other offsets of the same number of documents and tokens
    c["cu"].copy_(torch.tensor([0, 10, 900, 1040], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    want = _run(c)
    assert all(torch.equal(out[k], want[k]) for k in want)


def test_other_saved_sets_are_reported():
    c = _case([600, 700], 2, 2, False)
    a = (c["q"], c["k"], c["v"], c["slope"], c["cu"])
    ws = torch.empty(kda.kda_linattn_workspace_size(1300, 2, 2, 2, kda.KDA_OP_BWD_SAVED)[0], dtype=torch.uint8, device="cuda")
    sv = kda.kda_linattn_workspace_size(1300, 2, 2, 2, kda.KDA_OP_FWD)[1]
    for fill in (0, 255):
        kda.kda_linattn_bwd(*a, c["dO"], saved=torch.full((sv,), fill, dtype=torch.uint8, device="cuda"), ws=ws)
        assert kda.kda_read_device_status(ws) == kda.KDA_ERR_DEVICE_CHECK
    _, _, saved = kda.kda_linattn_fwd(*a)
    kda.kda_linattn_bwd(*a, c["dO"], saved=saved, ws=ws)
    assert kda.kda_read_device_status(ws) == kda.KDA_OK


# ---- single tokens ----

def _step_case(N, H, Hk, pool, seed=0):
    gen = torch.Generator("cpu").manual_seed(seed + N)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    qkv = rn(N, (2 * Hk + H) * D).bfloat16().cuda()
    q, k, v = qkv.split([Hk * D, Hk * D, H * D], 1)
    return (q.unflatten(1, (Hk, D)), k.unflatten(1, (Hk, D)), v.unflatten(1, (H, D)), (-torch.rand(H, generator=gen)).cuda(),
            rn(pool, H, D, D).cuda())


def _step_ref(q, k, v, slope, h, rows):
    H = v.shape[1]
    o, ht = linattn.linattn_fwd(_np(q)[rows], _np(k)[rows], _np(v)[rows], _np(slope), list(range(len(rows) + 1)), h, 0.25)
    return o, ht


@pytest.mark.parametrize("N,H,Hk", [(1, 1, 1), (1, 16, 16), (3, 6, 2), (40, 5, 5), (33, 8, 1)])
def test_step(N, H, Hk):
    q, k, v, slope, h = _step_case(N, H, Hk, N)
    before = h.clone()
    o, h1 = kda.kda_linattn_step(q, k, v, slope, h, scale=0.25, h_out=torch.empty_like(h))
    assert torch.equal(h, before)
    ro, rh = _step_ref(q, k, v, slope, _np(h), list(range(N)))
    # fp32 throughout: sums of 128 terms, 2^-24 each of the terms' root sum of squares, and the output's rounding
    assert (np.abs(_np(o) - ro) <= 2.0 ** -8 * np.abs(ro) + 1e-5 * np.abs(ro).max()).all()
    assert np.abs(_np(h1) - rh).max() <= 4 * 2.0 ** -24 * np.abs(rh).max() * 2
    o2, h2 = kda.kda_linattn_step(q, k, v, slope, h, scale=0.25)  # in place
    assert h2 is h and torch.equal(o2, o) and torch.equal(h, h1)


def test_step_slots():
    q, k, v, slope, h = _step_case(5, 3, 3, 9)
    slots = torch.tensor([7, -1, 0, 9, 3], dtype=torch.int32, device="cuda")
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    before = h.clone()
    o, _ = kda.kda_linattn_step(q, k, v, slope, h, scale=0.25, slots=slots, ws=ws)
    assert kda.kda_read_device_status(ws) == kda.KDA_ERR_DEVICE_CHECK  # slot 9 of 9
    ro, rh = _step_ref(q, k, v, slope, _np(before)[[7, 0, 3]], [0, 2, 4])
    assert (np.abs(_np(o)[[0, 2, 4]] - ro) <= 2.0 ** -8 * np.abs(ro) + 1e-5 * np.abs(ro).max()).all()
    assert not o[1].any() and not o[3].any()
    assert np.abs(_np(h)[[7, 0, 3]] - rh).max() <= 8 * 2.0 ** -24 * np.abs(rh).max()
    rest = [1, 2, 4, 5, 6, 8]
    assert torch.equal(h[rest], before[rest])
    slots[3] = 8
    kda.kda_linattn_step(q, k, v, slope, h, slots=slots, ws=ws)
    assert kda.kda_read_device_status(ws) == kda.KDA_OK


def test_steps_continue_a_prompt():
    c = _case([260, 3], 4, 2, False)
    cu = torch.tensor([0, 250, 250], dtype=torch.int32, device="cuda")
    sl = lambda t: torch.cat([t[:250]])  # noqa: E731
    _, h, _ = kda.kda_linattn_fwd(sl(c["q"]), sl(c["k"]), sl(c["v"]), c["slope"], cu, scale=c["scale"], save=False)
    o, ht, _ = kda.kda_linattn_fwd(c["q"], c["k"], c["v"], c["slope"], c["cu"], scale=c["scale"], save=False)
    for t in range(10):
        at = torch.tensor([250 + t, min(260 + t, 262)], device="cuda")
        y, _ = kda.kda_linattn_step(c["q"][at], c["k"][at], c["v"][at], c["slope"], h, scale=c["scale"],
                                    slots=torch.tensor([0, 1 if t < 3 else -1], dtype=torch.int32, device="cuda"))
        # bf16 scores and states on the chunked side: a few 2^-8 of the row
        want = o[at].float()
        for r in range(2 if t < 3 else 1):
            assert float((y[r].float() - want[r]).norm(dim=-1).div(want[r].norm(dim=-1)).max()) <= 4 * ROW
    _state("state", h, _np(ht))


def test_step_on_a_stream_and_in_a_graph():
    q, k, v, slope, h = _step_case(4, 2, 2, 4)
    want, hw = kda.kda_linattn_step(q, k, v, slope, h, h_out=torch.empty_like(h))
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(h)
    with torch.cuda.graph(g):
        o, _ = kda.kda_linattn_step(q, k, v, slope, h, h_out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(out, hw)


@pytest.mark.parametrize("lens,H", [([300, 40], 2), ([2500, 40], 2)])
def test_outputs_that_are_not_wanted(lens, H):
    # no final state, no dh0: the rows are the same but for values split more coarsely on their way into them
    import ctypes
    c = _case(lens, H, H, True, strided=False)
    want = _run(c)
    T, N = sum(lens), len(lens)
    pr = kda.kda_linattn_problem(T, N, H, H, D, kda.KDA_DT_BF16, c["scale"], 0, 0, 0, c["cu"].data_ptr())
    ws = torch.empty(kda.kda_linattn_workspace_size(T, N, H, H, kda.KDA_OP_BWD_REPLAY)[0], dtype=torch.uint8, device="cuda")
    o = torch.empty_like(c["v"])
    st = kda.lib().kda_linattn_fwd(ctypes.byref(pr), *(c[n].data_ptr() for n in ("q", "k", "v", "slope", "h0")), o.data_ptr(), None,
                                   None, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == kda.KDA_OK and kda.kda_read_device_status(ws) == kda.KDA_OK
    g = kda.kda_linattn_bwd(c["q"], c["k"], c["v"], c["slope"], c["cu"], c["dO"], h0=c["h0"], dht=c["dht"], scale=c["scale"], want_dh0=False)
    assert "dh0" not in g
    for name, a, b in [("o", o, want["o"])] + [(k, g[k], want[k]) for k in ("dq", "dk", "dv")]:
        # a split value differs by 2^-18 at most, which moves a rounding here and there
        assert float((a.float() - b.float()).norm() / b.float().norm()) <= 2.0 ** -9, name


def test_one_token_documents_are_single_steps():
    # a document of one token with a state in front of it is kda_linattn_step's call
    N, H = 9, 3
    c = _case([1] * N, H, H, True, strided=False)
    o, ht, _ = kda.kda_linattn_fwd(c["q"], c["k"], c["v"], c["slope"], c["cu"], h0=c["h0"], scale=c["scale"])
    y, h = kda.kda_linattn_step(c["q"], c["k"], c["v"], c["slope"], c["h0"], scale=c["scale"], h_out=torch.empty_like(c["h0"]))
    _state("ht", ht, _np(h))
    assert float((o.float() - y.float()).norm() / y.float().norm()) <= 2 * ROW
