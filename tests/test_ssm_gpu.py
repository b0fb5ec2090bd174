"""GPU parity of the selective state-space scan (kda_ssm_fwd / kda_ssm_bwd / kda_ssm_step) and of the
conv's serving forms against the FP64 oracles (oracle/ssm.py, oracle/conv1d.py) on the same inputs.

Bounds.  Everything is accumulated in fp32; a decay exp2(x) carries a relative error of 2^-22 and a
state remembers at most the document's tokens, so a state, and every sum built on states, is off
by at most (tokens remembered) 2^-22 of its size in the worst case: 300 tokens give 7e-5, and fp32
outputs are held to 1e-4 of their rms.  Outputs in bf16 / fp16 add the rounding of their own value,
eps / 2.  A state of one step is one multiply-add and one exp2: 4e-6.
"""
import numpy as np
import pytest
import torch

from linear_attention_chunked_gb300 import kda
from oracle import conv1d, ssm

pytestmark = pytest.mark.gpu

TOL = 1e-4
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _close(name, got, ref, tol=TOL):
    """|got - ref| <= tol rms(ref) + (eps / 2 of got's type, when it is below fp32) |ref|."""
    assert tuple(got.shape) == tuple(ref.shape), (name, got.shape, ref.shape)
    if ref.size == 0:
        return
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    g = _np(got)
    bound = tol * max(np.sqrt(np.mean(ref * ref)), 1e-30) * (1 + half) + half * np.abs(ref)
    if got.dtype == torch.float16:
        bound = bound + 2.0 ** -25  # half a step of fp16's subnormals
    bad = np.abs(g - ref) > bound
    assert np.isfinite(g).all() and not bad.any(), (name, float(np.max(np.abs(g - ref) / bound)), int(bad.sum()))


def _inputs(lens, C, S, G, dtype, seed, *, z=True, h0=False, D=True, bias=True, strided=False, dev="cuda"):
    gen = torch.Generator("cpu").manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    T, N, dt = sum(lens), len(lens), DT[dtype]
    wide = rn(T, 2 * C + 2 * G * S + 5).to(dt).to(dev)  # one projection; its columns are views
    cut = (lambda a, b: wide[:, a:b]) if strided else (lambda a, b: wide[:, a:b].contiguous())
    B = cut(2 * C + 1, 2 * C + 1 + G * S).unflatten(1, (G, S))
    Cm = cut(2 * C + 3 + G * S, 2 * C + 3 + 2 * G * S).unflatten(1, (G, S))
    a = dict(u=cut(0, C), dt=rn(T, C).to(dt).to(dev), A=(-torch.exp(0.5 * rn(C, S)) * torch.arange(1, S + 1)).to(dev),
             B=B, C=Cm, cu_seqlens=torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=dev))
    kw = dict(D=rn(C).to(dev) if D else None, dt_bias=(rn(C) - 3).to(dev) if bias else None,
              z=cut(C, 2 * C) if z else None, h0=rn(N, C, S).to(dev) if h0 else None)
    dy, dht = rn(T, C).to(dt).to(dev), rn(N, C, S).to(dev) if h0 else None
    return a, kw, dy, dht


def _ref_args(a, kw):
    return (dict(u=_np(a["u"]), dt=_np(a["dt"]), A=_np(a["A"]), B=_np(a["B"]), Cm=_np(a["C"]), cu_seqlens=a["cu_seqlens"].cpu().numpy()),
            {k: _np(v) for k, v in kw.items()})


CASES = {
    # one token, a chunk's edge, one past it, an empty document, several chunks
    "edges": dict(lens=[1, 64, 65, 0, 63, 200], C=40, S=16, G=1, dtype="bf16"),
    "h0_fp32": dict(lens=[3, 0, 129, 1], C=37, S=16, G=1, dtype="fp32", h0=True),
    "strided_groups": dict(lens=[70, 10], C=66, S=12, G=3, dtype="bf16", strided=True, h0=True),
    "states_1": dict(lens=[90], C=130, S=1, G=2, dtype="fp32", h0=True),
    "states_4": dict(lens=[66, 5], C=33, S=4, G=1, dtype="fp16"),
    "states_7": dict(lens=[130], C=50, S=7, G=1, dtype="fp32", h0=True),
    "states_8": dict(lens=[130], C=150, S=8, G=1, dtype="bf16"),
    "states_24": dict(lens=[20, 70], C=20, S=24, G=2, dtype="fp32", h0=True),
    "states_32": dict(lens=[67], C=35, S=32, G=1, dtype="bf16"),
    "states_64": dict(lens=[65, 2], C=18, S=64, G=2, dtype="fp32", h0=True),
    "plain": dict(lens=[100], C=24, S=16, G=1, dtype="fp32", z=False, D=False, bias=False),
    # more channels than a backward block's four tiles, in one and in two groups
    "many_channels": dict(lens=[80, 33], C=600, S=16, G=1, dtype="bf16", h0=True),
    "many_channels_2": dict(lens=[150], C=1040, S=8, G=2, dtype="fp32"),
}


@pytest.mark.parametrize("case", list(CASES))
def test_scan_forward_and_backward(case):
    a, kw, dy, dht = _inputs(**CASES[case], seed=len(case))
    ra, rk = _ref_args(a, kw)
    y_ref, ht_ref = ssm.ssm_fwd(**ra, **rk)
    y, ht, saved = kda.kda_ssm_fwd(**a, **kw)
    _close("y", y, y_ref)
    _close("ht", ht, ht_ref)
    y2, ht2, none = kda.kda_ssm_fwd(**a, **kw, save=False)
    assert none is None and torch.equal(y2, y) and torch.equal(ht2, ht)
    ref = ssm.ssm_bwd(**ra, dy=_np(dy), dht=_np(dht), **rk)
    got = kda.kda_ssm_bwd(**a, dy=dy, dht=dht, saved=saved, **kw)
    want = {"du", "ddt", "dA", "dB", "dC", "dh0"} | {n for n, k in (("dz", "z"), ("dD", "D"), ("ddt_bias", "dt_bias")) if kw[k] is not None}
    assert set(got) == want
    for k in got:
        _close(k, got[k], ref[k])
    replay = kda.kda_ssm_bwd(**a, dy=dy, dht=dht, **kw)
    for k in got:  # the recomputed states are the saved ones
        assert torch.equal(replay[k], got[k]), k


def test_scan_without_softplus():
    a, kw, dy, dht = _inputs([70, 9], 36, 16, 1, "fp32", 3, h0=True)
    a["dt"] = a["dt"].abs() * 0.1
    kw["dt_bias"] = kw["dt_bias"].abs() * 0.01
    ra, rk = _ref_args(a, kw)
    y_ref, ht_ref = ssm.ssm_fwd(**ra, **rk, softplus=False)
    y, ht, saved = kda.kda_ssm_fwd(**a, **kw, softplus=False)
    _close("y", y, y_ref)
    _close("ht", ht, ht_ref)
    ref = ssm.ssm_bwd(**ra, dy=_np(dy), dht=_np(dht), **rk, softplus=False)
    for k, v in kda.kda_ssm_bwd(**a, dy=dy, dht=dht, saved=saved, softplus=False, **kw).items():
        _close(k, v, ref[k])


def test_gradients_against_differences():
    # the kernels' own outputs differenced: L = sum(y dy) + sum(ht dht) is formed in fp64 from fp32
    # outputs, so a difference over 2e carries about 2^-22 rms(y) sqrt(T C) |dy| / (2 e) of rounding
    a, kw, dy, dht = _inputs([40, 70], 24, 8, 1, "fp32", 5, h0=True)
    got = kda.kda_ssm_bwd(**a, dy=dy, dht=dht, **kw)
    gen = torch.Generator("cpu").manual_seed(6)
    for name, g in dict(u="du", dt="ddt", A="dA", B="dB", C="dC", D="dD", dt_bias="ddt_bias", z="dz", h0="dh0").items():
        x = a[name] if name in a else kw[name]
        d = torch.randn(x.shape, generator=gen).cuda()
        e = 1e-2 if name in ("u", "B", "C", "D", "h0") else 1e-3  # the outputs are linear in the first
        outs = []
        for s in (e, -e):
            aa, kk = dict(a), dict(kw)
            (aa if name in aa else kk)[name] = x + s * d
            y, ht, _ = kda.kda_ssm_fwd(**aa, **kk, save=False)
            outs.append((y.double(), ht.double()))
        num = float((((outs[0][0] - outs[1][0]) * dy.double()).sum() + ((outs[0][1] - outs[1][1]) * dht.double()).sum()) / (2 * e))
        ana = float((got[g].double() * d.double()).sum())
        size = float(outs[0][0].norm() + outs[0][1].norm())
        assert abs(num - ana) <= 2.0 ** -20 * size / (2 * e) + 1e-3 * abs(ana) + 1e-3 * size * e, (name, num, ana)


def test_results_repeat_and_documents_are_isolated():
    lens = [70, 300, 5, 64]
    a, kw, dy, dht = _inputs(lens, 48, 16, 1, "bf16", 7, h0=True)
    run = lambda a, kw, dy, dht: (kda.kda_ssm_fwd(**a, **kw)[:2], kda.kda_ssm_bwd(**a, dy=dy, dht=dht, **kw))  # noqa: E731
    (y, ht), g = run(a, kw, dy, dht)
    (y2, ht2), g2 = run(a, kw, dy, dht)
    assert torch.equal(y, y2) and torch.equal(ht, ht2) and all(torch.equal(g[k], g2[k]) for k in g)
    cu = a["cu_seqlens"].tolist()
    for n in range(len(lens)):
        s, e = cu[n], cu[n + 1]
        part = {k: a[k][s:e].contiguous() for k in ("u", "dt", "B", "C")}
        pk = dict(kw, z=kw["z"][s:e].contiguous(), h0=kw["h0"][n:n + 1].contiguous())
        pa = dict(part, A=a["A"], cu_seqlens=torch.tensor([0, e - s], dtype=torch.int32, device="cuda"))
        (y1, h1), g1 = run(pa, pk, dy[s:e].contiguous(), dht[n:n + 1].contiguous())
        assert torch.equal(y1, y[s:e]) and torch.equal(h1[0], ht[n])
        for k in ("du", "ddt", "dB", "dC", "dz"):
            assert torch.equal(g1[k], g[k][s:e]), k
        assert torch.equal(g1["dh0"][0], g["dh0"][n])


def test_a_non_finite_document_leaves_the_others_alone():
    a, kw, dy, dht = _inputs([70, 80, 66], 40, 12, 1, "fp32", 8)
    (y, ht, _), g = kda.kda_ssm_fwd(**a, **kw), kda.kda_ssm_bwd(**a, dy=dy, **kw)
    bad = dict(a, u=a["u"].clone())
    bad["u"][75] = float("inf")
    bad["u"][80, 3] = float("nan")
    (y2, ht2, _), g2 = kda.kda_ssm_fwd(**bad, **kw), kda.kda_ssm_bwd(**bad, dy=dy, **kw)
    for s, e in ((0, 70), (150, 216)):
        assert torch.equal(y2[s:e], y[s:e])
        for k in ("du", "ddt", "dB", "dC", "dz"):
            assert torch.equal(g2[k][s:e], g[k][s:e]), k
    assert torch.equal(ht2[0], ht[0]) and torch.equal(ht2[2], ht[2])
    # causal inside the document, and an infinite input stays infinite where no state cancels it
    assert torch.equal(y2[70:75], y[70:75])


def test_extreme_steps():
    # delta from softplus(-80) = 1.8e-35 to 80: decays of 1 and 0, and no step at all
    a, kw, dy, dht = _inputs([65], 16, 16, 1, "fp32", 9, h0=True, bias=False)
    a["dt"] = torch.linspace(-80, 80, 65 * 16, device="cuda").reshape(65, 16).contiguous()
    ra, rk = _ref_args(a, kw)
    y_ref, ht_ref = ssm.ssm_fwd(**ra, **rk)
    y, ht, saved = kda.kda_ssm_fwd(**a, **kw)
    _close("y", y, y_ref)
    _close("ht", ht, ht_ref)
    ref = ssm.ssm_bwd(**ra, dy=_np(dy), dht=_np(dht), **rk)
    for k, v in kda.kda_ssm_bwd(**a, dy=dy, dht=dht, saved=saved, **kw).items():
        _close(k, v, ref[k])


def test_no_tokens():
    a, kw, dy, dht = _inputs([0, 0], 24, 16, 1, "bf16", 10, h0=True)
    y, ht, saved = kda.kda_ssm_fwd(**a, **kw)
    assert y.shape == (0, 24) and torch.equal(ht, kw["h0"])
    g = kda.kda_ssm_bwd(**a, dy=dy, dht=dht, saved=saved, **kw)
    assert torch.equal(g["dh0"], dht)
    for k in ("dA", "dD", "ddt_bias"):
        assert not g[k].any(), k


def test_malformed_offsets_set_the_status_and_write_nothing():
    a, kw, dy, _ = _inputs([40, 30], 24, 16, 1, "bf16", 11)
    for cu in ([0, 80, 70], [1, 40, 70], [0, 40, 69]):
        a["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        ws = torch.empty(kda.kda_ssm_workspace_size(70, 2, 24, 16, 1, kda.KDA_OP_FWD)[0], dtype=torch.uint8, device="cuda")
        y = torch.full((70, 24), 7.0, dtype=torch.bfloat16, device="cuda")
        ht = torch.full((2, 24, 16), 7.0, device="cuda")
        kda.kda_ssm_fwd(**a, **kw, save=False, ws=ws, y=y, ht=ht)
        assert kda.kda_read_device_status(ws) == kda.KDA_ERR_DEVICE_CHECK
        assert bool((y == 7).all()) and bool((ht == 7).all())


def test_on_another_stream():
    a, kw, dy, _ = _inputs([200], 64, 16, 1, "bf16", 12)
    want = kda.kda_ssm_fwd(**a, **kw)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = kda.kda_ssm_fwd(**a, **kw)[0]
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want)


def test_captured_in_a_graph():
    a, kw, dy, _ = _inputs([130, 20], 64, 16, 1, "bf16", 13)
    want = kda.kda_ssm_bwd(**a, dy=dy, **kw)  # also the device's set-up
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, ht, saved = kda.kda_ssm_fwd(**a, **kw)
        got = kda.kda_ssm_bwd(**a, dy=dy, saved=saved, **kw)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)


# ---- single tokens ----

STEP_CASES = {
    "one": dict(N=1, C=64, S=16, G=1, dtype="bf16"),
    "odd": dict(N=3, C=37, S=16, G=1, dtype="fp32", strided=True),
    "groups": dict(N=5, C=30, S=12, G=3, dtype="fp16", strided=True),
    "states_1": dict(N=4, C=300, S=1, G=1, dtype="fp32"),
    "states_4": dict(N=4, C=129, S=4, G=1, dtype="bf16"),
    "states_8": dict(N=2, C=40, S=8, G=2, dtype="bf16"),
    "states_32": dict(N=2, C=40, S=32, G=2, dtype="fp16"),
    "states_64": dict(N=7, C=21, S=64, G=1, dtype="fp32", z=False, D=False, bias=False),
}


@pytest.mark.parametrize("case", list(STEP_CASES))
def test_step(case):
    c = dict(STEP_CASES[case])
    N = c.pop("N")
    a, kw, _, _ = _inputs([1] * N, seed=N, h0=True, **c)
    ra, rk = _ref_args(a, kw)
    y_ref, ht_ref = ssm.ssm_fwd(**ra, **rk)
    h = kw.pop("h0")
    cu = a.pop("cu_seqlens")
    y, h_out = kda.kda_ssm_step(**a, h=h, **kw, h_out=torch.empty_like(h))
    _close("y", y, y_ref, 4e-6 * 8)  # S products more
    _close("h", h_out, ht_ref, 4e-6)
    # in place, through slots of a larger pool, an unused row between
    order = torch.randperm(N, generator=torch.Generator().manual_seed(1))
    pool = torch.full((N + 3, *h.shape[1:]), 5.0, device="cuda")
    pool[order.cuda() + 2] = h
    slots = (order + 2).to(torch.int32)
    slots[0] = -1
    y2, pool2 = kda.kda_ssm_step(**a, h=pool, **kw, slots=slots.cuda())
    assert pool2 is pool and not y2[0].any() and torch.equal(y2[1:], y[1:])
    assert torch.equal(pool[(order + 2)[1:].cuda()], h_out[1:])
    assert bool((pool[:2] == 5).all()) and bool((pool[N + 2:] == 5).all()) and torch.equal(pool[order[0] + 2], h[0])


def test_step_continues_a_prompt():
    lens = [70, 3]
    a, kw, _, _ = _inputs([n + 1 for n in lens], 64, 16, 1, "fp32", 14)
    y, ht, _ = kda.kda_ssm_fwd(**a, **kw)
    keep = torch.tensor([i for i in range(75) if i not in (70, 74)], device="cuda")
    last = torch.tensor([70, 74], device="cuda")
    part = lambda rows: ({k: a[k][rows].contiguous() for k in ("u", "dt", "B", "C")}, dict(kw, z=kw["z"][rows].contiguous()))  # noqa: E731
    pa, pk = part(keep)
    _, h, _ = kda.kda_ssm_fwd(**pa, A=a["A"], cu_seqlens=torch.tensor([0, 70, 73], dtype=torch.int32, device="cuda"), **pk)
    sa, sk = part(last)
    sk.pop("h0")
    y1, h1 = kda.kda_ssm_step(**sa, A=a["A"], h=h, **sk)
    _close("y", y1, _np(y[last]))
    _close("h", h1, _np(ht))


def test_step_reports_a_slot_out_of_range():
    a, kw, _, _ = _inputs([1, 1], 40, 16, 1, "bf16", 15, h0=True)
    h = kw.pop("h0")
    a.pop("cu_seqlens")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    before = h.clone()
    slots = torch.tensor([2, 1], dtype=torch.int32, device="cuda")
    y, _ = kda.kda_ssm_step(**a, h=h, **kw, slots=slots, ws=ws)
    assert kda.kda_read_device_status(ws) == kda.KDA_ERR_DEVICE_CHECK
    assert not y[0].any() and torch.equal(h[0], before[0]) and not torch.equal(h[1], before[1])


# ---- the conv's serving forms ----

@pytest.mark.parametrize("C", [8, 136, 2048])
@pytest.mark.parametrize("halo", [False, True])
def test_conv_tail_and_step_continue_a_prompt(C, halo):
    lens = [5, 0, 1, 2, 3, 70]
    N, gen = len(lens), torch.Generator("cpu").manual_seed(C)
    x = torch.randn((sum(lens), C), generator=gen).bfloat16().cuda()
    nxt = torch.randn((N, C), generator=gen).bfloat16().cuda()
    w, b = (torch.randn((C, 4), generator=gen) * 0.5).cuda(), (torch.randn(C, generator=gen) * 0.1).cuda()
    h = torch.randn((N, 3, C), generator=gen).bfloat16().cuda() if halo else None
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    tail = kda.kda_conv_tail(x, cu, halo=h)
    s = cu.tolist()
    for n in range(N):
        front = h[n] if halo else torch.zeros((3, C), dtype=torch.bfloat16, device="cuda")
        assert torch.equal(tail[n], torch.cat([front, x[s[n]:s[n + 1]]])[-3:])
    # the step's window is a halo: it is the conv of one-token documents, bit for bit in fp32 and bf16
    ones = torch.arange(N + 1, dtype=torch.int32, device="cuda")
    for act in (True, False):
        y_ref, _ = conv1d.conv_fwd(_np(nxt), _np(w), ones.cpu().numpy(), bias=_np(b), halo=_np(tail), activation=act)
        for dt in (torch.float32, torch.bfloat16):
            y, out = kda.kda_conv_step(nxt, w, tail, bias=b, activation=act, out_dtype=dt, win_out=torch.empty_like(tail))
            _close("y", y, y_ref, 1e-5)
            assert torch.equal(out, torch.cat([tail[:, 1:], nxt[:, None]], 1))
    pool = torch.full((N + 2, 3, C), 3.0, dtype=torch.bfloat16, device="cuda")
    pool[1:N + 1] = tail.flip(0)
    slots = torch.arange(N, 0, -1, dtype=torch.int32, device="cuda")
    slots[2] = -1
    slots[4] = N + 2
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    y2, _ = kda.kda_conv_step(nxt, w, pool, bias=b, activation=False, out_dtype=torch.bfloat16, slots=slots, ws=ws)
    assert kda.kda_read_device_status(ws) == kda.KDA_ERR_DEVICE_CHECK
    for n in range(N):
        if n in (2, 4):
            assert not y2[n].any() and torch.equal(pool[N - n], tail[n])
        else:
            assert torch.equal(y2[n], y[n]) and torch.equal(pool[N - n], out[n])
    assert bool((pool[0] == 3).all()) and bool((pool[N + 1] == 3).all())


def test_conv_step_large_batch_takes_the_same_rows():
    # 4 sequences per thread instead of one
    C, N = 4096, 700
    gen = torch.Generator("cuda").manual_seed(0)
    x = torch.randn((N, C), generator=gen, device="cuda").bfloat16()
    win = torch.randn((N, 3, C), generator=gen, device="cuda").bfloat16()
    w = torch.randn((C, 4), generator=gen, device="cuda")
    y, out = kda.kda_conv_step(x, w, win, win_out=torch.empty_like(win))
    for n in (0, 1, 2, 3, 4, 698, 699):
        y1, o1 = kda.kda_conv_step(x[n:n + 1], w, win[n:n + 1], win_out=torch.empty_like(win[:1]))
        assert torch.equal(y1[0], y[n]) and torch.equal(o1[0], out[n])


# ---- forms of the kernels, and long offsets ----

@pytest.mark.parametrize("S,G,dtype", [(1, 1, "fp32"), (4, 2, "bf16"), (7, 1, "fp16"), (16, 1, "bf16"), (24, 3, "fp32"), (64, 1, "bf16")])
def test_short_prompt_in_one_launch(S, G, dtype):
    # a pack of at most 64 tokens without a saved set: no plan, no carry; the same bits as with one
    for h0 in (False, True):
        a, kw, _, _ = _inputs([5, 0, 1, 37, 0], 12 * G + 3 * G, S, G, dtype, S, h0=h0, strided=True)
        ra, rk = _ref_args(a, kw)
        y_ref, ht_ref = ssm.ssm_fwd(**ra, **rk)
        before = kda.kda_launch_counter()
        y, ht, _ = kda.kda_ssm_fwd(**a, **kw, save=False)
        assert kda.kda_launch_counter() == before + 1
        _close("y", y, y_ref)
        _close("ht", ht, ht_ref)
        y2, ht2, _ = kda.kda_ssm_fwd(**a, **kw)
        assert torch.equal(y, y2) and torch.equal(ht, ht2)


def test_short_prompt_with_malformed_offsets():
    a, kw, _, _ = _inputs([30, 10], 24, 16, 1, "bf16", 11)
    for cu in ([0, 50, 40], [1, 30, 40], [0, 30, 39], [0, -1, 40]):
        a["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        ws = torch.empty(kda.kda_ssm_workspace_size(40, 2, 24, 16, 1, kda.KDA_OP_FWD)[0], dtype=torch.uint8, device="cuda")
        y = torch.full((40, 24), 7.0, dtype=torch.bfloat16, device="cuda")
        ht = torch.full((2, 24, 16), 7.0, device="cuda")
        kda.kda_ssm_fwd(**a, **kw, save=False, ws=ws, y=y, ht=ht)
        assert kda.kda_read_device_status(ws) == kda.KDA_ERR_DEVICE_CHECK
        assert bool((y == 7).all()) and bool((ht == 7).all())


def test_backward_reports_malformed_offsets():
    a, kw, dy, _ = _inputs([40, 30], 24, 16, 1, "bf16", 12)
    a["cu_seqlens"] = torch.tensor([0, 80, 70], dtype=torch.int32, device="cuda")
    _, _, saved = kda.kda_ssm_fwd(**a, **kw)
    for s, op in ((saved, kda.KDA_OP_BWD_SAVED), (None, kda.KDA_OP_BWD_REPLAY)):
        ws = torch.empty(kda.kda_ssm_workspace_size(70, 2, 24, 16, 1, op)[0], dtype=torch.uint8, device="cuda")
        kda.kda_ssm_bwd(**a, dy=dy, saved=s, ws=ws, **kw)
        assert kda.kda_read_device_status(ws) == kda.KDA_ERR_DEVICE_CHECK


def test_a_document_alone_equals_it_in_a_large_pack():
    # the pack takes the throughput forms (and four channel tiles a block in the backward), the document
    # alone the latency forms: the same bits
    lens = [2500, 100, 1900]
    a, kw, dy, dht = _inputs(lens, 4096, 16, 1, "bf16", 16, h0=True)
    y, ht, saved = kda.kda_ssm_fwd(**a, **kw)
    g = kda.kda_ssm_bwd(**a, dy=dy, dht=dht, saved=saved, **kw)
    s, e = 2500, 2600
    pa = dict({k: a[k][s:e].contiguous() for k in ("u", "dt", "B", "C")}, A=a["A"], cu_seqlens=torch.tensor([0, 100], dtype=torch.int32, device="cuda"))
    pk = dict(kw, z=kw["z"][s:e].contiguous(), h0=kw["h0"][1:2].contiguous())
    y1, h1, saved1 = kda.kda_ssm_fwd(**pa, **pk)
    g1 = kda.kda_ssm_bwd(**pa, dy=dy[s:e].contiguous(), dht=dht[1:2].contiguous(), saved=saved1, **pk)
    assert torch.equal(y1, y[s:e]) and torch.equal(h1[0], ht[1])
    for k in ("du", "ddt", "dB", "dC", "dz"):
        assert torch.equal(g1[k], g[k][s:e]), k
    assert torch.equal(g1["dh0"][0], g["dh0"][1])


def test_rows_beyond_32_bit_offsets():
    # 300 rows of one projection 2^23 columns wide: the last rows start past 2^31 elements
    T, C, S = 300, 24, 16
    a, kw, dy, _ = _inputs([T], C, S, 1, "bf16", 17)
    want_y, want_h, _ = kda.kda_ssm_fwd(**a, **kw)
    want = kda.kda_ssm_bwd(**a, dy=dy, **kw)
    wide = torch.empty((T, 1 << 23), dtype=torch.bfloat16, device="cuda")
    at = 0
    far = {}
    for name, t in (("u", a["u"]), ("dt", a["dt"]), ("z", kw["z"]), ("B", a["B"]), ("C", a["C"])):
        n = t[0].numel()
        wide[:, at:at + n] = t.reshape(T, n)
        far[name] = wide[:, at:at + n].unflatten(1, t.shape[1:]) if t.dim() > 2 else wide[:, at:at + n]
        at += n
    fa, fk = dict(a, **{k: far[k] for k in ("u", "dt", "B", "C")}), dict(kw, z=far["z"])
    y, h, _ = kda.kda_ssm_fwd(**fa, **fk)
    assert torch.equal(y, want_y) and torch.equal(h, want_h)
    g = kda.kda_ssm_bwd(**fa, dy=dy, **fk)
    assert all(torch.equal(g[k], want[k]) for k in want)


def test_slots_beyond_32_bit_offsets():
    C, S, n = 4096, 16, (1 << 31) // (4096 * 16) + 10  # the last states start past 2^31 elements
    a, kw, _, _ = _inputs([1, 1], C, S, 1, "bf16", 18, h0=True)
    h = kw.pop("h0")
    a.pop("cu_seqlens")
    y, h1 = kda.kda_ssm_step(**a, h=h, **kw, h_out=torch.empty_like(h))
    pool = torch.empty((n, C, S), device="cuda")
    slots = torch.tensor([n - 1, 3], dtype=torch.int32, device="cuda")
    pool[n - 1], pool[3] = h[0], h[1]
    y2, _ = kda.kda_ssm_step(**a, h=pool, **kw, slots=slots)
    assert torch.equal(y2, y) and torch.equal(pool[n - 1], h1[0]) and torch.equal(pool[3], h1[1])
    del pool
    m = (1 << 31) // (3 * 8192) + 10
    x = torch.randn((2, 8192), device="cuda").bfloat16()
    win, w = torch.randn((2, 3, 8192), device="cuda").bfloat16(), torch.randn((8192, 4), device="cuda")
    yc, wc = kda.kda_conv_step(x, w, win, win_out=torch.empty_like(win))
    pool = torch.empty((m, 3, 8192), dtype=torch.bfloat16, device="cuda")
    pool[m - 1], pool[3] = win[0], win[1]
    yc2, _ = kda.kda_conv_step(x, w, pool, slots=torch.tensor([m - 1, 3], dtype=torch.int32, device="cuda"))
    assert torch.equal(yc2, yc) and torch.equal(pool[m - 1], wc[0]) and torch.equal(pool[3], wc[1])


@pytest.mark.parametrize("S,C,dtype,G", [(1, 16384, "fp32", 1), (4, 16384, "bf16", 2), (7, 16384, "fp16", 1), (8, 16400, "fp32", 1),
                                         (12, 16384, "bf16", 4), (16, 16300, "fp32", 1), (16, 16384, "fp16", 1), (24, 8192, "fp32", 1),
                                         (32, 8192, "bf16", 2), (48, 4096, "fp32", 1), (64, 4096, "bf16", 1)])
def test_throughput_forms(S, C, dtype, G):
    # wide enough for the throughput forms of every kernel; the oracle takes the first and last channels of
    # each group, which alone have gradients (channels meet only in dB and dC)
    lens = [700, 0, 300]
    a, kw, dy, _ = _inputs(lens, C, S, G, dtype, S + G)
    Cg = C // G
    ch = np.concatenate([np.r_[g * Cg:g * Cg + 5, (g + 1) * Cg - 3:(g + 1) * Cg] for g in range(G)])
    mask = torch.zeros(C, dtype=dy.dtype, device="cuda")
    mask[torch.from_numpy(ch).cuda()] = 1
    dy = dy * mask
    pick = lambda t: None if t is None else _np(t)[..., ch]  # noqa: E731
    ra = dict(u=pick(a["u"]), dt=pick(a["dt"]), A=_np(a["A"])[ch], B=_np(a["B"]), Cm=_np(a["C"]), cu_seqlens=a["cu_seqlens"].cpu().numpy())
    rk = dict(D=pick(kw["D"]), dt_bias=pick(kw["dt_bias"]), z=pick(kw["z"]))
    y_ref, ht_ref = ssm.ssm_fwd(**ra, **rk)
    y, ht, saved = kda.kda_ssm_fwd(**a, **kw)
    idx = torch.from_numpy(ch).cuda()
    _close("y", y[:, idx], y_ref)
    _close("ht", ht[:, idx], ht_ref)
    ref = ssm.ssm_bwd(**ra, dy=_np(dy)[:, ch], **rk)
    got = kda.kda_ssm_bwd(**a, dy=dy, saved=saved, **kw)
    for k in ("du", "ddt", "dz", "dD", "ddt_bias"):
        _close(k, got[k][..., idx], ref[k])
    _close("dA", got["dA"][idx], ref["dA"])
    _close("dh0", got["dh0"][:, idx], ref["dh0"])
    _close("dB", got["dB"], ref["dB"])
    _close("dC", got["dC"], ref["dC"])
