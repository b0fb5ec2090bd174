"""The linear attention over documents that are cut into segments, and over many heads and documents, against the
same definition in 64 bits on the GPU (pairs of tokens within 64, states between); bounds as in test_linattn_gpu.py."""
import numpy as np
import pytest
import torch

from linear_attention_chunked_gb300 import kda
from test_linattn_gpu import D, ROW, STATE, _case, _run

pytestmark = pytest.mark.gpu


def _reference(c):
    """o, ht, dq, dk, dv, dh0 in fp64 and, for the rows' bounds, the root of the sum of their terms' squares."""
    f = torch.float64
    H, Hk = c["v"].shape[1], c["q"].shape[1]
    up = lambda x: x.to(f).repeat_interleave(H // x.shape[1], 1).transpose(0, 1)  # noqa: E731
    q, k, v, do = (up(c[n]) for n in ("q", "k", "v", "dO"))
    slope, scale, cu = c["slope"].to(f)[:, None], c["scale"], c["cu"].tolist()
    N, C = len(cu) - 1, 64

    def walk(query, key, value, s0, back, inside, by, power):
        """One walk (see kda_linattn): out and final state; power 2 takes every term's square."""
        out = torch.zeros_like(value)
        ends = torch.zeros((N, H, D, D), dtype=f, device="cuda")
        sl = slope * power
        for n in range(N):
            X = s0[n].to(f).clone() if s0 is not None else torch.zeros((H, D, D), dtype=f, device="cuda")
            if power == 2:
                X = X ** 2
            starts = list(range(cu[n], cu[n + 1], C))
            for a in reversed(starts) if back else starts:
                b = min(a + C, cu[n + 1])
                i = torch.arange(b - a, device="cuda", dtype=f)
                gap = (i[:, None] - i) * (-1 if back else 1)
                M = torch.where(gap >= 0, torch.exp(sl[:, :, None] * gap.clamp(min=0)), 0.0)
                e = (b - a - 1 - i) if back else i + 1  # decay of the state at a query
                P = (query[:, a:b] @ key[:, a:b].transpose(1, 2)) * M * inside
                out[:, a:b] = by * (P @ value[:, a:b] + torch.exp(sl * e)[:, :, None] * (query[:, a:b] @ X))
                w = torch.exp(sl * ((i + 1) if back else (b - a - 1 - i)))[:, :, None] * inside
                X = torch.exp(sl * (b - a))[:, :, None] * X + (key[:, a:b] * w).transpose(1, 2) @ value[:, a:b]
            ends[n] = X
        return out, ends

    t = lambda s: None if s is None else s.transpose(-1, -2)  # noqa: E731
    sq = lambda *x: [y ** 2 for y in x]  # noqa: E731
    o, ht = walk(q, k, v, c["h0"], False, 1.0, scale, 1)
    dq, _ = walk(do, v, k, t(c["h0"]), False, 1.0, scale, 1)
    dv, dh0 = walk(k, q, do, c["dht"], True, scale, 1.0, 1)
    dk, _ = walk(v, do, q, t(c["dht"]), True, scale, 1.0, 1)
    size = dict(o=walk(*sq(q, k, v), c["h0"], False, 1.0, scale ** 2, 2)[0], dq=walk(*sq(do, v, k), t(c["h0"]), False, 1.0, scale ** 2, 2)[0],
                dv=walk(*sq(k, q, do), c["dht"], True, scale ** 2, 1.0, 2)[0], dk=walk(*sq(v, do, q), t(c["dht"]), True, scale ** 2, 1.0, 2)[0])
    group = lambda x: x.unflatten(0, (Hk, H // Hk)).sum(1)  # noqa: E731
    ref = dict(o=o, dv=dv, dq=group(dq), dk=group(dk))
    size.update(dq=group(size["dq"]), dk=group(size["dk"]))
    back = lambda x: x.transpose(0, 1)  # noqa: E731
    return ({n: back(x) for n, x in ref.items()}, {n: back(x).sum(-1).sqrt() for n, x in size.items()}, dict(ht=ht, dh0=dh0))


def _check(c, got):
    rows, size, states = _reference(c)
    for n, ref in rows.items():
        err = (got[n].double() - ref).norm(dim=-1)
        tol = ROW * (ref.norm(dim=-1) + size[n]) + 1e-6
        assert bool((err <= tol).all()), (n, float((err / tol).max()))
    for n, ref in states.items():
        rel = float((got[n].double() - ref).norm() / ref.norm().clamp(min=1e-30))
        assert rel <= STATE, (n, rel)


# heads at both sides of every way of cutting (512, 1024, 2048 tokens a segment, the backward whole, both whole), documents at both
# sides of the length that is cut and of a segment's end
@pytest.mark.parametrize("lens,H,Hk", [
    ([2048, 2049, 1, 0, 4097], 2, 1), ([5000, 2047, 3000], 4, 4), ([2561, 2560, 2559], 3, 3), ([6145, 10], 8, 2), ([4096, 5555], 16, 16),
    ([9001], 23, 23), ([4200, 300], 24, 8), ([5000, 77], 40, 40), ([2300, 129], 64, 64), ([12345], 1, 1)])
def test_long_documents(lens, H, Hk):
    c = _case(lens, H, Hk, True, seed=H, slopes=(-torch.exp2(-10.0 * torch.rand(H, generator=torch.Generator().manual_seed(H)))).tolist())
    got = _run(c)
    _check(c, got)
    replay = _run(c, save=False)
    assert all(torch.equal(got[k], replay[k]) for k in got)


def test_no_initial_state_and_shared_heads():
    c = _case([3000, 2100], 6, 2, False)
    _check(c, dict(_run(c)))


@pytest.mark.parametrize("H", [2, 24, 64])
def test_a_long_document_alone_and_in_a_pack(H):
    lens = [700, 5000, 3, 2500]
    c = _case(lens, H, H, True)
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


def test_many_documents():
    # more documents than a warp has lanes (their order is the pack's), empty ones among them
    lens = [int(x) for x in np.random.default_rng(0).integers(0, 260, 70)]
    c = _case(lens, 4, 4, True)
    _check(c, _run(c))
    c = _case(lens[:33], 2, 2, True)
    c2 = dict(c, q=c["q"], cu=c["cu"])
    a, b = _run(c), _run(c2)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_long_weak_decays_keep_the_states_exact():
    # no decay at all, and decays whose tokens still weigh in the last state after thousands: held in 32 bits.  STATE is a
    # chunk's: its 24 additions round the running sum by 2^-23 of itself at most.  Where the tokens of m chunks weigh
    # (1 / |slope| tokens, at most all), the sum is rounded by m chunks' additions before the first of them fades: m STATE.
    slopes = [0.0, -1e-5, -1e-3, -2e-2]
    bound = [STATE * max(1.0, min(9000.0, 1 / max(-x, 1e-9)) / 128) for x in slopes]
    c = _case([9000], 4, 4, True, slopes=slopes)
    got = _run(c)
    _, _, states = _reference(c)
    for n, ref in states.items():
        for h in range(4):
            rel = float((got[n][:, h].double() - ref[:, h]).norm() / ref[:, h].norm())
            assert rel <= bound[h], (n, h, rel)


def test_non_finite_rows_of_a_long_document_stay_there():
    lens = [2600, 3000, 500]
    c = _case(lens, 2, 2, True)
    want = _run(c)
    d = {k: (x.clone() if torch.is_tensor(x) else x) for k, x in c.items()}
    for k in ("q", "k", "v", "dO"):
        d[k][2600:5600] = float("nan")
    got = _run(d)
    for k in ("o", "dq", "dk", "dv"):
        assert torch.equal(got[k][:2600], want[k][:2600]) and torch.equal(got[k][5600:], want[k][5600:]), k
    for k in ("ht", "dh0"):
        assert torch.equal(got[k][0], want[k][0]) and torch.equal(got[k][2], want[k][2]), k


def test_two_graphs_share_a_workspace():
    # calls on one workspace and saved set, captured apart and replayed in turn on one stream
    a, b = _case([2500, 100], 2, 2, True, seed=1), _case([2500, 100], 2, 2, True, seed=2)
    want = [_run(a), _run(b)]
    T, N, H = 2600, 2, 2
    ws = torch.empty(max(kda.kda_linattn_workspace_size(T, N, H, H, op)[0] for op in (0, 1, 2)), dtype=torch.uint8, device="cuda")
    saved = torch.empty(kda.kda_linattn_workspace_size(T, N, H, H, kda.KDA_OP_FWD)[1], dtype=torch.uint8, device="cuda")

    def call(c):
        x, kw = (c["q"], c["k"], c["v"], c["slope"], c["cu"]), dict(h0=c["h0"], scale=c["scale"])
        o, ht, _ = kda.kda_linattn_fwd(*x, **kw, saved=saved, ws=ws)
        return dict(kda.kda_linattn_bwd(*x, c["dO"], **kw, dht=c["dht"], saved=saved, ws=ws), o=o, ht=ht)

    graphs, outs = [], []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(c))
        graphs.append(g)
    for _ in range(2):
        for g, out, w in zip(graphs, outs, want):
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(out[k], w[k]) for k in w)


def test_offsets_beyond_32_bits():
    # rows of a projection of 2.3e9 elements, and a pool of 2.2e9 state elements
    T, wide = 36000, 64 * 1024
    big = torch.empty((T, wide), dtype=torch.bfloat16, device="cuda")
    c = _case([T - 1000, 1000], 1, 1, False, strided=False)
    views = {}
    for i, n in enumerate(("q", "k", "v")):
        views[n] = big[:, wide - 128 * (i + 1):wide - 128 * i].unflatten(1, (1, 128)).copy_(c[n])
    want, got = _run(c), _run(dict(c, **views))
    assert all(torch.equal(got[k], want[k]) for k in want)
    del big, views
    H, pool = 64, 2150
    gen = torch.Generator("cuda").manual_seed(0)
    q, k, v = (torch.randn((3, H, D), generator=gen, device="cuda").bfloat16() for _ in range(3))
    slope = -torch.rand(H, device="cuda")
    h = torch.empty((pool, H, D, D), device="cuda")
    slots = torch.tensor([pool - 1, 0, pool - 3], dtype=torch.int32, device="cuda")
    small = torch.randn((3, H, D, D), generator=gen, device="cuda")
    h[slots.long()] = small
    o, _ = kda.kda_linattn_step(q, k, v, slope, h, slots=slots)
    o2, small = kda.kda_linattn_step(q, k, v, slope, small)
    assert torch.equal(o, o2) and torch.equal(h[slots.long()], small)
