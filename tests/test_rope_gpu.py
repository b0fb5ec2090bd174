"""GPU parity of the norm and rotation of queries and keys (kda_rope_*) against the FP64 oracle.

Bounds, elementwise.  An output's rounding is eps / 2 of itself.  In fp32 a turned value takes the norm's factor (a sum
of D squares in a tree, a root and a division), a weight, cosine and sine (two ulp each, and the angle's own rounding to
24 bits of half a turn), two products and a sum: 16 units of 2^-24 of the pair's length.  A gradient adds the dot product
over the head: 32 units of the size of its parts.  dw sums T x heads terms, each off by 32 units, in chains below 512: the
terms' absolute sum times 2^-24 (32 + 512) bounds it.
"""
import numpy as np
import pytest
import torch

from linear_attention_chunked_gb300 import kda
from oracle import rope

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24


def _np(t):
    return None if t is None else t.detach().cpu().double().numpy()


def _case(T, Hq, Hk, C, R, dtype, norm, far=0, fused=True, seed=0):
    gen = torch.Generator("cpu").manual_seed(seed + T + C)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    dt = DT[dtype]

    def rows():
        if fused:
            x = (1.5 * rn(T, (Hq + 2 * Hk) * C)).to(dt).cuda()
            return x[:, :Hq * C].unflatten(1, (Hq, C)), x[:, Hq * C:(Hq + Hk) * C].unflatten(1, (Hk, C))
        return (1.5 * rn(T, Hq, C)).to(dt).cuda(), (1.5 * rn(T, Hk, C)).to(dt).cuda()

    q, k = rows()
    dq, dk = rows()
    pos = torch.randint(0, far + 1, (T,), generator=gen, dtype=torch.int32) if far else torch.arange(T, dtype=torch.int32)
    f, s = kda.kda_rope_frequencies(R, scaling="ramp", factor=8.0)
    return q, k, dq, dk, pos.cuda(), f, s, ((1 + 0.1 * rn(C)).cuda(), (1 + 0.1 * rn(C)).cuda()) if norm else (None, None)


def _pair_size(n, R, inter):
    """Length of the pair that a channel belongs to."""
    size = np.abs(n)
    i = np.arange(R // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, R // 2 + i)
    length = np.hypot(n[..., a], n[..., b])
    size[..., a] = length
    size[..., b] = length
    return size


def _check(c, inter, norm):
    q, k, dq, dk, pos, f, s, (wq, wk) = c
    C, R, half = q.shape[-1], 2 * f.numel(), torch.finfo(q.dtype).eps / 2
    kw = dict(wq=wq, wk=wk, norm=norm, interleaved=inter, scale=s)
    out = dict(zip("qk", kda.kda_rope_fwd(q, k, pos, f, **kw)))
    g = kda.kda_rope_bwd(q, k, pos, f, dq, dk, **kw)
    for name, x, dy, w in (("q", q, dq, wq), ("k", k, dk, wk)):
        o = dict(norm=norm, interleaved=inter, scale=s, w=_np(w))
        ref = rope.rope_fwd(_np(x), _np(pos), _np(f), **o)
        tol = half * np.abs(ref) + 16 * U * _pair_size(ref, R, inter) + 1e-30
        if q.dtype == torch.float16:
            tol = tol + 2.0 ** -25  # below its normal range
        err = np.abs(_np(out[name]) - ref)
        assert (err <= tol).all(), (name, float((err / tol).max()))
        dx, dw = rope.rope_bwd(_np(x), _np(pos), _np(f), _np(dy), **o)
        turned, _ = rope.rope_bwd(_np(x), _np(pos), _np(f), _np(dy), norm=False, interleaved=inter, scale=s)
        size = _pair_size(turned, R, inter)
        if norm:
            xn = _np(x)
            r = 1 / np.sqrt((xn ** 2).mean(-1, keepdims=True) + 1e-6)
            wa = np.abs(_np(w))
            part = r * (size * wa + np.abs(xn * r) * (size * wa * np.abs(xn * r)).mean(-1, keepdims=True))
            terms = (size * np.abs(xn * r)).sum((0, 1))
            err = np.abs(_np(g["dw" + name]) - dw)
            assert (err <= U * (32 + 512) * terms + 1e-30).all(), ("dw" + name, float(err.max()))
            size = part
        tol = half * np.abs(dx) + 32 * U * size + (2.0 ** -25 if q.dtype == torch.float16 else 1e-30)
        err = np.abs(_np(g["d" + name]) - dx)
        assert (err <= tol).all(), ("d" + name, float((err / tol).max()))
    again = kda.kda_rope_bwd(q, k, pos, f, dq, dk, **kw)
    assert all(torch.equal(again[n], g[n]) for n in g)


# head sizes of every lane group, parts that turn, widths that take single pairs, many rows
SHAPES = [(1, 1, 1, 2, 2), (1, 16, 16, 128, 128), (5, 3, 2, 128, 64), (7, 2, 1, 64, 64), (3, 1, 4, 256, 256), (9, 7, 3, 80, 52),
          (4, 5, 1, 96, 0), (6, 2, 2, 72, 40), (2, 3, 3, 254, 130), (33, 9, 5, 34, 10), (300, 40, 8, 128, 128), (1, 70, 3, 16, 8),
          (513, 5, 2, 128, 32)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("inter", [False, True])
def test_norm_and_rotation(shape, dtype, inter):
    for norm in (True, False):
        _check(_case(*shape, dtype, norm, fused=norm), inter, norm)


@pytest.mark.parametrize("T,Hq,Hk,C,R,dtype", [(5000, 8, 2, 128, 128, "bf16"), (4001, 3, 3, 64, 48, "fp32"), (3000, 5, 4, 50, 50, "fp16")])
def test_many_tokens(T, Hq, Hk, C, R, dtype):
    _check(_case(T, Hq, Hk, C, R, dtype, True), False, True)


@pytest.mark.parametrize("far", [10 ** 6, 2 ** 31 - 2])
def test_far_positions(far):
    # the oracle's own angles: pos freq in fp64 is off by 2^-53 of it, 2.4e-7 at 2^31 (below the bound's 16 2^-24)
    _check(_case(64, 2, 2, 128, 128, "fp32", False, far=far), True, False)


def test_negative_positions_turn_back():
    q, k, _, _, pos, f, _, _ = _case(20, 2, 2, 64, 64, "fp32", False)
    a, b = kda.kda_rope_fwd(q, k, pos, f)
    a, b = kda.kda_rope_fwd(a, b, -pos, f)
    assert float((a - q).abs().max()) <= 64 * U * float(q.abs().max()) * 2 and float((b - k).abs().max()) <= 64 * U * float(k.abs().max()) * 2


def test_in_place_and_into_strided_outputs():
    q, k, _, _, pos, f, s, (wq, wk) = _case(50, 6, 2, 128, 96, "bf16", True)
    kw = dict(wq=wq, wk=wk, norm=True, scale=s)
    a, b = kda.kda_rope_fwd(q, k, pos, f, **kw)
    wide = torch.zeros((50, 10 * 128 + 8), dtype=torch.bfloat16, device="cuda")
    qo, ko = wide[:, 8:8 + 6 * 128].unflatten(1, (6, 128)), wide[:, 8 + 6 * 128:8 + 8 * 128].unflatten(1, (2, 128))
    r = kda.kda_rope_fwd(q, k, pos, f, q_out=qo, k_out=ko, **kw)
    assert r[0] is qo and torch.equal(qo, a) and torch.equal(ko, b)
    assert not wide[:, :8].any() and not wide[:, 8 + 8 * 128:].any()
    kda.kda_rope_fwd(q, k, pos, f, q_out=q, k_out=k, **kw)
    assert torch.equal(q, a) and torch.equal(k, b)


def test_rows_at_odd_addresses():
    q, k, dq, dk, pos, f, s, (wq, wk) = _case(40, 3, 2, 128, 128, "bf16", True)
    odd = torch.empty((40, 3 * 128 + 3), dtype=torch.bfloat16, device="cuda")
    x = odd[:, 1:1 + 3 * 128].unflatten(1, (3, 128)).copy_(q)
    kw = dict(wq=wq, wk=wk, norm=True, scale=s)
    assert all(torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-5)  # (sums in another order)
               for a, b in zip(kda.kda_rope_fwd(x, k, pos, f, **kw), kda.kda_rope_fwd(q, k, pos, f, **kw)))


def test_one_side_alone_and_no_tokens():
    q, k, dq, dk, pos, f, s, (wq, wk) = _case(9, 4, 2, 64, 32, "fp16", True)
    kw = dict(norm=True, scale=s)
    a, b = kda.kda_rope_fwd(q, k, pos, f, wq=wq, wk=wk, **kw)
    a1, none = kda.kda_rope_fwd(q, None, pos, f, wq=wq, **kw)
    assert none is None and torch.equal(a1, a)
    g = kda.kda_rope_bwd(q, k, pos, f, dq, dk, wq=wq, wk=wk, **kw)
    g1 = kda.kda_rope_bwd(q, None, pos, f, dq, None, wq=wq, **kw)
    assert set(g1) == {"dq", "dwq"} and torch.equal(g1["dq"], g["dq"])
    e = torch.empty((0, 4, 64), device="cuda")
    p0 = torch.empty((0,), dtype=torch.int32, device="cuda")
    assert kda.kda_rope_fwd(e, e, p0, f)[0].shape == (0, 4, 64)
    g0 = kda.kda_rope_bwd(e, e, p0, f, e, e, wq=wq, wk=wk, norm=True)
    assert not g0["dwq"].any() and not g0["dwk"].any()


def test_non_finite_heads_stay_apart():
    q, k, dq, dk, pos, f, s, (wq, wk) = _case(6, 3, 2, 128, 128, "bf16", True, fused=False)
    kw = dict(wq=wq, wk=wk, norm=True, scale=s)
    a, b = kda.kda_rope_fwd(q, k, pos, f, **kw)
    q2 = q.clone()
    q2[2, 1, 5] = float("nan")
    a2, b2 = kda.kda_rope_fwd(q2, k, pos, f, **kw)
    assert torch.isnan(a2[2, 1]).all() and torch.equal(b2, b)
    a2[2, 1] = a[2, 1]
    assert torch.equal(a2, a)


def test_on_a_stream_and_in_a_graph():
    q, k, dq, dk, pos, f, s, (wq, wk) = _case(70, 4, 2, 128, 128, "bf16", True)
    kw = dict(wq=wq, wk=wk, norm=True, scale=s)
    call = lambda: dict(kda.kda_rope_bwd(q, k, pos, f, dq, dk, **kw), **dict(zip(("q", "k"), kda.kda_rope_fwd(q, k, pos, f, **kw))))  # noqa: E731
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(got[n], want[n]) for n in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[n], want[n]) for n in want)


def test_gradient_against_differences():
    # fp32 outputs differenced over 2e = 2e-2: rounding 2^-22 |y| / 2e, truncation e^2
    q, k, dq, dk, pos, f, s, (wq, wk) = _case(6, 2, 1, 96, 48, "fp32", True, fused=False)
    kw = dict(norm=True, scale=s)
    g = kda.kda_rope_bwd(q, k, pos, f, dq, dk, wq=wq, wk=wk, **kw)
    e, gen = 1e-2, torch.Generator("cuda").manual_seed(1)
    for i, n in enumerate(("dq", "dk", "dwq", "dwk")):
        args = [q, k, wq, wk]
        d = torch.randn(args[i].shape, generator=gen, device="cuda")
        out = []
        for sgn in (e, -e):
            t = list(args)
            t[i] = args[i] + sgn * d
            out.append([y.double() for y in kda.kda_rope_fwd(t[0], t[1], pos, f, wq=t[2], wk=t[3], **kw)])
        num = float(sum(((x - y) * z.double()).sum() for x, y, z in zip(out[0], out[1], (dq, dk))) / (2 * e))
        size = float(sum(x.norm() * z.norm() for x, z in zip(out[0], (dq, dk))))
        assert abs(num - float((g[n].double() * d.double()).sum())) <= 2.0 ** -22 * size / (2 * e) + 10 * e * e * size


def test_offsets_beyond_32_bits():
    T, wide = 36000, 64 * 1024
    big = torch.empty((T, wide), dtype=torch.bfloat16, device="cuda")
    q, k, dq, dk, pos, f, s, (wq, wk) = _case(T, 1, 1, 64, 64, "bf16", True, fused=False)
    x = big[:, wide - 64:].unflatten(1, (1, 64)).copy_(q)
    kw = dict(wq=wq, wk=wk, norm=True, scale=s)
    want, _ = kda.kda_rope_fwd(q, k, pos, f, **kw)
    got, _ = kda.kda_rope_fwd(x, k, pos, f, q_out=x, **kw)
    assert got is x and torch.equal(x, want)


def test_two_graphs_share_a_workspace():
    a, b = _case(70, 4, 2, 128, 128, "bf16", True, seed=1), _case(70, 4, 2, 128, 128, "bf16", True, seed=2)
    ws = torch.empty(kda.kda_rope_workspace_size(128), dtype=torch.uint8, device="cuda")

    def call(c, ws=None):
        q, k, dq, dk, pos, f, s, (wq, wk) = c
        return kda.kda_rope_bwd(q, k, pos, f, dq, dk, wq=wq, wk=wk, norm=True, scale=s, ws=ws)

    want, graphs, outs = [call(a), call(b)], [], []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(c, ws))
        graphs.append(g)
    for _ in range(2):
        for g, out, w in zip(graphs, outs, want):
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(out[k], w[k]) for k in w)
