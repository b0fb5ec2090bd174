"""The norm and rotation of queries and keys (kda_rope_*) where their arithmetic could leave its range: no eps, tiles that are
not full, rows far from one, values that are not finite.  Bounds as in test_rope_gpu.py."""
import numpy as np
import pytest
import torch

from linear_attention_chunked_gb300 import kda
from oracle import rope
from test_rope_gpu import U, _case, _np, _pair_size

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -126  # below it the kernels' results are zero


def _bounds(x, pos, f, dy, w, inter, scale, eps, half):
    """Definition and bounds of one tensor, forward and backward: {name: (value, tolerance)}."""
    R, o = 2 * len(f), dict(norm=True, interleaved=inter, scale=scale, w=w, eps=eps)
    y = rope.rope_fwd(x, pos, f, **o)
    dx, dw = rope.rope_bwd(x, pos, f, dy, **o)
    turned, _ = rope.rope_bwd(x, pos, f, dy, norm=False, interleaved=inter, scale=scale)
    size, wa = _pair_size(turned, R, inter), np.abs(w)
    r = 1 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    xr = np.abs(x * r)
    part = r * (size * wa + xr * (size * wa * xr).mean(-1, keepdims=True))
    least = 2.0 ** -25 if half == 2.0 ** -11 else TINY  # fp16: below its normal range
    return {"": (y, half * np.abs(y) + 16 * U * _pair_size(y, R, inter) + least),
            "d": (dx, half * np.abs(dx) + 32 * U * part + least),
            "dw": (dw, U * (32 + 512) * (size * xr).sum((0, 1)) + TINY)}


def _check(c, inter, eps):
    q, k, dq, dk, pos, f, s, (wq, wk) = c
    kw = dict(wq=wq, wk=wk, norm=True, interleaved=inter, scale=s, eps=eps)
    got = dict(zip("qk", kda.kda_rope_fwd(q, k, pos, f, **kw)))
    got.update(kda.kda_rope_bwd(q, k, pos, f, dq, dk, **kw))
    for n, x, dy, w in (("q", q, dq, wq), ("k", k, dk, wk)):
        eps32 = float(np.float32(eps))  # what the call takes
        for what, (ref, tol) in _bounds(_np(x), _np(pos), _np(f), _np(dy), _np(w), inter, s, eps32, torch.finfo(q.dtype).eps / 2).items():
            err = np.abs(_np(got[what + n]) - ref)
            assert (err <= tol).all(), (what + n, float(np.nanmax(err / tol)), int(np.isnan(err).sum()))


# tiles of tokens that the last ones do not fill, heads that a tile's groups do not share evenly, every pack width
PARTS = [(1, 1, 1, 128, 128), (37, 5, 3, 128, 64), (1777, 32, 8, 128, 128), (1777, 7, 3, 80, 52), (2500, 3, 1, 64, 64), (129, 11, 2, 96, 48),
         (33, 9, 5, 34, 10), (65, 3, 3, 254, 130), (4099, 2, 3, 128, 128)]


@pytest.mark.parametrize("shape", PARTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("inter", [False, True])
def test_no_eps(shape, dtype, inter):
    _check(_case(*shape, dtype, True), inter, 0.0)


# rows whose root mean square's inverse has no cube in fp32, both ways
@pytest.mark.parametrize("dtype,far,eps", [("bf16", 1e13, 1e-6), ("fp32", 1e13, 0.0), ("fp32", 3e16, 1e-6), ("bf16", 1e-12, 1e-30), ("fp32", 1e-13, 1e-30),
                                           ("fp32", 1e-14, 0.0), ("bf16", 1e-16, 0.0)])
@pytest.mark.parametrize("inter", [False, True])
def test_rows_far_from_one(dtype, far, eps, inter):
    for shape in ((77, 5, 3, 128, 64), (9, 7, 3, 80, 52), (5, 3, 3, 254, 130)):
        q, k, *rest = _case(*shape, dtype, True, fused=False)
        _check((q * far, k * far, *rest), inter, eps)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_rows_of_zeros(dtype):
    # x = 0 is an ordinary row where eps > 0: y = 0, dx = dy w / sqrt(eps) (in fp16's range where eps is not tiny)
    for eps in (1e-6,) if dtype == "fp16" else (1e-6, 1e-30):
        q, k, *rest = _case(21, 5, 3, 128, 64, dtype, True, fused=False)
        q[3], k[20, 1] = 0, 0
        q[7, 4] = 0
        _check((q, k, *rest), False, eps)


def _at(x, odd):
    """x as a view at an odd address with an odd token stride."""
    T, H, C = x.shape
    if not odd:
        return x
    return torch.empty((T, H * C + 3), dtype=x.dtype, device="cuda")[:, 1:1 + H * C].unflatten(1, (H, C)).copy_(x)


def _same(a, b):
    return torch.equal(torch.nan_to_num(a, 7.0), torch.nan_to_num(b, 7.0)) and torch.equal(torch.isnan(a), torch.isnan(b))


# every pack width, and the same rows where only single elements can be read
@pytest.mark.parametrize("C,R", [(128, 64), (128, 0), (80, 52), (72, 40), (96, 48), (34, 10), (254, 130), (16, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("odd", [False, True])
def test_channels_that_do_not_turn_pass_through(C, R, dtype, inter, odd):
    # without a norm an unturned channel is its input and no other channel depends on it, whatever it holds
    q, k, dq, dk, pos, f, s, _ = _case(11, 3, 2, C, R, dtype, False, fused=False)
    kw = dict(interleaved=inter, scale=s)
    a = [_at(x, odd) for x in (q, k)]
    fwd, bwd = kda.kda_rope_fwd(*a, pos, f, **kw), kda.kda_rope_bwd(*a, pos, f, _at(dq, odd), _at(dk, odd), **kw)
    rest = list(range(R, C))
    for bad in (float("inf"), float("nan")):
        for c in (rest[0], rest[len(rest) // 2], rest[-1]):
            x = [t.clone() for t in (q, k, dq, dk)]
            for t in x:
                t[4, 1, c] = bad
                t[0, 0, c] = -bad
                t[5, 0, R:] = bad
                t[6, 0, R:] = -0.0
            y = kda.kda_rope_fwd(_at(x[0], odd), _at(x[1], odd), pos, f, **kw)
            g = kda.kda_rope_bwd(*a, pos, f, _at(x[2], odd), _at(x[3], odd), **kw)
            for got, clean, given in ((y[0], fwd[0], x[0]), (y[1], fwd[1], x[1]), (g["dq"], bwd["dq"], x[2]), (g["dk"], bwd["dk"], x[3])):
                assert torch.equal(got[..., :R], clean[..., :R])
                assert _same(got[..., R:], given[..., R:])
                assert torch.equal(torch.signbit(got[6, 0, R:]), torch.signbit(given[6, 0, R:]))
    # with a norm an infinite channel takes the others of its head to zero and is no number itself
    x = q.clone()
    x[4, 1, rest[0]] = float("inf")
    y, _ = kda.kda_rope_fwd(_at(x, odd), a[1], pos, f, norm=True, **kw)
    want = torch.zeros(C, device="cuda")
    want[rest[0]] = float("nan")
    assert _same(y[4, 1].float(), want)


@pytest.mark.parametrize("C,R", [(128, 128), (80, 52), (34, 10)])
@pytest.mark.parametrize("inter", [False, True])
def test_frequencies_that_are_no_numbers(C, R, inter):
    # their pairs' angles are no numbers, at position 0 either; the other pairs turn as before
    q, k, dq, dk, pos, f, s, _ = _case(9, 3, 2, C, R, "fp32", False)
    kw = dict(interleaved=inter, scale=s)
    i = np.arange(R // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, R // 2 + i)
    call = lambda f: [*kda.kda_rope_fwd(q, k, pos, f, **kw), *kda.kda_rope_bwd(q, k, pos, f, dq, dk, **kw).values()]  # noqa: E731
    clean = call(f)
    for bad in (float("nan"), float("inf"), -float("inf")):
        g = f.clone()
        g[1] = g[R // 2 - 1] = bad
        lost = [int(x) for p in (1, R // 2 - 1) for x in (a[p], b[p])]
        kept = [c for c in range(C) if c not in lost]
        for got, want in zip(call(g), clean):
            assert torch.isnan(got[..., lost]).all() and torch.equal(got[..., kept], want[..., kept])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("inter", [False, True])
def test_rows_of_odd_addresses_and_strides(dtype, inter):
    # no word of two elements fits these rows, forward or backward
    for shape in ((40, 3, 2, 128, 128), (37, 5, 1, 80, 52), (9, 2, 3, 254, 130), (300, 1, 1, 2, 2), (65, 33, 4, 34, 10)):
        q, k, dq, dk, *rest = _case(*shape, dtype, True, fused=False)
        _check((*(_at(x, True) for x in (q, k, dq, dk)), *rest), inter, 1e-6)
