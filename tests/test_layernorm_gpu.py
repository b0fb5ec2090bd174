"""GPU parity of the layer norm (kda_layernorm_fwd / kda_layernorm_bwd) against the FP64 oracle.

Bounds.  Row sums of C terms in fp32 trees are off by a few 2^-24 of their terms' size, the column
sums of T rows by a few 2^-24 sqrt(T): fp32 outputs are held to 1e-5 of their rms.  Outputs in bf16
/ fp16 add the rounding of their own value, eps / 2.
"""
import numpy as np
import pytest
import torch

from linear_attention_chunked_gb300 import kda
from oracle import layernorm
from test_ssm_gpu import DT, _close, _np

pytestmark = pytest.mark.gpu

TOL = 1e-5

# widths at the edges of a warp's, 128 threads' and 512 threads' registers in whole vectors, odd
# widths, and rows too long for registers of either kind
SHAPES = [(1, 1), (3, 7), (5, 8), (9, 256), (4, 1024), (700, 64), (33, 513), (6, 2049), (3, 4096), (300, 2048), (2, 8200),
          (7, 16384), (2, 16392), (2, 8195), (40, 1111), (1300, 1024)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_layernorm(shape, dtype):
    T, C = shape
    dt, gen = DT[dtype], torch.Generator("cpu").manual_seed(T + C)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x, r, dy, ds = ((2 * rn(T, C) + 0.5).to(dt).cuda(), rn(T, C).to(dt).cuda(), rn(T, C).to(dt).cuda(), rn(T, C).to(dt).cuda())
    w, b = (1 + 0.1 * rn(C)).cuda(), (0.1 * rn(C)).cuda()
    for res, ww, bb in ((None, w, b), (r, w, b), (r, None, None)):
        y, total, mean, rstd = kda.kda_layernorm_fwd(x, ww, bb, res=res)
        if res is None:
            assert total is x
        else:
            assert torch.equal(total, (x.float() + r.float()).to(dt))
        yr, mr, rr = layernorm.layernorm_fwd(_np(total), _np(ww), _np(bb))
        if C > 1:
            _close("y", y, yr, TOL)
        else:  # one channel: the normalised value is zero
            assert torch.equal(y, torch.zeros_like(y) if bb is None else bb.to(dt).expand_as(y))
        _close("mean", mean, mr, TOL)
        _close("rstd", rstd, rr, TOL)
        for dsum in (None, ds):
            g = kda.kda_layernorm_bwd(total, ww, mean, rstd, dy, dsum=dsum)
            ref = layernorm.layernorm_bwd(_np(total), _np(dy), _np(ww), _np(dsum))
            if C > 1:
                _close("dx", g["dx"], ref["dx"], TOL)
                _close("dw", g["dw"], ref["dw"], TOL)
            else:
                assert torch.equal(g["dx"], torch.zeros_like(dy) if dsum is None else dsum)
                assert not g["dw"].any()
            _close("db", g["db"], ref["db"], TOL)
            again = kda.kda_layernorm_bwd(total, ww, mean, rstd, dy, dsum=dsum)
            assert all(torch.equal(again[k], g[k]) for k in g)


# more rows than the machine holds at once: blocks walk several rows (a row count that leaves a last
# step short), for a warp, 128, 256 and 512 threads a row, one, two and four vectors a thread
@pytest.mark.parametrize("dtype,T,C", [("bf16", 9999, 136), ("fp32", 9731, 200), ("fp16", 7500, 1000), ("bf16", 2501, 1032),
                                       ("fp32", 2437, 1024), ("bf16", 2000, 4096), ("bf16", 701, 8192), ("fp32", 1300, 2048),
                                       ("fp32", 613, 4096), ("bf16", 611, 16384), ("fp32", 620, 8192), ("bf16", 1500, 3001),
                                       # rows that start inside a vector, in every such form
                                       ("fp16", 9999, 61), ("bf16", 9999, 399), ("fp32", 10001, 131), ("bf16", 5000, 777), ("fp32", 2500, 555),
                                       ("fp32", 1300, 1111), ("fp16", 2600, 2047), ("fp32", 700, 3333), ("bf16", 1300, 7001), ("fp32", 640, 8001),
                                       ("bf16", 700, 15001), ("fp16", 3000, 10), ("fp32", 40000, 3)])
def test_layernorm_many_rows(dtype, T, C):
    gen, dt = torch.Generator("cuda").manual_seed(T), DT[dtype]
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, r, dy, ds = ((2 * rn(T, C) + 0.5).to(dt), rn(T, C).to(dt), rn(T, C).to(dt), rn(T, C).to(dt))
    w, b = 1 + 0.1 * rn(C), 0.1 * rn(C)
    for res, dsum in ((None, None), (r, ds)):
        y, total, mean, rstd = kda.kda_layernorm_fwd(x, w, b, res=res)
        if res is not None:
            assert torch.equal(total, (x.float() + r.float()).to(dt))
        yr, mr, rr = layernorm.layernorm_fwd(_np(total), _np(w), _np(b))
        # fp32 statistics: the mean's rounding, 2^-24 |x|, reaches a normalised value times rstd and a gradient
        # times rstd^2 (rows of three elements can lie close together; from tens of elements on rstd is below 1)
        cond = [2.0 ** -22 * float(total.abs().max()) * float(rr.max()) ** n for n in (1, 2)]
        _close("y", y, yr, TOL + cond[0])
        _close("mean", mean, mr, TOL)
        _close("rstd", rstd, rr, TOL + cond[0])
        g = kda.kda_layernorm_bwd(total, w, mean, rstd, dy, dsum=dsum)
        ref = layernorm.layernorm_bwd(_np(total), _np(dy), _np(w), _np(dsum))
        for k in g:
            _close(k, g[k], ref[k], TOL + (cond[1] if k == "dx" else cond[0]))


def test_large_offset_keeps_the_variance():
    # variance about the mean, not E[v^2] - mean^2: rows at 1000 with unit spread (the inputs' own fp32
    # rounding is part of the reference's input; subtracting the mean costs 1000 2^-24 of a unit)
    x = (1000 + torch.randn((8, 2048), generator=torch.Generator().manual_seed(0))).cuda()
    y, _, _, _ = kda.kda_layernorm_fwd(x)
    _close("y", y, layernorm.layernorm_fwd(_np(x))[0], 1000 * 2.0 ** -24 * 4)


def test_non_finite_rows_stay_apart():
    x = torch.randn((9, 1000), device="cuda")
    y, _, _, _ = kda.kda_layernorm_fwd(x)
    x2 = x.clone()
    x2[4, 3] = float("inf")
    y2, _, _, _ = kda.kda_layernorm_fwd(x2)
    keep = [0, 1, 2, 3, 5, 6, 7, 8]
    assert torch.equal(y2[keep], y[keep]) and bool(torch.isnan(y2[4]).all())


def test_no_rows():
    x = torch.empty((0, 64), device="cuda")
    y, _, mean, rstd = kda.kda_layernorm_fwd(x)
    g = kda.kda_layernorm_bwd(x, None, mean, rstd, x)
    assert y.shape == (0, 64) and not g["dw"].any() and not g["db"].any()


def test_gradient_against_differences():
    # outputs in fp32 differenced over 2e = 2e-2: rounding 2^-22 |y| / 2e, truncation e^2
    gen = torch.Generator("cpu").manual_seed(3)
    x, dy, w, b = (torch.randn(s, generator=gen).cuda() for s in ((6, 96), (6, 96), (96,), (96,)))
    _, _, mean, rstd = kda.kda_layernorm_fwd(x, w, b)
    g = kda.kda_layernorm_bwd(x, w, mean, rstd, dy)
    e = 1e-2
    for i, k in enumerate(("dx", "dw", "db")):
        args = [x, w, b]
        d = torch.randn(args[i].shape, generator=gen).cuda()
        outs = []
        for s in (e, -e):
            t = list(args)
            t[i] = args[i] + s * d
            outs.append(kda.kda_layernorm_fwd(*t)[0].double())
        num = float(((outs[0] - outs[1]) * dy.double()).sum() / (2 * e))
        size = float(outs[0].norm() * dy.norm())
        assert abs(num - float((g[k].double() * d.double()).sum())) <= 2.0 ** -22 * size / (2 * e) + 10 * e * e * size
