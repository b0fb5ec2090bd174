"""Documents of many chunks against the FP64 oracle, and layer norms whose column sums add several rows a
slot: the loops of the carries (16 chunks a turn) and of the re-reading norm kernels (32 row slots) go round
more than once.

Bounds of the scan.  A state takes one multiply-add and one decay per token of its chunk and one of each
per chunk before it, each off by at most 2^-22 of the value; a chunk's sum of steps, 64 fp32 additions, adds 16 of
them (64 roundings of 2^-24, over as many chunks as the state remembers), the step itself (softplus) 8.  Gradients are
products of two such values.
"""
import numpy as np
import pytest
import torch

from linear_attention_chunked_gb300 import kda
from oracle import layernorm, ssm
from test_ssm_gpu import DT, _close, _inputs, _np, _ref_args

pytestmark = pytest.mark.gpu


def _tol(lens):
    return (64 + -(-max(lens) // 64) + 16 + 8) * 2.0 ** -22


def _slow(a):
    """Decays from e^-0.0005 to e^-0.05 a token: states that remember chunks, and the whole document."""
    gen = torch.Generator("cpu").manual_seed(1)
    a["A"] = -torch.exp(torch.rand(a["A"].shape, generator=gen) * float(np.log(100.0)) + float(np.log(0.01))).cuda()


# 16, 17, 18 and 35 chunks, whole and ragged ones, an empty document and a short one between them
LENS = [1024, 1025, 0, 1088, 63, 1089, 2200]


@pytest.mark.parametrize("C,S,G,dtype,h0", [(12, 16, 1, "fp32", True), (10, 4, 2, "fp32", False), (9, 7, 1, "bf16", True), (8, 32, 1, "fp32", True)])
def test_many_chunks(C, S, G, dtype, h0):
    a, kw, dy, dht = _inputs(LENS, C, S, G, dtype, 21, h0=h0)
    _slow(a)
    ra, rk = _ref_args(a, kw)
    y_ref, ht_ref = ssm.ssm_fwd(**ra, **rk)
    y, ht, saved = kda.kda_ssm_fwd(**a, **kw)
    _close("y", y, y_ref, _tol(LENS))
    _close("ht", ht, ht_ref, _tol(LENS))
    y2, ht2, _ = kda.kda_ssm_fwd(**a, **kw, save=False)
    assert torch.equal(y2, y) and torch.equal(ht2, ht)
    ref = ssm.ssm_bwd(**ra, dy=_np(dy), dht=_np(dht), **rk)
    got = kda.kda_ssm_bwd(**a, dy=dy, dht=dht, saved=saved, **kw)
    for k in got:
        _close(k, got[k], ref[k], 2 * _tol(LENS))
    replay = kda.kda_ssm_bwd(**a, dy=dy, dht=dht, **kw)
    assert all(torch.equal(replay[k], got[k]) for k in got)


def test_many_chunks_in_the_throughput_forms():
    # 66 chunks x 32 blocks of channels; the oracle takes some channels, which alone have gradients
    lens, C = [2200, 1089, 700], 4096
    a, kw, dy, dht = _inputs(lens, C, 16, 1, "fp32", 22, h0=True)
    _slow(a)
    ch = np.r_[0:5, 2000:2003, C - 3:C]
    mask = torch.zeros(C, device="cuda")
    mask[torch.from_numpy(ch).cuda()] = 1
    dy, dht = dy * mask, dht * mask[:, None]
    pick = lambda t: _np(t)[..., ch]  # noqa: E731
    ra = dict(u=pick(a["u"]), dt=pick(a["dt"]), A=_np(a["A"])[ch], B=_np(a["B"]), Cm=_np(a["C"]), cu_seqlens=a["cu_seqlens"].cpu().numpy())
    rk = dict(D=pick(kw["D"]), dt_bias=pick(kw["dt_bias"]), z=pick(kw["z"]), h0=_np(kw["h0"])[:, ch])
    y_ref, ht_ref = ssm.ssm_fwd(**ra, **rk)
    y, ht, saved = kda.kda_ssm_fwd(**a, **kw)
    idx = torch.from_numpy(ch).cuda()
    _close("y", y[:, idx], y_ref, _tol(lens))
    _close("ht", ht[:, idx], ht_ref, _tol(lens))
    ref = ssm.ssm_bwd(**ra, dy=_np(dy)[:, ch], dht=_np(dht)[:, ch], **rk)
    got = kda.kda_ssm_bwd(**a, dy=dy, dht=dht, saved=saved, **kw)
    for k in ("du", "ddt", "dz", "dD", "ddt_bias"):
        _close(k, got[k][..., idx], ref[k], 2 * _tol(lens))
    _close("dA", got["dA"][idx], ref["dA"], 2 * _tol(lens))
    _close("dh0", got["dh0"][:, idx], ref["dh0"], 2 * _tol(lens))
    _close("dB", got["dB"], ref["dB"], 2 * _tol(lens))
    _close("dC", got["dC"], ref["dC"], 2 * _tol(lens))


# rows too long for the registers, whole and odd ones: more of them than the 32 slots that share the column sums.
# Sums of C terms by 1024 threads and a tree, and of T rows: a few 2^-24 of their size, held to 1e-5 of the rms
@pytest.mark.parametrize("T", [33, 65, 100])
@pytest.mark.parametrize("dtype,C", [("fp32", 8200), ("bf16", 16392), ("fp16", 16383)])
def test_long_rows(T, dtype, C):
    gen, dt = torch.Generator("cpu").manual_seed(T), DT[dtype]
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x, r, dy, ds = ((2 * rn(T, C) + 0.5).to(dt).cuda(), rn(T, C).to(dt).cuda(), rn(T, C).to(dt).cuda(), rn(T, C).to(dt).cuda())
    w, b = (1 + 0.1 * rn(C)).cuda(), (0.1 * rn(C)).cuda()
    for res, dsum in ((None, None), (r, ds)):
        y, total, mean, rstd = kda.kda_layernorm_fwd(x, w, b, res=res)
        yr, mr, rr = layernorm.layernorm_fwd(_np(total), _np(w), _np(b))
        for name, t, want in (("y", y, yr), ("mean", mean, mr), ("rstd", rstd, rr)):
            _close(name, t, want, 1e-5)
        g = kda.kda_layernorm_bwd(total, w, mean, rstd, dy, dsum=dsum)
        ref = layernorm.layernorm_bwd(_np(total), _np(dy), _np(w), _np(dsum))
        for k in g:
            _close(k, g[k], ref[k], 1e-5)


# Narrow rows, whose elements can lie close together: each row is held to a bound of its own.  With e the error of a
# normalised value, max|x| rstd 2^-21 (up to eight roundings of the mean, its factor and the difference) + 2^-21, and
# X = sqrt(C) its largest size, rstd is off by e X + 2^-21 of itself; d = dy w (largest D), mean(d xh) by
# D (e + X 2^-21), and dx = rstd (d - mean(d) - xh mean(d xh)) by rstd D (2 X e + (2 + X X) (e X + 2^-20))
@pytest.mark.parametrize("T,C", [(40000, 3), (40000, 2), (20000, 5), (37, 3)])
def test_narrow_rows(T, C):
    gen = torch.Generator("cuda").manual_seed(C)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x, dy, w, b = 2 * rn(T, C) + 0.5, rn(T, C), 1 + 0.1 * rn(C), 0.1 * rn(C)
    y, _, mean, rstd = kda.kda_layernorm_fwd(x, w, b)
    g = kda.kda_layernorm_bwd(x, w, mean, rstd, dy)
    v, wn = _np(x), _np(w)
    yr, _, rr = layernorm.layernorm_fwd(v, wn, _np(b))
    ref = layernorm.layernorm_bwd(v, _np(dy), wn)["dx"]
    X, u = np.sqrt(C), 2.0 ** -21
    e = np.abs(v).max(1) * rr * u + u
    D = np.abs(_np(dy) * wn).max(1)
    dy_err = np.abs(_np(y) - yr).max(1) / (np.abs(wn).max() * (e + X * (e * X + u)) + u * np.abs(yr).max(1))
    dx_err = np.abs(_np(g["dx"]) - ref).max(1) / (rr * D * (2 * X * e + (2 + X * X) * (e * X + 2 * u)))
    assert dy_err.max() <= 1 and dx_err.max() <= 1, (dy_err.max(), dx_err.max())
