"""Pins of the layer norm's FP64 oracle (CPU)."""
import numpy as np

from oracle import layernorm


def test_rows_have_zero_mean_and_unit_variance():
    v = np.random.default_rng(0).normal(size=(5, 17)) * 3 + 2
    y, mean, rstd = layernorm.layernorm_fwd(v, eps=0.0)
    assert np.allclose(y.mean(-1), 0, atol=1e-14) and np.allclose((y ** 2).mean(-1), 1)
    assert np.allclose(mean, v.mean(-1)) and np.allclose(rstd, 1 / v.std(-1))


def test_shift_and_scale_invariance():
    v = np.random.default_rng(1).normal(size=(4, 9))
    y, _, _ = layernorm.layernorm_fwd(v, eps=0.0)
    y2, _, _ = layernorm.layernorm_fwd(7 * v - 3, eps=0.0)
    assert np.allclose(y, y2)


def test_gradients_by_central_differences():
    r = np.random.default_rng(2)
    v, w, b, dy, ds = (r.normal(size=s) for s in ((3, 8), (8,), (8,), (3, 8), (3, 8)))
    g = layernorm.layernorm_bwd(v, dy, w, ds)
    loss = lambda v, w, b: (layernorm.layernorm_fwd(v, w, b)[0] * dy).sum() + (v * ds).sum()  # noqa: E731
    e = 1e-6
    for i, (x, got) in enumerate([(v, g["dx"]), (w, g["dw"]), (b, g["db"])]):
        d = r.normal(size=x.shape)
        args = [v, w, b]
        hi, lo = list(args), list(args)
        hi[i], lo[i] = x + e * d, x - e * d
        assert abs((loss(*hi) - loss(*lo)) / (2 * e) - (got * d).sum()) < 1e-7
