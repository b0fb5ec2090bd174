"""Pins of the FP64 oracle of the norm and rotation, and of the frequencies (CPU)."""
import math

import numpy as np
import pytest

from linear_attention_chunked_gb300 import build, kda
from oracle import rope


def test_a_quarter_turn_by_hand():
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    f = [math.pi / 2, math.pi]
    assert np.allclose(rope.rope_fwd(x, [1], f, interleaved=True), [[[-2, 1, -3, -4, 5, 6]]])
    assert np.allclose(rope.rope_fwd(x, [1], f), [[[-3, -2, 1, -4, 5, 6]]])


def test_lengths_and_relative_positions():
    r = np.random.default_rng(0)
    q, k, f = r.normal(size=(1, 1, 8)), r.normal(size=(1, 1, 8)), r.random(4)
    for inter in (False, True):
        turn = lambda x, p: rope.rope_fwd(x, [p], f, interleaved=inter)  # noqa: E731
        assert np.isclose((turn(q, 17) ** 2).sum(), (q ** 2).sum())
        assert np.isclose((turn(q, 17) * turn(k, 5)).sum(), (turn(q, 112) * turn(k, 100)).sum())
    x = rope.rope_fwd(q, [0], f, norm=True, eps=0.0)
    assert np.isclose((x ** 2).mean(), 1)


def test_layouts_are_a_permutation_apart():
    r = np.random.default_rng(1)
    x, f = r.normal(size=(3, 2, 8)), r.random(4)
    p = np.arange(8).reshape(4, 2).T.ravel()  # halves' channel j is neighbours' channel p[j]
    assert np.allclose(rope.rope_fwd(x[..., p], [0, 3, 9], f), rope.rope_fwd(x, [0, 3, 9], f, interleaved=True)[..., p])


@pytest.mark.parametrize("inter,norm,R", [(False, True, 8), (True, True, 4), (False, False, 6), (True, True, 0)])
def test_gradients_by_central_differences(inter, norm, R):
    r = np.random.default_rng(2)
    x, w, dy, f = r.normal(size=(3, 2, 8)), r.normal(size=8), r.normal(size=(3, 2, 8)), r.random(R // 2)
    kw = dict(norm=norm, interleaved=inter, scale=1.3)
    dx, dw = rope.rope_bwd(x, [2, 0, 7], f, dy, w=w if norm else None, **kw)
    loss = lambda x, w: (rope.rope_fwd(x, [2, 0, 7], f, w=w if norm else None, **kw) * dy).sum()  # noqa: E731
    e, d, dd = 1e-6, r.normal(size=x.shape), r.normal(size=8)
    assert abs((loss(x + e * d, w) - loss(x - e * d, w)) / (2 * e) - (dx * d).sum()) < 1e-7
    if norm:
        assert abs((loss(x, w + e * dd) - loss(x, w - e * dd)) / (2 * e) - (dw * dd).sum()) < 1e-7


def test_frequencies():
    build.build()
    freq = lambda R, **kw: kda.kda_rope_frequencies(R, device="cpu", **kw)  # noqa: E731
    f, s = freq(64)
    assert s == 1.0 and np.allclose(f.numpy(), 10000.0 ** (-2 * np.arange(32) / 64), rtol=1e-14)
    lin, _ = freq(64, scaling="linear", factor=4.0)
    assert np.allclose(lin.numpy(), f.numpy() / 4)
    base, _ = freq(64, scaling="base", factor=4.0)
    assert np.isclose(base[0], 1.0) and np.isclose(float(base[-1]), float(f[-1]) / 4)  # the slowest pair
    ramp, s = freq(64, scaling="ramp", factor=4.0, trained=4096, slow=1.0, fast=32.0)
    turns = 4096 * f.numpy() / (2 * np.pi)
    assert np.allclose(ramp.numpy()[turns >= 32], f.numpy()[turns >= 32])
    assert np.allclose(ramp.numpy()[turns <= 1], f.numpy()[turns <= 1] / 4) and (turns <= 1).any()
    between = (turns > 1) & (turns < 32)
    assert between.any() and (ramp.numpy()[between] < f.numpy()[between]).all() and (ramp.numpy()[between] > f.numpy()[between] / 4).all()
    assert np.isclose(s, 0.1 * np.log(4) + 1)
    assert freq(0)[0].numel() == 0
    for bad in (dict(R=3), dict(R=-2), dict(R=258), dict(R=8, base=0.0), dict(R=8, base=float("inf")),
                dict(R=8, scaling="linear", factor=0.5), dict(R=8, scaling="ramp", factor=2.0, slow=4.0, fast=4.0)):
        with pytest.raises(kda.KdaError):
            freq(**bad)
    with pytest.raises(ValueError, match="scaling must be"):
        freq(8, scaling="other")
