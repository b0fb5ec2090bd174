"""The state-space block of examples/ end to end: single tokens continue a prompt, and gradients train it."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_decoding_continues_the_prompt():
    from state_space_block import StateSpaceBlock, decode_error
    # the same tokens through matrix products of other shapes: bf16 roundings (2^-8 of a value) of the norm, u, dt
    # and y differ here and there; a few of them, on values up to four rms
    assert decode_error(StateSpaceBlock(width=128, channels=256)) <= 8 * 4 * 2.0 ** -8


def test_training_lowers_the_loss():
    from state_space_block import StateSpaceBlock, train
    losses = train(StateSpaceBlock(width=128, channels=256))
    assert losses[-1] < 0.5 * losses[0], losses


def test_gradient_of_the_whole_block():
    from state_space_block import StateSpaceBlock
    block = StateSpaceBlock(width=64, channels=128, seed=3)
    gen = torch.Generator("cuda").manual_seed(4)
    x, r, dy = (torch.randn((90, 64), generator=gen, device="cuda").bfloat16() for _ in range(3))
    cu = torch.tensor([0, 30, 90], dtype=torch.int32, device="cuda")
    y, _ = block.forward(x, r, cu)
    (y.float() * dy.float()).sum().backward()
    # D enters linearly: L(D + e v) - L(D - e v) = 2 e <dL/dD, v>, up to the bf16 rounding (2^-9 rms each) of y's
    # 90 x 64 and of the scan's 90 x 128 values, which add as a random walk weighted by dy
    v = torch.randn(block.D.shape, generator=gen, device="cuda")
    e, out = 0.5, []
    with torch.no_grad():
        for s in (e, -e):
            block.D += s * v
            out.append(block.forward(x, r, cu)[0].float())
            block.D -= s * v
    num = float(((out[0] - out[1]) * dy.float()).sum() / (2 * e))
    got = float((block.D.grad * v).sum())
    noise = 2.0 ** -8 * (90 * 64) ** 0.5 * float(y.float().square().mean().sqrt()) / (2 * e) * 4
    assert abs(num - got) <= noise + 2.0 ** -7 * abs(got), (num, got, noise)
