"""Every parameter's gradient of the linear-attention block in examples/ against the same block in 64 bits."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

D = 128


def _block(p, block, x, residual, cu, head_eps=1e-6, norm_eps=1e-5):
    """The block's output from its definition, elementary operations in fp64."""
    def layer_norm(t, w, b):
        t = t - t.mean(-1, keepdim=True)
        return t / (t.square().mean(-1, keepdim=True) + norm_eps).sqrt() * w + b

    normed = layer_norm(x + residual, p["norm_w"], p["norm_b"])
    q, k, v = block.split(normed @ p["w_in"])
    freq, half, out = block.freq, block.freq.numel(), []
    pos = torch.cat([torch.arange(b - a) for a, b in zip(cu, cu[1:])]).cuda().double()
    cos, sin = (f(pos[:, None] * freq)[:, None] for f in (torch.cos, torch.sin))

    def turned(t, w):
        t = t / (t.square().mean(-1, keepdim=True) + head_eps).sqrt() * w
        a, b, rest = t[..., :half], t[..., half:2 * half], t[..., 2 * half:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1)

    share = block.heads // block.key_heads
    q, k = (turned(t, p[n]).repeat_interleave(share, 1).transpose(0, 1) for t, n in ((q, "w_q"), (k, "w_k")))
    v = v.transpose(0, 1)
    for a, b in zip(cu, cu[1:]):
        i = torch.arange(b - a, device="cuda").double()
        gap = i[:, None] - i
        decay = torch.where(gap >= 0, torch.exp(block.slope.double()[:, None, None] * gap.clamp(min=0)), 0.0)
        out.append(D ** -0.5 * ((q[:, a:b] @ k[:, a:b].transpose(1, 2)) * decay) @ v[:, a:b])
    o = torch.cat(out, 1).transpose(0, 1)
    return layer_norm(o, p["out_w"], p["out_b"]).flatten(1) @ p["w_out"]


@pytest.mark.parametrize("width,heads,key_heads,turned,lens", [(64, 4, 2, 64, [30, 160]), (192, 3, 1, 128, [1, 300, 129]), (128, 2, 2, 32, [257])])
def test_gradients_of_every_parameter(width, heads, key_heads, turned, lens):
    # On the way forward nine tensors are rounded to bf16 (the sum, its norm, the projection, q and k, scores, state, o, its norm, y)
    # and on the way back as many gradients; each is off by at most 2^-8 of itself, o and the gradients of its inputs by twice that
    # (see test_linattn_gpu.py).  A gradient is linear in each of them along with the others, and the two norms'
    # Jacobians at most double what passes them: fewer than 32 such parts, were they all of one sign.  That is an eighth
    # of the gradient's own length; a missing or reversed part of any weight's gradient is far above.  The output has the way
    # forward's alone: half as many.
    from linear_attention_block import LinearAttentionBlock, _pack
    block = LinearAttentionBlock(width=width, heads=heads, key_heads=key_heads, turned=turned, seed=width)
    gen = torch.Generator("cuda").manual_seed(width + 1)
    x, r, dy = (torch.randn((sum(lens), width), generator=gen, device="cuda").bfloat16() for _ in range(3))
    names = ("norm_w", "norm_b", "w_in", "w_q", "w_k", "out_w", "out_b", "w_out")
    with torch.no_grad():  # weights that are not all alike
        for n in ("norm_w", "norm_b", "w_q", "w_k", "out_w", "out_b"):
            w = getattr(block, n)
            w += 0.2 * torch.randn(w.shape, generator=gen, device="cuda")
    cu = _pack(lens)
    y, total = block.forward(x, r, cu)
    (y.float() * dy.float()).sum().backward()
    p = {n: getattr(block, n).detach().double().requires_grad_() for n in names}
    want = _block(p, block, x.double(), r.double(), cu.tolist())
    (want * dy.double()).sum().backward()
    assert len(block.parameters()) == len(names)
    assert float((y.double() - want).norm() / want.norm()) <= 2.0 ** -4
    for n in names:
        got, ref = getattr(block, n).grad.double(), p[n].grad
        rel = float((got - ref).norm() / ref.norm())
        assert rel <= 2.0 ** -3, (n, rel)
