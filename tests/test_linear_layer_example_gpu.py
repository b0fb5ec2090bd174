"""The linear-attention block of examples/ end to end: the operators one after the other, in training, over prompts, token by
token and in a graph."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_decoding_continues_the_prompt():
    from linear_attention_block import LinearAttentionBlock, decode_error
    # the same tokens through matrix products of other shapes: bf16 roundings (2^-8 of a value) of the norms, q, k, v, the
    # scores, the state and o differ here and there; a few of them, on values up to four rms
    assert decode_error(LinearAttentionBlock(width=128)) <= 8 * 4 * 2.0 ** -8
    assert decode_error(LinearAttentionBlock(width=128, heads=3, key_heads=3, turned=128, context=4.0)) <= 8 * 4 * 2.0 ** -8


def test_it_trains():
    from linear_attention_block import LinearAttentionBlock, train
    block = LinearAttentionBlock(width=128)
    losses = train(block, steps=3)
    assert all(x == x and abs(x) < 1e9 for x in losses)
    assert all(p.grad is not None and bool(torch.isfinite(p.grad).all()) for p in block.parameters())


def test_gradients_of_the_whole_block():
    from linear_attention_block import LinearAttentionBlock, _pack
    block = LinearAttentionBlock(width=64, seed=3)
    gen = torch.Generator("cuda").manual_seed(4)
    x, r, dy = (torch.randn((190, 64), generator=gen, device="cuda").bfloat16() for _ in range(3))
    cu = _pack([30, 160])
    y, _ = block.forward(x, r, cu)
    (y.float() * dy.float()).sum().backward()
    # along a weight w: (L(w + e v) - L(w - e v)) / 2 e = <dL/dw, v> up to e^2 of the function's bend (outputs of norms: about
    # the loss itself times e^2) and the bf16 roundings of y and of the five tensors before it (2^-8 rms each, adding as a
    # random walk weighted by dy)
    e = 0.05
    for name in ("w_q", "w_k", "norm_w", "out_w"):
        w = getattr(block, name)
        v = torch.randn(w.shape, generator=gen, device="cuda")
        out = []
        with torch.no_grad():
            for s in (e, -e):
                w += s * v
                out.append(block.forward(x, r, cu)[0].float())
                w -= s * v
        num = float(((out[0] - out[1]) * dy.float()).sum() / (2 * e))
        got = float((w.grad * v).sum())
        noise = 6 * 2.0 ** -8 * float(y.detach().float().norm()) / (2 * e) * 2 + 4 * e * e * float(y.detach().float().norm() * dy.float().norm()) / 64 ** 0.5
        assert abs(num - got) <= noise + 2.0 ** -5 * abs(got), (name, num, got, noise)


def test_decode_step_replayed_from_a_graph():
    from linear_attention_block import LinearAttentionBlock, _pack
    block = LinearAttentionBlock(width=128)
    gen = torch.Generator("cuda").manual_seed(0)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    _, _, cache = block.prompt(rn(200, 128), rn(200, 128), _pack([70, 1, 129]))
    tokens = [(rn(3, 128), rn(3, 128)) for _ in range(4)]
    slots = torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda")
    eager = {k: v.clone() for k, v in cache.items()}
    want = [block.step(x, r, eager, slots) for x, r in tokens]
    x, r = (torch.empty_like(t) for t in tokens[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    scratch = {k: v.clone() for k, v in cache.items()}
    with torch.cuda.stream(side):  # warm-up on a cache of its own
        block.step(x.zero_(), r.zero_(), scratch, slots)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, total = block.step(x, r, cache, slots)
    for (tx, tr), (wy, wt) in zip(tokens, want):
        x.copy_(tx)
        r.copy_(tr)
        g.replay()
        assert torch.equal(y, wy) and torch.equal(total, wt)
    assert all(torch.equal(cache[k], eager[k]) for k in cache)
    assert cache["length"].tolist() == [74, 1, 133]
