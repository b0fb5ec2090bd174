"""A linear-attention block with a decay for each head, from the library's operators: trained on packed documents, run
over prompts and decoded token by token.

    x -> (x + residual, layer norm) -> [q | k | v] = in projection -> q, k = rotated(norm of every head)
      -> o = linear attention(q, k, v, slope) -> norm of every head of o -> out projection

The projections are plain matrix products; everything between them is kda_layernorm_*, kda_rope_* and
kda_linattn_*.  Run it on a GB300 (after `python -m linear_attention_chunked_gb300.build`):

    python examples/linear_attention_block.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from linear_attention_chunked_gb300 import kda  # noqa: E402

D = 128  # head dim


class LayerNorm(torch.autograd.Function):
    """(layer norm of x + residual, x + residual); without a residual the layer norm of x"""

    @staticmethod
    def forward(ctx, x, residual, w, b):
        y, total, mean, rstd = kda.kda_layernorm_fwd(x, w, b, res=residual)
        ctx.save_for_backward(total, w, mean, rstd)
        ctx.residual = residual is not None
        return (y, total) if ctx.residual else y

    @staticmethod
    def backward(ctx, dy, dsum=None):
        total, w, mean, rstd = ctx.saved_tensors
        g = kda.kda_layernorm_bwd(total, w, mean, rstd, dy.contiguous(), dsum=None if dsum is None else dsum.contiguous())
        return g["dx"], g["dx"] if ctx.residual else None, g["dw"], g["db"]


class Attention(torch.autograd.Function):
    """Norm and rotation of the heads' queries and keys, and the linear attention, of the columns of one projection."""

    @staticmethod
    def forward(ctx, qkv, wq, wk, block, pos, cu_seqlens):
        q, k, v = block.split(qkv)
        qr, kr = kda.kda_rope_fwd(q, k, pos, block.freq, wq=wq, wk=wk, norm=True)
        o, _, ctx.states = kda.kda_linattn_fwd(qr, kr, v, block.slope, cu_seqlens, scale=D ** -0.5)
        ctx.save_for_backward(qkv, wq, wk, qr, kr, pos, cu_seqlens)
        ctx.block = block
        return o

    @staticmethod
    def backward(ctx, do):
        qkv, wq, wk, qr, kr, pos, cu_seqlens = ctx.saved_tensors
        q, k, v = ctx.block.split(qkv)
        g = kda.kda_linattn_bwd(qr, kr, v, ctx.block.slope, cu_seqlens, do.contiguous(), saved=ctx.states, scale=D ** -0.5,
                                want_dh0=False)
        r = kda.kda_rope_bwd(q, k, pos, ctx.block.freq, g["dq"], g["dk"], wq=wq, wk=wk, norm=True)
        dqkv = torch.cat([r["dq"].flatten(1), r["dk"].flatten(1), g["dv"].flatten(1)], 1)
        return dqkv, r["dwq"], r["dwk"], None, None, None


def positions(cu_seqlens, tokens):
    """Each token's place in its document."""
    at = torch.arange(tokens, device=cu_seqlens.device, dtype=torch.int32)
    return at - cu_seqlens[torch.searchsorted(cu_seqlens[1:].contiguous(), at, right=True)]


class LinearAttentionBlock:
    """width: the residual stream's; heads of values, key_heads of queries and keys (each shared by heads / key_heads)."""

    def __init__(self, width=256, heads=4, key_heads=2, turned=64, context=1.0, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)

        def randn(*shape):
            return torch.randn(shape, generator=gen, device="cuda")

        self.heads, self.key_heads = heads, key_heads
        half = lambda t: t.bfloat16().requires_grad_()  # noqa: E731
        full = lambda t: t.contiguous().requires_grad_()  # noqa: E731
        ones, zeros = torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")
        self.norm_w, self.norm_b = full(ones), full(zeros)
        self.w_in = half(randn(width, (2 * key_heads + heads) * D) / math.sqrt(width))
        self.w_q, self.w_k = full(torch.ones(D, device="cuda")), full(torch.ones(D, device="cuda"))
        self.out_w, self.out_b = full(torch.ones(D, device="cuda")), full(torch.zeros(D, device="cuda"))
        self.w_out = half(randn(heads * D, width) / math.sqrt(heads * D))
        # decays: a geometric row over the heads; the rotation stretched to `context` times a trained length
        self.slope = -torch.exp2(-8.0 * (torch.arange(heads, device="cuda") + 1) / heads)
        self.freq, _ = kda.kda_rope_frequencies(turned, scaling="linear" if context > 1 else "plain", factor=context)

    def parameters(self):
        return [v for v in vars(self).values() if torch.is_tensor(v) and v.requires_grad]

    def split(self, qkv):
        a, b = self.key_heads * D, 2 * self.key_heads * D
        return (qkv[:, :a].unflatten(1, (self.key_heads, D)), qkv[:, a:b].unflatten(1, (self.key_heads, D)),
                qkv[:, b:].unflatten(1, (self.heads, D)))

    def _out(self, o):
        return LayerNorm.apply(o.reshape(-1, D), None, self.out_w, self.out_b).view(o.shape[0], -1) @ self.w_out

    def forward(self, x, residual, cu_seqlens):
        """Training: the block over packed documents; returns (output, residual stream)."""
        normed, total = LayerNorm.apply(x, residual, self.norm_w, self.norm_b)
        pos = positions(cu_seqlens, x.shape[0])
        return self._out(Attention.apply(normed @ self.w_in, self.w_q, self.w_k, self, pos, cu_seqlens)), total

    @torch.no_grad()
    def prompt(self, x, residual, cu_seqlens):
        """Prompts: as forward, and the cache that single tokens continue from."""
        normed, total, _, _ = kda.kda_layernorm_fwd(x, self.norm_w, self.norm_b, res=residual)
        q, k, v = self.split(normed @ self.w_in)
        pos = positions(cu_seqlens, x.shape[0])
        kda.kda_rope_fwd(q, k, pos, self.freq, wq=self.w_q, wk=self.w_k, norm=True, q_out=q, k_out=k)
        o, state, _ = kda.kda_linattn_fwd(q, k, v, self.slope, cu_seqlens, scale=D ** -0.5, save=False)
        return self._out(o), total, {"state": state, "length": (cu_seqlens[1:] - cu_seqlens[:-1]).contiguous()}

    @torch.no_grad()
    def step(self, x, residual, cache, slots=None):
        """One token per sequence; the cache is updated in place.  slots: each row's place in the cache
        (a negative one marks an unused row)."""
        normed, total, _, _ = kda.kda_layernorm_fwd(x, self.norm_w, self.norm_b, res=residual)
        q, k, v = self.split(normed @ self.w_in)
        length = cache["length"]
        if slots is None:
            pos = length[:x.shape[0]].clone()
            length[:x.shape[0]] += 1
        else:
            at, used = slots.clamp(min=0).long(), (slots >= 0).int()
            pos = length[at] * used
            length.index_add_(0, at, used)
        kda.kda_rope_fwd(q, k, pos, self.freq, wq=self.w_q, wk=self.w_k, norm=True, q_out=q, k_out=k)
        o, _ = kda.kda_linattn_step(q, k, v, self.slope, cache["state"], scale=D ** -0.5, slots=slots)
        return self._out(o), total


def _pack(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


def decode_error(block, lens=(70, 1, 330), tokens=5, seed=1):
    """Largest difference, over the outputs' rms, between decoding each document's last tokens one by one and running
    them as part of the prompt."""
    gen = torch.Generator("cuda").manual_seed(seed)
    width = block.w_in.shape[0]
    docs = [torch.randn((n + tokens, width), generator=gen, device="cuda").bfloat16() for n in lens]
    rest = [torch.randn((n + tokens, width), generator=gen, device="cuda").bfloat16() for n in lens]
    whole, _, _ = block.prompt(torch.cat(docs), torch.cat(rest), _pack([n + tokens for n in lens]))
    _, _, cache = block.prompt(torch.cat([d[:n] for d, n in zip(docs, lens)]), torch.cat([r[:n] for r, n in zip(rest, lens)]), _pack(list(lens)))
    worst, ends = 0.0, [sum(n + tokens for n in lens[:i]) for i in range(len(lens))]
    for t in range(tokens):
        y, _ = block.step(torch.stack([d[n + t] for d, n in zip(docs, lens)]), torch.stack([r[n + t] for r, n in zip(rest, lens)]), cache)
        want = torch.stack([whole[e + n + t] for e, n in zip(ends, lens)])
        worst = max(worst, float((y.float() - want.float()).abs().max() / want.float().square().mean().sqrt()))
    return worst


def train(block, steps=60, lens=(120, 40, 296), rate=0.005, seed=2):
    """Fits the block to a fixed random target on one pack; returns the losses."""
    gen = torch.Generator("cuda").manual_seed(seed)
    T, width = sum(lens), block.w_in.shape[0]
    x, residual, target = (torch.randn((T, width), generator=gen, device="cuda").bfloat16() for _ in range(3))
    cu = _pack(list(lens))
    opt = torch.optim.Adam(block.parameters(), lr=rate)
    losses = []
    for _ in range(steps):
        y, _ = block.forward(x, residual, cu)
        loss = (y.float() - target.float()).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


if __name__ == "__main__":
    b = LinearAttentionBlock()
    print("decoded against prompt: largest difference %.2g of the outputs' rms" % decode_error(b))
    curve = train(b)
    print("loss %.3f -> %.3f in %d steps" % (curve[0], curve[-1], len(curve)))
