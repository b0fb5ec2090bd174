"""A state-space block for packed documents, from the library's operators: trained, run over prompts and
decoded token by token.

    x -> (x + residual, layer norm) -> [u | z] = in projection -> u = silu(conv(u))
      -> [dt | B | C] = projection of u -> y = scan(u, dt, B, C) gated by z -> out projection

The projections are plain matrix products; everything between them is kda_layernorm_*, kda_conv_*
and kda_ssm_*.  Run it on a GB300 (after `python -m linear_attention_chunked_gb300.build`):

    python examples/state_space_block.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from linear_attention_chunked_gb300 import kda  # noqa: E402


class LayerNorm(torch.autograd.Function):
    """(layer norm of x + residual, x + residual)"""

    @staticmethod
    def forward(ctx, x, residual, w, b):
        y, total, mean, rstd = kda.kda_layernorm_fwd(x, w, b, res=residual)
        ctx.save_for_backward(total, w, mean, rstd)
        return y, total

    @staticmethod
    def backward(ctx, dy, dsum):
        total, w, mean, rstd = ctx.saved_tensors
        g = kda.kda_layernorm_bwd(total, w, mean, rstd, dy.contiguous(), dsum=dsum.contiguous())
        return g["dx"], g["dx"], g["dw"], g["db"]


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b, cu_seqlens):
        ctx.save_for_backward(x, w, b, cu_seqlens)
        return kda.kda_conv_fwd(x, w, cu_seqlens, bias=b)

    @staticmethod
    def backward(ctx, dy):
        x, w, b, cu_seqlens = ctx.saved_tensors
        g = kda.kda_conv_bwd(x, w, cu_seqlens, dy.contiguous(), bias=b)
        return g["dx"], g["dw"], g["dbias"], None


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, dt, A, B, C, D, dt_bias, z, cu_seqlens):
        y, _, ctx.states = kda.kda_ssm_fwd(u, dt, A, B, C, cu_seqlens, D=D, dt_bias=dt_bias, z=z)
        ctx.save_for_backward(u, dt, A, B, C, D, dt_bias, z, cu_seqlens)
        return y

    @staticmethod
    def backward(ctx, dy):
        u, dt, A, B, C, D, dt_bias, z, cu_seqlens = ctx.saved_tensors
        g = kda.kda_ssm_bwd(u, dt, A, B, C, cu_seqlens, dy.contiguous(), saved=ctx.states, D=D, dt_bias=dt_bias, z=z,
                            want_dh0=False)
        return g["du"], g["ddt"], g["dA"], g["dB"], g["dC"], g["dD"], g["ddt_bias"], g["dz"], None


class StateSpaceBlock:
    """width: the residual stream's; channels: the scan's (a multiple of 8); states per channel."""

    def __init__(self, width=256, channels=512, states=16, rank=16, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)

        def randn(*shape):
            return torch.randn(shape, generator=gen, device="cuda")

        self.channels, self.states, self.rank = channels, states, rank
        half = lambda t: t.bfloat16().requires_grad_()  # noqa: E731
        full = lambda t: t.contiguous().requires_grad_()  # noqa: E731
        self.norm_w, self.norm_b = full(torch.ones(width, device="cuda")), full(torch.zeros(width, device="cuda"))
        self.w_in = half(randn(width, 2 * channels) / math.sqrt(width))
        self.conv_w, self.conv_b = full(0.5 * randn(channels, 4)), full(torch.zeros(channels, device="cuda"))
        self.w_x = half(randn(channels, rank + 2 * states) / math.sqrt(channels))
        self.w_dt = half(randn(rank, channels) / math.sqrt(rank))
        # steps of 0.001 .. 0.1 at the start, as softplus(dt_bias)
        delta = torch.exp(torch.rand(channels, generator=gen, device="cuda") * math.log(100.0) + math.log(1e-3))
        self.dt_bias = full(delta + torch.log(-torch.expm1(-delta)))
        self.A_log = full(torch.log(torch.arange(1, states + 1, device="cuda", dtype=torch.float32)).expand(channels, states))
        self.D = full(torch.ones(channels, device="cuda"))
        self.w_out = half(randn(channels, width) / math.sqrt(channels))

    def parameters(self):
        return [v for v in vars(self).values() if torch.is_tensor(v)]

    def _inner(self, u):
        """dt, B, C of the conv's outputs; B and C stay columns of the projection."""
        p = u @ self.w_x
        r, s = self.rank, self.states
        return p[:, :r] @ self.w_dt, p[:, r:r + s], p[:, r + s:]

    def forward(self, x, residual, cu_seqlens):
        """Training: the block over packed documents; returns (output, residual stream)."""
        normed, total = LayerNorm.apply(x, residual, self.norm_w, self.norm_b)
        uz = normed @ self.w_in
        u = Conv.apply(uz[:, :self.channels].contiguous(), self.conv_w, self.conv_b, cu_seqlens)
        dt, B, C = self._inner(u)
        y = Scan.apply(u, dt, -torch.exp(self.A_log), B, C, self.D, self.dt_bias, uz[:, self.channels:], cu_seqlens)
        return y @ self.w_out, total

    @torch.no_grad()
    def prompt(self, x, residual, cu_seqlens):
        """Prompts: as forward, and the cache that single tokens continue from."""
        normed, total, _, _ = kda.kda_layernorm_fwd(x, self.norm_w, self.norm_b, res=residual)
        uz = normed @ self.w_in
        x_conv = uz[:, :self.channels].contiguous()
        u = kda.kda_conv_fwd(x_conv, self.conv_w, cu_seqlens, bias=self.conv_b)
        dt, B, C = self._inner(u)
        y, state, _ = kda.kda_ssm_fwd(u, dt, -torch.exp(self.A_log), B, C, cu_seqlens, D=self.D, dt_bias=self.dt_bias,
                                      z=uz[:, self.channels:], save=False)
        return y @ self.w_out, total, {"window": kda.kda_conv_tail(x_conv, cu_seqlens), "state": state}

    @torch.no_grad()
    def step(self, x, residual, cache, slots=None):
        """One token per sequence; the cache is updated in place.  slots: each row's place in the cache
        (a negative one marks an unused row)."""
        normed, total, _, _ = kda.kda_layernorm_fwd(x, self.norm_w, self.norm_b, res=residual)
        uz = normed @ self.w_in
        u, _ = kda.kda_conv_step(uz[:, :self.channels].contiguous(), self.conv_w, cache["window"], bias=self.conv_b, slots=slots)
        dt, B, C = self._inner(u)
        y, _ = kda.kda_ssm_step(u, dt, -torch.exp(self.A_log), B, C, cache["state"], D=self.D, dt_bias=self.dt_bias,
                                z=uz[:, self.channels:], slots=slots)
        return y @ self.w_out, total


def decode_error(block, lens=(70, 1, 130), tokens=5, seed=1):
    """Largest difference, over the outputs' rms, between decoding each document's last tokens one by one
    and running them as part of the prompt."""
    gen = torch.Generator("cuda").manual_seed(seed)
    width = block.w_in.shape[0]
    docs = [torch.randn((n + tokens, width), generator=gen, device="cuda").bfloat16() for n in lens]
    rest = [torch.randn((n + tokens, width), generator=gen, device="cuda").bfloat16() for n in lens]
    cu = lambda ns: torch.tensor([sum(ns[:i]) for i in range(len(ns) + 1)], dtype=torch.int32, device="cuda")  # noqa: E731
    whole, _, _ = block.prompt(torch.cat(docs), torch.cat(rest), cu([n + tokens for n in lens]))
    _, _, cache = block.prompt(torch.cat([d[:n] for d, n in zip(docs, lens)]), torch.cat([r[:n] for r, n in zip(rest, lens)]), cu(list(lens)))
    worst, ends = 0.0, [sum(n + tokens for n in lens[:i]) for i in range(len(lens))]
    for t in range(tokens):
        y, _ = block.step(torch.stack([d[n + t] for d, n in zip(docs, lens)]), torch.stack([r[n + t] for r, n in zip(rest, lens)]), cache)
        want = torch.stack([whole[e + n + t] for e, n in zip(ends, lens)])
        worst = max(worst, float((y.float() - want.float()).abs().max() / want.float().square().mean().sqrt()))
    return worst


def train(block, steps=60, lens=(120, 40, 96), rate=0.005, seed=2):
    """Fits the block to a fixed random target on one pack; returns the losses."""
    gen = torch.Generator("cuda").manual_seed(seed)
    T, width = sum(lens), block.w_in.shape[0]
    x, residual, target = (torch.randn((T, width), generator=gen, device="cuda").bfloat16() for _ in range(3))
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
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
    b = StateSpaceBlock()
    print("decoded against prompt: largest difference %.2g of the outputs' rms" % decode_error(b))
    curve = train(b)
    print("loss %.3f -> %.3f in %d steps" % (curve[0], curve[-1], len(curve)))
