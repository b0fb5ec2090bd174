"""The state-space block's serving and norm calls in captured graphs."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def test_decode_step_replayed_from_a_graph():
    from state_space_block import StateSpaceBlock
    block = StateSpaceBlock(width=128, channels=256)
    gen = torch.Generator("cuda").manual_seed(0)
    cu = torch.tensor([0, 70, 71, 200], dtype=torch.int32, device="cuda")
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    _, _, cache = block.prompt(rn(200, 128), rn(200, 128), cu)
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


FIRST_CALLS = """
import torch
from linear_attention_chunked_gb300 import kda
gen = torch.Generator("cuda").manual_seed(0)
rn = lambda *s: torch.randn(s, generator=gen, device="cuda")
bf = torch.bfloat16
def scan(T, C, S):
    return (rn(T, C).to(bf), rn(T, C).to(bf), -torch.exp(rn(C, S)), rn(T, S).to(bf), rn(T, S).to(bf),
            torch.tensor([0, T], dtype=torch.int32, device="cuda"))
kda.kda_ssm_fwd(*scan(70, 16, 16))  # sets the device up
x, dy, w = rn(700, 8192).to(bf), rn(700, 8192).to(bf), rn(8192)
short = scan(40, 512, 4)
u, dt, A, B, C, _ = scan(5, 64, 8)
h, win, taps = rn(5, 64, 8), rn(5, 3, 64).to(bf), rn(64, 4)
ws = torch.empty(256, dtype=torch.uint8, device="cuda")
def calls():
    y, _, mean, rstd = kda.kda_layernorm_fwd(x, w)
    g = kda.kda_layernorm_bwd(x, w, mean, rstd, dy)
    p, ht, _ = kda.kda_ssm_fwd(*short, save=False)
    s, h1 = kda.kda_ssm_step(u, dt, A, B, C, h, h_out=torch.empty_like(h), ws=ws)
    c, w1 = kda.kda_conv_step(u, taps, win, win_out=torch.empty_like(win), ws=ws)
    return [y, mean, rstd, g["dx"], g["dw"], g["db"], p, ht, s, h1, c, w1]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = calls()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, calls()))
print("equal")
"""


def test_shapes_first_met_inside_a_capture():
    # after a device's first call other shapes may be met first inside a capture: a process of its own
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("equal"), r.stderr[-2000:]
