"""Batches of single tokens so large that a block walks several groups of sequences: each row takes what it takes in a
small batch, bit for bit."""
import pytest
import torch

from linear_attention_chunked_gb300 import kda

pytestmark = pytest.mark.gpu


# one block of channels, and several; a count of sequences that leaves the last group and the last walk short
@pytest.mark.parametrize("N,C,S,dtype", [(16001, 64, 16, torch.bfloat16), (30003, 200, 4, torch.float32), (9001, 130, 12, torch.float16),
                                         (15002, 16, 64, torch.float32)])
def test_rows_of_a_large_batch(N, C, S, dtype):
    gen = torch.Generator("cuda").manual_seed(S)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    u, dt, z, B, Cm = (rn(N, k).to(dtype) for k in (C, C, C, S, S))
    A, D, bias, pool = -torch.exp(rn(C, S)), rn(C), rn(C), rn(N + 5, C, S)
    slots = torch.randperm(N + 5, generator=gen, device="cuda")[:N].to(torch.int32)
    slots[7] = -1
    slots[N - 1] = N + 5
    before, ws = pool.clone(), torch.empty(256, dtype=torch.uint8, device="cuda")
    y, _ = kda.kda_ssm_step(u, dt, A, B, Cm, pool, D=D, dt_bias=bias, z=z, slots=slots, ws=ws)
    assert kda.kda_read_device_status(ws) == kda.KDA_ERR_DEVICE_CHECK
    want = before.clone()
    for i in range(0, N, 500):
        r = slice(i, min(i + 500, N))
        yi, _ = kda.kda_ssm_step(u[r], dt[r], A, B[r], Cm[r], want, D=D, dt_bias=bias, z=z[r], slots=slots[r])
        assert torch.equal(yi, y[r])
    assert torch.equal(want, pool)
    touched = torch.zeros(N + 5, dtype=torch.bool, device="cuda")
    touched[slots[(slots >= 0) & (slots < N + 5)].long()] = True
    assert torch.equal(pool[~touched], before[~touched])
