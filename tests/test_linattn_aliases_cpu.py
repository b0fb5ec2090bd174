"""Outputs of the linear attention that are inputs still being read are refused before any CUDA call.  No GPU needed."""
import ctypes

import pytest
import torch

from linear_attention_chunked_gb300 import build, kda

Z = ctypes.c_void_p(0)
BIG = 1 << 40  # more than any workspace here
FWD = "q k v slope h0 o ht saved".split()
BWD = "q k v slope h0 dO dht saved dq dk dv dh0".split()


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kda.lib()


@pytest.mark.parametrize("T,H", [(100, 4), (5000, 4), (5000, 64)])  # whole and cut documents alike
def test_outputs_that_are_inputs(lib, T, H):
    pr = kda.kda_linattn_problem(T, 2, H, H, 128, kda.KDA_DT_BF16, 1.0, 0, 0, 0, 256)

    def call(fn, names, **same):
        at = {n: 4096 * (i + 1) for i, n in enumerate(names)}  # (no CUDA call is reached: these are no addresses)
        at.update({a: at[b] for a, b in same.items()})
        return fn(ctypes.byref(pr), *[ctypes.c_void_p(at[n]) for n in names], ctypes.c_void_p(1 << 20), BIG, Z)

    assert call(lib.kda_linattn_fwd, FWD, ht="h0") == kda.KDA_ERR_INVALID_ARG
    for out, ins in (("dh0", ("h0", "dht")), *((d, ("q", "k", "v", "dO")) for d in ("dq", "dk", "dv"))):
        for i in ins:
            assert call(lib.kda_linattn_bwd, BWD, **{out: i}) == kda.KDA_ERR_INVALID_ARG, (out, i)


def test_state_in_place():
    bf = torch.bfloat16
    q, h = torch.zeros(6, 2, 128, dtype=bf), torch.zeros(1, 2, 128, 128)
    cu = torch.tensor([0, 6], dtype=torch.int32)
    with pytest.raises(ValueError, match="ht is h0"):
        kda.kda_linattn_fwd(q, q, q, torch.zeros(2), cu, h0=h, ht=h)
