"""Checks of the binding that keep a tensor the kernels could not read from reaching them: offsets of the conv's
window, workspaces and saved sets.  No GPU needed: what fits ends at the refusal of tensors on the CPU."""
import pytest
import torch

from linear_attention_chunked_gb300 import build, kda

bf = torch.bfloat16
FITS = "expected a CUDA device"


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return kda.lib()


@pytest.mark.parametrize("cu,word", [
    (torch.tensor([0, 2, 5]), "cu_seqlens is torch.int64"),
    (torch.tensor([0.0, 2.0, 5.0]), "cu_seqlens is torch.float32"),
    (torch.tensor([0, 9, 2, 9, 5, 9], dtype=torch.int32)[::2], "cu_seqlens has strides"),
    (torch.tensor([[0, 2, 5]], dtype=torch.int32), "cu_seqlens has shape"),
    (torch.empty(3, dtype=torch.int32, device="meta"), "cu_seqlens is on meta"),
    (torch.tensor([0, 2, 5], dtype=torch.int32), FITS),
])
def test_offsets_of_the_conv_window(cu, word):
    with pytest.raises(ValueError, match=word):
        kda.kda_conv_tail(torch.zeros(5, 16, dtype=bf), cu)
