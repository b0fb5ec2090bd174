"""The scan's backward follows a saved set's plan only where that set was written for the call's sizes: any other
buffer is reported through the device status and leads to no access."""
import ctypes

import pytest
import torch

from linear_attention_chunked_gb300 import kda
from test_ssm_gpu import _inputs

pytestmark = pytest.mark.gpu


def _bwd(a, kw, dy, saved):
    """The gradients, pre-filled so that what the call leaves alone shows, and the call's status."""
    N, S = a["cu_seqlens"].numel() - 1, a["A"].shape[1]
    pr = kda._ssm_problem("kda_ssm_bwd", a["u"], a["dt"], a["A"], a["B"], a["C"], kw["z"], kw["D"], kw["dt_bias"], True, N, a["cu_seqlens"])
    ws = torch.full((kda.kda_ssm_workspace_size(pr.T, N, pr.C, S, pr.G, kda.KDA_OP_BWD_SAVED)[0],), 0x5a, dtype=torch.uint8, device="cuda")
    out = [torch.full_like(t, 7.0, memory_format=torch.contiguous_format)
           for t in (a["u"], a["dt"], a["A"], a["B"], a["C"], kw["D"], kw["dt_bias"], kw["z"], a["A"].expand(N, *a["A"].shape))]
    kda._call("kda_ssm_bwd", a["u"].device, ctypes.byref(pr), *(t.data_ptr() for t in (a["u"], a["dt"], a["A"], a["B"], a["C"])),
              kw["D"].data_ptr(), kw["dt_bias"].data_ptr(), kw["z"].data_ptr(), None, dy.data_ptr(), None, saved.data_ptr(),
              *(t.data_ptr() for t in out), ws.data_ptr(), ws.numel())
    return out, kda.kda_read_device_status(ws)


# the latency forms, and the throughput forms of every kernel
@pytest.mark.parametrize("lens,C", [([150, 0, 70], 40), ([2200, 1089, 700], 4096)])
def test_a_set_for_other_sizes_is_refused(lens, C):
    a, kw, dy, _ = _inputs(lens, C, 16, 1, "bf16", 1)
    size = kda.kda_ssm_workspace_size(sum(lens), len(lens), C, 16, 1, kda.KDA_OP_FWD)[1]
    sets = [torch.full((size,), v, dtype=torch.uint8, device="cuda") for v in (0, 1, 0xff)]  # buffers that no forward wrote
    for other, Co, S, G in ((lens + [500], C, 16, 1), (lens, C, 32, 1), (lens, 2 * C, 16, 1), (lens, C, 16, 2), ([n + 64 for n in lens], C, 16, 1)):
        oa, ok, _, _ = _inputs(other, Co, S, G, "bf16", 2)
        sets.append(kda.kda_ssm_fwd(**oa, **ok)[2])
    for i, saved in enumerate(sets):
        out, status = _bwd(a, kw, dy, saved)
        assert status == kda.KDA_ERR_DEVICE_CHECK, i
        assert all(bool((t == 7).all()) for t in out), i
    out, status = _bwd(a, kw, dy, kda.kda_ssm_fwd(**a, **kw)[2])
    want = kda.kda_ssm_bwd(**a, dy=dy, **kw)
    assert status == kda.KDA_OK
    for t, k in zip(out, ("du", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dz", "dh0")):
        assert torch.equal(t, want[k]), k
    # and the entry point itself
    ws = torch.empty(kda.kda_ssm_workspace_size(sum(lens), len(lens), C, 16, 1, kda.KDA_OP_BWD_SAVED)[0], dtype=torch.uint8, device="cuda")
    kda.kda_ssm_bwd(**a, dy=dy, saved=sets[3], ws=ws, **kw)
    assert kda.kda_read_device_status(ws) == kda.KDA_ERR_DEVICE_CHECK
