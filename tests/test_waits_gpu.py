"""Waits that run out, in part of a warp alone as well."""
import pytest
import torch

from linear_attention_chunked_gb300 import kda
from test_linattn_gpu import _case, _check, _run

pytestmark = pytest.mark.gpu


def test_a_warp_gives_up_together():
    # half of the lanes wait for what never comes, the others for what has come: all of them are told to give up (a device
    # check's status says that they were not), and the next call works
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        kda.kda_selftest_wait_timeout(ws, limit_us=1000)
        assert kda.kda_read_device_status(ws) == kda.KDA_ERR_TIMEOUT
    c = _case([300, 1, 90], 2, 2, True)
    _check(c, _run(c))
