"""The device status of the single-token calls: that of the latest call, whatever the word held before."""
import pytest
import torch

from linear_attention_chunked_gb300 import kda

pytestmark = pytest.mark.gpu


def _steps():
    C, S, N = 40, 16, 3
    gen = torch.Generator("cuda").manual_seed(0)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    u, dt, B, Cm = rn(N, C).to(bf), rn(N, C).to(bf), rn(N, S).to(bf), rn(N, S).to(bf)
    A, h, w, win = -torch.exp(rn(C, S)), rn(N, C, S), rn(C, 4), rn(N, 3, C).to(bf)
    return {"scan": lambda slots, ws: kda.kda_ssm_step(u, dt, A, B, Cm, h, slots=slots, ws=ws),
            "conv": lambda slots, ws: kda.kda_conv_step(u, w, win, slots=slots, ws=ws)}


@pytest.mark.parametrize("op", ["scan", "conv"])
def test_status_is_the_latest_calls(op):
    step = _steps()[op]
    good, bad, unused = (torch.tensor(s, dtype=torch.int32, device="cuda") for s in ([2, 0, 1], [2, 3, 1], [2, -1, 1]))
    ws = torch.full((256,), 0x5a, dtype=torch.uint8, device="cuda")  # memory as an allocator hands it out
    for slots in (None, good, unused):
        ws.fill_(0x5a)
        step(slots, ws)
        assert kda.kda_read_device_status(ws) == kda.KDA_OK, slots
    step(bad, ws)
    assert kda.kda_read_device_status(ws) == kda.KDA_ERR_DEVICE_CHECK
    step(bad, ws)
    step(good, ws)  # the next call's own
    assert kda.kda_read_device_status(ws) == kda.KDA_OK
