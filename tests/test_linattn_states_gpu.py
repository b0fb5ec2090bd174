"""The linear attention's states over weak decays, held to what each path adds up; bounds in units of
2^-24 where nothing is summed."""
import pytest
import torch

from linear_attention_chunked_gb300 import kda
from test_linattn_gpu import _case

pytestmark = pytest.mark.gpu

SLOPES = [0.0, -1e-5, -1e-3, -2e-2]


@pytest.mark.parametrize("n,H,tokens", [(1000, 4, (999, 930, 896, 895, 700, 300, 0)), (960, 4, (767, 760, 600)), (5000, 4, (4999, 4700, 4608, 4600, 4300, 3000, 5)),
                                        (2500, 64, (2499, 2400, 2300, 1700, 0))])
def test_what_one_token_leaves_in_a_state(n, H, tokens):
    # One token's term alone: lambda^dist k v^T, all other values zero, so nothing is summed and each element is off by its own
    # roundings.  Units of 2^-24: a factor's exponential 4 and its argument |slope| dist, its product with the value 1, three
    # planes' products cut to 24 bits twice 2; then each chunk's factor and product 5.  Documents that are cut take
    # one more factor, and one a segment and one a chunk of the last segment instead: 40 in place of 16.  A token that weighs below
    # 1/64 may be rounded besides to two bf16 numbers: the first leaves at most 2^-8 of it, the second 2^-9 of that.
    scale = 0.25
    c = _case([n], H, H, False, slopes=SLOPES * (H // 4), strided=False)
    a, slope = (c["q"], c["k"]), c["slope"].double()
    for t in tokens:
        v, dO = torch.zeros_like(c["v"]), torch.zeros_like(c["dO"])
        v[t], dO[n - 1 - t] = c["v"][t], c["dO"][n - 1 - t]
        _, ht, _ = kda.kda_linattn_fwd(*a, v, c["slope"], c["cu"], scale=scale, save=False)
        g = kda.kda_linattn_bwd(*a, v, c["slope"], c["cu"], dO, scale=scale)
        b = n - 1 - t
        for name, got, dist, key, value, f in (("ht", ht, n - 1 - t, c["k"][t], c["v"][t], 1.0), ("dh0", g["dh0"], b + 1, c["q"][b], c["dO"][b], scale)):
            weight = torch.exp(slope * dist)[:, None, None]
            ref = f * weight * key.double()[:, :, None] * value.double()[:, None, :]
            units = (40 if n > 2048 and H < 64 else 16) + 5 * (-(-dist // 128)) + slope.abs()[:, None, None] * dist
            tol = ref.abs() * (units * 2.0 ** -24 + torch.where(weight > 1 / 64, 0.0, 2.0 ** -17)) + 2.0 ** -120
            err = (got[0].double() - ref).abs()
            assert bool((err <= tol).all()), (name, t, float((err / tol).max()))
