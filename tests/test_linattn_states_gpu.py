"""The linear attention's states over weak decays and over many documents, held to what each path adds up; bounds in units of
2^-24 where nothing is summed, else as in test_linattn_long_gpu.py."""
import numpy as np
import pytest
import torch

from linear_attention_chunked_gb300 import kda
from test_linattn_gpu import D, STATE, _case, _check, _run
from test_linattn_long_gpu import _check as _check_long
from test_linattn_long_gpu import _reference

pytestmark = pytest.mark.gpu

SLOPES = [0.0, -1e-5, -1e-3, -2e-2]


@pytest.mark.parametrize("H", [4, 64])
def test_weak_decays(H):
    # 64 heads: one walk over 71 chunks; its sum is rounded by the chunks that weigh before the first of them fades (1 / |slope|
    # tokens, at most all), a chunk's 24 additions and decay by STATE.  4 heads: 18 segments of at most 4 chunks, of which a
    # state's path adds up one segment's 4, walks at most 4 more, and takes 17 sums and factors (2^-22 for the factor, the
    # same one each time, and 2^-24).
    c = _case([9000], H, H, True, slopes=SLOPES * (H // 4))
    got = _run(c)
    _, _, states = _reference(c)
    for h in range(H):
        chunks = max(1.0, min(9000.0, 1 / max(-SLOPES[h % 4], 1e-9)) / 128)
        bound = STATE * chunks if H == 64 else STATE * min(chunks, 8) + 17 * 1.25 * 2.0 ** -22
        for n, ref in states.items():
            rel = float((got[n][:, h].double() - ref[:, h]).norm() / ref[:, h].norm())
            assert rel <= bound, (n, h, rel, bound)


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


@pytest.mark.parametrize("N", [1, 2, 31, 32, 33, 70])
def test_documents_around_a_warps_lanes(N):
    # whole documents: up to 32 are walked longest first
    lens = [int(x) for x in np.random.default_rng(N).integers(0, 2048 // N, N)]
    c = _case(lens, 2, 2, True)
    _check(c, _run(c))


def test_many_whole_documents_of_many_heads():
    lens = [40] * 32 + [0, 2300]
    c = _case(lens, 64, 64, True)
    _check_long(c, _run(c))
