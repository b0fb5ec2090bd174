"""The scan with decays of zero: A = -inf forgets a state at every token.  Its term of the gradient of dt, A times
a decay of 0, counts as 0, as for any large finite A; everything is finite, in the channels concerned and in the others."""
import pytest
import torch

from linear_attention_chunked_gb300 import kda
from oracle import ssm
from test_ssm_gpu import _close, _inputs, _np, _ref_args

pytestmark = pytest.mark.gpu


# the last channel, which the lanes past the group's channels repeat, and one inside; documents whose last
# chunk ends inside a run of tokens, and one that does not
@pytest.mark.parametrize("lens,C,S,G,dtype", [([70, 9, 64], 40, 16, 1, "fp32"), ([3], 24, 4, 2, "bf16"), ([130, 66], 37, 7, 1, "fp32"),
                                              ([65], 20, 64, 1, "bf16"), ([64, 128], 64, 16, 1, "fp32")])
def test_states_that_are_forgotten_at_once(lens, C, S, G, dtype):
    a, kw, dy, dht = _inputs(lens, C, S, G, dtype, 5, h0=True)
    gone = [C - 1, 3]
    a["A"][gone[0]] = -float("inf")
    a["A"][gone[1], S // 2] = -float("inf")
    ra, rk = _ref_args(a, kw)
    ra["A"][ra["A"] == -float("inf")] = -1e30
    y_ref, ht_ref = ssm.ssm_fwd(**ra, **rk)
    ref = ssm.ssm_bwd(**ra, dy=_np(dy), dht=_np(dht), **rk)
    y, ht, saved = kda.kda_ssm_fwd(**a, **kw)
    _close("y", y, y_ref)
    _close("ht", ht, ht_ref)
    for sv in (saved, None):
        got = kda.kda_ssm_bwd(**a, dy=dy, dht=dht, saved=sv, **kw)
        for k in got:
            _close(k, got[k], ref[k])
