"""Pins of the selective scan's FP64 oracle (CPU): closed forms, the pack's structure and central
finite differences of every gradient."""
import numpy as np
import pytest

from oracle import ssm


def _case(lens, C, S, G, seed, *, z=True, h0=True, D=True, bias=True):
    r = np.random.default_rng(seed)
    T, N = sum(lens), len(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    a = dict(u=r.normal(size=(T, C)), dt=r.normal(size=(T, C)), A=-np.exp(r.normal(size=(C, S))),
             B=r.normal(size=(T, G, S)), Cm=r.normal(size=(T, G, S)), cu_seqlens=cu)
    kw = dict(D=r.normal(size=C) if D else None, dt_bias=r.normal(size=C) if bias else None,
              z=r.normal(size=(T, C)) if z else None, h0=r.normal(size=(N, C, S)) if h0 else None)
    return a, kw


def test_constant_decay_is_a_geometric_sum():
    # delta = d and u = B = C = 1: h_t = d (1 + q + .. + q^t) with q = exp(-d a)
    T, d, a = 12, 0.3, 1.7
    one = np.ones((T, 1))
    y, ht = ssm.ssm_fwd(one, d * one, [[-a]], one[:, :, None], one[:, :, None], [0, T], softplus=False)
    q = np.exp(-d * a)
    want = d * (1 - q ** np.arange(1, T + 1)) / (1 - q)
    assert np.allclose(y[:, 0], want, rtol=1e-13) and np.allclose(ht[0, 0, 0], want[-1], rtol=1e-13)


def test_zero_decay_is_a_prefix_sum_within_each_document():
    a, _ = _case([5, 0, 3], 2, 1, 1, 0)
    a["A"] = np.zeros((2, 1))
    y, ht = ssm.ssm_fwd(**a, softplus=False)
    du = a["dt"] * a["u"] * a["B"][:, 0]
    for n, (s, e) in enumerate([(0, 5), (5, 5), (5, 8)]):
        assert np.allclose(y[s:e], a["Cm"][s:e, 0] * np.cumsum(du[s:e], 0))
        assert np.allclose(ht[n, :, 0], du[s:e].sum(0))


def test_pack_equals_its_documents_and_a_cut_document_hands_its_state_over():
    a, kw = _case([4, 7], 6, 3, 2, 1)
    y, ht = ssm.ssm_fwd(**a, **kw)
    for n, (s, e) in enumerate([(0, 4), (4, 11)]):
        part = {k: a[k][s:e] for k in ("u", "dt", "B", "Cm")}
        pk = dict(kw, z=kw["z"][s:e], h0=kw["h0"][n:n + 1])
        y1, h1 = ssm.ssm_fwd(**part, A=a["A"], cu_seqlens=[0, e - s], **pk)
        assert np.array_equal(y1, y[s:e]) and np.array_equal(h1[0], ht[n])
        m = s + 2
        cut = lambda lo, hi, h: ssm.ssm_fwd(**{k: a[k][lo:hi] for k in ("u", "dt", "B", "Cm")}, A=a["A"],  # noqa: E731
                                            cu_seqlens=[0, hi - lo], **dict(kw, z=kw["z"][lo:hi], h0=h))
        ya, ha = cut(s, m, kw["h0"][n:n + 1])
        yb, hb = cut(m, e, ha)
        assert np.array_equal(np.concatenate([ya, yb]), y[s:e]) and np.array_equal(hb[0], ht[n])


def test_groups_read_their_own_B_and_C():
    a, kw = _case([6], 4, 2, 2, 2, z=False)
    y, _ = ssm.ssm_fwd(**a, **kw)
    for g in range(2):
        ch = slice(2 * g, 2 * g + 2)
        y1, _ = ssm.ssm_fwd(a["u"][:, ch], a["dt"][:, ch], a["A"][ch], a["B"][:, g], a["Cm"][:, g], [0, 6],
                            D=kw["D"][ch], dt_bias=kw["dt_bias"][ch], h0=kw["h0"][:, ch])
        assert np.array_equal(y1, y[:, ch])


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("z", [True, False])
def test_gradients_by_central_differences(softplus, z):
    a, kw = _case([3, 0, 5], 4, 3, 2, 3, z=z)
    r = np.random.default_rng(9)
    dy, dht = r.normal(size=a["u"].shape), r.normal(size=kw["h0"].shape)
    grads = ssm.ssm_bwd(**a, dy=dy, dht=dht, softplus=softplus, **kw)

    def outputs(name, x):
        aa, kk = dict(a), dict(kw)
        (aa if name in aa else kk)[name] = x
        return ssm.ssm_fwd(**aa, softplus=softplus, **kk)

    names = dict(u="du", dt="ddt", A="dA", B="dB", Cm="dC", D="dD", dt_bias="ddt_bias", h0="dh0")
    if z:
        names["z"] = "dz"
    for name, g in names.items():
        x = a[name] if name in a else kw[name]
        direction = r.normal(size=x.shape)
        e = 1e-5
        hi, lo = outputs(name, x + e * direction), outputs(name, x - e * direction)
        # the outputs are subtracted before the loss is formed: a growing recurrence (negative steps
        # without softplus) makes the loss itself too large to difference
        num = (((hi[0] - lo[0]) * dy).sum() + ((hi[1] - lo[1]) * dht).sum()) / (2 * e)
        got = (grads[g] * direction).sum()
        # central differences: truncation ~ e^2, and each output's rounding over e
        rounding = sum(np.finfo(float).eps * (abs(p) * abs(q)).sum() / e for p, q in zip(hi, (dy, dht)))
        assert abs(num - got) <= 1e-7 * (1 + abs(got)) + rounding, (name, num, got)
