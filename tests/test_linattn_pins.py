"""Pins of the FP64 oracle of the linear attention with a decay for each head (CPU)."""
import numpy as np

from oracle import linattn


def _case(T=9, H=2, Hk=1, d=3, cu=(0, 4, 4, 9), seed=0):
    r = np.random.default_rng(seed)
    n = len(cu) - 1
    return dict(q=r.normal(size=(T, Hk, d)), k=r.normal(size=(T, Hk, d)), v=r.normal(size=(T, H, d)), slope=-r.random(H),
                cu=list(cu)), dict(h0=r.normal(size=(n, H, d, d))), r


def test_two_tokens_by_hand():
    # one channel, lam = 1/2: S = 3*5 = 15 after token 0 from S = 4 -> 2 + 15 = 17, then 8.5 + 2*7 = 22.5
    one = lambda *x: np.array(x, float).reshape(-1, 1, 1)  # noqa: E731
    o, ht = linattn.linattn_fwd(one(10, 100), one(3, 2), one(5, 7), [np.log(0.5)], [0, 2], h0=one(4).reshape(1, 1, 1, 1), scale=0.1)
    assert np.allclose(o.ravel(), [17, 225]) and np.allclose(ht.ravel(), [22.5])
    # G_1 = dht + scale q dO = 1 + 0.1*100*2 = 21; G_0 = 10.5 + 0.1*10*3 = 13.5
    g = linattn.linattn_bwd(one(10, 100), one(3, 2), one(5, 7), [np.log(0.5)], [0, 2], one(3, 2), h0=one(4).reshape(1, 1, 1, 1),
                            dht=one(1).reshape(1, 1, 1, 1), scale=0.1)
    assert np.allclose(g["dk"].ravel(), [13.5 * 5, 21 * 7]) and np.allclose(g["dv"].ravel(), [13.5 * 3, 21 * 2])
    assert np.allclose(g["dq"].ravel(), [0.1 * 17 * 3, 0.1 * 22.5 * 2]) and np.allclose(g["dh0"].ravel(), [6.75])


def test_no_decay_is_a_running_sum_and_no_memory_a_token_alone():
    a, s, _ = _case()
    a["slope"] = np.zeros(2)
    o, _ = linattn.linattn_fwd(**a)
    for n in range(3):
        sl = slice(a["cu"][n], a["cu"][n + 1])
        P = np.tril(a["q"][sl, 0] @ a["k"][sl, 0].T)
        for h in range(2):
            assert np.allclose(o[sl, h], P @ a["v"][sl, h])
    a["slope"] = np.full(2, -np.inf)
    o, ht = linattn.linattn_fwd(**a, **s)
    assert np.allclose(o, (a["q"] * a["k"]).sum(-1, keepdims=True) * a["v"])
    assert np.allclose(ht[1], s["h0"][1])  # the empty document


def test_a_document_cut_in_two():
    a, s, r = _case(cu=(0, 9))
    o, ht = linattn.linattn_fwd(**a, **s)
    cut = lambda lo, hi: {**{k: a[k][lo:hi] for k in "qkv"}, "slope": a["slope"], "cu": [0, hi - lo]}  # noqa: E731
    o1, mid = linattn.linattn_fwd(**cut(0, 5), **s)
    o2, end = linattn.linattn_fwd(**cut(5, 9), h0=mid)
    assert np.allclose(np.concatenate([o1, o2]), o) and np.allclose(end, ht)
    dO, dht = r.normal(size=o.shape), r.normal(size=ht.shape)
    g = linattn.linattn_bwd(**a, dO=dO, dht=dht, **s)
    g2 = linattn.linattn_bwd(**cut(5, 9), dO=dO[5:], h0=mid, dht=dht)
    g1 = linattn.linattn_bwd(**cut(0, 5), dO=dO[:5], dht=g2["dh0"], **s)
    for k in ("dq", "dk", "dv"):
        assert np.allclose(np.concatenate([g1[k], g2[k]]), g[k])
    assert np.allclose(g1["dh0"], g["dh0"])


def test_gradients_by_central_differences():
    a, s, r = _case(H=4, Hk=2)
    dO, dht = r.normal(size=(9, 4, 3)), r.normal(size=(3, 4, 3, 3))
    g = linattn.linattn_bwd(**a, dO=dO, dht=dht, scale=0.7, **s)

    def loss(**kw):
        o, ht = linattn.linattn_fwd(**{**a, **s, **kw}, scale=0.7)
        return (o * dO).sum() + (ht * dht).sum()

    e = 1e-6
    for name, got in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("h0", "dh0")):
        x = s["h0"] if name == "h0" else a[name]
        d = r.normal(size=x.shape)
        assert abs((loss(**{name: x + e * d}) - loss(**{name: x - e * d})) / (2 * e) - (g[got] * d).sum()) < 1e-6
