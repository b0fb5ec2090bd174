"""Calls of the linear-attention layer's operators that their documentation allows and the other tests do not make."""
import ctypes

import pytest
import torch

from linear_attention_chunked_gb300 import kda
from test_linattn_gpu import D, ROW, STATE, _run
from test_linattn_gpu import _case as _lin_case
from test_rope_gpu import DT, _case

pytestmark = pytest.mark.gpu


def _rope_problem(T, Hq, Hk, C, R, dtype, inter, norm, s):
    return kda.kda_rope_problem(T, Hq, Hk, C, R, kda.KDA_ROPE_PAIRS if inter else kda.KDA_ROPE_HALF, norm, kda._DTYPES[DT[dtype]], 1e-6, s,
                                0, 0, 0, 0)


def _p(t):
    return None if t is None else t.data_ptr()


def _stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("shape", [(300, 5, 3, 128, 64), (70, 3, 2, 80, 52), (33, 9, 5, 34, 10), (65, 3, 3, 254, 254), (4000, 2, 1, 128, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("inter", [False, True])
def test_rotation_gradients_in_place(shape, dtype, inter):
    # dq and dk may be dq_out and dk_out where those are dense
    for norm in (1, 0):
        q, k, dq, dk, pos, f, s, (wq, wk) = _case(*shape, dtype, bool(norm), fused=False)
        want = kda.kda_rope_bwd(q, k, pos, f, dq, dk, wq=wq, wk=wk, norm=bool(norm), interleaved=inter, scale=s)
        pr = _rope_problem(*shape, dtype, inter, norm, s)
        ws = torch.empty(max(kda.kda_rope_workspace_size(shape[3]), 16), dtype=torch.uint8, device="cuda")
        dwq, dwk = (torch.empty(shape[3], device="cuda") for _ in range(2))
        st = kda.lib().kda_rope_bwd(ctypes.byref(pr), _p(q), _p(k), _p(pos), _p(f), _p(wq), _p(wk), _p(dq), _p(dk), _p(dq), _p(dk),
                                    _p(dwq) if norm else None, _p(dwk) if norm else None, _p(ws), ws.numel(), _stream())
        assert st == kda.KDA_OK
        assert torch.equal(dq, want["dq"]) and torch.equal(dk, want["dk"])
        assert not norm or (torch.equal(dwq, want["dwq"]) and torch.equal(dwk, want["dwk"]))


@pytest.mark.parametrize("C,R", [(128, 64), (34, 10)])
def test_rotation_of_keys_alone_and_weights_of_one_side(C, R):
    q, k, dq, dk, pos, f, s, (wq, wk) = _case(90, 4, 2, C, R, "bf16", True, fused=False)
    kw = dict(norm=True, scale=s)
    _, want = kda.kda_rope_fwd(q, k, pos, f, wq=wq, wk=wk, **kw)
    out = torch.empty_like(k)
    pr = _rope_problem(90, 0, 2, C, R, "bf16", False, 1, s)
    assert kda.lib().kda_rope_fwd(ctypes.byref(pr), None, _p(k), _p(pos), _p(f), None, _p(wk), None, _p(out), _stream()) == kda.KDA_OK
    assert torch.equal(out, want)
    g = kda.kda_rope_bwd(q, k, pos, f, dq, dk, wq=wq, wk=wk, **kw)
    ones = torch.ones(C, device="cuda")
    h = kda.kda_rope_bwd(q, k, pos, f, dq, dk, wk=wk, **kw)
    plain = kda.kda_rope_bwd(q, k, pos, f, dq, dk, wq=ones, wk=ones, **kw)
    none = kda.kda_rope_bwd(q, k, pos, f, dq, dk, **kw)
    assert set(h) == {"dq", "dk", "dwk"} and torch.equal(h["dk"], g["dk"]) and torch.equal(h["dwk"], g["dwk"])
    assert torch.equal(h["dq"], plain["dq"]) and set(none) == {"dq", "dk"}
    assert torch.equal(none["dq"], plain["dq"]) and torch.equal(none["dk"], plain["dk"])


def test_rotation_of_many_heads():
    # as many heads as a call takes: one token's rows are walked by every group of a block
    H, f = 65535, kda.kda_rope_frequencies(16)[0]
    x = torch.randn((3, H, 16), device="cuda")
    pos = torch.tensor([0, 7, -5], dtype=torch.int32, device="cuda")
    y, z = kda.kda_rope_fwd(x, x[:, :1], pos, f)
    part, _ = kda.kda_rope_fwd(x[:, 65000:], None, pos, f)
    assert torch.equal(y[:, 65000:], part) and torch.equal(z, y[:, :1])
    g = kda.kda_rope_bwd(x, None, -pos, f, x, None)  # the turn undone at -pos is the turn at pos
    assert float((g["dq"] - y).abs().max()) <= 16 * 2.0 ** -24 * float(x.abs().max()) * 2


def test_as_many_documents_as_a_call_takes():
    # 65535 documents of one token, and of none here and there: each is a single step
    N = 65535
    gen = torch.Generator("cuda").manual_seed(0)
    lens = torch.ones(N, dtype=torch.int64, device="cuda")
    lens[::7] = 0
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), lens.cumsum(0)]).int()
    T = int(cu[-1])
    q, k, v = (torch.randn((T, 1, D), generator=gen, device="cuda").bfloat16() for _ in range(3))
    slope, h0 = torch.tensor([-0.1], device="cuda"), torch.randn((N, 1, D, D), generator=gen, device="cuda")
    o, ht, _ = kda.kda_linattn_fwd(q, k, v, slope, cu, h0=h0, scale=D ** -0.5)
    assert torch.equal(ht[::7], h0[::7])
    full = lens.nonzero()[:, 0]
    slots = full.int()
    y, h = kda.kda_linattn_step(q, k, v, slope, h0, scale=D ** -0.5, slots=slots)
    assert float((ht[full] - h[full]).norm() / h[full].norm()) <= STATE
    assert float((o.float() - y.float()).norm() / y.float().norm()) <= 2 * ROW


def test_two_calls_at_once():
    # on two streams, each with its own workspace
    cases = [_lin_case([9000, 300], 4, 2, True, seed=1), _lin_case([700, 2000], 64, 64, True, seed=2)]
    want = [_run(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(_run(cases[i]))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        assert all(torch.equal(r[n], w[n]) for r in runs for n in w)


def test_queries_keys_and_values_of_one_tensor():
    # inputs may overlap each other
    c = _lin_case([400, 2300], 3, 3, True, strided=False)
    x = c["v"]
    a, b = _run(dict(c, q=x, k=x)), _run(dict(c, q=x.clone(), k=x.clone()))
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_a_very_long_document():
    # 300000 tokens of two heads: 586 segments; the states against the same walk in two calls, the first one's state handed on
    T, cut = 300000, 123000
    c = _lin_case([T], 2, 1, True, slopes=[-1e-3, -1e-5], strided=False)
    o, ht, _ = kda.kda_linattn_fwd(c["q"], c["k"], c["v"], c["slope"], c["cu"], h0=c["h0"], scale=c["scale"], save=False)
    h, parts = c["h0"], []
    for a, b in ((0, cut), (cut, T)):
        cu = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        y, h, _ = kda.kda_linattn_fwd(c["q"][a:b], c["k"][a:b], c["v"][a:b], c["slope"], cu, h0=h, scale=c["scale"], save=False)
        parts.append(y)
    # both sums carry some 600 segments, each factor and addition off by 1.25 2^-22 at most, and 8 chunks' additions
    assert float((h - ht).norm() / ht.norm()) <= 2 * (8 * STATE + 600 * 1.25 * 2.0 ** -22)
    y = torch.cat(parts)
    # scores and states are rounded at other places: each row's two errors of 2^-8 of its terms, twice
    rel = (y.float() - o.float()).norm(dim=-1) / o.float().norm(dim=-1).clamp(min=1e-3)
    assert float(rel.median()) <= 4 * ROW and float((y.float() - o.float()).norm() / o.float().norm()) <= 4 * ROW
