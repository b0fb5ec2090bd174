"""Refusals of the linear attention's and the rotation's entry points: bad arguments are answered with a status
(or, for tensors that do not fit the call, a ValueError) before any CUDA call.  No GPU needed."""
import ctypes

import pytest
import torch

from linear_attention_chunked_gb300 import build, kda

Z, A, MIS, ODD = (ctypes.c_void_p(v) for v in (0, 4096, 4104, 4097))
BAD, UNS = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kda.lib()


def _lin(**kw):
    pr = kda.kda_linattn_problem(5000, 2, 8, 4, 128, kda.KDA_DT_BF16, 1.0, 0, 0, 0, 256)
    for k, v in kw.items():
        setattr(pr, k, v)
    return pr


FWD = "q k v slope h0 o ht saved".split()
BWD = "q k v slope h0 dO dht saved dq dk dv dh0".split()


def _fwd(lib, pr, ws=A, **at):  # 16 bytes: never enough to run
    return lib.kda_linattn_fwd(ctypes.byref(pr), *[at.get(n, A) for n in FWD], ws, 16, Z)


def _bwd(lib, pr, ws=A, **at):
    return lib.kda_linattn_bwd(ctypes.byref(pr), *[at.get(n, A) for n in BWD], ws, 16, Z)


@pytest.mark.parametrize("field,value,status", [
    ("T", -1, BAD), ("T", 2 ** 31 - 1, BAD), ("N", 0, BAD), ("N", 65536, BAD), ("H", 0, BAD), ("H", 65536, BAD), ("H", 6, BAD),
    ("Hk", 0, BAD), ("Hk", 3, BAD), ("Hk", 16, BAD), ("d", 64, UNS), ("d", 0, UNS), ("dtype", kda.KDA_DT_FP16, UNS),
    ("dtype", kda.KDA_DT_FP32, UNS), ("dtype", 3, BAD), ("ld_q", 511, BAD), ("ld_q", 516, BAD), ("ld_k", 504, BAD),
    ("ld_v", 1016, BAD), ("ld_v", -1024, BAD), ("cu_seqlens", None, BAD), ("cu_seqlens", 257, BAD),
])
def test_linattn_problem(lib, field, value, status):
    pr = _lin(**{field: value})
    assert lib.kda_linattn_workspace_size(ctypes.byref(pr), kda.KDA_OP_FWD, None, None) == status
    assert _fwd(lib, pr) == status and _bwd(lib, pr) == status
    if field not in ("T", "cu_seqlens"):  # the step reads neither
        assert lib.kda_linattn_step(ctypes.byref(pr), A, A, A, A, Z, 4, A, A, A, Z, Z) == status


def test_linattn_pointers(lib):
    pr = _lin()
    short = kda.KDA_ERR_WORKSPACE
    for n in FWD:
        assert _fwd(lib, pr, **{n: MIS}) == BAD, n
        assert _fwd(lib, pr, **{n: Z}) == (short if n in ("h0", "ht", "saved") else BAD), n
    for n in BWD:
        assert _bwd(lib, pr, **{n: MIS}) == BAD, n
        assert _bwd(lib, pr, **{n: Z}) == (short if n in ("h0", "dht", "saved", "dh0") else BAD), n
    for ws in (Z, MIS):
        assert _fwd(lib, pr, ws=ws) == BAD and _bwd(lib, pr, ws=ws) == BAD
    assert lib.kda_linattn_workspace_size(ctypes.byref(pr), kda.KDA_OP_WALK, None, None) == BAD
    assert lib.kda_linattn_workspace_size(None, kda.KDA_OP_FWD, None, None) == BAD
    assert lib.kda_linattn_workspace_size(ctypes.byref(_lin(N=65535, H=65535, Hk=1)), kda.KDA_OP_FWD, None, None) == UNS


def test_linattn_step_arguments(lib):
    pr = _lin()
    step = lambda slots, n, *p: lib.kda_linattn_step(ctypes.byref(pr), A, A, A, A, slots, n, *p, Z)  # noqa: E731
    assert step(Z, 1, A, A, A, Z) == BAD  # two rows, one state
    assert step(A, 0, A, A, A, Z) == BAD and step(ODD, 2, A, A, A, Z) == BAD and step(Z, 2, A, A, A, MIS) == BAD
    for i in range(3):
        for bad in (Z, MIS):
            p = [A, A, A]
            p[i] = bad
            assert step(Z, 2, *p, Z) == BAD
    for i in range(4):
        for bad in (Z, MIS):
            p = [A, A, A, A]
            p[i] = bad
            assert lib.kda_linattn_step(ctypes.byref(pr), *p, Z, 2, A, A, A, Z, Z) == BAD
    assert lib.kda_linattn_step(None, A, A, A, A, Z, 4, A, A, A, Z, Z) == BAD


def _rope(**kw):
    pr = kda.kda_rope_problem(10, 4, 2, 128, 64, kda.KDA_ROPE_HALF, 1, kda.KDA_DT_BF16, 1e-6, 1.0, 0, 0, 0, 0)
    for k, v in kw.items():
        setattr(pr, k, v)
    return pr


RF = "q k pos freq wq wk q_out k_out".split()
RB = "q k pos freq wq wk dq_out dk_out dq dk dwq dwk".split()


@pytest.mark.parametrize("field,value,status", [
    ("T", -1, BAD), ("T", 2 ** 31, BAD), ("Hq", -1, BAD), ("Hq", 65536, BAD), ("Hk", -1, BAD), ("D", 0, BAD), ("D", 127, BAD),
    ("D", 258, UNS), ("R", -2, BAD), ("R", 63, BAD), ("R", 130, BAD), ("layout", 2, BAD), ("norm", 2, BAD), ("dtype", 3, BAD),
    ("eps", -1.0, BAD), ("eps", float("nan"), BAD), ("ld_q", 511, BAD), ("ld_k", 255, BAD), ("ld_qo", -512, BAD), ("ld_ko", 1, BAD),
])
def test_rope_problem(lib, field, value, status):
    pr = _rope(**{field: value})
    assert lib.kda_rope_workspace_size(ctypes.byref(pr), None) == status
    assert lib.kda_rope_fwd(ctypes.byref(pr), *([A] * 8), Z) == status
    assert lib.kda_rope_bwd(ctypes.byref(pr), *([A] * 12), A, 16, Z) == status


def test_rope_pointers(lib):
    pr = ctypes.byref(_rope())
    assert lib.kda_rope_workspace_size(ctypes.byref(_rope(Hq=0, Hk=0)), None) == BAD
    for n in RF:
        assert lib.kda_rope_fwd(pr, *[ODD if m == n else A for m in RF], Z) == BAD, n
        if n not in ("wq", "wk"):
            assert lib.kda_rope_fwd(pr, *[Z if m == n else A for m in RF], Z) == BAD, n
    for n in RB:
        assert lib.kda_rope_bwd(pr, *[ODD if m == n else A for m in RB], A, 16, Z) == BAD, n
        want = kda.KDA_ERR_WORKSPACE if n in ("wq", "wk", "dwq", "dwk") else BAD
        assert lib.kda_rope_bwd(pr, *[Z if m == n else A for m in RB], A, 16, Z) == want, n
    assert lib.kda_rope_bwd(pr, *([A] * 12), Z, 0, Z) == BAD
    assert lib.kda_rope_bwd(pr, *([A] * 12), A, 16, Z) == kda.KDA_ERR_WORKSPACE


def test_tensors_that_do_not_fit_the_call():
    bf, i32 = torch.bfloat16, torch.int32
    T, H, Hk = 6, 4, 2
    a = dict(q=torch.zeros(T, Hk, 128, dtype=bf), k=torch.zeros(T, Hk, 128, dtype=bf), v=torch.zeros(T, H, 128, dtype=bf),
             slope=torch.zeros(H), cu_seqlens=torch.tensor([0, T], dtype=i32))
    wide = torch.zeros(T, 4 * 128 + 4, dtype=bf)
    for change, word in ((dict(v=a["v"].half()), "v is"), (dict(q=a["q"].float()), "q is"), (dict(k=a["k"][:, :1]), "k has shape"),
                         (dict(v=a["v"][:, :3]), "do not divide"), (dict(v=a["v"][..., :64]), "head dim"),
                         (dict(q=a["q"][0]), "expected \\[T, heads"), (dict(v=torch.zeros(H, T, 128, dtype=bf).transpose(0, 1)), "v has strides"),
                         (dict(v=wide[:, :512].unflatten(1, (4, 128))), "v is not aligned"),
                         (dict(slope=torch.zeros(Hk)), "slope has shape"), (dict(slope=torch.zeros(H, dtype=bf)), "slope is"),
                         (dict(cu_seqlens=torch.tensor([0, T])), "cu_seqlens is"), (dict(h0=torch.zeros(1, H, 128, 64)), "h0 has shape"),
                         (dict(o=torch.zeros(T, H, 128)), "o is"), (dict(ht=torch.zeros(2, H, 128, 128)), "ht has shape"),
                         (dict(saved=torch.zeros(4)), "saved holds")):
        with pytest.raises(ValueError, match=word):
            kda.kda_linattn_fwd(**{**a, **change})
    with pytest.raises(ValueError, match="CUDA device"):
        kda.kda_linattn_fwd(**a)
    for change, word in ((dict(dO=a["q"]), "dO has shape"), (dict(dht=torch.zeros(1, H, 128, 128, dtype=bf)), "dht is"),
                         (dict(saved=torch.zeros(4)), "saved holds")):
        with pytest.raises(ValueError, match=word):
            kda.kda_linattn_bwd(**{**a, "dO": a["v"], **change})
    s = {k: v for k, v in a.items() if k != "cu_seqlens"}
    for kw, word in ((dict(h=torch.zeros(T - 1, H, 128, 128)), "need as many states"), (dict(h=torch.zeros(T, H, 128, 64)), "h has shape"),
                     (dict(h=torch.zeros(T, H, 128, 128), slots=torch.zeros(T, dtype=torch.int64)), "slots is"),
                     (dict(h=torch.zeros(T, H, 128, 128), ws=torch.zeros(2)), "ws holds")):
        with pytest.raises(ValueError, match=word):
            kda.kda_linattn_step(**s, **kw)


def test_rope_tensors_that_do_not_fit_the_call():
    f = torch.ones(8, dtype=torch.float64)
    a = dict(q=torch.zeros(5, 3, 32), k=torch.zeros(5, 1, 32), pos=torch.zeros(5, dtype=torch.int32), freq=f)
    for change, word in ((dict(q=a["q"].double()), "q is"), (dict(k=a["k"].half()), "k is"), (dict(k=a["k"][:4]), "k has shape"),
                         (dict(k=torch.zeros(5, 1, 16)), "k has shape"), (dict(pos=a["pos"].long()), "pos is"),
                         (dict(pos=a["pos"][:4]), "pos has shape"), (dict(freq=f.float()), "freq is"),
                         (dict(freq=torch.ones(17, dtype=torch.float64)), "turn more channels"), (dict(wq=torch.ones(32)), "belong to the norm"),
                         (dict(wq=torch.ones(16), norm=True), "wq has shape"), (dict(wk=torch.ones(32).half(), norm=True), "wk is"),
                         (dict(q=torch.zeros(3, 5, 32).transpose(0, 1)), "q has strides"), (dict(q_out=torch.zeros(5, 3, 16)), "q_out has shape"),
                         (dict(k_out=torch.zeros(5, 1, 32).half()), "k_out is"), (dict(k=None, k_out=a["k"]), "needs a k"),
                         (dict(q=a["q"][0]), "must be")):
        with pytest.raises(ValueError, match=word):
            kda.kda_rope_fwd(**{**a, **change})
    for change, word in ((dict(dq_out=a["k"]), "dq_out has shape"), (dict(dk_out=a["k"].half()), "dk_out is"), (dict(k=None), "needs a k"),
                         (dict(ws=torch.zeros(2), wq=torch.ones(32), norm=True), None)):
        with pytest.raises((ValueError, kda.KdaError), match=word):
            kda.kda_rope_bwd(**{**a, "dq_out": a["q"], "dk_out": a["k"], **change})
