"""Refusals of the selective scan's, the conv serving forms' and the layer norm's entry points: bad
arguments are answered with a status (or, for tensors that do not fit the call, a ValueError)
before any CUDA call.  No GPU needed."""
import ctypes

import pytest
import torch

from linear_attention_chunked_gb300 import build, kda

Z, A, MIS, ODD = (ctypes.c_void_p(v) for v in (0, 4096, 4104, 4097))
BAD = kda.KDA_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kda.lib()


def _ssm(**kw):
    pr = kda.kda_ssm_problem(100, 2, 64, 16, 2, kda.KDA_DT_BF16, 1, 0, 0, 0, 0, 0, 256)
    for k, v in kw.items():
        setattr(pr, k, v)
    return pr


def _fwd(lib, pr, **at):
    args = [A] * 12  # u dt A B C D dt_bias z h0 y ht saved
    for k, v in at.items():
        args["u dt A B C D dt_bias z h0 y ht saved".split().index(k)] = v
    return lib.kda_ssm_fwd(ctypes.byref(pr), *args, at.get("ws", A), 16, Z)  # 16 bytes: never enough to run


@pytest.mark.parametrize("field,value,status", [
    ("T", -1, BAD), ("T", 2 ** 31 - 1, BAD), ("N", 0, BAD), ("N", 65536, BAD), ("C", 0, BAD), ("C", 63, BAD),
    ("S", 0, BAD), ("S", 65, kda.KDA_ERR_UNSUPPORTED), ("G", 0, BAD), ("G", 3, BAD), ("dtype", 3, BAD), ("dtype", -1, BAD),
    ("dt_softplus", 2, BAD), ("ld_u", 63, BAD), ("ld_dt", -64, BAD), ("ld_z", 1, BAD), ("ld_b", 31, BAD), ("ld_c", 16, BAD),
    ("cu_seqlens", None, BAD), ("cu_seqlens", 257, BAD),
])
def test_scan_problem(lib, field, value, status):
    pr = _ssm(**{field: value})
    assert lib.kda_ssm_workspace_size(ctypes.byref(pr), kda.KDA_OP_FWD, None, None) == status
    assert _fwd(lib, pr) == status
    assert lib.kda_ssm_bwd(ctypes.byref(pr), *([A] * 21), A, 16, Z) == status
    if field not in ("T", "cu_seqlens"):  # the step reads neither
        assert lib.kda_ssm_step(ctypes.byref(pr), *([A] * 8), Z, 4, A, A, A, Z, Z) == status


def test_scan_grid_limit(lib):
    pr = _ssm(T=2 ** 30, N=1, C=1 << 20, G=1)
    assert lib.kda_ssm_workspace_size(ctypes.byref(pr), kda.KDA_OP_FWD, None, None) == kda.KDA_ERR_UNSUPPORTED


def test_scan_pointers(lib):
    pr = _ssm()
    for name in ("u", "dt", "A", "B", "C", "y"):
        assert _fwd(lib, pr, **{name: Z}) == BAD, name
    for name in ("u", "dt", "B", "C", "z"):  # element alignment is enough: only the workspace is too small
        assert _fwd(lib, pr, **{name: ODD}) == BAD, name
        assert _fwd(lib, pr, **{name: ctypes.c_void_p(4098)}) == kda.KDA_ERR_WORKSPACE, name
    for name in ("A", "D", "dt_bias", "h0", "y", "ht", "saved"):
        assert _fwd(lib, pr, **{name: MIS}) == BAD, name
    for name in ("D", "dt_bias", "z", "h0", "ht", "saved"):
        assert _fwd(lib, pr, **{name: Z}) == kda.KDA_ERR_WORKSPACE, name
    names = "u dt A B C D dt_bias z h0 dy dht saved du ddt dA dB dC dD ddt_bias dz dh0".split()
    for name in names:
        args = [MIS if n == name else A for n in names]
        want = kda.KDA_ERR_WORKSPACE if name in ("u", "dt", "B", "C", "z") else BAD
        assert lib.kda_ssm_bwd(ctypes.byref(pr), *args, A, 16, Z) == want, name
        args = [Z if n == name else A for n in names]
        want = kda.KDA_ERR_WORKSPACE if name in ("D", "dt_bias", "h0", "dht", "saved", "dD", "ddt_bias", "dh0", "z") else BAD
        assert lib.kda_ssm_bwd(ctypes.byref(pr), *args, A, 16, Z) == want, name
    assert lib.kda_ssm_workspace_size(ctypes.byref(pr), kda.KDA_OP_WALK, None, None) == BAD


def test_scan_sizes_do_not_depend_on_types_or_strides(lib):
    a = kda.kda_ssm_workspace_size(1000, 3, 64, 16, 1, kda.KDA_OP_FWD)
    assert a == kda.kda_ssm_workspace_size(1000, 3, 64, 16, 1, kda.KDA_OP_FWD, dtype=torch.float32)
    chunks = -(-1000 // 64) + 3
    # four states per 64-token chunk in the saved set; a forward without one keeps the chunks' starts
    assert a[1] >= 4 * chunks * 64 * 16 * 4 and a[0] >= chunks * 64 * 16 * 4
    saved, replay = (kda.kda_ssm_workspace_size(1000, 3, 64, 16, 1, op)[0] for op in (kda.KDA_OP_BWD_SAVED, kda.KDA_OP_BWD_REPLAY))
    assert replay >= saved + 4 * chunks * 64 * 16 * 4  # the same states in the workspace


def test_step_arguments(lib):
    pr = _ssm()
    step = lambda slots, n, hin, hout, y, ws: lib.kda_ssm_step(ctypes.byref(pr), *([A] * 8), slots, n, hin, hout, y, ws, Z)  # noqa: E731
    assert step(Z, 1, A, A, A, Z) == BAD  # two rows, one state
    assert step(A, 0, A, A, A, Z) == BAD
    assert step(MIS, 0, A, A, A, Z) == BAD
    assert step(ODD, 2, A, A, A, Z) == BAD
    for i in range(3):
        args = [A, A, A]
        for bad in (Z, MIS):
            args[i] = bad
            assert step(Z, 2, *args, Z) == BAD
    assert step(Z, 2, A, A, A, MIS) == BAD
    assert lib.kda_ssm_step(None, *([A] * 8), Z, 4, A, A, A, Z, Z) == BAD


def test_conv_serving_arguments(lib):
    pr = kda.make_conv_problem(100, 2, 64)
    pr.cu_seqlens = 256
    ref = ctypes.byref(pr)
    for args in ((Z, Z, A), (MIS, Z, A), (A, MIS, A), (A, Z, Z), (A, Z, MIS)):
        assert lib.kda_conv_tail(ref, *args, Z) == BAD
    for args in ((Z, A, A), (A, Z, A), (A, A, MIS), (MIS, A, A)):
        assert lib.kda_conv_step(ref, *args, Z, 2, A, A, A, Z, Z) == BAD
    for args in ((Z, A, A), (A, Z, A), (A, A, Z), (MIS, A, A), (A, MIS, A), (A, A, MIS)):
        assert lib.kda_conv_step(ref, A, A, Z, Z, 2, *args, Z, Z) == BAD
    assert lib.kda_conv_step(ref, A, A, Z, Z, 1, A, A, A, Z, Z) == BAD
    assert lib.kda_conv_step(ref, A, A, Z, A, 0, A, A, A, Z, Z) == BAD
    assert lib.kda_conv_step(ref, A, A, Z, Z, 2, A, A, A, MIS, Z) == BAD
    for field, value in (("C", 12), ("N", 0), ("activation", 2), ("out_fp32", 5)):
        bad = kda.make_conv_problem(100, 2, 64)
        setattr(bad, field, value)
        assert lib.kda_conv_step(ctypes.byref(bad), A, A, Z, Z, 4, A, A, A, Z, Z) == BAD


def test_layernorm_arguments(lib):
    mk = lambda **kw: kda.kda_layernorm_problem(**dict(dict(T=4, C=64, dtype=kda.KDA_DT_BF16, eps=1e-5), **kw))  # noqa: E731
    for kw in (dict(T=-1), dict(C=0), dict(C=(1 << 24) + 1), dict(dtype=3), dict(eps=-1.0), dict(eps=float("nan"))):
        pr = mk(**kw)
        assert lib.kda_layernorm_workspace_size(ctypes.byref(pr), None) == BAD
        assert lib.kda_layernorm_fwd(ctypes.byref(pr), *([A] * 8), Z) == BAD
        assert lib.kda_layernorm_bwd(ctypes.byref(pr), *([A] * 10), 1 << 30, Z) == BAD
    pr = ctypes.byref(mk())
    names = "x res w b sum y mean rstd".split()
    for name in names:
        assert lib.kda_layernorm_fwd(pr, *[MIS if n == name else A for n in names], Z) == BAD, name
    for name in ("x", "y", "res"):  # (a sum without a residual)
        assert lib.kda_layernorm_fwd(pr, *[Z if n == name else A for n in names], Z) == BAD, name
    names = "x w mean rstd dy dsum dx dw db ws".split()
    for name in names:
        assert lib.kda_layernorm_bwd(pr, *[MIS if n == name else A for n in names], 1 << 30, Z) == BAD, name
    for name in ("x", "mean", "rstd", "dy", "dx", "ws"):
        assert lib.kda_layernorm_bwd(pr, *[Z if n == name else A for n in names], 1 << 30, Z) == BAD, name
    assert lib.kda_layernorm_bwd(pr, *([A] * 10), 16, Z) == kda.KDA_ERR_WORKSPACE


def test_tensors_that_do_not_fit_the_call():
    f, bf = torch.float32, torch.bfloat16
    T, C, S = 6, 16, 4
    a = dict(u=torch.zeros(T, C, dtype=bf), dt=torch.zeros(T, C, dtype=bf), A=torch.zeros(C, S), B=torch.zeros(T, 2, S, dtype=bf),
             C=torch.zeros(T, 2, S, dtype=bf), cu_seqlens=torch.tensor([0, T], dtype=torch.int32))
    for change, word in ((dict(u=a["u"].double()), "u is"), (dict(dt=a["dt"].float()), "dt is"), (dict(A=a["A"].to(bf)), "A is"),
                         (dict(A=torch.zeros(C + 1, S)), "A has shape"), (dict(C=a["C"][:, :1]), "C has shape"),
                         (dict(B=torch.zeros(T, S, 2, dtype=bf).transpose(1, 2)), "B has strides"),
                         (dict(u=torch.zeros(C, T, dtype=bf).t()), "u has strides"),
                         (dict(u=torch.zeros(1, C, dtype=bf).expand(T, C)), "u has strides"),
                         (dict(z=torch.zeros(T, C)), "z is"), (dict(D=torch.zeros(C - 1)), "D has shape"),
                         (dict(h0=torch.zeros(2, C, S)), "h0 has shape"), (dict(y=torch.zeros(T, C)), "y is"),
                         (dict(saved=torch.zeros(4)), "saved holds"), (dict(cu_seqlens=torch.tensor([0, T])), "cu_seqlens is")):
        with pytest.raises(ValueError, match=word):
            kda.kda_ssm_fwd(**{**a, "ws": torch.zeros(8), "ht": torch.zeros(1, C, S), "y": torch.zeros(T, C, dtype=bf), **change})
    with pytest.raises(ValueError, match="dy has shape"):
        kda.kda_ssm_bwd(**a, dy=a["u"][1:])
    with pytest.raises(ValueError, match="dht is"):
        kda.kda_ssm_bwd(**a, dy=a["u"], dht=torch.zeros(1, C, S, dtype=bf))
    s = {k: v for k, v in a.items() if k != "cu_seqlens"}
    with pytest.raises(ValueError, match="need as many states"):
        kda.kda_ssm_step(**s, h=torch.zeros(T - 1, C, S))
    with pytest.raises(ValueError, match="slots is"):
        kda.kda_ssm_step(**s, h=torch.zeros(T, C, S), slots=torch.zeros(T, dtype=torch.int64))
    with pytest.raises(ValueError, match="h has strides"):
        kda.kda_ssm_step(**s, h=torch.zeros(T, S, C).transpose(1, 2))
    x, w, win = torch.zeros(2, 8, dtype=bf), torch.zeros(8, 4), torch.zeros(2, 3, 8, dtype=bf)
    with pytest.raises(ValueError, match="win is"):
        kda.kda_conv_step(x, w, win.float())
    with pytest.raises(ValueError, match="w has shape"):
        kda.kda_conv_step(x, w.t(), win)
    with pytest.raises(ValueError, match="need as many states"):
        kda.kda_conv_step(x, w, win[:1])
    with pytest.raises(ValueError, match="halo has shape"):
        kda.kda_conv_tail(x, torch.tensor([0, 2], dtype=torch.int32), halo=win)
    with pytest.raises(ValueError, match="x has strides"):
        kda.kda_layernorm_fwd(torch.zeros(4, 6).t())
    with pytest.raises(ValueError, match="res is"):
        kda.kda_layernorm_fwd(torch.zeros(4, 6), res=torch.zeros(4, 6, dtype=bf))
    with pytest.raises(ValueError, match="needs a residual"):
        kda.kda_layernorm_fwd(torch.zeros(4, 6), sum=torch.zeros(4, 6), y=torch.zeros(4, 6))
    with pytest.raises(ValueError, match="w has shape"):
        kda.kda_layernorm_bwd(torch.zeros(4, 6, dtype=f), torch.zeros(4), torch.zeros(4), torch.zeros(4), torch.zeros(4, 6))
