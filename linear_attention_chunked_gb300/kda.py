"""ctypes binding of the C ABI in include/kda.h (argument marshalling only).

Every function here has the name of the C entry point it calls.  PyTorch supplies device memory
and the current stream; all arithmetic runs in the CUDA kernels of libkda_gb300.so.  If that
library has not been built this module raises -- there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

from . import build as _build

D = 128
CHUNK = 64

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_WORKSPACE = 0, 1, 2, 3
KDA_ERR_CUDA, KDA_ERR_TIMEOUT, KDA_ERR_DEVICE_CHECK, KDA_ERR_TOO_LARGE = 4, 5, 6, 7
KDA_STATIC_WS_BYTES = 64 << 20
KDA_GATE_G, KDA_GATE_RAW = 0, 1
KDA_OP_FWD, KDA_OP_BWD_SAVED, KDA_OP_BWD_REPLAY, KDA_OP_FRAGMENT, KDA_OP_WALK = 0, 1, 2, 3, 4
KDA_FRAG_FWD, KDA_FRAG_BWD = 0, 1
KDA_DT_BF16, KDA_DT_FP16, KDA_DT_FP32 = 0, 1, 2
_DTYPES = {torch.bfloat16: KDA_DT_BF16, torch.float16: KDA_DT_FP16, torch.float32: KDA_DT_FP32}
KDA_WALK_FP32, KDA_WALK_TF32, KDA_WALK_TF32_HILO, KDA_WALK_BF16X3, KDA_WALK_BF16X3_HW = 0, 1, 2, 3, 4
WALK_PRECISIONS = {"fp32": KDA_WALK_FP32, "tf32": KDA_WALK_TF32, "tf32_hilo": KDA_WALK_TF32_HILO,
                   "bf16x3": KDA_WALK_BF16X3, "bf16x3_hw": KDA_WALK_BF16X3_HW}
WALK_DEFAULT = KDA_WALK_BF16X3_HW  # the format the pages ship as the default walk

EXPORTS = ("kda_workspace_size", "kda_fwd", "kda_fwd_static_ws", "kda_bwd", "kda_fragment_summary",
           "kda_transfer_walk", "kda_conv_workspace_size", "kda_conv_fwd", "kda_conv_bwd",
           "kda_conv_tail", "kda_conv_step", "kda_ssm_workspace_size", "kda_ssm_fwd", "kda_ssm_bwd",
           "kda_ssm_step", "kda_layernorm_workspace_size", "kda_layernorm_fwd",
           "kda_layernorm_bwd", "kda_read_device_status", "kda_profile_enable",
           "kda_profile_collect", "kda_kernel_count", "kda_kernel_name", "kda_launch_counter",
           "kda_status_string")


class KdaError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: {kda_status_string(status)} (status {status})")


class kda_conv_problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("N", ctypes.c_int32), ("C", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("out_fp32", ctypes.c_int32),
                ("cu_seqlens", ctypes.c_void_p)]


class kda_problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("N", ctypes.c_int32), ("H", ctypes.c_int32),
                ("d", ctypes.c_int32), ("gate", ctypes.c_int32), ("l2norm", ctypes.c_int32),
                ("out_fp32", ctypes.c_int32), ("group_chunks", ctypes.c_int32),
                ("scale", ctypes.c_float), ("l2_eps", ctypes.c_float),
                ("cu_seqlens", ctypes.c_void_p)]


class kda_ssm_problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("N", ctypes.c_int32), ("C", ctypes.c_int32),
                ("S", ctypes.c_int32), ("G", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("dt_softplus", ctypes.c_int32), ("ld_u", ctypes.c_int64),
                ("ld_dt", ctypes.c_int64), ("ld_z", ctypes.c_int64), ("ld_b", ctypes.c_int64),
                ("ld_c", ctypes.c_int64), ("cu_seqlens", ctypes.c_void_p)]


class kda_layernorm_problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("C", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("eps", ctypes.c_float)]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def lib():
    """Loads libkda_gb300.so (raises if it was not built)."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not os.path.exists(path):
                raise RuntimeError(f"CUDA library {path} is missing: run "
                                   "`python -m linear_attention_chunked_gb300.build` first")
            L = ctypes.CDLL(path)
            P, I, S, V = ctypes.POINTER(kda_problem), ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
            L.kda_workspace_size.argtypes = [P, I, ctypes.POINTER(S), ctypes.POINTER(S)]
            L.kda_fwd.argtypes = [P] + [V] * 11 + [V, S, V]
            L.kda_fwd_static_ws.argtypes = [P] + [V] * 10 + [V]
            L.kda_bwd.argtypes = [P] + [V] * 19 + [V, S, V]
            L.kda_fragment_summary.argtypes = [P, I] + [V] * 10 + [V, S, V]
            L.kda_transfer_walk.argtypes = [ctypes.c_int32, V, ctypes.c_int32, ctypes.c_int32,
                                            V, V, V, I, I, V, V, V, V]
            CP = ctypes.POINTER(kda_conv_problem)
            L.kda_conv_workspace_size.argtypes = [CP, ctypes.POINTER(S)]
            L.kda_conv_fwd.argtypes = [CP, V, V, V, V, V, V]
            L.kda_conv_bwd.argtypes = [CP] + [V] * 9 + [V, S, V]
            L.kda_conv_tail.argtypes = [CP, V, V, V, V]
            L.kda_conv_step.argtypes = [CP, V, V, V, V, ctypes.c_int64, V, V, V, V, V]
            SP = ctypes.POINTER(kda_ssm_problem)
            L.kda_ssm_workspace_size.argtypes = [SP, I, ctypes.POINTER(S), ctypes.POINTER(S)]
            L.kda_ssm_fwd.argtypes = [SP] + [V] * 12 + [V, S, V]
            L.kda_ssm_bwd.argtypes = [SP] + [V] * 21 + [V, S, V]
            L.kda_ssm_step.argtypes = [SP] + [V] * 9 + [ctypes.c_int64] + [V] * 5
            NP = ctypes.POINTER(kda_layernorm_problem)
            L.kda_layernorm_workspace_size.argtypes = [NP, ctypes.POINTER(S)]
            L.kda_layernorm_fwd.argtypes = [NP] + [V] * 9
            L.kda_layernorm_bwd.argtypes = [NP] + [V] * 10 + [S, V]
            L.kda_read_device_status.argtypes = [V, ctypes.POINTER(I), V]
            L.kda_selftest_wait_timeout.argtypes = [V, ctypes.c_uint32, V]
            L.kda_profile_enable.argtypes = [I]
            L.kda_profile_collect.argtypes = [V, V]
            L.kda_kernel_count.argtypes = []
            L.kda_kernel_name.argtypes = [I]
            L.kda_kernel_name.restype = ctypes.c_char_p
            L.kda_launch_counter.argtypes = []
            L.kda_launch_counter.restype = ctypes.c_uint64
            L.kda_status_string.argtypes = [I]
            L.kda_status_string.restype = ctypes.c_char_p
            for name in ("kda_workspace_size", "kda_fwd", "kda_fwd_static_ws", "kda_bwd", "kda_fragment_summary",
                         "kda_transfer_walk", "kda_conv_workspace_size", "kda_conv_fwd",
                         "kda_conv_bwd", "kda_conv_tail", "kda_conv_step", "kda_ssm_workspace_size",
                         "kda_ssm_fwd", "kda_ssm_bwd", "kda_ssm_step",
                         "kda_layernorm_workspace_size", "kda_layernorm_fwd",
                         "kda_layernorm_bwd", "kda_read_device_status", "kda_selftest_wait_timeout",
                         "kda_profile_enable",
                         "kda_profile_collect", "kda_kernel_count"):
                getattr(L, name).restype = ctypes.c_int
            _lib = L
    return _lib


def kda_status_string(status: int) -> str:
    return lib().kda_status_string(int(status)).decode()


def _check(fn, status):
    if status != KDA_OK:
        raise KdaError(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _gate(gate):
    if gate in ("g", KDA_GATE_G):
        return KDA_GATE_G
    if gate in ("raw", KDA_GATE_RAW):
        return KDA_GATE_RAW
    raise ValueError(f"gate must be 'g' or 'raw', got {gate!r}")


def make_problem(T, N, H, cu_seqlens=None, *, gate="g", l2norm=False, scale=1.0, eps=1e-6,
                 d=D, out_dtype=torch.float32, group_chunks=0):
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("out_dtype must be torch.float32 or torch.bfloat16")
    return kda_problem(int(T), int(N), int(H), int(d), _gate(gate), int(bool(l2norm)),
                       int(out_dtype == torch.float32), int(group_chunks), float(scale), float(eps),
                       None if cu_seqlens is None else cu_seqlens.data_ptr())


def kda_workspace_size(T, N, H, op, **kw):
    """Returns (workspace bytes, saved-set bytes) of op for (T, N, H)."""
    pr = make_problem(T, N, H, **kw)
    if pr.cu_seqlens is None:
        pr.cu_seqlens = 16  # size queries never read it; any aligned non-null value passes
    ws, sv = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check("kda_workspace_size",
           lib().kda_workspace_size(ctypes.byref(pr), int(op), ctypes.byref(ws), ctypes.byref(sv)))
    return ws.value, sv.value


def _check_dtypes(tensors, dtype):
    """The library writes outputs in the dtype the problem declares: a caller's tensor must match."""
    for name, t in tensors.items():
        if t.dtype != dtype:
            raise ValueError(f"{name} is {t.dtype}, the call writes {dtype}")


def _empty_bytes(n, device):
    return torch.empty(max(int(n), 256), dtype=torch.uint8, device=device)


def _shape(q, cu_seqlens):
    T, H, d = q.shape
    return T, cu_seqlens.numel() - 1, H, d


def kda_fwd(q, k, v, beta, g_or_a, cu_seqlens, *, gate="g", A_log=None, dt_bias=None, h0=None,
            l2norm=False, scale=1.0, eps=1e-6, save=True, out_dtype=torch.float32, o=None, ht=None,
            saved=None, ws=None, group_chunks=0):
    """Forward.  Returns (o, ht, saved) -- saved is None when save=False.  group_chunks > 0 cuts
    documents into groups of that many chunks whose summaries are composed by the walk."""
    T, N, H, d = _shape(q, cu_seqlens)
    dev = q.device
    pr = make_problem(T, N, H, cu_seqlens, gate=gate, l2norm=l2norm, scale=scale, eps=eps, d=d,
                      out_dtype=out_dtype, group_chunks=group_chunks)
    ws_b, sv_b = kda_workspace_size(T, N, H, KDA_OP_FWD, group_chunks=group_chunks)
    if ws is None:
        ws = _empty_bytes(ws_b, dev)
    if save and saved is None:
        saved = _empty_bytes(sv_b, dev)
    if not save:
        saved = None
    if o is None:
        o = torch.empty(q.shape, dtype=out_dtype, device=dev)
    _check_dtypes({"o": o}, out_dtype)
    if ht is None:
        ht = torch.empty((N, H, d, d), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        st = lib().kda_fwd(ctypes.byref(pr), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g_or_a),
                           _ptr(A_log), _ptr(dt_bias), _ptr(h0), _ptr(o), _ptr(ht), _ptr(saved),
                           _ptr(ws), ws.numel(), _stream(dev))
    _check("kda_fwd", st)
    return o, ht, saved


def kda_fwd_static_ws(q, k, v, beta, g_or_a, cu_seqlens, *, gate="g", A_log=None, dt_bias=None,
                      h0=None, l2norm=False, scale=1.0, eps=1e-6, out_dtype=torch.float32,
                      o=None, ht=None):
    """Forward through the allocation-free entry point (its scratch is a static device array of
    the library).  Returns (o, ht).  The output tensors are the caller's (allocated here when not
    given, as any caller would); the library itself allocates nothing."""
    T, N, H, d = _shape(q, cu_seqlens)
    dev = q.device
    pr = make_problem(T, N, H, cu_seqlens, gate=gate, l2norm=l2norm, scale=scale, eps=eps, d=d,
                      out_dtype=out_dtype)
    if o is None:
        o = torch.empty(q.shape, dtype=out_dtype, device=dev)
    _check_dtypes({"o": o}, out_dtype)
    if ht is None:
        ht = torch.empty((N, H, d, d), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        st = lib().kda_fwd_static_ws(ctypes.byref(pr), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                     _ptr(g_or_a), _ptr(A_log), _ptr(dt_bias), _ptr(h0), _ptr(o),
                                     _ptr(ht), _stream(dev))
    _check("kda_fwd_static_ws", st)
    return o, ht


def kda_bwd(q, k, v, beta, g_or_a, cu_seqlens, dO, *, saved=None, gate="g", A_log=None,
            dt_bias=None, h0=None, dht=None, l2norm=False, scale=1.0, eps=1e-6, want_dh0=True,
            out_dtype=torch.float32, out=None, ws=None, group_chunks=0):
    """Backward (saved=None: checkpoint replay).  Returns a dict of gradients.  group_chunks must
    be the forward's."""
    T, N, H, d = _shape(q, cu_seqlens)
    dev = q.device
    g_ = _gate(gate)
    pr = make_problem(T, N, H, cu_seqlens, gate=gate, l2norm=l2norm, scale=scale, eps=eps, d=d,
                      out_dtype=out_dtype, group_chunks=group_chunks)
    op = KDA_OP_BWD_SAVED if saved is not None else KDA_OP_BWD_REPLAY
    ws_b, _ = kda_workspace_size(T, N, H, op, group_chunks=group_chunks)
    if ws is None:
        ws = _empty_bytes(ws_b, dev)
    if out is None:
        od = dict(dtype=out_dtype, device=dev)
        out = dict(dq=torch.empty(q.shape, **od), dk=torch.empty(k.shape, **od),
                   dv=torch.empty(v.shape, **od), dbeta=torch.empty(beta.shape, **od),
                   dg=torch.empty_like(g_or_a))
        if g_ == KDA_GATE_RAW:
            out["dA_log"] = torch.empty((H,), dtype=torch.float32, device=dev)
            out["ddt_bias"] = torch.empty((H, d), dtype=torch.float32, device=dev)
        if want_dh0:
            out["dh0"] = torch.empty((N, H, d, d), dtype=torch.float32, device=dev)
    _check_dtypes({k: out[k] for k in ("dq", "dk", "dv", "dbeta")}, out_dtype)
    _check_dtypes({k: out[k] for k in ("dg", "dA_log", "ddt_bias", "dh0") if out.get(k) is not None},
                  torch.float32)
    with torch.cuda.device(dev):
        st = lib().kda_bwd(ctypes.byref(pr), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g_or_a),
                           _ptr(A_log), _ptr(dt_bias), _ptr(h0), _ptr(dO), _ptr(dht), _ptr(saved),
                           _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dbeta"]),
                           _ptr(out["dg"]), _ptr(out.get("dA_log")), _ptr(out.get("ddt_bias")),
                           _ptr(out.get("dh0")), _ptr(ws), ws.numel(), _stream(dev))
    _check("kda_bwd", st)
    return out


def kda_fragment_summary(q, k, v, beta, g_or_a, frag_cu, *, mode=KDA_FRAG_FWD, dO=None,
                         gate="g", A_log=None, dt_bias=None, l2norm=False, scale=1.0, eps=1e-6,
                         M=None, B_or_C=None, ws=None):
    """mode KDA_FRAG_FWD -> (M, B); mode KDA_FRAG_BWD -> C.  Fragments = documents of frag_cu."""
    T, F, H, d = _shape(q, frag_cu)
    dev = q.device
    pr = make_problem(T, F, H, frag_cu, gate=gate, l2norm=l2norm, scale=scale, eps=eps, d=d)
    ws_b, _ = kda_workspace_size(T, F, H, KDA_OP_FRAGMENT)
    if ws is None:
        ws = _empty_bytes(ws_b, dev)
    if mode == KDA_FRAG_FWD and M is None:
        M = torch.empty((F, H, d, d), dtype=torch.float32, device=dev)
    if B_or_C is None:
        B_or_C = torch.empty((F, H, d, d), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        st = lib().kda_fragment_summary(ctypes.byref(pr), int(mode), _ptr(q), _ptr(k), _ptr(v),
                                        _ptr(beta), _ptr(g_or_a), _ptr(A_log), _ptr(dt_bias),
                                        _ptr(dO), _ptr(M), _ptr(B_or_C), _ptr(ws), ws.numel(),
                                        _stream(dev))
    _check("kda_fragment_summary", st)
    return (M, B_or_C) if mode == KDA_FRAG_FWD else B_or_C


def kda_transfer_walk(doc_frag, M, B, S0=None, *, reverse=False, precision=None, S_in=None,
                      S_final=None, ws=None):
    """Returns (S_in [F,H,d,d], S_final [N,H,d,d]).  precision: a KDA_WALK_* product format
    (default WALK_DEFAULT); ws (optional, >= 256 bytes) receives the device status."""
    F, H, d, _ = M.shape
    N = doc_frag.numel() - 1
    dev = M.device
    if precision is None:
        precision = WALK_DEFAULT
    if S_in is None:
        S_in = torch.empty_like(M)
    if S_final is None:
        S_final = torch.empty((N, H, d, d), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        st = lib().kda_transfer_walk(N, _ptr(doc_frag), F, H, _ptr(M), _ptr(B), _ptr(S0),
                                     int(bool(reverse)), int(precision), _ptr(S_in),
                                     _ptr(S_final), _ptr(ws), _stream(dev))
    _check("kda_transfer_walk", st)
    return S_in, S_final


def make_conv_problem(T, N, C, cu_seqlens=None, *, activation=True, out_dtype=torch.bfloat16):
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("out_dtype must be torch.float32 or torch.bfloat16")
    return kda_conv_problem(int(T), int(N), int(C), int(bool(activation)),
                            int(out_dtype == torch.float32),
                            None if cu_seqlens is None else cu_seqlens.data_ptr())


def kda_conv_workspace_size(T, N, C):
    pr = make_conv_problem(T, N, C)
    pr.cu_seqlens = 16  # size queries never read it
    ws = ctypes.c_size_t(0)
    _check("kda_conv_workspace_size", lib().kda_conv_workspace_size(ctypes.byref(pr), ctypes.byref(ws)))
    return ws.value


def _conv_shape(x, cu_seqlens):
    T = x.shape[0]
    C = x.numel() // max(T, 1) if T else int(torch.tensor(x.shape[1:]).prod())
    return T, cu_seqlens.numel() - 1, C


def kda_conv_fwd(x, w, cu_seqlens, *, bias=None, halo=None, activation=True,
                 out_dtype=torch.bfloat16, y=None):
    """Width-4 causal conv1d (+ SiLU) of x [T, ...] (bf16, C channels per token) with taps w
    [C, 4] fp32; halo [N, 3, C] bf16 or None.  Returns y with x's shape in out_dtype."""
    T, N, C = _conv_shape(x, cu_seqlens)
    pr = make_conv_problem(T, N, C, cu_seqlens, activation=activation, out_dtype=out_dtype)
    if y is None:
        y = torch.empty(x.shape, dtype=out_dtype, device=x.device)
    _check_dtypes({"y": y}, out_dtype)
    with torch.cuda.device(x.device):
        st = lib().kda_conv_fwd(ctypes.byref(pr), _ptr(x), _ptr(w), _ptr(bias), _ptr(halo), _ptr(y),
                                _stream(x.device))
    _check("kda_conv_fwd", st)
    return y


def kda_conv_bwd(x, w, cu_seqlens, dy, *, bias=None, halo=None, activation=True, want_dhalo=None,
                 ws=None):
    """Backward of L = sum(y * dy) (dy in y's dtype).  Returns dict dx (dy's dtype, x's shape),
    dw [C, 4], dbias [C] (when bias is given), dhalo [N, 3, C] (when halo is given)."""
    T, N, C = _conv_shape(x, cu_seqlens)
    out_dtype = dy.dtype
    pr = make_conv_problem(T, N, C, cu_seqlens, activation=activation, out_dtype=out_dtype)
    dev = x.device
    if ws is None:
        ws = _empty_bytes(kda_conv_workspace_size(T, N, C), dev)
    out = dict(dx=torch.empty(x.shape, dtype=out_dtype, device=dev),
               dw=torch.empty((C, 4), dtype=torch.float32, device=dev))
    if bias is not None:
        out["dbias"] = torch.empty((C,), dtype=torch.float32, device=dev)
    if halo is not None and want_dhalo is not False:
        out["dhalo"] = torch.empty((N, 3, C), dtype=out_dtype, device=dev)
    with torch.cuda.device(dev):
        st = lib().kda_conv_bwd(ctypes.byref(pr), _ptr(x), _ptr(w), _ptr(bias), _ptr(halo),
                                _ptr(dy), _ptr(out["dx"]), _ptr(out["dw"]), _ptr(out.get("dbias")),
                                _ptr(out.get("dhalo")), _ptr(ws), ws.numel(), _stream(dev))
    _check("kda_conv_bwd", st)
    return out


def _check_tensor(fn, name, t, shape, dtype, device, strided=False):
    """A tensor handed to the library has the shape, type and device the call works on and dense
    rows; `strided` ones (views of a projection) may have any row stride."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        return
    if t.dtype != dtype:
        raise ValueError(f"{fn}: {name} is {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{fn}: {name} is on {t.device}, expected {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        dims, st, inner = t.shape, t.stride(), 1
        rows = strided and t.numel() > 0
        for k in range(t.dim() - 1, 0, -1):  # the inner dimensions lie dense
            rows = rows and (dims[k] == 1 or st[k] == inner)
            inner *= dims[k]
        if not rows or (dims[0] > 1 and st[0] < inner):
            raise ValueError(f"{fn}: {name} has strides {t.stride()}, expected dense "
                             f"{'rows' if strided else 'storage'}")


def _check_bytes(fn, name, t, need, device):
    """A workspace or saved set (of any type) is dense, lies on the call's device and holds `need`
    bytes.  Returns the bytes it holds."""
    if t.device != device:
        raise ValueError(f"{fn}: {name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{fn}: {name} has strides {t.stride()}, expected dense storage")
    n = t.numel() * t.element_size()
    if n < need:
        raise ValueError(f"{fn}: {name} holds {n} bytes, needs {need}")
    return n


def _workspace(fn, ws, need, device):
    """The caller's workspace or a new one, and its bytes (the library refuses too few)."""
    if ws is None:
        ws = _empty_bytes(need, device)
        return ws, ws.numel()
    return ws, _check_bytes(fn, "ws", ws, 0, device)


def _row_stride(t):
    """The row stride of a tensor whose rows are dense (0, the library's dense, where it has at
    most one row)."""
    return 0 if t is None or t.shape[0] < 2 else t.stride(0)


def _slots(fn, slots, rows, pool, dev):
    if slots is None:
        if pool < rows:
            raise ValueError(f"{fn}: {rows} rows need as many states, the pool has {pool}")
    else:
        _check_tensor(fn, "slots", slots, (rows,), torch.int32, dev)


def _at(t):
    return None if t is None else t.data_ptr()


def _call(fn, dev, *args):
    """Calls an entry point on dev's current stream.  A decode step is a handful of such calls of a
    few microseconds each, so the device is only switched when it is not the current one."""
    if dev.type != "cuda":
        raise ValueError(f"{fn}: the tensors are on {dev}, expected a CUDA device")
    f = getattr(_lib or lib(), fn)
    if dev.index == torch.cuda.current_device():
        st = f(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        with torch.cuda.device(dev):
            st = f(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    if st != KDA_OK:
        raise KdaError(fn, st)


def kda_conv_tail(x, cu_seqlens, *, halo=None, tail=None):
    """The conv window that a prompt leaves: tail [N, 3, C] bf16, the three rows before each
    document's end (from halo [N, 3, C], or zero, where the document is shorter).  As for
    kda_conv_fwd, malformed offsets give unspecified rows."""
    fn = "kda_conv_tail"
    T, N, C = _conv_shape(x, cu_seqlens)
    dev = x.device
    if tail is None:
        tail = torch.empty((N, 3, C), dtype=torch.bfloat16, device=dev)
    _check_tensor(fn, "x", x, x.shape, torch.bfloat16, dev)
    _check_tensor(fn, "cu_seqlens", cu_seqlens, (N + 1,), torch.int32, dev)
    _check_tensor(fn, "halo", halo, (N, 3, C), torch.bfloat16, dev)
    _check_tensor(fn, "tail", tail, (N, 3, C), torch.bfloat16, dev)
    pr = make_conv_problem(T, N, C, cu_seqlens)
    _call(fn, dev, ctypes.byref(pr), x.data_ptr(), _at(halo), tail.data_ptr())
    return tail


def kda_conv_step(x, w, win, *, bias=None, activation=True, slots=None, out_dtype=torch.bfloat16,
                  win_out=None, y=None, ws=None):
    """The conv of one token per sequence: x [N, C] bf16, taps w [C, 4] fp32, windows win
    [n_slots, 3, C] bf16 (row n's is win[slots[n]], win[n] without slots).  Returns (y [N, C] in
    out_dtype, win_out); win_out defaults to win, updated in place.  A negative slot marks an
    unused row; ws (optional, >= 256 bytes) receives the device status of this call."""
    fn = "kda_conv_step"
    N, C = x.shape
    dev = x.device
    if win_out is None:
        win_out = win
    if y is None:
        y = torch.empty((N, C), dtype=out_dtype, device=dev)
    else:
        _check_tensor(fn, "y", y, (N, C), out_dtype, dev)
    _check_tensor(fn, "x", x, (N, C), torch.bfloat16, dev)
    _check_tensor(fn, "w", w, (C, 4), torch.float32, dev)
    _check_tensor(fn, "bias", bias, (C,), torch.float32, dev)
    _check_tensor(fn, "win", win, (win.shape[0], 3, C), torch.bfloat16, dev)
    if win_out is not win:
        _check_tensor(fn, "win_out", win_out, win.shape, torch.bfloat16, dev)
    _slots(fn, slots, N, win.shape[0], dev)
    if ws is not None:
        _check_bytes(fn, "ws", ws, 256, dev)
    pr = make_conv_problem(N, N, C, activation=activation, out_dtype=out_dtype)
    _call(fn, dev, ctypes.byref(pr), x.data_ptr(), w.data_ptr(), _at(bias), _at(slots), win.shape[0],
          win.data_ptr(), win_out.data_ptr(), y.data_ptr(), _at(ws))
    return y, win_out


def _ssm_problem(fn, u, dt, A, B, C, z, D, dt_bias, softplus, N, cu_seqlens):
    """Checks the scan's inputs and describes the call: B, C [T, G, S] or [T, S] (one group)."""
    T, ch = u.shape
    S, dev, dtype = A.shape[-1], u.device, u.dtype
    G = B.shape[1] if B.dim() == 3 else 1
    if dtype not in _DTYPES:
        raise ValueError(f"{fn}: u is {dtype}, expected one of bfloat16, float16, float32")
    _check_tensor(fn, "u", u, (T, ch), dtype, dev, True)
    _check_tensor(fn, "dt", dt, (T, ch), dtype, dev, True)
    _check_tensor(fn, "z", z, (T, ch), dtype, dev, True)
    bc = (T, G, S) if B.dim() == 3 else (T, S)
    _check_tensor(fn, "B", B, bc, dtype, dev, True)
    _check_tensor(fn, "C", C, bc, dtype, dev, True)
    _check_tensor(fn, "A", A, (ch, S), torch.float32, dev)
    _check_tensor(fn, "D", D, (ch,), torch.float32, dev)
    _check_tensor(fn, "dt_bias", dt_bias, (ch,), torch.float32, dev)
    if cu_seqlens is not None:
        _check_tensor(fn, "cu_seqlens", cu_seqlens, (N + 1,), torch.int32, dev)
    return kda_ssm_problem(T, N, ch, S, G, _DTYPES[dtype], int(bool(softplus)), _row_stride(u),
                           _row_stride(dt), _row_stride(z), _row_stride(B), _row_stride(C),
                           None if cu_seqlens is None else cu_seqlens.data_ptr())


@functools.lru_cache(maxsize=256)  # the sizes are a function of these numbers alone
def _ssm_sizes(T, N, C, S, G, op):
    pr = kda_ssm_problem(T, N, C, S, G, KDA_DT_BF16, 1, 0, 0, 0, 0, 0, 16)  # cu_seqlens is not read
    ws, sv = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check("kda_ssm_workspace_size",
           lib().kda_ssm_workspace_size(ctypes.byref(pr), int(op), ctypes.byref(ws), ctypes.byref(sv)))
    return ws.value, sv.value


def kda_ssm_workspace_size(T, N, C, S, G, op, *, dtype=torch.bfloat16):
    """Returns (workspace bytes, saved-set bytes) of the scan's op (whatever its type)."""
    if dtype not in _DTYPES:
        raise ValueError(f"kda_ssm_workspace_size: dtype is {dtype}, expected one of bfloat16, float16, float32")
    return _ssm_sizes(T, N, C, S, G, op)


def kda_ssm_fwd(u, dt, A, B, C, cu_seqlens, *, D=None, dt_bias=None, z=None, h0=None,
                softplus=True, save=True, y=None, ht=None, saved=None, ws=None):
    """Selective state-space scan of packed documents: u, dt, z [T, ch], B, C [T, G, S] (or [T, S])
    of one type (bf16, fp16, fp32; views with a row stride are taken as they are), A [ch, S], D,
    dt_bias [ch], h0 [N, ch, S] fp32.  Returns (y [T, ch], ht [N, ch, S], saved) -- saved is None
    when save=False."""
    fn = "kda_ssm_fwd"
    N, dev = cu_seqlens.numel() - 1, u.device
    pr = _ssm_problem(fn, u, dt, A, B, C, z, D, dt_bias, softplus, N, cu_seqlens)
    ws_b, sv_b = _ssm_sizes(pr.T, N, pr.C, pr.S, pr.G, KDA_OP_FWD)
    state = (N, pr.C, pr.S)
    ws, ws_n = _workspace(fn, ws, ws_b, dev)
    if not save:
        saved = None
    elif saved is None:
        saved = _empty_bytes(sv_b, dev)
    else:
        _check_bytes(fn, "saved", saved, sv_b, dev)
    if y is None:  # dense rows, whatever u's strides are
        y = torch.empty_like(u, memory_format=torch.contiguous_format)
    else:
        _check_tensor(fn, "y", y, u.shape, u.dtype, dev)
    if ht is None:
        ht = torch.empty(state, dtype=torch.float32, device=dev)
    else:
        _check_tensor(fn, "ht", ht, state, torch.float32, dev)
    _check_tensor(fn, "h0", h0, state, torch.float32, dev)
    _call(fn, dev, ctypes.byref(pr), u.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(),
          _at(D), _at(dt_bias), _at(z), _at(h0), y.data_ptr(), ht.data_ptr(), _at(saved), ws.data_ptr(), ws_n)
    return y, ht, saved


def kda_ssm_bwd(u, dt, A, B, C, cu_seqlens, dy, *, saved=None, D=None, dt_bias=None, z=None,
                h0=None, dht=None, softplus=True, want_dh0=True, ws=None):
    """Backward of the scan for L = sum(y * dy) + sum(ht * dht) (saved=None: the states are
    recomputed).  Returns a dict: du, ddt, dB, dC and (with z) dz in the inputs' type, dA and, for
    what was given, dD, ddt_bias fp32, and dh0 fp32 when wanted."""
    fn = "kda_ssm_bwd"
    N, dev, dtype = cu_seqlens.numel() - 1, u.device, u.dtype
    pr = _ssm_problem(fn, u, dt, A, B, C, z, D, dt_bias, softplus, N, cu_seqlens)
    state = (N, pr.C, pr.S)
    _check_tensor(fn, "dy", dy, u.shape, dtype, dev)
    _check_tensor(fn, "h0", h0, state, torch.float32, dev)
    _check_tensor(fn, "dht", dht, state, torch.float32, dev)
    ws_b, sv_b = _ssm_sizes(pr.T, N, pr.C, pr.S, pr.G, KDA_OP_BWD_REPLAY if saved is None else KDA_OP_BWD_SAVED)
    if saved is not None:
        _check_bytes(fn, "saved", saved, sv_b, dev)
    ws, ws_n = _workspace(fn, ws, ws_b, dev)
    # (like dy: dense rows whatever the inputs' strides are)
    out = dict(du=torch.empty_like(dy), ddt=torch.empty_like(dy), dA=torch.empty_like(A),
               dB=torch.empty(B.shape, dtype=dtype, device=dev),
               dC=torch.empty(B.shape, dtype=dtype, device=dev))
    if D is not None:
        out["dD"] = torch.empty_like(D)
    if dt_bias is not None:
        out["ddt_bias"] = torch.empty_like(dt_bias)
    if z is not None:
        out["dz"] = torch.empty_like(dy)
    if want_dh0:
        out["dh0"] = torch.empty(state, dtype=torch.float32, device=dev)
    _call(fn, dev, ctypes.byref(pr), u.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(),
          _at(D), _at(dt_bias), _at(z), _at(h0), dy.data_ptr(), _at(dht), _at(saved),
          *(_at(out.get(k)) for k in ("du", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dz", "dh0")),
          ws.data_ptr(), ws_n)
    return out


def kda_ssm_step(u, dt, A, B, C, h, *, D=None, dt_bias=None, z=None, softplus=True, slots=None,
                 h_out=None, y=None, ws=None):
    """The scan of one token per sequence: rows are sequences, h [n_slots, ch, S] fp32 the states
    (row n's is h[slots[n]], h[n] without slots).  Returns (y, h_out); h_out defaults to h, updated
    in place.  A negative slot marks an unused row; ws (optional, >= 256 bytes) receives the
    device status of this call."""
    fn = "kda_ssm_step"
    N, dev = u.shape[0], u.device
    pr = _ssm_problem(fn, u, dt, A, B, C, z, D, dt_bias, softplus, N, None)
    if h_out is None:
        h_out = h
    else:
        _check_tensor(fn, "h_out", h_out, h.shape, torch.float32, dev)
    if y is None:  # dense rows, whatever u's strides are
        y = torch.empty_like(u, memory_format=torch.contiguous_format)
    else:
        _check_tensor(fn, "y", y, u.shape, u.dtype, dev)
    _check_tensor(fn, "h", h, (h.shape[0], pr.C, pr.S), torch.float32, dev)
    _slots(fn, slots, N, h.shape[0], dev)
    if ws is not None:
        _check_bytes(fn, "ws", ws, 256, dev)
    _call(fn, dev, ctypes.byref(pr), u.data_ptr(), dt.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(),
          _at(D), _at(dt_bias), _at(z), _at(slots), h.shape[0], h.data_ptr(), h_out.data_ptr(),
          y.data_ptr(), _at(ws))
    return y, h_out


def _layernorm_problem(fn, x, eps):
    if x.dtype not in _DTYPES:
        raise ValueError(f"{fn}: x is {x.dtype}, expected one of bfloat16, float16, float32")
    _check_tensor(fn, "x", x, x.shape, x.dtype, x.device)
    C = x.shape[-1]
    return kda_layernorm_problem(x.numel() // max(C, 1), C, _DTYPES[x.dtype], float(eps))


@functools.lru_cache(maxsize=256)  # a function of these numbers alone
def kda_layernorm_workspace_size(T, C, *, dtype=torch.bfloat16):
    if dtype not in _DTYPES:
        raise ValueError(f"kda_layernorm_workspace_size: dtype is {dtype}, expected one of bfloat16, float16, float32")
    pr = kda_layernorm_problem(int(T), int(C), _DTYPES[dtype], 0.0)
    ws = ctypes.c_size_t(0)
    _check("kda_layernorm_workspace_size",
           lib().kda_layernorm_workspace_size(ctypes.byref(pr), ctypes.byref(ws)))
    return ws.value


def kda_layernorm_fwd(x, w=None, b=None, *, res=None, eps=1e-5, y=None, sum=None):
    """Layer norm of x [..., C] (bf16, fp16, fp32) over the last axis, of x + res when res is given;
    w, b fp32 [C].  Returns (y, sum, mean, rstd): sum is x + res in x's type (x itself without
    res), mean and rstd fp32 one per row -- what kda_layernorm_bwd takes."""
    fn = "kda_layernorm_fwd"
    pr = _layernorm_problem(fn, x, eps)
    dev = x.device
    if y is None:
        y = torch.empty_like(x)
    else:
        _check_tensor(fn, "y", y, x.shape, x.dtype, dev)
    if res is None:
        if sum is not None:
            raise ValueError(f"{fn}: a sum needs a residual")
    else:
        _check_tensor(fn, "res", res, x.shape, x.dtype, dev)
        if sum is None:
            sum = torch.empty_like(x)
        else:
            _check_tensor(fn, "sum", sum, x.shape, x.dtype, dev)
    _check_tensor(fn, "w", w, (pr.C,), torch.float32, dev)
    _check_tensor(fn, "b", b, (pr.C,), torch.float32, dev)
    mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev)
    _call(fn, dev, ctypes.byref(pr), x.data_ptr(), _at(res), _at(w), _at(b), _at(sum), y.data_ptr(),
          mean.data_ptr(), rstd.data_ptr())
    return y, x if res is None else sum, mean, rstd


def kda_layernorm_bwd(x, w, mean, rstd, dy, *, dsum=None, ws=None):
    """Backward of the layer norm: x is what was normalised (the forward's sum), dsum the gradient
    that reaches it past the norm.  Returns dict dx, dw, db (w may be None: ones)."""
    fn = "kda_layernorm_bwd"
    pr = _layernorm_problem(fn, x, 0.0)
    dev = x.device
    _check_tensor(fn, "dy", dy, x.shape, x.dtype, dev)
    _check_tensor(fn, "dsum", dsum, x.shape, x.dtype, dev)
    _check_tensor(fn, "w", w, (pr.C,), torch.float32, dev)
    _check_tensor(fn, "mean", mean, x.shape[:-1], torch.float32, dev)
    _check_tensor(fn, "rstd", rstd, x.shape[:-1], torch.float32, dev)
    ws, ws_n = _workspace(fn, ws, kda_layernorm_workspace_size(pr.T, pr.C, dtype=x.dtype), dev)
    out = dict(dx=torch.empty_like(x),
               dw=torch.empty((pr.C,), dtype=torch.float32, device=dev),
               db=torch.empty((pr.C,), dtype=torch.float32, device=dev))
    _call(fn, dev, ctypes.byref(pr), x.data_ptr(), _at(w), mean.data_ptr(), rstd.data_ptr(), dy.data_ptr(),
          _at(dsum), out["dx"].data_ptr(), out["dw"].data_ptr(), out["db"].data_ptr(), ws.data_ptr(),
          ws_n)
    return out


def kda_read_device_status(ws) -> int:
    v = ctypes.c_int(0)
    with torch.cuda.device(ws.device):
        _check("kda_read_device_status",
               lib().kda_read_device_status(_ptr(ws), ctypes.byref(v), _stream(ws.device)))
    return v.value


def kda_selftest_wait_timeout(ws, limit_us=20000):
    """Runs a kernel whose bounded wait must time out; its KDA_ERR_TIMEOUT lands in ws's status."""
    with torch.cuda.device(ws.device):
        _check("kda_selftest_wait_timeout",
               lib().kda_selftest_wait_timeout(_ptr(ws), ctypes.c_uint32(int(limit_us)), _stream(ws.device)))


def kda_profile_enable(enable=True):
    _check("kda_profile_enable", lib().kda_profile_enable(int(bool(enable))))


def kda_profile_collect():
    """{kernel name: (summed device ms, launches)} since the last collect (waits for events)."""
    n = lib().kda_kernel_count()
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_uint64 * n)()
    _check("kda_profile_collect", lib().kda_profile_collect(ms, cnt))
    return {lib().kda_kernel_name(i).decode(): (ms[i], cnt[i]) for i in range(n)}


def kda_launch_counter() -> int:
    return int(lib().kda_launch_counter())
