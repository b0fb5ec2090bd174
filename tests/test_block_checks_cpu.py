"""Checks of the binding that keep a tensor the kernels could not read from reaching them: offsets of the conv's
window, workspaces and saved sets.  No GPU needed: what fits ends at the refusal of tensors on the CPU."""
import pytest
import torch

from linear_attention_chunked_gb300 import build, kda

bf = torch.bfloat16
FITS = "expected a CUDA device"


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return kda.lib()


@pytest.mark.parametrize("cu,word", [
    (torch.tensor([0, 2, 5]), "cu_seqlens is torch.int64"),
    (torch.tensor([0.0, 2.0, 5.0]), "cu_seqlens is torch.float32"),
    (torch.tensor([0, 9, 2, 9, 5, 9], dtype=torch.int32)[::2], "cu_seqlens has strides"),
    (torch.tensor([[0, 2, 5]], dtype=torch.int32), "cu_seqlens has shape"),
    (torch.empty(3, dtype=torch.int32, device="meta"), "cu_seqlens is on meta"),
    (torch.tensor([0, 2, 5], dtype=torch.int32), FITS),
])
def test_offsets_of_the_conv_window(cu, word):
    with pytest.raises(ValueError, match=word):
        kda.kda_conv_tail(torch.zeros(5, 16, dtype=bf), cu)


def _calls():
    """Every call that takes a workspace: (call of keywords, its smallest workspace in bytes)."""
    T, C, S = 6, 16, 4
    x = torch.zeros(T, C, dtype=bf)
    bc = torch.zeros(T, S, dtype=bf)
    cu = torch.tensor([0, T], dtype=torch.int32)
    a, cs = (x, x, torch.zeros(C, S), bc, bc), torch.zeros(C)
    size = lambda op: kda.kda_ssm_workspace_size(T, 1, C, S, 1, op)  # noqa: E731
    ws, saved = size(kda.KDA_OP_FWD)
    st = torch.zeros(T)
    return {
        "kda_ssm_fwd": (lambda **kw: kda.kda_ssm_fwd(*a, cu, save=False, **kw), ws),
        "kda_ssm_bwd": (lambda **kw: kda.kda_ssm_bwd(*a, cu, x, saved=torch.zeros(saved, dtype=torch.uint8), **kw), size(kda.KDA_OP_BWD_SAVED)[0]),
        "kda_ssm_bwd replay": (lambda **kw: kda.kda_ssm_bwd(*a, cu, x, **kw), size(kda.KDA_OP_BWD_REPLAY)[0]),
        "kda_ssm_step": (lambda **kw: kda.kda_ssm_step(*a, torch.zeros(T, C, S), **kw), 256),
        "kda_conv_step": (lambda **kw: kda.kda_conv_step(x, torch.zeros(C, 4), torch.zeros(T, 3, C, dtype=bf), **kw), 256),
        "kda_layernorm_bwd": (lambda **kw: kda.kda_layernorm_bwd(x, cs, st, st, x, **kw), kda.kda_layernorm_workspace_size(T, C)),
    }


@pytest.mark.parametrize("name", ["kda_ssm_fwd", "kda_ssm_bwd", "kda_ssm_bwd replay", "kda_ssm_step", "kda_conv_step", "kda_layernorm_bwd"])
def test_workspaces(name, monkeypatch):
    call, need = _calls()[name]
    u8 = torch.uint8
    for ws, word in ((torch.empty(need, dtype=u8, device="meta"), "ws is on meta"),
                     (torch.zeros(2 * need, dtype=u8)[::2], "ws has strides"),
                     (torch.zeros(need, dtype=u8), FITS), (torch.zeros(need // 4), FITS)):
        with pytest.raises(ValueError, match=word):
            call(ws=ws)
    if "step" in name:
        with pytest.raises(ValueError, match="ws holds 255 bytes, needs 256"):
            call(ws=torch.zeros(255, dtype=u8))
    else:  # the library, which refuses too few, is told the bytes whatever the tensor's type is
        told = []
        monkeypatch.setattr(kda, "_call", lambda fn, dev, *args: told.append(args[-1]))
        call(ws=torch.zeros(need // 4 + 1))
        assert told == [4 * (need // 4 + 1)]


def test_saved_sets():
    T, C, S = 6, 16, 4
    x, bc, cu = torch.zeros(T, C, dtype=bf), torch.zeros(T, S, dtype=bf), torch.tensor([0, T], dtype=torch.int32)
    a = (x, x, torch.zeros(C, S), bc, bc, cu)
    need = kda.kda_ssm_workspace_size(T, 1, C, S, 1, kda.KDA_OP_FWD)[1]
    u8 = torch.uint8
    for saved, word in ((torch.empty(need, dtype=u8, device="meta"), "saved is on meta"),
                        (torch.zeros(2 * need, dtype=u8)[::2], "saved has strides"),
                        (torch.zeros(need - 1, dtype=u8), f"saved holds {need - 1} bytes, needs {need}"),
                        (torch.zeros(need, dtype=u8), FITS), (torch.zeros(need // 4), FITS)):
        with pytest.raises(ValueError, match=word):
            kda.kda_ssm_fwd(*a, saved=saved)
        with pytest.raises(ValueError, match=word):
            kda.kda_ssm_bwd(*a, x, saved=saved)


def test_size_queries_refuse_other_types():
    for size in (lambda **kw: kda.kda_ssm_workspace_size(6, 1, 16, 4, 1, kda.KDA_OP_FWD, **kw), lambda **kw: kda.kda_layernorm_workspace_size(6, 16, **kw)):
        with pytest.raises(ValueError, match="dtype is torch.float64"):
            size(dtype=torch.float64)
