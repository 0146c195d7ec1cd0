"""The Python binding's buffer checks, without a GPU.

The C ABI takes plain pointers, so the binding checks what the library
cannot see: each buffer's device, dtype and element count against the call's
map.  CPU tensors stand in for device tensors here: a call whose buffers pass
the checks reaches the pointer conversion, which refuses non-CUDA tensors
with ValueError before anything is launched.  (The device check compares
CUDA device indices and needs two GPUs to fail.)
"""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def wb():
    spec = importlib.util.spec_from_file_location(
        "_wbmm_build", os.path.join(ROOT, "windowed_matmul_conv_b200", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    build.build()
    import windowed_matmul_conv_b200 as mod
    return mod


BF = torch.bfloat16


def maps(B=2, C=3, H=28, W=28, dtype=BF):
    return torch.zeros((B, C, H, W), dtype=dtype)


def status_of(fn, *a):
    import windowed_matmul_conv_b200 as mod
    try:
        fn(*a)
    except mod.WbmmError as e:
        return e.status
    except ValueError:
        return "passed"          # checks passed; only the CUDA pointer was refused
    raise AssertionError("no exception")


def test_forward_buffers(wb):
    x, T, y = maps(), torch.zeros((3, 729), dtype=BF), maps()
    assert status_of(wb.wbmm_forward, x, T, y, 14) == "passed"
    assert status_of(wb.wbmm_forward, x, T[:2], y, 14) == 1            # table too short
    assert status_of(wb.wbmm_forward, x, T, y[:1], 14) == 1            # output too short
    assert status_of(wb.wbmm_forward, x, T.float(), y, 14) == 3        # table dtype
    assert status_of(wb.wbmm_forward, x, T, y.float(), 14) == 3        # output dtype
    # a longer table than the window needs is fine (the library rejects the shape)
    assert status_of(wb.wbmm_forward, x, T, y, 7) == "passed"


def test_backward_buffers(wb):
    x, dY, dX = maps(), maps(), maps()
    T = torch.zeros((3, 729), dtype=BF)
    dT = torch.zeros((3, 729), dtype=torch.float32)
    ws = torch.zeros(16, dtype=torch.float32)
    assert status_of(wb.wbmm_backward, x, T, dY, dX, dT, ws, 14) == "passed"
    assert status_of(wb.wbmm_backward, None, T, dY, dX, None, None, 14) == "passed"
    assert status_of(wb.wbmm_backward, x, None, dY, None, dT, ws, 14) == "passed"
    assert status_of(wb.wbmm_backward, x[:1], T, dY, dX, dT, ws, 14) == 1
    assert status_of(wb.wbmm_backward, x, T, dY, dX[:1], dT, ws, 14) == 1
    assert status_of(wb.wbmm_backward, x, T, dY, dX, dT[:2], ws, 14) == 1
    assert status_of(wb.wbmm_backward, x, T, dY, dX, dT.to(BF), ws, 14) == 3   # dT is fp32
    assert status_of(wb.wbmm_backward, x.float(), T, dY, dX, dT, ws, 14) == 3
    assert status_of(wb.wbmm_backward_dt_static, x, dY, dT, 14) == "passed"
    assert status_of(wb.wbmm_backward_dt_static, x, dY, dT[:1], 14) == 1
    assert status_of(wb.wbmm_backward_dt_static, x[:1], dY, dT, 14) == 1


def test_cached_path_buffers(wb):
    T = torch.zeros((3, 729), dtype=BF)
    M = torch.zeros((3, 196, 196), dtype=BF)
    assert status_of(wb.wbmm_cache_matrices, T, M, 14) == "passed"
    assert status_of(wb.wbmm_cache_matrices, T, M[:2], 14) == 1
    assert status_of(wb.wbmm_cache_matrices, T[:, :169], M, 14) == 1
    Tk = torch.zeros((3, 169), dtype=BF)
    assert status_of(wb.wbmm_reparam_merge, T, Tk, M, 14, 7) == "passed"
    assert status_of(wb.wbmm_reparam_merge, T, Tk[:, :25], M, 14, 7) == 1
    assert status_of(wb.wbmm_reparam_merge, T, Tk.float(), M, 14, 7) == 3
    x, out = maps(), maps()
    K = torch.zeros((3, 1, 3, 3), dtype=BF)
    assert status_of(wb.wbmm_forward_cached, x, M, None, out, 14) == "passed"
    assert status_of(wb.wbmm_forward_cached, x, M, K, out, 14) == "passed"
    assert status_of(wb.wbmm_forward_cached, x, M[:1], K, out, 14) == 1
    assert status_of(wb.wbmm_forward_cached, x, M, K[:2], out, 14) == 1
    assert status_of(wb.wbmm_forward_cached, x, M, K, out[:, :2], 14) == 1
    assert status_of(wb.wbmm_dw3x3, x, K, out) == "passed"
    assert status_of(wb.wbmm_dw3x3, x, K.float(), out) == 3
    assert status_of(wb.wbmm_dw3x3, x, K, out[:1]) == 1


def test_workspace_size_dtypes(wb):
    assert wb.wbmm_backward_workspace_bytes(2, 3, 28, 28, 14, torch.float32) > 0
    with pytest.raises(TypeError):
        wb.wbmm_backward_workspace_bytes(2, 3, 28, 28, 14, torch.float16)


def test_checkpoint_buffers(wb):
    x = maps()
    codes, exps = torch.zeros(x.numel(), dtype=torch.uint8), torch.zeros(24, dtype=torch.uint8)
    for f in (lambda c, e: wb.wbmm_checkpoint(x, c, e, 14), lambda c, e: wb.wbmm_checkpoint_restore(c, e, x, 14)):
        assert status_of(f, codes, exps) == "passed"
        assert status_of(f, codes[1:], exps) == 1
        assert status_of(f, codes, exps[1:]) == 1
        assert status_of(f, codes.to(torch.int8), exps) == 3
        assert status_of(f, codes, exps.int()) == 3
    T, dY, dX = torch.zeros((3, 729), dtype=BF), maps(), maps()
    dT, ws = torch.zeros((3, 729)), torch.zeros(16)
    assert status_of(wb.wbmm_backward_checkpoint, codes, exps, T, dY, dX, dT, ws, 14) == "passed"
    assert status_of(wb.wbmm_backward_checkpoint, codes[1:], exps, T, dY, dX, dT, ws, 14) == 1
    assert status_of(wb.wbmm_backward_checkpoint, codes, exps[1:], T, dY, dX, dT, ws, 14) == 1
    assert status_of(wb.wbmm_backward_checkpoint, codes, exps, T[:2], dY, dX, dT, ws, 14) == 1
    assert status_of(wb.wbmm_backward_checkpoint, codes, exps, T, dY, dX, dT.to(BF), ws, 14) == 3


def test_recurrence_buffers(wb):
    B, C, L = 2, 3, 300
    x, u8 = torch.zeros((B, C, L), dtype=BF), torch.uint8
    h, n = torch.zeros((B, C)), torch.zeros(B, dtype=torch.int32)
    st, cd, ex = torch.zeros((B, C, 2)), torch.zeros((B, C, L), dtype=u8), torch.zeros((B, C, 5), dtype=u8)
    good = dict(v=x, g=x, h0=h, lengths=n, y=x, hT=h, states=st, vc=cd, ve=ex, gc=cd, ge=ex)

    def fwd(**k):
        return status_of(wb.wbmm_scan_forward, *{**good, **k}.values())
    assert fwd() == "passed" and fwd(h0=None, lengths=None, hT=None, states=None) == "passed"
    assert fwd(g=x[:1]) == 1 and fwd(y=x[:, :1]) == 1 and fwd(h0=h[:1]) == 1 and fwd(hT=h[:, :2]) == 1
    assert fwd(lengths=n[:1]) == 1 and fwd(states=st[:, :, :1]) == 1 and fwd(gc=cd[:1]) == 1 and fwd(ve=ex[:1]) == 1
    assert fwd(g=x.float()) == 3 and fwd(h0=h.to(BF)) == 3 and fwd(lengths=n.long()) == 3 and fwd(vc=ex.int()) == 3
    good2 = dict(v=x, g=x, states=st, lengths=n, dY=x, dhT=h, dv=x, dg=x, dh0=h)

    def bwd(**k):
        return status_of(wb.wbmm_scan_backward, *{**good2, **k}.values())
    assert bwd() == "passed" and bwd(dhT=None, dh0=None, lengths=None) == "passed"
    assert bwd(v=x[:1]) == 1 and bwd(dg=x[:1]) == 1 and bwd(states=st[:1]) == 1 and bwd(dh0=h[:1]) == 1
    assert bwd(dv=x.float()) == 3 and bwd(dhT=h.double()) == 3
    good3 = dict(vc=cd, ve=ex, gc=cd, ge=ex, states=st, lengths=n, dY=x, dhT=h, dv=x, dg=x, dh0=h)

    def bwd8(**k):
        return status_of(wb.wbmm_scan_backward_checkpoint, *{**good3, **k}.values())
    assert bwd8() == "passed" and bwd8(vc=cd[:1]) == 1 and bwd8(ge=ex[:, :, :4]) == 1 and bwd8(vc=cd.int()) == 3
    s = x[:, :, 0].contiguous()
    assert status_of(wb.wbmm_scan_step, s, s, h, s, h) == "passed"
    assert status_of(wb.wbmm_scan_step, s, s[:1], h, s, h) == 1
    assert status_of(wb.wbmm_scan_step, s, s, h[:1], s, h) == 1
    assert status_of(wb.wbmm_scan_step, s, s, h, s, h.double()) == 3
    with pytest.raises(ValueError):
        wb.wbmm_scan_step(x, x, h, x, h)
    with pytest.raises(ValueError):
        wb.scan_forward(x[0, 0], x[0, 0])
    # more positions than the C ABI's int holds (an expanded view: no memory)
    huge = torch.zeros(1, dtype=BF).expand(1, 1, 1 << 32)
    with pytest.raises(wb.WbmmError) as e:
        wb.wbmm_scan_forward(huge, huge, None, None, huge, *[None] * 6)
    assert e.value.status == 5
