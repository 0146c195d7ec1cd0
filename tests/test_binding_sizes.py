"""Sizes beyond the C ABI's ints are refused by the binding: ctypes would cut
them to 32 bits, and the call would run on other sizes than its buffers were
checked for.  Expanded views stand in for maps that large; no GPU."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, U8 = torch.bfloat16, torch.uint8
CUT = 1 << 32                   # what 32 bits do not see


@pytest.fixture(scope="module")
def wb():
    spec = importlib.util.spec_from_file_location(
        "_wbmm_build", os.path.join(ROOT, "windowed_matmul_conv_b200", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    build.build()
    import windowed_matmul_conv_b200 as mod
    return mod


def wide(*shape, dtype=BF):
    return torch.zeros(1, dtype=dtype).expand(*shape)


def refused(wb, fn, *a):
    with pytest.raises(wb.WbmmError) as e:
        fn(*a)
    return e.value.status == 5


def test_window_sizes(wb):
    x, codes = torch.zeros((2, 3, 28, 28), dtype=BF), torch.zeros(2 * 3 * 28 * 28, dtype=U8)
    short = torch.zeros(1, dtype=U8)    # a window of 14 has 24 exponent bytes here
    T, dT, ws = torch.zeros((3, 729), dtype=BF), torch.zeros((3, 729)), torch.zeros(16)
    for w in (CUT + 14, 14 - CUT):
        assert refused(wb, wb.wbmm_checkpoint, x, codes, short, w)
        assert refused(wb, wb.wbmm_checkpoint_restore, codes, short, x, w)
        assert refused(wb, wb.wbmm_backward_checkpoint, codes, short, T, x, x, dT, ws, w)
        assert refused(wb, wb.wbmm_backward_checkpoint_workspace_bytes, 2, 3, 28, 28, w, BF)
        assert refused(wb, wb.wbmm_backward_workspace_bytes, 2, 3, 28, 28, w, BF)


def test_map_sizes(wb):
    for shape in ((CUT + 2, 1, 2, 2), (1, CUT + 1, 2, 2), (1, 1, CUT + 2, 2), (1, 1, 2, CUT + 2)):
        x, codes, exps = wide(*shape), wide(*shape, dtype=U8), wide(*shape, dtype=U8)
        T, M, K = wide(shape[1], 9), wide(shape[1], 4, 4), wide(shape[1], 1, 3, 3)
        dT = wide(shape[1], 9, dtype=torch.float32)
        assert refused(wb, wb.wbmm_checkpoint, x, codes, exps, 2)
        assert refused(wb, wb.wbmm_checkpoint_restore, codes, exps, x, 2)
        assert refused(wb, wb.checkpoint_restore, codes, exps, shape, 2, BF)
        assert refused(wb, wb.wbmm_backward_checkpoint, codes, exps, T, x, x, dT, dT, 2)
        assert refused(wb, wb.wbmm_backward_checkpoint_workspace_bytes, *shape, 2, BF)
        assert refused(wb, wb.wbmm_forward, x, T, x, 2)
        assert refused(wb, wb.wbmm_backward, x, T, x, x, dT, dT, 2)
        assert refused(wb, wb.wbmm_backward_dt_static, x, x, dT, 2)
        assert refused(wb, wb.wbmm_backward_workspace_bytes, *shape, 2, BF)
        assert refused(wb, wb.wbmm_forward_cached, x, M, None, x, 2)
        assert refused(wb, wb.wbmm_dw3x3, x, K, x)
    C = CUT + 1
    assert refused(wb, wb.wbmm_cache_matrices, wide(C, 9), wide(C, 4, 4), 2)
    assert refused(wb, wb.wbmm_reparam_merge, wide(C, 9), wide(C, 1), wide(C, 4, 4), 2, 1)


def test_sequence_sizes(wb):
    for B, C, L in ((CUT + 1, 1, 2), (1, CUT + 1, 2), (1, 1, CUT + 1)):
        x, f = wide(B, C, L), wide(B, C, dtype=torch.float32)
        states = wide(B, C, -(-L // 256), dtype=torch.float32)
        assert refused(wb, wb.wbmm_scan_forward, x, x, None, None, x, *[None] * 6)
        assert refused(wb, wb.wbmm_scan_backward, x, x, states, None, x, None, x, x, None)
        assert refused(wb, wb.wbmm_scan_states_bytes, B, C, L)
        if L == 2:
            assert refused(wb, wb.wbmm_scan_step, x[:, :, 0], x[:, :, 0], f, x[:, :, 0], f)
    assert wb.wbmm_scan_states_bytes(1, 1, (1 << 31) - 1) == 4 << 23


def test_large_maps_with_sizes_that_fit_pass(wb):
    """More than 2^31 elements are no reason to refuse."""
    x, u8 = wide(1 << 10, 1 << 10, 56, 56), wide(1 << 10, 1 << 10, 56, 56, dtype=U8)
    with pytest.raises(ValueError):     # the checks passed; only the CPU pointer is refused
        wb.wbmm_checkpoint(x, u8, u8, 14)
