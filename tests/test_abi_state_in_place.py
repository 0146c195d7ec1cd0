"""Only the state may be updated in place: the exemption from the overlap
checks of the recurrence's entry points is for its own pair of buffers, not
for any input that starts where they do.  No GPU: every call is refused."""
import ctypes
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, I = ctypes.c_void_p, ctypes.c_int
A = [0x10000000 * k for k in range(1, 12)]
SHAPE = (2, 4, 100)


@pytest.fixture(scope="module")
def lib():
    spec = importlib.util.spec_from_file_location(
        "_wbmm_build", os.path.join(ROOT, "windowed_matmul_conv_b200", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    return ctypes.CDLL(build.build())


def proto(lib, name, pointers, ints):
    f = getattr(lib, name)
    f.restype, f.argtypes = I, [P] * pointers + [I] * ints + [P]
    return f


def test_forward(lib):
    f = proto(lib, "wbmm_scan_forward", 11, 4)
    rest = (None,) * 5
    # v, g, h0, lengths, y, hT: hT in h0's buffer, which is an input's too
    assert f(A[2], A[1], A[2], None, A[4], A[2], *rest, *SHAPE, 0, None) == 1
    assert f(A[0], A[2], A[2], None, A[4], A[2], *rest, *SHAPE, 0, None) == 1
    assert f(A[0], A[1], A[2], A[2], A[4], A[2], *rest, *SHAPE, 0, None) == 1


def test_backward(lib):
    f = proto(lib, "wbmm_scan_backward", 9, 4)
    # v, g, states, lengths, dY, dhT, dv, dg, dh0
    for k in (0, 1, 2, 3, 4):
        a = [A[0], A[1], A[2], A[3], A[4], A[5], A[6], A[7], A[5]]
        a[k] = A[5]
        assert f(*a, *SHAPE, 0, None) == 1, k


def test_backward_from_checkpoints(lib):
    f = proto(lib, "wbmm_scan_backward_checkpoint", 11, 4)
    # v_codes, v_exps, g_codes, g_exps, states, lengths, dY, dhT, dv, dg, dh0
    for k in range(7):
        a = [A[0], A[1], A[2], A[3], A[4], A[5], A[6], A[7], A[8], A[9], A[7]]
        a[k] = A[7]
        assert f(*a, *SHAPE, 0, None) == 1, k


def test_step(lib):
    f = proto(lib, "wbmm_scan_step", 5, 3)
    assert f(A[2], A[1], A[2], A[3], A[2], 2, 4, 0, None) == 1
    assert f(A[0], A[2], A[2], A[3], A[2], 2, 4, 0, None) == 1
