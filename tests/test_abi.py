"""The C ABI without a GPU: the library loads, exports every symbol the header
declares, and rejects bad arguments before touching the device."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "wbmm.h")


def declared_symbols():
    text = open(HEADER).read()
    return re.findall(r"WBMM_API\s+[\w\s\*]+?\b(wbmm_\w+)\s*\(", text)


@pytest.fixture(scope="module")
def lib():
    # by path: the package's __init__ refuses to import before the library exists
    import importlib.util
    spec = importlib.util.spec_from_file_location(
        "_wbmm_build", os.path.join(ROOT, "windowed_matmul_conv_b200", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    return ctypes.CDLL(build.build())


def test_header_declares_the_entry_points():
    names = declared_symbols()
    for required in ("wbmm_forward", "wbmm_backward", "wbmm_backward_workspace_bytes",
                     "wbmm_cache_matrices", "wbmm_forward_cached", "wbmm_dw3x3"):
        assert required in names


def test_library_exports_every_declared_symbol(lib):
    for name in declared_symbols():
        assert hasattr(lib, name), name


def test_binding_mirrors_the_header(lib):
    import windowed_matmul_conv_b200 as wb
    assert sorted(wb.EXPORTS) == sorted(declared_symbols())
    for name in wb.EXPORTS:
        assert callable(getattr(wb, name))


def _fwd(lib, x, T, y, B, C, H, W, w, dt):
    f = lib.wbmm_forward
    f.restype = ctypes.c_int
    f.argtypes = [ctypes.c_void_p] * 3 + [ctypes.c_int] * 6 + [ctypes.c_void_p]
    return f(x, T, y, B, C, H, W, w, dt, None)


def test_argument_checks_need_no_device(lib):
    a, b, c = 0x10000, 0x20000000, 0x40000000       # never dereferenced
    assert _fwd(lib, None, b, c, 1, 1, 14, 14, 7, 1) == 1   # null input
    assert _fwd(lib, a, b, c, 1, 1, 14, 15, 7, 1) == 2      # W % w
    assert _fwd(lib, a, b, c, 0, 1, 14, 14, 7, 1) == 1      # B = 0
    assert _fwd(lib, a, b, c, 1, 1, 14, 14, 7, 9) == 3      # dtype
    assert _fwd(lib, a + 2, b, c, 1, 1, 14, 14, 7, 1) == 4  # bf16 needs 16 B
    assert _fwd(lib, a, b, a + 64, 1, 1, 14, 14, 7, 1) == 1  # y overlaps x
    assert _fwd(lib, a, b, c, 1, 1, 130, 130, 65, 1) == 5   # w beyond limit


def test_workspace_size_formula(lib):
    f = lib.wbmm_backward_workspace_bytes
    f.restype = ctypes.c_size_t
    f.argtypes = [ctypes.c_int] * 6
    # bf16, tensor-core path: a fixed region of 65536 arrival counters, then
    # one partial table per (channel, CTA range) segment, at most
    # n = C + min(256, tiles) - 1 of them.
    def tc(C, grid, tsz=729):
        n = C + grid - 1
        return (65536 + n * tsz) * 4
    # training workload: 64-window tiles of 32 two-window bands, 8 tiles per
    # channel, 2048 tiles -> 256 + 255 tables
    assert f(128, 256, 28, 28, 14, 1) == tc(256, 256)
    # 64 images of 56x56: 16 bands/tile, 16 tiles/channel, 2048 tiles
    assert f(64, 128, 56, 56, 14, 1) == tc(128, 256)
    # 32 images of 112x112: 8 bands/tile, 32 tiles/channel, 128 tiles
    assert f(32, 4, 112, 112, 14, 1) == tc(4, 128)
    # 2 images of 112x112, w = 7: 64-window tiles of 4 bands, 8 tiles/channel
    assert f(2, 4, 112, 112, 7, 1) == tc(4, 32, 169)
    # fp32, CUDA-core path, 4 <= w <= 14: tiles of whole bands (at most 64
    # windows); all channels' tiles split into min(148, tiles) contiguous
    # ranges; a channel spans at most 2 + (n - 2) // (fewest tiles of a
    # range) of them (n tiles per channel, capped at n), one partial table
    # slot each
    assert f(2, 3, 14, 28, 7, 0) == (65536 + 3 * 1 * 169) * 4
    # training workload: 8 tiles per channel, 2048 tiles in ranges of 13 or 14
    assert f(128, 256, 28, 28, 14, 0) == (65536 + 256 * 2 * 729) * 4
    # 3 tiles per channel, 6 tiles, one per range: 3 slots
    assert f(3, 2, 56, 56, 7, 0) == (65536 + 2 * 3 * 169) * 4
    # w > 14: chunks of 8 bands per channel
    assert f(2, 3, 40, 40, 20, 0) == (65536 + 3 * 1 * 1521) * 4
    assert f(9, 1, 40, 40, 20, 0) == (65536 + 1 * 3 * 1521) * 4
    assert f(1, 1, 14, 15, 7, 1) == 0


def test_status_strings(lib):
    f = lib.wbmm_status_string
    f.restype = ctypes.c_char_p
    f.argtypes = [ctypes.c_int]
    for s in range(9):
        assert f(s).decode().startswith("WBMM_")


def _proto(lib, name, argtypes):
    f = getattr(lib, name)
    f.restype = ctypes.c_int
    f.argtypes = argtypes
    return f


P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t

# Addresses that are never dereferenced: every call below must be rejected by
# the host-side checks, before any device call.  Blocks are 256 MB apart so
# that buffers of the shapes used never overlap unless a test says so.
A0, A1, A2, A3, A4 = (0x10000000 * k for k in (1, 2, 3, 4, 5))


def test_backward_argument_checks(lib):
    f = _proto(lib, "wbmm_backward", [P, P, P, P, P, P, S] + [I] * 6 + [P])
    ws = lib.wbmm_backward_workspace_bytes
    ws.restype, ws.argtypes = S, [I] * 6
    need = ws(2, 4, 28, 28, 14, 1)
    assert need > 0

    def call(x=A0, T=A1, dY=A2, dX=A3, dT=A4, work=A4 + 0x100000, nbytes=need,
             shape=(2, 4, 28, 28, 14), dt=1):
        return f(x, T, dY, dX, dT, work, nbytes, *shape, dt, None)

    assert call(dt=2) == 3                               # dtype
    assert call(dY=None) == 1                            # dY is required
    assert call(T=None) == 1                             # dX needs the table
    assert call(x=None) == 1                             # dT needs the input
    assert call(shape=(2, 4, 28, 30, 14)) == 2           # W % w
    assert call(shape=(2, 4, 28, 28, 0)) == 1            # w = 0
    assert call(shape=(2, 4, 130, 130, 65)) == 5         # w beyond limit
    assert call(dX=A3 + 8) == 4                          # bf16 maps need 16 B
    assert call(dT=A4 + 2) == 4                          # dT is fp32
    assert call(dX=A2 + 64) == 1                         # dX overlaps dY
    assert call(dT=A0 + 64) == 1                         # dT overlaps x
    assert call(work=None) == 6                          # dT needs a workspace
    assert call(nbytes=need - 4) == 6                    # ... of the stated size
    assert call(work=A4 + 0x100008) == 4                 # ... 16-byte aligned
    assert call(work=A4 + 64) == 1                       # ... not overlapping dT
    assert call(work=A2 + 64) == 1                       # ... nor dY
    # dX only: neither x nor a workspace is needed, so the first failing check
    # is the misaligned dX
    assert call(dT=None, x=None, work=None, nbytes=0, dX=A3 + 8) == 4
    # dT only: no table needed
    assert call(dX=None, T=None, dT=A4 + 2) == 4


def test_cache_and_merge_argument_checks(lib):
    cache = _proto(lib, "wbmm_cache_matrices", [P, P, I, I, I, P])
    assert cache(A0, A1, 4, 14, 3, None) == 3
    assert cache(None, A1, 4, 14, 1, None) == 1
    assert cache(A0, A1, 0, 14, 1, None) == 1
    assert cache(A0, A1, 4, 65, 1, None) == 5
    assert cache(A0, A1 + 2, 4, 14, 1, None) == 4
    assert cache(A0, A0 + 128, 4, 14, 1, None) == 1      # M overlaps T
    merge = _proto(lib, "wbmm_reparam_merge", [P, P, P, I, I, I, I, P])
    assert merge(A0, A1, A2, 4, 14, 7, 5, None) == 3
    assert merge(A0, None, A2, 4, 14, 7, 1, None) == 1
    assert merge(A0, A1, A2, 4, 14, 5, 1, None) == 1     # k must divide w
    assert merge(A0, A1, A2, 4, 14, 0, 1, None) == 1
    assert merge(A0, A1, A2, 4, 70, 7, 1, None) == 5
    assert merge(A0, A1, A2 + 8, 4, 14, 7, 1, None) == 4
    assert merge(A0, A2 + 64, A2, 4, 14, 7, 1, None) == 1  # M overlaps the small table


def test_cached_and_dw_argument_checks(lib):
    fc = _proto(lib, "wbmm_forward_cached", [P, P, P, P] + [I] * 6 + [P])
    assert fc(A0, A1, None, A2, 1, 4, 28, 28, 14, 4, None) == 3
    assert fc(A0, None, None, A2, 1, 4, 28, 28, 14, 1, None) == 1
    assert fc(A0, A1, None, A2, 1, 4, 28, 21, 14, 1, None) == 2
    assert fc(A0, A1, A3 + 2, A2, 1, 4, 28, 28, 14, 1, None) == 4   # 3x3 weights
    assert fc(A0, A1, None, A0 + 16, 1, 4, 28, 28, 14, 1, None) == 1  # out overlaps x
    assert fc(A0, A1, A2 + 16, A2, 1, 4, 28, 28, 14, 1, None) == 1  # out overlaps the weights
    dw = _proto(lib, "wbmm_dw3x3", [P, P, P] + [I] * 5 + [P])
    assert dw(A0, A1, A2, 1, 4, 9, 13, 7, None) == 3
    assert dw(A0, A1, None, 1, 4, 9, 13, 1, None) == 1
    assert dw(A0, A1, A2, 1, 4, 0, 13, 1, None) == 1
    assert dw(A0 + 8, A1, A2, 1, 4, 9, 13, 1, None) == 4
    assert dw(A0, A1, A0 + 32, 1, 4, 9, 13, 1, None) == 1           # in place is refused


def test_static_table_gradient_argument_checks(lib):
    f = _proto(lib, "wbmm_backward_dt_static", [P, P, P] + [I] * 6 + [P])
    assert f(A0, A1, A2, 2, 4, 28, 28, 14, 2, None) == 3
    assert f(A0, None, A2, 2, 4, 28, 28, 14, 1, None) == 1
    assert f(A0, A1, A2, 2, 4, 28, 27, 14, 1, None) == 2
    assert f(A0, A1, A2, 2, 4, 130, 130, 65, 1, None) == 5
    assert f(A0, A1 + 8, A2, 2, 4, 28, 28, 14, 1, None) == 4
    assert f(A0, A1, A0 + 64, 2, 4, 28, 28, 14, 1, None) == 1       # dT overlaps x
    # more partial tables than the 4 MiB static array holds
    assert f(A0, A1, A2, 1, 2048, 14, 14, 14, 1, None) == 6


def test_checkpoint_argument_checks(lib):
    st = _proto(lib, "wbmm_checkpoint", [P, P, P] + [I] * 6 + [P])
    re_ = _proto(lib, "wbmm_checkpoint_restore", [P, P, P] + [I] * 6 + [P])
    shape = (2, 4, 28, 28, 14)
    assert st(A0, A1, A2, *shape, 2, None) == 3
    assert st(None, A1, A2, *shape, 1, None) == 1
    assert st(A0, None, A2, *shape, 1, None) == 1
    assert st(A0, A1, None, *shape, 1, None) == 1
    assert st(A0, A1, A2, 2, 4, 28, 29, 14, 1, None) == 2
    assert st(A0, A1, A2, 0, 4, 28, 28, 14, 1, None) == 1
    assert st(A0, A1, A2, 1, 4, 130, 130, 65, 1, None) == 5
    assert st(A0 + 2, A1, A2, *shape, 1, None) == 4
    assert st(A0, A1 + 8, A2, *shape, 1, None) == 4
    assert st(A0, A0 + 16, A2, *shape, 1, None) == 1     # codes overlap x
    assert st(A0, A1, A1 + 6271, *shape, 1, None) == 1   # exponents overlap the codes' last byte
    assert st(A0, A1, A0, *shape, 1, None) == 1
    assert re_(A0, A1, A2, *shape, 7, None) == 3
    assert re_(A0, A1, None, *shape, 1, None) == 1
    assert re_(A0 + 4, A1, A2, *shape, 1, None) == 4
    assert re_(A0, A1, A2 + 4, *shape, 1, None) == 4
    assert re_(A0, A1, A0 + 16, *shape, 1, None) == 1
    assert re_(A0, A1, A2, 2, 4, 27, 28, 14, 1, None) == 2


def test_backward_checkpoint_argument_checks(lib):
    f = _proto(lib, "wbmm_backward_checkpoint", [P] * 7 + [S] + [I] * 6 + [P])
    ws = lib.wbmm_backward_checkpoint_workspace_bytes
    ws.restype, ws.argtypes = S, [I] * 6
    need = ws(2, 4, 28, 28, 14, 1)
    plain = lib.wbmm_backward_workspace_bytes
    plain.restype, plain.argtypes = S, [I] * 6
    assert need >= plain(2, 4, 28, 28, 14, 1) > 0
    assert ws(1, 1, 14, 15, 7, 1) == 0 and ws(1, 1, 14, 14, 7, 3) == 0
    exps = 0x60000000

    def call(codes=A0, exps=exps, T=A1, dY=A2, dX=A3, dT=A4, work=A4 + 0x100000, nbytes=need,
             shape=(2, 4, 28, 28, 14), dt=1):
        return f(codes, exps, T, dY, dX, dT, work, nbytes, *shape, dt, None)

    assert call(dt=2) == 3
    assert call(dY=None) == 1
    assert call(T=None) == 1
    assert call(codes=None) == 1
    assert call(exps=None) == 1
    assert call(shape=(2, 4, 28, 30, 14)) == 2
    assert call(shape=(2, 4, 28, 28, 0)) == 1
    assert call(codes=A0 + 8) == 4
    assert call(dX=A3 + 8) == 4
    assert call(dT=A4 + 2) == 4
    assert call(dX=A2 + 64) == 1
    assert call(dX=A0 + 64) == 1                         # dX overlaps the codes
    assert call(dT=exps) == 1                            # dT overlaps the exponents
    assert call(work=None) == 6
    assert call(nbytes=need - 4) == 6
    assert call(work=A4 + 0x100008) == 4
    assert call(work=A0 + 64) == 1
    assert call(work=A4 + 64) == 1
    assert call(dT=None, codes=None, exps=None, work=None, nbytes=0, dX=A3 + 8) == 4


def test_recurrence_argument_checks(lib):
    f = _proto(lib, "wbmm_scan_forward", [P] * 11 + [I] * 4 + [P])
    A = [0x10000000 * k for k in range(1, 13)]

    def fwd(v=A[0], g=A[1], h0=A[2], n=A[3], y=A[4], hT=A[5], st=A[6], vc=A[7], ve=A[8], gc=A[9], ge=A[10],
            shape=(2, 4, 100), dt=1):
        return f(v, g, h0, n, y, hT, st, vc, ve, gc, ge, *shape, dt, None)

    assert fwd(dt=2) == 3
    assert fwd(v=None) == 1 and fwd(g=None) == 1 and fwd(y=None) == 1
    assert fwd(vc=None) == 1 and fwd(ve=None) == 1 and fwd(gc=None) == 1 and fwd(ge=None) == 1
    for shape in ((0, 4, 100), (2, 0, 100), (2, 4, 0), (2, -1, 100)):
        assert fwd(shape=shape) == 1
    assert fwd(v=A[0] + 2) == 4 and fwd(y=A[4] + 8) == 4 and fwd(vc=A[7] + 4) == 4
    assert fwd(h0=A[2] + 2) == 4 and fwd(n=A[3] + 1) == 4 and fwd(st=A[6] + 2) == 4 and fwd(hT=A[5] + 2) == 4
    assert fwd(v=A[0] + 2, dt=0) == 4
    assert fwd(shape=(1 << 16, 1 << 15, 1), v=1 << 40, g=1 << 41, y=1 << 42, h0=None, n=None, hT=None, st=None,
               vc=None, ve=None, gc=None, ge=None) == 5
    assert fwd(shape=(1, 1, (1 << 31) - 65536), v=1 << 40, g=1 << 41, y=1 << 42, h0=None, n=None, hT=None, st=None,
               vc=None, ve=None, gc=None, ge=None) == 5
    assert fwd(y=A[0] + 16) == 1 and fwd(y=A[1]) == 1
    assert fwd(hT=A[2] + 4) == 1                          # in place only as a whole
    assert fwd(st=A[5]) == 1 and fwd(vc=A[9]) == 1 and fwd(hT=A[3]) == 1 and fwd(ge=A[4] + 1599) == 1

    b = _proto(lib, "wbmm_scan_backward", [P] * 9 + [I] * 4 + [P])

    def bwd(v=A[0], g=A[1], st=A[2], n=A[3], dy=A[4], dhT=A[5], dv=A[6], dg=A[7], dh0=A[8], shape=(2, 4, 100), dt=1):
        return b(v, g, st, n, dy, dhT, dv, dg, dh0, *shape, dt, None)

    assert bwd(dt=5) == 3
    for k in ("v", "g", "st", "dy", "dv", "dg"):
        assert bwd(**{k: None}) == 1
    assert bwd(shape=(2, 4, -3)) == 1
    assert bwd(v=A[0] + 2) == 4 and bwd(dg=A[7] + 2) == 4 and bwd(dh0=A[8] + 2) == 4
    assert bwd(dv=A[0]) == 1 and bwd(dv=A[4]) == 1 and bwd(dg=A[6]) == 1 and bwd(dh0=A[2]) == 1
    assert bwd(dh0=A[5] + 4) == 1

    c = _proto(lib, "wbmm_scan_backward_checkpoint", [P] * 11 + [I] * 4 + [P])

    def bwd8(vc=A[0], ve=A[1], gc=A[2], ge=A[3], st=A[4], n=A[5], dy=A[6], dhT=A[7], dv=A[8], dg=A[9], dh0=A[10],
             shape=(2, 4, 100), dt=1):
        return c(vc, ve, gc, ge, st, n, dy, dhT, dv, dg, dh0, *shape, dt, None)

    assert bwd8(dt=5) == 3
    for k in ("vc", "ve", "gc", "ge", "st", "dy", "dv", "dg"):
        assert bwd8(**{k: None}) == 1
    assert bwd8(vc=A[0] + 8) == 4 and bwd8(gc=A[2] + 1) == 4
    assert bwd8(dv=A[0]) == 1 and bwd8(dg=A[3]) == 1 and bwd8(dh0=A[1]) == 1

    s = _proto(lib, "wbmm_scan_step", [P] * 5 + [I] * 3 + [P])
    assert s(A[0], A[1], A[2], A[3], A[4], 2, 4, 3, None) == 3
    assert s(A[0], A[1], None, A[3], A[4], 2, 4, 1, None) == 1
    assert s(A[0], A[1], A[2], A[3], None, 2, 4, 1, None) == 1
    assert s(A[0], A[1], A[2], A[3], A[4], 2, 0, 1, None) == 1
    assert s(A[0] + 8, A[1], A[2], A[3], A[4], 2, 4, 1, None) == 4
    assert s(A[0], A[1], A[2] + 2, A[3], A[4], 2, 4, 1, None) == 4
    assert s(A[0], A[1], A[2], A[0], A[4], 2, 4, 1, None) == 1
    assert s(A[0], A[1], A[2], A[3], A[2] + 8, 2, 4, 1, None) == 1

    n = lib.wbmm_scan_states_bytes
    n.restype, n.argtypes = S, [I] * 3
    assert n(2, 3, 1) == 24 and n(2, 3, 256) == 24 and n(2, 3, 257) == 48 and n(1, 1, (1 << 31) - 1) == 4 << 23
    assert n(0, 3, 1) == 0 and n(2, -3, 1) == 0 and n(2, 3, 0) == 0
