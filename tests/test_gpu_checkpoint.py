"""GPU parity of the 8-bit checkpoints of maps and of the WBMM backward that
reads them: codes and exponents equal the fp64 oracle's, restored values are
exact, dT equals the backward of the restored map bit for bit and meets the
oracle within every parity test's tolerances; and one training step with all
of them together."""
import numpy as np
import pytest
import torch

import oracle
import synth
from oracle import recurrence as orc
from parity_util import check_bf16, check_f32, dt_bound, forward_rowbound, to_np
from scan_util import bounds

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import windowed_matmul_conv_b200 as wb  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
DEV = "cuda:0"


def gen(shape, seed, kind, scale=1.0):
    return synth.draw_tensor(shape, seed, "f32", scale).to(DT[kind]).to(DEV)


SHAPES = [
    (2, 3, 28, 28, 14), (9, 3, 56, 56, 14), (1, 2, 14, 14, 14), (3, 2, 14, 42, 14),
    (2, 4, 35, 49, 7), (1, 5, 7, 7, 7), (2, 2, 40, 24, 8), (3, 2, 40, 40, 5), (2, 3, 9, 15, 3),
    (2, 3, 5, 7, 1), (1, 2, 8, 6, 2), (2, 2, 39, 13, 13), (1, 2, 32, 48, 16), (1, 1, 56, 84, 28),
    (1, 2, 31, 62, 31), (1, 1, 64, 128, 64), (1, 1, 7, 700, 7), (2, 1, 14, 1400, 14), (1, 1, 40, 4000, 40),
]


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_codes_and_restored_values(shape, kind):
    B, C, H, W, w = shape
    x = gen((B, C, H, W), 1, kind)
    x = (x * torch.exp(4 * gen((B, C, 1, 1), 2, "fp32"))).to(DT[kind])
    codes, exps = wb.checkpoint(x, w)
    back = wb.checkpoint_restore(codes, exps, x.shape, w, x.dtype)
    torch.cuda.synchronize()
    wc, we = orc.encode(orc.windows(to_np(x), w))
    assert np.array_equal(exps.cpu().numpy(), we)
    assert np.array_equal(codes.cpu().numpy(), wc)
    assert np.array_equal(to_np(back), orc.unwindows(orc.decode(wc, we), x.shape, w))
    again = wb.checkpoint(back, w)
    assert torch.equal(again[0], codes) and torch.equal(again[1], exps)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("w", [3, 7, 14, 28])
def test_special_values(w, kind):
    """Zeros, denormals, values next to the type's largest, ties, NaN and
    infinities, one kind a window; the other windows keep theirs."""
    x = gen((1, 2, 2 * w, 4 * w), 3, kind)
    big = torch.finfo(DT[kind]).max
    x[0, 0, :w, :w] = 0
    x[0, 0, :w, w:2 * w] = 1e-40
    x[0, 0, 0, w] = -1e-38
    x[0, 0, :w, 2 * w:3 * w] *= 1e37
    x[0, 0, 1, 2 * w] = big
    x[0, 0, 2, 3 * w - 1] = -big
    x[0, 0, :w, 3 * w:] = 0.5
    x[0, 0, 0, 3 * w:3 * w + 3] = torch.tensor([64.0, 2.5, -1.5], device=DEV).to(DT[kind])
    x[0, 1, w - 1, w - 1] = float("nan")
    x[0, 1, w, w] = float("-inf")
    codes, exps = wb.checkpoint(x, w)
    back = wb.checkpoint_restore(codes, exps, x.shape, w, x.dtype)
    wc, we = orc.encode(orc.windows(x.detach().double().cpu().numpy(), w))
    assert np.array_equal(exps.cpu().numpy(), we) and np.array_equal(codes.cpu().numpy(), wc)
    want = orc.unwindows(orc.decode(wc, we), x.shape, w)
    assert np.array_equal(back.double().cpu().numpy(), want, equal_nan=True)
    assert np.isnan(want).sum() == 2 * w * w


def test_checkpoint_guards():
    for kind in ("bf16", "fp32"):
        for B, C, H, W, w in ((2, 3, 35, 49, 7), (1, 3, 28, 42, 14), (1, 1, 5, 5, 5)):
            x = gen((B, C, H, W), 5, kind)
            n, m = x.numel(), x.numel() // (w * w)
            codes = torch.full((n + 64,), 7, dtype=torch.uint8, device=DEV)
            exps = torch.full((m + 65,), 7, dtype=torch.uint8, device=DEV)
            out = torch.full((n + 64,), 7, dtype=DT[kind], device=DEV)
            wb.wbmm_checkpoint(x, codes, exps[1:], w)     # exponents at an odd address
            wb.wbmm_checkpoint_restore(codes, exps[1:], out[:n].view(x.shape), w)
            torch.cuda.synchronize()
            assert (codes[n:] == 7).all() and (exps[1 + m:] == 7).all() and exps[0] == 7
            assert (out[n:] == 7).all()
            want = wb.checkpoint(x, w)
            assert torch.equal(codes[:n], want[0].reshape(-1))
            assert torch.equal(exps[1:m + 1], want[1].reshape(-1))


BWD_SHAPES = [s for s in SHAPES if s[4] in (2, 3, 5, 7, 8, 13, 14, 16)] + [
    (2, 2, 28, 28, 28), (5, 2, 105, 112, 7), (4, 2, 39, 104, 13), (2, 2, 24, 96, 12), (3, 3, 48, 64, 16),
    (1, 9, 7, 56, 7), (3, 5, 7, 8, 1), (2, 2, 63, 63, 9), (5, 3, 42, 28, 14), (1, 3, 14, 28, 14)] + [
    (3, 2, 2 * w, 8 * w, w) for w in range(2, 17)]


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", BWD_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_backward_from_checkpoint(shape, kind):
    B, C, H, W, w = shape
    x, dy = gen((B, C, H, W), 6, kind), gen((B, C, H, W), 7, kind)
    T = gen((C, (2 * w - 1) ** 2), 8, kind, 0.02)
    codes, exps = wb.checkpoint(x, w)
    xh = wb.checkpoint_restore(codes, exps, x.shape, w, x.dtype)
    dX, dT = wb.backward_checkpoint(codes, exps, T, dy, w)
    torch.cuda.synchronize()
    assert wb.wbmm_get_device_status() == 0
    pX, pT = wb.backward(xh, T, dy, w)
    assert torch.equal(dX, pX) and torch.equal(dT, pT)
    only_x = wb.backward_checkpoint(None, None, T, dy, w, need_dt=False)
    assert only_x[1] is None
    assert torch.equal(only_x[0], wb.backward(None, T, dy, w, need_dt=False)[0])
    only_t = wb.backward_checkpoint(codes, exps, None, dy, w, need_dx=False)
    assert only_t[0] is None
    assert torch.equal(only_t[1], wb.backward(xh, None, dy, w, need_dx=False)[1])
    if H * W * B > 40000 and w > 14:
        return
    xr, gr, Tr = to_np(xh), to_np(dy), to_np(T)
    if kind == "bf16":
        check_bf16(to_np(dX), oracle.backward_dx(gr, Tr, w), forward_rowbound(gr, Tr[:, ::-1].copy(), w), "dX")
        check_bf16(to_np(dT), oracle.backward_dt(xr, gr, w), dt_bound(xr, gr, w), "dT")
    else:
        check_f32(to_np(dX), oracle.backward_dx(gr, Tr, w), oracle.backward_dx(np.abs(gr), np.abs(Tr), w), "dX")
        check_f32(to_np(dT), oracle.backward_dt(xr, gr, w), oracle.backward_dt(np.abs(xr), np.abs(gr), w), "dT")


def test_bad_windows_reach_the_table_gradient():
    """A window that overflowed gives NaN in its channel's dT, no other."""
    for shape in ((4, 3, 28, 28, 14), (2, 3, 15, 20, 5)):
        B, C, H, W, w = shape
        x, dy = gen((B, C, H, W), 6, "bf16"), gen((B, C, H, W), 7, "bf16")
        x[1, 1, 0, 0] = float("inf")
        codes, exps = wb.checkpoint(x, w)
        _, dT = wb.backward_checkpoint(codes, exps, None, dy, w, need_dx=False)
        assert torch.isnan(dT[1]).all() and torch.isfinite(dT[0]).all() and torch.isfinite(dT[2]).all()


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_workspace_shared_by_calls_and_graphs(kind):
    """One workspace for calls of several shapes, of wbmm_backward and of
    wbmm_backward_checkpoint, eager and captured, one after the other."""
    cases = []
    for k, (B, C, H, W, w) in enumerate(((5, 6, 56, 56, 14), (2, 3, 35, 49, 7), (9, 2, 56, 56, 14))):
        x, dy = gen((B, C, H, W), 10 + k, kind), gen((B, C, H, W), 20 + k, kind)
        T = gen((C, (2 * w - 1) ** 2), 30 + k, kind, 0.02)
        codes, exps = wb.checkpoint(x, w)
        want = wb.backward_checkpoint(codes, exps, T, dy, w)
        dX, dT = torch.empty_like(dy), torch.empty_like(want[1])
        cases.append((codes, exps, T, dy, dX, dT, w, want, x))
    need = max(max(wb.wbmm_backward_checkpoint_workspace_bytes(*c[3].shape, c[6], DT[kind]),
                   wb.wbmm_backward_workspace_bytes(*c[3].shape, c[6], DT[kind])) for c in cases)
    ws = torch.zeros(need // 4 + 1, device=DEV)
    graphs = []
    for codes, exps, T, dy, dX, dT, w, want, x in cases:
        wb.wbmm_backward_checkpoint(codes, exps, T, dy, dX, dT, ws, w)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            wb.wbmm_backward_checkpoint(codes, exps, T, dy, dX, dT, ws, w)
        graphs.append(g)
    for _ in range(3):
        for g, (codes, exps, T, dy, dX, dT, w, want, x) in zip(graphs, cases):
            dX.zero_(), dT.zero_()
            g.replay()
            wb.wbmm_backward(x, T, dy, torch.empty_like(dX), torch.empty_like(dT), ws, w)
            torch.cuda.synchronize()
            assert torch.equal(dX, want[0]) and torch.equal(dT, want[1])
    assert (ws[:65536].view(torch.int32) == 0).all()


def test_training_step_together():
    """WBMM, then the gated recurrence over its map, then both backward passes
    from 8-bit checkpoints, against the oracle on the same tensors; captured
    and replayed it gives the same bits."""
    B, C, H, W, w = 4, 6, 56, 56, 14
    x = gen((B, C, H, W), 41, "bf16")
    T = gen((C, (2 * w - 1) ** 2), 42, "bf16", 0.05)
    K = gen((C, 1, 3, 3), 43, "bf16", 0.3)
    g, dz = gen((B, C, H, W), 44, "bf16"), gen((B, C, H, W), 45, "bf16")

    def step():
        codes, exps = wb.checkpoint(x, w)
        y = wb.forward(x, T, w)
        z, hT, saved = wb.scan_forward_train(y, g, checkpoint=True)
        dy, dg, _ = wb.scan_backward(saved, dz)
        dX, dT = wb.backward_checkpoint(codes, exps, T, dy, w)
        return codes, exps, y, z, hT, dy, dg, dX, dT, wb.dw3x3(z, K)

    out = step()
    torch.cuda.synchronize()
    assert wb.wbmm_get_device_status() == 0
    codes, exps, y, z, hT, dy, dg, dX, dT, _ = out
    flat = (B, C, H * W)
    rz, rh = orc.scan(to_np(y).reshape(flat), to_np(g).reshape(flat))
    v8, g8 = (orc.seq_decode(*orc.seq_encode(to_np(t).reshape(flat))) for t in (y, g))
    rdv, rdg, _ = orc.scan_backward(v8, g8, to_np(dz).reshape(flat), states=rh[:, :, 0:H * W:orc.TILE])
    tol = bounds(to_np(y).reshape(flat), to_np(g).reshape(flat), "bf16", None, None,
                 to_np(dz).reshape(flat), None, v8, g8)
    for got, want, t in ((z, rz, "y"), (dy, rdv, "dv"), (dg, rdg, "dg")):
        assert (np.abs(to_np(got).reshape(flat) - want) <= tol[t]).all(), t
    xh, gr, Tr = to_np(wb.checkpoint_restore(codes, exps, x.shape, w, x.dtype)), to_np(dy), to_np(T)
    check_bf16(to_np(dX), oracle.backward_dx(gr, Tr, w), forward_rowbound(gr, Tr[:, ::-1].copy(), w), "dX")
    check_bf16(to_np(dT), oracle.backward_dt(xh, gr, w), dt_bound(xh, gr, w), "dT")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = step()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, cap):
        assert torch.equal(a, b)


@pytest.mark.parametrize("shape", [(5, 6, 56, 56, 14), (64, 256, 28, 28, 14), (2, 3, 35, 49, 7), (1, 3, 14, 28, 14)],
                         ids=lambda s: "x".join(map(str, s)))
def test_workspace_content_does_not_matter(shape):
    """Channels split between CTAs and whole ones, both gradients and dT alone,
    on a workspace full of garbage."""
    B, C, H, W, w = shape
    for kind in ("bf16", "fp32"):
        x, dy = gen((B, C, H, W), 51, kind), gen((B, C, H, W), 52, kind)
        T = gen((C, (2 * w - 1) ** 2), 53, kind, 0.02)
        codes, exps = wb.checkpoint(x, w)
        xh = wb.checkpoint_restore(codes, exps, x.shape, w, x.dtype)
        n = wb.wbmm_backward_checkpoint_workspace_bytes(B, C, H, W, w, DT[kind])
        ws = torch.full((n,), 0x7f, dtype=torch.uint8, device=DEV)
        for dx in (True, False):
            want = wb.backward(xh, T, dy, w, need_dx=dx)
            dX = torch.empty_like(dy) if dx else None
            dT = torch.empty_like(want[1])
            wb.wbmm_backward_checkpoint(codes, exps, T, dy, dX, dT, ws, w)
            assert torch.equal(dT, want[1]) and (not dx or torch.equal(dX, want[0]))
            ws.fill_(0x7f)


def test_offsets_past_32_bits():
    """A map of more than 2^31 elements: the codes of its last image, and the
    table gradient of the whole."""
    B, C, H, W, w = 700, 64, 224, 224, 14
    x = torch.zeros((B, C, H, W), dtype=torch.bfloat16, device=DEV)
    x[-1] = gen((1, C, H, W), 61, "bf16")[0]
    codes, exps = wb.checkpoint(x, w)
    want = wb.checkpoint(x[-1:].contiguous(), w)
    n = (H // w) * (W // w)
    assert torch.equal(codes[:, -n:], want[0]) and torch.equal(exps[:, -n:], want[1])
    assert (codes[:, :-n] == 128).all() and (exps[:, :-n] == 1).all()
    back = wb.checkpoint_restore(codes, exps, x.shape, w, x.dtype)
    assert torch.equal(back[-1:], wb.checkpoint_restore(*want, (1, C, H, W), w, x.dtype))
    assert (back[:-1] == 0).all()
    dy = torch.zeros_like(x)
    dy[-1] = gen((1, C, H, W), 62, "bf16")[0]
    _, dT = wb.backward_checkpoint(codes, exps, None, dy, w, need_dx=False)
    _, pT = wb.backward(back, None, dy, w, need_dx=False)
    assert torch.equal(dT, pT) and dT.abs().max() > 0
