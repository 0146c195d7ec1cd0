"""The table-gradient kernel's pipeline where it reads 8-bit codes: a skipped
tile load ends in a status that the host reads and leaves the workspace's
counters zero; results do not depend on the ring's depth, nor on a second call
on another stream."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import windowed_matmul_conv_b200 as wb  # noqa: E402

DEV = "cuda:0"
SHORT_BUDGET = 20_000_000       # SM cycles, about 10 ms


def make(B, C, H, W, w, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV).to(torch.bfloat16)
    x, dy, T = normal(B, C, H, W), normal(B, C, H, W), 0.02 * normal(C, (2 * w - 1) ** 2)
    return (*wb.checkpoint(x, w), T, dy, w)


@pytest.mark.parametrize("shape", [(9, 3, 56, 56, 14), (9, 3, 56, 56, 7)], ids=lambda s: "x".join(map(str, s)))
def test_a_skipped_load_ends_in_a_status(shape):
    """Channels are split between CTAs here, so that counters are in use."""
    B, C, H, W, w = shape
    codes, exps, _, dy, _ = make(*shape, 1)
    want = wb.backward_checkpoint(codes, exps, None, dy, w, need_dx=False)[1]
    assert torch.isfinite(want).all() and wb.wbmm_get_device_status() == 0
    n = wb.wbmm_backward_checkpoint_workspace_bytes(B, C, H, W, w, torch.bfloat16)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    dT = torch.empty_like(want)
    wb.wbmm_set_wait_budget(SHORT_BUDGET)
    try:
        wb.wbmm_debug_set(wb.WBMM_DEBUG_SKIP_LOAD_TABLE_GRAD, 0)
        wb.wbmm_backward_checkpoint(codes, exps, None, dy, None, dT, ws, w)
        assert wb.wbmm_get_device_status() == 8
        assert (ws[:4 * C] == 0).all()          # the counters of the call's channels
    finally:
        wb.wbmm_set_wait_budget(0)
        wb.wbmm_debug_set(wb.WBMM_DEBUG_SKIP_LOAD_TABLE_GRAD, -1)
        wb.wbmm_get_device_status()
    wb.wbmm_backward_checkpoint(codes, exps, None, dy, None, dT, ws, w)
    assert wb.wbmm_get_device_status() == 0
    assert torch.equal(dT, want)


@pytest.mark.parametrize("shape", [(9, 3, 56, 56, 14), (6, 8, 40, 40, 5), (64, 40, 56, 56, 14), (8, 96, 112, 112, 7)],
                         ids=lambda s: "x".join(map(str, s)))
def test_ring_depth_does_not_change_results(shape):
    codes, exps, T, dy, w = make(*shape, 2)

    def run():
        out = (*wb.backward_checkpoint(codes, exps, T, dy, w),
               wb.backward_checkpoint(codes, exps, None, dy, w, need_dx=False)[1])
        assert wb.wbmm_get_device_status() == 0
        return out
    want = run()
    try:
        wb.wbmm_debug_set(wb.WBMM_DEBUG_RING_CAP, 2)
        got = run()
    finally:
        wb.wbmm_debug_set(wb.WBMM_DEBUG_RING_CAP, 0)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    """Each call has a workspace of its own."""
    args = [make(*s, 3) for s in ((9, 12, 56, 56, 14), (8, 24, 56, 56, 7), (16, 8, 35, 49, 7))]
    want = [wb.backward_checkpoint(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    got = []
    for _ in range(6):
        for a, s in zip(args, streams):
            got.append(wb.backward_checkpoint(*a, stream=s))
    torch.cuda.synchronize()
    assert wb.wbmm_get_device_status() == 0
    for k, g in enumerate(got):
        for a, b in zip(g, want[k % len(args)]):
            assert torch.equal(a, b)
