"""Convenience calls on a given stream: the results are those of a call on the
current stream, outputs and workspaces are that stream's memory, and the
current stream's own allocations meanwhile change nothing."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import windowed_matmul_conv_b200 as wb  # noqa: E402

DEV = "cuda:0"


def pool_of(t):
    """The stream whose memory pool a tensor's block belongs to."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not an allocation")


def flat(out):
    for t in out if isinstance(out, tuple) else (out,):
        if isinstance(t, tuple):
            yield from flat(t)
        elif t is not None:
            yield t


def test_every_call_on_a_given_stream(monkeypatch):
    gen = torch.Generator(device=DEV).manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV).to(torch.bfloat16)
    B, C, H, W, w = 8, 24, 56, 56, 14
    x, dY, g, T, Tk = normal(B, C, H, W), normal(B, C, H, W), normal(B, C, H, W), normal(C, 729), normal(C, 169)
    K, M = normal(C, 1, 3, 3), wb.cache_matrices(T, w)
    codes, exps = wb.checkpoint(x, w)
    saved = wb.scan_forward_train(x, g, checkpoint=True)[2]
    h = torch.zeros(B, C, device=DEV)
    step = x[:, :, 0, 0].contiguous()
    calls = [lambda s: wb.forward(x, T, w, s), lambda s: wb.backward(x, T, dY, w, stream=s),
             lambda s: wb.cache_matrices(T, w, s), lambda s: wb.reparam_merge(T, Tk, w, 7, s),
             lambda s: wb.forward_cached(x, M, w, K, s), lambda s: wb.dw3x3(x, K, s),
             lambda s: wb.checkpoint(x, w, s),
             lambda s: wb.checkpoint_restore(codes, exps, x.shape, w, x.dtype, s),
             lambda s: wb.backward_checkpoint(codes, exps, T, dY, w, stream=s),
             lambda s: wb.scan_forward(x, g, h, stream=s),
             lambda s: wb.scan_forward_train(x, g, h, checkpoint=True, stream=s)[:2],
             lambda s: wb.scan_backward(saved, dY, h, stream=s), lambda s: wb.scan_step(step, step, h, s)]
    spaces = []
    for name, at in (("wbmm_backward", 5), ("wbmm_backward_checkpoint", 6)):
        def note(*a, _call=getattr(wb, name), _at=at):
            spaces.append(pool_of(a[_at]))
            return _call(*a)
        monkeypatch.setattr(wb, name, note)
    want = [list(flat(c(None))) for c in calls]
    own = {pool_of(t) for ts in want for t in ts}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    assert s.cuda_stream not in own
    del spaces[:]
    for _ in range(3):
        got = []
        for call in calls:
            got.append(list(flat(call(s))))
            # what the current stream is given now must not be the call's
            for n in (1 << 12, 1 << 19, 1 << 22):
                torch.full((n,), 255, dtype=torch.uint8, device=DEV)
        s.synchronize()
        for ts, ws in zip(got, want):
            assert len(ts) == len(ws)
            for a, b in zip(ts, ws):
                assert torch.equal(a, b) and pool_of(a) == s.cuda_stream
    assert spaces == [s.cuda_stream] * 6


def test_a_given_stream_is_checked():
    x = torch.zeros(1, 2, 14, 14, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    with pytest.raises(ValueError):
        wb.checkpoint(x.cpu(), 14, s)
    with pytest.raises(wb.WbmmError) as e:
        wb.scan_forward(x, x[:, :1].contiguous(), stream=s)
    assert e.value.status == 1
    assert torch.cuda.current_stream() != s
