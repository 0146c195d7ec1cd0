"""The convenience functions' `stream` argument: outputs and workspaces come
from that stream's memory.  From another stream's they would be handed out
again, or still be in use there, while the call's kernels run.  The library
and the streams are stand-ins; no GPU."""
import contextlib
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


class FakeStream:
    cuda_stream, device_index = 7, 0


class FakeLib:
    """Every entry point succeeds and notes the stream it was given."""

    def __init__(self, size):
        self.streams, self.size = [], size

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: self.size

        def call(*a):
            self.streams.append(a[-1])
            return 0
        return call


BF = torch.bfloat16
X = torch.zeros((2, 3, 28, 28), dtype=BF)
T = torch.zeros((3, 729), dtype=BF)
CODES, EXPS = torch.zeros(X.numel(), dtype=torch.uint8), torch.zeros(24, dtype=torch.uint8)
H = torch.zeros((2, 3))
S = X[:, :, 0, 0].contiguous()
M, K = torch.zeros((3, 196, 196), dtype=BF), torch.zeros((3, 1, 3, 3), dtype=BF)
STATES = torch.zeros((2, 3, 4))

CALLS = {
    "forward": lambda wb, s: wb.forward(X, T, 14, s),
    "backward": lambda wb, s: wb.backward(X, T, X, 14, stream=s),
    "cache_matrices": lambda wb, s: wb.cache_matrices(T, 14, s),
    "reparam_merge": lambda wb, s: wb.reparam_merge(T, T[:, :169].contiguous(), 14, 7, s),
    "forward_cached": lambda wb, s: wb.forward_cached(X, M, 14, stream=s),
    "dw3x3": lambda wb, s: wb.dw3x3(X, K, s),
    "checkpoint": lambda wb, s: wb.checkpoint(X, 14, s),
    "checkpoint_restore": lambda wb, s: wb.checkpoint_restore(CODES, EXPS, X.shape, 14, BF, s),
    "backward_checkpoint": lambda wb, s: wb.backward_checkpoint(CODES, EXPS, T, X, 14, stream=s),
    "scan_forward": lambda wb, s: wb.scan_forward(X, X, H, stream=s),
    "scan_forward_train": lambda wb, s: wb.scan_forward_train(X, X, H, stream=s),
    "scan_forward_train8": lambda wb, s: wb.scan_forward_train(X, X, H, checkpoint=True, stream=s),
    "scan_backward": lambda wb, s: wb.scan_backward(wb.ScanSaved(X, X, None, None, STATES, None), X, stream=s),
    "scan_step": lambda wb, s: wb.scan_step(S, S, H, s),
}


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("given", [False, True], ids=["current", "given"])
def test_allocations_are_made_on_the_calls_stream(wb, monkeypatch, name, given):
    current, seen = [], []

    @contextlib.contextmanager
    def use(stream):
        current.append(stream)
        yield
        current.pop()

    def noting(alloc):
        def call(*a, **k):
            seen.append(current[-1] if current else None)
            return alloc(*a, **k)
        return call

    lib = FakeLib(1 << 16)
    stream = FakeStream() if given else None
    monkeypatch.setattr(wb, "_lib", lib)
    monkeypatch.setattr(wb, "_p", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(wb, "_ptrs", lambda *ts: [None if t is None else t.data_ptr() for t in ts])
    monkeypatch.setattr(wb, "_stream", lambda s, ref=None: (s or (current or [None])[-1] or FakeStream).cuda_stream)
    monkeypatch.setattr(torch.cuda, "stream", use)
    for fn in ("empty", "zeros", "empty_like"):
        monkeypatch.setattr(torch, fn, noting(getattr(torch, fn)))
    monkeypatch.setattr(torch.Tensor, "new_empty", noting(torch.Tensor.new_empty))
    CALLS[name](wb, stream)
    assert seen and all(s is stream for s in seen)
    assert lib.streams == [7] and not current
