"""A missing buffer is the library's to refuse (WBMM_ERR_INVALID_ARG): the
binding passes None on as a null pointer, whichever argument it is.  CPU
tensors stand in for device tensors, and a stand-in for the library takes the
pointers."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, U8 = torch.bfloat16, torch.uint8


@pytest.fixture(scope="module")
def wb():
    spec = importlib.util.spec_from_file_location(
        "_wbmm_build", os.path.join(ROOT, "windowed_matmul_conv_b200", "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    build.build()
    import windowed_matmul_conv_b200 as mod
    return mod


class Tensor(torch.Tensor):
    is_cuda = True


def on_device(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype).as_subclass(Tensor)


def test_missing_buffers(wb, monkeypatch):
    lib, calls = wb._lib, []

    class Lib:
        def __getattr__(self, name):
            def call(*a):
                if name != "wbmm_status_string":
                    calls.append(name)
                return getattr(lib, name)(*a)       # refused before the device is touched
            return call
    monkeypatch.setattr(wb, "_lib", Lib())
    monkeypatch.setattr(wb, "_stream", lambda s, ref=None: None)
    x, h, n = on_device(2, 3, 300), on_device(2, 3, dtype=torch.float32), on_device(2, dtype=torch.int32)
    st, cd, ex = on_device(2, 3, 2, dtype=torch.float32), on_device(2, 3, 300, dtype=U8), on_device(2, 3, 5, dtype=U8)
    m, mc, me = on_device(2, 3, 28, 28), on_device(4704, dtype=U8), on_device(24, dtype=U8)
    s = on_device(2, 3)
    wanted = [(wb.wbmm_scan_forward, [x, x, h, n, x, h, st, cd, ex, cd, ex], (1, 4, 7, 8, 9, 10)),
              (wb.wbmm_scan_backward, [x, x, st, n, x, h, x, x, h], (0, 1, 2, 6, 7)),
              (wb.wbmm_scan_backward_checkpoint, [cd, ex, cd, ex, st, n, x, h, x, x, h], (0, 1, 2, 3, 4, 8, 9)),
              (wb.wbmm_scan_step, [s, s, h, s, h], (1, 2, 3, 4)),
              (wb.wbmm_checkpoint, [m, mc, me, 14], (1, 2)),
              (wb.wbmm_checkpoint_restore, [mc, me, m, 14], (0, 1))]
    for fn, args, needed in wanted:
        for k in needed:
            a = list(args)
            a[k] = None
            with pytest.raises(wb.WbmmError) as e:
                fn(*a)
            assert e.value.status == 1, (fn.__name__, k)
    assert len(calls) == sum(len(w[2]) for w in wanted)


def test_buffers_off_the_device_are_refused(wb):
    x, u8 = torch.zeros((2, 3, 28, 28), dtype=BF), torch.zeros(4704, dtype=U8)
    with pytest.raises(ValueError):
        wb.wbmm_checkpoint_restore(None, u8, x, 14)
    with pytest.raises(ValueError):
        wb.wbmm_scan_backward(None, x, torch.zeros((2, 3, 4)), None, x, None, x, x, None)
