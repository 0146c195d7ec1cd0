"""A map that holds no whole window is refused for its shape, as by every
other call, although it has no exponent bytes to point to.  No GPU."""
import pytest
import torch

from test_binding_missing import on_device, wb  # noqa: F401


@pytest.mark.parametrize("shape", [(1, 1, 5, 5), (2, 3, 28, 5), (2, 3, 5, 28)])
def test_checkpoint_of_a_map_smaller_than_a_window(wb, monkeypatch, shape):  # noqa: F811
    monkeypatch.setattr(wb, "_stream", lambda s, ref=None: None)
    x = on_device(*shape)
    with pytest.raises(wb.WbmmError) as e:
        wb.forward(x, on_device(shape[1], 169), 7)
    assert e.value.status == 2
    with pytest.raises(wb.WbmmError) as e:
        wb.checkpoint(x, 7)
    assert e.value.status == 2
    for w in (0, -7):
        with pytest.raises(wb.WbmmError) as e:
            wb.checkpoint(x, w)
        assert e.value.status == 1
