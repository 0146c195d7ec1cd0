"""The fp64 torch form of the gated recurrence that the GPU tests use for many
rows, against the step-by-step oracle."""
import numpy as np
import pytest
import torch

import recurrence_f64 as ref
from oracle import recurrence as orc


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("L", [1, 2, 63, 64, 65, 256, 257, 700])
def test_agrees_with_the_oracle(L, ragged):
    gen = torch.Generator().manual_seed(L)
    B, C = 4, 3
    v, g, dY = (torch.randn(B, C, L, generator=gen, dtype=torch.float64) for _ in range(3))
    g = 2 * g + 1
    h0, dhT = (torch.randn(B, C, generator=gen, dtype=torch.float64) for _ in range(2))
    n = torch.tensor([0, L, (L + 1) // 2, L // 3], dtype=torch.int32) if ragged else None
    nn = None if n is None else n.numpy()
    y, h = orc.scan(v.numpy(), g.numpy(), h0.numpy(), nn)
    fwd = ref.forward(v, g, h0, n, "fp32")

    def same(got, want):
        assert np.allclose(got.numpy(), want, rtol=1e-12, atol=1e-13)
    same(fwd["y"][0], y)
    same(fwd["hT"][0], h[:, :, -1])
    same(fwd["states"][0], h[:, :, 0:L:orc.TILE])
    for a in (v, g):
        back, codes, exps = ref.through_8_bits(a * 10.0 ** torch.arange(-1, 2)[None, :, None], n)
        wc, we = orc.seq_encode((a * 10.0 ** torch.arange(-1, 2)[None, :, None]).numpy(), nn)
        assert np.array_equal(codes.numpy(), wc) and np.array_equal(exps.numpy(), we)
        assert np.array_equal(back.numpy(), orc.seq_decode(wc, we))
    for quantised in (False, True):
        vb, gb = (ref.through_8_bits(a, n)[0] for a in (v, g)) if quantised else (v, g)
        want = orc.scan_backward(vb.numpy(), gb.numpy(), dY.numpy(), dhT.numpy(), h0.numpy(), nn,
                                 h[:, :, 0:L:orc.TILE] if quantised else None)
        bwd = ref.backward(fwd, vb, gb, dY, dhT, n, "fp32")
        for name, w in zip(("dv", "dg", "dh0"), want):
            same(bwd[name][0], w)


def test_group_step_ties_and_ends():
    top = torch.tensor([127.5, 127.4999, 63.75, 0.0, 3e38, 1e-45, 2.0 ** -120, 255.0, 254.9], dtype=torch.float64)
    x = torch.zeros(1, 1, 64 * top.numel(), dtype=torch.float64)
    x[0, 0, ::64] = top
    assert list(ref.through_8_bits(x, None)[2][0, 0].numpy() - 127.0) == list(orc.group_step(top.numpy()))
