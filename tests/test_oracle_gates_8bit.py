"""What 8 bits cost a gate: f and 1 - f of a restored gate are within a factor
of exp(half its group's step) of the gate's own, by the definitions (no GPU)."""
import numpy as np
import pytest

from oracle import recurrence as orc


@pytest.mark.parametrize("shift,spread", [(0.0, 1.0), (6.0, 1.0), (-6.0, 1.0), (0.0, 8.0), (2.0, 30.0)])
def test_factor_of_a_restored_gate(shift, spread):
    g = shift + spread * np.random.default_rng(1).normal(size=(3, 4, 1000))
    codes, exps = orc.seq_encode(g)
    back = orc.seq_decode(codes, exps)
    half = np.repeat(np.ldexp(0.5, exps.astype(int) - 127), orc.SEQ_GROUP, axis=2)[:, :, :1000]
    slack = 1 + 1e-12                   # of the fp64 definitions
    for a, b in zip(orc.gates(g, None), orc.gates(back, None)):
        assert np.all(b <= a * np.exp(half) * slack) and np.all(a <= b * np.exp(half) * slack)


@pytest.mark.parametrize("top,percent", [(4.0, 3.2), (7.9, 3.2), (8.0, 6.5), (15.9, 6.5)])
def test_percentages_by_the_largest_gate(top, percent):
    step = np.ldexp(1.0, int(orc.group_step(top)))
    assert np.expm1(step / 2) <= percent / 100


def test_small_groups_are_within_half_the_smallest_step():
    a = np.ldexp(np.random.default_rng(2).normal(size=(50, 9)), np.arange(-160, -110)[:, None])
    back = orc.decode(*orc.encode(a))
    far, top = np.abs(back - a).max(axis=1), np.abs(a).max(axis=1)
    assert np.all(far <= np.maximum(2.0 ** -127, top / 127))
    assert (far > top / 127).any()      # where the exponent is at its end
