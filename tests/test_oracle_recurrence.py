"""Pins of the fp64 oracle of the 8-bit checkpoints and the gated recurrence:
closed forms, brute force and central differences (no GPU)."""
import numpy as np
import pytest

import oracle
from oracle import recurrence as orc


def rng(seed):
    return np.random.default_rng(seed)


# ------------------------------------------------------------- checkpoints

def test_group_step_by_brute_force():
    r = rng(0)
    tops = np.concatenate([np.exp(r.normal(0, 20, 200)), 2.0 ** np.arange(-130, 128),
                           127.5 * 2.0 ** np.arange(-30, 30), 127.49 * 2.0 ** np.arange(-30, 30), [0.0]])
    for top in tops:
        fits = [e for e in range(-126, 122) if np.rint(top * 2.0 ** -e) <= 127]
        assert orc.group_step(top) == (fits[0] if fits else 121), top


def test_codes_are_the_nearest_step():
    a = rng(1).normal(size=(50, 23)) * np.exp(rng(2).normal(0, 10, size=(50, 1)))
    codes, exps = orc.encode(a)
    back = orc.decode(codes, exps)
    step = 2.0 ** (exps.astype(float) - 127)
    assert np.all(np.abs(back - a) <= step[:, None] / 2)
    # half a step is at most 1/127 of the largest value, and no code is spare
    assert np.all(step / 2 <= np.abs(a).max(axis=1) / 127)
    assert np.all(np.abs(codes.astype(int) - 128).max(axis=1) >= 64)
    again = orc.encode(back)
    assert np.array_equal(again[0], codes) and np.array_equal(again[1], exps)


def test_special_groups():
    a = np.zeros((5, 4))
    a[1, 2] = np.nan
    a[2, 0] = -np.inf
    a[3] = [3.4e38, -3.4e38, 1e38, 0]
    a[4] = [1e-45, -1e-45, 0, 2.0 ** -126]
    codes, exps = orc.encode(a)
    assert list(exps) == [1, 255, 255, 248, 1]
    back = orc.decode(codes, exps)
    assert np.all(back[0] == 0) and np.isnan(back[1]).all() and np.isnan(back[2]).all()
    assert back[3, 0] == 127 * 2.0 ** 121 and back[3, 1] == -back[3, 0]
    assert list(back[4]) == [0, 0, 0, 2.0 ** -126]


def test_window_order_and_sequence_groups():
    x = np.arange(2 * 1 * 4 * 6, dtype=float).reshape(2, 1, 4, 6)
    a = orc.windows(x, 2)
    assert a.shape == (1, 12, 4)
    assert list(a[0, 1]) == [2, 3, 8, 9] and list(a[0, 3]) == [12, 13, 18, 19]
    assert list(a[0, 6]) == [24, 25, 30, 31]
    assert np.array_equal(orc.unwindows(a, x.shape, 2), x)
    s = rng(3).normal(size=(2, 3, 130))
    codes, exps = orc.seq_encode(s, [130, 70])
    assert exps.shape == (2, 3, 3)
    full = orc.encode(s[:, :, 64:128])
    assert np.array_equal(codes[0, :, 64:128], full[0][0])
    assert np.all(codes[1, :, 70:] == 128) and np.all(exps[1, :, 2] == 1)
    assert np.abs(orc.seq_decode(codes, exps)[0] - s[0]).max() < 4 / 127


# -------------------------------------------------------------- recurrence

def test_constant_gate_closed_form():
    # with f constant, h_t = f^(t+1) h0 + (1 - f^(t+1)) v
    g, v, h0 = 1.3, 0.7, -2.0
    f = 1 / (1 + np.exp(-g))
    y, h = orc.scan(np.full((1, 1, 40), v), np.full((1, 1, 40), g), np.full((1, 1), h0))
    want = f ** np.arange(1, 41) * h0 + (1 - f ** np.arange(1, 41)) * v
    assert np.allclose(y[0, 0], want, rtol=1e-13)
    assert h[0, 0, 0] == h0 and h[0, 0, -1] == y[0, 0, -1]


def test_open_and_shut_gates():
    v = rng(4).normal(size=(1, 2, 9))
    y, _ = orc.scan(v, np.full(v.shape, 800.0), np.full((1, 2), 3.0))
    assert np.all(y == 3.0)
    y, _ = orc.scan(v, np.full(v.shape, -800.0), np.full((1, 2), 3.0))
    assert np.array_equal(y, v)


def test_lengths_stop_a_sequence():
    v, g = rng(5).normal(size=(3, 2, 8)), rng(6).normal(size=(3, 2, 8))
    h0 = rng(7).normal(size=(3, 2))
    v[0, :, 5:] = np.nan
    y, h = orc.scan(v, g, h0, [5, 0, 8])
    assert np.array_equal(y[0, :, :5], orc.scan(v[:1, :, :5], g[:1, :, :5], h0[:1])[0][0])
    assert np.all(y[0, :, 5:] == 0) and np.all(y[1] == 0)
    assert np.array_equal(h[1, :, -1], h0[1]) and np.array_equal(h[0, :, -1], y[0, :, 4])


@pytest.mark.parametrize("lengths", [None, [6, 0]])
def test_backward_by_central_differences(lengths):
    r = rng(8)
    v, g = r.normal(size=(2, 2, 7)), r.normal(size=(2, 2, 7)) + 1
    h0, dY, dhT = r.normal(size=(2, 2)), r.normal(size=(2, 2, 7)), r.normal(size=(2, 2))

    def loss(v, g, h0):
        y, h = orc.scan(v, g, h0, lengths)
        return (y * dY).sum() + (h[:, :, -1] * dhT).sum()

    dv, dg, dh0 = orc.scan_backward(v, g, dY, dhT, h0, lengths)
    for x, d, k in ((v, dv, 0), (g, dg, 1), (h0, dh0, 2)):
        for at in np.ndindex(x.shape):
            args = [v.copy(), g.copy(), h0.copy()]
            args[k][at] += 1e-5
            up = loss(*args)
            args[k][at] -= 2e-5
            assert abs((up - loss(*args)) / 2e-5 - d[at]) < 1e-8


def test_backward_from_kept_states_is_the_same():
    r = rng(9)
    v, g, dY = (r.normal(size=(1, 2, 600)) for _ in range(3))
    _, h = orc.scan(v, g)
    a = orc.scan_backward(v, g, dY)
    b = orc.scan_backward(v, g, dY, states=h[:, :, 0:600:256])
    for p, q in zip(a, b):
        assert np.array_equal(p, q)
    # and a wrong state is noticed
    bad = h[:, :, 0:600:256].copy()
    bad[:, :, 1] += 1
    assert not np.allclose(orc.scan_backward(v, g, dY, states=bad)[1], a[1])


def test_planted_mistakes_fail():
    """The differences test above tells apart the usual slips of the backward
    formulas."""
    r = rng(10)
    v, g, dY = (r.normal(size=(1, 1, 6)) for _ in range(3))
    f, i = orc.gates(g, None)
    _, h = orc.scan(v, g)
    dv, dg, _ = orc.scan_backward(v, g, dY)
    c, wrong_state, wrong_carry = 0.0, [], []
    for t in range(5, -1, -1):
        dh = dY[0, 0, t] + c
        wrong_state.append(f[0, 0, t] * i[0, 0, t] * (h[0, 0, t + 1] - v[0, 0, t]) * dh)
        wrong_carry.append(i[0, 0, t] * dh)
        c = f[0, 0, t] * dY[0, 0, t]            # drops the carry
    assert not np.allclose(wrong_state[::-1], dg[0, 0])
    assert not np.allclose(wrong_carry[::-1], dv[0, 0])


def test_table_gradient_of_a_checkpoint():
    """dT from a checkpoint is linear in the restored map (the oracle's dT)."""
    x, dy = rng(11).normal(size=(2, 1, 6, 6)), rng(12).normal(size=(2, 1, 6, 6))
    xh = orc.unwindows(orc.decode(*orc.encode(orc.windows(x, 3))), x.shape, 3)
    far = oracle.backward_dt(x, dy, 3) - oracle.backward_dt(xh, dy, 3)
    assert np.allclose(far, oracle.backward_dt(x - xh, dy, 3))
    assert np.abs(x - xh).max() <= np.abs(x).max() / 127
