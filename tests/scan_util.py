"""Error bounds of the gated recurrence's kernels (test infrastructure).

U = 2^-24 is half a step of fp32, relative to a value.  With exp(-g) off by
eps_e, f = 1 / (1 + e) is off by i * eps_e + 2U and i = e f by eps_e + 3U
(relative; one rounding each of 1 + e, of its reciprocal and of the product;
the fast reciprocal of the bf16 path adds 2 ulp, 4U, to each).
  fp32 path: expf is within 2 ulp:               eps_e = 4U
  bf16 path: __expf within 2 + |1.173 g| ulp:    eps_e = 2U (2 + 1.173 |g|)
             (both documented bounds; an ulp is at most 2U relative)
A state is the sum over k of i_k v_k prod f_j, each product formed by one
multiplication a factor, in whatever order, and summed with one rounding an
addition; a term meets at most one multiplication and one addition for each
position it passes, besides 3 for each of the 13 joins of a tile (8 steps
within a lane, 5 exchanges).  So the running bound is
  b_t = f_t b_{t-1} + f_t a_{t-1} (i eps_e + 6U + 4U) + a_t' (eps_e + 7U + 4U),
a the same recurrence over magnitudes, plus 40U a_t once for the joins of each
tile (counted at every position's read-out, and carried by the recurrence from
tile to tile through the 4U of each step).
"""
import numpy as np

from oracle import recurrence as orc

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}      # half a step, relative


def eps_e(g, kind):
    return 4 * U if kind == "fp32" else 2 * U * (2 + 1.173 * np.abs(g))


def run_bound(f, i, src, src_err, start, kind, g):
    """Magnitudes a_t and bounds b_t of s_t = f_t s_{t-1} + src_t, along the
    last axis; src_err bounds src's own error, start is |s_{-1}| (exact)."""
    ee = eps_e(g, kind)
    a = np.zeros(f.shape[:2] + (f.shape[2] + 1,))
    b = np.zeros_like(a)
    a[:, :, 0] = start
    for t in range(f.shape[2]):
        ft, it = f[:, :, t], i[:, :, t]
        e = ee if np.isscalar(ee) else ee[:, :, t]
        on = it != 0
        a[:, :, t + 1] = ft * a[:, :, t] + src[:, :, t]
        b[:, :, t + 1] = (ft * b[:, :, t] + np.where(on, ft * a[:, :, t] * (it * e + 10 * U), 0.0)
                          + src_err[:, :, t] + 4 * U * src[:, :, t])
    return a, b


def bounds(v, g, kind, h0, lengths, dY=None, dhT=None, v8=None, g8=None):
    """Bounds of y and the states and, with dY, of dv, dg and dh0.  v8, g8: the
    inputs as the backward pass has them."""
    m = orc.masked(np.nan_to_num(v), lengths)
    f, i = orc.gates(np.nan_to_num(g), lengths)
    e = eps_e(np.nan_to_num(g), kind)
    src = i * np.abs(m)
    a, b = run_bound(f, i, src, src * (e + 7 * U), np.abs(h0) if h0 is not None else 0.0, kind,
                     np.nan_to_num(g))
    state = b + 40 * U * a
    out = {"h": state, "y": state[:, :, 1:] + HALF[kind] * (a + state)[:, :, 1:]}
    if dY is None:
        return out
    m = orc.masked(np.nan_to_num(v if v8 is None else v8), lengths)
    gg = np.nan_to_num(g if g8 is None else g8)
    f, i = orc.gates(gg, lengths)
    e = eps_e(gg, kind)
    # replayed states: the kept state's error, and the replay's own over
    # magnitudes that restart at each tile no larger than |state| there
    src = i * np.abs(m)
    before = np.zeros_like(f)
    L = f.shape[2]
    for t0 in range(0, L, orc.TILE):
        s = slice(t0, min(L, t0 + orc.TILE))
        aa, bb = run_bound(f[:, :, s], i[:, :, s], src[:, :, s],
                           src[:, :, s] * ((e if np.isscalar(e) else e[:, :, s]) + 7 * U),
                           a[:, :, t0], kind, gg[:, :, s])
        bb[:, :, 0] += 0
        carry = state[:, :, t0, None] * np.concatenate(
            [np.ones(f.shape[:2] + (1,)), np.cumprod(f[:, :, s], axis=2)], axis=2)
        before[:, :, s] = (bb + 40 * U * aa + carry)[:, :, :-1]
    mag = np.zeros_like(f)
    for t0 in range(0, L, orc.TILE):
        s = slice(t0, min(L, t0 + orc.TILE))
        aa, _ = run_bound(f[:, :, s], i[:, :, s], src[:, :, s], 0 * src[:, :, s], a[:, :, t0], kind,
                          gg[:, :, s])
        mag[:, :, s] = aa[:, :, :-1]
    d = np.abs(orc.masked(np.nan_to_num(dY), lengths))
    # c_t = f_t (dy_t + c_{t+1}): reversed, with source f_t dy_t
    r = slice(None, None, -1)
    srcc = f * d
    ie = i * e + 10 * U
    ac, bc = run_bound(f[:, :, r], i[:, :, r], srcc[:, :, r], (srcc * ie)[:, :, r],
                       np.abs(dhT) if dhT is not None else 0.0, kind, gg[:, :, r])
    bc = bc + 40 * U * ac
    after_a, after_b = ac[:, :, -2::-1], bc[:, :, -2::-1]      # c_{t+1}
    dh = d + after_a
    dh_b = after_b + 2 * U * dh
    dv = i * dh
    dv_b = i * dh_b + dv * (e + 8 * U)
    gap = mag + np.abs(m)
    dg = f * dv * gap
    dg_b = f * dv_b * gap + dv * f * (before + 2 * U * gap) + dg * (i * e + 12 * U)
    out["dv"] = dv_b + HALF[kind] * (dv + dv_b)
    out["dg"] = dg_b + HALF[kind] * (dg + dg_b)
    out["dh0"] = bc[:, :, -1]
    return out
