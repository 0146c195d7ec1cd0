"""The gated recurrence in fp64 torch, all rows at once on any device, and
error bounds of its kernels (test infrastructure; held to the step-by-step
oracle by tests/test_recurrence_f64.py).

U = 2^-24 is half a step of fp32, relative to a value.  The kernels' gates are
e = 2^(-g log2 e) by ex2.approx (relative error at most 2^-22 = 4U), then
f = rcp.approx(1 + e) (an ulp, at most 2U, beside the sum's U) and i = e f:
  fp32: the exponent's rounding and the constant's next bits are put back by
        one fma (U); what is left of the correction is its square, below
        2^-35:                                        eps_e = 5.1 U
  bf16: the product -g log2 e is rounded (|t| U in the exponent) and the
        constant is off by 0.23 U of itself; times ln 2, in e:
                                                      eps_e = (4 + 1.23 |g|) U
so f is off by i eps_e + 3U and i by eps_e + 4U.

A state is the sum over k of i_k v_k prod f_j.  A term meets at most one
multiplication and one addition a position that it passes, and 3 roundings for
each of the at most 13 joins of its tile (8 steps in a lane, 5 exchanges).  The
running bound takes 4U a position, 2U more than these need, so that the 512 U
left over in a tile cover a join of tiles; the 13 joins of the first tile are
40 U at every read-out:
  b_t = f_t b_{t-1} + f_t a_{t-1} (i eps_e + 3U + 4U) + |src_t| (eps_src + 4U),
a the same recurrence over magnitudes.
"""
import torch

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}      # half a step, relative
TILE, GROUP = 256, 64


def recur(a, b, start=None):
    """h_t = a_t h_{t-1} + b_t along the last axis, by doubling."""
    if start is not None:
        b = torch.cat([b[..., :1] + a[..., :1] * start[..., None], b[..., 1:]], dim=-1)
    L, d = a.shape[-1], 1
    while d < L:
        b = torch.cat([b[..., :d], b[..., d:] + a[..., d:] * b[..., :-d]], dim=-1)
        a = torch.cat([a[..., :d], a[..., d:] * a[..., :-d]], dim=-1)
        d *= 2
    return b


def live(x, lengths):
    if lengths is None:
        return torch.ones_like(x, dtype=torch.bool)
    at = torch.arange(x.shape[-1], device=x.device)
    return (at[None, None] < lengths.to(x.device)[:, None, None]).expand_as(x)


def gates(g, on):
    f, i = 1.0 / (1.0 + torch.exp(-g)), 1.0 / (1.0 + torch.exp(g))
    return torch.where(on, f, 1.0), torch.where(on, i, 0.0)


def through_8_bits(x, lengths):
    """x as its 8-bit form keeps it: groups of 64 positions share the smallest
    step 2^e with max |x| < 127.5 steps, -126 <= e <= 121."""
    x = torch.where(live(x, lengths), x, 0.0)
    L = x.shape[-1]
    a = torch.nn.functional.pad(x, (0, -L % GROUP)).unflatten(-1, (-1, GROUP))
    m, e = torch.frexp(a.abs().amax(dim=-1))
    e = torch.where(128.0 * m < 127.5, e - 7, e - 6)
    e = torch.where(m > 0, e, -126).clamp(-126, 121)
    q = torch.round(torch.ldexp(a, -e[..., None])).clamp(-127, 127)
    codes = (q + 128).to(torch.uint8).flatten(-2)[..., :L].contiguous()
    return torch.ldexp(q, e[..., None]).flatten(-2)[..., :L], codes, (e + 127).to(torch.uint8)


def _starts(h0, h):
    return h0.double() if h0 is not None else torch.zeros_like(h[..., 0])


def _before(h, start):
    return torch.cat([start[..., None], h[..., :-1]], dim=-1)


def _tiles(x, fill):
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % TILE), value=fill).unflatten(-1, (-1, TILE))


def _replay(f, src, into):
    """States before every position, each tile started from `into`."""
    L = f.shape[-1]
    h = recur(_tiles(f, 1.0), _tiles(src, 0.0), into)
    return torch.cat([into[..., None], h[..., :-1]], dim=-1).flatten(-2)[..., :L]


def _eps_e(g, kind):
    return 5.1 * U * torch.ones_like(g) if kind == "fp32" else (4.0 + 1.23 * g.abs()) * U


def forward(v, g, h0, lengths, kind):
    """Values and allowed errors: dict of name -> (value, tolerance)."""
    v, g, on = v.double(), g.double(), live(v, lengths)
    v, g = torch.where(on, v, 0.0), torch.where(on, g, 0.0)
    f, i = gates(g, on)
    start = _starts(h0, v)
    h = recur(f, i * v, start)
    ee = _eps_e(g, kind)
    src = i * v.abs()
    a = recur(f, src, start.abs())
    ap = _before(a, start.abs())
    b = recur(f, torch.where(on, f * ap * (i * ee + 7 * U), 0.0) + src * (ee + 9 * U))
    tol = b + 40 * U * a
    every = slice(None, None, TILE)
    zero = torch.zeros_like(start)
    return dict(y=(torch.where(on, h, 0.0), torch.where(on, tol + HALF[kind] * (a + tol), 0.0)),
                hT=(h[..., -1], tol[..., -1]),
                states=(_before(h, start)[..., every], _before(tol, zero)[..., every]),
                magnitudes=ap[..., every])


def backward(fwd, v, g, dY, dhT, lengths, kind):
    """From forward()'s result; v and g as the backward pass has them."""
    on = live(v, lengths)
    v, g, dY = (torch.where(on, x.double(), 0.0) for x in (v, g, dY))
    f, i = gates(g, on)
    ee = _eps_e(g, kind)
    into, into_tol = fwd["states"]
    mag = fwd["magnitudes"]
    src = i * v.abs()
    before = _replay(f, i * v, into)
    ap = _replay(f, src, mag)
    bp = _replay(f, torch.where(on, f * ap * (i * ee + 7 * U), 0.0) + src * (ee + 9 * U), into_tol)
    before_tol = bp + 40 * U * ap
    end = _starts(dhT, v)

    def back(a, b, s):
        return recur(a.flip(-1), b.flip(-1), s).flip(-1)

    def after(c, s):
        return torch.cat([c[..., 1:], s[..., None]], dim=-1)
    c = back(f, f * dY, end)
    dh = dY + after(c, end)
    srcc = f * dY.abs()
    ac = back(f, srcc, end.abs())
    an = after(ac, end.abs())
    bc = back(f, torch.where(on, f * an * (i * ee + 7 * U), 0.0) + srcc * (i * ee + 8 * U), torch.zeros_like(end))
    bc = bc + 40 * U * ac
    dha = dY.abs() + an
    dhb = after(bc, torch.zeros_like(end)) + 2 * U * dha
    dva = i * dha
    dvb = i * dhb + dva * (ee + 8 * U)
    gap = ap + v.abs()
    dga = f * dva * gap
    dgb = f * dvb * gap + dva * f * (before_tol + 2 * U * gap) + dga * (i * ee + 12 * U)

    def out(x, tol, m):
        return torch.where(on, x, 0.0), torch.where(on, tol + HALF[kind] * (m + tol), 0.0)
    return dict(dv=out(i * dh, dvb, dva), dg=out(f * i * (before - v) * dh, dgb, dga), dh0=(c[..., 0], bc[..., 0]))
