"""Oracle of the 8-bit checkpoints and of the gated recurrence: test
infrastructure only.

Plain fp64 numpy, step by step, sharing no code with
``windowed_matmul_conv_b200``.  Pinned by tests/test_oracle_recurrence.py
against closed forms, brute force and central differences.
"""
import numpy as np

SEQ_GROUP = 64
TILE = 256      # positions per kept state


def group_step(top):
    """The smallest e, -126 <= e <= 121, with rint(top / 2^e) <= 127."""
    top = np.asarray(top, dtype=np.float64)
    # top / 2^e is at least 256 where e is not at an end (frexp gives 0 for 0)
    e = np.where(top > 0, np.clip(np.frexp(top)[1] - 9, -126, 121), -126)
    while True:
        more = (e < 121) & (np.rint(np.ldexp(top, -e)) > 127)
        if not more.any():
            return e
        e = e + more


def encode(a):
    """Groups along the last axis of `a` -> uint8 codes, uint8 exponent bytes."""
    a = np.asarray(a, dtype=np.float64)
    bad = ~np.isfinite(a).all(axis=-1)
    a = np.where(bad[..., None], 0.0, a)
    e = group_step(np.abs(a).max(axis=-1))
    q = np.clip(np.rint(np.ldexp(a, -e[..., None])), -127, 127) + 128
    return q.astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def decode(codes, exps):
    e = exps.astype(np.int64)
    val = np.ldexp(codes.astype(np.float64) - 128.0, (e - 127)[..., None])
    val[e == 255] = np.nan
    return val


def windows(x, w):
    """[B,C,H,W] -> [C, B*nh*nw, w*w], windows in (b, i, j) order."""
    B, C, H, W = x.shape
    out = np.empty((C, B * (H // w) * (W // w), w * w), dtype=x.dtype)
    for c in range(C):
        n = 0
        for b in range(B):
            for i in range(0, H, w):
                for j in range(0, W, w):
                    out[c, n] = x[b, c, i:i + w, j:j + w].reshape(-1)
                    n += 1
    return out


def unwindows(a, shape, w):
    B, C, H, W = shape
    x = np.empty(shape, dtype=a.dtype)
    for c in range(C):
        n = 0
        for b in range(B):
            for i in range(0, H, w):
                for j in range(0, W, w):
                    x[b, c, i:i + w, j:j + w] = a[c, n].reshape(w, w)
                    n += 1
    return x


def seq_encode(x, lengths=None):
    """[B,C,L] -> codes [B,C,L], exponent bytes [B,C,ceil(L/64)]; positions
    behind a sequence's end count as zero."""
    x = masked(np.asarray(x, dtype=np.float64), lengths)
    B, C, L = x.shape
    pad = -L % SEQ_GROUP
    a = np.concatenate([x, np.zeros((B, C, pad))], axis=2).reshape(B, C, -1, SEQ_GROUP)
    codes, exps = encode(a)
    return codes.reshape(B, C, -1)[:, :, :L], exps


def seq_decode(codes, exps):
    B, C, L = codes.shape
    pad = -L % SEQ_GROUP
    a = np.concatenate([codes, np.full((B, C, pad), 128, np.uint8)], axis=2)
    return decode(a.reshape(B, C, -1, SEQ_GROUP), exps).reshape(B, C, -1)[:, :, :L]


def live(shape, lengths):
    B, C, L = shape
    n = np.full(B, L) if lengths is None else np.clip(np.asarray(lengths), 0, L)
    return np.broadcast_to(np.arange(L)[None, None] < n[:, None, None], shape)


def masked(x, lengths):
    return np.where(live(x.shape, lengths), x, 0.0)


def gates(g, lengths):
    """f and 1 - f; the identity step (1, 0) behind a sequence's end."""
    on = live(g.shape, lengths)
    with np.errstate(over="ignore"):
        f, i = 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))
    return np.where(on, f, 1.0), np.where(on, i, 0.0)


def scan(v, g, h0=None, lengths=None):
    """y [B,C,L], the state before every position and after the last
    [B,C,L+1]."""
    v, g = np.asarray(v, dtype=np.float64), np.asarray(g, dtype=np.float64)
    B, C, L = v.shape
    f, i = gates(g, lengths)
    u = i * masked(v, lengths)
    h = np.zeros((B, C, L + 1))
    if h0 is not None:
        h[:, :, 0] = h0
    for t in range(L):
        h[:, :, t + 1] = f[:, :, t] * h[:, :, t] + u[:, :, t]
    return masked(h[:, :, 1:], lengths), h


def scan_backward(v, g, dY, dhT=None, h0=None, lengths=None, states=None):
    """dv, dg, dh0.  With `states` [B,C,tiles], the state is set to them before
    every TILE-th position."""
    v, g = masked(np.asarray(v, np.float64), lengths), np.asarray(g, np.float64)
    B, C, L = v.shape
    f, i = gates(g, lengths)
    before = np.zeros((B, C, L))
    s = np.zeros((B, C)) if h0 is None else np.asarray(h0, np.float64)
    for t in range(L):
        if states is not None and t % TILE == 0:
            s = states[:, :, t // TILE]
        before[:, :, t] = s
        s = f[:, :, t] * s + i[:, :, t] * v[:, :, t]
    dY = masked(np.asarray(dY, np.float64), lengths)
    c = np.zeros((B, C)) if dhT is None else np.asarray(dhT, np.float64)
    dv, dg = np.zeros((B, C, L)), np.zeros((B, C, L))
    for t in range(L - 1, -1, -1):
        dh = dY[:, :, t] + c
        dv[:, :, t] = i[:, :, t] * dh
        dg[:, :, t] = f[:, :, t] * i[:, :, t] * (before[:, :, t] - v[:, :, t]) * dh
        c = f[:, :, t] * dh
    return dv, dg, c
