"""What is timed of the 8-bit activation checkpoints and the gated recurrence.

Every case is one pass of an operator as a training or serving program calls
it.  `run` computes it in plain torch operations, or, with `own` set, through
`windowed_matmul_conv_b200`.

Kinds of case
  roundtrip  a map [B,C,H,W] stored in 8 bits by windows and restored
  wbmm_bwd   the WBMM backward (dX, dT) whose input map is such a checkpoint
  prefill    the gated recurrence over [B,C,L] with a carried state
  train      its forward and backward pass
  train8     the same, its inputs kept as 8-bit checkpoints in between
  step       one token for every sequence of a batch
"""
import torch

own = False

DEV = "cuda"
SEQ_GROUP = 64          # positions of a sequence that share one step
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the benchmark's training workload: its input map kept in 8 bits
        dict(name="roundtrip_train_bf16", kind="roundtrip", dtype="bf16", B=128, C=256, H=28, W=28, w=14),
        # an odd window and a ragged map in fp32, as the CUDA-core tests use
        dict(name="roundtrip_odd_fp32", kind="roundtrip", dtype="fp32", B=9, C=37, H=35, W=63, w=7),
        # the backward call of the benchmark's training workload
        dict(name="wbmm_bwd_train_bf16", kind="wbmm_bwd", dtype="bf16", B=128, C=256, H=28, W=28, w=14),
        # small windows on a larger map, few channels
        dict(name="wbmm_bwd_w7_bf16", kind="wbmm_bwd", dtype="bf16", B=8, C=96, H=112, W=112, w=7),
        # the high-resolution map as one sequence a channel: few rows, long ones
        dict(name="prefill_hires_bf16", kind="prefill", dtype="bf16", B=8, C=96, L=50176, carry=True, ragged=False),
        # a padded batch of odd-length sequences, one of them empty
        dict(name="prefill_ragged_fp32", kind="prefill", dtype="fp32", B=5, C=333, L=777, carry=True, ragged=True),
        # training over 56 x 56 maps
        dict(name="train_map_bf16", kind="train", dtype="bf16", B=32, C=256, L=3136, carry=False, ragged=False),
        # training on a padded batch of odd length with a carried state
        dict(name="train_odd_fp32", kind="train", dtype="fp32", B=3, C=517, L=1001, carry=True, ragged=True),
        # the 56 x 56 maps again, inputs kept in 8 bits
        dict(name="train8_map_bf16", kind="train8", dtype="bf16", B=32, C=256, L=3136, carry=False, ragged=False),
        # one long sequence in 128 channels: work has to be split along it
        dict(name="train8_long_bf16", kind="train8", dtype="bf16", B=1, C=128, L=65536, carry=True, ragged=False),
        # serving: a single sequence, latency only; and a large batch
        dict(name="step_single_bf16", kind="step", dtype="bf16", B=1, C=256),
        dict(name="step_batch_bf16", kind="step", dtype="bf16", B=256, C=8192),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    kind = rng.choice(["roundtrip", "wbmm_bwd", "prefill", "train", "train8", "step"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if kind in ("roundtrip", "wbmm_bwd"):
        w = rng.choice([5, 7, 8, 12, 14])
        nh, nw = rng.randint(1, 112 // w), rng.randint(1, 112 // w)
        C = _log_int(rng, 3, 256)
        cap = 25_000_000 if kind == "roundtrip" else 12_000_000
        most = max(1, cap // (C * nh * nw * w * w))
        B = _log_int(rng, 1, min(128, most))
        return dict(kind=kind, dtype=dtype, B=B, C=C, H=nh * w, W=nw * w, w=w)
    if kind == "step":
        B = _log_int(rng, 1, 256)
        return dict(kind=kind, dtype=dtype, B=B, C=_log_int(rng, 17, 8192))
    L = _log_int(rng, 2, 50_000)
    if rng.random() < 0.5 and L >= 16:
        L = L // 8 * 8
    B = rng.randint(1, 32)
    C = _log_int(rng, 8, max(9, min(1024, 20_000_000 // (L * B))))
    return dict(kind=kind, dtype=dtype, B=B, C=C, L=L, carry=rng.random() < 0.5,
                ragged=rng.random() < 0.4)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    s = dict(case=case)
    B, C = case["B"], case["C"]
    if case["kind"] in ("roundtrip", "wbmm_bwd"):
        H, W, w = case["H"], case["W"], case["w"]
        # channels of an activation map differ in scale
        x = (normal(B, C, H, W) * torch.exp(0.7 * normal(1, C, 1, 1))).to(dt)
        if case["kind"] == "roundtrip":
            s["x"] = x
        else:
            # a backward pass has the checkpoint in hand, not the map
            codes, exps = _encode(_windows(x.float(), w))
            s["codes"], s["exps"] = codes, exps
            s["T"] = (0.02 * normal(C, (2 * w - 1) ** 2)).to(dt)
            s["dY"] = normal(B, C, H, W).to(dt)
        return s
    if case["kind"] == "step":
        s["v"] = normal(B, C).to(dt)
        s["g"] = (normal(B, C) + 2.0).to(dt)
        s["h"] = normal(B, C)
        return s
    L = case["L"]
    s["v"] = normal(B, C, L).to(dt)
    # a forget-gate bias per channel, so channels differ in how far they remember
    s["g"] = (normal(B, C, L) + 3.0 * torch.rand(1, C, 1, generator=gen, device=DEV)).to(dt)
    s["h0"] = normal(B, C) if case["carry"] else None
    s["lengths"] = None
    if case["ragged"]:
        n = torch.randint(0, L + 1, (B,), generator=gen, device=DEV, dtype=torch.int32)
        n[0] = L
        if B > 2:
            n[1] = 0
        s["lengths"] = n
    if case["kind"] != "prefill":
        s["dy"] = normal(B, C, L).to(dt)
        s["dhT"] = normal(B, C) if case["carry"] else None
    return s


# ------------------------------------------------------------- plain forms

def _windows(x, w):
    """[B,C,H,W] -> [C, windows, w*w], windows in (b, i, j) order."""
    B, C, H, W = x.shape
    x = x.reshape(B, C, H // w, w, W // w, w)
    return x.permute(1, 0, 2, 4, 3, 5).reshape(C, -1, w * w)


def _unwindows(a, B, C, H, W, w):
    a = a.reshape(C, B, H // w, W // w, w, w)
    return a.permute(1, 0, 2, 4, 3, 5).reshape(B, C, H, W)


def _encode(a):
    """Groups along the last axis -> uint8 codes of the same shape, uint8 exponents."""
    top = a.abs().amax(dim=-1)
    bad = ~torch.isfinite(a).all(dim=-1)
    # the exponent field of the fp32 maximum, one more where 127.5 / 64 is reached
    e = ((torch.where(bad, torch.zeros_like(top), top).view(torch.int32) + 0x10000) >> 23) - 6
    e = e.clamp(1, 248)
    step = (e << 23).view(torch.float32)
    q = torch.round(a / step[..., None]).clamp(-127, 127) + 128
    q = torch.where(bad[..., None], torch.full_like(q, 128), q)
    return q.to(torch.uint8), torch.where(bad, torch.full_like(e, 255), e).to(torch.uint8)


def _decode(codes, exps):
    step = (exps.to(torch.int32) << 23).view(torch.float32)
    return (codes.float() - 128.0) * step[..., None]


def _through_8_bits(x):
    """A sequence tensor [B,C,L] as its checkpoint keeps it."""
    L = x.shape[-1]
    pad = -L % SEQ_GROUP
    a = torch.cat([x, x.new_zeros(*x.shape[:-1], pad)], dim=-1)
    a = a.reshape(*x.shape[:-1], -1, SEQ_GROUP)
    return _decode(*_encode(a)).reshape(*x.shape[:-1], -1)[..., :L]


def _offsets(w, device):
    i = torch.arange(w, device=device)
    p, q = i.repeat_interleave(w), i.repeat(w)
    return (p[:, None] - p[None] + w - 1) * (2 * w - 1) + (q[:, None] - q[None] + w - 1)


def _recurrence(a, b):
    """h_t = a_t h_{t-1} + b_t along the last axis, by doubling."""
    L, d = a.shape[-1], 1
    while d < L:
        b = torch.cat([b[..., :d], b[..., d:] + a[..., d:] * b[..., :-d]], dim=-1)
        a = torch.cat([a[..., :d], a[..., d:] * a[..., :-d]], dim=-1)
        d *= 2
    return b


def _live(s):
    L = s["case"]["L"]
    if s["lengths"] is None:
        return None
    return torch.arange(L, device=DEV)[None, None] < s["lengths"][:, None, None]


def _gates(v, g, live):
    f = 1.0 / (1.0 + torch.exp(-g))
    i = 1.0 / (1.0 + torch.exp(g))
    u = i * v
    if live is not None:
        f = torch.where(live, f, 1.0)
        u = torch.where(live, u, 0.0)
    return f, i, u


def _scan(v, g, h0, live):
    f, i, u = _gates(v, g, live)
    if h0 is not None:
        u = torch.cat([u[..., :1] + f[..., :1] * h0[..., None], u[..., 1:]], dim=-1)
    return f, i, _recurrence(f, u)


def _zero(x, live):
    return x if live is None else torch.where(live, x, 0.0)


def _plain(s):
    case = s["case"]
    kind, dt = case["kind"], DTYPES[case["dtype"]]
    if kind == "roundtrip":
        dims = [case[k] for k in ("B", "C", "H", "W", "w")]
        return _unwindows(_decode(*_encode(_windows(s["x"].float(), case["w"]))), *dims).to(dt)
    if kind == "wbmm_bwd":
        dims = [case[k] for k in ("B", "C", "H", "W", "w")]
        w = case["w"]
        x, dy = _decode(s["codes"], s["exps"]), _windows(s["dY"].float(), w)
        at = _offsets(w, DEV)
        M = s["T"].float()[:, at]
        dX = _unwindows(dy @ M, *dims).to(dt)
        G = dy.transpose(1, 2) @ x
        dT = torch.zeros(case["C"], (2 * w - 1) ** 2, device=DEV)
        dT.index_add_(1, at.reshape(-1), G.reshape(case["C"], -1))
        return dX, dT
    if kind == "step":
        v, g = s["v"].float(), s["g"].float()
        h = s["h"] / (1.0 + torch.exp(-g)) + v / (1.0 + torch.exp(g))
        return h.to(dt), h
    live = _live(s)
    v, g = s["v"].float(), s["g"].float()
    f, i, h = _scan(v, g, s["h0"], live)
    y, hT = _zero(h, live).to(dt), h[..., -1].contiguous()
    if kind == "prefill":
        return y, hT
    start = s["h0"][..., None] if s["h0"] is not None else torch.zeros_like(h[..., :1])
    if kind == "train8":
        # the backward pass has the inputs as the checkpoint keeps them; the
        # states at every 256th position are those of the forward pass; what
        # lies behind a sequence's end counts as zero
        v, g = _through_8_bits(_zero(v, live)), _through_8_bits(_zero(g, live))
        f, i, u = _gates(v, g, live)
        L = f.shape[-1]
        pad = -L % 256
        fb = torch.cat([f, f.new_ones(*f.shape[:-1], pad)], dim=-1).unflatten(-1, (-1, 256))
        ub = torch.cat([u, u.new_zeros(*u.shape[:-1], pad)], dim=-1).unflatten(-1, (-1, 256))
        into = torch.cat([start, h[..., 255::256]], dim=-1)[..., :fb.shape[-2], None]
        ub = torch.cat([ub[..., :1] + fb[..., :1] * into, ub[..., 1:]], dim=-1)
        hb = _recurrence(fb, ub)
        before = torch.cat([into, hb[..., :-1]], dim=-1).flatten(-2)[..., :L]
    else:
        before = torch.cat([start, h[..., :-1]], dim=-1)
    dy = _zero(s["dy"].float(), live)
    b = f * dy
    if s["dhT"] is not None:
        b = torch.cat([b[..., :-1], b[..., -1:] + f[..., -1:] * s["dhT"][..., None]], dim=-1)
    c = _recurrence(f.flip(-1), b.flip(-1)).flip(-1)
    end = s["dhT"][..., None] if s["dhT"] is not None else torch.zeros_like(c[..., :1])
    dh = dy + torch.cat([c[..., 1:], end], dim=-1)
    dv = _zero(dh * i, live).to(dt)
    dg = _zero(dh * (before - v) * f * i, live).to(dt)
    return y, hT, dv, dg, c[..., 0].contiguous()


# ------------------------------------------------------ the framework's calls

def _own(s):
    import windowed_matmul_conv_b200 as wb
    case = s["case"]
    kind = case["kind"]
    if kind == "roundtrip":
        codes, exps = wb.checkpoint(s["x"], case["w"])
        return wb.checkpoint_restore(codes, exps, s["x"].shape, case["w"], s["x"].dtype)
    if kind == "wbmm_bwd":
        return wb.backward_checkpoint(s["codes"], s["exps"], s["T"], s["dY"], case["w"])
    if kind == "step":
        return wb.scan_step(s["v"], s["g"], s["h"])
    if kind == "prefill":
        return wb.scan_forward(s["v"], s["g"], s["h0"], s["lengths"])
    y, hT, saved = wb.scan_forward_train(s["v"], s["g"], s["h0"], s["lengths"],
                                         checkpoint=kind == "train8")
    dv, dg, dh0 = wb.scan_backward(saved, s["dy"], s["dhT"])
    return y, hT, dv, dg, dh0


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work

def work(case):
    sz = 2 if case["dtype"] == "bf16" else 4
    rows = case["B"] * case["C"]
    kind = case["kind"]
    if kind in ("roundtrip", "wbmm_bwd"):
        n, d = rows * case["H"] * case["W"], case["w"] ** 2
        t = case["C"] * (2 * case["w"] - 1) ** 2
        kept = n + n // d
        if kind == "roundtrip":
            return {"bytes": 2 * sz * n + kept, "flops": 4 * n}
        return {"bytes": 2 * sz * n + kept + (sz + 4) * t, "flops": 4 * d * n}
    if kind == "step":
        return {"bytes": rows * (3 * sz + 8), "flops": 8 * rows}
    n = rows * case["L"]
    state = 4 * rows
    if kind == "prefill":
        return {"bytes": 3 * sz * n + state * (1 + case["carry"]), "flops": 8 * n}
    # the forward pass reads v and g and writes y; the backward pass reads dy
    # and the kept v and g and writes dv and dg (in 8 bits the kept ones are
    # written and read at a byte and a 64th each)
    kept = 2 * 2 * (n + n // SEQ_GROUP) if kind == "train8" else 2 * sz * n
    return {"bytes": 6 * sz * n + kept + state * (2 + 2 * case["carry"]), "flops": 26 * n}


# ------------------------------------------------------------- definition

def exact(case, seed):
    """The definition in 64 bits: sequences step by step, windows one offset
    at a time."""
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "step":
        f = torch.sigmoid(s["g"].double())
        h = f * s["h"].double() + torch.sigmoid(-s["g"].double()) * s["v"].double()
        return h, h
    if kind in ("roundtrip", "wbmm_bwd"):
        B, C, H, W, w = (case[k] for k in ("B", "C", "H", "W", "w"))
        if kind == "roundtrip":
            x = s["x"].double()
            a = x.unfold(2, w, w).unfold(3, w, w)             # B C nh nw w w
            top = a.abs().amax(dim=(-2, -1))
            step = _step64(top)
            val = torch.round(a / step[..., None, None]) * step[..., None, None]
            return val.permute(0, 1, 2, 4, 3, 5).reshape(B, C, H, W)
        nh, nw = H // w, W // w
        two = _two64(s["exps"].double() - 127.0)
        x = ((s["codes"].double() - 128.0) * two[..., None]).reshape(C, -1, w, w)
        dy = s["dY"].double().unfold(2, w, w).unfold(3, w, w)
        dy = dy.permute(1, 0, 2, 3, 4, 5).reshape(C, -1, w, w)
        T = s["T"].double().reshape(C, 2 * w - 1, 2 * w - 1)
        dx = torch.zeros_like(dy)
        dT = torch.zeros_like(T)
        for a in range(-(w - 1), w):                          # a = p - r, b = q - s
            p0, p1 = max(0, a), min(w, w + a)
            for b in range(-(w - 1), w):
                q0, q1 = max(0, b), min(w, w + b)
                part = dy[:, :, p0:p1, q0:q1]
                at = (slice(None), slice(None), slice(p0 - a, p1 - a), slice(q0 - b, q1 - b))
                dx[at] += part * T[:, a + w - 1, b + w - 1, None, None, None]
                dT[:, a + w - 1, b + w - 1] = (part * x[at]).sum(dim=(1, 2, 3))
        dx = dx.reshape(C, B, nh, nw, w, w).permute(1, 0, 2, 4, 3, 5).reshape(B, C, H, W)
        return dx, dT.reshape(C, -1)

    B, C, L = case["B"], case["C"], case["L"]
    n = s["lengths"]

    def rows(x):                                              # position first
        return x.double().reshape(B * C, L).t().contiguous()

    def back(x, dt=None):
        return x.t().reshape(B, C, L)

    v, g = rows(s["v"]), rows(s["g"])
    f, i = torch.sigmoid(g), torch.sigmoid(-g)
    on = None
    if n is not None:
        on = torch.arange(L, device=DEV)[:, None] < n.repeat_interleave(C)[None]
        f = torch.where(on, f, 1.0)
        i = torch.where(on, i, 0.0)
    u = i * v
    h0 = s["h0"].double().reshape(-1) if s["h0"] is not None else torch.zeros(B * C, device=DEV, dtype=torch.float64)
    h = torch.empty(L + 1, B * C, device=DEV, dtype=torch.float64)
    h[0] = h0
    for t in range(L):
        torch.addcmul(u[t], f[t], h[t], out=h[t + 1])
    y = h[1:] if on is None else torch.where(on, h[1:], 0.0)
    hT = h[L].reshape(B, C).clone()
    if kind == "prefill":
        return back(y), hT
    y = back(y)
    if kind == "train8":
        def kept(x):
            out = torch.empty_like(x)
            for t in range(0, L, SEQ_GROUP):
                part = x[t:t + SEQ_GROUP]
                step = _step64(part.abs().amax(dim=0))
                out[t:t + SEQ_GROUP] = torch.round(part / step) * step
            return out
        if on is not None:
            v, g = torch.where(on, v, 0.0), torch.where(on, g, 0.0)
        v, g = kept(v), kept(g)
        f, i = torch.sigmoid(g), torch.sigmoid(-g)
        if on is not None:
            f = torch.where(on, f, 1.0)
            i = torch.where(on, i, 0.0)
        u = i * v
        k = torch.empty(L, B * C, device=DEV, dtype=torch.float64)
        for t in range(L):
            # the state before position t: kept exactly at every 256th
            k[t] = h[t] if t % 256 == 0 else f[t - 1] * k[t - 1] + u[t - 1]
        before = k
    else:
        before = h[:L]
    dy = rows(s["dy"])
    if on is not None:
        dy = torch.where(on, dy, 0.0)
    c = s["dhT"].double().reshape(-1) if s["dhT"] is not None else torch.zeros_like(h0)
    dh = torch.empty_like(dy)
    for t in range(L - 1, -1, -1):
        torch.add(dy[t], c, out=dh[t])
        c = f[t] * dh[t]
    return y, hT, back(dh * i), back(dh * (before - v) * f * i), c.reshape(B, C)


def _step64(top):
    """Smallest 2^e with rint(top / 2^e) <= 127."""
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 127.0)) - 1
    for _ in range(2):
        e = e + (torch.round(top / _two64(e)) > 127).double()
    return _two64(e.clamp(-126, 121))


def _two64(e):
    """2^e for whole e, from its bits: pow() may be off in the last place, and
    half steps are common among bf16 inputs."""
    return ((e.clamp(-1000, 1000).to(torch.int64) + 1023) << 52).view(torch.float64)
