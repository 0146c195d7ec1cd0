"""GPU parity of the gated recurrence (forward, backward, from 8-bit
checkpoints, single position) against the fp64 oracle, within bounds derived
in scan_util.py; carried states, padded batches, NaN behind a sequence's end,
guard bands, graph replays and other streams."""
import numpy as np
import pytest
import torch

from oracle import recurrence as orc
from scan_util import bounds

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import windowed_matmul_conv_b200 as wb  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
DEV = "cuda:0"


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(B, C, L, kind, seed, carry=True, ragged=False, gate=1.0):
    gen = torch.Generator().manual_seed(seed)
    dt = DT[kind]
    d = dict(v=torch.randn(B, C, L, generator=gen).to(dt),
             g=(torch.randn(B, C, L, generator=gen) * 2 + gate).to(dt),
             dY=torch.randn(B, C, L, generator=gen).to(dt),
             h0=torch.randn(B, C, generator=gen) if carry else None,
             dhT=torch.randn(B, C, generator=gen) if carry else None, lengths=None)
    if ragged:
        n = torch.randint(0, L + 1, (B,), generator=gen, dtype=torch.int32)
        n[0] = 0
        n[-1] = L + 5                      # taken as L
        if B > 3:
            n[1] = -7                      # taken as 0
        d["lengths"] = n
    return {k: t.to(DEV) if t is not None else None for k, t in d.items()}


def close(got, want, tol, what):
    got = np64(got)
    assert np.isfinite(got).all(), what
    far = np.abs(got - want) - tol
    at = np.unravel_index(far.argmax(), far.shape)
    assert far.max() <= 0, f"{what} at {at}: {got[at]} against {want[at]}, allowed {tol[at]:.3e}"


def check_train(d, kind, checkpoint):
    v, g, dY, h0, dhT, n = (np64(d[k]) for k in ("v", "g", "dY", "h0", "dhT", "lengths"))
    y, hT, saved = wb.scan_forward_train(d["v"], d["g"], d["h0"], d["lengths"], checkpoint=checkpoint)
    dv, dg, dh0 = wb.scan_backward(saved, d["dY"], d["dhT"])
    torch.cuda.synchronize()
    assert wb.wbmm_get_device_status() == 0
    ry, rh = orc.scan(v, g, h0, n)
    v8 = g8 = states = None
    if checkpoint:
        for x, c, e in ((v, saved.v, saved.v_exps), (g, saved.g, saved.g_exps)):
            wc, we = orc.seq_encode(x, n)
            assert np.array_equal(c.cpu().numpy(), wc) and np.array_equal(e.cpu().numpy(), we)
        v8, g8 = (orc.seq_decode(*orc.seq_encode(x, n)) for x in (v, g))
        states = rh[:, :, 0:v.shape[2]:orc.TILE]
    bv, bg = (v8, g8) if checkpoint else (v, g)
    rdv, rdg, rdh0 = orc.scan_backward(bv, bg, dY, dhT, h0, n, states)
    tol = bounds(v, g, kind, h0, n, dY, dhT, v8, g8)
    close(y, ry, tol["y"], "y")
    close(hT, rh[:, :, -1], tol["h"][:, :, -1], "hT")
    close(dv, rdv, tol["dv"], "dv")
    close(dg, rdg, tol["dg"], "dg")
    close(dh0, rdh0, tol["dh0"], "dh0")
    # a plain forward gives the same bits, and so does a second run
    y2, hT2 = wb.scan_forward(d["v"], d["g"], d["h0"], d["lengths"])
    assert torch.equal(y, y2) and torch.equal(hT, hT2)
    again = wb.scan_backward(saved, d["dY"], d["dhT"])
    assert torch.equal(dv, again[0]) and torch.equal(dg, again[1]) and torch.equal(dh0, again[2])


LENGTHS = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 127, 128, 129, 196, 255, 256, 257, 512, 777, 1024, 2049]


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("L", LENGTHS)
def test_lengths_one_to_many(L, kind):
    check_train(make(2, 5, L, kind, L), kind, False)
    check_train(make(2, 5, L, kind, L + 1), kind, True)


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 1, 16384), (1, 3, 5003), (3, 2, 20000), (40, 100, 49), (37, 33, 300),
                                   (2, 700, 1000), (700, 2, 120)],
                         ids=lambda s: "x".join(map(str, s)))
def test_few_and_many_rows(shape, kind, checkpoint):
    check_train(make(*shape, kind, sum(shape), carry=shape[0] != 3), kind, checkpoint)


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("L", [1, 5, 13, 30, 60, 64, 100, 256, 1000, 4104])
def test_padded_batch(L, kind, checkpoint):
    check_train(make(5, 4, L, kind, 100 + L, carry=L % 8 == 0, ragged=True), kind, checkpoint)


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("L", [20, 120, 1000, 3000])
def test_nothing_behind_the_end_counts(L, checkpoint):
    """NaN and infinities behind a sequence's end change no bit of any result,
    and the rows there are zero."""
    for kind in ("bf16", "fp32"):
        d = make(4, 3, L, kind, 7, ragged=True)
        on = torch.arange(L, device=DEV)[None, None] < d["lengths"][:, None, None]

        def run(d):
            y, hT, saved = wb.scan_forward_train(d["v"], d["g"], d["h0"], d["lengths"],
                                                 checkpoint=checkpoint)
            return (y, hT) + wb.scan_backward(saved, d["dY"], d["dhT"])
        a = run(d)
        bad = dict(d)
        for k, x in (("v", float("nan")), ("g", float("inf")), ("dY", float("nan"))):
            bad[k] = torch.where(on, d[k], torch.full_like(d[k], x))
        for p, q in zip(a, run(bad)):
            assert torch.equal(p, q)
        for k in (0, 2, 3):
            assert (a[k].masked_select(~on) == 0).all()
        assert torch.equal(a[1][0], d["h0"][0])         # an empty sequence keeps its state


def test_nan_within_a_sequence_spreads_forward_only():
    for L in (40, 700):
        d = make(2, 2, L, "fp32", 3)
        d["v"][0, 1, L // 2] = float("nan")
        y, hT = wb.scan_forward(d["v"], d["g"], d["h0"])
        assert torch.isfinite(y[0, 0]).all() and torch.isfinite(y[1]).all()
        assert torch.isfinite(y[0, 1, :L // 2]).all() and torch.isnan(y[0, 1, L // 2:]).all()
        assert torch.isnan(hT[0, 1]) and torch.isfinite(hT[1]).all()


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_extreme_gates(kind):
    """Gates at both ends of the type's range, infinities among them: an open
    gate keeps the state, a shut one takes the input."""
    B, C, L = 1, 2, 600
    big = torch.finfo(DT[kind]).max
    for top in (big, float("inf"), 500.0):
        d = make(B, C, L, kind, 5)
        g = torch.full((B, C, L), top, dtype=DT[kind], device=DEV)
        y, hT = wb.scan_forward(d["v"], g, d["h0"])
        assert torch.equal(hT, d["h0"])
        assert torch.equal(y, d["h0"].to(DT[kind])[:, :, None].expand_as(y))
        y, hT = wb.scan_forward(d["v"], -g, d["h0"])
        assert torch.equal(y, d["v"])
        _, _, saved = wb.scan_forward_train(d["v"], -g, d["h0"])
        dv, dg, dh0 = wb.scan_backward(saved, d["dY"], d["dhT"])
        assert torch.equal(dv[:, :, :-1], d["dY"][:, :, :-1])
        assert dg.abs().max() < 1e-30 and dh0.abs().max() < 1e-30


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_long_memory(kind):
    """Gates close to 1 over thousands of positions."""
    check_train(make(1, 3, 6000, kind, 11, gate=8.0), kind, False)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_step_and_carried_state(kind):
    """A prefill of 75 positions, then single positions, against one call; a
    step is the forward of one position, in place or not."""
    d = make(3, 17, 90, kind, 21)
    v, g = d["v"], d["g"]
    want, last = orc.scan(np64(v), np64(g), np64(d["h0"]))
    tol = bounds(np64(v), np64(g), kind, np64(d["h0"]), None)
    cut = 75
    h = d["h0"].clone()
    y = torch.empty(3, 17, cut, dtype=DT[kind], device=DEV)
    wb.wbmm_scan_forward(v[:, :, :cut].contiguous(), g[:, :, :cut].contiguous(), h, None, y, h, None,
                         None, None, None, None)       # the state updated in place
    close(y, want[:, :, :cut], tol["y"][:, :, :cut], "prefill")
    for t in range(cut, 90):
        vt, gt = v[:, :, t].contiguous(), g[:, :, t].contiguous()
        y1, h1 = wb.scan_step(vt, gt, h)
        y2, h2 = wb.scan_forward(vt, gt, h)
        assert torch.equal(y1, y2) and torch.equal(h1, h2)
        wb.wbmm_scan_step(vt, gt, h, y2, h)            # in place
        assert torch.equal(y1, y2) and torch.equal(h1, h)
        close(y1, want[:, :, t], tol["y"][:, :, t], "step")
    close(h, last[:, :, -1], tol["h"][:, :, -1], "state")


@pytest.mark.parametrize("rows", [(1, 1), (1, 7), (1, 256), (3, 333), (64, 1000), (256, 8192)])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_step_sizes(rows, kind):
    d = make(*rows, 1, kind, 31)
    v, g = (d[k][:, :, 0].contiguous() for k in ("v", "g"))
    y, h = wb.scan_step(v, g, d["h0"])
    want, s = orc.scan(np64(d["v"]), np64(d["g"]), np64(d["h0"]))
    tol = bounds(np64(d["v"]), np64(d["g"]), kind, np64(d["h0"]), None)
    close(y, want[:, :, 0], tol["y"][:, :, 0], "y")
    close(h, s[:, :, 1], tol["h"][:, :, 1], "h")


@pytest.mark.parametrize("shape", [(3, 5, 1), (3, 5, 7), (3, 5, 100), (3, 5, 333), (1, 2, 9001)])
def test_nothing_outside_the_outputs_is_written(shape):
    B, C, L = shape
    for kind in ("bf16", "fp32"):
        d = make(*shape, kind, 41, ragged=True)
        n = B * C * L
        st = wb.wbmm_scan_states_bytes(B, C, L) // 4
        ng = B * C * -(-L // 64)

        def guarded(count, dtype):
            return torch.full((count + 128,), 77, dtype=dtype, device=DEV)

        y, dv, dg = (guarded(n, DT[kind]) for _ in range(3))
        hT, dh0 = guarded(B * C, torch.float32), guarded(B * C, torch.float32)
        states = guarded(st, torch.float32)
        vc, gc = guarded(n, torch.uint8), guarded(n, torch.uint8)
        ve, ge = guarded(ng, torch.uint8), guarded(ng, torch.uint8)
        wb.wbmm_scan_forward(d["v"], d["g"], d["h0"], d["lengths"], y, hT, states, vc, ve, gc, ge)
        wb.wbmm_scan_backward_checkpoint(vc, ve, gc, ge, states, d["lengths"], d["dY"], d["dhT"], dv, dg, dh0)
        torch.cuda.synchronize()
        for t, count in ((y, n), (dv, n), (dg, n), (hT, B * C), (dh0, B * C), (states, st), (vc, n),
                         (gc, n), (ve, ng), (ge, ng)):
            assert (t[count:] == 77).all()
        ref = wb.scan_forward_train(d["v"], d["g"], d["h0"], d["lengths"], checkpoint=True)
        assert torch.equal(ref[0].reshape(-1), y[:n])
        assert torch.equal(wb.scan_backward(ref[2], d["dY"], d["dhT"])[1].reshape(-1), dg[:n])


def test_offset_pointers():
    """Buffers that start inside an allocation: fp32 needs 4-byte alignment
    only, and single states and lengths too."""
    B, C, L = 2, 3, 264
    d = make(B, C, L, "fp32", 51, ragged=True)
    want = wb.scan_forward_train(d["v"], d["g"], d["h0"], d["lengths"])
    wgrad = wb.scan_backward(want[2], d["dY"], d["dhT"])

    def moved(t):
        s = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view(t.shape)
        return s.copy_(t)
    m = {k: moved(t) for k, t in d.items()}
    y, hT, states = moved(d["v"]), moved(d["h0"]), moved(want[2].states)
    wb.wbmm_scan_forward(m["v"], m["g"], m["h0"], m["lengths"], y, hT, states, None, None, None, None)
    assert torch.equal(y, want[0]) and torch.equal(hT, want[1])
    dv, dg, dh0 = moved(y), moved(y), moved(hT)
    wb.wbmm_scan_backward(m["v"], m["g"], states, m["lengths"], m["dY"], m["dhT"], dv, dg, dh0)
    for a, b in zip((dv, dg, dh0), wgrad):
        assert torch.equal(a, b)


@pytest.mark.parametrize("shape", [(2, 3, 1), (2, 30, 196), (1, 4, 20000)])
def test_graph_replay_and_side_stream(shape):
    """A captured forward and backward pass, replayed with new inputs in place,
    gives the eager call's bits; so does a call on another stream."""
    a, b = make(*shape, "bf16", 61), make(*shape, "bf16", 62)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    live = {k: t.clone() for k, t in a.items() if t is not None}

    def step(d):
        y, hT, saved = wb.scan_forward_train(d["v"], d["g"], d["h0"], checkpoint=True)
        return (y, hT) + wb.scan_backward(saved, d["dY"], d["dhT"])
    with torch.cuda.stream(s):
        first = step(live)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(live)
    for d in (b, a, b):
        for k, t in live.items():
            t.copy_(d[k])
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(out, step(d)):
            assert torch.equal(p, q)
    for p, q in zip(first, step(a)):
        assert torch.equal(p, q)


def test_gradients_against_differences():
    """The kernels' own forward, by central differences of a sum in fp64; the
    map is smooth, so the step's error is about 1e-4 of the values and fp32's
    rounding about 2^-24 / 2e-2 of them."""
    B, C, L = 1, 2, 70
    d = make(B, C, L, "fp32", 71)
    _, _, saved = wb.scan_forward_train(d["v"], d["g"], d["h0"])
    grads = dict(zip(("v", "g", "h0"), wb.scan_backward(saved, d["dY"], d["dhT"])))

    def loss(x):
        y, hT = wb.scan_forward(x["v"], x["g"], x["h0"])
        return ((y.double() * d["dY"].double()).sum() + (hT.double() * d["dhT"].double()).sum()).item()
    eps = 2e-2
    for k, at in (("v", (0, 0, 0)), ("v", (0, 1, 69)), ("v", (0, 1, 33)), ("g", (0, 0, 0)), ("g", (0, 0, 40)),
                  ("g", (0, 1, 69)), ("h0", (0, 0)), ("h0", (0, 1))):
        up, down = dict(d), dict(d)
        up[k], down[k] = d[k].clone(), d[k].clone()
        up[k][at] += eps
        down[k][at] -= eps
        diff = (loss(up) - loss(down)) / (2 * eps)
        assert abs(diff - grads[k][at].item()) < 1e-3, (k, at)


def test_maps_as_sequences():
    """A [B,C,H,W] map is its H*W positions in row-major order."""
    d = make(2, 3, 7 * 28, "bf16", 81)
    y, hT = wb.scan_forward(d["v"], d["g"])
    y4, hT4 = wb.scan_forward(d["v"].view(2, 3, 7, 28), d["g"].view(2, 3, 7, 28))
    assert y4.shape == (2, 3, 7, 28) and torch.equal(y4.view_as(y), y) and torch.equal(hT, hT4)


def test_offsets_past_32_bits():
    """A tensor of more than 2^31 elements; the rows at its end."""
    B, C, L = 1, 3, 1 << 30
    v = torch.zeros(B, C, L, dtype=torch.bfloat16, device=DEV)
    g = torch.zeros(B, C, L, dtype=torch.bfloat16, device=DEV)
    tail = make(1, 1, 4096, "bf16", 91, carry=False)
    v[0, 2, -4096:], g[0, 2, -4096:] = tail["v"][0, 0], tail["g"][0, 0]
    y, hT = wb.scan_forward(v, g)
    want, last = wb.scan_forward(tail["v"], tail["g"])
    assert torch.equal(y[0, 2, -4096:], want[0, 0]) and torch.equal(hT[0, 2], last[0, 0])
    assert (y[0, 2, :-4096] == 0).all() and (hT[0, :2] == 0).all()


@pytest.mark.parametrize("shape", [(2, 3, 5), (2, 3, 200), (2, 3, 300), (1, 2, 9000), (40, 50, 700)])
def test_states_updated_in_place(shape):
    """hT in h0's buffer and dh0 in dhT's, whichever kernel takes the rows."""
    d = make(*shape, "bf16", 101)
    y, hT, saved = wb.scan_forward_train(d["v"], d["g"], d["h0"])
    dv, dg, dh0 = wb.scan_backward(saved, d["dY"], d["dhT"])
    for _ in range(3):
        h, c, y2, dv2, dg2 = d["h0"].clone(), d["dhT"].clone(), *(torch.empty_like(y) for _ in range(3))
        wb.wbmm_scan_forward(d["v"], d["g"], h, None, y2, h, saved.states, None, None, None, None)
        wb.wbmm_scan_backward(d["v"], d["g"], saved.states, None, d["dY"], c, dv2, dg2, c)
        for a, b in ((h, hT), (y2, y), (c, dh0), (dv2, dv), (dg2, dg)):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    """Calls that overlap on the GPU share nothing."""
    ds = [make(1, 8, 30000 + 8 * k, "bf16", 111 + k) for k in range(2)]
    want = []
    for d in ds:
        y, hT, saved = wb.scan_forward_train(d["v"], d["g"], d["h0"], checkpoint=True)
        want.append((y, hT) + wb.scan_backward(saved, d["dY"], d["dhT"]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    got = []
    for _ in range(5):
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                y, hT, saved = wb.scan_forward_train(d["v"], d["g"], d["h0"], checkpoint=True)
                got.append((y, hT) + wb.scan_backward(saved, d["dY"], d["dhT"]))
    torch.cuda.synchronize()
    for k, g in enumerate(got):
        for a, b in zip(g, want[k % 2]):
            assert torch.equal(a, b)


def test_saved_of_another_shape_is_refused():
    d = make(2, 3, 40, "bf16", 121)
    saved = wb.scan_forward_train(d["v"], d["g"])[2]
    before = wb.wbmm_launch_count()
    for dY in (d["dY"][:, :, :32].contiguous(), d["dY"].reshape(3, 2, 40)):
        with pytest.raises(wb.WbmmError) as e:
            wb.scan_backward(saved, dY)
        assert e.value.status == 1
    with pytest.raises(ValueError):
        wb.scan_forward(d["v"].transpose(0, 1), d["g"].transpose(0, 1))
    with pytest.raises(wb.WbmmError) as e:      # bf16 rows that start between 16-byte boundaries
        wb.scan_forward(d["v"].reshape(-1)[1:41].view(1, 1, 40), d["g"].reshape(-1)[1:41].view(1, 1, 40))
    assert e.value.status == 4
    assert wb.wbmm_launch_count() == before


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(2, 3, 250), (2, 3, 257), (2, 3, 519), (2, 3, 1279), (2, 3, 1024), (1, 2, 9001)])
def test_one_states_array_serves_both_backward_calls(shape, kind):
    """The kept states are those before every 256th position, with 8-bit forms
    or without, so that either forward call's serve the other's backward."""
    d = make(*shape, kind, 121)
    plain = wb.scan_forward_train(d["v"], d["g"], d["h0"])[2]
    coded = wb.scan_forward_train(d["v"], d["g"], d["h0"], checkpoint=True)[2]
    v, g, h0 = np64(d["v"]), np64(d["g"]), np64(d["h0"])
    every = slice(0, shape[2], orc.TILE)
    want, tol = orc.scan(v, g, h0)[1][:, :, every], bounds(v, g, kind, h0, None)["h"][:, :, every]
    close(plain.states, want, tol, "states")
    close(coded.states, want, tol, "states beside 8-bit forms")
    for a, b in ((plain, coded), (coded, plain)):
        for p, q in zip(wb.scan_backward(a, d["dY"], d["dhT"]),
                        wb.scan_backward(a._replace(states=b.states), d["dY"], d["dhT"])):
            assert torch.equal(p, q)
