"""GPU parity of the gated recurrence's kernels for many rows (a warp a row,
from 10 rows an SM on) and for walks of more than 32 tiles a warp, every row
against the fp64 form, within bounds derived in recurrence_f64.py."""
import pytest
import torch

import recurrence_f64 as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import windowed_matmul_conv_b200 as wb  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
DEV = "cuda:0"


def make(B, C, L, kind, seed, carry, ragged):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = DT[kind]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)
    d = dict(v=normal(B, C, L).to(dt), g=(2 * normal(B, C, L) + 1).to(dt), dY=normal(B, C, L).to(dt),
             h0=normal(B, C) if carry else None, dhT=normal(B, C) if carry else None, lengths=None)
    if ragged:
        n = torch.randint(0, L + 1, (B,), generator=gen, device=DEV, dtype=torch.int32)
        n[0], n[1], n[2] = 0, L, max(1, L - 1)
        d["lengths"] = n
    return d


def close(got, want, what):
    value, tol = want
    assert torch.isfinite(got).all(), what
    far = (got.double() - value).abs() - tol
    k = int(far.argmax())
    at = [int(q) for q in torch.unravel_index(torch.tensor(k), far.shape)]
    assert far.max() <= 0, (f"{what} at {at}: {got.flatten()[k].item()} against "
                            f"{value.flatten()[k].item()}, allowed {tol.flatten()[k].item():.3e}")


def check(d, kind, checkpoint):
    v, g, dY, h0, dhT, n = (d[k] for k in ("v", "g", "dY", "h0", "dhT", "lengths"))
    y, hT, saved = wb.scan_forward_train(v, g, h0, n, checkpoint=checkpoint)
    dv, dg, dh0 = wb.scan_backward(saved, dY, dhT)
    torch.cuda.synchronize()
    assert wb.wbmm_get_device_status() == 0
    fwd = ref.forward(v, g, h0, n, kind)
    close(y, fwd["y"], "y")
    close(hT, fwd["hT"], "hT")
    # states are kept up to a sequence's end
    at = torch.arange(saved.states.shape[-1], device=DEV) * 256
    kept = at[None, None] < (n if n is not None else torch.full((v.shape[0],), v.shape[2], device=DEV))[:, None, None]
    close(torch.where(kept, saved.states, 0.0),
          tuple(torch.where(kept, x, 0.0) for x in fwd["states"]), "states")
    vb, gb = v.double(), g.double()
    if checkpoint:
        vb, vc, ve = ref.through_8_bits(vb, n)
        gb, gc, ge = ref.through_8_bits(gb, n)
        for name, a, b in (("codes of v", saved.v, vc), ("codes of g", saved.g, gc),
                           ("exponents of v", saved.v_exps, ve), ("exponents of g", saved.g_exps, ge)):
            assert torch.equal(a, b), name
    bwd = ref.backward(fwd, vb, gb, dY, dhT, n, kind)
    close(dv, bwd["dv"], "dv")
    close(dg, bwd["dg"], "dg")
    close(dh0, bwd["dh0"], "dh0")
    # a plain forward gives the same bits, and so does a second run
    y2, hT2 = wb.scan_forward(v, g, h0, n)
    assert torch.equal(y, y2) and torch.equal(hT, hT2)
    for a, b in zip((dv, dg, dh0), wb.scan_backward(saved, dY, dhT)):
        assert torch.equal(a, b)


def many_rows():
    """A batch and a channel count of some more rows than a warp a row takes."""
    C = torch.cuda.get_device_properties(0).multi_processor_count * 2 + 3
    return 5, C


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("L", [257, 300, 512, 1000, 1003, 2048, 2049])
def test_a_warp_a_row(L, kind, checkpoint):
    check(make(*many_rows(), L, kind, L, carry=L % 2 == 0, ragged=False), kind, checkpoint)


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("L", [272, 777, 1280])
def test_a_warp_a_row_of_a_padded_batch(L, kind, checkpoint):
    check(make(*many_rows(), L, kind, L, carry=L % 2 == 1, ragged=True), kind, checkpoint)


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("L", [8448, 9001, 16640])
def test_a_warp_a_row_of_more_than_32_tiles(L, kind, checkpoint):
    """33, 36 and 65 tiles: the kept states and exponent bytes of a second and
    a third 32 tiles."""
    check(make(*many_rows(), L, kind, L, carry=True, ragged=L == 9001), kind, checkpoint)


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(4, 100, 40000), (4, 25, 140001)], ids=lambda s: "x".join(map(str, s)))
def test_teams_of_more_than_32_tiles_a_warp(shape, kind, checkpoint):
    check(make(*shape, kind, sum(shape), carry=True, ragged=shape[2] % 2 == 1), kind, checkpoint)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("rows", [(1, 7), (3, 333), (64, 1000), (256, 8192)], ids=lambda s: "x".join(map(str, s)))
def test_a_step_is_a_row_of_one_position(rows, kind):
    """Against calls that the row kernels take: a forward call that keeps states,
    and one with lengths."""
    d = make(*rows, 1, kind, 31, carry=True, ragged=False)
    y, h = wb.scan_step(d["v"][:, :, 0].contiguous(), d["g"][:, :, 0].contiguous(), d["h0"])
    y1, h1, saved = wb.scan_forward_train(d["v"], d["g"], d["h0"])
    assert torch.equal(y, y1[:, :, 0]) and torch.equal(h, h1)
    assert torch.equal(saved.states[:, :, 0], d["h0"])
    n = torch.ones(rows[0], dtype=torch.int32, device=DEV)
    y2, h2 = wb.scan_forward(d["v"], d["g"], d["h0"], n)
    assert torch.equal(y, y2[:, :, 0]) and torch.equal(h, h2)
