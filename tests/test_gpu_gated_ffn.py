"""GPU parity of gated_ffn_fwd and gated_ffn_bwd against float64, from one row to many, at sizes that no tile divides."""
import math

import pytest
import torch

from block_ref import BF, F32, check, ffn_reference
from gpu_common import announce
from selective_state_space_vjp_amd import binding as bd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def inputs(M, D, F, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    return [t.to(dtype) for t in (rn(M, D), rn(F, D) * D**-0.5, rn(F, D) * D**-0.5, rn(M, F))]


SIZES = [(1, 8, 8), (1, 256, 520), (2, 64, 16), (5, 136, 72), (16, 128, 128), (17, 104, 264), (33, 72, 136), (64, 64, 64),
         (65, 200, 96), (100, 512, 144), (129, 88, 328), (257, 264, 136), (300, 136, 512), (520, 128, 264)]


@pytest.mark.parametrize("M,D,F", SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_forward_and_gradients(M, D, F, act, dtype):
    announce(f"gated ffn {act} {dtype} M={M} D={D} F={F}")
    x, wg, wu, dh = inputs(M, D, F, dtype, M + D + F)
    ref = ffn_reference(x, wg, wu, dh, act, dtype=dtype)
    t = [v.to(DEV) for v in (x, wg, wu, dh)]
    out = bd.gated_ffn_fwd(*t[:3], act=act, want_saved=True)
    for k in ("h", "gate", "up"):
        check(out[k], *ref[k], k)
    lean = bd.gated_ffn_fwd(*t[:3], act=act)
    assert torch.equal(lean["h"], out["h"]) and lean["gate"] is None
    got = bd.gated_ffn_bwd(t[3], *t[:3], act=act)
    for k in ("dx", "dw_gate", "dw_up"):
        check(got[k], *ref[k], k + " formed again")
    saved = (out["gate"], out["up"])
    ref = ffn_reference(x, wg, wu, dh, act, saved=[s.cpu() for s in saved], dtype=dtype)
    got = bd.gated_ffn_bwd(t[3], *t[:3], act=act, saved=saved)
    for k in ("dx", "dw_gate", "dw_up"):
        check(got[k], *ref[k], k + " kept")


def near(got, want, tol, where):
    err = float((got.double() - want).norm() / want.norm())
    print(where, f"{err:.1e} of {tol:.1e}", flush=True)
    assert err <= tol, (where, err, tol)


# 128 x 128 with k in parts; whole; 256 x 256 of the forward, of dx, of the weights' gradients, of all but dx
@pytest.mark.parametrize("M,D,F", [(777, 1000, 2712), (1030, 1544, 1032), (2048, 512, 2560), (2100, 72, 4104), (4104, 4104, 72),
                                   (264, 2056, 4360), (2056, 2048, 12296)])
def test_large_tiles(M, D, F):
    """Norms of the errors: a rounding of bf16 leaves at most 2^-8 of the norm, dgate's and dup's roundings 2^-8 of
    independent terms more, float32 sums far less."""
    announce(f"gated ffn large {M} {D} {F}")
    x, wg, wu, dh = (v.to(DEV) for v in inputs(M, D, F, BF, 5))
    out = bd.gated_ffn_fwd(x, wg, wu, want_saved=True)
    X, G, Uw, H = (v.double() for v in (x, wg, wu, dh))
    gate, up = torch.mm(X, G.T), torch.mm(X, Uw.T)
    near(out["gate"], gate, 2.0**-8, "gate")
    near(out["up"], up, 2.0**-8, "up")
    near(out["h"], gate * torch.sigmoid(gate) * up, 2.0**-8, "h")
    for saved in (None, (out["gate"], out["up"])):
        if saved:
            gate, up = (v.double() for v in saved)
        s = torch.sigmoid(gate)
        dg, du = H * up * (s + gate * s * (1 - s)), H * gate * s
        got = bd.gated_ffn_bwd(dh, x, wg, wu, saved=saved)
        near(got["dx"], torch.mm(dg, G) + torch.mm(du, Uw), 2.0**-7, "dx")
        near(got["dw_gate"], torch.mm(dg.T, X), 2.0**-7, "dw_gate")
        near(got["dw_up"], torch.mm(du.T, X), 2.0**-7, "dw_up")


def agrees(M, D, F, dtype):
    """Norms of the errors: bf16 as above.  float32: a sum of k products wanders off by about 2^-24 sqrt(k / 6) of its
    norm, what the activation adds is a few roundings, and the second product passes the first one's on."""
    announce(f"gated ffn tiles {M} {D} {F} {dtype}")
    x, wg, wu, dh = (v.to(DEV) for v in inputs(M, D, F, dtype, 6))
    out = bd.gated_ffn_fwd(x, wg, wu, want_saved=True)
    first, rows, cols = ((2.0**-8, 2.0**-7, 2.0**-7) if dtype is BF else
                         [2.0**-24 * (16 + math.sqrt(D) + math.sqrt(k)) for k in (0, 2 * F, M)])
    X, G, Uw, H = (v.double() for v in (x, wg, wu, dh))
    gate, up = torch.mm(X, G.T), torch.mm(X, Uw.T)
    near(out["gate"], gate, first, "gate")
    near(out["up"], up, first, "up")
    near(out["h"], gate * torch.sigmoid(gate) * up, first, "h")
    assert torch.equal(bd.gated_ffn_fwd(x, wg, wu)["h"], out["h"])
    for saved in (None, (out["gate"], out["up"])):
        if saved:
            gate, up = (v.double() for v in saved)
        s = torch.sigmoid(gate)
        dg, du = H * up * (s + gate * s * (1 - s)), H * gate * s
        got = bd.gated_ffn_bwd(dh, x, wg, wu, saved=saved)
        near(got["dx"], torch.mm(dg, G) + torch.mm(du, Uw), rows, "dx")
        near(got["dw_gate"], torch.mm(dg.T, X), cols, "dw_gate")
        near(got["dw_up"], torch.mm(du.T, X), cols, "dw_up")
    only = bd.gated_ffn_bwd(dh, x, wg, wu, saved=saved, want_dw=False)
    assert only["dw_gate"] is None
    near(only["dx"], torch.mm(dg, G) + torch.mm(du, Uw), rows, "dx alone")
    only = bd.gated_ffn_bwd(dh, x, wg, wu, saved=saved, want_dx=False)
    assert only["dx"] is None  # another call may cut k elsewhere
    near(only["dw_gate"], torch.mm(dg.T, X), cols, "dw_gate without dx")
    near(only["dw_up"], torch.mm(du.T, X), cols, "dw_up without dx")


# 256 x 256 of the forward and of what it forms again; of dx; of the weights' gradients; of dx with k in parts
@pytest.mark.parametrize("M,D,F,dtype", [(2100, 72, 4104, F32), (4104, 4104, 72, F32), (264, 2056, 4360, F32),
                                         (1024, 2048, 12296, F32), (1000, 4096, 12288, BF)])
def test_large_tiles_of_both_types(M, D, F, dtype):
    agrees(M, D, F, dtype)


# The smaller tiles of dx (32 x 64, 128 x 64, 128 x 128) beside those of the weights' gradients (128 x 64, 128 x 128), each
# whole and with k in parts, and the forward's
@pytest.mark.parametrize("M,D,F,dtype", [
    (177, 1912, 1088, BF), (1, 1904, 1248, BF), (891, 8, 472, BF), (31, 48, 8, BF), (2236, 1864, 264, BF), (2219, 1912, 352, BF),
    (2331, 392, 2376, BF), (2356, 520, 1416, BF), (34, 1648, 1720, BF), (2474, 200, 2760, BF), (1345, 8, 1368, BF),
    (2222, 1360, 408, BF), (2192, 1736, 8, BF), (133, 1728, 2760, BF),
    (172, 1616, 520, F32), (1137, 72, 1320, F32), (562, 16, 8, F32), (31, 48, 8, F32), (1762, 1800, 648, F32),
    (2065, 1584, 536, F32), (2438, 72, 936, F32), (2053, 72, 872, F32), (113, 1376, 1208, F32), (1510, 1064, 8, F32),
    (2220, 664, 8, F32), (867, 1840, 368, F32), (2290, 1640, 40, F32)])
def test_every_pair_of_tiles(M, D, F, dtype):
    agrees(M, D, F, dtype)


@pytest.mark.parametrize("M,D,F", [(48, 392, 8), (1, 64, 2584), (1, 3208, 16), (30, 16, 1232), (3, 8, 8), (2500, 8, 200),
                                   (700, 128, 8), (1, 1000, 4104), (33, 400, 96), (1, 2000, 8200)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_few_values_are_formed_from_two_parts(M, D, F, act):
    """A gradient is off by its own rounding, 2^-8 of it at most, and by what two parts of dgate and dup leave: 2^-16 of
    every term, with the float32 errors of the products and the sums (a few 2^-22) 2^-15.  act' has a zero, near which its
    error is not one of itself: with u = 2^-24 and |z| <= 5, s is off by (|z| + 4) s (1 - s) u <= 2 u, f = z s by 11 u,
    f (1 - s) by 11 u + 5 * 2 u, act' by 24 u; in GELU's f (1 - s) <= 0.2 meets a factor of at most 1.6 (1 + 0.13 z^2) <= 7
    and is off by (|2 v| + 6) <= 40 u of itself where that is more than u, so by 56 u: 2^-18 of dh up in dgate.
    gate and up that are formed again are sums of D terms: each addition rounds a partial sum of at most 5 by 5 u to either
    side, D of them wander off by 5 u sqrt(D / 3), six times that is below 2^-19 sqrt(D); |act'| and |act''| <= 1.2."""
    announce(f"gated ffn two parts {act} {M} {D} {F}")
    x, wg, wu, dh = (v.to(DEV) for v in inputs(M, D, F, BF, 8))
    out = bd.gated_ffn_fwd(x, wg, wu, act=act, want_saved=True)
    X, G, Uw, H = (v.double() for v in (x, wg, wu, dh))
    for saved in (None, (out["gate"], out["up"])):
        gate, up = (v.double() for v in saved) if saved else (torch.mm(X, G.T), torch.mm(X, Uw.T))
        gate.requires_grad_(True)
        f = gate * torch.sigmoid(gate) if act == "silu" else torch.nn.functional.gelu(gate, approximate="tanh")
        df, = torch.autograd.grad(f.sum(), gate)
        dg, du = H * up * df, H * f.detach()
        eg = 2.0**-15 * dg.abs() + 2.0**-18 * (H * up).abs()
        eu = 2.0**-15 * du.abs()
        if not saved:
            wander = 1.2 * 2.0**-19 * math.sqrt(D)
            eg += wander * (H.abs() + (H * up).abs())
            eu += wander * H.abs()
        got = bd.gated_ffn_bwd(dh, x, wg, wu, act=act, saved=saved)
        for k, want, left in (("dx", torch.mm(dg, G) + torch.mm(du, Uw), torch.mm(eg, G.abs()) + torch.mm(eu, Uw.abs())),
                              ("dw_gate", torch.mm(dg.T, X), torch.mm(eg.T, X.abs())),
                              ("dw_up", torch.mm(du.T, X), torch.mm(eu.T, X.abs()))):
            over = (got[k].double() - want).abs() - 2.0**-8 * want.abs() - left
            assert float(over.max()) <= 0, (k, float(over.max()))


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_rows_are_independent(dtype):
    """A row's result does not depend on which rows stand beside it where the same kernel runs, a NaN row harms no other,
    and the zeros that fill a tile never meet it."""
    announce(f"gated ffn rows {dtype}")
    for M in (3, 70, 300):
        x, wg, wu, dh = (v.to(DEV) for v in inputs(M, 136, 264, dtype, 3))
        clean = bd.gated_ffn_fwd(x, wg, wu, want_saved=True)
        x2 = x.clone()
        x2[M // 2] = math.nan
        got = bd.gated_ffn_fwd(x2, wg, wu, want_saved=True)
        rest = torch.ones(M, dtype=torch.bool)
        rest[M // 2] = False
        for k in clean:
            assert torch.equal(got[k][rest], clean[k][rest]) and torch.isnan(got[k][M // 2]).all()
        g = bd.gated_ffn_bwd(dh, x, wg, wu, saved=(clean["gate"], clean["up"]))
        d2 = dh.clone()
        d2[M // 2] = math.inf
        g2 = bd.gated_ffn_bwd(d2, x, wg, wu, saved=(clean["gate"], clean["up"]))
        assert torch.equal(g2["dx"][rest], g["dx"][rest])


def test_extreme_projections():
    """act and its derivative far out: finite where the formula is."""
    announce("gated ffn extremes")
    for act in ("silu", "gelu"):
        x = torch.tensor([[-300.0, 0, 0, 0, 0, 0, 0, 0], [300.0, 0, 0, 0, 0, 0, 0, 0], [0.0] * 8], device=DEV)
        w = torch.eye(8, device=DEV)
        out = bd.gated_ffn_fwd(x, w, torch.ones(8, 8, device=DEV), act=act)
        assert torch.isfinite(out["h"]).all()
        assert out["h"][0, 0] == 0 and float(out["h"][1, 0]) == 300.0 * 300.0 and out["h"][2, 0] == 0
        g = bd.gated_ffn_bwd(torch.ones(3, 8, device=DEV), x, w, torch.ones(8, 8, device=DEV), act=act)
        assert all(torch.isfinite(v).all() for v in g.values())


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_projections_whose_square_overflows(act):
    """act'(z) is 1 above and 0 below, act(z) is z and 0, in the epilogue that forms gate again and from the kept one."""
    announce(f"gated ffn far {act}")
    x = torch.zeros(2, 8, device=DEV)
    x[0, 0], x[1, 0] = 1e20, -1e20
    w, one = torch.eye(8, device=DEV), torch.zeros(8, 8, device=DEV)
    one[:, 1] = 1.0
    x[:, 1] = 1.0  # up = 1
    out = bd.gated_ffn_fwd(x, w, one, act=act, want_saved=True)
    assert float(out["h"][0, 0]) == float(x[0, 0]) and float(out["h"][1, 0]) == 0.0
    for saved in (None, (out["gate"], out["up"])):
        g = bd.gated_ffn_bwd(torch.ones(2, 8, device=DEV), x, w, one, act=act, saved=saved)
        # dw_up[0, 0] = act(1e20) 1e20 is past float32's largest
        assert torch.isfinite(g["dx"]).all() and torch.isfinite(g["dw_gate"]).all() and float(g["dw_up"][0, 0]) == math.inf
        assert float(g["dx"][0, 0]) == 1.0 and float(g["dx"][1, 0]) == 0.0


def test_optional_outputs_empty_batches_and_streams():
    announce("gated ffn options")
    x, wg, wu, dh = (v.to(DEV) for v in inputs(40, 64, 96, BF, 7))
    full = bd.gated_ffn_bwd(dh, x, wg, wu)
    only = bd.gated_ffn_bwd(dh, x, wg, wu, want_dw=False)
    assert torch.equal(only["dx"], full["dx"]) and only["dw_gate"] is None and only["dw_up"] is None
    only = bd.gated_ffn_bwd(dh, x, wg, wu, want_dx=False)
    assert torch.equal(only["dw_up"], full["dw_up"]) and torch.equal(only["dw_gate"], full["dw_gate"]) and only["dx"] is None
    e = bd.gated_ffn_fwd(x[:0], wg, wu, want_saved=True)
    assert e["h"].shape == (0, 96)
    g = bd.gated_ffn_bwd(dh[:0], x[:0], wg, wu)
    assert (g["dw_gate"] == 0).all() and (g["dw_up"] == 0).all() and g["dx"].shape == (0, 64)
    # leading axes, another stream, a graph replayed on other values
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    h = bd.gated_ffn_fwd(x.view(4, 10, 64), wg, wu, stream=other)["h"]
    other.synchronize()
    assert h.shape == (4, 10, 96) and torch.equal(h.view(40, 96), bd.gated_ffn_fwd(x, wg, wu)["h"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f = bd.gated_ffn_fwd(x, wg, wu, want_saved=True)
        b = bd.gated_ffn_bwd(dh, x, wg, wu, saved=(f["gate"], f["up"]))
        b2 = bd.gated_ffn_bwd(dh, x, wg, wu)
    for _ in range(3):
        x.copy_(torch.randn(40, 64, device=DEV))
        g.replay()
        torch.cuda.synchronize()
        wf = bd.gated_ffn_fwd(x, wg, wu, want_saved=True)
        wb, wb2 = bd.gated_ffn_bwd(dh, x, wg, wu, saved=(wf["gate"], wf["up"])), bd.gated_ffn_bwd(dh, x, wg, wu)
        for got, want in ((f, wf), (b, wb), (b2, wb2)):
            for k in want:
                assert torch.equal(got[k], want[k]), k
