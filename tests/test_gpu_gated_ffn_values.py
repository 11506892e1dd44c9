"""gated_ffn_fwd and gated_ffn_bwd on every kind of tile, each value against float64 and its own bound: beside the norms,
which a wrong fragment of a large output hardly moves (one 16 x 16 of 25 million values adds 3e-3 of the norm)."""
import pytest
import torch

from block_ref import BF, F32, ffn_reference
from gpu_common import announce
from selective_state_space_vjp_amd import binding as bd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def inputs(M, D, F, dtype):
    gen = torch.Generator(DEV).manual_seed(M + D + F)
    rn = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    return [t.to(dtype) for t in (rn(M, D), rn(F, D) * D**-0.5, rn(F, D) * D**-0.5, rn(M, F))]


def within(got, want, bound, where):
    """Every value within its bound, and no 16 x 16 of them (the values that one fragment forms) off by a third of its
    norm: a fragment that is missing or another's is off by all of it, a rounding of bf16 by 2^-8 of every value, dgate's
    and dup's by as much of independent terms."""
    err = (got.double() - want).abs()
    over = float((err - bound).max())
    print(f"{where}: {float((err / (bound + 1e-30)).max()):.2f} of the bound", flush=True)
    assert torch.isfinite(got).all() and over <= 0, (where, over)
    m, n = -want.shape[0] % 16, -want.shape[1] % 16
    block = lambda v: torch.nn.functional.pad(v * v, (0, n, 0, m)).unflatten(1, (-1, 16)).unflatten(0, (-1, 16)).sum((1, 3))  # noqa: E731
    worst = float((block(err) / block(want)).max()) ** 0.5
    assert worst <= 1 / 3, (where, worst)


# test_ffn_plans.py says which tiles these sizes get: every kind that each product has, whole and with k in parts, and every
# kind of dx beside every kind of the weights' gradients.
SIZES = [
    (777, 1000, 2712, BF), (1030, 1544, 1032, BF), (2048, 512, 2560, BF), (2100, 72, 4104, BF), (4104, 4104, 72, BF),
    (264, 2056, 4360, BF), (2056, 2048, 12296, BF), (1000, 4096, 12288, BF), (1016, 12296, 4088, BF), (12296, 2040, 2040, BF),
    (177, 1912, 1088, BF), (1, 1904, 1248, BF), (891, 8, 472, BF), (31, 48, 8, BF), (2236, 1864, 264, BF), (2219, 1912, 352, BF),
    (2331, 392, 2376, BF), (2356, 520, 1416, BF), (34, 1648, 1720, BF), (2474, 200, 2760, BF), (1345, 8, 1368, BF),
    (2222, 1360, 408, BF), (2192, 1736, 8, BF), (133, 1728, 2760, BF),
    (2100, 72, 4104, F32), (4104, 4104, 72, F32), (264, 2056, 4360, F32), (1024, 2048, 12296, F32), (1016, 6152, 4088, F32),
    (6152, 2040, 2040, F32), (643, 824, 1344, F32), (172, 1616, 520, F32), (1137, 72, 1320, F32), (562, 16, 8, F32), (31, 48, 8, F32),
    (1762, 1800, 648, F32), (2065, 1584, 536, F32), (2438, 72, 936, F32), (2053, 72, 872, F32), (113, 1376, 1208, F32),
    (1510, 1064, 8, F32), (2220, 664, 8, F32), (867, 1840, 368, F32), (2290, 1640, 40, F32),
    (5, 136, 72, F32)]


@pytest.mark.parametrize("M,D,F,dtype", SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_every_value(act, M, D, F, dtype):
    announce(f"gated ffn values {act} {dtype} {M} {D} {F}")
    x, wg, wu, dh = inputs(M, D, F, dtype)
    ref = ffn_reference(x, wg, wu, dh, act, dtype=dtype)
    out = bd.gated_ffn_fwd(x, wg, wu, act=act, want_saved=True)
    for k in ("h", "gate", "up"):
        within(out[k], *ref[k], k)
    got = bd.gated_ffn_bwd(dh, x, wg, wu, act=act)
    for k in ("dx", "dw_gate", "dw_up"):
        within(got[k], *ref[k], k + " formed again")
    saved = (out["gate"], out["up"])
    ref = ffn_reference(x, wg, wu, dh, act, saved=saved, dtype=dtype)
    got = bd.gated_ffn_bwd(dh, x, wg, wu, act=act, saved=saved)
    for k in ("dx", "dw_gate", "dw_up"):
        within(got[k], *ref[k], k + " kept")
    # by themselves they may get other tiles and parts
    within(bd.gated_ffn_bwd(dh, x, wg, wu, act=act, saved=saved, want_dw=False)["dx"], *ref["dx"], "dx alone")
    got = bd.gated_ffn_bwd(dh, x, wg, wu, act=act, saved=saved, want_dx=False)
    for k in ("dw_gate", "dw_up"):
        within(got[k], *ref[k], k + " without dx")
