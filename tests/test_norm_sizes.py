"""Layer norm at the largest sizes the header names: the host's checks and the backward's
workspace (CPU), and rows of millions of values (GPU)."""
import ctypes

import pytest
import torch

from gpu_common import announce
from selective_state_space_vjp_amd import binding as bd

U32 = 2.0**-24
DEV = "cuda:0"


def query(fn, rows, groups, dim, dtype):
    n = ctypes.c_size_t(0)
    d = bd.NormDesc(rows, groups, dim, 1e-5, dtype)
    return getattr(bd.lib(), fn + "_workspace")(ctypes.byref(d), ctypes.byref(n)), n.value


@pytest.mark.parametrize("dtype", [bd.F32, bd.BF16])
@pytest.mark.parametrize("rows,groups,dim,status", [
    (3, 1, 1 << 20, bd.OK),
    (3, 1, (1 << 21) + 3, bd.OK),
    (1 << 20, 1, 1 << 24, bd.OK),
    (2, 1, (1 << 26) - 17, bd.OK),
    (2, 1, (1 << 26) - 16, bd.EUNSUPPORTED),
    (2, 64, (1 << 20) - 1, bd.OK),
    (2, 64, 1 << 20, bd.EUNSUPPORTED),
    (1, (1 << 24) - 2049, 1, bd.OK),
    (1, (1 << 24) - 2048, 1, bd.EUNSUPPORTED),
    ((1 << 31) - 1, 1, 1, bd.OK),
    (1 << 31, 1, 1, bd.EUNSUPPORTED),
])
def test_sizes_named_by_the_header(rows, groups, dim, status, dtype):
    for fn in ("layer_norm_fwd", "layer_norm_bwd"):
        assert query(fn, rows, groups, dim, dtype)[0] == status


@pytest.mark.parametrize("dtype", [bd.F32, bd.BF16])
@pytest.mark.parametrize("groups,dim", [(1, 1000), (1, 1 << 20), (3, (1 << 23) + 1), (1, (1 << 26) - 17), (8191, 8192)])
def test_partial_sums_fit_the_workspace_and_the_grid(groups, dim, dtype):
    """256 columns and one share of the rows a workgroup, fewer than 2^24 workgroups of 256: the shares that the
    workspace has room for, two sums each."""
    st, n = query("layer_norm_bwd", 100000, groups, dim, dtype)
    assert st == bd.OK
    parts = n // (2 * groups * dim * 4)
    assert parts * 2 * groups * dim * 4 == n and 1 <= parts <= -(-512 // groups)
    if dim > 8192:
        assert parts * groups * -(-dim // 256) < 1 << 24


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,dim", [(3, (1 << 21) + 3), (5, 1 << 20)])
def test_rows_of_millions(rows, dim, dtype):
    announce(f"norm {rows} x {dim} {dtype}")
    gen = torch.Generator(DEV).manual_seed(4)
    rn = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    x, dy = (rn(rows, dim) + 0.5).to(dtype), rn(rows, dim).to(dtype)
    w, b = 1.0 + 0.1 * rn(dim), 0.1 * rn(dim)
    f = bd.layer_norm_fwd(x, w, b)
    g = bd.layer_norm_bwd(dy, x, f["mean"], f["rstd"], w)
    x64, dy64, w64 = x.double(), dy.double(), w.double()
    mean = x64.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((x64 - mean) ** 2).mean(-1, keepdim=True) + 1e-5)
    # a thread adds dim / 256 terms one behind the other, each rounding at most 2^-24 of a sum of that many absolute
    # values; 16 more for the tree.  As an error of the mean: that times mean|x|.
    s = (dim / 256 + 16) * U32
    size = x64.abs().mean(-1)
    assert ((f["mean"].double() - mean[:, 0]).abs() <= s * size).all()
    assert ((f["rstd"].double() / rstd[:, 0] - 1).abs() <= s + (s * size) ** 2).all()
    mean, rstd = f["mean"].double()[:, None], f["rstd"].double()[:, None]
    h = (x64 - mean) * rstd
    half = torch.finfo(dtype).eps / 2
    # h is formed from a difference and a product, y from two more operations (2^-24 each, on the absolute values)
    y = h * w64 + b.double()
    assert ((f["y"].double() - y).abs() <= half * y.abs() + 4 * U32 * ((x64.abs() + mean.abs()) * rstd * w64.abs() + b.abs())).all()
    t = dy64 * w64
    c1, c2 = t.mean(-1, keepdim=True), (t * h).mean(-1, keepdim=True)
    dx = rstd * (t - c1 - h * c2)
    room = rstd * ((s + 4 * U32) * (t.abs().mean(-1, keepdim=True) + h.abs() * (t * h).abs().mean(-1, keepdim=True)) + 4 * U32 * t.abs())
    assert ((g["dx"].double() - dx).abs() <= half * dx.abs() + room).all()
    # rows terms, each of three operations
    for name, terms in (("dweight", dy64 * h), ("dbias", dy64)):
        size = (dy64.abs() * ((x64.abs() + mean.abs()) * rstd)).sum(0) if name == "dweight" else dy64.abs().sum(0)
        assert ((g[name].double() - terms.sum(0)).abs() <= (rows + 3) * U32 * size).all(), name
