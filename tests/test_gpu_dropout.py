"""dropout_fwd and dropout_bwd against the generator word by word in Python integers."""
import math

import pytest
import torch

from block_ref import BF, F32, HALF, U, dropout_reference, keep_mask
from gpu_common import announce
from selective_state_space_vjp_amd import binding as bd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def rng(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device=DEV)


@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (9,), (3, 5, 7), (2048,), (2049,), (33, 1001), (5, 4096)], ids=str)
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.93, 1.0])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_against_the_generator(shape, p, dtype):
    announce(f"dropout {shape} {p} {dtype}")
    gen = torch.Generator().manual_seed(1)
    x, res = torch.randn(shape, generator=gen).to(dtype), torch.randn(shape, generator=gen).to(dtype)
    seed, offset = -0x123456789ABCDEF, (1 << 40) + 17
    t = rng(seed, offset)
    for r in (None, res):
        want, keep = dropout_reference(x, p, seed, offset, r)
        got = bd.dropout_fwd(x.to(DEV), t, None if r is None else r.to(DEV), p=p).double().cpu()
        # the scale, the product and the sum in float32, then one rounding
        bound = (HALF[dtype] * want.abs() + 3 * U * (want.abs() + (0 if r is None else r.double().abs()))) * (1 + U)
        assert ((got - want).abs() <= bound).all()
        assert torch.equal(got[~keep], torch.zeros_like(want)[~keep] if r is None else r.double()[~keep])
    want, _ = dropout_reference(x, p, seed, offset)
    dx = bd.dropout_bwd(x.to(DEV), t, p=p)
    assert torch.equal(dx, bd.dropout_fwd(x.to(DEV), t, p=p))


def test_seeds_offsets_and_determinism():
    announce("dropout seeds")
    x = torch.ones(1 << 16, device=DEV)
    base = bd.dropout_fwd(x, rng(5, 0), p=0.5)
    assert torch.equal(base, bd.dropout_fwd(x, rng(5, 0), p=0.5))
    for s, o in ((6, 0), (5, 1), (5 + (1 << 32), 0), (5, 1 << 32)):
        other = bd.dropout_fwd(x, rng(s, o), p=0.5)
        assert 0.45 < float((other == base).double().mean()) < 0.55, (s, o)
    assert abs(float(base.double().mean()) - 1) < 0.02


def test_dropped_values_leave_no_trace_and_in_place():
    announce("dropout nan, in place")
    n = 5000
    keep = keep_mask(n, 0.4, 3, 9).to(DEV)
    x = torch.where(keep, 1.0, math.nan)
    y = bd.dropout_fwd(x, rng(3, 9), p=0.4)
    assert torch.isfinite(y).all() and (y[~keep] == 0).all()
    for dtype in (F32, BF):
        x, r = torch.randn(n, device=DEV).to(dtype), torch.randn(n, device=DEV).to(dtype)
        want = bd.dropout_fwd(x, rng(3, 9), r, p=0.4)
        a = x.clone()
        assert bd.dropout_fwd(a, rng(3, 9), r, p=0.4, out=a) is a and torch.equal(a, want)
        b = r.clone()
        bd.dropout_fwd(x, rng(3, 9), b, p=0.4, out=b)
        assert torch.equal(b, want)
        # odd element offsets
        f = torch.empty(n + 1, device=DEV, dtype=dtype)
        f[1:] = x
        assert torch.equal(bd.dropout_fwd(f[1:], rng(3, 9), r, p=0.4), want)


def test_captured_call_reads_the_generator_state():
    """A replay draws from the rng as it is then."""
    announce("dropout graph")
    t, x = rng(1, 0), torch.ones(3000, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = bd.dropout_fwd(x, t, p=0.5)
        t[1] += 1
    seen = []
    t.copy_(rng(1, 0))
    for k in range(4):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, bd.dropout_fwd(x, rng(1, k), p=0.5))
        seen.append(y.clone())
    assert not torch.equal(seen[0], seen[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z = bd.dropout_fwd(x, rng(1, 2), p=0.5, stream=s)
    s.synchronize()
    assert torch.equal(z, seen[2])


def test_empty():
    assert bd.dropout_fwd(torch.empty(0, 4, device=DEV), rng(0, 0), p=0.3).shape == (0, 4)
