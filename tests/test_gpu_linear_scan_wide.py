"""The linear recurrence over many groups of tiles and many slabs of channels at once, and on inputs of more than 128 MB,
which the kernels read by streaming loads.  Channels know nothing of each other and a channel's operations are the same
in every slab and with either kind of load, so every output is that of its channels by themselves, bit for bit: those
are one slab, or inputs below that size, which the other tests hold to the definition in float64."""
import math

import pytest
import torch

from block_ref import BF, C, F32
from gpu_common import announce
from selective_state_space_vjp_amd import binding as bd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def make(form, n, T, D, dtype, borders, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    b = n if borders is None else len(borders) - 1
    t = dict(x=rn(n, T, D).to(dtype), dh=rn(n, T, D).to(dtype), h0=rn(b, D), dh_final=rn(b, D), input_gate=None, decay=None,
             seq_offsets=None if borders is None else torch.tensor(borders, dtype=torch.int32, device=DEV))
    if form == "gated":
        t.update(gate=rn(n, T, D).to(dtype), input_gate=rn(n, T, D).to(dtype), decay=torch.linspace(-9.0, -2.5, D, device=DEV))
    else:
        t["gate"] = rn(n, T, D).abs_() * -torch.exp(torch.linspace(math.log(0.001), math.log(2.0), D, device=DEV))
    return t


def run(t):
    kw = dict(input_gate=t["input_gate"], decay=t["decay"], c=C, seq_offsets=t["seq_offsets"])
    f = bd.linear_scan_fwd(t["x"], t["gate"], t["h0"], want_ckpt=True, **kw)
    kept = bd.linear_scan_bwd(t["x"], t["gate"], t["dh"], t["h0"], t["dh_final"], ckpt=f["ckpt"], **kw)
    again = bd.linear_scan_bwd(t["x"], t["gate"], t["dh"], t["h0"], t["dh_final"], **kw)
    torch.cuda.synchronize()
    return {**f, **kept, **{k + " again": v for k, v in again.items()}}


def compare(t, own, width):
    D = t["x"].shape[2]
    whole = run(t)
    for c0 in range(0, D, width):
        cut = {k: v if v is None or k == "seq_offsets" else v[..., c0:c0 + width].contiguous() for k, v in t.items()}
        part = run(cut)
        for k, v in part.items():
            assert (v is None) == (whole[k] is None), k
            if v is None:
                continue
            got = whole[k][..., c0:c0 + width]
            if v.shape == cut["x"].shape:  # rows that a sequence owns
                got, v = got[:, own], v[:, own]
            assert torch.isfinite(v).all() and torch.equal(got, v), (k, c0)


def owned(t):
    T = t["x"].shape[1]
    return slice(0, T) if t["seq_offsets"] is None else slice(int(t["seq_offsets"][0]), int(t["seq_offsets"][-1]))


@pytest.mark.parametrize("borders", [None, [3, 2200, 2200, 2230, 5000, 5064]], ids=["equal", "packed"])
@pytest.mark.parametrize("n,D,width", [(2, 300, 128), (1, 1000, 128), (2, 131, 64)])
@pytest.mark.parametrize("form,dtype", [("log", F32), ("gated", BF), ("log", BF), ("gated", F32)])
def test_groups_and_slabs(form, dtype, n, D, width, borders):
    """2 to 5 groups of 16 tiles of 128 (forward) and 64 (backward) tokens, 3 to 8 slabs; 131: one channel a lane."""
    T = 2300 if borders is None else 5100
    announce(f"linear scan groups and slabs {form} {dtype} n={n} T={T} D={D}")
    t = make(form, n if borders is None else 1, T, D, dtype, borders, n + D)
    compare(t, owned(t), width)


@pytest.mark.parametrize("borders", [None, [0, 3000, 3001, 5801]], ids=["equal", "packed"])
@pytest.mark.parametrize("form,dtype", [("log", F32), ("gated", BF), ("log", BF), ("gated", F32)])
def test_inputs_that_are_streamed(form, dtype, borders):
    """23.8 million values: 143 MB at the least that both passes read, 95 MB at the most of a quarter of the channels."""
    n, T, D = (2, 2900, 4096) if borders is None else (1, 5801, 4096)
    announce(f"linear scan streamed {form} {dtype} n={n} T={T}")
    t = make(form, n, T, D, dtype, borders, T)
    values = n * T * D
    size = t["x"].element_size()
    first = values * (3 * size if form == "gated" else size + 4)
    assert first > 128 << 20 and (first + values * size) // 4 <= 128 << 20
    compare(t, owned(t), D // 4)
