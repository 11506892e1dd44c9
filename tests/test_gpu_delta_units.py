"""dbeta and dg where a workgroup of the gradients kernel goes from unit to unit and from value head to
value head: their gates, row sums and column sums are carried or loaded ahead from one to the next."""
import pytest
import torch

from delta_ref import BF, TOL_BF16, TOL_SPLIT, check, inputs, reference
from gpu_common import announce
from selective_state_space_vjp_amd import binding as bd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("shape", [
    (24, 24, 64, 32),   # one value head a qk head, 768 units
    (24, 48, 64, 32),   # two
    (24, 72, 128, 16),  # three: the double buffer of the gates changes sides at every unit
    (16, 32, 16, 16),   # few cells (terms of dg from float32 states), 512 units
], ids=str)
def test_gate_gradients_over_many_units(shape):
    announce(f"delta dbeta and dg {shape}")
    H, HV, K, V = shape
    lens = [130, 0, 1, 64, 65, 200, 0, 63] * 2
    d = inputs(1, sum(lens), H, HV, K, V, BF, True, lens, seed=HV)
    t = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    run = lambda: bd.delta_chunk_bwd(t["q"], t["k"], t["v"], t["beta"], t["g"], t["S0"], t["d_o"], t["dS"],  # noqa: E731
                                     scale=t["scale"], seq_offsets=t["offsets"])
    got = run()
    ref = reference(d)
    tol = dict(dq=TOL_BF16, dk=TOL_BF16, dv=TOL_BF16, dbeta=TOL_SPLIT, dg=TOL_SPLIT, dS0=TOL_SPLIT)
    check(got, ref, tol, "all")
    at = 0
    for i, n in enumerate(lens):  # and of every sequence by itself: one bad unit is not lost in the norm of all
        part = {m: got[m][:, at:at + n] for m in ("dbeta", "dg")}
        want = {m: ref[m][:, at:at + n] for m in ref if m in ("dbeta", "dg", "scale of dbeta", "scale of dg")}
        check(part, want, dict(dbeta=TOL_SPLIT, dg=TOL_SPLIT), f"sequence {i} of {n}")
        at += n
    again = run()
    for m in got:
        assert torch.equal(got[m], again[m]), m
