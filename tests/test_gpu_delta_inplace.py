"""Gradients of the chunked delta rule with dS0 written over S0, which the header allows, at sizes
whose workgroups cannot all be resident at once: what the forward walk reads must not yet be
overwritten by the reverse walk."""
import pytest
import torch

from delta_ref import BF, inputs
from gpu_common import announce
from selective_state_space_vjp_amd import binding as bd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def bwd(t, dS0=None):
    """Into tensors of sevens, which stay where no sequence owns a row; dS0 into a tensor of the caller's."""
    like = dict(dq="q", dk="k", dv="v", dbeta="beta", dg="g", dS0="S0")
    out = {n: torch.full_like(t[x], 7.0) for n, x in like.items()}
    if dS0 is not None:
        out["dS0"] = dS0
    return bd.delta_chunk_bwd(t["q"], t["k"], t["v"], t["beta"], t["g"], t["S0"], t["d_o"], t["dS"], scale=t["scale"],
                              seq_offsets=t["offsets"], out=out)


# workgroups per walk: 32 columns of a head's state each; a workgroup takes a CU, of which there are 256
@pytest.mark.parametrize("shape", [
    (1, 2048, 16, 48, 128, 128, None),                     # 192
    (3, 70, 8, 32, 128, 128, None),                        # 384
    (3, 70, 8, 32, 64, 128, None),                         # the same, K <= 64
    (36, 400, 8, 8, 64, 32, [0, 1, 20, 63, 0, 2] * 6),     # 288, empty and short sequences
    (64, 20, 8, 8, 16, 16, None),                          # 512, few cells
    (40, 100, 2, 8, 16, 32, [0, 3, 0, 1, 6] * 8),          # 320, few cells, empty and short sequences
    (1, 130, 1, 2, 128, 32, None),                         # few cells, K > 64
], ids=str)
def test_state_gradient_over_the_initial_state(shape):
    announce(f"delta dS0 over S0 {shape}")
    b, T, H, HV, K, V, packed = shape
    d = inputs(b, T, H, HV, K, V, BF, True, packed, seed=T + V)
    t = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    for name in ("S0", "dS", "both"):
        u = dict(t)
        if name == "both":  # one buffer for the initial state, the gradient given and the gradient returned
            want = bwd(dict(t, dS=t["S0"]))
            over = u["S0"] = u["dS"] = t["S0"].clone()
        else:
            want = bwd(t)
            over = u[name] = t[name].clone()
        got = bwd(u, over)
        for n in want:
            assert torch.equal(got[n], want[n]), (name, n)
