"""The gated linear recurrence with decays near and past float32's largest."""
import math

import pytest
import torch

from block_ref import C
from gpu_common import announce
from selective_state_space_vjp_amd import binding as bd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_decays_whose_rate_overflows():
    """c softplus(decay) log2(e) past float32's largest: a = 0 wherever the recurrence gate is not shut (sigmoid(-200) is 0
    in float32: a = 1 there), h = sigmoid(i) x and its gradients, nothing of the decay's or the gate's."""
    announce("linear scan decays that overflow")
    T, D = 200, 6
    gen = torch.Generator().manual_seed(5)
    x, ig, dh = (torch.randn(1, T, D, generator=gen).to(DEV) for _ in range(3))
    gate = torch.randn(1, T, D, generator=gen).to(DEV)
    gate[..., 3:] = -200.0
    decay = torch.tensor([1e38, 3.4e38, math.inf] * 2, device=DEV)
    kw = dict(input_gate=ig, decay=decay, c=C)
    h0 = torch.ones(1, D, device=DEV)
    out = bd.linear_scan_fwd(x, gate, h0, **kw)
    got = bd.linear_scan_bwd(x, gate, dh, h0, h0, **kw)
    for k, v in {**out, **got}.items():
        assert v is None or torch.isfinite(v).all(), k
    w, X, H = torch.sigmoid(ig.double()), x.double(), dh.double()
    lam = H.clone()
    lam[:, -1] += 1.0
    u = 16 * 2.0**-24  # sigmoid and two products
    for name, have, want in (("h", out["h"], w * X), ("dx", got["dx"], lam * w), ("dinput_gate", got["dinput_gate"], lam * w * (1 - w) * X)):
        err = (have.double() - want)[..., :3].abs()
        assert (err <= 4 * u * (lam.abs() * X.abs() + X.abs() + lam.abs())[..., :3]).all(), name
    assert (got["dgate"] == 0).all() and (got["ddecay"] == 0).all() and (got["dh0"][:, :3] == 0).all()
    # shut: the state stays, x never enters
    assert (out["h"][..., 3:] == 1).all() and (got["dx"][..., 3:] == 0).all()
    step = h0.clone()
    h = bd.linear_scan_step(x[:, 0].contiguous(), gate[:, 0].contiguous(), step, input_gate=ig[:, 0].contiguous(), decay=decay, c=C)
    assert torch.equal(h, out["h"][:, 0]) and torch.equal(step, h)
