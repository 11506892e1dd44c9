"""The debug finiteness mode on the outputs of the linear recurrence, the gated feed-forward projections and dropout."""
import math

import pytest
import torch

from block_ref import BF, C, F32, make_scan
from gpu_common import announce
from selective_state_space_vjp_amd import binding as bd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAN = math.nan


@pytest.fixture
def mode(monkeypatch):
    monkeypatch.setenv("SSMVJP_CHECK_FINITE", "1")


def nonfinite(fn):
    with pytest.raises(bd.SsmVjpError) as e:
        fn()
    assert e.value.status == bd.ENONFINITE


@pytest.mark.parametrize("form", ["log", "gated"])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_scan(mode, form, dtype):
    announce(f"finite scan {form} {dtype}")
    d = make_scan(form, 1, 0, 20, dtype, lens=[50, 0, 90], first=30, tail=30, seed=1)
    for k in ("x", "gate", "dh", "input_gate"):
        if d[k] is not None:
            d[k][:, :30] = NAN
            d[k][:, 170:] = NAN
    t = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    args = dict(input_gate=t["input_gate"], decay=t["decay"], c=C, seq_offsets=t["seq_offsets"])
    fwd = lambda x, **kw: bd.linear_scan_fwd(x, t["gate"], t["h0"], **args, **kw)  # noqa: E731
    bwd = lambda dh, **kw: bd.linear_scan_bwd(t["x"], t["gate"], dh, t["h0"], t["dh_final"], **args, **kw)  # noqa: E731
    # rows that no sequence owns say nothing
    o = fwd(t["x"], want_ckpt=True)
    bwd(t["dh"], ckpt=o["ckpt"])
    bwd(t["dh"])
    for at in (30, 79, 80, 169):
        x = t["x"].clone()
        x[0, at, 19] = NAN
        nonfinite(lambda: fwd(x))
        nonfinite(lambda: fwd(x, want_final=False))
        dh = t["dh"].clone()
        dh[0, at, 0] = math.inf
        nonfinite(lambda: bwd(dh))


def test_step(mode):
    announce("finite step")
    x, g = torch.randn(3, 40, device=DEV), -torch.rand(3, 40, device=DEV)
    pool = torch.randn(6, 40, device=DEV)
    pool[5] = NAN  # a state that no request names
    slots = torch.tensor([4, -1, 0], dtype=torch.int32, device=DEV)
    bd.linear_scan_step(x, g, pool, slots=slots)
    pool[0, 39] = NAN
    nonfinite(lambda: bd.linear_scan_step(x, g, pool, slots=slots))


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_ffn_and_dropout(mode, dtype):
    announce(f"finite ffn, dropout {dtype}")
    x, w, dh = torch.randn(70, 64, device=DEV).to(dtype), torch.randn(96, 64, device=DEV).to(dtype), torch.randn(70, 96, device=DEV).to(dtype)
    o = bd.gated_ffn_fwd(x, w, w, want_saved=True)
    bd.gated_ffn_bwd(dh, x, w, w, saved=(o["gate"], o["up"]))
    x2 = x.clone()
    x2[69, 63] = NAN
    nonfinite(lambda: bd.gated_ffn_fwd(x2, w, w))
    nonfinite(lambda: bd.gated_ffn_bwd(dh, x2, w, w))
    nonfinite(lambda: bd.gated_ffn_bwd(dh, x2, w, w, want_dx=False, saved=(o["gate"], o["up"])))
    rng = torch.tensor([1, 2], dtype=torch.int64, device=DEV)
    bd.dropout_fwd(x, rng, x, p=0.3)
    nonfinite(lambda: bd.dropout_fwd(x, rng, x2, p=0.3))
    bd.dropout_fwd(x2, rng, p=1.0)  # dropped: it leaves no trace
    nonfinite(lambda: bd.dropout_bwd(x2, rng, p=0.0))
