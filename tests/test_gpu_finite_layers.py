"""The debug finiteness mode on what the delta rule writes in part: the token rows of packed
sequences (o and every token gradient) and the states that a one-token call names."""
import pytest
import torch

from delta_ref import BF, F32, inputs
from gpu_common import announce
from selective_state_space_vjp_amd import binding as bd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAN = float("nan")


@pytest.fixture
def mode(monkeypatch):
    monkeypatch.setenv("SSMVJP_CHECK_FINITE", "1")


def dev(d):
    return {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def fwd(t, **kw):
    return bd.delta_chunk_fwd(t["q"], t["k"], t["v"], t["beta"], t["g"], t["S0"], scale=t["scale"],
                              seq_offsets=t["offsets"], **kw)


def bwd(t, **kw):
    return bd.delta_chunk_bwd(t["q"], t["k"], t["v"], t["beta"], t["g"], t["S0"], t["d_o"], t["dS"], scale=t["scale"],
                              seq_offsets=t["offsets"], **kw)


def nonfinite(fn):
    with pytest.raises(bd.SsmVjpError) as e:
        fn()
    assert e.value.status == bd.ENONFINITE


def case(dtype):
    """Three sequences in the middle of 200 tokens; NaN in the inputs of the tokens that none owns."""
    d = inputs(3, 200, 1, 2, 64, 48, dtype, True, [50, 0, 90], seed=1)
    d["offsets"] += 30
    for n in ("q", "k", "v", "beta", "g", "d_o"):
        d[n][:, :30] = NAN
        d[n][:, 170:] = NAN
    return dev(d)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_packed_outputs_without_states(mode, dtype):
    """With no final state asked for, o alone can show a value that is not a number."""
    announce(f"finite packed forward {dtype}")
    t = case(dtype)
    o = torch.full_like(t["v"], NAN)  # rows that no sequence owns stay as they are, and say nothing
    fwd(t, out=dict(o=o, S_final=None))
    assert torch.isnan(o[:, :30]).all() and torch.isnan(o[:, 170:]).all() and torch.isfinite(o[:, 30:170]).all()
    for at in (30, 79, 80, 169):  # the first and last tokens of both sequences
        bad = dict(t, v=t["v"].clone())
        bad["v"][0, at, 1, 47] = NAN
        nonfinite(lambda: fwd(bad, want_final=False))


def test_packed_gradients_without_states(mode):
    announce("finite packed backward")
    t = case(BF)
    like = dict(dq="q", dk="k", dv="v", dbeta="beta", dg="g")
    out = {n: torch.full_like(t[x], NAN) for n, x in like.items()}
    bwd(t, out=dict(out, dS0=None))
    for n in out:
        assert torch.isnan(out[n][:, :30]).all() and torch.isfinite(out[n][:, 30:170]).all(), n
    for at in (30, 79, 80, 169):
        bad = dict(t, d_o=t["d_o"].clone())
        bad["d_o"][0, at, 0, 0] = float("inf")
        nonfinite(lambda: bwd(bad, want_dS0=False))


@pytest.mark.parametrize("slotted", [False, True])
def test_states_of_one_token_calls(mode, slotted):
    """q = 0: o is zero whatever the state becomes, and only the state shows that it left float32's range."""
    announce(f"finite one token, slots={slotted}")
    n, HV, K, V = 6, 2, 32, 48
    q, k = torch.zeros(3, 1, K, device=DEV), torch.zeros(3, 1, K, device=DEV)
    v, beta, g = torch.zeros(3, HV, V, device=DEV), torch.full((3, HV), -1.0, device=DEV), torch.zeros(3, HV, device=DEV)
    k[:, :, 5] = 1.0
    slots = torch.tensor([4, -1, 1], dtype=torch.int32, device=DEV) if slotted else None
    good = torch.ones(n, HV, K, V, device=DEV)
    good[5] = NAN  # no request's
    if slotted:
        good[0] = float("inf")
    pool = good.clone()
    o = bd.delta_step(q, k, v, beta, g, pool, scale=1.0, slots=slots)
    assert (o == 0).all()
    pool = good.clone()
    pool[1, 1, 5, 47] = 3e38  # r = -3e38, beta = -1: the row doubles
    nonfinite(lambda: bd.delta_step(q, k, v, beta, g, pool, scale=1.0, slots=slots))
    assert torch.isinf(pool[1, 1, 5, 47])
