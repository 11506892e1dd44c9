"""A value that is not finite reaches its own token and those behind it, in the chunked forward of
the delta rule as in the definition: garbage behind the end of a padded sequence leaves the tokens
before it alone."""
import pytest
import torch

from delta_ref import BF, inputs, reference
from gpu_common import announce
from selective_state_space_vjp_amd import binding as bd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAN, INF = float("nan"), float("inf")


def fwd(d):
    t = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    out = bd.delta_chunk_fwd(t["q"], t["k"], t["v"], t["beta"], t["g"], t["S0"], scale=t["scale"], seq_offsets=t["offsets"])
    return {n: x.cpu() for n, x in out.items()}


def put(d, name, at, value):
    d = dict(d, **{name: d[name].clone()})
    d[name][at] = value
    return d


# equal sequences; packed ones with their second border inside a chunk; the state before, narrow and wide heads
SHAPES = [(2, 150, 2, 4, 128, 48, None), (1, 150, 1, 2, 48, 32, None), (3, 170, 1, 2, 64, 64, [40, 0, 130])]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("name,value", [("v", NAN), ("v", INF), ("k", NAN), ("k", -INF), ("q", NAN), ("q", INF), ("beta", NAN),
                                        ("beta", INF), ("g", NAN)])
def test_only_the_tokens_behind_it(shape, name, value):
    announce(f"delta causal {shape} {name} {value}")
    b, T, H, HV, K, V, packed = shape
    d = inputs(b, T, H, HV, K, V, BF, True, packed, seed=K)
    clean = fwd(d)
    row = b - 1 if packed is None else 0
    for t in (0, 1, 5, 15, 16, 31, 32, 40, 50, 62, 63, 64, 95, 100, 127, 128, 149):
        at = (row, t, -1) if name in ("beta", "g") else (row, t, -1, 7)
        bad = put(d, name, at, value)
        got, ref = fwd(bad), reference(bad, grads=False)
        for n in ("o", "S_final"):
            ok = torch.isfinite(ref[n])
            assert torch.equal(torch.isfinite(got[n]), ok), (n, t)
            assert torch.equal(got[n][ok], clean[n][ok]), (n, t)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_lost_columns_of_the_initial_state(shape):
    announce(f"delta causal S0 {shape}")
    b, T, H, HV, K, V, packed = shape
    d = inputs(b, T, H, HV, K, V, BF, True, packed, seed=V)
    clean = fwd(d)
    bad = put(d, "S0", (b - 1, 1, 3, 17), NAN)
    got, ref = fwd(bad), reference(bad, grads=False)
    for n in ("o", "S_final"):
        ok = torch.isfinite(ref[n])
        assert torch.equal(torch.isfinite(got[n]), ok) and torch.equal(got[n][ok], clean[n][ok]), n


def test_padded_batch():
    """Sequences of 100, 33 and 150 tokens in 150: NaN in every input behind their ends."""
    announce("delta causal padding")
    d = inputs(3, 150, 2, 4, 128, 64, BF, True, None, seed=9)
    clean = fwd(d)
    bad, lens = {k: (v.clone() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}, (100, 33, 150)
    for i, n in enumerate(lens):
        for name in ("q", "k", "v", "beta", "g"):
            bad[name][i, n:] = NAN
    got = fwd(bad)
    for i, n in enumerate(lens):
        assert torch.equal(got["o"][i, :n], clean["o"][i, :n]), i
        assert torch.isnan(got["o"][i, n:]).all()
    assert torch.equal(got["S_final"][2], clean["S_final"][2])
