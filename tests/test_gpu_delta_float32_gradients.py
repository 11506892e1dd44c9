"""The float32 gradients of delta_chunk_fwd as the header says they are to be had: delta_rule_bwd
with the gate repeated over the key channels, heads padded with zeros to 128 keys and a multiple
of 32 columns, sequences one by one."""
import pytest
import torch
from torch.nn.functional import pad

from delta_ref import F32, TOL_F32, check, inputs, reference, spans
from gpu_common import announce
from selective_state_space_vjp_amd import binding as bd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
OUT = ("dq", "dk", "dv", "dbeta", "dg", "dS0")


def status(fn):
    with pytest.raises(bd.SsmVjpError) as e:
        fn()
    return e.value.status


@pytest.mark.parametrize("shape", [
    (2, 70, 2, 4, 128, 64, None),
    (1, 33, 1, 3, 48, 16, None),
    (3, 100, 1, 2, 80, 112, [41, 0, 59]),
], ids=str)
def test_padded_delta_rule_bwd(shape):
    announce(f"delta float32 gradients {shape}")
    b, T, H, HV, K, V, packed = shape
    d = inputs(b, T, H, HV, K, V, F32, True, packed, seed=T)
    t = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    assert status(lambda: bd.delta_chunk_bwd(t["q"], t["k"], t["v"], t["beta"], t["g"], t["S0"], t["d_o"], t["dS"],
                                             scale=t["scale"], seq_offsets=t["offsets"])) == bd.EUNSUPPORTED
    pk, pv = 128 - K, -V % 32
    got = {n: torch.zeros_like(t[x]) for n, x in zip(OUT, ("q", "k", "v", "beta", "g", "S0"))}
    for i, (row, a, e) in enumerate(spans(d)):
        if a == e:
            got["dS0"][i] = t["dS"][i]
            continue
        one = lambda n: t[n][row:row + 1, a:e]  # noqa: E731
        call = lambda q, k, v, g, S0, do, dS: bd.delta_rule_bwd(  # noqa: E731
            *(x.clone(memory_format=torch.contiguous_format)  # a sequence's rows may start off 16 bytes
              for x in (q, k, v, one("beta"), g, S0, do, dS)), scale=t["scale"])
        g = one("g")[..., None]
        if pk or pv:  # without the padding it takes no such head
            assert status(lambda: call(one("q"), one("k"), one("v"), g.expand(*g.shape[:-1], K), t["S0"][i:i + 1],
                                       one("d_o"), t["dS"][i:i + 1])) == bd.EUNSUPPORTED
        r = call(pad(one("q"), (0, pk)), pad(one("k"), (0, pk)), pad(one("v"), (0, pv)), g.expand(*g.shape[:-1], 128),
                 pad(t["S0"][i:i + 1], (0, pv, 0, pk)), pad(one("d_o"), (0, pv)), pad(t["dS"][i:i + 1], (0, pv, 0, pk)))
        got["dq"][row, a:e], got["dk"][row, a:e] = r["dq"][0, ..., :K], r["dk"][0, ..., :K]
        got["dv"][row, a:e], got["dbeta"][row, a:e] = r["dv"][0, ..., :V], r["dbeta"][0]
        got["dg"][row, a:e], got["dS0"][i] = r["dg"][0].sum(-1), r["dS0"][0, :, :K, :V]
    check(got, reference(d), {n: TOL_F32 for n in OUT}, str(shape))


def test_bf16_values_as_float32_keep_the_states():
    """States of 300 tokens from the same values in both types: two bf16 parts against float32 throughout."""
    announce("delta float32 states")
    d = inputs(2, 300, 1, 2, 64, 64, torch.bfloat16, True, None, seed=5)
    ref = reference(d, grads=False)
    wide = {k: (v.to(DEV).float() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    f = bd.delta_chunk_fwd(*(wide[n] for n in ("q", "k", "v", "beta", "g", "S0")), scale=wide["scale"])
    # 300 tokens, each with a product, two sums of 64 terms and an update, of independent roundings of 2^-24 / sqrt(3):
    # sqrt(300 * 8) of them in the mean square (a sum in a tree of 6 levels)
    check(f, ref, dict(S_final=(300 * 8 / 3) ** 0.5 * 2.0**-24), "states")
