"""The reference of the delta rule with one gate per value head (tests/delta_ref.py), in
float64 on the CPU: its gradients against differences of its own forward, and its forward
against the recurrence written out."""
import numpy as np
import torch

from delta_ref import F32, inputs, reference, spans


def _objective(d):
    r = reference(d, grads=False)
    return float((r["o"] * d["d_o"].double()).sum() + (r["S_final"] * d["dS"].double()).sum())


def _case():
    d = inputs(1, 11, 2, 4, 16, 16, F32, True, [4, 0, 7], seed=2, rate=0.4)
    return {n: (t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t) for n, t in d.items()}


def test_gradients_against_differences():
    d = _case()
    ref = reference(d)
    gen = torch.Generator().manual_seed(9)
    h = 1e-5
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("beta", "dbeta"), ("g", "dg"), ("S0", "dS0")):
        for _ in range(3):
            x, e = d[name], torch.randn(d[name].shape, generator=gen, dtype=torch.float64)
            j = []
            for s in (h, -h):
                d[name] = x + s * e
                j.append(_objective(d))
            d[name] = x
            got = (j[0] - j[1]) / (2 * h)
            want = float((ref[grad] * e).sum())
            # central differences: h^2 of the third derivative, and 2^-53 of J over h
            assert abs(got - want) <= 1e-7 * (1 + abs(want) + float(ref[grad].norm() * e.norm())), (name, got, want)


def test_forward_is_the_recurrence():
    d = _case()
    ref = reference(d, grads=False)
    q, k, v, beta, g = (d[n].numpy() for n in ("q", "k", "v", "beta", "g"))
    rep = v.shape[2] // q.shape[2]
    for i, (row, a, e) in enumerate(spans(d)):
        for hv in range(v.shape[2]):
            S = d["S0"][i, hv].numpy().copy()
            for t in range(a, e):
                S *= np.exp(g[row, t, hv])
                r = v[row, t, hv] - k[row, t, hv // rep] @ S
                S += np.outer(k[row, t, hv // rep], beta[row, t, hv] * r)
                np.testing.assert_allclose(ref["o"][row, t, hv].numpy(), d["scale"] * q[row, t, hv // rep] @ S, atol=1e-13)
            np.testing.assert_allclose(ref["S_final"][i, hv].numpy(), S, atol=1e-13)
