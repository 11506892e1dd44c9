"""The float64 references of the linear recurrence, the gated feed-forward block and dropout: gradients
against differences, the generator against its published test vectors, no value beyond its own bound."""
import pytest
import torch

from block_ref import BF, F32, act, coefficients, ffn_reference, keep_mask, make_scan, philox, scan_forward, scan_reference


def test_generator_known_answers():
    """The known answers that the generator's authors publish beside it."""
    assert philox((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    f = 0xFFFFFFFF
    assert philox((f, f, f, f), (f, f)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    pi = (0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344)
    assert philox(pi, (0xA4093822, 0x299F31D0)) == [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


def test_mask_has_its_probability():
    for p in (0.1, 0.5, 0.9):
        n = 40000
        kept = float(keep_mask(n, p, 12345, 7).double().mean())
        assert abs(kept - (1 - p)) < 5 * (p * (1 - p) / n) ** 0.5
    assert keep_mask(100, 0.0, 1, 2).all() and not keep_mask(100, 1.0, 1, 2).any()


@pytest.mark.parametrize("form", ["log", "gated"])
def test_scan_gradients_against_differences(form):
    d = make_scan(form, 1, 0, 3, F32, lens=[4, 0, 3], seed=3, first=1, tail=2)
    ref = scan_reference(d)
    name = {"x": "dx", "gate": "dgate", "input_gate": "dinput_gate", "decay": "ddecay", "h0": "dh0"}

    def J(e):
        hs, last = scan_forward(e)
        v = (last * d["dh_final"].double()).sum()
        at = d["first"]
        for h in hs:
            v = v + (h * d["dh"][0, at:at + len(h)].double()).sum()
            at += len(h)
        return float(v)

    checked = 0
    for k, g in name.items():
        if d[k] is None:
            continue
        flat = d[k].double().reshape(-1)
        for i in range(flat.numel()):
            v = []
            for s in (1e-5, -1e-5):
                e = flat.clone()
                e[i] += s
                v.append(J(dict(d, **{k: e.reshape(d[k].shape)})))
            assert abs((v[0] - v[1]) / 2e-5 - float(ref[g][0].reshape(-1)[i])) < 1e-7, (k, i)
            checked += 1
    assert checked > 50


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_ffn_gradients_against_differences(name):
    gen = torch.Generator().manual_seed(1)
    x, wg, wu, dh = (torch.randn(s, generator=gen, dtype=torch.float64) for s in ((3, 4), (5, 4), (5, 4), (3, 5)))
    ref = ffn_reference(x, wg, wu, dh, name)
    J = lambda x, wg, wu: float((dh * act(name, x @ wg.T) * (x @ wu.T)).sum())  # noqa: E731
    ts = [x, wg, wu]
    for j, g in enumerate(("dx", "dw_gate", "dw_up")):
        for i in range(ts[j].numel()):
            v = []
            for s in (1e-6, -1e-6):
                e = [t.clone() for t in ts]
                e[j].view(-1)[i] += s
                v.append(J(*e))
            assert abs((v[0] - v[1]) / 2e-6 - float(ref[g][0].reshape(-1)[i])) < 1e-7


@pytest.mark.parametrize("form", ["log", "gated"])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_float32_loop_stays_inside_the_bounds(form, dtype):
    """The definition token by token in float32: what the bounds are meant to allow."""
    d = make_scan(form, 2, 150, 6, dtype, seed=5, reset=True)
    ref = scan_reference(d)
    a, u = (t.float() for t in coefficients(d))
    h = d["h0"].clone()
    for t in range(150):
        h = a[:, t] * h + u[:, t]
    want, bound = ref["h_final"]
    assert ((h.double() - want).abs() <= bound).all()
    assert float((bound / want.abs().clamp(min=1e-3)).max()) < 0.05  # and no more than that
