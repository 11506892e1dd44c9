"""linear_scan_fwd and linear_scan_bwd on borders that are not ascending: a border below one before it counts as that
one, so every output is that of the ascending borders, bit for bit; and on borders of no sequence at all."""
import math

import pytest
import torch

from block_ref import BF, C, F32, make_scan
from gpu_common import announce
from selective_state_space_vjp_amd import binding as bd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# the second border of a pair that falls lies above the one before it, below an earlier one: its sequence has no tokens
FALLS = [[0, 300, 7, 200, 900],
         [0, 300, 7, 299, 300, 301, 900],
         [0, 500, 400, 450, 100, 200, 499, 500, 640, 3, 900],
         [40, 5, 20, 39, 900, 1, 899, 900],
         [0, 1000000, -3, 5, 900],
         [900, 0, 900],
         [0] + [800] + [k % 700 for k in range(0, 900, 11)] + [900],
         [3 * k if k % 3 == 0 else 2 * k + k % 3 for k in range(301)],
         [3 * k if k % 2 else 2 * k for k in range(301)]]  # (falls, and no such sequence)


def rising(borders, T):
    out, most = [], 0
    for b in borders:
        most = max(most, min(max(b, 0), T))
        out.append(most)
    return out


def scan(form, dtype, borders, D, state, seed):
    d = make_scan(form, 1, 900, D, dtype, seed=seed)
    t = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    gen = torch.Generator().manual_seed(seed + 1)
    n = len(borders) - 1
    t["h0"], t["dh_final"] = (torch.randn(n, D, generator=gen).to(DEV) for _ in range(2)) if state else (None, None)
    return t


def outputs(t, borders, keep):
    """Every output of both directions, over NaN where the call does not write (rows of tokens: over 7)."""
    off = torch.tensor(borders, dtype=torch.int32, device=DEV)
    n, D = len(borders) - 1, t["x"].shape[2]
    new = lambda *s: torch.full(s, math.nan, device=DEV)  # noqa: E731
    gated = t["decay"] is not None
    kw = dict(input_gate=t["input_gate"], decay=t["decay"], c=C, seq_offsets=off)
    f = {"h": torch.full_like(t["x"], 7.0), "h_final": new(n, D), "ckpt": new(900 // 64 + n, D)}
    bd.linear_scan_fwd(t["x"], t["gate"], t["h0"], out=f, **kw)
    g = {"dx": torch.full_like(t["x"], 7.0), "dgate": torch.full_like(t["gate"], 7.0), "dh0": new(n, D)}
    if gated:
        g.update(dinput_gate=torch.full_like(t["x"], 7.0), ddecay=new(D))
    bd.linear_scan_bwd(t["x"], t["gate"], t["dh"], t["h0"], t["dh_final"], ckpt=f["ckpt"] if keep else None, out=g, **kw)
    torch.cuda.synchronize()
    return {**f, **g}


@pytest.mark.parametrize("borders", FALLS, ids=lambda b: f"{len(b) - 1} sequences {b[:5]}")
@pytest.mark.parametrize("form,dtype,D,state", [("log", F32, 16, True), ("gated", BF, 300, True), ("gated", F32, 5, False),
                                                ("log", BF, 1, True)])
def test_every_output_is_that_of_ascending_borders(form, dtype, D, state, borders):
    announce(f"linear scan falling borders {form} {dtype} D={D} {len(borders) - 1} sequences {borders[:5]}")
    t = scan(form, dtype, borders, D, state, seed=len(borders))
    up = rising(borders, 900)
    empty = torch.tensor([a == b for a, b in zip(up, up[1:])], device=DEV)
    assert any(a == b and c < d for a, b, c, d in zip(up, up[1:], borders, borders[1:])) or borders is FALLS[-1]
    for keep in (True, False):
        got, want = outputs(t, borders, keep), outputs(t, up, keep)
        for k in want:
            assert torch.equal(got[k], want[k]), (k, keep)
        # a sequence without tokens passes its state on
        for k, given in (("h_final", t["h0"]), ("dh0", t["dh_final"])):
            given = torch.zeros_like(got[k]) if given is None else given
            assert torch.equal(got[k][empty], given[empty]), (k, keep)
            assert torch.isfinite(got[k]).all(), (k, keep)


@pytest.mark.parametrize("form", ["log", "gated"])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_finiteness_mode_scans_what_ascending_borders_own(monkeypatch, form, dtype):
    """Rows that only the borders as they stand would give to a sequence say nothing; those that one owns do."""
    announce(f"linear scan falling borders, finiteness mode {form} {dtype}")
    monkeypatch.setenv("SSMVJP_CHECK_FINITE", "1")
    borders = [5, 300, 0, 4, 800] + [k % 700 for k in range(90)] + [850]  # 0 .. 4 and 850 .. 899 are nobody's
    t = scan(form, dtype, borders, 20, True, seed=3)
    own = torch.zeros(900, dtype=torch.bool)
    own[5:850] = True
    for k in ("x", "gate", "dh", "input_gate"):
        if t[k] is not None:
            t[k][0, ~own] = math.nan
    off = torch.tensor(borders, dtype=torch.int32, device=DEV)
    kw = dict(input_gate=t["input_gate"], decay=t["decay"], c=C, seq_offsets=off)

    def both(x, dh):
        out = {"h": torch.full_like(x, math.nan), "h_final": torch.empty_like(t["h0"])}  # unowned rows are left as they are
        bd.linear_scan_fwd(x, t["gate"], t["h0"], out=out, **kw)
        g = {"dx": torch.full_like(x, math.nan), "dgate": torch.full_like(t["gate"], math.nan), "dh0": torch.empty_like(t["h0"])}
        if form == "gated":
            g.update(dinput_gate=torch.full_like(x, math.nan), ddecay=torch.empty_like(t["decay"]))
        bd.linear_scan_bwd(t["x"], t["gate"], dh, t["h0"], t["dh_final"], out=g, **kw)

    both(t["x"], t["dh"])
    for at in (5, 299, 300, 799, 849):
        for k in ("x", "dh"):
            bad = t[k].clone()
            bad[0, at, 19] = math.nan
            with pytest.raises(bd.SsmVjpError) as e:
                both(*((bad, t["dh"]) if k == "x" else (t["x"], bad)))
            assert e.value.status == bd.ENONFINITE, (k, at)


@pytest.mark.parametrize("form", ["log", "gated"])
@pytest.mark.parametrize("T", [1, 64, 200, 5000])
def test_kept_states_of_no_sequences(form, T):
    """Packed tokens that no sequence owns, for there is none: rows of ckpt that no token has are zeros all the same."""
    announce(f"linear scan no sequences {form} T={T}")
    d = make_scan(form, 1, T, 70, BF, seed=T)
    t = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    kw = dict(input_gate=t["input_gate"], decay=t["decay"], c=C, seq_offsets=torch.tensor([3], dtype=torch.int32, device=DEV))
    none = torch.empty(0, 70, device=DEV)
    out = {"h": torch.full_like(t["x"], 7.0), "h_final": none, "ckpt": torch.full((T // 64, 70), math.nan, device=DEV)}
    bd.linear_scan_fwd(t["x"], t["gate"], none, out=out, **kw)
    assert (out["h"] == 7.0).all() and (out["ckpt"] == 0).all()
    for ckpt in (out["ckpt"], None):
        g = {"dx": torch.full_like(t["x"], 7.0), "dgate": torch.full_like(t["gate"], 7.0), "dh0": none}
        if form == "gated":
            g.update(dinput_gate=torch.full_like(t["x"], 7.0), ddecay=torch.full((70,), math.nan, device=DEV))
        bd.linear_scan_bwd(t["x"], t["gate"], t["dh"], none, none, ckpt=ckpt, out=g, **kw)
        assert all((v == (0.0 if k == "ddecay" else 7.0)).all() for k, v in g.items())
