"""GPU parity of linear_scan_fwd, linear_scan_bwd and linear_scan_step against the definition in float64, at the
lengths, widths and borders where they can go wrong."""
import math

import pytest
import torch

from block_ref import BF, C, F32, HALF, U, check, coefficients, make_scan, owned, scan_reference
from gpu_common import announce
from selective_state_space_vjp_amd import binding as bd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dev(d):
    return {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def fwd(t, **kw):
    return bd.linear_scan_fwd(t["x"], t["gate"], t["h0"], input_gate=t["input_gate"], decay=t["decay"], c=C,
                              seq_offsets=t["seq_offsets"], **kw)


def bwd(t, **kw):
    return bd.linear_scan_bwd(t["x"], t["gate"], t["dh"], t["h0"], t["dh_final"], input_gate=t["input_gate"], decay=t["decay"],
                              c=C, seq_offsets=t["seq_offsets"], **kw)


def ckpt_rows(d):
    """Where the state before each 64th token belongs, and which token that is."""
    rows, at = [], d["first"]
    if d["lens"] is None:
        n, T = d["x"].shape[:2]
        return [((i, j), (i, 64 * j)) for i in range(n) for j in range(-(-T // 64))]
    for s, k in enumerate(d["lens"]):
        rows += [((at // 64 + s + j,), (0, at + 64 * j)) for j in range(-(-k // 64))]
        at += k
    return rows


def compare(d, what):
    ref = scan_reference(d)
    t = dev(d)
    own = owned(d)
    out = fwd(t, want_ckpt=True)
    torch.cuda.synchronize()
    check(out["h"], *ref["h"], f"{what} h", own)
    check(out["h_final"], *ref["h_final"], f"{what} h_final")
    # a kept state is the state before its token: the h of the token before, to the bound of a state
    kept = out["ckpt"].double().cpu()
    seen = torch.zeros(kept.shape[:-1], dtype=torch.bool)
    h, bound = ref["h"]
    starts = {}
    for s, (row, at) in enumerate([(r, 0) for r in range(d["x"].shape[0])] if d["lens"] is None else
                                  [(0, d["first"] + sum(d["lens"][:i])) for i in range(len(d["lens"]))]):
        starts.setdefault((row, at), []).append(s)
    for where, (row, tok) in ckpt_rows(d):
        seen[where] = True
        if (row, tok) in starts:
            s = [q for q in starts[(row, tok)] if d["lens"] is None or d["lens"][q]][-1]
            want = torch.zeros(h.shape[-1], dtype=torch.float64) if d["h0"] is None else d["h0"][s].double()
            assert torch.equal(kept[where], want), (what, "ckpt", where)
        else:
            assert ((kept[where] - h[row, tok - 1]).abs() <= bound[row, tok - 1]).all(), (what, "ckpt", where)
    assert (kept[~seen] == 0).all()
    for ckpt in (out["ckpt"], None):
        got = bwd(t, ckpt=ckpt)
        torch.cuda.synchronize()
        for k, v in got.items():
            if v is None or (k == "dh0" and d["h0"] is None):
                continue
            check(v, *ref[k], f"{what} {k} {'kept' if ckpt is not None else 'formed again'}", own if v.dim() == 3 else None)
        assert (got["ddecay"] is None) == (d["form"] == "log")


EQUAL = [(1, 1, 1), (2, 1, 130), (1, 2, 7), (3, 15, 64), (1, 16, 128), (2, 17, 129), (1, 63, 3), (1, 64, 256), (2, 65, 2),
         (1, 127, 66), (1, 128, 130), (2, 129, 5), (1, 200, 1001), (2, 300, 258), (1, 1025, 33)]


@pytest.mark.parametrize("n,T,D", EQUAL)
@pytest.mark.parametrize("form", ["log", "gated"])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_equal_sequences(form, dtype, n, T, D):
    announce(f"linear scan {form} {dtype} n={n} T={T} D={D}")
    compare(make_scan(form, n, T, D, dtype, seed=n + T + D, state=(n + T) % 2 == 0), f"{form} {n}x{T}x{D}")


@pytest.mark.parametrize("lens,D,first,tail", [([5], 4, 0, 0), ([0, 0, 3], 9, 0, 0), ([64, 1, 0, 63, 65, 128], 66, 0, 0),
                                               ([1] * 70, 10, 0, 0), ([130, 0, 257, 2], 130, 30, 77), ([0], 5, 3, 3),
                                               ([700, 5, 600], 3, 1, 0)], ids=str)
@pytest.mark.parametrize("form", ["log", "gated"])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_packed_sequences(form, dtype, lens, D, first, tail):
    announce(f"linear scan packed {form} {dtype} {lens} D={D}")
    compare(make_scan(form, 1, 0, D, dtype, lens=lens, seed=len(lens) + D, reset=True, first=first, tail=tail), f"{form} {lens}")


@pytest.mark.parametrize("form", ["log", "gated"])
def test_long_sequences(form):
    """Many groups of tiles behind one another, equal and packed."""
    announce(f"linear scan long {form}")
    compare(make_scan(form, 1, 9001, 6, F32, seed=2), f"{form} 9001")
    compare(make_scan(form, 1, 0, 4, BF, lens=[4200, 1, 8300], seed=4, first=7, tail=60), f"{form} 4200,1,8300")


@pytest.mark.parametrize("form", ["log", "gated"])
def test_states_kept_over_thousands_of_tokens(form):
    """Norms of the errors of the final states and of dh0, float32, a within 0.0005 to 0.002 of one.  A state adds up the
    last tau = 1 / (1 - a) <= 2000 tokens; each has met tau roundings of half a step, 2^-25, in a, in the products of a
    and in the sums: three walks of sqrt(tau) 2^-25 = 1.3e-6, 4e-6 if all go one way.  The plain bound of a state, which
    takes every a to be off by its worst to one side, is hundreds of times that."""
    T, D, b = 12000, 64, 2
    d = make_scan(form, b, T, D, F32, seed=11)
    rate = torch.exp(torch.linspace(math.log(0.0005), math.log(0.002), D))
    if form == "log":
        d["gate"] = -rate * torch.rand(b, T, D, generator=torch.Generator().manual_seed(1)).add(0.5)
    else:  # sigmoid(gate) is 1/2 in the middle
        d["decay"] = torch.log(torch.expm1((2 * rate / C).double())).float()
    t = dev(d)
    a, u = coefficients(d)
    h, l = d["h0"].double(), d["dh_final"].double()
    for i in range(T):
        h = a[:, i] * h + u[:, i]
        l = a[:, T - 1 - i] * (l + d["dh"][:, T - 1 - i].double())
    out, got = fwd(t), bwd(t)
    for where, have, want in (("h_final", out["h_final"], h), ("dh0", got["dh0"], l)):
        err = float((have.double().cpu() - want).norm() / want.norm())
        print(form, where, f"{err:.1e}", flush=True)
        assert err <= 3 * math.sqrt(2000) * 2.0**-25, (where, err)


def test_states_that_span_every_channel_tile():
    announce("linear scan wide")
    compare(make_scan("gated", 1, 140, 5000, BF, seed=6), "wide")


@pytest.mark.parametrize("form", ["log", "gated"])
def test_no_state_no_final(form):
    """Outputs that are not asked for; T = 0 and no sequences at all."""
    announce(f"linear scan optional {form}")
    d = make_scan(form, 2, 70, 12, F32, seed=1, state=False)
    t, ref = dev(d), scan_reference(d)
    out = fwd(t, want_final=False)
    assert out["h_final"] is None and out["ckpt"] is None
    check(out["h"], *ref["h"], "h")
    got = bwd(t, want_dh0=False)
    assert got["dh0"] is None
    check(got["dx"], *ref["dx"], "dx")
    for n, T in ((2, 0), (0, 5)):
        d = make_scan(form, n, T, 12, F32, seed=1)
        t = dev(d)
        out = fwd(t, want_ckpt=True)
        assert torch.equal(out["h_final"], t["h0"]) and out["h"].shape == (n, T, 12)
        got = bwd(t)
        assert torch.equal(got["dh0"], t["dh_final"])
        if form == "gated":
            assert (got["ddecay"] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_rows_that_no_sequence_owns_are_left(dtype):
    announce("linear scan unowned rows")
    d = make_scan("gated", 1, 0, 40, dtype, lens=[90, 0, 70], first=33, tail=100, seed=8)
    own = owned(d)[0]
    for k in ("x", "gate", "input_gate", "dh"):
        d[k][0, ~own] = math.nan
    t = dev(d)
    out = {"h": torch.full_like(t["x"], 7.0), "h_final": torch.empty(3, 40, device=DEV), "ckpt": None}
    fwd(t, out=out)
    assert (out["h"][0, ~own] == 7.0).all() and torch.isfinite(out["h"]).all()
    g = {k: torch.full_like(t["x"], 7.0) for k in ("dx", "dgate", "dinput_gate")}
    g.update(ddecay=torch.empty(40, device=DEV), dh0=torch.empty(3, 40, device=DEV))
    bwd(t, out=g)
    for k in ("dx", "dgate", "dinput_gate"):
        assert (g[k][0, ~own] == 7.0).all() and torch.isfinite(g[k]).all()
    assert torch.isfinite(g["ddecay"]).all()


def test_borders_outside_the_tokens_are_clamped():
    announce("linear scan clamped borders")
    d = make_scan("log", 1, 0, 16, F32, lens=[60, 140], seed=9)
    t = dev(d)
    want = fwd(t)
    t["seq_offsets"] = torch.tensor([-5, 60, 100000], dtype=torch.int32, device=DEV)
    got = fwd(t)
    assert torch.equal(got["h"], want["h"]) and torch.equal(got["h_final"], want["h_final"])


def test_borders_that_go_back_count_as_the_largest_before():
    """Tiles wait for each other: no borders may leave one waiting."""
    announce("linear scan borders out of order")
    d = make_scan("gated", 1, 0, 16, F32, lens=[300, 0, 500, 100], seed=9)
    t = dev(d)
    want, wg = fwd(t, want_ckpt=True), bwd(t)
    t["seq_offsets"] = torch.tensor([0, 300, 7, 800, 900], dtype=torch.int32, device=DEV)
    got, gg = fwd(t, want_ckpt=True), bwd(t)
    torch.cuda.synchronize()
    assert torch.equal(got["h"], want["h"]) and torch.equal(got["ckpt"], want["ckpt"])
    for k in ("dx", "dgate", "dinput_gate", "ddecay"):
        assert torch.equal(gg[k], wg[k])


def test_more_sequences_than_a_wave():
    """The slot of a tile among hundreds of sequences, most of them empty."""
    announce("linear scan many sequences")
    lens = [0] * 70 + [130] + [0] * 63 + [1, 64, 65] + [0] * 128 + [200, 0]
    compare(make_scan("log", 1, 0, 3, F32, lens=lens, seed=19, first=5, tail=70), "many")
    compare(make_scan("gated", 1, 0, 2, F32, lens=[0] * 200, seed=20, tail=130), "all empty")


@pytest.mark.parametrize("form", ["log", "gated"])
def test_whole_tiles_that_no_sequence_owns(form):
    """Tiles of tokens before the first sequence and behind the last."""
    announce(f"linear scan unowned tiles {form}")
    d = make_scan(form, 1, 0, 10, BF, lens=[40, 150], seed=21, first=700, tail=600)
    own = owned(d)[0]
    for k in ("x", "gate", "input_gate", "dh"):
        if d[k] is not None:
            d[k][0, ~own] = math.nan
    t = dev(d)
    out = {"h": torch.full_like(t["x"], 7.0), "h_final": torch.empty(2, 10, device=DEV), "ckpt": None}
    fwd(t, out=out)
    g = {"dx": torch.full_like(t["x"], 7.0), "dgate": torch.full_like(t["gate"], 7.0), "dh0": torch.empty(2, 10, device=DEV)}
    if form == "gated":
        g.update(dinput_gate=torch.full_like(t["x"], 7.0), ddecay=torch.empty(10, device=DEV))
    bwd(t, out=g)
    for k, v in {"h": out["h"], **{k: g[k] for k in ("dx", "dgate", "dinput_gate") if k in g}}.items():
        assert (v[0, ~own] == 7.0).all() and torch.isfinite(v).all(), k
    assert all(torch.isfinite(v).all() for v in (out["h_final"], g["dh0"], g.get("ddecay", out["h_final"])))
    for k in ("x", "gate", "input_gate", "dh"):
        if d[k] is not None:
            d[k][0, ~own] = 0
    compare(d, "unowned tiles")


@pytest.mark.parametrize("form", ["log", "gated"])
def test_values_that_are_not_numbers_stay_causal(form):
    announce(f"linear scan nan {form}")
    d = make_scan(form, 2, 400, 20, F32, seed=10)
    t = dev(d)
    clean = fwd(t)["h"]
    for at in (0, 63, 130, 399):
        for bad in (math.nan, math.inf):
            x = t["x"].clone()
            x[1, at, 7] = bad
            got = fwd(dict(t, x=x))["h"]
            same = torch.ones_like(got, dtype=torch.bool)
            same[1, at:, 7] = False
            assert torch.equal(got[same], clean[same])
            assert not torch.isfinite(got[1, at, 7])


def test_extreme_gates():
    """Gates that saturate: nothing is forgotten, everything is; decays at both ends of float32."""
    announce("linear scan extreme gates")
    n, T, D = 1, 130, 8
    gen = torch.Generator().manual_seed(11)
    x = torch.randn(n, T, D, generator=gen)
    gate = torch.zeros(n, T, D)
    gate[..., 0], gate[..., 1], gate[..., 2] = 200.0, -200.0, -90.0
    decay = torch.full((D,), -4.0)
    decay[3], decay[4], decay[5], decay[6] = -100.0, 30.0, -20.0, 80.0
    ig = torch.randn(n, T, D, generator=gen)
    ig[..., 7] = -200.0
    t = dict(x=x.to(DEV), gate=gate.to(DEV), input_gate=ig.to(DEV), decay=decay.to(DEV), h0=torch.ones(n, D, device=DEV),
             seq_offsets=None, dh=torch.ones(n, T, D, device=DEV), dh_final=torch.ones(n, D, device=DEV))
    out, g = fwd(t), bwd(t)
    for k, v in {**out, **g}.items():
        if v is not None:
            assert torch.isfinite(v).all(), k
    # a = 1 and m = 0 as sigmoid(-200) is below float32's smallest: the state stays as it was and x never enters
    assert (out["h"][0, :, 1] == 1).all() and (g["dx"][0, :, 1] == 0).all() and (out["h"][0, :, 7] <= 1).all()


@pytest.mark.parametrize("form", ["log", "gated"])
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("b,D", [(1, 1), (1, 258), (5, 33), (70, 256), (3, 1001)])
def test_step(form, dtype, b, D):
    """One token of every request is the recurrence's next one; the states that no request names stay."""
    announce(f"linear scan step {form} {dtype} b={b} D={D}")
    d = make_scan(form, b, 1, D, dtype, seed=b + D)
    gen = torch.Generator().manual_seed(1)
    pool = torch.randn(b + 3, D, generator=gen)
    slots = torch.randperm(b + 3, generator=gen)[:b].to(torch.int32)
    d["h0"] = pool[slots.long()]
    ref = scan_reference(d)
    t = dev(d)
    sq = lambda v: None if v is None else v[:, 0].contiguous() if v.dim() == 3 else v  # noqa: E731
    args = dict(input_gate=sq(t["input_gate"]), decay=t["decay"], c=C)
    state = pool.to(DEV)
    h = bd.linear_scan_step(sq(t["x"]), sq(t["gate"]), state, slots=slots.to(DEV), **args)
    check(h[:, None], *ref["h"], "h")
    check(state[slots.long().to(DEV)], *ref["h_final"], "state")
    rest = torch.ones(b + 3, dtype=torch.bool)
    rest[slots.long()] = False
    assert torch.equal(state.cpu()[rest], pool[rest])
    # without slots: request i has state i
    state2 = d["h0"].to(DEV)
    h2 = bd.linear_scan_step(sq(t["x"]), sq(t["gate"]), state2, **args)
    assert torch.equal(h2, h) and torch.equal(state2, state[slots.long().to(DEV)])


def test_step_bad_and_repeated_slots():
    announce("linear scan step slots")
    gen = torch.Generator().manual_seed(2)
    b, D = 200, 70
    x, gate = torch.randn(b, D, generator=gen).to(DEV), -torch.rand(b, D, generator=gen).to(DEV)
    pool = torch.randn(8, D, generator=gen).to(DEV)
    slots = torch.full((b,), -1, dtype=torch.int32)
    slots[3], slots[4], slots[5], slots[150], slots[151], slots[199] = 2, 8, 2, 7, -2**31, 7
    state = pool.clone()
    h = bd.linear_scan_step(x, gate, state, slots=slots.to(DEV))
    live = [3, 150]
    a = torch.exp(gate.double())
    for i, s in ((3, 2), (150, 7)):
        want = a[i] * pool[s].double() + x[i].double()
        assert ((h[i].double() - want).abs() <= 16 * U * (a[i] * pool[s].double()).abs() + 2 * U * want.abs()).all()
        assert torch.equal(state[s], h[i])
    dead = [i for i in range(b) if i not in live]
    assert (h[dead] == 0).all()
    rest = [s for s in range(8) if s not in (2, 7)]
    assert torch.equal(state[rest], pool[rest])


def test_sequence_by_steps():
    """A prompt by linear_scan_fwd, then tokens one by one: the whole sequence in one call."""
    announce("linear scan prompt and steps")
    d = make_scan("gated", 3, 90, 34, BF, seed=12)
    t, ref = dev(d), scan_reference(d)
    cut = {k: (v[:, :80].contiguous() if isinstance(v, torch.Tensor) and v.dim() == 3 else v) for k, v in t.items()}
    out = fwd(cut)
    state = out["h_final"].clone()
    hs = [out["h"]]
    for i in range(80, 90):
        hs.append(bd.linear_scan_step(t["x"][:, i].contiguous(), t["gate"][:, i].contiguous(), state,
                                      input_gate=t["input_gate"][:, i].contiguous(), decay=t["decay"], c=C)[:, None])
    check(torch.cat(hs, 1), *ref["h"], "h")
    check(state, *ref["h_final"], "state")


def test_unaligned_and_repeated():
    """Tensors at odd element offsets, two calls bit for bit alike, other streams, a given workspace."""
    announce("linear scan alignment, determinism, streams")
    for dtype in (F32, BF):
        d = make_scan("gated", 2, 150, 36, dtype, seed=13)
        t = dev(d)
        want_f, want_b = fwd(t, want_ckpt=True), bwd(t)

        def shift(v):
            if not isinstance(v, torch.Tensor):
                return v
            flat = torch.empty(v.numel() + 1, dtype=v.dtype, device=DEV)
            flat[1:] = v.reshape(-1)
            return flat[1:].view(v.shape)

        s = {k: shift(v) for k, v in t.items()}
        for a, b in ((fwd(s, want_ckpt=True), want_f), (bwd(s), want_b)):
            for k in b:
                assert torch.equal(a[k], b[k]), (dtype, k)
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device=DEV)
        other.wait_stream(torch.cuda.current_stream())
        got_f, got_b = fwd(t, want_ckpt=True, stream=other, workspace=ws), bwd(t, stream=other, workspace=ws)
        other.synchronize()
        for a, b in ((got_f, want_f), (got_b, want_b)):
            for k in b:
                assert torch.equal(a[k], b[k]), (dtype, k)


def test_captured_calls_share_a_workspace():
    """Two graphs on one workspace, replayed in turn with other inputs and eager calls between."""
    announce("linear scan graphs")
    a, b = dev(make_scan("gated", 2, 700, 130, BF, seed=14)), dev(make_scan("log", 1, 1500, 64, F32, seed=15))
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device=DEV)
    graphs = []
    for t in (a, b):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            fwd(t, want_ckpt=True, workspace=ws)
            bwd(t, workspace=ws)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            f = fwd(t, want_ckpt=True, workspace=ws)
            r = bwd(t, ckpt=f["ckpt"], workspace=ws)
            r2 = bwd(t, workspace=ws)
        graphs.append((t, g, f, r, r2))
    for turn in range(4):
        for t, g, f, r, r2 in graphs:
            t["x"].copy_(torch.randn(t["x"].shape, device=DEV) * (turn + 1))
            g.replay()
            ws_fill = torch.full((1 << 20,), turn, device=DEV)  # the program's own work between the replays
            torch.cuda.synchronize()
            wf, wb = fwd(t, want_ckpt=True), bwd(t)
            for got, want in ((f, wf), (r, wb), (r2, wb)):
                for k in want:
                    if want[k] is not None:
                        assert torch.equal(got[k], want[k]), (turn, k)
            ws[:64].fill_(turn)
            assert int(ws_fill[0]) == turn


def test_two_calls_at_once():
    announce("linear scan concurrent")
    a, b = dev(make_scan("gated", 2, 2000, 130, BF, seed=16)), dev(make_scan("gated", 2, 2000, 130, BF, seed=17))
    want = [fwd(a), fwd(b)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [fwd(a, stream=s[0]), fwd(b, stream=s[1])]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g["h"], w["h"]) and torch.equal(g["h_final"], w["h_final"])


def test_coefficients_of_the_reference_are_the_documented_ones():
    d = make_scan("gated", 1, 3, 2, F32, seed=1)
    a, u = coefficients(d)
    x, r, i, dec = (d[k].double() for k in ("x", "gate", "input_gate", "decay"))
    want = torch.exp(-C * torch.log1p(torch.exp(dec)) / (1 + torch.exp(-r)))
    assert torch.allclose(a, want, rtol=1e-12)
    assert torch.allclose(u, torch.sqrt(1 - want**2) / (1 + torch.exp(-i)) * x, rtol=1e-9)
    assert HALF[BF] == torch.finfo(BF).eps / 2
