"""GPU parity of the gated delta rule with one gate per head (delta_chunk_fwd,
delta_chunk_bwd, delta_step) against the float64 oracle, through the binding."""
import numpy as np
import pytest
import torch

from delta_ref import BF, F32, TOL_BF16, TOL_F32, TOL_SPLIT, check, inputs, reference, spans
from gpu_common import announce
from selective_state_space_vjp_amd import binding as bd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FWD = dict(o=TOL_BF16, S_final=TOL_SPLIT)
FWD32 = dict(o=TOL_F32, S_final=TOL_F32)
BWD = dict(dq=TOL_BF16, dk=TOL_BF16, dv=TOL_BF16, dbeta=TOL_SPLIT, dg=TOL_SPLIT, dS0=TOL_SPLIT)


def dev(d):
    return {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def fwd(t, **kw):
    return bd.delta_chunk_fwd(t["q"], t["k"], t["v"], t["beta"], t["g"], t["S0"], scale=t["scale"],
                              seq_offsets=t["offsets"], **kw)


def bwd(t, **kw):
    return bd.delta_chunk_bwd(t["q"], t["k"], t["v"], t["beta"], t["g"], t["S0"], t["d_o"], t["dS"], scale=t["scale"],
                              seq_offsets=t["offsets"], **kw)


SHAPES = [
    # b, T, H, HV, K, V, state, lengths of packed sequences
    (1, 1, 1, 1, 16, 16, True, None),
    (2, 2, 1, 2, 32, 48, False, None),
    (1, 15, 2, 2, 128, 128, True, None),
    (2, 16, 1, 3, 48, 16, True, None),
    (1, 17, 2, 4, 64, 80, False, None),
    (1, 63, 1, 1, 128, 32, True, None),
    (3, 64, 2, 2, 80, 64, True, None),
    (1, 65, 3, 3, 112, 144, True, None),
    (2, 130, 1, 4, 128, 96, False, None),
    (1, 257, 2, 4, 96, 176, True, None),
    (9, 400, 2, 4, 128, 64, True, [1, 0, 63, 64, 65, 0, 129, 2, 76]),
    (3, 150, 1, 1, 64, 16, False, [0, 0, 150]),
    (70, 200, 1, 2, 32, 32, True, [3, 1, 0, 4, 6, 2, 4] * 10),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_backward_parity(shape):
    announce(f"delta_chunk {shape}")
    b, T, H, HV, K, V, state, packed = shape
    d = inputs(b, T, H, HV, K, V, BF, state, packed, seed=T + V)
    ref = reference(d)
    t = dev(d)
    check(fwd(t), ref, FWD, "fwd")
    check(bwd(t), ref, BWD, "bwd")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_float32(shape):
    announce(f"delta_chunk f32 {shape}")
    b, T, H, HV, K, V, state, packed = shape
    d = inputs(b, T, H, HV, K, V, F32, state, packed, seed=T + V)
    check(fwd(dev(d)), reference(d, grads=False), FWD32, "fwd f32")


@pytest.mark.parametrize("case", ["no_decay", "no_write", "full_write", "strong", "resets", "same_key", "zero_keys"])
def test_degenerate_gates_and_keys(case):
    """g = 0, beta = 0 and 1, gates that underflow, hard resets, one key for all tokens, no keys."""
    announce(f"delta_chunk {case}")
    d = inputs(2, 140, 1, 2, 64, 48, BF, True, None, seed=5)
    if case == "no_decay":
        d["g"].zero_()
    elif case == "no_write":
        d["beta"].zero_()
    elif case == "full_write":
        d["beta"].fill_(1.0)
    elif case == "strong":
        d["g"].fill_(-87.0)
    elif case == "resets":
        d["g"][:, 3::50] = float("-inf")
    elif case == "same_key":
        d["k"][:] = d["k"][:, :1]
        d["beta"].fill_(1.0)
        d["g"].zero_()
    else:
        d["k"].zero_()
    t = dev(d)
    if case == "resets":
        # the oracle's exp(-inf) = 0 is the definition; the kernels' e^-88 is 6e-39 of the state
        ref = reference(d, grads=False)
        check(fwd(t), ref, FWD, case)
        got = bwd(t)
        assert all(torch.isfinite(got[n]).all() for n in BWD)
        d["g"] = d["g"].clamp(min=-88.0)
        check(got, reference(d), dict(BWD, dg=2 * TOL_SPLIT), case)  # gates of e^-88: sums of 88 round to 2^-18
        return
    ref = reference(d)
    tol, btol, floors = dict(FWD), dict(BWD), {}
    if case == "strong":
        # e^-87 = 1.6e-38 is as small as float32's normal numbers get.  dS0 = e^-87 (q scale dO - k mu) of the
        # first token: each of the two operands e^-87 scale dO and e^-87 mu is a bf16 number below 2^-126, where
        # steps are 2^-133, and |q_k|, |k_k| <= 1.  dg: at most 64 terms of three float32 products there, steps
        # 2^-149.
        floors = {"dS0": 2 * 2.0**-134, "dg": 64 * 3 * 2.0**-150}
    if case == "same_key":
        # r_t = v_t - v_{t-1} for every token: T R cancels sums of 64 terms of the size of r,
        # sqrt(64) times the relative error of a generic chunk
        tol["S_final"] *= 8
        for n in ("dbeta", "dg", "dS0"):
            btol[n] *= 8
    check(fwd(t), ref, tol, case)
    check(bwd(t), ref, btol, case, floors)


def test_empty_inputs():
    announce("delta_chunk empty")
    d = inputs(2, 0, 1, 2, 32, 32, BF, True, None)
    t = dev(d)
    assert torch.equal(fwd(t)["S_final"], t["S0"])
    assert torch.equal(bwd(t)["dS0"], t["dS"])
    for dt in (BF, F32):
        d = inputs(0, 7, 1, 2, 32, 32, dt, False, None)
        assert fwd(dev(d))["o"].shape == (0, 7, 2, 32)
    d = inputs(0, 40, 1, 2, 32, 32, BF, False, [])
    t = dev(d)
    out = dict(o=torch.full_like(t["v"], 7.0), S_final=None)
    fwd(t, out=out)
    assert (out["o"] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_without_a_sequence_are_left_alone(dtype):
    """Tokens before the first and behind the last border: NaN there is neither read nor overwritten."""
    announce("delta_chunk unowned rows")
    d = inputs(3, 200, 1, 2, 64, 48, dtype, True, [50, 0, 90])
    d["offsets"] += 30
    own = torch.zeros(200, dtype=torch.bool)
    own[30:170] = True
    for n in ("q", "k", "v", "beta", "g", "d_o"):
        d[n][:, ~own] = float("nan")
    t = dev(d)
    ref = reference({**d, **{n: torch.nan_to_num(d[n]) for n in ("q", "k", "v", "beta", "g", "d_o")}})
    out = dict(o=torch.full_like(t["v"], 7.0), S_final=torch.empty_like(t["S0"]))
    fwd(t, out=out)
    assert (out["o"][:, ~own] == 7.0).all()
    out["o"][:, ~own] = 0
    check(out, ref, FWD if dtype == BF else FWD32, "fwd")
    if dtype == F32:
        return
    like = dict(dq="q", dk="k", dv="v", dbeta="beta", dg="g")
    out = {n: torch.full_like(t[x], 7.0) for n, x in like.items()}
    out["dS0"] = torch.empty_like(t["S0"])
    bwd(t, out=out)
    for n in like:
        assert (out[n][:, ~own] == 7.0).all(), n
        out[n][:, ~own] = 0
    check(out, ref, BWD, "bwd")


def test_bad_borders_stay_inside_the_tensors():
    """Borders past the ends are clamped and a descending pair is an empty sequence: the documented
    meaning, on borders that the kernels' own checks bring into range."""
    announce("delta_chunk clamped borders")
    d = inputs(3, 100, 1, 1, 32, 32, BF, True, [40, 30, 30])
    ref = reference(d, grads=False)
    t = dev(d)
    t["offsets"] = torch.tensor([-5, 40, 70, 1 << 20], dtype=torch.int32, device=DEV)
    check(fwd(t), ref, FWD, "clamped")
    for dt in (BF, F32):
        t = dev(inputs(3, 100, 1, 1, 32, 32, dt, True, [40, 30, 30]))
        t["offsets"] = torch.tensor([0, 100, 40, 40], dtype=torch.int32, device=DEV)
        got = fwd(t)
        assert torch.equal(got["S_final"][1:], t["S0"][1:])


def test_two_chained_calls_equal_one():
    announce("delta_chunk chaining")
    d = inputs(2, 200, 1, 2, 64, 64, BF, True, None, seed=8)
    t = dev(d)
    cut = 77
    a = {k: (v[:, :cut].contiguous() if k in ("q", "k", "v", "beta", "g", "d_o") else v) for k, v in t.items()}
    z = {k: (v[:, cut:].contiguous() if k in ("q", "k", "v", "beta", "g", "d_o") else v) for k, v in t.items()}
    fa = fwd(a)
    z["S0"] = fa["S_final"]
    fz = fwd(z)
    ref = reference(d)
    check(dict(o=torch.cat([fa["o"], fz["o"]], 1), S_final=fz["S_final"]), ref, FWD, "fwd")
    gz = bwd(z)
    a["dS"] = gz["dS0"]
    ga = bwd(a)
    both = {n: torch.cat([ga[n], gz[n]], 1) for n in ("dq", "dk", "dv", "dbeta", "dg")}
    check(dict(both, dS0=ga["dS0"]), ref, BWD, "bwd")


def test_null_states_and_unwanted_outputs():
    announce("delta_chunk NULL states")
    d = inputs(1, 100, 1, 2, 64, 64, BF, True, None, seed=9)
    for drop in (("S0",), ("dS",), ("S0", "dS")):
        c = dict(d, **{n: None for n in drop})
        ref = reference(c)
        t = dev(c)
        check(fwd(t), ref, FWD, str(drop))
        check(bwd(t), ref, BWD, str(drop))
    t = dev(d)
    assert fwd(t, want_final=False)["S_final"] is None
    got = bwd(t, want_dS0=False)
    assert got["dS0"] is None
    full = bwd(t)
    for n in ("dq", "dk", "dv", "dbeta", "dg"):
        assert torch.equal(got[n], full[n]), n


def test_deterministic_and_independent_of_the_workspace():
    announce("delta_chunk determinism")
    t = dev(inputs(5, 300, 2, 6, 128, 80, BF, True, [100, 3, 0, 64, 133], seed=3))
    f, g = fwd(t), bwd(t)
    desc = bd.delta_chunk_desc(t["q"], t["v"], t["scale"], t["offsets"])
    for fn, name, first in ((fwd, "delta_chunk_fwd_workspace", f), (bwd, "delta_chunk_bwd_workspace", g)):
        ws = torch.full((bd._query(name, desc),), 255, dtype=torch.uint8, device=DEV)  # NaN patterns
        for _ in range(2):
            again = fn(t, workspace=ws)
            for n in first:
                assert torch.equal(first[n], again[n]), n


def test_stacked_heads_and_sequences_do_not_mix():
    """A NaN in one sequence's tokens stays in that sequence, a NaN in one value head in that head (and, in
    dq and dk, in its qk head)."""
    announce("delta_chunk isolation")
    d = inputs(3, 200, 2, 4, 64, 64, BF, True, [70, 60, 70], seed=4)
    clean_f, clean_b = fwd(dev(d)), bwd(dev(d))
    d["v"][0, 100, 1, 5] = float("nan")  # sequence 1, value head 1 (qk head 0)
    f, g = fwd(dev(d)), bwd(dev(d))
    other = [h for h in range(4) if h != 1]
    assert torch.equal(f["o"][:, :70], clean_f["o"][:, :70]) and torch.equal(f["o"][:, 130:], clean_f["o"][:, 130:])
    assert torch.equal(f["o"][:, :, other], clean_f["o"][:, :, other])
    assert torch.equal(f["S_final"][:, other], clean_f["S_final"][:, other])
    for n in ("dv", "dbeta", "dg"):
        assert torch.equal(g[n][:, :, other], clean_b[n][:, :, other]), n
    for n in ("dq", "dk"):
        assert torch.equal(g[n][:, :, 1], clean_b[n][:, :, 1]), n
        assert torch.equal(g[n][:, :70], clean_b[n][:, :70]) and torch.equal(g[n][:, 130:], clean_b[n][:, 130:]), n
    assert torch.isnan(f["o"][:, 100:130, 1]).any()


def test_gradients_against_differences():
    """<gradient, direction> against the central difference of J = <d_o, o> + <dS, S_final> in the float64
    reference, for every input: only the kernel's own errors enter, J being smooth (step 1e-4: the
    difference's own error is the third derivative times 1e-8 / 6)."""
    announce("delta_chunk differences")
    d = inputs(1, 90, 1, 2, 32, 32, BF, True, None, seed=12)
    g = bwd(dev(d))

    def J(x):
        r = reference(x, grads=False)
        return float((r["o"] * d["d_o"].double()).sum() + (r["S_final"] * d["dS"].double()).sum())

    gen = torch.Generator().manual_seed(1)
    base = {n: (v.double() if isinstance(v, torch.Tensor) and n != "offsets" else v) for n, v in d.items()}
    for n, tol in (("q", TOL_BF16), ("k", TOL_BF16), ("v", TOL_BF16), ("beta", TOL_SPLIT), ("g", TOL_SPLIT), ("S0", TOL_SPLIT)):
        dirn = torch.randn(d[n].shape, generator=gen, dtype=torch.float64)
        h = 1e-4
        want = (J({**base, n: base[n] + h * dirn}) - J({**base, n: base[n] - h * dirn})) / (2 * h)
        grad = g["d" + n].double().cpu()
        # the gradient's error is a vector of tol |grad| in no particular direction: its product with a
        # random direction is off by tol |grad| times a standard normal number; 5 of them, and 1e-6 of
        # |grad| |direction| for the difference itself
        bound = (5 * tol + 1e-6 * float(dirn.norm())) * float(grad.norm())
        assert abs(float((grad * dirn).sum()) - want) <= bound, (n, float((grad * dirn).sum()), want, bound)


# ------------------------------------------------------------------ one token
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("per_key", [False, True])
@pytest.mark.parametrize("shape", [(1, 1, 1, 16, 16), (3, 2, 4, 128, 128), (5, 1, 3, 80, 112), (70, 2, 2, 48, 32)], ids=str)
def test_step_parity(shape, per_key, dtype):
    announce(f"delta_step {shape} per_key={per_key} {dtype}")
    b, H, HV, K, V = shape
    import oracle

    gen = torch.Generator().manual_seed(b + K)
    rn = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    q, k = (torch.nn.functional.normalize(rn(b, H, K), dim=-1).to(dtype) for _ in range(2))
    v, beta = rn(b, HV, V).to(dtype), torch.sigmoid(rn(b, HV)).float()
    g = (-torch.nn.functional.softplus(rn(*((b, HV, K) if per_key else (b, HV))))).float()
    state = (0.5 * rn(b + 3, HV, K, V)).float()
    slots = torch.randperm(b + 3, generator=gen)[:b].to(torch.int32)
    gk = (g if per_key else g[..., None].expand(b, HV, K)).double().numpy()
    o, s = oracle.kda_fwd(*(x.double().numpy()[:, None] for x in (q, k, v, beta)), np.ascontiguousarray(gk[:, None]),
                          state[slots.long()].double().numpy(), scale=0.7)
    want = state.double().clone()
    want[slots.long()] = torch.from_numpy(s)
    pool = state.to(DEV)
    got = bd.delta_step(q.to(DEV), k.to(DEV), v.to(DEV), beta.to(DEV), g.to(DEV), pool, scale=0.7, slots=slots.to(DEV))
    check(dict(o=got, state=pool), dict(o=torch.from_numpy(o[:, 0]), state=want),
          dict(o=TOL_BF16 if dtype == BF else TOL_F32, state=TOL_F32), "step")
    idle = [i for i in range(b + 3) if i not in slots.tolist()]
    assert torch.equal(pool.cpu()[idle], state[idle])


def test_step_padding_repeated_slots_and_no_slots():
    announce("delta_step slots")
    gen = torch.Generator().manual_seed(2)
    b, H, HV, K, V, n = 70, 1, 2, 32, 48, 40
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    q, k = (torch.nn.functional.normalize(rn(b, H, K), dim=-1).to(BF).to(DEV) for _ in range(2))
    v, beta, g = rn(b, HV, V).to(BF).to(DEV), torch.sigmoid(rn(b, HV)).to(DEV), -rn(b, HV).abs().to(DEV)
    state = rn(n, HV, K, V).to(DEV)
    slots = torch.full((b,), -1, dtype=torch.int32)
    slots[1], slots[3], slots[4] = 7, n, 1 << 30     # 3 and 4 outside
    slots[2], slots[69], slots[68] = 7, 7, 9         # 2 and 69 repeat 1's
    live = [1, 68]
    pool = state.clone()
    got = bd.delta_step(q, k, v, beta, g, pool, scale=1.0, slots=slots.to(DEV))
    one = state.clone()
    want = bd.delta_step(*(x[live].contiguous() for x in (q, k, v, beta, g)), one, scale=1.0,
                         slots=slots[live].to(DEV))
    assert torch.equal(pool, one) and torch.equal(got[live], want)
    dead = [i for i in range(b) if i not in live]
    assert (got[dead] == 0).all()
    # no slots: request i uses state i
    pool = state.clone()
    a = bd.delta_step(*(x[:n].contiguous() for x in (q, k, v, beta, g)), pool, scale=1.0)
    one = state.clone()
    z = bd.delta_step(*(x[:n].contiguous() for x in (q, k, v, beta, g)), one, scale=1.0,
                      slots=torch.arange(n, dtype=torch.int32, device=DEV))
    assert torch.equal(a, z) and torch.equal(pool, one)
    with pytest.raises(bd.SsmVjpError) as e:
        bd.delta_step(q, k, v, beta, g, pool, scale=1.0)  # 70 requests, 40 states
    assert e.value.status == bd.EINVAL


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_then_tokens(dtype):
    """A prompt through delta_chunk_fwd and its continuation through delta_step against the whole sequence
    through the reference."""
    announce("delta prompt then tokens")
    d = inputs(3, 90, 2, 4, 64, 80, dtype, True, None, seed=6)
    t = dev(d)
    cut = 70
    head = {k: (v[:, :cut].contiguous() if k in ("q", "k", "v", "beta", "g") else v) for k, v in t.items()}
    f = fwd(head)
    pool, o = f["S_final"], [f["o"]]
    for i in range(cut, 90):
        o.append(bd.delta_step(*(t[n][:, i].contiguous() for n in ("q", "k", "v", "beta", "g")), pool, scale=t["scale"])[:, None])
    check(dict(o=torch.cat(o, 1), S_final=pool), reference(d, grads=False), FWD if dtype == BF else FWD32, "prompt + tokens")


# ------------------------------------------------------------- streams, graphs
def test_other_streams_and_two_calls_at_once():
    announce("delta streams")
    ts = [dev(inputs(2, 150, 1, 2, 64, 64, BF, True, None, seed=s)) for s in (1, 2)]
    want = [(fwd(t), bwd(t)) for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    got = []
    for _ in range(3):
        for s, t in zip(streams, ts):
            got.append((fwd(t, stream=s), bwd(t, stream=s)))
    torch.cuda.synchronize()
    for i, (f, b) in enumerate(got):
        for n, x in {**want[i % 2][0], **want[i % 2][1]}.items():
            assert torch.equal(x, {**f, **b}[n]), n


def test_captured_and_replayed():
    """Forward, backward and a token in one graph, replayed with eager calls between."""
    announce("delta graph")
    d = inputs(4, 150, 1, 2, 64, 64, BF, True, [60, 0, 65, 25], seed=7)
    t = dev(d)
    tok = {n: t[n][0, :4].contiguous() for n in ("q", "k", "v", "beta", "g")}
    pool = t["S0"].clone()

    def run():
        return fwd(t), bwd(t), bd.delta_step(*tok.values(), pool, scale=t["scale"])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f, b, o = run()
    gen = torch.Generator().manual_seed(3)
    for i in range(4):
        t["v"].copy_(torch.randn(t["v"].shape, generator=gen))
        pool.copy_(torch.randn(pool.shape, generator=gen))
        if i == 2:  # other borders, same graph
            t["offsets"].copy_(torch.tensor([0, 10, 75, 75, 150], dtype=torch.int32))
        start = pool.clone()
        graph.replay()
        torch.cuda.synchronize()
        after = pool.clone()
        pool.copy_(start)
        f2, b2, o2 = run()
        torch.cuda.synchronize()
        for n in f:
            assert torch.equal(f[n], f2[n]), (i, n)
        for n in b:
            assert torch.equal(b[n], b2[n]), (i, n)
        assert torch.equal(o, o2) and torch.equal(after, pool)


def test_long_sequence_slice():
    """The kda workload's sizes (b=2, T=4096, H=16, HV=32, K=V=128), one qk head of each sequence."""
    announce("delta full size")
    d = inputs(2, 4096, 16, 32, 128, 128, BF, False, None, seed=2, rate=0.02)
    t = dev(d)
    f, g = fwd(t), bwd(t)
    for bi, h in ((0, 3), (1, 15)):
        pick = lambda x, heads: x[bi:bi + 1, :, heads].contiguous()  # noqa: E731
        nv = [2 * h, 2 * h + 1]
        sub = {"q": pick(d["q"], [h]), "k": pick(d["k"], [h]), **{n: pick(d[n], nv) for n in ("v", "beta", "g", "d_o")},
               "S0": None, "dS": None, "scale": d["scale"], "offsets": None}
        got = {"o": pick(f["o"], nv), "S_final": f["S_final"][bi:bi + 1, nv], "dq": pick(g["dq"], [h]), "dk": pick(g["dk"], [h]),
               "dv": pick(g["dv"], nv), "dbeta": pick(g["dbeta"], nv), "dg": pick(g["dg"], nv), "dS0": g["dS0"][bi:bi + 1, nv]}
        check(got, reference(sub), {**FWD, **BWD}, f"sequence {bi} head {h}")
    assert spans(d)[1] == (1, 0, 4096)
