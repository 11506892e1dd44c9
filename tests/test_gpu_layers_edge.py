"""The chunked delta rule, its one-token form and layer norm where calls get unusual: the
debug finiteness mode, results written over inputs, values that are not numbers, borders
that do not fit, the largest heads, and pools past 2^31 elements."""
import pytest
import torch

from delta_ref import BF, F32, TOL_BF16, TOL_SPLIT, check, inputs, reference
from gpu_common import announce
from selective_state_space_vjp_amd import binding as bd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def dev(d):
    return {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def fwd(t, **kw):
    return bd.delta_chunk_fwd(t["q"], t["k"], t["v"], t["beta"], t["g"], t["S0"], scale=t["scale"],
                              seq_offsets=t["offsets"], **kw)


def bwd(t, **kw):
    return bd.delta_chunk_bwd(t["q"], t["k"], t["v"], t["beta"], t["g"], t["S0"], t["d_o"], t["dS"], scale=t["scale"],
                              seq_offsets=t["offsets"], **kw)


def step(t, pool):
    return bd.delta_step(*(t[n][:, 0].contiguous() for n in ("q", "k", "v", "beta", "g")), pool, scale=t["scale"])


def _nonfinite(fn):
    with pytest.raises(bd.SsmVjpError) as e:
        fn()
    assert e.value.status == bd.ENONFINITE


@pytest.mark.parametrize("dtype", [BF, F32])
def test_nonfinite_outputs_are_reported(dtype, monkeypatch):
    announce(f"delta and norm finite check {dtype}")
    monkeypatch.delenv("SSMVJP_CHECK_FINITE", raising=False)
    t = dev(inputs(2, 70, 1, 2, 32, 32, dtype, True, None, seed=4))
    x, w = torch.randn(30, 40, device=DEV).to(dtype), torch.ones(40, device=DEV)

    def calls(t, x):
        f = fwd(t)
        n = bd.layer_norm_fwd(x, w, w, want_ckpt8=True)
        out = {**f, **n, "step": step(t, t["S0"].clone())}
        if dtype == BF:
            out.update(bwd(t))
        out.update(bd.layer_norm_bwd(x, x, n["mean"], n["rstd"], w))
        return out

    plain = calls(t, x)
    torch.cuda.synchronize()
    monkeypatch.setenv("SSMVJP_CHECK_FINITE", "1")
    for n, v in calls(t, x).items():
        assert torch.equal(v, plain[n]), n
    bad = dict(t, v=t["v"].clone())
    bad["v"][1, 0, 1, 3] = float("nan")
    _nonfinite(lambda: fwd(bad))
    _nonfinite(lambda: step(bad, t["S0"].clone()))
    if dtype == BF:
        _nonfinite(lambda: bwd(dict(t, d_o=bad["v"])))
    y = x.clone()
    y[7, 3] = float("inf")
    _nonfinite(lambda: bd.layer_norm_fwd(y, w, w))
    n = bd.layer_norm_fwd(x, w, w)
    _nonfinite(lambda: bd.layer_norm_bwd(y, x, n["mean"], n["rstd"], w))
    monkeypatch.delenv("SSMVJP_CHECK_FINITE", raising=False)
    fwd(bad)
    torch.cuda.synchronize()


@pytest.mark.parametrize("packed", [None, [70, 0, 1, 69]])
def test_states_written_over_the_states_read(packed):
    announce("delta in place")
    for dtype in (BF, F32):
        t = dev(inputs(2, 140, 1, 2, 64, 48, dtype, True, packed, seed=3))
        want = fwd(t)
        S0 = t["S0"].clone()
        got = fwd(dict(t, S0=S0), out={"o": torch.empty_like(t["v"]), "S_final": S0})
        for n in want:
            assert torch.equal(got[n], want[n]), (dtype, n)
    t = dev(inputs(2, 140, 1, 2, 64, 48, BF, True, packed, seed=3))
    want = bwd(t)
    for name in ("dS", "S0"):
        u = dict(t)
        u[name] = t[name].clone()
        out = {n: torch.empty_like(v) for n, v in want.items()}
        out["dS0"] = u[name]
        got = bwd(u, out=out)
        for n in want:
            assert torch.equal(got[n], want[n]), (name, n)


def test_not_a_number_stays_in_its_head_and_sequence():
    announce("delta nan")
    for dtype in (BF, F32):
        d = inputs(1, 200, 2, 4, 64, 32, dtype, True, [66, 134], seed=8)
        t = dev(d)
        ok = fwd(t), (bwd(t) if dtype == BF else {})
        bad = dev(d)
        bad["v"][0, 70, 3, 5] = float("nan")   # second sequence, last value head (second qk head)
        bad["d_o"][0, 90, 3, 1] = float("inf")
        f, b = fwd(bad), (bwd(bad) if dtype == BF else {})
        assert torch.isnan(f["o"][0, 70, 3]).any()
        for n, x in f.items():
            r = ok[0][n]
            if n == "o":
                assert torch.equal(x[0, :66], r[0, :66]) and torch.equal(x[0, :, :3], r[0, :, :3])
            else:
                assert torch.equal(x[0], r[0]) and torch.equal(x[1, :3], r[1, :3])
        for n, x in b.items():
            r = ok[1][n]
            if n == "dS0":
                assert torch.equal(x[0], r[0]) and torch.equal(x[1, :3], r[1, :3])
            else:
                clean = 1 if n in ("dq", "dk") else 3
                assert torch.equal(x[0, :66], r[0, :66]) and torch.equal(x[0, :, :clean], r[0, :, :clean]), n


def test_nan_gates_are_not_taken_for_resets():
    announce("delta nan gate")
    t = dev(inputs(1, 40, 1, 1, 16, 16, BF, True, None, seed=8))
    t["g"][0, 20, 0] = float("nan")
    assert torch.isnan(fwd(t)["S_final"]).any()
    assert torch.isnan(bwd(t)["dS0"]).any()


def test_many_heads_narrow_and_wide():
    """Many value heads of one qk head, and one wide one."""
    announce("delta heads")
    for shape in ((1, 20, 1, 40, 16, 16), (1, 70, 1, 1, 16, 1040), (2, 5, 24, 24, 16, 16)):
        b, T, H, HV, K, V = shape
        d = inputs(b, T, H, HV, K, V, BF, True, None, seed=T)
        t, ref = dev(d), reference(d)
        check(fwd(t), ref, dict(o=TOL_BF16, S_final=TOL_SPLIT), str(shape))
        check(bwd(t), ref, dict(dq=TOL_BF16, dk=TOL_BF16, dv=TOL_BF16, dbeta=TOL_SPLIT, dg=TOL_SPLIT, dS0=TOL_SPLIT),
              str(shape))


def test_pool_past_32_bit_offsets():
    """A pool of 2^31 + elements (8.6 GB): the last state's request reads and writes the last state."""
    announce("delta_step large pool")
    n, HV, K, V = (1 << 31) // (8 * 128 * 128) + 3, 8, 128, 128
    d = inputs(2, 1, 8, HV, K, V, BF, True, None, seed=6)
    t = dev(d)
    tok = [t[x][:, 0].contiguous() for x in ("q", "k", "v", "beta", "g")]
    small = t["S0"].clone()
    want = bd.delta_step(*tok, small, scale=d["scale"])
    pool = torch.empty(n, HV, K, V, device=DEV)
    pool[0], pool[n - 1] = t["S0"][0], t["S0"][1]
    pool[1], pool[n - 2] = 5.0, 7.0
    slots = torch.tensor([0, n - 1], dtype=torch.int32, device=DEV)
    got = bd.delta_step(*tok, pool, scale=d["scale"], slots=slots)
    assert torch.equal(got, want)
    assert torch.equal(pool[0], small[0]) and torch.equal(pool[n - 1], small[1])
    assert bool((pool[1] == 5.0).all()) and bool((pool[n - 2] == 7.0).all())


def test_strided_tensors_are_refused_not_copied():
    t = dev(inputs(1, 20, 1, 2, 32, 32, BF, True, None, seed=4))
    wide = torch.zeros(1, 20, 2, 64, dtype=BF, device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        fwd(dict(t, v=wide[..., :32]))
    x = torch.zeros(8, 64, dtype=BF, device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        bd.layer_norm_fwd(x[:, :32])
    flat = torch.zeros(20 * 2 * 32 + 1, dtype=BF, device=DEV)[1:]  # contiguous, two bytes off
    with pytest.raises(bd.SsmVjpError) as e:
        fwd(dict(t, v=flat.view(1, 20, 2, 32)))
    assert e.value.status == bd.EINVAL


def test_more_long_rows_than_one_grid():
    """Rows past the registers' length, more than 2^20 of them: the last rows as in a small call."""
    announce("norm many long rows")
    n = (1 << 20) + 3
    gen = torch.Generator(DEV).manual_seed(2)
    x = torch.randn(n, 2049, generator=gen, device=DEV, dtype=BF)
    f = bd.layer_norm_fwd(x)
    few = torch.cat([x[:2], x[-4:]])
    want = bd.layer_norm_fwd(few)
    for name in want:
        assert torch.equal(torch.cat([f[name][:2], f[name][-4:]]), want[name]), name
    x = x.view(-1)[:n * 1025].view(n, 1025)
    st = bd.layer_norm_fwd(x)
    dy = f["y"].view(-1)[:n * 1025].view(n, 1025)
    b = bd.layer_norm_bwd(dy, x, st["mean"], st["rstd"])
    pick = torch.tensor([0, 1, n - 4, n - 3, n - 2, n - 1], device=DEV)
    want = bd.layer_norm_bwd(dy[pick], x[pick], st["mean"][pick], st["rstd"][pick])
    assert torch.equal(b["dx"][pick], want["dx"])


@pytest.mark.parametrize("shape", [
    (3, 130, 4, 8, 64, 64),     # both walks in one launch, K <= 64
    (3, 130, 4, 8, 128, 48),    # the same, K > 64
    (8, 70, 4, 32, 64, 32),     # a full round of 256 workgroups: two launches, K <= 64
    (8, 70, 4, 32, 80, 32),     # the same, K > 64
    (5, 3, 2, 6, 16, 32),       # few cells: float32 terms of dg, K <= 64
    (1, 65, 1, 3, 112, 48),     # the same, K > 64
], ids=str)
def test_every_form_of_the_backward(shape):
    announce(f"delta backward form {shape}")
    b, T, H, HV, K, V = shape
    d = inputs(b, T, H, HV, K, V, BF, True, None, seed=T + K)
    tol = dict(dq=TOL_BF16, dk=TOL_BF16, dv=TOL_BF16, dbeta=TOL_SPLIT, dg=TOL_SPLIT, dS0=TOL_SPLIT)
    t = dev(d)
    got = bwd(t)
    check(got, reference(d), tol, str(shape))
    for n, x in bwd(t).items():
        assert torch.equal(x, got[n]), n


def test_more_units_than_the_gradients_grid():
    """More (chunk, qk head) units than workgroups of the gradients kernel, some of them without tokens: the same
    bits as sequence by sequence."""
    announce("delta gradients units")
    lens = [130, 0, 1, 64, 65, 200, 0, 63] * 2
    d = inputs(1, sum(lens), 24, 24, 64, 32, BF, True, lens, seed=12)
    t = dev(d)
    got = bwd(t)
    at = 0
    for i, n in enumerate(lens):
        if n:
            one = {k: (t[k][:, at:at + n].contiguous() if k in ("q", "k", "v", "beta", "g", "d_o") else t[k]) for k in t}
            one.update(S0=t["S0"][i:i + 1], dS=t["dS"][i:i + 1], offsets=None)
            w = bwd(one)
            for k in ("dq", "dk", "dv"):
                assert torch.equal(got[k][:, at:at + n], w[k]), (i, k)
            assert torch.equal(got["dS0"][i], w["dS0"][0]), i
        at += n
