"""GPU parity of layer_norm_fwd and layer_norm_bwd, with the input itself and with
its 8-bit form, against the formulas in float64; and the norms and the gated delta
rule run together as a layer runs them."""
import math

import numpy as np
import pytest
import torch

from delta_ref import BF, F32, TOL_BF16, TOL_SPLIT
from gpu_common import announce
from selective_state_space_vjp_amd import binding as bd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5
U32 = 2.0**-24
# sums of n float32 terms in a tree of partial sums of at most 64 serial additions each:
# every level adds 64 roundings, 3 levels at most for the sizes here, in the worst case
SUM32 = 3 * 64 * U32


def reference(x, w, b, dy=None, stats=None, eps=EPS):
    """Everything in float64; stats: mean and rstd as given instead of x's own."""
    x = x.double()
    mean = x.mean(-1, keepdim=True) if stats is None else stats[0].double()[..., None]
    rstd = (1 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)) if stats is None else stats[1].double()[..., None]
    h = (x - mean) * rstd
    w = torch.ones((), dtype=torch.float64) if w is None else w.double()
    out = {"y": h * w + (0 if b is None else b.double()), "mean": mean[..., 0], "rstd": rstd[..., 0]}
    if dy is not None:
        dy = dy.double()
        t = dy * w
        out["dx"] = rstd * (t - t.mean(-1, keepdim=True) - h * (t * h).mean(-1, keepdim=True))
        lead = tuple(range(x.dim() - (w.dim() or 1)))
        out["dweight"], out["dbias"] = (dy * h).sum(lead), dy.sum(lead)
    return out


def codes(x):
    """The 8-bit form as the header defines it, in numpy float32."""
    x = x.float().numpy()
    D = x.shape[-1]
    q, s = np.zeros(x.shape, np.int8), np.zeros(x.shape[:-1] + (-(-D // 64),), np.float32)
    for j in range(s.shape[-1]):
        blk = x[..., 64 * j:64 * j + 64]
        top = np.abs(blk).max(-1)
        some = top >= np.float32(1e-36)
        inv = np.float32(127) * (np.float32(1) / np.where(some, top, np.float32(1)))
        q[..., 64 * j:64 * j + 64] = np.rint(blk * np.where(some, inv, np.float32(0))[..., None])
        s[..., j] = np.where(some, top * np.float32(1 / 127), np.float32(0))
    return torch.from_numpy(q), torch.from_numpy(s)


def kept(q, s, D):
    return (q.float() * s.repeat_interleave(64, -1)[..., :D]).double()


def near(got, want, tol, where):
    """|error| <= tol * (largest value of the row / column it belongs to, at least the mean square)."""
    got, want = got.double().cpu(), want.double()
    assert got.shape == want.shape, (where, got.shape, want.shape)
    if not want.numel():
        return
    assert torch.isfinite(got).all(), where
    rms = float(want.norm()) / math.sqrt(want.numel())
    err = float(((got - want).abs() / want.abs().clamp(min=max(rms, 1e-30))).max())
    print(where, f"{err:.1e} of {tol:.1e}", flush=True)
    assert err <= tol, (where, err, tol)


def case(shape, dtype, affine, groups, seed, shift=0):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731

    def place(t):  # `shift` elements behind an aligned address
        if not shift or t is None:
            return t
        flat = torch.empty(t.numel() + shift, dtype=t.dtype)
        out = flat[shift:].view(t.shape)
        out.copy_(t)
        return out

    x = (1.5 * rn(*shape) + 0.5 * rn(*shape[:-1], 1)).to(dtype)
    ws = shape[-2:] if groups else shape[-1:]
    w, b = (1 + 0.2 * rn(*ws), 0.2 * rn(*ws)) if affine else (None, None)
    return place(x), place(w), place(b), place(rn(*shape).to(dtype))


def to_dev(t, shift=0):
    if t is None:
        return None
    if not shift:
        return t.to(DEV)
    out = torch.empty(t.numel() + shift, dtype=t.dtype, device=DEV)[shift:].view(t.shape)
    return out.copy_(t)


SHAPES = [  # shape, weights per head
    ((1, 1), False), ((5, 2), False), ((3, 16), False), ((700, 64), False), ((33, 5, 128), True), ((2, 3, 4, 256), True),
    ((9, 1000), False), ((4, 3, 333), True), ((300, 2048), False), ((11, 2049), False), ((6, 4096), False),
    ((7, 2, 8192), True), ((3, 16384), False), ((2, 20000), False), ((3, 9001), False), ((0, 64), False), ((1030, 1, 24), True),
]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape,groups", SHAPES, ids=str)
def test_parity(shape, groups, dtype):
    for affine in ((True,) if groups else (True, False)):
        for shift in (0, 1):
            announce(f"layer_norm {shape} groups={groups} {dtype} affine={affine} shift={shift}")
            x, w, b, dy = case(shape, dtype, affine, groups, seed=shape[-1])
            X, W, B, DY = (to_dev(t, shift) for t in (x, w, b, dy))
            f = bd.layer_norm_fwd(X, W, B, eps=EPS, want_ckpt8=True)
            ref = reference(x, w, b)
            out = 2.0**-8 + 8 * SUM32 if dtype == BF else 16 * SUM32
            near(f["mean"], ref["mean"], 8 * SUM32, "mean")
            near(f["rstd"], ref["rstd"], 8 * SUM32, "rstd")
            near(f["y"], ref["y"], out, "y")
            plain = bd.layer_norm_fwd(X, W, B, eps=EPS)
            assert "x8" not in plain
            for n in plain:
                assert torch.equal(plain[n], f[n]), n
            q, s = codes(x)
            assert torch.equal(f["x8"].cpu(), q) and torch.equal(f["x8_scale"].cpu(), s)
            stats = f["mean"].cpu(), f["rstd"].cpu()
            for ck in (False, True):
                g = bd.layer_norm_bwd(DY, None if ck else X, f["mean"], f["rstd"], W,
                                      ckpt8=(f["x8"], f["x8_scale"]) if ck else None)
                r = reference(kept(q, s, shape[-1]) if ck else x, w, b, dy, stats)
                near(g["dx"], r["dx"], out, f"dx ck={ck}")
                if affine:
                    near(g["dweight"], r["dweight"], 16 * SUM32, f"dweight ck={ck}")
                    near(g["dbias"], r["dbias"], 16 * SUM32, f"dbias ck={ck}")
                else:
                    assert g["dweight"] is None and g["dbias"] is None


def test_large_mean_constant_rows_and_zero_variance():
    announce("layer_norm large mean")
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(64, 512, generator=gen) + 1e4  # E[x^2] - mean^2 would keep no digit of the variance
    x[3] = 5.0
    x[4] = 0.0
    f = bd.layer_norm_fwd(x.to(DEV), eps=EPS)
    ref = reference(x, None, None)
    # the mean is rounded to 2^-24 of 1e4 (6e-4), which shifts every h by 6e-4
    near(f["y"], ref["y"], 2e-3, "y")
    assert (f["y"][3:5] == 0).all()
    assert abs(float(f["rstd"][4]) * math.sqrt(EPS) - 1) < 1e-6


def test_not_a_number_stays_in_its_row():
    announce("layer_norm NaN")
    x, w, b, dy = case((300, 3, 128), BF, True, True, seed=1)
    X, W, B, DY = (t.to(DEV) for t in (x, w, b, dy))
    clean = bd.layer_norm_fwd(X, W, B, want_ckpt8=True)
    gc = bd.layer_norm_bwd(DY, X, clean["mean"], clean["rstd"], W)
    for bad in (float("nan"), float("inf")):
        Y = X.clone()
        Y[17, 1, 5] = bad
        f = bd.layer_norm_fwd(Y, W, B, want_ckpt8=True)
        g = bd.layer_norm_bwd(DY, Y, f["mean"], f["rstd"], W)
        g8 = bd.layer_norm_bwd(DY, None, f["mean"], f["rstd"], W, ckpt8=(f["x8"], f["x8_scale"]))
        keep = torch.ones(300, 3, dtype=torch.bool, device=DEV)
        keep[17, 1] = False
        assert torch.equal(f["y"][keep], clean["y"][keep]) and torch.equal(g["dx"][keep], gc["dx"][keep])
        assert torch.isnan(f["y"][17, 1]).any() and torch.isnan(g["dx"][17, 1]).all() and torch.isnan(g8["dx"][17, 1]).all()
        assert torch.equal(g["dweight"][[0, 2]], gc["dweight"][[0, 2]])


def test_tiny_and_empty_blocks_of_the_8_bit_form():
    announce("layer_norm 8-bit blocks")
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(4, 200, generator=gen)
    x[0, :64] = 0
    x[1, 64:128] *= 1e-37
    x[2] *= 1e-30
    x[3] *= 1e30
    f = bd.layer_norm_fwd(x.to(DEV), want_ckpt8=True)
    q, s = codes(x)
    assert torch.equal(f["x8"].cpu(), q) and torch.equal(f["x8_scale"].cpu(), s)
    v = kept(q, s, 200)
    top = torch.nn.functional.pad(x, (0, 56)).reshape(4, 4, 64).abs().amax(-1).double().repeat_interleave(64, -1)[:, :200]
    ok = top >= 1e-36
    # half a step, and the roundings of the scale, its inverse and the product (4 of 2^-24 of 127 steps)
    assert ((v - x.double()).abs()[ok] <= (top[ok] / 254) * (1 + 254 * 4 * U32)).all()
    assert (v[~ok] == 0).all()


def test_gradients_against_differences():
    announce("layer_norm differences")
    x, w, b, dy = case((40, 2, 72), F32, True, True, seed=4)
    X, W, B, DY = (t.to(DEV) for t in (x, w, b, dy))
    f = bd.layer_norm_fwd(X, W, B)
    g = bd.layer_norm_bwd(DY, X, f["mean"], f["rstd"], W)
    gen = torch.Generator().manual_seed(5)
    J = lambda x_, w_, b_: float((reference(x_, w_, b_)["y"] * dy.double()).sum())  # noqa: E731
    at = dict(x=x.double(), w=w.double(), b=b.double())
    for n, o in (("x", "dx"), ("w", "dweight"), ("b", "dbias")):
        dirn = torch.randn(at[n].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        args = [{**at, n: at[n] + s * h * dirn} for s in (1, -1)]
        want = (J(**{k + "_": v for k, v in args[0].items()}) - J(**{k + "_": v for k, v in args[1].items()})) / (2 * h)
        grad = g[o].double().cpu()
        # as for the delta rule: 5 standard deviations of the gradient's error, and the difference's own
        assert abs(float((grad * dirn).sum()) - want) <= (5 * 16 * SUM32 + 1e-7 * float(dirn.norm())) * float(grad.norm()), n


def test_deterministic_captured_and_on_other_streams():
    announce("layer_norm streams, graph")
    x, w, b, dy = case((500, 4, 128), BF, True, True, seed=6)
    X, W, B, DY = (t.to(DEV) for t in (x, w, b, dy))

    def run(**kw):
        f = bd.layer_norm_fwd(X, W, B, want_ckpt8=True, **kw)
        return {**f, **bd.layer_norm_bwd(DY, None, f["mean"], f["rstd"], W, ckpt8=(f["x8"], f["x8_scale"]), **kw)}

    want = run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [run(stream=s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    for o in got:
        for n in want:
            assert torch.equal(want[n], o[n]), n
    graph = torch.cuda.CUDAGraph()
    s = streams[0]
    with torch.cuda.stream(s):
        run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        o = run()
    gen = torch.Generator().manual_seed(3)
    for _ in range(3):
        X.copy_(torch.randn(X.shape, generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        e = run()
        torch.cuda.synchronize()
        for n in e:
            assert torch.equal(e[n], o[n]), n


# ---------------------------------------------------------------- as a layer
def test_norm_delta_rule_norm_forward_and_backward():
    """A layer's path: the input norm (its input kept in 8 bits), the delta rule on slices of its output, the
    norm of every head's readout, and back; then one more token through delta_step and the heads' norm.
    Against torch's autograd in float64 on the same path from the values that the kernels passed on
    (each operator's inputs as it got them, so that only its own errors count)."""
    announce("norm + delta rule + norm")
    gen = torch.Generator().manual_seed(9)
    b, T, H, HV, K, V = 2, 100, 2, 4, 32, 48
    width = 2 * H * K + HV * V
    x = torch.randn(b, T, width, generator=gen).to(BF).to(DEV)
    w1, b1 = (1 + 0.1 * torch.randn(width, generator=gen)).to(DEV), (0.1 * torch.randn(width, generator=gen)).to(DEV)
    w2, b2 = (1 + 0.1 * torch.randn(HV, V, generator=gen)).to(DEV), (0.1 * torch.randn(HV, V, generator=gen)).to(DEV)
    beta = torch.rand(b, T, HV, generator=gen).to(DEV)
    g = (-0.2 * torch.rand(b, T, HV, generator=gen)).to(DEV)
    dz = torch.randn(b, T, HV, V, generator=gen).to(BF).to(DEV)
    scale = 1 / K

    n1 = bd.layer_norm_fwd(x, w1, b1, eps=EPS, want_ckpt8=True)
    q, k, v = n1["y"].split([H * K, H * K, HV * V], -1)
    q, k, v = q.reshape(b, T, H, K), (q.reshape(b, T, H, K) * 0 + k.reshape(b, T, H, K) / K**0.5), v.reshape(b, T, HV, V)
    q, k, v = (t.contiguous() for t in (q, k, v))
    f = bd.delta_chunk_fwd(q, k, v, beta, g, scale=scale)
    n2 = bd.layer_norm_fwd(f["o"], w2, b2, eps=EPS)
    g2 = bd.layer_norm_bwd(dz, f["o"], n2["mean"], n2["rstd"], w2)
    gd = bd.delta_chunk_bwd(q, k, v, beta, g, None, g2["dx"], scale=scale)
    dy1 = torch.cat([gd["dq"].reshape(b, T, -1), (gd["dk"] / K**0.5).reshape(b, T, -1), gd["dv"].reshape(b, T, -1)], -1).contiguous()
    g1 = bd.layer_norm_bwd(dy1, None, n1["mean"], n1["rstd"], w1, ckpt8=(n1["x8"], n1["x8_scale"]))
    torch.cuda.synchronize()

    c = lambda t: t.detach().double().cpu()  # noqa: E731
    qr, kr, vr, br, gr = (c(t).requires_grad_() for t in (q, k, v, beta, g))
    S = torch.zeros(b, HV, K, V, dtype=torch.float64)
    rep, outs = HV // H, []
    for t in range(T):
        kt, qt = kr[:, t].repeat_interleave(rep, 1), qr[:, t].repeat_interleave(rep, 1)
        S = torch.exp(gr[:, t])[..., None, None] * S
        r = vr[:, t] - (kt[..., None] * S).sum(-2)
        S = S + (br[:, t, :, None] * kt)[..., None] * r[..., None, :]
        outs.append(scale * (qt[..., None] * S).sum(-2))
    o = torch.stack(outs, 1)
    rel = lambda a, e: float((c(a) - e).norm() / e.norm())  # noqa: E731
    assert rel(f["o"], o.detach()) <= TOL_BF16 and rel(f["S_final"], S.detach()) <= TOL_SPLIT
    grads = torch.autograd.grad((o * c(g2["dx"])).sum(), (qr, kr, vr, br, gr))
    for n, e, tol in zip(("dq", "dk", "dv", "dbeta", "dg"), grads, [TOL_BF16] * 3 + [TOL_SPLIT] * 2):
        assert rel(gd[n], e) <= tol, (n, rel(gd[n], e))
    r2 = reference(c(f["o"]), c(w2), c(b2), c(dz))
    assert rel(n2["y"], r2["y"]) <= TOL_BF16 and rel(g2["dx"], r2["dx"]) <= TOL_BF16
    r1 = reference(kept(n1["x8"].cpu(), n1["x8_scale"].cpu(), width), c(w1), c(b1), c(dy1), (c(n1["mean"]), c(n1["rstd"])))
    assert rel(g1["dx"], r1["dx"]) <= TOL_BF16 and rel(g1["dweight"], r1["dweight"]) <= 16 * SUM32
    # what the 8 bits cost: the exact gradient of the same path.  A kept value is off by max|x| / 254 / sqrt(3) of a
    # block of 64 (max about 2.6 standard deviations): 0.6 % of h, which enters dx only through h sum(t h) / D
    full = reference(c(x), c(w1), c(b1), c(dy1))
    assert rel(g1["dx"], full["dx"]) <= TOL_BF16 + 2.6 / 254 and rel(g1["dweight"], full["dweight"]) <= 2.6 / 254

    # the next token of every sequence
    tok = [torch.randn(b, n, d, generator=gen).to(BF).to(DEV) for n, d in ((H, K), (H, K), (HV, V))]
    tok[1] = torch.nn.functional.normalize(tok[1].float(), dim=-1).to(BF)
    pool = f["S_final"].clone()
    o1 = bd.delta_step(*tok, beta[:, 0].contiguous(), g[:, 0].contiguous(), pool, scale=scale)
    z1 = bd.layer_norm_fwd(o1, w2, b2, eps=EPS)["y"]
    kt, qt = (c(t).repeat_interleave(rep, 1) for t in (tok[1], tok[0]))
    S1 = torch.exp(c(g[:, 0]))[..., None, None] * c(f["S_final"])
    S1 = S1 + (c(beta[:, 0])[..., None] * kt)[..., None] * (c(tok[2]) - (kt[..., None] * S1).sum(-2))[..., None, :]
    assert rel(pool, S1) <= SUM32
    assert rel(z1, reference(c(o1), c(w2), c(b2))["y"]) <= TOL_BF16
