"""Float64 reference of the gated delta rule with one gate per value head: the
oracle's delta rule (one gate per key channel) with the gate repeated over the
channels and its gradient summed over them, sequence by sequence."""
import math

import numpy as np
import torch

import oracle

BF, F32 = torch.bfloat16, torch.float32

# Tolerances, as the 2-norm of the error over the 2-norm of the result.
#
# bf16 results: one rounding is off by at most half a step, 2^-8 of the value,
# 2^-8 / sqrt(3) in the mean square.  A readout or a gradient that is a sum of
# products passes at most four independent ones: its own, and one of each of
# three computed operands (state, r or mu, pair weights).
TOL_BF16 = 2.0**-8 * math.sqrt(4 / 3)
# float32 results of the chunked form: a computed operand is kept in two bf16
# parts, off by at most 2^-16, 2^-16 / 3 in the mean square; a product of two
# such operands also drops lo * lo, as large again.  At most five such products
# lie between the inputs and a result (K S, T R, K dS, T^T dU, K^T u): sqrt(15)
# errors, times 2 for the norm of the triangular inverse.
TOL_SPLIT = 2 * math.sqrt(15) * 2.0**-16 / 3
# float32 kernels: 2^-24 per operation, sums of up to 128 rows over up to a few
# hundred tokens, added in quadrature with the same factor 2.
TOL_F32 = 2 * math.sqrt(128 * 256) * 2.0**-24


def inputs(b, T, H, HV, K, V, dtype=BF, state=True, packed=None, seed=0, rate=0.1):
    """CPU tensors q, k, v, beta, g, S0, d_o, dS as the kernels get them; packed: lengths."""
    gen = torch.Generator().manual_seed(seed)

    def rn(*s):
        return torch.randn(s, generator=gen, dtype=torch.float64)

    n = 1 if packed is not None else b
    ns = len(packed) if packed is not None else b

    def unit(x):
        return (x / x.norm(dim=-1, keepdim=True)).to(dtype)

    d = dict(q=unit(rn(n, T, H, K)), k=unit(rn(n, T, H, K)), v=rn(n, T, HV, V).to(dtype),
             beta=torch.sigmoid(rn(n, T, HV)).float(),
             g=(-rate * torch.nn.functional.softplus(rn(n, T, HV))).float(),
             S0=(0.3 * rn(ns, HV, K, V)).float() if state else None, d_o=rn(n, T, HV, V).to(dtype),
             dS=(0.3 * rn(ns, HV, K, V)).float() if state else None, scale=K**-0.5, offsets=None)
    if packed is not None:
        edges = np.concatenate([[0], np.cumsum(packed)])
        d["offsets"] = torch.tensor(edges, dtype=torch.int32)
    return d


def spans(d):
    """(row of the token tensors' first axis, first token, last token + 1) of every sequence."""
    if d["offsets"] is None:
        return [(i, 0, d["q"].shape[1]) for i in range(d["q"].shape[0])]
    o = d["offsets"].tolist()
    return [(0, a, e) for a, e in zip(o, o[1:])]


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _sum_scales(x, S0, dS, scale):
    """Per token and head, the root of the sum of the squared terms of dbeta_t = sum_v r_v du_v and of
    dg_t = sum_kv (S_dec)_kv (dS_dec)_kv, in float64 (one sequence, arrays [T,...]).

    Both are sums of products whose factors carry independent errors of relative size e, so that the sum is
    off by e times this, however much of the sum itself cancels."""
    T, HV = x["beta"].shape
    rep = HV // x["q"].shape[1]
    q, k = (np.repeat(x[n], rep, axis=1) for n in ("q", "k"))
    S = np.zeros((HV, q.shape[-1], x["v"].shape[-1])) if S0 is None else S0.copy()
    dS = np.zeros_like(S) if dS is None else dS.copy()
    decs, rs = [], []
    for t in range(T):
        dec = np.exp(x["g"][t])[:, None, None] * S
        r = x["v"][t] - np.einsum("hk,hkv->hv", k[t], dec)
        S = dec + np.einsum("hk,hv->hkv", k[t], x["beta"][t][:, None] * r)
        decs.append(dec)
        rs.append(r)
    yb, yg = np.zeros((T, HV)), np.zeros((T, HV))
    for t in reversed(range(T)):
        dS = dS + scale * np.einsum("hk,hv->hkv", q[t], x["d_o"][t])
        du = np.einsum("hk,hkv->hv", k[t], dS)
        yb[t] = np.sqrt(((rs[t] * du) ** 2).sum(-1))
        ddec = dS - np.einsum("hk,hv->hkv", k[t], x["beta"][t][:, None] * du)
        yg[t] = np.sqrt(((decs[t] * ddec) ** 2).sum((-1, -2)))
        dS = np.exp(x["g"][t])[:, None, None] * ddec
    return yb, yg


def reference(d, grads=True):
    """Outputs of delta_chunk_fwd and, with grads, of delta_chunk_bwd as float64 tensors (rows that
    no sequence owns stay zero)."""
    K = d["q"].shape[-1]
    x = {n: _np(d[n]) for n in ("q", "k", "v", "beta", "g", "d_o")}
    out = {"o": np.zeros_like(x["v"])}
    if grads:
        out.update({"d" + n: np.zeros_like(x[n]) for n in ("q", "k", "v", "beta", "g")})
        out.update({n: np.zeros_like(x["beta"]) for n in ("scale of dbeta", "scale of dg")})
    sf, ds0 = [], []
    for i, (row, a, e) in enumerate(spans(d)):
        c = {n: np.ascontiguousarray(x[n][row:row + 1, a:e]) for n in x}
        gk = np.repeat(c["g"][..., None], K, axis=-1)
        S0 = None if d["S0"] is None else _np(d["S0"][i:i + 1])
        o, s = oracle.kda_fwd(c["q"], c["k"], c["v"], c["beta"], gk, S0, scale=d["scale"])
        out["o"][row, a:e] = o[0]
        sf.append(s[0])
        if grads:
            r = oracle.kda_bwd(c["q"], c["k"], c["v"], c["beta"], gk, S0, c["d_o"],
                               None if d["dS"] is None else _np(d["dS"][i:i + 1]), scale=d["scale"])
            for n in ("dq", "dk", "dv", "dbeta"):
                out[n][row, a:e] = r[n][0]
            out["dg"][row, a:e] = r["dg"][0].sum(-1)
            ds0.append(r["dS0"][0])
            if e - a <= 1000:
                yb, yg = _sum_scales({n: v[0] for n, v in c.items()}, None if S0 is None else S0[0],
                                     None if d["dS"] is None else _np(d["dS"][i]), d["scale"])
                out["scale of dbeta"][row, a:e], out["scale of dg"][row, a:e] = yb, yg
    out["S_final"] = np.stack(sf)
    if grads:
        out["dS0"] = np.stack(ds0)
    return {n: torch.from_numpy(v) for n, v in out.items()}


def check(got, ref, tols, where="", floors={}):
    """got[n] against ref[n] for n in tols: the 2-norm as a whole, and every value within
    8 tol of the larger of itself and the root mean square (five standard deviations of the
    operands' errors and one whole rounding of the largest values).  floors[n] is an absolute
    error that every value of n may have besides."""
    errs = {}
    for n, tol in tols.items():
        a, e = got[n].detach().double().cpu(), ref[n].double()
        assert a.shape == e.shape, (n, a.shape, e.shape)
        if not e.numel():
            continue
        assert torch.isfinite(a).all(), (where, n)
        err = ((a - e).abs() - floors.get(n, 0.0)).clamp(min=0.0)
        norm = max(float(e.norm()), float(ref["scale of " + n].norm()) if "scale of " + n in ref else 0.0)
        if norm == 0:
            assert float(a.abs().max()) == 0, (where, n)
            continue
        rms = norm / math.sqrt(e.numel())
        rel = float(err.norm()) / norm
        big = float((err / e.abs().clamp(min=rms)).max())
        errs[n] = (rel, big, tol)
    print(where, {n: f"{r:.1e}/{b:.1e}" for n, (r, b, _) in errs.items()}, flush=True)
    bad = {n: v for n, v in errs.items() if v[0] > v[2] or v[1] > 8 * v[2]}
    assert not bad, (where, bad)
