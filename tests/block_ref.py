"""The linear recurrence, the gated feed-forward projections and dropout in float64 on the CPU,
each beside a bound of the float32 error that their kernels may have.

Roundings: u = 2^-24 relative for each float32 operation; half a step of the type for a stored value
(bf16 2^-8).  `unit` is the relative error of one token's coefficients:
  log form:   exp of |g| <= 8: the product with log2 e is off by u (8 log2 e) and the power by 2 u: 16 u
  gated form: sigmoid of |r| <= 8 to 14 u, c softplus(decay) to 4 u, so L to 20 u and a (L <= 2) to 44 u;
              1 - a^2 where 2 L >= 0.25 is off by 2 * 44 u * 0.78 / 0.22 = 312 u of itself in the worst case
              (all errors of a of one sign), its root by half of that; sigmoid(i) and two products 17 u: 176 u
A state's error then obeys e_t <= a e_{t-1} + unit (a |h_{t-1}| + |u_t|), whatever the grouping of the
products: every token's factor is used at most once between two tokens.  The adjoint's likewise.
"""
import math

import torch

U = 2.0**-24
UNIT = {"log": 16 * U, "gated": 176 * U}
HALF = {torch.float32: U, torch.bfloat16: 2.0**-8}
F32, BF = torch.float32, torch.bfloat16
C = 8.0


def lengths_of(n, T, lens):
    return [T] * n if lens is None else list(lens)


def make_scan(form, n, T, D, dtype, lens=None, state=True, seed=0, reset=False, first=0, tail=0):
    """CPU inputs.  lens: packed sequences of these lengths, `first` tokens before them and `tail` behind."""
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen).clamp(-4, 4)  # noqa: E731
    b = n if lens is None else len(lens)
    if lens is not None:
        n, T = 1, first + sum(lens) + tail
    d = dict(form=form, x=rn(n, T, D).to(dtype), lens=lens, first=first, dh=rn(n, T, D).to(dtype), input_gate=None, decay=None,
             h0=rn(b, D) if state else None, dh_final=rn(b, D) if state else None, seq_offsets=None)
    if form == "gated":
        d["gate"], d["input_gate"] = rn(n, T, D).to(dtype), rn(n, T, D).to(dtype)
        d["decay"] = torch.linspace(-9.0, -2.5, D)  # a from 0.999 down to 0.55 and below
    else:
        rate = torch.exp(torch.linspace(math.log(0.001), math.log(2.0), D))
        d["gate"] = -(rate * torch.nn.functional.softplus(rn(n, T, D))).clamp(max=8)
        if reset:
            d["gate"][torch.rand(n, T, D, generator=gen) < 0.02] = -math.inf
    if lens is not None:
        edges = [first]
        for k in lens:
            edges.append(edges[-1] + k)
        d["seq_offsets"] = torch.tensor(edges, dtype=torch.int32)
    return d


def coefficients(d):
    """a, u (float64, differentiable in what d holds) of every token."""
    x = d["x"].double()
    if d["form"] == "log":
        return torch.exp(d["gate"].double()), x
    L = C * torch.nn.functional.softplus(d["decay"].double()) * torch.sigmoid(d["gate"].double())
    return torch.exp(-L), torch.sqrt(-torch.expm1(-2 * L)) * torch.sigmoid(d["input_gate"].double()) * x


def spans(d):
    """(row of the batch axis, first token, length) of every sequence."""
    if d["lens"] is None:
        return [(i, 0, d["x"].shape[1]) for i in range(d["x"].shape[0])]
    out, at = [], d["first"]
    for k in d["lens"]:
        out.append((0, at, k))
        at += k
    return out


def scan_forward(d):
    """h per sequence (lists of [len, D]), the final states."""
    a, u = coefficients(d)
    hs, last = [], []
    for s, (row, at, n) in enumerate(spans(d)):
        h = torch.zeros(a.shape[-1], dtype=torch.float64) if d["h0"] is None else d["h0"][s].double()
        seq = []
        for t in range(at, at + n):
            h = a[row, t] * h + u[row, t]
            seq.append(h)
        hs.append(torch.stack(seq) if seq else a.new_zeros(0, a.shape[-1]))
        last.append(h)
    return hs, (torch.stack(last) if last else a.new_zeros(0, a.shape[-1]))


def scan_reference(d):
    """Values and gradients (torch's own differentiation of the loop) with the bounds of their float32 errors."""
    leaves = {k: d[k].double().clone().requires_grad_(True) for k in ("x", "gate", "input_gate", "decay", "h0") if d[k] is not None}
    e = dict(d, **leaves)
    hs, last = scan_forward(e)
    J = (last * d["dh_final"].double()).sum() if d["dh_final"] is not None else 0.0 * last.sum()
    for (row, at, n), h in zip(spans(d), hs):
        J = J + (h * d["dh"][row, at:at + n].double()).sum()
    g = dict(zip(leaves, torch.autograd.grad(J, list(leaves.values()), allow_unused=True)))
    g = {k: (torch.zeros_like(leaves[k]) if v is None else torch.nan_to_num(v)) for k, v in g.items()}
    unit = UNIT[d["form"]]
    a, u = (t.detach() for t in coefficients(d))
    shape = d["x"].shape
    z = lambda: torch.zeros(shape, dtype=torch.float64)  # noqa: E731
    h, eh, hp, ehp, lam, el = z(), z(), z(), z(), z(), z()
    el_last, eh_last = torch.zeros_like(last), torch.zeros_like(last)
    for s, (row, at, n) in enumerate(spans(d)):
        cur = torch.zeros(shape[-1], dtype=torch.float64) if d["h0"] is None else d["h0"][s].double()
        err = torch.zeros_like(cur)
        for t in range(at, at + n):
            hp[row, t], ehp[row, t] = cur, err
            err = a[row, t] * err + unit * ((a[row, t] * cur).abs() + u[row, t].abs())
            cur = a[row, t] * cur + u[row, t]
            h[row, t], eh[row, t] = cur, err
        eh_last[s] = err
        cur = torch.zeros_like(cur) if d["dh_final"] is None else d["dh_final"][s].double()
        err = torch.zeros_like(cur)
        for t in reversed(range(at, at + n)):
            lam[row, t] = cur + d["dh"][row, t].double()
            el[row, t] = err + unit * (cur.abs() + lam[row, t].abs())
            cur, err = a[row, t] * lam[row, t], a[row, t] * (el[row, t] + unit * lam[row, t].abs())
        el_last[s] = err
    half = HALF[d["x"].dtype]
    out = {"h": (h, eh + half * (h.abs() + eh)), "h_final": (last.detach(), eh_last + U * last.detach().abs())}
    if d["form"] == "log":
        dg = lam * a * hp
        out["dx"] = (g["x"], el + half * (lam.abs() + el))
        out["dgate"] = (g["gate"], el * (a * hp).abs() + (lam * a).abs() * ehp + 2 * unit * dg.abs())
    else:
        x = d["x"].double()
        r, w = torch.sigmoid(d["gate"].double()), torch.sigmoid(d["input_gate"].double())
        sp = torch.nn.functional.softplus(d["decay"].double())
        L = C * sp * r
        m = torch.sqrt(-torch.expm1(-2 * L))
        t1, t2 = w * x * a * a * L / m, L * a * hp
        eE = el * (t1 - t2).abs() + lam.abs() * (3 * unit * (t1.abs() + t2.abs()) + L * a * ehp)
        bx = el * m * w + 2 * unit * (lam * m * w).abs()
        out["dx"] = (g["x"], bx + half * (g["x"].abs() + bx))
        bi = (bx + unit * (lam * m * w).abs()) * x.abs() * (1 - w) + 16 * U * (lam * m * w * x).abs()
        out["dinput_gate"] = (g["input_gate"], bi + half * (g["input_gate"].abs() + bi))
        bg = eE * (1 - r) + 16 * U * (lam * (t1 - t2)).abs()
        out["dgate"] = (g["gate"], bg + half * (g["gate"].abs() + bg))
        slope = torch.sigmoid(d["decay"].double()) / sp
        E = (lam * (t1 - t2)).abs()
        # the sum over the tokens: at most 16 + 64 + 8 serial float32 additions in each of three levels
        out["ddecay"] = (g["decay"], slope * (eE.sum((0, 1)) + (3 * 88 * U + 8 * U) * E.sum((0, 1))))
    if d["h0"] is not None:
        out["dh0"] = (g["h0"], el_last + 2 * unit * g["h0"].abs())
    return out


def check(got, want, bound, where, mask=None):
    """|got - want| <= bound everywhere (mask: where it is looked at)."""
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (where, got.shape, want.shape)
    if mask is not None:
        got, want, bound = got[mask], want[mask], bound[mask]
    if not want.numel():
        return
    assert torch.isfinite(got).all(), (where, "not finite")
    over = (got - want).abs() - bound - 1e-30
    worst = float(((got - want).abs() / (bound + 1e-30)).max())
    print(f"{where}: {worst:.2f} of the bound", flush=True)
    assert (over <= 0).all(), (where, worst, int((over > 0).sum()), got.numel())


def owned(d):
    """Which tokens a sequence owns, [n, T]."""
    m = torch.zeros(d["x"].shape[:2], dtype=torch.bool)
    for row, at, n in spans(d):
        m[row, at:at + n] = True
    return m


# ---------------------------------------------------------------------------------------------- feed-forward
def act(name, z):
    if name == "silu":
        return z * torch.sigmoid(z)
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z**3)))


def ffn_reference(x, wg, wu, dh, name, saved=None, dtype=F32):
    """Values and gradients with bounds: a sum of K products in float32 is off by at most K u sum |products|,
    act and its derivative (both with a slope below 1.2) by 24 u where |z| <= 8; dgate and dup are rounded to dtype once."""
    x, wg, wu, dh = (t.double() for t in (x, wg, wu, dh))
    half = HALF[dtype]
    K, F, M = x.shape[1], wg.shape[0], x.shape[0]
    gate, up = x @ wg.T, x @ wu.T
    eg, eu = K * U * (x.abs() @ wg.abs().T), K * U * (x.abs() @ wu.abs().T)
    f = act(name, gate)
    h = f * up
    eh = 1.2 * eg * up.abs() + (f.abs() + 1.2 * eg) * eu + 24 * U * (gate.abs() * up.abs())
    out = {"h": (h, eh + half * (h.abs() + eh)), "gate": (gate, eg + half * (gate.abs() + eg)), "up": (up, eu + half * (up.abs() + eu))}
    if saved is not None:
        gate, up = (t.double() for t in saved)
        eg, eu = torch.zeros_like(gate), torch.zeros_like(up)
    z = gate.clone().requires_grad_(True)
    df, = torch.autograd.grad(act(name, z).sum(), z)
    f = act(name, gate)
    dg, du = dh * up * df, dh * f
    edg = dh.abs() * (1.2 * (eu + eg * up.abs()) + 32 * U * up.abs() * (1 + gate.abs()))
    edu = dh.abs() * (1.2 * eg + 24 * U * gate.abs())
    edg, edu = edg + half * (dg.abs() + edg), edu + half * (du.abs() + edu)
    for n, v, e in (("dx", dg @ wg + du @ wu, edg @ wg.abs() + edu @ wu.abs() + 2 * F * U * (dg.abs() @ wg.abs() + du.abs() @ wu.abs())),
                    ("dw_gate", dg.T @ x, edg.T @ x.abs() + M * U * (dg.abs().T @ x.abs())),
                    ("dw_up", du.T @ x, edu.T @ x.abs() + M * U * (du.abs().T @ x.abs()))):
        out[n] = (v, e + half * (v.abs() + e))
    return out


# ---------------------------------------------------------------------------------------------------- dropout
def philox(counter, key):
    """Philox 4x32-10 in Python integers."""
    c, k, low = list(counter), list(key), 0xFFFFFFFF
    for _ in range(10):
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(q >> 32) ^ c[1] ^ k[0], q & low, (p >> 32) ^ c[3] ^ k[1], p & low]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    return c


def keep_mask(n, p, seed, offset):
    t = round(65536 * p)
    seed, offset, low = seed % 2**64, offset % 2**64, 0xFFFFFFFF
    out = []
    for b in range((n + 7) // 8):
        for w in philox((b & low, b >> 32, offset & low, offset >> 32), (seed & low, seed >> 32)):
            out += [(w & 0xFFFF) >= t, (w >> 16) >= t]
    return torch.tensor(out[:n], dtype=torch.bool)


def dropout_reference(x, p, seed, offset, residual=None):
    t = round(65536 * p)
    keep = keep_mask(x.numel(), p, seed, offset).reshape(x.shape)
    y = torch.where(keep, x.double() * (65536 / (65536 - t) if t < 65536 else 0.0), 0.0)
    return (y if residual is None else y + residual.double()), keep
