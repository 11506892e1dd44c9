"""The measured cases of the gated delta rule (chunked and recurrent) and of the layer norm behind it.

Operators, all of ``selective_state_space_vjp_amd.binding``:

* ``delta_chunk_fwd``   the gated delta rule with one log gate per value head, over whole sequences
* ``delta_chunk_bwd``   its gradients
* ``delta_step``        one token per request on a pool of states, in place
* ``layer_norm_fwd``    layer norm of the last axis, one weight row per group of rows (heads) or one for all
* ``layer_norm_bwd``    its gradients
* both with ``ckpt8``   the forward leaves its input in 8 bits, the backward reads that

Per value head, with S_{-1} = S0 and a_t = exp(g_t):
    r_t = v_t - k_t^T (a_t S_{t-1});  S_t = a_t S_{t-1} + (beta_t k_t) (x) r_t;  o_t = (scale q_t)^T S_t
Per row of D values: y = (x - mean) rstd w + b.  The 8-bit form of x: for each block of 64 values of a row the
scale is max|x| / 127 and the codes are x * (127 / max|x|), rounded half to even, all in float32 (a block whose
max|x| is below 1e-36 is stored as zeros).
"""
import math
import random

import torch

own = False
BLOCK = 64  # values per 8-bit scale
EPS = 1e-5


# ------------------------------------------------------------------------------------------------ cases
def listed():
    bf = "bfloat16"
    return [
        # prefill or the forward half of a training step of one layer: the sizes of the repository's kda workload
        dict(name="delta fwd layer", op="fwd", b=2, T=4096, packed=False, state=False, H=16, HV=32, K=128, V=128, dtype=bf),
        # prompts of different lengths packed behind one another, continued from kept states
        dict(name="delta fwd packed", op="fwd", b=13, T=2989, packed=True, state=True, H=8, HV=8, K=128, V=128, dtype=bf),
        # the backward half of a training step of one layer
        dict(name="delta bwd layer", op="bwd", b=2, T=4096, packed=False, state=False, H=16, HV=32, K=128, V=128, dtype=bf),
        # packed documents in a small model with narrow heads, truncated at kept states
        dict(name="delta bwd packed", op="bwd", b=7, T=3001, packed=True, state=True, H=4, HV=8, K=64, V=80, dtype=bf),
        # one request's next token: launch and latency
        dict(name="step 1", op="step", b=1, slots=4, H=16, HV=32, K=128, V=128, gate="head", dtype=bf),
        # a full serving batch: the states' traffic
        dict(name="step 256", op="step", b=256, slots=300, H=16, HV=32, K=128, V=128, gate="head", dtype=bf),
        # the norm of every head's readout, each head with its own weights
        dict(name="norm fwd heads", op="norm_fwd", rows=2 * 4096, G=32, D=128, dtype=bf, affine=True),
        # the same for the tokens of one decode step
        dict(name="norm fwd few", op="norm_fwd", rows=9, G=32, D=128, dtype=bf, affine=True),
        # a layer's input norm over the model width, training
        dict(name="norm bwd width", op="norm_bwd", rows=8192, G=1, D=4096, dtype=bf, affine=True),
        # odd width, float32
        dict(name="norm bwd odd", op="norm_bwd", rows=777, G=1, D=1001, dtype="float32", affine=True),
        # forward and backward with the input kept in 8 bits between them, over the model width
        dict(name="norm ckpt8 width", op="norm_ckpt8", rows=8192, G=1, D=4096, dtype=bf, affine=True),
        # the same per head
        dict(name="norm ckpt8 heads", op="norm_ckpt8", rows=4096, G=32, D=128, dtype=bf, affine=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "norm_fwd", "norm_bwd", "norm_ckpt8"])
    if op in ("fwd", "bwd"):
        H = rng.choice([1, 2, 3, 4, 8, 16])
        HV = H * rng.choice([1, 1, 2, 3, 4])
        K, V = 16 * rng.randint(1, 8), 16 * rng.randint(1, 12)
        packed = rng.random() < 0.5
        T = _log(rng, 1, 8192)
        b = rng.randint(1, 24) if packed else rng.randint(1, 4)
        tokens = T if packed else b * T
        most = 8192 * 32 * 128 // (HV * max(K, V))
        if tokens > most:
            T = max(1, most if packed else most // b)
        dtype = "float32" if op == "fwd" and rng.random() < 0.25 else "bfloat16"
        return dict(op=op, b=b, T=T, packed=packed, state=rng.random() < 0.5, H=H, HV=HV, K=K, V=V, dtype=dtype)
    if op == "step":
        H = rng.choice([1, 2, 3, 4, 8, 16])
        HV = H * rng.choice([1, 2, 4])
        b = _log(rng, 1, 256)
        return dict(op=op, b=b, slots=b + rng.randint(0, 40), H=H, HV=HV, K=16 * rng.randint(1, 8), V=16 * rng.randint(1, 8),
                    gate=rng.choice(["head", "key"]), dtype=rng.choice(["bfloat16", "float32"]))
    D = _log(rng, 16, 12000)
    G = rng.choice([1, 1, 2, 5, 16, 32])
    rows = _log(rng, 1, max(1, min(100000, 8192 * 4096 // (D * G))))
    return dict(op=op, rows=rows, G=G, D=D, dtype=rng.choice(["bfloat16", "bfloat16", "float32"]), affine=rng.random() < 0.8)


def _lengths(c):
    """Lengths of a packed case's sequences: uneven, one of them empty where there are three or more."""
    rng = random.Random(c["T"] * 131 + c["b"])
    cuts = sorted(rng.randint(0, c["T"]) for _ in range(c["b"] - 1))
    if len(cuts) >= 2:
        cuts[1] = cuts[0]
    edges = [0] + cuts + [c["T"]]
    return [y - x for x, y in zip(edges, edges[1:])]


def work(c):
    e = 2 if c["dtype"] == "bfloat16" else 4
    if c["op"] in ("fwd", "bwd"):
        tok = c["T"] if c["packed"] else c["b"] * c["T"]
        qk, v, gates = tok * c["H"] * c["K"], tok * c["HV"] * c["V"], tok * c["HV"]
        st = c["b"] * c["HV"] * c["K"] * c["V"] * 4
        # the recurrence itself: k^T S, the update and q^T S are 2 K V operations each per token and head
        kv = tok * c["HV"] * c["K"] * c["V"]
        if c["op"] == "fwd":
            return {"bytes": e * (2 * qk + 2 * v) + 8 * gates + st * (2 if c["state"] else 1), "flops": 6 * kv}
        return {"bytes": e * (4 * qk + 3 * v) + 16 * gates + st * (3 if c["state"] else 0), "flops": 18 * kv}
    if c["op"] == "step":
        kv = c["b"] * c["HV"] * c["K"] * c["V"]
        gate = 4 * c["b"] * c["HV"] * (c["K"] if c["gate"] == "key" else 1)
        return {"bytes": 8 * kv + e * c["b"] * (2 * c["H"] * c["K"] + 2 * c["HV"] * c["V"]) + gate + 4 * c["b"] * (c["HV"] + 1), "flops": 6 * kv}
    n, r, w = c["rows"] * c["G"] * c["D"], c["rows"] * c["G"], (c["G"] * c["D"] * 4 if c["affine"] else 0)
    blocks = r * ((c["D"] + BLOCK - 1) // BLOCK)
    if c["op"] == "norm_fwd":
        return {"bytes": 2 * e * n + 8 * r + 2 * w, "flops": 8 * n}
    if c["op"] == "norm_bwd":
        return {"bytes": 3 * e * n + 8 * r + 3 * w, "flops": 14 * n}
    # x, dy read, y, dx written, the codes written and read
    return {"bytes": (4 * e + 2) * n + 16 * r + 8 * blocks + 5 * w, "flops": 26 * n}


# ------------------------------------------------------------------------------------------------ inputs
def prepare(c, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = getattr(torch, c["dtype"])

    def rn(*shape):
        return torch.randn(shape, device=dev, generator=gen)

    def unit(x):  # rows of length one, as the layers pass q and k
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    s = dict(c=c, scale=c["K"] ** -0.5 if "K" in c else 1.0)
    if c["op"] in ("fwd", "bwd"):
        n, T = (1, c["T"]) if c["packed"] else (c["b"], c["T"])
        s["q"], s["k"] = unit(rn(n, T, c["H"], c["K"])), unit(rn(n, T, c["H"], c["K"]))
        s["v"] = rn(n, T, c["HV"], c["V"]).to(dt)
        s["beta"] = torch.sigmoid(rn(n, T, c["HV"]))
        # heads that forget within a few tokens beside heads that keep thousands
        rate = torch.exp(torch.linspace(math.log(0.002), math.log(1.0), c["HV"], device=dev))
        s["g"] = -rate * torch.nn.functional.softplus(rn(n, T, c["HV"]))
        s["S0"] = 0.3 * rn(c["b"], c["HV"], c["K"], c["V"]) if c["state"] else None
        s["offsets"] = None
        if c["packed"]:
            edges = [0]
            for length in _lengths(c):
                edges.append(edges[-1] + length)
            s["offsets"] = torch.tensor(edges, dtype=torch.int32, device=dev)
        if c["op"] == "bwd":
            s["d_o"] = rn(n, T, c["HV"], c["V"]).to(dt)
            s["dS"] = 0.3 * rn(c["b"], c["HV"], c["K"], c["V"]) if c["state"] else None
    elif c["op"] == "step":
        b = c["b"]
        s["q"], s["k"] = unit(rn(b, c["H"], c["K"])), unit(rn(b, c["H"], c["K"]))
        s["v"] = rn(b, c["HV"], c["V"]).to(dt)
        s["beta"] = torch.sigmoid(rn(b, c["HV"]))
        s["g"] = -0.1 * torch.nn.functional.softplus(rn(*((b, c["HV"]) if c["gate"] == "head" else (b, c["HV"], c["K"]))))
        s["state"] = 0.3 * rn(c["slots"], c["HV"], c["K"], c["V"])
        s["slots"] = torch.randperm(c["slots"], device=dev, generator=gen)[:b].to(torch.int32)
    else:
        shape = (c["rows"], c["G"], c["D"]) if c["G"] > 1 else (c["rows"], c["D"])
        s["x"] = (rn(*shape) * 1.5 + 0.3 * rn(*shape[:-1], 1)).to(dt)
        wshape = (c["G"], c["D"]) if c["G"] > 1 else (c["D"],)
        s["w"] = 1.0 + 0.1 * rn(*wshape) if c["affine"] else None
        s["b"] = 0.1 * rn(*wshape) if c["affine"] else None
        if c["op"] != "norm_fwd":
            s["dy"] = rn(*shape).to(dt)
        if c["op"] == "norm_bwd":  # what the forward pass left
            x = s["x"].double()
            s["mean"] = x.mean(-1).float()
            s["rstd"] = (x.var(-1, unbiased=False) + EPS).rsqrt().float()
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    op = s["c"]["op"]
    if own:
        from selective_state_space_vjp_amd import binding as bd

        if op == "fwd":
            return bd.delta_chunk_fwd(s["q"], s["k"], s["v"], s["beta"], s["g"], s["S0"], scale=s["scale"], seq_offsets=s["offsets"])
        if op == "bwd":
            out = bd.delta_chunk_bwd(s["q"], s["k"], s["v"], s["beta"], s["g"], s["S0"], s["d_o"], s["dS"], scale=s["scale"],
                                     seq_offsets=s["offsets"], want_dS0=s["c"]["state"])
            return {k: x for k, x in out.items() if x is not None}
        if op == "step":
            o = bd.delta_step(s["q"], s["k"], s["v"], s["beta"], s["g"], s["state"], scale=s["scale"], slots=s["slots"])
            return {"o": o, "state": s["state"]}
        if op == "norm_fwd":
            return bd.layer_norm_fwd(s["x"], s["w"], s["b"], eps=EPS)
        if op == "norm_bwd":
            out = bd.layer_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["w"])
            return {k: x for k, x in out.items() if x is not None}
        f = bd.layer_norm_fwd(s["x"], s["w"], s["b"], eps=EPS, want_ckpt8=True)
        out = bd.layer_norm_bwd(s["dy"], None, f["mean"], f["rstd"], s["w"], ckpt8=(f["x8"], f["x8_scale"]))
        return {"y": f["y"], "mean": f["mean"], "rstd": f["rstd"], **{k: x for k, x in out.items() if x is not None}}
    return _PLAIN[op](s)


# ------------------------------------------------------------------------------------------------ plain forms
L = 64  # chunk of the plain form


def _index(s):
    """Rows of the token axis of each padded sequence ([b, C*L], -1 behind a sequence's end), on the GPU."""
    c = s["c"]
    dev = s["q"].device
    if c["packed"]:
        lens = _lengths(c)
        starts = [sum(lens[:i]) for i in range(len(lens))]
        longest = max(lens)
    else:
        lens, starts, longest = [c["T"]] * c["b"], [i * c["T"] for i in range(c["b"])], c["T"]
    n = max(1, -(-longest // L)) * L
    t = torch.arange(n, device=dev)
    st, ln = torch.tensor(starts, device=dev), torch.tensor(lens, device=dev)
    return torch.where(t < ln[:, None], st[:, None] + t, -1)


def _rows(x, idx):
    """[.., tokens, heads, ...] -> [b, heads, C, L, ...] in float32, zeros behind the ends."""
    flat = x.reshape(-1, *x.shape[2:])
    got = flat[idx.clamp(min=0)].float() * (idx >= 0).reshape(*idx.shape, *([1] * (flat.dim() - 1)))
    return got.reshape(idx.shape[0], idx.shape[1] // L, L, *flat.shape[1:]).movedim(3, 1)


def _back(y, idx, like):
    """The inverse of _rows, in like's type and shape."""
    flat = y.movedim(1, 3).reshape(idx.numel(), *like.shape[2:])
    out = torch.empty_like(like).reshape(-1, *like.shape[2:])
    at = idx.reshape(-1)
    out[at[at >= 0]] = flat[at >= 0].to(like.dtype)
    return out.reshape(like.shape)


def _delta_common(s):
    """What both directions need of every chunk of every head, all [b, HV, C, ...]."""
    c = s["c"]
    rep = c["HV"] // c["H"]
    idx = _index(s)
    q, k = (_rows(s[n], idx).repeat_interleave(rep, 1) for n in ("q", "k"))
    v, beta = _rows(s["v"], idx), _rows(s["beta"], idx)
    G = _rows(s["g"], idx).double().cumsum(-1).float()
    lower = torch.ones(L, L, device=q.device).tril()
    gam = torch.exp((G[..., :, None] - G[..., None, :]) * lower) * lower
    kk = k @ k.mT
    A = (beta[..., :, None] * gam * kk).tril(-1)
    # (I + A)^-1 by doubling: the inverse of every diagonal block of 2 n from those of n
    inv = torch.eye(L, device=q.device).expand_as(A)
    i = torch.arange(L, device=q.device)
    n = 1
    while n < L:
        below = ((i[:, None] // (2 * n) == i // (2 * n)) & (i[:, None] // n > i // n)).float()
        inv = inv - inv @ (A * below) @ inv
        n *= 2
    return idx, q, k, v, beta, G, gam, kk, inv


def _walk(s, q, k, v, beta, G, inv):
    """The state before each chunk, the updates u of each chunk, and the last state (the recurrence is what loops)."""
    S = s["S0"].clone() if s["S0"] is not None else torch.zeros(v.shape[0], v.shape[1], k.shape[-1], v.shape[-1], device=v.device)
    eG, end = torch.exp(G)[..., None], G[..., -1:]
    w, uv = inv @ (beta[..., None] * eG * k), inv @ (beta[..., None] * v)
    kend = (torch.exp(end - G)[..., None] * k).mT.contiguous()
    states, us = [], []
    for j in range(v.shape[2]):
        u = uv[:, :, j] - w[:, :, j] @ S
        states.append(S)
        us.append(u)
        S = torch.exp(end[:, :, j])[..., None] * S + kend[:, :, j] @ u
    return torch.stack(states, 2), torch.stack(us, 2), S


def _plain_fwd(s):
    idx, q, k, v, beta, G, gam, kk, inv = _delta_common(s)
    S, u, last = _walk(s, q, k, v, beta, G, inv)
    o = s["scale"] * (torch.exp(G)[..., None] * (q @ S) + ((q @ k.mT) * gam) @ u)
    return {"o": _back(o, idx, s["v"]), "S_final": last}


def _plain_bwd(s):
    c = s["c"]
    idx, q, k, v, beta, G, gam, kk, inv = _delta_common(s)
    S, u, last = _walk(s, q, k, v, beta, G, inv)
    do = s["scale"] * _rows(s["d_o"], idx)
    eG, end = torch.exp(G)[..., None], G[..., -1:]
    P = (q @ k.mT) * gam
    kend, qin, kin = torch.exp(end - G)[..., None] * k, (eG * q).mT.contiguous(), (beta[..., None] * eG * k).mT.contiguous()
    du0, invT = P.mT @ do, inv.mT.contiguous()
    dS = s["dS"].clone() if s["dS"] is not None else torch.zeros_like(last)
    dSs, lams = [], []
    for j in reversed(range(v.shape[2])):  # the recurrence of the state's gradient
        dSs.append(dS)
        lam = invT[:, :, j] @ (du0[:, :, j] + kend[:, :, j] @ dS)
        lams.append(lam)
        dS = torch.exp(end[:, :, j])[..., None] * dS + qin[:, :, j] @ do[:, :, j] - kin[:, :, j] @ lam
    dSn, lam = torch.stack(dSs[::-1], 2), torch.stack(lams[::-1], 2)
    dP, dA = (do @ u.mT).tril(), -(lam @ u.mT).tril(-1)
    M = dP * P + dA * (beta[..., None] * gam * kk)
    x1, x2, x3 = do @ S.mT, lam @ S.mT, u @ dSn.mT
    Dg, Eg = dP * gam, dA * gam
    b1 = beta[..., None]
    dq = eG * x1 + Dg @ k
    src = torch.exp(end - G)[..., None] * x3
    dk = src + Dg.mT @ q - b1 * eG * x2 + b1 * (Eg @ k) + Eg.mT @ (b1 * k)
    kx2 = eG[..., 0] * (k * x2).sum(-1)
    dbeta = (lam * v).sum(-1) - kx2 + (Eg * kk).sum(-1)
    ksrc = (k * src).sum(-1)
    dG = eG[..., 0] * (q * x1).sum(-1) - beta * kx2 + M.sum(-1) - M.sum(-2) - ksrc
    tail = ksrc.sum(-1) + torch.exp(end[..., 0]) * (S * dSn).sum((-1, -2))
    dg = dG.double().flip(-1).cumsum(-1).flip(-1).float() + tail[..., None]
    rep = c["HV"] // c["H"]
    dq, dk = (x.reshape(x.shape[0], c["H"], rep, *x.shape[2:]).sum(2) for x in (dq, dk))
    out = {"dq": _back(dq, idx, s["q"]), "dk": _back(dk, idx, s["k"]), "dv": _back(b1 * lam, idx, s["v"]),
           "dbeta": _back(dbeta, idx, s["beta"]), "dg": _back(dg, idx, s["g"])}
    if c["state"]:
        out["dS0"] = dS
    return out


def _plain_step(s):
    c = s["c"]
    rep = c["HV"] // c["H"]
    q, k = (s[n].float().repeat_interleave(rep, 1) for n in ("q", "k"))
    at = s["slots"].long()
    gate = torch.exp(s["g"])
    S = (gate[..., None, None] if c["gate"] == "head" else gate[..., None]) * s["state"][at]
    r = s["v"].float() - (k[..., None] * S).sum(-2)
    S = S + (s["beta"][..., None] * k)[..., None] * r[..., None, :]
    s["state"][at] = S
    o = s["scale"] * (q[..., None] * S).sum(-2)
    return {"o": o.to(s["v"].dtype), "state": s["state"]}


def _norm_stats(s, x):
    mean = x.mean(-1)
    d = x - mean[..., None]
    return d, mean, ((d * d).mean(-1) + EPS).rsqrt()


def _plain_norm_fwd(s):
    d, mean, rstd = _norm_stats(s, s["x"].float())
    y = d * rstd[..., None]
    if s["w"] is not None:
        y = y * s["w"] + s["b"]
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _norm_grads(s, x, mean, rstd):
    dy = s["dy"].float()
    h = (x - mean[..., None]) * rstd[..., None]
    t = dy * s["w"] if s["w"] is not None else dy
    dx = rstd[..., None] * (t - t.mean(-1, keepdim=True) - h * (t * h).mean(-1, keepdim=True))
    out = {"dx": dx.to(s["dy"].dtype)}
    if s["w"] is not None:
        out["dweight"], out["dbias"] = (dy * h).sum(0), dy.sum(0)
    return out


def _plain_norm_bwd(s):
    return _norm_grads(s, s["x"].float(), s["mean"], s["rstd"])


def _kept8(x):
    """The values that the 8-bit form of x stands for (float32)."""
    D = x.shape[-1]
    n = -(-D // BLOCK)
    p = torch.nn.functional.pad(x, (0, n * BLOCK - D)).reshape(*x.shape[:-1], n, BLOCK)
    top = p.abs().amax(-1, keepdim=True)
    some = top >= 1e-36
    codes = torch.round(p * torch.where(some, 127.0 / top, 0.0))
    return (codes * torch.where(some, top / 127.0, 0.0)).reshape(*x.shape[:-1], n * BLOCK)[..., :D]


def _plain_norm_ckpt8(s):
    f = _plain_norm_fwd(s)
    return {**f, **_norm_grads(s, _kept8(s["x"].float()), f["mean"], f["rstd"])}


_PLAIN = {"fwd": _plain_fwd, "bwd": _plain_bwd, "step": _plain_step, "norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd,
          "norm_ckpt8": _plain_norm_ckpt8}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _exact_delta(s):
    """Token by token, the forward and the adjoint of each token's update."""
    c = s["c"]
    rep = c["HV"] // c["H"]
    lens = _lengths(c) if c["packed"] else [c["T"]] * c["b"]
    starts = [sum(lens[:i]) for i in range(c["b"])] if c["packed"] else [i * c["T"] for i in range(c["b"])]
    tok = {n: s[n].reshape(-1, *s[n].shape[2:]).double() for n in ("q", "k", "v", "beta", "g", "d_o") if n in s}
    order = sorted(range(c["b"]), key=lambda i: -lens[i])  # longest first: the live sequences are a prefix
    dev = s["q"].device
    S = (s["S0"].double() if s["S0"] is not None else torch.zeros(c["b"], c["HV"], c["K"], c["V"], dtype=torch.float64, device=dev))[order].clone()
    top = max(lens)
    first = torch.tensor([starts[i] for i in order], device=dev)
    live = [sum(1 for i in order if lens[i] > t) for t in range(top)]

    def token(t, m):
        r = first[:m] + t
        q, k = (tok[n][r].repeat_interleave(rep, 1) for n in ("q", "k"))
        return r, q, k, tok["v"][r], tok["beta"][r][..., None], torch.exp(tok["g"][r])[..., None, None]

    def forward(t, S):
        m = live[t]
        r, q, k, v, beta, a = token(t, m)
        dec = a * S[:m]
        res = v - (k[..., None] * dec).sum(-2)
        return m, r, q, k, beta, a, dec, res, dec + (beta * k)[..., None] * res[..., None, :]

    out_o = torch.zeros_like(tok["v"])
    seg, kept = 64, []
    for t in range(top):
        if t % seg == 0:
            kept.append(S.clone())
        m, r, q, k, beta, a, dec, res, new = forward(t, S)
        S[:m] = new
        if c["op"] == "fwd":
            out_o[r] = s["scale"] * (q[..., None] * new).sum(-2)
    inverse = torch.tensor(sorted(range(c["b"]), key=lambda i: order[i]), device=dev)
    if c["op"] == "fwd":
        return {"o": out_o.reshape(s["v"].shape), "S_final": S[inverse]}
    g = {n: torch.zeros_like(tok[n]) for n in ("q", "k", "v", "beta", "g")}
    dS = (s["dS"].double() if s["dS"] is not None else torch.zeros_like(S))[order].clone()
    for j in reversed(range(len(kept))):
        S = kept[j]
        steps = []
        for t in range(j * seg, min(top, (j + 1) * seg)):
            got = forward(t, S)
            S[: got[0]] = got[8]
            steps.append(got)
        for m, r, q, k, beta, a, dec, res, new in reversed(steps):
            do = s["scale"] * tok["d_o"][r]
            group = lambda x: x.reshape(m, c["H"], rep, -1).sum(2)  # noqa: E731
            g["q"][r] = s["scale"] * group((new * tok["d_o"][r][..., None, :]).sum(-1))
            d = dS[:m] + q[..., None] * do[..., None, :]
            dw = (d * res[..., None, :]).sum(-1)  # of beta k
            dres = ((beta * k)[..., None] * d).sum(-2)
            g["beta"][r] = (dw * k).sum(-1)
            g["v"][r] = dres
            g["k"][r] = group(beta * dw - (dec * dres[..., None, :]).sum(-1))
            ddec = d - k[..., None] * dres[..., None, :]
            g["g"][r] = (ddec * dec).sum((-1, -2))
            dS[:m] = a * ddec
    out = {"d" + n: x.reshape(s[n].shape) for n, x in g.items()}
    if c["state"]:
        out["dS0"] = dS[inverse]
    return out


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] in ("fwd", "bwd"):
        return _exact_delta(s)
    if c["op"] == "step":
        rep = c["HV"] // c["H"]
        state = s["state"].double()
        o = torch.empty(s["v"].shape, dtype=torch.float64, device=state.device)
        for i, slot in enumerate(s["slots"].tolist()):
            q, k = s["q"][i].double().repeat_interleave(rep, 0), s["k"][i].double().repeat_interleave(rep, 0)
            gate = torch.exp(s["g"][i].double()).reshape(c["HV"], -1, 1)
            dec = gate * state[slot]
            res = s["v"][i].double() - torch.einsum("hk,hkv->hv", k, dec)
            state[slot] = dec + torch.einsum("hk,hv->hkv", k * s["beta"][i].double()[:, None], res)
            o[i] = s["scale"] * torch.einsum("hk,hkv->hv", q, state[slot])
        return {"o": o, "state": state}
    x = s["x"].double()
    if c["op"] == "norm_bwd":  # from the statistics as they were kept
        mean, rstd = s["mean"].double()[..., None], s["rstd"].double()[..., None]
    else:
        mean = x.mean(-1, keepdim=True)
        rstd = 1.0 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + EPS)
    w = s["w"].double() if s["w"] is not None else torch.ones((), dtype=torch.float64, device=x.device)
    out = {}
    if c["op"] != "norm_bwd":
        y = (x - mean) * rstd * w
        out = {"y": y + s["b"].double() if s["b"] is not None else y, "mean": mean[..., 0], "rstd": rstd[..., 0]}
    if c["op"] == "norm_fwd":
        return out
    if c["op"] == "norm_ckpt8":  # the codes are defined in float32: the only values here that are not in 64 bits
        kept = []
        for block in s["x"].float().split(BLOCK, -1):
            top = block.abs().max(-1, keepdim=True).values
            scale = torch.where(top < 1e-36, 0.0, top / 127.0)
            code = torch.round(block * torch.where(top < 1e-36, 0.0, 127.0 / top))
            kept.append(code.double() * scale.double())
        x = torch.cat(kept, -1)
    dy = s["dy"].double()
    h = (x - mean) * rstd
    D = x.shape[-1]
    t = dy * w
    out["dx"] = rstd * (t - t.sum(-1, keepdim=True) / D - h * ((t * h).sum(-1, keepdim=True) / D))
    if s["w"] is not None:
        out["dweight"], out["dbias"] = (dy * h).sum(0), dy.sum(0)
    return out
