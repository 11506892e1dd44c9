"""The measured cases of the linear recurrence, the gated feed-forward projections and dropout.

Operators, all of ``selective_state_space_vjp_amd.binding``; together they are one residual layer of a recurrent
model (mixer, feed-forward, dropout on both branches):

* ``linear_scan_fwd``   a recurrence with one state value per channel, over whole sequences
* ``linear_scan_bwd``   its gradients
* ``linear_scan_step``  one token per request on a pool of states, in place
* ``gated_ffn_fwd``     both projections of a gated feed-forward block, the activation and the product
* ``gated_ffn_bwd``     its gradients, from the projections the forward kept or by forming them again
* ``dropout_fwd``       dropout from a counter-based generator, added to a residual
* ``dropout_bwd``       its gradient, the mask drawn again

Recurrence, per channel, with h_{-1} = h0 (or zeros):
    log form:    h_t = exp(g_t) h_{t-1} + x_t
    gated form:  L_t = c softplus(decay) sigmoid(r_t);  a_t = exp(-L_t);
                 h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t
The forward can keep the state before every 64th token of a sequence (``ckpt``): sequence s of equal ones owns row s of
[b, ceil(T/64), D]; of packed ones the rows start/64 + s + j of [T/64 + b, D], start being its first token; rows
that no token has are zeros.
Feed-forward: gate = x Wg^T, up = x Wu^T, h = act(gate) up; act is silu or gelu in its tanh form.
Dropout: the Philox 4x32-10 generator (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
2011), key = the seed's low and high 32 bits, counter = (low, high of e // 8, low, high of the offset) for element e
of the flattened tensor, which takes 16-bit half e % 8 of the four words, low halves first.  It is kept where that draw
is at least t = rint(65536 p), and multiplied by 65536 / (65536 - t).
"""
import math
import random

import torch

own = False
CHUNK = 64  # tokens per kept state
C = 8.0     # c of the gated form


# ------------------------------------------------------------------------------------------------ cases
def listed():
    bf = "bfloat16"
    return [
        # the forward half of a training step of one mixer layer, its states kept for the backward
        dict(name="scan fwd layer", op="scan_fwd", form="gated", b=2, T=4096, D=4096, packed=False, state=False, ckpt=True, dtype=bf),
        # long prompts of different lengths packed behind one another, continued from kept states
        dict(name="scan fwd packed", op="scan_fwd", form="log", b=5, T=32771, D=2560, packed=True, state=True, ckpt=False, dtype=bf),
        # the backward half of a training step
        dict(name="scan bwd layer", op="scan_bwd", form="gated", b=2, T=4096, D=4096, packed=False, state=False, ckpt=True, dtype=bf),
        # packed documents of a small model with an odd width in float32, truncated at kept states, nothing kept by the forward
        dict(name="scan bwd odd", op="scan_bwd", form="log", b=7, T=3001, D=1001, packed=True, state=True, ckpt=False, dtype="float32"),
        # one request's next token: launch and latency
        dict(name="scan step 1", op="scan_step", form="gated", b=1, slots=4, D=4096, dtype=bf),
        # a full serving batch
        dict(name="scan step 256", op="scan_step", form="gated", b=256, slots=300, D=4096, dtype=bf),
        # the feed-forward half of a layer in training, its projections kept
        dict(name="ffn fwd layer", op="ffn_fwd", M=8192, D=4096, F=12288, act="silu", saved=True, dtype=bf),
        # the tokens of one decode step of a few requests: the weights' traffic
        dict(name="ffn fwd few", op="ffn_fwd", M=5, D=4096, F=12288, act="silu", saved=False, dtype=bf),
        # its backward in training
        dict(name="ffn bwd layer", op="ffn_bwd", M=8192, D=4096, F=12288, act="silu", saved=True, dtype=bf),
        # odd sizes of a small model, the projections formed again
        dict(name="ffn bwd odd", op="ffn_bwd", M=777, D=1000, F=2712, act="gelu", saved=False, dtype=bf),
        # a residual branch in training
        dict(name="dropout fwd layer", op="drop_fwd", rows=8192, D=4096, p=0.1, residual=True, dtype=bf),
        # a short batch of odd width, its gradient
        dict(name="dropout bwd few", op="drop_bwd", rows=9, D=1001, p=0.25, residual=False, dtype="float32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "scan_step", "ffn_fwd", "ffn_fwd", "ffn_bwd", "ffn_bwd", "drop_fwd", "drop_bwd"])
    dtype = rng.choice(["bfloat16", "bfloat16", "bfloat16", "float32"])
    if op in ("scan_fwd", "scan_bwd"):
        packed = rng.random() < 0.5
        T, D = _log(rng, 1, 65536), _log(rng, 1, 8192)
        b = rng.randint(1, 24) if packed else rng.randint(1, 8)
        most = 2 * 4096 * 4096 // D
        if T * (1 if packed else b) > most:
            T = max(1, most if packed else most // b)
        return dict(op=op, form=rng.choice(["gated", "log"]), b=b, T=T, D=D, packed=packed, state=rng.random() < 0.5, ckpt=rng.random() < 0.5, dtype=dtype)
    if op == "scan_step":
        b = _log(rng, 1, 256)
        return dict(op=op, form=rng.choice(["gated", "log"]), b=b, slots=b + rng.randint(0, 40), D=_log(rng, 1, 8192), dtype=dtype)
    if op in ("ffn_fwd", "ffn_bwd"):
        M, D, F = _log(rng, 1, 8192), 8 * _log(rng, 1, 640), 8 * _log(rng, 1, 1536)
        if dtype == "float32":  # a smaller model
            M, D, F = max(1, M // 4), 8 * max(1, D // 16), 8 * max(1, F // 16)
        return dict(op=op, M=M, D=D, F=F, act=rng.choice(["silu", "gelu"]), saved=rng.random() < 0.5, dtype=dtype)
    D = _log(rng, 1, 8192)
    rows = _log(rng, 1, max(1, 8192 * 4096 // D))
    return dict(op=op, rows=rows, D=D, p=round(rng.choice([0.0, 0.05, 0.1, rng.random(), 0.5]), 4), residual=op == "drop_fwd" and rng.random() < 0.6, dtype=dtype)


def _lengths(c):
    """Lengths of a case's sequences; packed ones are uneven, one of them empty where there are three or more."""
    if not c["packed"]:
        return [c["T"]] * c["b"]
    rng = random.Random(c["T"] * 131 + c["b"])
    cuts = sorted(rng.randint(0, c["T"]) for _ in range(c["b"] - 1))
    if len(cuts) >= 2:
        cuts[1] = cuts[0]
    edges = [0] + cuts + [c["T"]]
    return [y - x for x, y in zip(edges, edges[1:])]


def _ckpt_rows(c):
    return c["T"] // CHUNK + c["b"] if c["packed"] else c["b"] * -(-c["T"] // CHUNK)


def work(c):
    e = 2 if c["dtype"] == "bfloat16" else 4
    gated = c.get("form") == "gated"
    if c["op"] in ("scan_fwd", "scan_bwd"):
        n, st = (c["T"] if c["packed"] else c["b"] * c["T"]) * c["D"], 4 * c["b"] * c["D"]
        kept = 4 * _ckpt_rows(c) * c["D"] if c["ckpt"] else 0
        ins = (3 * e if gated else e + 4) * n + (4 * c["D"] if gated else 0)
        if c["op"] == "scan_fwd":
            return {"bytes": ins + e * n + kept + st * (2 if c["state"] else 1), "flops": (24 if gated else 3) * n}
        outs = (3 * e if gated else e + 4) * n + (4 * c["D"] if gated else 0)
        return {"bytes": ins + e * n + outs + kept + st * (3 if c["state"] else 0), "flops": (48 if gated else 7) * n}
    if c["op"] == "scan_step":
        n = c["b"] * c["D"]
        return {"bytes": (4 * e if gated else 2 * e + 4) * n + 8 * n + 4 * c["b"] + (4 * c["D"] if gated else 0), "flops": (24 if gated else 3) * n}
    if c["op"] in ("ffn_fwd", "ffn_bwd"):
        x, h, w = c["M"] * c["D"], c["M"] * c["F"], 2 * c["D"] * c["F"]
        if c["op"] == "ffn_fwd":
            return {"bytes": e * (x + w + h * (3 if c["saved"] else 1)), "flops": 2 * c["M"] * w}
        return {"bytes": e * (2 * x + 2 * w + h * (3 if c["saved"] else 1)), "flops": (4 if c["saved"] else 6) * c["M"] * w}
    n = c["rows"] * c["D"]
    return {"bytes": e * n * (3 if c["residual"] else 2) + 16, "flops": 2 * n}


# ------------------------------------------------------------------------------------------------ inputs
def prepare(c, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = getattr(torch, c["dtype"])

    def rn(*shape):
        return torch.randn(shape, device=dev, generator=gen)

    s = dict(c=c)
    D = c["D"]
    if c["op"] in ("scan_fwd", "scan_bwd", "scan_step"):
        lead = (c["b"],) if c["op"] == "scan_step" else (1 if c["packed"] else c["b"], c["T"])
        s["x"] = rn(*lead, D).to(dt)
        if c["form"] == "gated":
            s["gate"], s["input_gate"] = rn(*lead, D).to(dt), rn(*lead, D).to(dt)
            # exp(-c softplus(decay)) from 0.9 to 0.999 over the channels
            soft = -torch.log(torch.linspace(0.9, 0.999, D, device=dev)) / C
            s["decay"] = torch.log(torch.expm1(soft))
        else:
            # channels that forget within a few tokens beside channels that keep thousands, and a reset now and then
            rate = torch.exp(torch.linspace(math.log(0.001), math.log(1.0), D, device=dev))
            s["gate"] = -rate * torch.nn.functional.softplus(rn(*lead, D))
            s["gate"][torch.rand(lead, device=dev, generator=gen) < 0.0005] = -math.inf
            s["input_gate"] = s["decay"] = None
        if c["op"] == "scan_step":
            s["state"] = rn(c["slots"], D)
            s["slots"] = torch.randperm(c["slots"], device=dev, generator=gen)[: c["b"]].to(torch.int32)
            return s
        s["h0"] = rn(c["b"], D) if c["state"] else None
        s["offsets"] = None
        if c["packed"]:
            edges = [0]
            for length in _lengths(c):
                edges.append(edges[-1] + length)
            s["offsets"] = torch.tensor(edges, dtype=torch.int32, device=dev)
        if c["op"] == "scan_bwd":
            s["dh"] = rn(*lead, D).to(dt)
            s["dh_final"] = rn(c["b"], D) if c["state"] else None
            s["ckpt"] = None
            if c["ckpt"]:  # what the forward pass left
                a, u, _ = _gates(s)
                s["ckpt"] = _kept(s, _states(s, a, u))
    elif c["op"] in ("ffn_fwd", "ffn_bwd"):
        s["x"] = rn(c["M"], D).to(dt)
        s["w_gate"], s["w_up"] = ((rn(c["F"], D) * D ** -0.5).to(dt) for _ in range(2))
        if c["op"] == "ffn_bwd":
            s["dh"] = rn(c["M"], c["F"]).to(dt)
            s["saved"] = None
            if c["saved"]:  # what the forward pass left
                s["saved"] = tuple((s["x"].float() @ s[n].float().T).to(dt) for n in ("w_gate", "w_up"))
    else:
        s["x"] = rn(c["rows"], D).to(dt)
        s["residual"] = rn(c["rows"], D).to(dt) if c["residual"] else None
        s["rng"] = torch.tensor([seed * 0x9E3779B97F4A7C15 % 2 ** 63, seed * 1000003 + (5 << 32)], dtype=torch.int64, device=dev)
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    if not own:
        return _PLAIN[s["c"]["op"]](s)
    from selective_state_space_vjp_amd import binding as bd

    c = s["c"]
    op = c["op"]
    if op == "scan_fwd":
        out = bd.linear_scan_fwd(s["x"], s["gate"], s["h0"], input_gate=s["input_gate"], decay=s["decay"], c=C, seq_offsets=s["offsets"], want_ckpt=c["ckpt"])
    elif op == "scan_bwd":
        out = bd.linear_scan_bwd(s["x"], s["gate"], s["dh"], s["h0"], s["dh_final"], input_gate=s["input_gate"], decay=s["decay"], c=C, ckpt=s["ckpt"],
                                 seq_offsets=s["offsets"], want_dh0=c["state"])
    elif op == "scan_step":
        h = bd.linear_scan_step(s["x"], s["gate"], s["state"], input_gate=s["input_gate"], decay=s["decay"], c=C, slots=s["slots"])
        out = {"h": h, "state": s["state"]}
    elif op == "ffn_fwd":
        out = bd.gated_ffn_fwd(s["x"], s["w_gate"], s["w_up"], act=c["act"], want_saved=c["saved"])
    elif op == "ffn_bwd":
        out = bd.gated_ffn_bwd(s["dh"], s["x"], s["w_gate"], s["w_up"], act=c["act"], saved=s["saved"])
    elif op == "drop_fwd":
        out = {"y": bd.dropout_fwd(s["x"], s["rng"], s["residual"], p=c["p"])}
    else:
        out = {"dx": bd.dropout_bwd(s["x"], s["rng"], p=c["p"])}
    return {k: x for k, x in out.items() if x is not None}


# ------------------------------------------------------------------------------------------------ plain forms
def _edges(c):
    """Rows of the flattened token axis that begin and end each sequence that has tokens, and which sequences those are."""
    begin, end, seq, at = [], [], [], 0
    for i, n in enumerate(_lengths(c)):
        if n:
            begin.append(at)
            end.append(at + n - 1)
            seq.append(i)
        at += n
    return begin, end, seq


def _flat(x):
    return x.reshape(-1, x.shape[-1]).float()


def _gates(s):
    """a_t and what h_t adds to a_t h_{t-1}, and the parts that the gradients need."""
    x, gate = _flat(s["x"]), _flat(s["gate"])
    if s["decay"] is None:
        return torch.exp(gate), x, None
    soft = torch.log1p(torch.exp(s["decay"]))
    sr, si = 1 / (1 + torch.exp(-gate)), 1 / (1 + torch.exp(-_flat(s["input_gate"])))
    L = C * soft * sr
    m = torch.sqrt(-torch.expm1(-2 * L))
    return torch.exp(-L), m * si * x, (x, soft, sr, si, L, m)


def _solve(a, u):
    """y_t = a_t y_{t-1} + u_t along the first axis, y_{-1} = 0: by doubling."""
    n = 1
    while n < u.shape[0]:
        u = torch.cat([u[:n], u[n:] + a[n:] * u[:-n]])
        a = torch.cat([a[:n], a[n:] * a[:-n]])
        n *= 2
    return u


def _states(s, a, u):
    """h of every token, flat."""
    begin, _, seq = _edges(s["c"])
    if not begin:
        return u
    a, u = a.clone(), u.clone()
    if s["h0"] is not None:
        u[begin] += a[begin] * s["h0"][seq]
    a[begin] = 0
    return _solve(a, u)


def _before(s, h):
    """h_{t-1} of every token."""
    begin, _, seq = _edges(s["c"])
    prev = torch.zeros_like(h)
    prev[1:] = h[:-1]
    if begin:
        prev[begin] = s["h0"][seq] if s["h0"] is not None else 0.0
    return prev


def _kept(s, h):
    """The state before every 64th token of each sequence, in the layout of ckpt."""
    c = s["c"]
    rows, tokens, at = [], [], 0
    for i, n in enumerate(_lengths(c)):
        for j in range(-(-n // CHUNK)):
            rows.append(at // CHUNK + i + j if c["packed"] else i * -(-c["T"] // CHUNK) + j)
            tokens.append(at + CHUNK * j)
        at += n
    out = torch.zeros(_ckpt_rows(c), c["D"], dtype=h.dtype, device=h.device)
    if rows:
        dev = h.device
        out[torch.tensor(rows, device=dev)] = _before(s, h)[torch.tensor(tokens, device=dev)]
    return out if c["packed"] else out.reshape(c["b"], -1, c["D"])


def _plain_scan_fwd(s):
    c = s["c"]
    a, u, _ = _gates(s)
    h = _states(s, a, u)
    begin, end, seq = _edges(c)
    last = s["h0"].clone() if s["h0"] is not None else torch.zeros(c["b"], c["D"], device=h.device)
    last[seq] = h[end]
    out = {"h": h.to(s["x"].dtype).reshape(s["x"].shape), "h_final": last}
    if c["ckpt"]:
        out["ckpt"] = _kept(s, h)
    return out


def _plain_scan_bwd(s):
    c = s["c"]
    a, u, parts = _gates(s)
    prev = _before(s, _states(s, a, u))
    begin, end, seq = _edges(c)
    lam = _flat(s["dh"]).clone()
    if s["dh_final"] is not None:
        lam[end] += s["dh_final"][seq]
    nxt = torch.zeros_like(a)
    nxt[:-1] = a[1:]
    nxt[end] = 0
    lam = _solve(nxt.flip(0), lam.flip(0)).flip(0)
    shape, dt = s["x"].shape, s["x"].dtype
    if parts is None:
        out = {"dx": lam.to(dt).reshape(shape), "dgate": (lam * a * prev).reshape(shape)}
    else:
        x, soft, sr, si, L, m = parts
        E = lam * (si * x * a * a * (L / m) - L * a * prev)
        out = {"dx": (lam * m * si).to(dt).reshape(shape), "dgate": (E * (1 - sr)).to(dt).reshape(shape),
               "dinput_gate": (lam * m * x * si * (1 - si)).to(dt).reshape(shape),
               "ddecay": E.double().sum(0).float() / (soft * (1 + torch.exp(-s["decay"])))}
    if c["state"]:
        dh0 = s["dh_final"].clone()
        dh0[seq] = a[begin] * lam[begin]
        out["dh0"] = dh0
    return out


def _plain_scan_step(s):
    a, u, _ = _gates(s)
    at = s["slots"].long()
    h = a * s["state"][at] + u
    s["state"][at] = h
    return {"h": h.to(s["x"].dtype), "state": s["state"]}


def _act(name, z):
    """The activation and its derivative."""
    if name == "silu":
        g = 1 / (1 + torch.exp(-z))
        return z * g, g * (1 + z * (1 - g))
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)


def _plain_ffn_fwd(s):
    x = s["x"].float()
    gate, up = x @ s["w_gate"].float().T, x @ s["w_up"].float().T
    dt = s["x"].dtype
    out = {"h": (_act(s["c"]["act"], gate)[0] * up).to(dt)}
    if s["c"]["saved"]:
        out["gate"], out["up"] = gate.to(dt), up.to(dt)
    return out


def _plain_ffn_bwd(s):
    x, wg, wu, dh = (s[n].float() for n in ("x", "w_gate", "w_up", "dh"))
    gate, up = (t.float() for t in s["saved"]) if s["saved"] else (x @ wg.T, x @ wu.T)
    f, df = _act(s["c"]["act"], gate)
    dgate, dup = dh * up * df, dh * f
    dt = s["x"].dtype
    return {"dx": (dgate @ wg + dup @ wu).to(dt), "dw_gate": (dgate.T @ x).to(dt), "dw_up": (dup.T @ x).to(dt)}


def _keep(rng, n, t):
    """Which of n elements are kept, in 64-bit integers: a product of two 32-bit words wraps, its high word is masked out of the shift."""
    low = 0xFFFFFFFF
    j = torch.arange((n + 7) // 8, device=rng.device)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    c0, c1 = j & low, j >> 32
    c2, c3 = (rng[1] & low).expand_as(j), ((rng[1] >> 32) & low).expand_as(j)
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & low) ^ c1 ^ k0, p1 & low, ((p0 >> 32) & low) ^ c3 ^ k1, p0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    draws = torch.stack([h for w in (c0, c1, c2, c3) for h in (w & 0xFFFF, w >> 16)], -1)
    return draws.reshape(-1)[:n] >= t


def _plain_drop(s):
    x = s["x"]
    t = int(round(65536 * s["c"]["p"]))
    y = torch.where(_keep(s["rng"], x.numel(), t).reshape(x.shape), x.float() * (65536 / (65536 - t) if t < 65536 else 0.0), 0.0)
    if s["residual"] is not None:
        y = s["residual"].float() + y
    return {("y" if s["c"]["op"] == "drop_fwd" else "dx"): y.to(x.dtype)}


_PLAIN = {"scan_fwd": _plain_scan_fwd, "scan_bwd": _plain_scan_bwd, "scan_step": _plain_scan_step, "ffn_fwd": _plain_ffn_fwd,
          "ffn_bwd": _plain_ffn_bwd, "drop_fwd": _plain_drop, "drop_bwd": _plain_drop}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _exact_coefficients(s):
    """Per token: log a, the factor of x, and sigmoid(r), sigmoid(i) in the gated form."""
    x, gate = s["x"].double(), s["gate"].double()
    if s["decay"] is None:
        return gate, torch.ones_like(x), None, None
    r, i = torch.sigmoid(gate), torch.sigmoid(s["input_gate"].double())
    la = -C * torch.logaddexp(s["decay"].double(), torch.zeros((), dtype=torch.float64, device=x.device)) * r
    return la, (1 - torch.exp(2 * la)).sqrt(), r, i


def _exact_scan(s):
    """Token by token over the time axis; packed sequences one behind the other in it."""
    c = s["c"]
    la, m, r, i = _exact_coefficients(s)
    a, x = torch.exp(la), s["x"].double()
    add = x * m if i is None else x * m * i
    n, T, D = x.shape
    lens = _lengths(c)
    zero = torch.zeros(c["b"], D, dtype=torch.float64, device=x.device)
    h0 = zero if s["h0"] is None else s["h0"].double()
    starts, ends = {}, {}
    at = 0
    if c["packed"]:
        for q, length in enumerate(lens):
            if length:
                starts[at], ends[at + length - 1] = [q], [q]
            at += length
    else:
        starts[0] = ends[T - 1] = list(range(n))
    h = torch.empty_like(x)
    last = h0.clone()
    cur = h0[:n].clone()
    for t in range(T):
        if t in starts:
            cur = h0[starts[t]]
        cur = a[:, t] * cur + add[:, t]
        h[:, t] = cur
        if t in ends:
            last[ends[t]] = cur
    if c["op"] == "scan_fwd":
        out = {"h": h, "h_final": last}
        if c["ckpt"]:
            rows = torch.zeros(_ckpt_rows(c), D, dtype=torch.float64, device=x.device)
            at = 0
            for q, length in enumerate(lens):
                for j in range(0, length, CHUNK):
                    if c["packed"]:
                        rows[at // CHUNK + q + j // CHUNK] = h[0, at + j - 1] if j else h0[q]
                    else:
                        rows[q * -(-T // CHUNK) + j // CHUNK] = h[q, j - 1] if j else h0[q]
                at += length
            out["ckpt"] = rows if c["packed"] else rows.reshape(n, -1, D)
        return out
    prev = torch.empty_like(h)
    prev[:, 1:] = h[:, :-1]
    for t, which in starts.items():
        prev[:, t] = h0[which]
    dlast = zero if s["dh_final"] is None else s["dh_final"].double()
    dh, lam = s["dh"].double(), torch.empty_like(x)
    dh0 = dlast.clone()
    cur = torch.zeros_like(cur)
    for t in reversed(range(T)):
        if t in ends:
            cur = dlast[ends[t]]
        lam[:, t] = cur + dh[:, t]
        cur = a[:, t] * lam[:, t]
        if t in starts:
            dh0[starts[t]] = cur
    dla = lam * a * prev
    out = {"dx": lam * m if i is None else lam * m * i}
    if i is None:
        out["dgate"] = dla
    else:
        # d sqrt(1 - a^2) / d log a = -a^2 / sqrt(1 - a^2)
        dla = dla - lam * i * x * a * a / m
        out["dgate"] = dla * la * (1 - r)
        out["dinput_gate"] = lam * m * x * i * (1 - i)
        slope = torch.sigmoid(s["decay"].double())
        out["ddecay"] = (dla * -C * r).sum((0, 1)) * slope
    if c["state"]:
        out["dh0"] = dh0
    return out


def _exact_keep(rng, n, t):
    """The generator word by word in Python's unbounded integers, on object arrays of numpy's 64-bit unsigned halves."""
    import numpy as np

    seed, offset = (int(v) % 2 ** 64 for v in rng.tolist())
    u, sh, lo = np.uint64, np.uint64(32), np.uint64(0xFFFFFFFF)
    blocks = np.arange((n + 7) // 8, dtype=u)
    word = [blocks & lo, blocks >> sh, np.full_like(blocks, offset & 0xFFFFFFFF), np.full_like(blocks, offset >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        first, second = word[0] * u(0xD2511F53), word[2] * u(0xCD9E8D57)
        word = [(second >> sh) ^ word[1] ^ u(key[0]), second & lo, (first >> sh) ^ word[3] ^ u(key[1]), first & lo]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    draws = np.empty((blocks.size, 8), dtype=np.int64)
    for k in range(4):
        draws[:, 2 * k] = (word[k] & u(0xFFFF)).astype(np.int64)
        draws[:, 2 * k + 1] = (word[k] >> u(16)).astype(np.int64)
    return torch.from_numpy(draws.reshape(-1)[:n] >= t)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] in ("scan_fwd", "scan_bwd"):
        return _exact_scan(s)
    if c["op"] == "scan_step":
        la, m, _, i = _exact_coefficients(s)
        state = s["state"].double()
        h = torch.empty_like(la)
        for q, slot in enumerate(s["slots"].tolist()):
            h[q] = torch.exp(la[q]) * state[slot] + m[q] * (1 if i is None else i[q]) * s["x"][q].double()
            state[slot] = h[q]
        return {"h": h, "state": state}
    if c["op"] in ("ffn_fwd", "ffn_bwd"):
        x, wg, wu = (s[n].double() for n in ("x", "w_gate", "w_up"))
        kept = s.get("saved")
        gate, up = (t.double() for t in kept) if kept else (torch.mm(x, wg.T), torch.mm(x, wu.T))
        if c["act"] == "silu":
            sg = torch.sigmoid(gate)
            f, df = gate * sg, sg + gate * sg * (1 - sg)
        else:
            # tanh(z) = 2 sigmoid(2 z) - 1, so 0.5 (1 + tanh(z)) = sigmoid(2 z)
            z = 2 * math.sqrt(2 / math.pi) * (gate + 0.044715 * gate * gate * gate)
            sg = torch.sigmoid(z)
            f, df = gate * sg, sg + gate * sg * (1 - sg) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * gate * gate)
        if c["op"] == "ffn_fwd":
            return {"h": f * up, **({"gate": gate, "up": up} if c["saved"] else {})}
        dh = s["dh"].double()
        dgate, dup = df * up * dh, f * dh
        return {"dx": torch.mm(dgate, wg) + torch.mm(dup, wu), "dw_gate": torch.mm(dgate.T, x), "dw_up": torch.mm(dup.T, x)}
    t = round(65536 * c["p"])
    keep = _exact_keep(s["rng"], s["x"].numel(), t).reshape(s["x"].shape).to(s["x"].device)
    y = s["x"].double() * keep * (65536 / (65536 - t) if t < 65536 else 0.0)
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return {("y" if c["op"] == "drop_fwd" else "dx"): y}
