"""The linear recurrence, dropout, layer norm and the gated feed-forward projections together, as a residual layer runs
them: values and gradients against torch's differentiation of the same layer in float64 on the CPU, a captured training
step, and a prompt followed by single tokens."""
import pytest
import torch

from block_ref import BF, C, F32, U, UNIT, act, keep_mask
from gpu_common import announce
from selective_state_space_vjp_amd import binding as bd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D, F = 64, 160
P = 0.2
# relative to the norm: 12 stages of sums of at most 160 terms (160 u each in the worst case) and the recurrence's
# coefficients in both directions, each amplified at most four times by what follows (norms of rows of deviation near 1)
TOL = 4 * (12 * 160 * U + 2 * UNIT["gated"])


def weights(seed, dtype=F32):
    gen = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    w = {k: (rn(D, D) * D**-0.5).to(dtype) for k in ("wr", "wi", "wx", "wo")}
    w.update(decay=torch.linspace(-8.0, -4.0, D), g1=1 + 0.1 * rn(D), b1=0.1 * rn(D), g2=1 + 0.1 * rn(D), b2=0.1 * rn(D),
             wg=(rn(F, D) * D**-0.5).to(dtype), wu=(rn(F, D) * D**-0.5).to(dtype), wd=(rn(D, F) * F**-0.5).to(dtype))
    return w


def mm(x, w):
    return (x.reshape(-1, x.shape[-1]) @ w.T).view(*x.shape[:-1], w.shape[0])


def layer(x, w, rng, offsets=None, h0=None):
    """The forward pass and what its backward reads."""
    s = {"x": x}
    s["n1"] = bd.layer_norm_fwd(x, w["g1"], w["b1"])
    n = s["n1"]["y"]
    s["r"], s["i"], s["u"] = mm(n, w["wr"]), mm(n, w["wi"]), mm(n, w["wx"])
    s["scan"] = bd.linear_scan_fwd(s["u"], s["r"], h0, input_gate=s["i"], decay=w["decay"], c=C, seq_offsets=offsets, want_ckpt=True)
    s["x1"] = bd.dropout_fwd(mm(s["scan"]["h"], w["wo"]), rng[0], x, p=P)
    s["n2"] = bd.layer_norm_fwd(s["x1"], w["g2"], w["b2"])
    s["ffn"] = bd.gated_ffn_fwd(s["n2"]["y"], w["wg"], w["wu"], want_saved=True)
    return bd.dropout_fwd(mm(s["ffn"]["h"], w["wd"]), rng[1], s["x1"], p=P), s


def layer_bwd(dy, s, w, rng, offsets=None, h0=None):
    g = {}
    flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
    d = bd.dropout_bwd(dy, rng[1], p=P)
    g["wd"] = flat(d).T @ flat(s["ffn"]["h"])
    f = bd.gated_ffn_bwd(flat(d) @ w["wd"], flat(s["n2"]["y"]), w["wg"], w["wu"], saved=(flat(s["ffn"]["gate"]), flat(s["ffn"]["up"])))
    g["wg"], g["wu"] = f["dw_gate"], f["dw_up"]
    n = bd.layer_norm_bwd(f["dx"].view(dy.shape), s["x1"], s["n2"]["mean"], s["n2"]["rstd"], w["g2"])
    g["g2"], g["b2"] = n["dweight"], n["dbias"]
    dx1 = dy + n["dx"]
    d = bd.dropout_bwd(dx1, rng[0], p=P)
    g["wo"] = flat(d).T @ flat(s["scan"]["h"])
    dh = (flat(d) @ w["wo"]).view(dy.shape)
    b = bd.linear_scan_bwd(s["u"], s["r"], dh, h0, input_gate=s["i"], decay=w["decay"], c=C, ckpt=s["scan"]["ckpt"], seq_offsets=offsets,
                           want_dh0=h0 is not None)
    g["decay"], g["h0"] = b["ddecay"], b["dh0"]
    n1 = flat(s["n1"]["y"])
    g["wr"], g["wi"], g["wx"] = (flat(b[k]).T @ n1 for k in ("dgate", "dinput_gate", "dx"))
    dn = (flat(b["dgate"]) @ w["wr"] + flat(b["dinput_gate"]) @ w["wi"] + flat(b["dx"]) @ w["wx"]).view(dy.shape)
    n = bd.layer_norm_bwd(dn, s["x"], s["n1"]["mean"], s["n1"]["rstd"], w["g1"])
    g["g1"], g["b1"], g["x"] = n["dweight"], n["dbias"], dx1 + n["dx"]
    return g


def reference(x, w, masks, spans, h0):
    ln = lambda t, g, b: torch.nn.functional.layer_norm(t, (D,), g, b, 1e-5)  # noqa: E731
    n = ln(x, w["g1"], w["b1"])
    r, i, u = n @ w["wr"].T, n @ w["wi"].T, n @ w["wx"].T
    L = C * torch.nn.functional.softplus(w["decay"]) * torch.sigmoid(r)
    a, v = torch.exp(-L), torch.sqrt(-torch.expm1(-2 * L)) * torch.sigmoid(i) * u
    hs = []
    for k, (row, at, m) in enumerate(spans):
        h = h0[k] if h0 is not None else torch.zeros(D, dtype=torch.float64)
        for t in range(at, at + m):
            h = a[row, t] * h + v[row, t]
            hs.append(h)
    h = torch.stack(hs).view(x.shape)
    x1 = x + (h @ w["wo"].T) * masks[0]
    n = ln(x1, w["g2"], w["b2"])
    f = act("silu", n @ w["wg"].T) * (n @ w["wu"].T)
    return x1 + (f @ w["wd"].T) * masks[1]


@pytest.mark.parametrize("lens", [None, [70, 0, 3, 127]], ids=["equal", "packed"])
def test_layer_and_its_gradients(lens):
    announce(f"residual layer {lens}")
    n, T = (2, 140) if lens is None else (1, sum(lens))
    gen = torch.Generator().manual_seed(3)
    x, dy = torch.randn(n, T, D, generator=gen), torch.randn(n, T, D, generator=gen)
    w = weights(1)
    h0 = torch.randn(2 if lens is None else len(lens), D, generator=gen)
    seeds = ((7, 1), (7, 2))
    rng = [torch.tensor(s, dtype=torch.int64, device=DEV) for s in seeds]
    edges = None if lens is None else torch.tensor([sum(lens[:k]) for k in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
    W = {k: v.to(DEV) for k, v in w.items()}
    y, s = layer(x.to(DEV), W, rng, edges, h0.to(DEV))
    g = layer_bwd(dy.to(DEV), s, W, rng, edges, h0.to(DEV))
    leaf = {k: v.double().requires_grad_(True) for k, v in {**w, "x": x, "h0": h0}.items()}
    t = round(65536 * P)
    masks = [keep_mask(x.numel(), P, *q).view(x.shape).double() * (65536 / (65536 - t)) for q in seeds]
    spans = [(k, 0, T) for k in range(n)] if lens is None else [(0, sum(lens[:k]), lens[k]) for k in range(len(lens))]
    want = reference(leaf["x"], leaf, masks, spans, leaf["h0"])
    grads = dict(zip(leaf, torch.autograd.grad((want * dy.double()).sum(), list(leaf.values()))))
    for k, got, ref in [("y", y, want.detach())] + [(k, g[k], grads[k]) for k in grads]:
        err = float((got.double().cpu() - ref).norm() / ref.norm())
        print(f"{k}: {err:.1e} of {TOL:.1e}", flush=True)
        assert err <= TOL, (k, err)


def test_captured_training_step():
    """Forward and backward of the layer in one graph, replayed on other inputs with eager work between: every replay is
    the eager result, masks included."""
    announce("residual layer graph")
    W = {k: v.to(DEV) for k, v in weights(2, BF).items()}
    x, dy = torch.randn(2, 200, D, device=DEV).to(BF), torch.randn(2, 200, D, device=DEV).to(BF)
    rng = [torch.tensor([5, k], dtype=torch.int64, device=DEV) for k in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer_bwd(dy, layer(x, W, rng)[1], W, rng)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, s = layer(x, W, rng)
        g = layer_bwd(dy, s, W, rng)
    for turn in range(4):
        x.copy_(torch.randn(2, 200, D, device=DEV))
        rng[0][1] += 2
        graph.replay()
        torch.cuda.synchronize()
        ye, se = layer(x, W, rng)
        ge = layer_bwd(dy, se, W, rng)
        assert torch.equal(y, ye), turn
        for k in ge:
            if ge[k] is not None:
                assert torch.equal(g[k], ge[k]), (turn, k)


def test_prompt_then_tokens():
    """Serving: a packed batch of prompts, then tokens one by one with the states in a pool, is the layer over the whole
    sequences (no dropout), to the roundings of bf16 where the values pass through it."""
    announce("residual layer serving")
    W = {k: v.to(DEV) for k, v in weights(4).items()}
    lens, more = [5, 33, 70], 6
    gen = torch.Generator().manual_seed(5)
    seqs = [torch.randn(1, k + more, D, generator=gen).to(DEV) for k in lens]

    def mixer(n, state, slots=None, offsets=None):
        r, i, u = mm(n, W["wr"]), mm(n, W["wi"]), mm(n, W["wx"])
        if slots is not None:
            return bd.linear_scan_step(u, r, state, input_gate=i, decay=W["decay"], c=C, slots=slots)
        o = bd.linear_scan_fwd(u, r, input_gate=i, decay=W["decay"], c=C, seq_offsets=offsets)
        if state is not None:
            state[:] = o["h_final"]
        return o["h"]

    def block(x, *a, **kw):
        x1 = x + mm(mixer(bd.layer_norm_fwd(x, W["g1"], W["b1"])["y"], *a, **kw), W["wo"])
        n = bd.layer_norm_fwd(x1, W["g2"], W["b2"])["y"]
        return x1 + mm(bd.gated_ffn_fwd(n, W["wg"], W["wu"])["h"], W["wd"])

    want = [block(s, None)[0] for s in seqs]
    state = torch.zeros(3, D, device=DEV)
    edges = torch.tensor([0, 5, 38, 108], dtype=torch.int32, device=DEV)
    y = block(torch.cat([s[:, :k] for s, k in zip(seqs, lens)], 1), state, offsets=edges)[0]
    pool = torch.zeros(8, D, device=DEV)
    slots = torch.tensor([6, 1, 3], dtype=torch.int32, device=DEV)
    pool[slots.long()] = state
    at = 0
    for k, ref in zip(lens, want):
        assert float((y[at:at + k] - ref[:k]).norm() / ref[:k].norm()) <= TOL
        at += k
    for t in range(more):
        y = block(torch.cat([s[:, k + t] for s, k in zip(seqs, lens)]), pool, slots=slots)
        for q, (k, ref) in enumerate(zip(lens, want)):
            assert float((y[q] - ref[k + t]).norm() / ref[k + t].norm()) <= TOL, (q, t)
    assert (pool[[0, 2, 4, 5, 7]] == 0).all()
