"""Host-side argument checks of the binding of the linear recurrence, the gated feed-forward projections and
dropout: every mismatch of a tensor with the sizes that the others fix is refused before any call; CPU tensors of
the right shapes are refused for their device alone."""
import pytest
import torch

from selective_state_space_vjp_amd import binding as bd

f32, bf16, i32 = torch.float32, torch.bfloat16, torch.int32


def scan(b=2, T=9, D=6, dtype=bf16, gated=True, packed=False):
    n = 1 if packed else b
    z = lambda *s, t=dtype: torch.zeros(*s, dtype=t)  # noqa: E731
    return dict(x=z(n, T, D), gate=z(n, T, D, t=dtype if gated else f32), dh=z(n, T, D), h0=z(b, D, t=f32), dh_final=z(b, D, t=f32),
                input_gate=z(n, T, D) if gated else None, decay=z(D, t=f32) if gated else None,
                ckpt=z(T // 64 + b, D, t=f32) if packed else z(b, 1, D, t=f32),
                seq_offsets=torch.zeros(b + 1, dtype=i32) if packed else None)


def fwd(a, **kw):
    return bd.linear_scan_fwd(a["x"], a["gate"], a["h0"], input_gate=a["input_gate"], decay=a["decay"], seq_offsets=a["seq_offsets"], **kw)


def bwd(a, **kw):
    return bd.linear_scan_bwd(a["x"], a["gate"], a["dh"], a["h0"], a["dh_final"], input_gate=a["input_gate"], decay=a["decay"],
                              ckpt=a["ckpt"], seq_offsets=a["seq_offsets"], **kw)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("call", [fwd, bwd])
def test_scan_correct_shapes_refused_only_for_the_device(call, packed, gated):
    with pytest.raises(ValueError, match="GPU tensor"):
        call(scan(packed=packed, gated=gated))


BAD = [("x", torch.zeros(2, 9, 7, dtype=bf16)), ("gate", torch.zeros(2, 8, 6, dtype=bf16)), ("gate", torch.zeros(2, 9, 1, dtype=bf16)),
       ("input_gate", torch.zeros(1, 9, 6, dtype=bf16)), ("decay", torch.zeros(7)), ("decay", torch.zeros(1)), ("h0", torch.zeros(1, 6)),
       ("h0", torch.zeros(6))]


@pytest.mark.parametrize("key,bad", BAD, ids=lambda x: x if isinstance(x, str) else str(tuple(x.shape)))
def test_scan_rejects_mismatched_inputs(key, bad):
    for call in (fwd, bwd):
        a = scan()
        a[key] = bad
        with pytest.raises(ValueError, match="shape"):
            call(a)


@pytest.mark.parametrize("key,bad", [("dh", torch.zeros(2, 9, 5, dtype=bf16)), ("dh_final", torch.zeros(2, 5)), ("ckpt", torch.zeros(2, 2, 6)),
                                     ("ckpt", torch.zeros(2, 6))], ids=str)
def test_scan_backward_rejects_mismatched_gradients(key, bad):
    a = scan()
    a[key] = bad
    with pytest.raises(ValueError, match="shape"):
        bwd(a)


def test_scan_types_forms_and_layout():
    for key in ("gate", "input_gate", "decay", "h0"):
        for call in (fwd, bwd):
            a = scan()
            a[key] = a[key].to(torch.float16)
            with pytest.raises(TypeError):
                call(a)
    a = scan()
    a["x"] = a["x"].to(torch.float16)
    with pytest.raises(TypeError):
        fwd(a)
    with pytest.raises(TypeError):  # the log form's gate is float32
        fwd(dict(scan(gated=False), gate=torch.zeros(2, 9, 6, dtype=bf16)))
    for key in ("input_gate", "decay"):
        with pytest.raises(ValueError, match="belong together"):
            fwd(dict(scan(), **{key: None}))
    for key in ("x", "gate"):
        with pytest.raises(ValueError, match="required"):
            fwd(dict(scan(), **{key: None}))
    with pytest.raises(ValueError, match="required"):
        bwd(dict(scan(), dh=None))
    with pytest.raises(ValueError, match="contiguous"):
        fwd(dict(scan(), gate=torch.zeros(2, 9, 12, dtype=bf16)[..., ::2]))
    with pytest.raises(ValueError, match="packed"):
        fwd(dict(scan(), seq_offsets=torch.zeros(3, dtype=i32)))
    with pytest.raises(TypeError):
        fwd(dict(scan(packed=True), seq_offsets=torch.zeros(3, dtype=torch.int64)))
    with pytest.raises(ValueError, match=r"\[b,T,D\]"):
        fwd(dict(scan(), x=torch.zeros(9, 6, dtype=bf16)))


def test_scan_outputs_are_checked():
    a = scan()
    with pytest.raises(ValueError, match="out is missing 'h'"):
        fwd(a, out={"h": None})
    with pytest.raises(ValueError, match="shape"):
        fwd(a, out={"h": torch.zeros(2, 9, 5, dtype=bf16)})
    with pytest.raises(ValueError, match="shape"):
        fwd(a, out={"h": torch.zeros_like(a["x"]), "ckpt": torch.zeros(2, 2, 6)})
    with pytest.raises(ValueError, match="out is missing"):
        bwd(a, out={"dx": torch.zeros_like(a["x"])})
    good = {"dx": torch.zeros_like(a["x"]), "dgate": torch.zeros_like(a["x"]), "dinput_gate": torch.zeros_like(a["x"]), "ddecay": torch.zeros(6)}
    with pytest.raises(ValueError, match="shape"):
        bwd(a, out=dict(good, ddecay=torch.zeros(5)))
    with pytest.raises(ValueError, match="shape"):
        bwd(a, out=dict(good, dh0=torch.zeros(1, 6)))


def test_step_checks():
    x, st = torch.zeros(3, 6, dtype=bf16), torch.zeros(4, 6)
    args = dict(input_gate=x, decay=torch.zeros(6))
    with pytest.raises(ValueError, match="GPU tensor"):
        bd.linear_scan_step(x, x, st, slots=torch.zeros(3, dtype=i32), **args)
    with pytest.raises(ValueError, match="GPU tensor"):
        bd.linear_scan_step(x, torch.zeros(3, 6), st)
    for bad in (dict(state=torch.zeros(4, 5)), dict(gate=torch.zeros(3, 5, dtype=bf16)), dict(slots=torch.zeros(2, dtype=i32)),
                dict(decay=torch.zeros(5)), dict(input_gate=torch.zeros(2, 6, dtype=bf16)), dict(out=torch.zeros(3, 7, dtype=bf16))):
        kw = dict(gate=x, state=st, **args)
        kw.update(bad)
        with pytest.raises(ValueError, match="shape"):
            bd.linear_scan_step(x, kw.pop("gate"), kw.pop("state"), **kw)
    with pytest.raises(TypeError):
        bd.linear_scan_step(x, x, st.to(bf16), **args)
    with pytest.raises(TypeError):
        bd.linear_scan_step(x, x, st)  # the log form's gate is float32
    with pytest.raises(ValueError, match="required"):
        bd.linear_scan_step(x, x, None, **args)
    with pytest.raises(ValueError, match="belong together"):
        bd.linear_scan_step(x, x, st, input_gate=x)


def test_ffn_checks():
    x, w, h = torch.zeros(3, 8, dtype=bf16), torch.zeros(16, 8, dtype=bf16), torch.zeros(3, 16, dtype=bf16)
    with pytest.raises(ValueError, match="GPU tensor"):
        bd.gated_ffn_fwd(x, w, w, want_saved=True)
    with pytest.raises(ValueError, match="GPU tensor"):
        bd.gated_ffn_bwd(h, x, w, w, saved=(h, h), act="gelu")
    with pytest.raises(ValueError, match="GPU tensor"):
        bd.gated_ffn_fwd(torch.zeros(2, 3, 8, dtype=bf16), w, w)
    with pytest.raises(ValueError, match="act"):
        bd.gated_ffn_fwd(x, w, w, act="relu")
    for bad in ((torch.zeros(3, 16, dtype=bf16), w, w), (x, w, torch.zeros(8, 8, dtype=bf16)), (x, w, torch.zeros(16, 16, dtype=bf16))):
        with pytest.raises(ValueError, match="shape"):
            bd.gated_ffn_fwd(*bad)
    for kw in (dict(dh=torch.zeros(3, 8, dtype=bf16)), dict(saved=(h, torch.zeros(2, 16, dtype=bf16)))):
        with pytest.raises(ValueError, match="shape"):
            bd.gated_ffn_bwd(kw.pop("dh", h), x, w, w, **kw)
    with pytest.raises(ValueError, match="required"):
        bd.gated_ffn_bwd(h, x, w, w, saved=(h, None))
    with pytest.raises(ValueError, match="required"):
        bd.gated_ffn_bwd(None, x, w, w)
    with pytest.raises(TypeError):
        bd.gated_ffn_fwd(x, w, w.float())
    with pytest.raises(TypeError):
        bd.gated_ffn_fwd(x.half(), w.half(), w.half())
    with pytest.raises(ValueError, match="contiguous"):
        bd.gated_ffn_fwd(x, torch.zeros(16, 16, dtype=bf16)[:, ::2], w)
    with pytest.raises(ValueError, match="out is missing"):
        bd.gated_ffn_fwd(x, w, w, want_saved=True, out={"h": h})
    with pytest.raises(ValueError, match="shape"):
        bd.gated_ffn_bwd(h, x, w, w, want_dx=False, out={"dw_gate": w, "dw_up": x})


def test_dropout_checks():
    x, r = torch.zeros(3, 5), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU tensor"):
        bd.dropout_fwd(x, r, x, p=0.5)
    with pytest.raises(ValueError, match="GPU tensor"):
        bd.dropout_bwd(x, r, p=0.5)
    for p in (-0.1, 1.1, float("nan")):
        with pytest.raises(ValueError, match="p must be"):
            bd.dropout_fwd(x, r, p=p)
    with pytest.raises(ValueError, match="shape"):
        bd.dropout_fwd(x, r, torch.zeros(3, 4), p=0.5)
    with pytest.raises(ValueError, match="shape"):
        bd.dropout_fwd(x, torch.zeros(3, dtype=torch.int64), p=0.5)
    with pytest.raises(TypeError):
        bd.dropout_fwd(x, torch.zeros(2, dtype=i32), p=0.5)
    with pytest.raises(TypeError):
        bd.dropout_fwd(x, r, x.to(bf16), p=0.5)
    with pytest.raises(TypeError):
        bd.dropout_fwd(x.double(), r, p=0.5)
    with pytest.raises(ValueError, match="contiguous"):
        bd.dropout_bwd(torch.zeros(3, 10)[:, ::2], r, p=0.5)
    with pytest.raises(ValueError, match="required"):
        bd.dropout_fwd(x, None, p=0.5)
    with pytest.raises(ValueError, match="shape"):
        bd.dropout_fwd(x, r, p=0.5, out=torch.zeros(15))
