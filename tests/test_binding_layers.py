"""Host-side argument checks of the binding of the chunked delta rule, its one-token
form and layer norm.  The C entry points see only pointers, so every mismatch of a
tensor with the sizes that q, v or x fix is refused before any call; CPU tensors of
the right shapes are refused for their device alone."""
import pytest
import torch

from selective_state_space_vjp_amd import binding as bd

f32, bf16, i32 = torch.float32, torch.bfloat16, torch.int32


def _chunk(b=1, T=8, H=1, HV=2, K=16, V=32, dtype=bf16, packed=False):
    ns = 3 if packed else b
    return dict(q=torch.zeros(b, T, H, K, dtype=dtype), k=torch.zeros(b, T, H, K, dtype=dtype),
                v=torch.zeros(b, T, HV, V, dtype=dtype), beta=torch.zeros(b, T, HV), g=torch.zeros(b, T, HV),
                S0=torch.zeros(ns, HV, K, V), d_o=torch.zeros(b, T, HV, V, dtype=dtype),
                dS_final=torch.zeros(ns, HV, K, V),
                seq_offsets=torch.tensor([0, 2, 5, 8], dtype=i32) if packed else None)


def _fwd(a, **kw):
    return bd.delta_chunk_fwd(a["q"], a["k"], a["v"], a["beta"], a["g"], a["S0"], scale=1.0,
                              seq_offsets=a["seq_offsets"], **kw)


def _bwd(a, **kw):
    return bd.delta_chunk_bwd(a["q"], a["k"], a["v"], a["beta"], a["g"], a["S0"], a["d_o"], a["dS_final"], scale=1.0,
                              seq_offsets=a["seq_offsets"], **kw)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_chunk_correct_shapes_refused_only_for_the_device(call, packed):
    with pytest.raises(ValueError, match="GPU tensor"):
        call(_chunk(packed=packed))


CHUNK_BAD = [
    ("k", torch.zeros(1, 8, 2, 16, dtype=bf16)), ("k", torch.zeros(1, 7, 1, 16, dtype=bf16)),
    ("v", torch.zeros(1, 9, 2, 32, dtype=bf16)), ("v", torch.zeros(2, 8, 2, 32, dtype=bf16)),
    ("beta", torch.zeros(1, 8, 1)), ("g", torch.zeros(1, 8, 2, 16)), ("g", torch.zeros(8, 2)),
    ("S0", torch.zeros(1, 2, 32, 16)), ("S0", torch.zeros(2, 2, 16, 32)),
]


@pytest.mark.parametrize("key,bad", CHUNK_BAD, ids=lambda x: x if isinstance(x, str) else str(tuple(x.shape)))
def test_chunk_rejects_mismatched_inputs(key, bad):
    for call in (_fwd, _bwd):
        a = _chunk()
        a[key] = bad
        with pytest.raises(ValueError, match="shape"):
            call(a)


@pytest.mark.parametrize("key,bad", [("d_o", torch.zeros(1, 8, 2, 16, dtype=bf16)), ("dS_final", torch.zeros(1, 1, 16, 32))],
                         ids=["d_o", "dS_final"])
def test_chunk_backward_rejects_mismatched_gradients(key, bad):
    a = _chunk()
    a[key] = bad
    with pytest.raises(ValueError, match="shape"):
        _bwd(a)


@pytest.mark.parametrize("key", ["q", "k", "v", "beta", "g"])
def test_chunk_rejects_missing_and_wrong_types(key):
    for call in (_fwd, _bwd):
        a = _chunk()
        a[key] = None
        with pytest.raises(ValueError, match="required"):
            call(a)
        a = _chunk()
        a[key] = a[key].to(torch.float16)
        with pytest.raises(TypeError):
            call(a)


def test_chunk_rejects_strided_inputs():
    a = _chunk(T=16)
    a["v"] = torch.zeros(1, 32, 2, 32, dtype=bf16)[:, ::2]
    with pytest.raises(ValueError, match="contiguous"):
        _fwd(a)


def test_chunk_rejects_bad_offsets():
    a = _chunk(packed=True)
    a["seq_offsets"] = a["seq_offsets"].long()
    with pytest.raises(TypeError):
        _fwd(a)
    a["seq_offsets"] = torch.zeros(2, 2, dtype=i32)
    with pytest.raises(ValueError, match="seq_offsets"):
        _fwd(a)
    a["seq_offsets"] = torch.zeros(0, dtype=i32)
    with pytest.raises(ValueError, match="seq_offsets"):
        _fwd(a)
    a = _chunk(b=2, packed=True)
    with pytest.raises(ValueError, match="packed"):
        _fwd(a)
    a = _chunk(packed=True)
    a["S0"] = torch.zeros(1, 2, 16, 32)  # one state for three sequences
    with pytest.raises(ValueError, match="shape"):
        _fwd(a)


def _step(b=3, H=1, HV=2, K=16, V=32, n=5, dtype=bf16, per_key=False):
    return dict(q=torch.zeros(b, H, K, dtype=dtype), k=torch.zeros(b, H, K, dtype=dtype),
                v=torch.zeros(b, HV, V, dtype=dtype), beta=torch.zeros(b, HV),
                g=torch.zeros((b, HV, K) if per_key else (b, HV)), state=torch.zeros(n, HV, K, V),
                slots=torch.zeros(b, dtype=i32))


def _call_step(a, **kw):
    return bd.delta_step(a["q"], a["k"], a["v"], a["beta"], a["g"], a["state"], scale=1.0, slots=a["slots"], **kw)


@pytest.mark.parametrize("per_key", [False, True])
def test_step_correct_shapes_refused_only_for_the_device(per_key):
    with pytest.raises(ValueError, match="GPU tensor"):
        _call_step(_step(per_key=per_key))


@pytest.mark.parametrize("key,bad", [
    ("k", torch.zeros(2, 1, 16, dtype=bf16)), ("v", torch.zeros(2, 2, 32, dtype=bf16)), ("beta", torch.zeros(3, 1)),
    ("g", torch.zeros(3, 2, 8)), ("g", torch.zeros(2, 2)), ("state", torch.zeros(5, 2, 32, 16)),
    ("state", torch.zeros(5, 1, 16, 32)), ("slots", torch.zeros(2, dtype=i32)),
], ids=lambda x: x if isinstance(x, str) else str(tuple(x.shape)))
def test_step_rejects_mismatched_inputs(key, bad):
    a = _step()
    a[key] = bad
    with pytest.raises(ValueError, match="shape"):
        _call_step(a)


def test_step_rejects_types_ranks_and_missing_tensors():
    for key in ("q", "k", "v", "beta", "g", "state"):
        a = _step()
        a[key] = None
        with pytest.raises(ValueError, match="required"):
            _call_step(a)
    for key in ("k", "v", "beta", "g", "state"):
        a = _step()
        a[key] = a[key].double()
        with pytest.raises(TypeError):
            _call_step(a)
    a = _step()
    a["slots"] = a["slots"].long()
    with pytest.raises(TypeError):
        _call_step(a)
    a = _step()
    a["q"] = a["q"][None]
    with pytest.raises(ValueError, match="must be"):
        _call_step(a)
    a = _step()
    a["state"] = torch.zeros(5, 2, 32, 16).transpose(2, 3)  # the right shape, strided
    with pytest.raises(ValueError, match="contiguous"):
        _call_step(a)


def test_norm_correct_shapes_refused_only_for_the_device():
    x = torch.zeros(4, 2, 8, dtype=bf16)
    for w in (None, torch.ones(8), torch.ones(2, 8)):
        with pytest.raises(ValueError, match="GPU tensor"):
            bd.layer_norm_fwd(x, w, w)
        with pytest.raises(ValueError, match="GPU tensor"):
            bd.layer_norm_bwd(x, x, torch.zeros(4, 2), torch.zeros(4, 2), w)
    with pytest.raises(ValueError, match="GPU tensor"):
        bd.layer_norm_bwd(x, None, torch.zeros(4, 2), torch.zeros(4, 2),
                          ckpt8=(torch.zeros(4, 2, 8, dtype=torch.int8), torch.zeros(4, 2, 1)))


def test_norm_rejects_mismatched_inputs():
    x, st = torch.zeros(4, 2, 8, dtype=bf16), torch.zeros(4, 2)
    for w in (torch.ones(4), torch.ones(4, 8), torch.ones(2, 2, 8)):
        with pytest.raises(ValueError):
            bd.layer_norm_fwd(x, w)
        with pytest.raises(ValueError):
            bd.layer_norm_bwd(x, x, st, st, w)
    with pytest.raises(ValueError):
        bd.layer_norm_fwd(x, torch.ones(8), torch.ones(2, 8))
    with pytest.raises(ValueError, match="weight"):
        bd.layer_norm_fwd(x, None, torch.ones(8))
    with pytest.raises(TypeError):
        bd.layer_norm_fwd(x, torch.ones(8, dtype=bf16))
    with pytest.raises(TypeError):
        bd.layer_norm_fwd(x.half())
    with pytest.raises(ValueError, match="contiguous"):
        bd.layer_norm_fwd(x.transpose(0, 1))
    with pytest.raises(ValueError):
        bd.layer_norm_fwd(torch.zeros(4, 0))
    with pytest.raises(ValueError):
        bd.layer_norm_fwd(torch.zeros(()))
    with pytest.raises(ValueError):
        bd.layer_norm_bwd(x, x[:3].contiguous(), st, st)
    with pytest.raises(TypeError):
        bd.layer_norm_bwd(x, x.float(), st, st)
    with pytest.raises(ValueError):
        bd.layer_norm_bwd(x, x, torch.zeros(4), st)
    with pytest.raises(ValueError, match="exactly one"):
        bd.layer_norm_bwd(x, None, st, st)
    x8, s8 = torch.zeros(4, 2, 8, dtype=torch.int8), torch.zeros(4, 2, 1)
    with pytest.raises(ValueError, match="exactly one"):
        bd.layer_norm_bwd(x, x, st, st, ckpt8=(x8, s8))
    with pytest.raises(ValueError):
        bd.layer_norm_bwd(x, None, st, st, ckpt8=(x8, torch.zeros(4, 2)))
    with pytest.raises(TypeError):
        bd.layer_norm_bwd(x, None, st, st, ckpt8=(x8.float(), s8))
    with pytest.raises(ValueError, match="required"):
        bd.layer_norm_bwd(x, None, st, st, ckpt8=(x8, None))
