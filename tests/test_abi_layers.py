"""Host-only checks of the C ABI of the chunked delta rule, its one-token form and
layer norm: descriptors, workspaces and the refusals that come before any launch."""
import ctypes

import pytest

from selective_state_space_vjp_amd import binding as bd


def _chunk(**kw):
    d = dict(batch=2, seqlen=100, nqk_heads=2, nv_heads=4, dk=128, dv=64, scale=0.1, dtype=bd.BF16, packed=0, reserved=0)
    d.update(kw)
    return bd.DeltaChunkDesc(**d)


def _step(**kw):
    d = dict(batch=3, nslots=5, nqk_heads=2, nv_heads=4, dk=128, dv=64, scale=0.1, dtype=bd.BF16,
             gate=bd.GATE_PER_HEAD, reserved=0)
    d.update(kw)
    return bd.DeltaStepDesc(**d)


def _norm(**kw):
    d = dict(rows=10, groups=1, dim=100, eps=1e-5, dtype=bd.BF16)
    d.update(kw)
    return bd.NormDesc(**d)


def _ws(fn, desc):
    n = ctypes.c_size_t(0)
    st = getattr(bd.lib(), fn)(ctypes.byref(desc), ctypes.byref(n))
    return st, n.value


def _fake(n):
    """Aligned addresses that no refused call reads."""
    return [ctypes.c_void_p(4096 * (i + 1)) for i in range(n)]


WS = ctypes.c_void_p(1 << 20)
BIG = 1 << 40

HEADS = [
    (dict(), bd.OK),
    (dict(nv_heads=3), bd.EINVAL),      # not a multiple of the qk heads
    (dict(nqk_heads=0), bd.EINVAL),
    (dict(nv_heads=0), bd.EINVAL),
    (dict(dk=0), bd.EINVAL),
    (dict(dv=-16), bd.EINVAL),
    (dict(dtype=2), bd.EINVAL),
    (dict(reserved=1), bd.EINVAL),
    (dict(batch=-1), bd.EINVAL),
    (dict(dk=16, dv=16), bd.OK),
    (dict(dk=112, dv=48), bd.OK),
    (dict(dk=120), bd.EUNSUPPORTED),
    (dict(dk=144), bd.EUNSUPPORTED),
    (dict(dv=40), bd.EUNSUPPORTED),
    (dict(dv=65536 + 16), bd.EUNSUPPORTED),
    (dict(nqk_heads=1 << 17, nv_heads=1 << 17), bd.EUNSUPPORTED),  # H*K reaches 2^24
    (dict(nqk_heads=1, nv_heads=1 << 18), bd.EUNSUPPORTED),        # HV*V reaches 2^24
    (dict(nqk_heads=1 << 62, nv_heads=1 << 62), bd.EUNSUPPORTED),
    (dict(batch=1 << 40), bd.EUNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", HEADS + [
    (dict(seqlen=-1), bd.EINVAL),
    (dict(packed=2), bd.EINVAL),
    (dict(seqlen=0), bd.OK),
    (dict(batch=0), bd.OK),
    (dict(packed=1), bd.OK),
    (dict(seqlen=1 << 40), bd.EUNSUPPORTED),
], ids=str)
def test_chunk_descriptor_validation(kw, status):
    for fn in ("delta_chunk_fwd_workspace", "delta_chunk_bwd_workspace"):
        assert _ws(fn, _chunk(**kw))[0] == status
    L = bd.lib()
    for fn, n in (("delta_chunk_fwd", 9), ("delta_chunk_bwd", 15)):
        if status != bd.OK:
            assert getattr(L, fn)(ctypes.byref(_chunk(**kw)), *_fake(n), WS, BIG, None) == status


@pytest.mark.parametrize("kw,status", HEADS + [
    (dict(nslots=-1), bd.EINVAL),
    (dict(gate=2), bd.EINVAL),
    (dict(gate=bd.GATE_PER_KEY), bd.OK),
    (dict(batch=0), bd.OK),
    (dict(nslots=1 << 40), bd.EUNSUPPORTED),
], ids=str)
def test_step_descriptor_validation(kw, status):
    assert _ws("delta_step_workspace", _step(**kw))[0] == status
    if status != bd.OK:
        assert bd.lib().delta_step(ctypes.byref(_step(**kw)), *_fake(8), WS, BIG, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(), bd.OK),
    (dict(rows=0), bd.OK),
    (dict(rows=-1), bd.EINVAL),
    (dict(groups=0), bd.EINVAL),
    (dict(dim=0), bd.EINVAL),
    (dict(dtype=-1), bd.EINVAL),
    (dict(eps=-1e-9), bd.EINVAL),
    (dict(eps=float("nan")), bd.EINVAL),
    (dict(eps=0.0), bd.OK),
    (dict(groups=64, dim=1), bd.OK),
    (dict(rows=1 << 32), bd.EUNSUPPORTED),
    (dict(rows=1 << 16, groups=1 << 16), bd.EUNSUPPORTED),
    (dict(dim=1 << 36), bd.EUNSUPPORTED),
    (dict(rows=1 << 30, dim=1 << 34), bd.EUNSUPPORTED),  # byte offsets past 64 bits
], ids=str)
def test_norm_descriptor_validation(kw, status):
    assert _ws("layer_norm_fwd_workspace", _norm(**kw))[0] == status
    assert _ws("layer_norm_bwd_workspace", _norm(**kw))[0] == status
    if status != bd.OK:
        assert bd.lib().layer_norm_fwd(ctypes.byref(_norm(**kw)), *_fake(8), WS, BIG, None) == status
        assert bd.lib().layer_norm_bwd(ctypes.byref(_norm(**kw)), *_fake(10), WS, BIG, None) == status


def test_backward_of_the_chunked_rule_is_bf16_only():
    d = _chunk(dtype=bd.F32)
    assert _ws("delta_chunk_fwd_workspace", d)[0] == bd.OK
    assert _ws("delta_chunk_bwd_workspace", d)[0] == bd.EUNSUPPORTED
    assert bd.lib().delta_chunk_bwd(ctypes.byref(d), *_fake(15), WS, BIG, None) == bd.EUNSUPPORTED


def test_null_descriptors_and_sizes():
    L = bd.lib()
    n = ctypes.c_size_t(0)
    for fn, d in (("delta_chunk_fwd", _chunk()), ("delta_chunk_bwd", _chunk()), ("delta_step", _step()),
                  ("layer_norm_fwd", _norm()), ("layer_norm_bwd", _norm())):
        q = getattr(L, fn + "_workspace")
        assert q(None, ctypes.byref(n)) == bd.EINVAL
        assert q(ctypes.byref(d), None) == bd.EINVAL


# per entry point: descriptor, number of pointers, the optional ones, alignments (16 unless named)
CALLS = {
    "delta_chunk_fwd": (_chunk, 9, {5, 6, 8}, {3: 4, 4: 4}),
    "delta_chunk_bwd": (_chunk, 15, {5, 7, 8, 14}, {3: 4, 4: 4, 12: 4, 13: 4}),
    "delta_step": (_step, 8, {6}, {3: 4, 4: 4, 6: 4}),
    "layer_norm_fwd": (_norm, 8, {1, 2, 4, 5, 6, 7}, {0: 2, 1: 4, 2: 4, 3: 2, 4: 4, 5: 4, 6: 1, 7: 4}),
    "layer_norm_bwd": (_norm, 10, {1, 2, 3, 6, 8, 9}, {0: 2, 1: 2, 2: 1, 3: 4, 4: 4, 5: 4, 6: 4, 7: 2, 8: 4, 9: 4}),
}


def _pointers(fn, n):
    p = _fake(n)
    if fn == "delta_chunk_fwd":
        p[6] = None  # seq_offsets, packed only
    elif fn == "delta_chunk_bwd":
        p[8] = None
    elif fn == "layer_norm_bwd":
        p[2] = p[3] = None  # the 8-bit form, in place of x
    return p


@pytest.mark.parametrize("fn", CALLS)
def test_null_and_misaligned_pointers_are_refused(fn):
    make, n, optional, align = CALLS[fn]
    call, d = getattr(bd.lib(), fn), make()
    good = _pointers(fn, n)
    for i in range(n):
        if i not in optional:
            p = list(good)
            p[i] = None
            assert call(ctypes.byref(d), *p, WS, BIG, None) == bd.EINVAL, i
        a = align.get(i, 16)
        if good[i] is not None and a > 1:
            p = list(good)
            p[i] = ctypes.c_void_p(p[i].value + a // 2)
            assert call(ctypes.byref(d), *p, WS, BIG, None) == bd.EINVAL, i


@pytest.mark.parametrize("fn", ["delta_chunk_fwd", "delta_chunk_bwd", "layer_norm_bwd"])
def test_workspace_is_checked(fn):
    make, n, _, _ = CALLS[fn]
    call, d, p = getattr(bd.lib(), fn), make(), _pointers(fn, n)
    st, need = _ws(fn + "_workspace", d)
    assert st == bd.OK and need > 0
    assert call(ctypes.byref(d), *p, None, need, None) == bd.EWORKSPACE
    assert call(ctypes.byref(d), *p, WS, need - 1, None) == bd.EWORKSPACE
    assert call(ctypes.byref(d), *p, ctypes.c_void_p(WS.value + 16), need, None) == bd.EWORKSPACE


def test_offsets_belong_to_packed_calls():
    L = bd.lib()
    for fn, n, at in (("delta_chunk_fwd", 9, 6), ("delta_chunk_bwd", 15, 8)):
        p = _fake(n)
        assert getattr(L, fn)(ctypes.byref(_chunk()), *p, WS, BIG, None) == bd.EINVAL
        p[at] = None
        assert getattr(L, fn)(ctypes.byref(_chunk(packed=1)), *p, WS, BIG, None) == bd.EINVAL
        p[at] = ctypes.c_void_p(4096 + 2)
        assert getattr(L, fn)(ctypes.byref(_chunk(packed=1)), *p, WS, BIG, None) == bd.EINVAL


def test_step_without_slots_needs_a_state_for_every_request():
    p = _fake(8)
    p[6] = None
    assert bd.lib().delta_step(ctypes.byref(_step(batch=6)), *p, None, 0, None) == bd.EINVAL
    # per-key gates are read in 16-byte pieces
    p = _fake(8)
    p[4] = ctypes.c_void_p(4096 * 5 + 4)
    assert bd.lib().delta_step(ctypes.byref(_step(gate=bd.GATE_PER_KEY)), *p, None, 0, None) == bd.EINVAL


def test_norm_takes_one_form_of_its_input():
    L, d = bd.lib(), _norm()
    p = _fake(10)
    assert L.layer_norm_bwd(ctypes.byref(d), *p, WS, BIG, None) == bd.EINVAL  # x and x8
    q = list(p)
    q[1] = q[2] = q[3] = None                                               # neither
    assert L.layer_norm_bwd(ctypes.byref(d), *q, WS, BIG, None) == bd.EINVAL
    q = list(p)
    q[1] = q[3] = None                                                      # codes without scales
    assert L.layer_norm_bwd(ctypes.byref(d), *q, WS, BIG, None) == bd.EINVAL
    q = _fake(8)
    q[7] = None
    assert L.layer_norm_fwd(ctypes.byref(d), *q, None, 0, None) == bd.EINVAL


def test_nothing_to_do_reads_no_pointer():
    L = bd.lib()
    assert L.delta_chunk_fwd(ctypes.byref(_chunk(batch=0)), *([None] * 9), None, 0, None) == bd.OK
    assert L.delta_chunk_bwd(ctypes.byref(_chunk(batch=0)), *([None] * 15), None, 0, None) == bd.OK
    assert L.delta_step(ctypes.byref(_step(batch=0)), *([None] * 8), None, 0, None) == bd.OK
    assert L.layer_norm_fwd(ctypes.byref(_norm(rows=0)), *([None] * 8), None, 0, None) == bd.OK


def test_debug_mode_adds_its_flag_to_every_workspace(monkeypatch):
    queries = [("delta_chunk_fwd", _chunk()), ("delta_chunk_bwd", _chunk()), ("delta_step", _step()),
               ("layer_norm_fwd", _norm()), ("layer_norm_bwd", _norm())]
    monkeypatch.delenv("SSMVJP_CHECK_FINITE", raising=False)
    off = [_ws(fn + "_workspace", d) for fn, d in queries]
    monkeypatch.setenv("SSMVJP_CHECK_FINITE", "1")
    for (fn, d), (st0, n0) in zip(queries, off):
        st, n = _ws(fn + "_workspace", d)
        assert st == st0 == bd.OK and n == (n0 + 255) // 256 * 256 + 256, fn
        p = _pointers(fn, CALLS[fn][1])
        assert getattr(bd.lib(), fn)(ctypes.byref(d), *p, WS, n0, None) == bd.EWORKSPACE


def test_backward_workspace_grows_with_the_chunks_not_the_steps():
    n64 = _ws("delta_chunk_bwd_workspace", _chunk(batch=1, seqlen=64))[1]
    assert _ws("delta_chunk_bwd_workspace", _chunk(batch=1, seqlen=1))[1] == n64
    assert _ws("delta_chunk_bwd_workspace", _chunk(batch=1, seqlen=128))[1] <= 2 * n64
