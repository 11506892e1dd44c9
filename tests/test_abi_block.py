"""Host-only checks of the C ABI of the linear recurrence, the gated feed-forward projections and dropout:
descriptors, workspaces and the refusals that come before any launch."""
import ctypes

import pytest

from selective_state_space_vjp_amd import binding as bd

WS = ctypes.c_void_p(1 << 20)
BIG = 1 << 45
INF, NAN = float("inf"), float("nan")


def _scan(**kw):
    d = dict(batch=2, seqlen=300, dim=100, c=8.0, form=bd.SCAN_GATED, dtype=bd.BF16, packed=0)
    d.update(kw)
    return bd.LinearScanDesc(**d)


def _step(**kw):
    d = dict(batch=3, nslots=5, dim=100, c=8.0, form=bd.SCAN_GATED, dtype=bd.BF16, reserved=0)
    d.update(kw)
    return bd.LinearStepDesc(**d)


def _ffn(**kw):
    d = dict(rows=10, dim=64, hidden=96, act=bd.ACT_SILU, dtype=bd.BF16)
    d.update(kw)
    return bd.FfnDesc(**d)


def _drop(**kw):
    d = dict(n=1000, p=0.1, dtype=bd.BF16, reserved=0)
    d.update(kw)
    return bd.DropoutDesc(**d)


def _ws(fn, desc):
    n = ctypes.c_size_t(0)
    st = getattr(bd.lib(), fn + "_workspace")(ctypes.byref(desc), ctypes.byref(n))
    return st, n.value


def _fake(n):
    """Aligned addresses that no refused call reads."""
    return [ctypes.c_void_p(4096 * (i + 1)) for i in range(n)]


def _call(fn, desc, ptrs, ws=WS, nws=BIG):
    return getattr(bd.lib(), fn)(ctypes.byref(desc), *ptrs, ws, nws, None)


COMMON = [
    (dict(), bd.OK),
    (dict(dim=0), bd.EINVAL),
    (dict(dim=-4), bd.EINVAL),
    (dict(dtype=2), bd.EINVAL),
    (dict(form=2), bd.EINVAL),
    (dict(form=-1), bd.EINVAL),
    (dict(c=0.0), bd.EINVAL),
    (dict(c=-1.0), bd.EINVAL),
    (dict(c=INF), bd.EINVAL),
    (dict(c=NAN), bd.EINVAL),
    (dict(c=NAN, form=bd.SCAN_LOG), bd.OK),  # not used
    (dict(batch=-1), bd.EINVAL),
    (dict(batch=0), bd.OK),
    (dict(dim=1), bd.OK),
    (dict(dim=(1 << 24) - 1, batch=1), bd.OK),
    (dict(dim=1 << 24), bd.EUNSUPPORTED),
    (dict(batch=1 << 40), bd.EUNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(seqlen=-1), bd.EINVAL),
    (dict(seqlen=0), bd.OK),
    (dict(packed=2), bd.EINVAL),
    (dict(packed=1), bd.OK),
    (dict(seqlen=1 << 40), bd.EUNSUPPORTED),
    (dict(seqlen=1 << 24, dim=1 << 13), bd.EUNSUPPORTED),      # launches of 2^32 threads
    (dict(seqlen=1 << 30, batch=1 << 30), bd.EUNSUPPORTED),
], ids=str)
def test_scan_descriptor_validation(kw, status):
    for fn, n in (("linear_scan_fwd", 9), ("linear_scan_bwd", 14)):
        assert _ws(fn, _scan(**kw))[0] == status
        if status != bd.OK:
            assert _call(fn, _scan(**kw), _fake(n)) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(reserved=1), bd.EINVAL),
    (dict(nslots=-1), bd.EINVAL),
    (dict(nslots=1 << 40), bd.EUNSUPPORTED),
], ids=str)
def test_step_descriptor_validation(kw, status):
    assert _ws("linear_scan_step", _step(**kw))[0] == status
    if status != bd.OK:
        assert _call("linear_scan_step", _step(**kw), _fake(7)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(), bd.OK),
    (dict(rows=0), bd.OK),
    (dict(rows=-1), bd.EINVAL),
    (dict(dim=0), bd.EINVAL),
    (dict(hidden=0), bd.EINVAL),
    (dict(act=2), bd.EINVAL),
    (dict(dtype=-1), bd.EINVAL),
    (dict(dim=8, hidden=8, rows=1), bd.OK),
    (dict(dim=60), bd.EUNSUPPORTED),
    (dict(hidden=100), bd.EUNSUPPORTED),
    (dict(dim=1 << 20), bd.EUNSUPPORTED),
    (dict(hidden=1 << 20), bd.EUNSUPPORTED),
    (dict(dim=(1 << 20) - 8, hidden=(1 << 20) - 8), bd.EUNSUPPORTED),  # the weights' gradients' tiles
    (dict(rows=1 << 30), bd.EUNSUPPORTED),
    (dict(rows=1 << 40), bd.EUNSUPPORTED),
], ids=str)
def test_ffn_descriptor_validation(kw, status):
    for fn, n in (("gated_ffn_fwd", 6), ("gated_ffn_bwd", 9)):
        assert _ws(fn, _ffn(**kw))[0] == status
        if status != bd.OK:
            assert _call(fn, _ffn(**kw), _fake(n)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(), bd.OK),
    (dict(n=0), bd.OK),
    (dict(n=-1), bd.EINVAL),
    (dict(p=-1e-9), bd.EINVAL),
    (dict(p=1.0000001), bd.EINVAL),
    (dict(p=NAN), bd.EINVAL),
    (dict(p=1.0), bd.OK),
    (dict(reserved=1), bd.EINVAL),
    (dict(dtype=7), bd.EINVAL),
    (dict(n=1 << 60), bd.EUNSUPPORTED),
], ids=str)
def test_dropout_descriptor_validation(kw, status):
    for fn, n in (("dropout_fwd", 4), ("dropout_bwd", 3)):
        assert _ws(fn, _drop(**kw))[0] == status
        if status != bd.OK:
            assert _call(fn, _drop(**kw), _fake(n)) == status


# the calls, their pointers by name, which may be NULL; (x, gate, igate, decay, h0, off, h, h_final, ckpt)
CALLS = [
    ("linear_scan_fwd", _scan(), ["x", "gate", "input_gate", "decay", "h0?", "off!", "h", "h_final?", "ckpt?"]),
    ("linear_scan_bwd", _scan(), ["x", "gate", "input_gate", "decay", "h0?", "ckpt?", "dh", "dh_final?", "off!", "dx", "dgate",
                                  "dinput_gate", "ddecay", "dh0?"]),
    ("linear_scan_step", _step(), ["x", "gate", "input_gate", "decay", "state", "slots?", "h"]),
    ("gated_ffn_fwd", _ffn(), ["x", "w_gate", "w_up", "h", "gate&", "up&"]),
    ("gated_ffn_bwd", _ffn(), ["dh", "x", "w_gate", "w_up", "gate&", "up&", "dx?", "dw_gate?", "dw_up?"]),
    ("dropout_fwd", _drop(), ["x", "residual?", "rng", "y"]),
    ("dropout_bwd", _drop(), ["dy", "rng", "dx"]),
]


@pytest.mark.parametrize("fn,desc,names", CALLS, ids=lambda v: v if isinstance(v, str) else "")
def test_pointers(fn, desc, names):
    """Each required pointer NULL, each pointer off its alignment; "!" must be NULL here, "&" both or neither."""
    good = [None if n.endswith("!") else p for n, p in zip(names, _fake(len(names)))]
    for i, n in enumerate(names):
        bad = list(good)
        if n.endswith("!"):
            bad[i] = ctypes.c_void_p(4096)  # borders without packed sequences
            assert _call(fn, desc, bad) == bd.EINVAL, n
            continue
        if not n.endswith("?"):
            bad[i] = None
            assert _call(fn, desc, bad) == bd.EINVAL, n
        bad[i] = ctypes.c_void_p(good[i].value + 1)
        assert _call(fn, desc, bad) == bd.EINVAL, n
    need = _ws(fn, desc)[1]
    if need:
        assert _call(fn, desc, good, None, BIG) == bd.EWORKSPACE
        assert _call(fn, desc, good, WS, need - 1) == bd.EWORKSPACE
        assert _call(fn, desc, good, ctypes.c_void_p((1 << 20) + 8), BIG) == bd.EWORKSPACE
    assert getattr(bd.lib(), fn + "_workspace")(ctypes.byref(desc), None) == bd.EINVAL
    assert getattr(bd.lib(), fn)(None, *good, WS, BIG, None) == bd.EINVAL


def test_forms_and_aliases_of_the_scan():
    p = _fake(9)
    p[5] = None
    log = _scan(form=bd.SCAN_LOG)
    assert _call("linear_scan_fwd", log, p) == bd.EINVAL  # input_gate and decay with the log form
    q = list(p)
    q[7] = q[4]  # h_final over h0
    assert _call("linear_scan_fwd", _scan(), q) == bd.EINVAL
    q = list(p)
    assert _call("linear_scan_fwd", _scan(packed=1), q) == bd.EINVAL  # no borders
    b = _fake(14)
    b[8] = None
    assert _call("linear_scan_bwd", log, b) == bd.EINVAL
    c = list(b)
    c[13] = c[7]  # dh0 over dh_final
    assert _call("linear_scan_bwd", _scan(), c) == bd.EINVAL
    c = list(b)
    c[2] = c[3] = None
    assert _call("linear_scan_bwd", log, c) == bd.EINVAL  # ddecay and dinput_gate with the log form
    s = _fake(7)
    s[5] = None
    assert _call("linear_scan_step", _step(nslots=2), s) == bd.EINVAL  # request i without a state i


def test_workspaces_grow_with_what_they_hold():
    one = _ws("linear_scan_fwd", _scan(seqlen=128))[1]
    assert one == 0  # a sequence of one tile waits for none
    assert _ws("linear_scan_fwd", _scan(seqlen=129))[1] > 0
    assert _ws("linear_scan_bwd", _scan(seqlen=4096))[1] > _ws("linear_scan_bwd", _scan(seqlen=2048))[1]
    assert _ws("gated_ffn_fwd", _ffn(rows=4096, dim=4096, hidden=8192))[1] == 0
    assert _ws("gated_ffn_bwd", _ffn(rows=777))[1] >= 4 * 777 * 96


@pytest.mark.parametrize("rows", [0, 1, 31, 32, 33, 200, 5000])
def test_ffn_workspace_of_every_kind_of_tile(rows):
    for dim, hidden in ((8, 8), (64, 12288), (12288, 64), (4096, 4096)):
        for dtype in (bd.F32, bd.BF16):
            st, n = _ws("gated_ffn_bwd", _ffn(rows=rows, dim=dim, hidden=hidden, dtype=dtype))
            assert st == bd.OK and n >= 2 * rows * hidden * (4 if dtype == bd.F32 else 2)


def test_finiteness_mode_asks_for_its_flag(monkeypatch):
    for fn, desc, _ in CALLS:
        off = _ws(fn, desc)[1]
        monkeypatch.setenv("SSMVJP_CHECK_FINITE", "1")
        on = _ws(fn, desc)[1]
        monkeypatch.delenv("SSMVJP_CHECK_FINITE")
        assert on == (off + 255) // 256 * 256 + 256
