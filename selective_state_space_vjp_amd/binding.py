"""ctypes binding of libssmvjp (C ABI in include/ssmvjp.h).

Argument marshalling only: shape/dtype checks, output and workspace
allocation through torch's caching allocator, and the current HIP stream.
Every step of the computation runs in the HIP kernels; there is no CPU path.
If the library is missing the calls raise.
"""
from __future__ import annotations

import ctypes
from pathlib import Path

import torch

LIB_PATH = Path(__file__).resolve().parent / "libssmvjp.so"

OK, EINVAL, EUNSUPPORTED, EWORKSPACE, EHIP, ENONFINITE = 0, 1, 2, 3, 4, 5
F32, BF16 = 0, 1
DECAY_PER_HEAD, DECAY_PER_STATE = 0, 1
FORM_MAMBA2, FORM_RAW = 0, 1
GATE_PER_HEAD, GATE_PER_KEY = 0, 1
DELTA_CKPT, DELTA_BWD, DELTA_REDUCE, DELTA_ALL = 1, 2, 4, 7

_STATUS_FNS = ("ssm_scan_bwd_workspace", "ssm_scan_bwd", "ssm_scan_bwd_dA", "ssd_chunk_bwd_workspace",
               "ssd_chunk_bwd", "ssd_chunk_bwd_dA", "ssd_chunk_bwd_states", "ssd_chunk_bwd_grads", "ssd_chunk_bwd_noalloc",
               "ssd_chunk_fwd_workspace", "ssd_chunk_fwd", "delta_rule_bwd_workspace", "delta_rule_bwd",
               "delta_rule_bwd_stages", "delta_chunk_fwd_workspace", "delta_chunk_fwd",
               "delta_chunk_bwd_workspace", "delta_chunk_bwd", "delta_step_workspace",
               "delta_step", "layer_norm_fwd_workspace", "layer_norm_fwd", "layer_norm_bwd_workspace", "layer_norm_bwd")
EXPORTS = _STATUS_FNS + ("ssmvjp_status_str", "ssmvjp_version")


class ScanDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("decay", ctypes.c_int32), ("dtype", ctypes.c_int32), ("ckpt_every", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class SsdDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64),
                ("mimo_rank", ctypes.c_int64), ("chunk_len", ctypes.c_int64),
                ("form", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class DeltaDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nqk_heads", ctypes.c_int64),
                ("nv_heads", ctypes.c_int64), ("dk", ctypes.c_int64), ("dv", ctypes.c_int64),
                ("scale", ctypes.c_float), ("reserved", ctypes.c_int32)]


class DeltaChunkDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nqk_heads", ctypes.c_int64),
                ("nv_heads", ctypes.c_int64), ("dk", ctypes.c_int64), ("dv", ctypes.c_int64),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int32), ("packed", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class DeltaStepDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("nslots", ctypes.c_int64), ("nqk_heads", ctypes.c_int64),
                ("nv_heads", ctypes.c_int64), ("dk", ctypes.c_int64), ("dv", ctypes.c_int64),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int32), ("gate", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class NormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("groups", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("eps", ctypes.c_float), ("dtype", ctypes.c_int32)]


class SsmVjpError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: status {status} ({status_str(status)})")


_lib = None


def lib():
    """Load libssmvjp.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not LIB_PATH.exists():
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(str(LIB_PATH))
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        L.ssm_scan_bwd_workspace.argtypes = [ctypes.POINTER(ScanDesc), ctypes.POINTER(sz)]
        L.ssm_scan_bwd.argtypes = [ctypes.POINTER(ScanDesc)] + [vp] * 14 + [sz, vp]
        L.ssm_scan_bwd_dA.argtypes = [ctypes.POINTER(ScanDesc)] + [vp] * 15 + [sz, vp]
        L.ssd_chunk_bwd_workspace.argtypes = [ctypes.POINTER(SsdDesc), ctypes.POINTER(sz)]
        L.ssd_chunk_bwd.argtypes = [ctypes.POINTER(SsdDesc)] + [vp] * 14 + [sz, vp]
        L.ssd_chunk_bwd_dA.argtypes = [ctypes.POINTER(SsdDesc)] + [vp] * 15 + [sz, vp]
        L.ssd_chunk_bwd_states.argtypes = [ctypes.POINTER(SsdDesc)] + [vp] * 10 + [sz, vp]
        L.ssd_chunk_bwd_grads.argtypes = [ctypes.POINTER(SsdDesc)] + [vp] * 11 + [sz, vp]
        L.ssd_chunk_bwd_noalloc.argtypes = [ctypes.POINTER(SsdDesc)] + [vp] * 14
        L.ssd_chunk_fwd_workspace.argtypes = [ctypes.POINTER(SsdDesc), ctypes.POINTER(sz)]
        L.ssd_chunk_fwd.argtypes = [ctypes.POINTER(SsdDesc)] + [vp] * 9 + [sz, vp]
        L.delta_rule_bwd_workspace.argtypes = [ctypes.POINTER(DeltaDesc), ctypes.POINTER(sz)]
        L.delta_rule_bwd.argtypes = [ctypes.POINTER(DeltaDesc)] + [vp] * 15 + [sz, vp]
        L.delta_rule_bwd_stages.argtypes = [ctypes.POINTER(DeltaDesc), ctypes.c_int32] + [vp] * 15 + [sz, vp]
        for name, desc, nptr in (("delta_chunk_fwd", DeltaChunkDesc, 9), ("delta_chunk_bwd", DeltaChunkDesc, 15),
                                 ("delta_step", DeltaStepDesc, 8),
                                 ("layer_norm_fwd", NormDesc, 8), ("layer_norm_bwd", NormDesc, 10)):
            getattr(L, name + "_workspace").argtypes = [ctypes.POINTER(desc), ctypes.POINTER(sz)]
            getattr(L, name).argtypes = [ctypes.POINTER(desc)] + [vp] * nptr + [vp, sz, vp]
        for name in _STATUS_FNS:
            getattr(L, name).restype = ctypes.c_int
        L.ssmvjp_status_str.argtypes = [ctypes.c_int]
        L.ssmvjp_status_str.restype = ctypes.c_char_p
        L.ssmvjp_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_str(status):
    return lib().ssmvjp_status_str(int(status)).decode()


def version():
    return lib().ssmvjp_version().decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t):
    dtype = t.dtype
    if dtype is torch.float32:
        return F32
    if dtype is torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t.dtype}; big tensors are float32 or bfloat16")


def _need(t, name, dtype, shape, device):
    """Check an optional tensor argument (None passes): shape, dtype and layout.
    The device is checked by _on_gpu once every shape has been checked."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_gpu(device, *tensors):
    """Every tensor handed to the library lives on the same GPU (there is no CPU path)."""
    if not device.type == "cuda":
        raise ValueError("inputs must be GPU tensors (there is no CPU path)")
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"a tensor is on {t.device}, expected {device} (there is no CPU path)")


def _check_out(out, spec, device):
    """Every tensor of a caller-supplied ``out`` dict must match what the call writes:
    the kernels see only pointers, so a wrong size would be written out of bounds."""
    for name, (dtype, shape) in spec.items():
        if name not in out or out[name] is None:
            raise ValueError(f"out is missing '{name}'")
        _need(out[name], f"out['{name}']", dtype, shape, device)


def _workspace(nbytes, device, workspace):
    if nbytes == 0:
        return None, 0
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError("workspace too small")
        if not workspace.is_contiguous() or not workspace.is_cuda or workspace.device != device:
            raise ValueError(f"workspace must be a contiguous tensor on {device}")
        return workspace, workspace.numel() * workspace.element_size()
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


def _check(fn, status):
    if status != OK:
        raise SsmVjpError(fn, status)


# --------------------------------------------------------------------------- #
def scan_desc(x, A, B, ckpt_every=0):
    b, T, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    decay = DECAY_PER_STATE if A.dim() == 2 else DECAY_PER_HEAD
    return ScanDesc(b, T, H, P, N, G, decay, _dtype_code(x), int(ckpt_every), 0)


def ssm_scan_bwd_workspace(desc):
    n = ctypes.c_size_t(0)
    _check("ssm_scan_bwd_workspace", lib().ssm_scan_bwd_workspace(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def ssm_scan_bwd(x, dt, A, B, C, s0, dy, ds_final, *, ckpt_every=0, want_dA=False, out=None, workspace=None,
                 stream=None):
    """Sequential selective-scan backward.  Returns dict dx, d_dt, dB, dC, d_s0
    (and dA, shaped like A, with want_dA=True).

    x, dy [b,T,H,P] and B, C [b,T,G,N] are float32 or bfloat16 (all the same);
    dt [b,T,H], A [H] (Mamba-2) or [H,N] (Mamba-1), s0, ds_final [b,H,P,N] float32
    (s0 / ds_final may be None = zeros).
    """
    if x is None or B is None or A is None or x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [b,T,H,P], B [b,T,G,N] and A [H] or [H,N]")
    desc = scan_desc(x, A, B, ckpt_every)
    b, T, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dev, big = x.device, x.dtype
    _need(x, "x", big, (b, T, H, P), dev)
    _need(dy, "dy", big, (b, T, H, P), dev)
    _need(B, "B", big, (b, T, G, N), dev)
    _need(C, "C", big, (b, T, G, N), dev)
    for name, t in (("dt", dt), ("C", C), ("dy", dy)):
        if t is None:
            raise ValueError(f"{name} is required")
    _need(dt, "dt", torch.float32, (b, T, H), dev)
    if A.dim() not in (1, 2):
        raise ValueError("A must be [H] (per-head decay) or [H,N] (per-state decay)")
    _need(A, "A", torch.float32, (H,) if A.dim() == 1 else (H, N), dev)
    _need(s0, "s0", torch.float32, (b, H, P, N), dev)
    _need(ds_final, "ds_final", torch.float32, (b, H, P, N), dev)
    spec = dict(dx=(big, (b, T, H, P)), d_dt=(torch.float32, (b, T, H)), dB=(big, (b, T, G, N)),
                dC=(big, (b, T, G, N)), d_s0=(torch.float32, (b, H, P, N)))
    if out is None:
        out = dict(dx=torch.empty_like(x), d_dt=torch.empty_like(dt), dB=torch.empty_like(B),
                   dC=torch.empty_like(C), d_s0=torch.empty((b, H, P, N), dtype=torch.float32, device=dev))
    _check_out(out, spec, dev)
    _on_gpu(dev, x, dt, A, B, C, s0, dy, ds_final, *out.values())
    ws, wsb = _workspace(ssm_scan_bwd_workspace(desc), dev, workspace)
    args = (_ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(s0), _ptr(dy), _ptr(ds_final), _ptr(out["dx"]),
            _ptr(out["d_dt"]), _ptr(out["dB"]), _ptr(out["dC"]), _ptr(out["d_s0"]))
    if want_dA:
        if "dA" not in out:
            out["dA"] = torch.empty_like(A)
        _need(out["dA"], "out['dA']", torch.float32, tuple(A.shape), dev)
        st = lib().ssm_scan_bwd_dA(ctypes.byref(desc), *args, _ptr(out["dA"]), _ptr(ws), wsb, _stream(stream))
        _check("ssm_scan_bwd_dA", st)
    else:
        st = lib().ssm_scan_bwd(ctypes.byref(desc), *args, _ptr(ws), wsb, _stream(stream))
        _check("ssm_scan_bwd", st)
    return out


class ScanCall:
    """A prepared ssm_scan_bwd call on fixed device buffers (for repeated timing):
    arguments are checked once, ``run()`` only enqueues the backward."""

    def __init__(self, x, dt, A, B, C, s0, dy, ds_final, *, ckpt_every=0, stream=None):
        self.out = ssm_scan_bwd(x, dt, A, B, C, s0, dy, ds_final, ckpt_every=ckpt_every, stream=stream)
        self.desc = scan_desc(x, A, B, ckpt_every)
        self.ws, self.wsb = _workspace(ssm_scan_bwd_workspace(self.desc), x.device, None)
        self.stream = stream
        p, o = _ptr, self.out
        self._args = (p(x), p(dt), p(A), p(B), p(C), p(s0), p(dy), p(ds_final), p(o["dx"]), p(o["d_dt"]), p(o["dB"]),
                      p(o["dC"]), p(o["d_s0"]))
        self._keep = (x, dt, A, B, C, s0, dy, ds_final)

    def run(self):
        st = lib().ssm_scan_bwd(ctypes.byref(self.desc), *self._args, _ptr(self.ws), self.wsb, _stream(self.stream))
        _check("ssm_scan_bwd", st)


# --------------------------------------------------------------------------- #
def ssd_desc(xv, B, chunk_len, form):
    if form == FORM_MAMBA2:
        b, T, H, P = xv.shape
        M = 1
        G, N = B.shape[2], B.shape[3]
    else:
        b, T, M, H, P = xv.shape
        G, N = B.shape[3], B.shape[4]
    return SsdDesc(b, T, H, P, N, G, M, int(chunk_len), form, _dtype_code(xv))


def _ssd_inputs(xv, dtda, A, B, C, s0, form, chunk_len):
    """Descriptor of a chunked call after checking every input against the shapes
    x/v fixes: B, C [b,T,G,N] (RAW: [b,T,M,G,N]), dt/da [b,T,H], A [H], states
    [b,H,P,N]."""
    if xv is None or B is None:
        raise ValueError("x/v and B are required")
    if xv.dim() != (4 if form == FORM_MAMBA2 else 5):
        raise ValueError(f"x/v must be {'[b,T,H,P]' if form == FORM_MAMBA2 else '[b,T,M,H,P]'}")
    if B.dim() != xv.dim():
        raise ValueError(f"B must be {'[b,T,G,N]' if form == FORM_MAMBA2 else '[b,T,M,G,N]'}")
    desc = ssd_desc(xv, B, chunk_len, form)
    b, T, H, P, N, G, M = desc.batch, desc.seqlen, desc.nheads, desc.headdim, desc.dstate, desc.ngroups, desc.mimo_rank
    dev, big = xv.device, xv.dtype
    bc = (b, T, G, N) if form == FORM_MAMBA2 else (b, T, M, G, N)
    _need(xv, "x/v", big, tuple(xv.shape), dev)
    _need(B, "B", big, bc, dev)
    _need(C, "C", big, bc, dev)
    _need(dtda, "dt/da", torch.float32, (b, T, H), dev)
    if form == FORM_MAMBA2:
        _need(A, "A", torch.float32, (H,), dev)
    _need(s0, "s0", torch.float32, (b, H, P, N), dev)
    if C is None or dtda is None or (form == FORM_MAMBA2 and A is None):
        raise ValueError("C, dt/da (and A in the Mamba-2 form) are required")
    return desc


def _ssd_grad_spec(desc, xv, form):
    b, T, H, P, N, G, M = (desc.batch, desc.seqlen, desc.nheads, desc.headdim, desc.dstate, desc.ngroups,
                           desc.mimo_rank)
    big = xv.dtype
    bc = (b, T, G, N) if form == FORM_MAMBA2 else (b, T, M, G, N)
    names = ("dx", "d_dt") if form == FORM_MAMBA2 else ("dv", "d_da")
    return {names[0]: (big, tuple(xv.shape)), names[1]: (torch.float32, (b, T, H)), "dB": (big, bc),
            "dC": (big, bc), "d_s0": (torch.float32, (b, H, P, N))}


def ssd_chunk_bwd_workspace(desc):
    n = ctypes.c_size_t(0)
    _check("ssd_chunk_bwd_workspace", lib().ssd_chunk_bwd_workspace(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def ssd_chunk_bwd(xv, dtda, A, B, C, s0, dy, ds_final, *, chunk_len, want_dA=False, out=None, workspace=None,
                  stream=None):
    """Chunked SSD backward.

    Mamba-2 form (A given): xv = x [b,T,H,P], dtda = dt [b,T,H] (raw),
    B, C [b,T,G,N]; returns dict dx, d_dt, dB, dC, d_s0 (and dA [H] with
    want_dA=True).
    RAW form (A None): xv = v [b,T,M,H,P], dtda = da [b,T,H], B, C [b,T,M,G,N];
    returns dict dv, d_da, dB, dC, d_s0.
    """
    form = FORM_MAMBA2 if A is not None else FORM_RAW
    desc = _ssd_inputs(xv, dtda, A, B, C, s0, form, chunk_len)
    b, T, H, P, N = desc.batch, desc.seqlen, desc.nheads, desc.headdim, desc.dstate
    dev, big = xv.device, xv.dtype
    if dy is None:
        raise ValueError("dy is required")
    _need(dy, "dy", big, tuple(xv.shape), dev)
    _need(ds_final, "ds_final", torch.float32, (b, H, P, N), dev)
    names = ("dx", "d_dt") if form == FORM_MAMBA2 else ("dv", "d_da")
    if out is None:
        out = {names[0]: torch.empty_like(xv), names[1]: torch.empty_like(dtda), "dB": torch.empty_like(B),
               "dC": torch.empty_like(C), "d_s0": torch.empty((b, H, P, N), dtype=torch.float32, device=dev)}
    _check_out(out, _ssd_grad_spec(desc, xv, form), dev)
    _on_gpu(dev, xv, dtda, A, B, C, s0, dy, ds_final, *out.values())
    ws, wsb = _workspace(ssd_chunk_bwd_workspace(desc), dev, workspace)
    args = (_ptr(xv), _ptr(dtda), _ptr(A), _ptr(B), _ptr(C), _ptr(s0), _ptr(dy), _ptr(ds_final),
            _ptr(out[names[0]]), _ptr(out[names[1]]), _ptr(out["dB"]), _ptr(out["dC"]), _ptr(out["d_s0"]))
    if want_dA:
        if form != FORM_MAMBA2:
            raise ValueError("dA needs the Mamba-2 (x, dt, A) form")
        if "dA" not in out:
            out["dA"] = torch.empty_like(A)
        _need(out["dA"], "out['dA']", torch.float32, (H,), dev)
        st = lib().ssd_chunk_bwd_dA(ctypes.byref(desc), *args, _ptr(out["dA"]), _ptr(ws), wsb, _stream(stream))
        _check("ssd_chunk_bwd_dA", st)
    else:
        st = lib().ssd_chunk_bwd(ctypes.byref(desc), *args, _ptr(ws), wsb, _stream(stream))
        _check("ssd_chunk_bwd", st)
    return out


NOALLOC_SCRATCH_BYTES = 96 << 20  # SSMVJP_NOALLOC_SCRATCH_BYTES


def ssd_chunk_bwd_noalloc(xv, dtda, A, B, C, s0, dy, ds_final, *, chunk_len, out, stream=None):
    """ssd_chunk_bwd on the library's own device array instead of a workspace.

    ``out`` (required: this call allocates nothing) holds the output tensors,
    as returned by ssd_chunk_bwd.  Shapes whose workspace exceeds
    NOALLOC_SCRATCH_BYTES raise (SSMVJP_EWORKSPACE).
    """
    form = FORM_MAMBA2 if A is not None else FORM_RAW
    desc = _ssd_inputs(xv, dtda, A, B, C, s0, form, chunk_len)
    if dy is None or out is None:
        raise ValueError("dy and out are required")
    dev = xv.device
    _need(dy, "dy", xv.dtype, tuple(xv.shape), dev)
    _need(ds_final, "ds_final", torch.float32, (desc.batch, desc.nheads, desc.headdim, desc.dstate), dev)
    _check_out(out, _ssd_grad_spec(desc, xv, form), dev)
    _on_gpu(dev, xv, dtda, A, B, C, s0, dy, ds_final, *out.values())
    names = ("dx", "d_dt") if form == FORM_MAMBA2 else ("dv", "d_da")
    st = lib().ssd_chunk_bwd_noalloc(ctypes.byref(desc), _ptr(xv), _ptr(dtda), _ptr(A), _ptr(B), _ptr(C), _ptr(s0),
                                     _ptr(dy), _ptr(ds_final), _ptr(out[names[0]]), _ptr(out[names[1]]),
                                     _ptr(out["dB"]), _ptr(out["dC"]), _ptr(out["d_s0"]), _stream(stream))
    _check("ssd_chunk_bwd_noalloc", st)
    return out


def ssd_chunk_fwd_workspace(desc):
    n = ctypes.c_size_t(0)
    _check("ssd_chunk_fwd_workspace", lib().ssd_chunk_fwd_workspace(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def ssd_chunk_fwd(xv, dtda, A, B, C, s0=None, *, chunk_len=64, out=None, want_final=True, workspace=None,
                  stream=None):
    """Chunked SSD forward.  Returns dict y (like xv) and s_final [b,H,P,N] float32.

    Mamba-2 form (A given): xv = x [b,T,H,P], dtda = dt [b,T,H] (raw), B, C [b,T,G,N].
    RAW form (A None): xv = v [b,T,M,H,P], dtda = da [b,T,H], B, C [b,T,M,G,N].
    s0 None = zeros; want_final=False leaves s_final out (None).
    """
    form = FORM_MAMBA2 if A is not None else FORM_RAW
    desc = _ssd_inputs(xv, dtda, A, B, C, s0, form, chunk_len)
    b, T, H, P, N = desc.batch, desc.seqlen, desc.nheads, desc.headdim, desc.dstate
    dev, big = xv.device, xv.dtype
    if out is None:
        out = {"y": torch.empty_like(xv),
               "s_final": torch.empty((b, H, P, N), dtype=torch.float32, device=dev) if want_final else None}
    if out.get("y") is None:
        raise ValueError("out is missing 'y'")
    _need(out["y"], "out['y']", big, tuple(xv.shape), dev)
    _need(out.get("s_final"), "out['s_final']", torch.float32, (b, H, P, N), dev)
    _on_gpu(dev, xv, dtda, A, B, C, s0, out["y"], out.get("s_final"))
    ws, wsb = _workspace(ssd_chunk_fwd_workspace(desc), dev, workspace)
    st = lib().ssd_chunk_fwd(ctypes.byref(desc), _ptr(xv), _ptr(dtda), _ptr(A), _ptr(B), _ptr(C), _ptr(s0),
                             _ptr(out["y"]), _ptr(out["s_final"]), _ptr(ws), wsb, _stream(stream))
    _check("ssd_chunk_fwd", st)
    return out


class SsdCall:
    """A prepared ssd_chunk_bwd call on fixed device buffers (for repeated timing).

    ``run()`` enqueues the whole backward; ``states()`` then ``grads()`` enqueue
    its two stages separately (together they are exactly ``run()``).
    """

    def __init__(self, xv, dtda, A, B, C, s0, dy, ds_final, *, chunk_len, out=None, stream=None):
        self.form = FORM_MAMBA2 if A is not None else FORM_RAW
        self.desc = _ssd_inputs(xv, dtda, A, B, C, s0, self.form, chunk_len)
        d = self.desc
        dev = xv.device
        if dy is None:
            raise ValueError("dy is required")
        _need(dy, "dy", xv.dtype, tuple(xv.shape), dev)
        _need(ds_final, "ds_final", torch.float32, (d.batch, d.nheads, d.headdim, d.dstate), dev)
        names = ("dx", "d_dt") if self.form == FORM_MAMBA2 else ("dv", "d_da")
        if out is None:
            out = {names[0]: torch.empty_like(xv), names[1]: torch.empty_like(dtda), "dB": torch.empty_like(B),
                   "dC": torch.empty_like(C),
                   "d_s0": torch.empty((d.batch, d.nheads, d.headdim, d.dstate), dtype=torch.float32, device=dev)}
        _check_out(out, _ssd_grad_spec(d, xv, self.form), dev)
        _on_gpu(dev, xv, dtda, A, B, C, s0, dy, ds_final, *out.values())
        self.out = out
        self.ws, self.wsb = _workspace(ssd_chunk_bwd_workspace(d), dev, None)
        self.stream = stream
        p = _ptr
        self._in = (p(xv), p(dtda), p(A), p(B), p(C))
        self._s0, self._dy, self._dsf = p(s0), p(dy), p(ds_final)
        self._o = (p(out[names[0]]), p(out[names[1]]), p(out["dB"]), p(out["dC"]))
        self._ds0 = p(out["d_s0"])
        self._keep = (xv, dtda, A, B, C, s0, dy, ds_final)

    def run(self):
        st = lib().ssd_chunk_bwd(ctypes.byref(self.desc), *self._in, self._s0, self._dy, self._dsf, *self._o,
                                 self._ds0, _ptr(self.ws), self.wsb, _stream(self.stream))
        _check("ssd_chunk_bwd", st)

    def states(self):
        st = lib().ssd_chunk_bwd_states(ctypes.byref(self.desc), *self._in, self._s0, self._dy, self._dsf,
                                        self._ds0, _ptr(self.ws), self.wsb, _stream(self.stream))
        _check("ssd_chunk_bwd_states", st)

    def grads(self):
        st = lib().ssd_chunk_bwd_grads(ctypes.byref(self.desc), *self._in, self._dy, *self._o, _ptr(self.ws),
                                       self.wsb, _stream(self.stream))
        _check("ssd_chunk_bwd_grads", st)


# --------------------------------------------------------------------------- #
def delta_desc(q, v, scale):
    b, T, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    return DeltaDesc(b, T, H, HV, K, V, float(scale), 0)


def delta_rule_bwd_workspace(desc):
    n = ctypes.c_size_t(0)
    _check("delta_rule_bwd_workspace", lib().delta_rule_bwd_workspace(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def _delta_args(q, k, v, beta, g, S0, d_o, dS_final, want_dS0, out):
    if q is None or v is None or q.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be [b,T,H,K] and v [b,T,HV,V]")
    desc = delta_desc(q, v, 1.0)
    b, T, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    dev, f32 = q.device, torch.float32
    _need(q, "q", f32, (b, T, H, K), dev)
    _need(k, "k", f32, (b, T, H, K), dev)
    _need(v, "v", f32, (b, T, HV, V), dev)
    _need(beta, "beta", f32, (b, T, HV), dev)
    _need(g, "g", f32, (b, T, HV, K), dev)
    _need(S0, "S0", f32, (b, HV, K, V), dev)
    _need(d_o, "d_o", f32, (b, T, HV, V), dev)
    _need(dS_final, "dS_final", f32, (b, HV, K, V), dev)
    for name, t in (("q", q), ("k", k), ("v", v), ("beta", beta), ("g", g), ("d_o", d_o)):
        if t is None:
            raise ValueError(f"{name} is required")
    if out is None:
        out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v), dg=torch.empty_like(g),
                   dbeta=torch.empty_like(beta),
                   dS0=torch.empty((b, HV, K, V), dtype=f32, device=dev) if want_dS0 else None)
    _check_out(out, dict(dq=(f32, (b, T, H, K)), dk=(f32, (b, T, H, K)), dv=(f32, (b, T, HV, V)),
                         dg=(f32, (b, T, HV, K)), dbeta=(f32, (b, T, HV))), dev)
    _need(out.get("dS0"), "out['dS0']", f32, (b, HV, K, V), dev)
    _on_gpu(dev, q, k, v, beta, g, S0, d_o, dS_final, *out.values())
    p = _ptr
    args = (p(q), p(k), p(v), p(beta), p(g), p(S0), p(d_o), p(dS_final), p(out["dq"]), p(out["dk"]), p(out["dv"]),
            p(out["dg"]), p(out["dbeta"]), p(out.get("dS0")))
    return desc, out, args


def delta_rule_bwd(q, k, v, beta, g, S0, d_o, dS_final=None, *, scale, want_dS0=True, out=None, workspace=None,
                   stream=None):
    """KDA gated delta-rule backward (float32).  Returns dict dq, dk, dv, dg, dbeta, dS0."""
    desc, out, args = _delta_args(q, k, v, beta, g, S0, d_o, dS_final, want_dS0, out)
    desc.scale = float(scale)
    ws, wsb = _workspace(delta_rule_bwd_workspace(desc), q.device, workspace)
    st = lib().delta_rule_bwd(ctypes.byref(desc), *args, _ptr(ws), wsb, _stream(stream))
    _check("delta_rule_bwd", st)
    return out


class DeltaCall:
    """A prepared delta_rule_bwd call on fixed device buffers (for repeated timing).

    ``run()`` enqueues the whole backward; ``stage(DELTA_CKPT)``,
    ``stage(DELTA_BWD)`` and ``stage(DELTA_REDUCE)`` in that order enqueue its
    three kernels separately (together they are exactly ``run()``).
    """

    def __init__(self, q, k, v, beta, g, S0, d_o, dS_final=None, *, scale, want_dS0=True, out=None, stream=None):
        self.desc, self.out, self._args = _delta_args(q, k, v, beta, g, S0, d_o, dS_final, want_dS0, out)
        self.desc.scale = float(scale)
        self.ws, self.wsb = _workspace(delta_rule_bwd_workspace(self.desc), q.device, None)
        self.stream = stream
        self._keep = (q, k, v, beta, g, S0, d_o, dS_final)

    def stage(self, stages):
        st = lib().delta_rule_bwd_stages(ctypes.byref(self.desc), int(stages), *self._args, _ptr(self.ws), self.wsb,
                                         _stream(self.stream))
        _check("delta_rule_bwd_stages", st)

    def run(self):
        self.stage(DELTA_ALL)


# --------------------------------------------------------------------------- #
class _Here:
    """The current stream of the current device: nothing to switch."""

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_HERE = _Here()


def _scope(dev, stream):
    """Where a call's launches and allocations go: the given stream, or the current
    stream of the tensors' device (which need not be the current device)."""
    if dev.type != "cuda":
        raise ValueError("inputs must be GPU tensors (there is no CPU path)")
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
        return torch.cuda.stream(stream)
    return _HERE if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _required(**tensors):
    for name, t in tensors.items():
        if t is None:
            raise ValueError(f"{name} is required")


def _fits(t, dtype, shape):
    """What _need checks, as a truth value: these calls are made once per token, and a
    check that passes must cost no more than the comparison."""
    return t.dtype is dtype and t.shape == shape and t.is_contiguous()


def _query(name, desc):
    n = ctypes.c_size_t(0)
    _check(name, getattr(lib(), name)(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


_entry = {}  # entry points by name, looked up once


def _enqueue(name, desc, args, dev, workspace, needs=True):
    """Workspace and launch of one of the entry points that end in (workspace, bytes, stream).
    needs=False: the call takes a workspace only in the debug finiteness mode, and says so."""
    fn = _entry.get(name)
    if fn is None:
        fn = _entry[name] = getattr(lib(), name)
    d = ctypes.byref(desc)
    ptrs = [None if t is None else t.data_ptr() for t in args]
    stream = torch._C._cuda_getCurrentRawStream(dev.index)
    st = EWORKSPACE
    if not needs and workspace is None:
        st = fn(d, *ptrs, None, 0, stream)
    if st == EWORKSPACE:
        ws, wsb = _workspace(_query(name + "_workspace", desc), dev, workspace)
        st = fn(d, *ptrs, None if ws is None else ws.data_ptr(), wsb, stream)
    if st != OK:
        raise SsmVjpError(name, st)


def delta_chunk_desc(q, v, scale, seq_offsets=None):
    n, T, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    packed = seq_offsets is not None
    return DeltaChunkDesc(seq_offsets.shape[0] - 1 if packed else n, T, H, HV, K, V, float(scale), _dtype_code(q),
                          int(packed), 0)


def _delta_chunk_inputs(q, k, v, beta, g, S0, scale, seq_offsets):
    _required(q=q, k=k, v=v, beta=beta, g=g)
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be [b,T,H,K] and v [b,T,HV,V]")
    n, T, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    dev, big, f32 = q.device, q.dtype, torch.float32
    if seq_offsets is not None:
        if n != 1:
            raise ValueError("packed sequences (seq_offsets given) need token tensors [1,T,...]")
        if seq_offsets.dim() != 1 or seq_offsets.shape[0] < 1:
            raise ValueError("seq_offsets must be [sequences + 1]")
        _need(seq_offsets, "seq_offsets", torch.int32, tuple(seq_offsets.shape), dev)
    desc = delta_chunk_desc(q, v, scale, seq_offsets)
    _need(q, "q", big, (n, T, H, K), dev)
    _need(k, "k", big, (n, T, H, K), dev)
    _need(v, "v", big, (n, T, HV, V), dev)
    _need(beta, "beta", f32, (n, T, HV), dev)
    _need(g, "g", f32, (n, T, HV), dev)
    _need(S0, "S0", f32, (desc.batch, HV, K, V), dev)
    return desc


def delta_chunk_fwd(q, k, v, beta, g, S0=None, *, scale, seq_offsets=None, want_final=True, out=None, workspace=None,
                    stream=None):
    """Gated delta rule with one log gate per value head.  Returns dict o (like v) and
    S_final [b,HV,K,V] float32 (None with want_final=False).

    q, k [b,T,H,K] and v [b,T,HV,V] float32 or bfloat16 (all the same), beta, g [b,T,HV]
    and S0 [b,HV,K,V] (None = zeros) float32.  With seq_offsets (int32 [n+1] on the GPU,
    ascending) the token tensors are [1,T,...], sequence i owns the tokens
    seq_offsets[i] .. seq_offsets[i+1]-1, and the states are [n,HV,K,V]; rows of o that no
    sequence owns are left as they were.
    """
    desc = _delta_chunk_inputs(q, k, v, beta, g, S0, scale, seq_offsets)
    dev = q.device
    with _scope(dev, stream):
        if out is None:
            shape = (desc.batch, desc.nv_heads, desc.dk, desc.dv)
            out = {"o": torch.empty_like(v),
                   "S_final": torch.empty(shape, dtype=torch.float32, device=dev) if want_final else None}
        if out.get("o") is None:
            raise ValueError("out is missing 'o'")
        S_final = out.get("S_final")
        _need(out["o"], "out['o']", v.dtype, tuple(v.shape), dev)
        _need(S_final, "out['S_final']", torch.float32, (desc.batch, desc.nv_heads, desc.dk, desc.dv), dev)
        _on_gpu(dev, q, k, v, beta, g, S0, seq_offsets, out["o"], S_final)
        _enqueue("delta_chunk_fwd", desc, (q, k, v, beta, g, S0, seq_offsets, out["o"], S_final), dev, workspace)
    return out


def delta_chunk_bwd(q, k, v, beta, g, S0, d_o, dS_final=None, *, scale, seq_offsets=None, want_dS0=True, out=None,
                    workspace=None, stream=None):
    """Gradients of delta_chunk_fwd (bfloat16 q, k, v, d_o).  Returns dict dq, dk (like q), dv (like v),
    dbeta, dg (float32) and dS0 [b,HV,K,V] float32 (None with want_dS0=False).

    Arguments as for delta_chunk_fwd; d_o like v, dS_final [b,HV,K,V] float32 (None = zeros).
    Rows that no sequence of a packed call owns are left as they were.
    There is no float32 form (EUNSUPPORTED): delta_rule_bwd has it for equal sequences, K = 128
    and V a multiple of 32, with g repeated over the key channels and dg summed over them.
    """
    desc = _delta_chunk_inputs(q, k, v, beta, g, S0, scale, seq_offsets)
    _required(d_o=d_o)
    dev, big, f32 = q.device, q.dtype, torch.float32
    state = (desc.batch, desc.nv_heads, desc.dk, desc.dv)
    _need(d_o, "d_o", big, tuple(v.shape), dev)
    _need(dS_final, "dS_final", f32, state, dev)
    with _scope(dev, stream):
        if out is None:
            out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
                       dbeta=torch.empty_like(beta), dg=torch.empty_like(g),
                       dS0=torch.empty(state, dtype=f32, device=dev) if want_dS0 else None)
        _check_out(out, dict(dq=(big, tuple(q.shape)), dk=(big, tuple(q.shape)), dv=(big, tuple(v.shape)),
                             dbeta=(f32, tuple(beta.shape)), dg=(f32, tuple(g.shape))), dev)
        dS0 = out.get("dS0")
        _need(dS0, "out['dS0']", f32, state, dev)
        args = (q, k, v, beta, g, S0, d_o, dS_final, seq_offsets, out["dq"], out["dk"], out["dv"], out["dbeta"],
                out["dg"], dS0)
        _on_gpu(dev, *args)
        _enqueue("delta_chunk_bwd", desc, args, dev, workspace)
    return out


def delta_step(q, k, v, beta, g, state, *, scale, slots=None, out=None, workspace=None, stream=None):
    """One token of the gated delta rule per request; updates ``state`` in place and returns o.

    q, k [b,H,K] and v, o [b,HV,V] float32 or bfloat16 (all the same), beta [b,HV] float32,
    g float32 [b,HV] (one log gate per head) or [b,HV,K] (per key channel), state
    [n,HV,K,V] float32.  slots (int32 [b] on the GPU, None = request i uses state i): a
    request whose slot is outside [0,n) or was named by an earlier request gets zeros and
    touches no state.
    """
    if q is None or k is None or v is None or beta is None or g is None or state is None:
        _required(q=q, k=k, v=v, beta=beta, g=g, state=state)
    if q.dim() != 3 or v.dim() != 3 or state.dim() != 4 or g.dim() not in (2, 3):
        raise ValueError("q must be [b,H,K], v [b,HV,V], g [b,HV] or [b,HV,K] and state [n,HV,K,V]")
    b, H, K = q.shape
    HV, V = v.shape[1], v.shape[2]
    dev, big, f32 = q.device, q.dtype, torch.float32
    per_key = g.dim() == 3
    qs, hs, gs, ss = (b, H, K), (b, HV), ((b, HV, K) if per_key else (b, HV)), (state.shape[0], HV, K, V)
    if not (_fits(q, big, qs) and _fits(k, big, qs) and _fits(v, big, (b, HV, V)) and _fits(beta, f32, hs)
            and _fits(g, f32, gs) and _fits(state, f32, ss) and (slots is None or _fits(slots, torch.int32, (b,)))):
        for name, t, dtype, shape in (("q", q, big, qs), ("k", k, big, qs), ("v", v, big, (b, HV, V)), ("beta", beta, f32, hs),
                                      ("g", g, f32, gs), ("state", state, f32, ss), ("slots", slots, torch.int32, (b,))):
            _need(t, name, dtype, shape, dev)
    desc = DeltaStepDesc(b, state.shape[0], H, HV, K, V, float(scale), _dtype_code(q),
                         GATE_PER_KEY if per_key else GATE_PER_HEAD, 0)
    with _scope(dev, stream):
        if out is None:
            o = torch.empty_like(v)
        else:
            o = out
            _need(o, "out", big, (b, HV, V), dev)
        args = (q, k, v, beta, g, state, slots, o)
        _on_gpu(dev, *args)
        _enqueue("delta_step", desc, args, dev, workspace, needs=False)
    return o


# --------------------------------------------------------------------------- #
def norm_desc(x, weight, eps):
    """x [..., D] with weight None or [D], or x [..., G, D] with weight [G, D]."""
    shape = x.shape
    if len(shape) < 1:
        raise ValueError("x must have at least one axis")
    D = shape[-1]
    G = 1
    if weight is not None:
        wdim = weight.dim()
        if wdim == 2:
            if len(shape) < 2:
                raise ValueError("a weight [G,D] needs x [...,G,D]")
            G = shape[-2]
        elif wdim != 1:
            raise ValueError("weight must be [D] or [G,D]")
    if D == 0 or G == 0:
        raise ValueError("x has an empty last axis")
    return NormDesc(x.numel() // (G * D), G, D, eps, _dtype_code(x))


def _norm_wshape(desc, weight):
    return (desc.groups, desc.dim) if weight.dim() == 2 else (desc.dim,)


def layer_norm_fwd(x, weight=None, bias=None, *, eps=1e-5, want_ckpt8=False, out=None, workspace=None, stream=None):
    """Layer norm of the last axis.  Returns dict y (like x), mean and rstd (float32, x's shape
    without the last axis) and, with want_ckpt8=True, x8 (int8, like x) and x8_scale
    [..., ceil(D/64)]: the 8-bit form of x that layer_norm_bwd can read in its place.

    x [..., D] float32 or bfloat16; weight and bias float32 [D], or [G,D] for x [..., G, D]
    (every head its own), or None.
    """
    if x is None:
        _required(x=x)
    if weight is None and bias is not None:
        raise ValueError("a bias needs a weight")
    desc = norm_desc(x, weight, eps)
    dev, f32 = x.device, torch.float32
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if weight is not None:
        ws = _norm_wshape(desc, weight)
        for name, t in (("weight", weight), ("bias", bias)):
            if t is not None and not _fits(t, f32, ws):
                _need(t, name, f32, ws, dev)
    stat = x.shape[:-1]
    with _scope(dev, stream):
        if out is None:
            mean = x.new_empty(stat, dtype=f32)
            out = {"y": torch.empty_like(x), "mean": mean, "rstd": torch.empty_like(mean)}
            if want_ckpt8:
                out["x8"] = x.new_empty(x.shape, dtype=torch.int8)
                out["x8_scale"] = x.new_empty(stat + ((desc.dim + 63) // 64,), dtype=f32)
        else:
            spec = {"y": (x.dtype, x.shape), "mean": (f32, stat), "rstd": (f32, stat)}
            if want_ckpt8:
                spec.update(x8=(torch.int8, x.shape), x8_scale=(f32, stat + ((desc.dim + 63) // 64,)))
            _check_out(out, spec, dev)
        x8, x8s = (out["x8"], out["x8_scale"]) if want_ckpt8 else (None, None)
        args = (x, weight, bias, out["y"], out["mean"], out["rstd"], x8, x8s)
        _on_gpu(dev, *args)
        _enqueue("layer_norm_fwd", desc, args, dev, workspace, needs=False)
    return out


def layer_norm_bwd(dy, x, mean, rstd, weight=None, *, ckpt8=None, out=None, workspace=None, stream=None):
    """Gradients of layer_norm_fwd.  Returns dict dx (like dy), dweight and dbias (float32, like
    weight; None without a weight).

    x is the forward's input, or None with ckpt8=(x8, x8_scale) from a forward with
    want_ckpt8=True; mean and rstd are the forward's.
    """
    if dy is None or mean is None or rstd is None:
        _required(dy=dy, mean=mean, rstd=rstd)
    if (x is None) == (ckpt8 is None):
        raise ValueError("exactly one of x and ckpt8 must be given")
    desc = norm_desc(dy, weight, 0.0)
    dev, f32 = dy.device, torch.float32
    stat = dy.shape[:-1]
    x8, x8s = (None, None) if ckpt8 is None else ckpt8
    if ckpt8 is not None:
        _required(x8=x8, x8_scale=x8s)
    ws = None if weight is None else _norm_wshape(desc, weight)
    shape, blocks = dy.shape, None if x8 is None else stat + ((desc.dim + 63) // 64,)
    if not (_fits(dy, dy.dtype, shape) and _fits(mean, f32, stat) and _fits(rstd, f32, stat)
            and (x is None or _fits(x, dy.dtype, shape)) and (weight is None or _fits(weight, f32, ws))
            and (x8 is None or (_fits(x8, torch.int8, shape) and _fits(x8s, f32, blocks)))):
        for name, t, dtype, want in (("dy", dy, dy.dtype, shape), ("x", x, dy.dtype, shape), ("mean", mean, f32, stat),
                                     ("rstd", rstd, f32, stat), ("x8", x8, torch.int8, shape),
                                     ("x8_scale", x8s, f32, blocks), ("weight", weight, f32, ws)):
            _need(t, name, dtype, want, dev)
    with _scope(dev, stream):
        if out is None:
            out = {"dx": torch.empty_like(dy), "dweight": None if weight is None else torch.empty_like(weight),
                   "dbias": None if weight is None else torch.empty_like(weight)}
        else:
            spec = {"dx": (dy.dtype, dy.shape)}
            if weight is not None:
                spec.update(dweight=(f32, ws), dbias=(f32, ws))
            _check_out(out, spec, dev)
        dw, db = (out["dweight"], out["dbias"]) if weight is not None else (None, None)
        args = (dy, x, x8, x8s, mean, rstd, weight, out["dx"], dw, db)
        _on_gpu(dev, *args)
        _enqueue("layer_norm_bwd", desc, args, dev, workspace)
    return out
