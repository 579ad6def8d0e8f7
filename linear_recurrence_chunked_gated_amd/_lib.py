"""ctypes binding of libsf_gdn.so (the C ABI in include/sf_gdn.h).

Argument marshalling only: torch provides device memory and the stream, and
every step of the computation runs in the library's HIP kernels.  There is no
fallback: if the library is missing or fails, calls raise.  The decoding calls,
the norms, linear attention with a decay and the rotation, whose kernels can be
shorter than their marshalling in Python, check and call through the native
module _calls (csrc/sf_gdn_calls.cpp) on the same entry points.

Every call takes ``stream``, the current one when None.  On another, its
kernels are in no order with the current stream's work but what the caller sets
up; outputs that it makes are that stream's memory, marked as used by the
current one too.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsf_gdn.so")

SF_OK, SF_ERR_INVALID_ARG, SF_ERR_UNSUPPORTED, SF_ERR_WORKSPACE, SF_ERR_HIP = range(5)
SF_DTYPE_F32, SF_DTYPE_BF16 = 0, 1

_DTYPES = {torch.float32: SF_DTYPE_F32, torch.bfloat16: SF_DTYPE_BF16}

# Every function the header declares, with (restype, argtypes).
_vp, _cvp, _fp = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
_sz = ctypes.c_size_t


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("Dk", ctypes.c_int), ("Dv", ctypes.c_int), ("dtype", ctypes.c_int),
                ("seg_blocks", ctypes.c_int)]


class ConvShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("C", ctypes.c_int),
                ("W", ctypes.c_int), ("dtype", ctypes.c_int), ("act", ctypes.c_int)]


class StepShape(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int), ("n_tok", ctypes.c_int), ("n_slots", ctypes.c_int),
                ("Hk", ctypes.c_int), ("Hv", ctypes.c_int), ("Dk", ctypes.c_int),
                ("Dv", ctypes.c_int), ("dtype", ctypes.c_int), ("update", ctypes.c_int),
                ("q_stride", ctypes.c_longlong), ("k_stride", ctypes.c_longlong),
                ("v_stride", ctypes.c_longlong)]


class ConvStepShape(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int), ("n_tok", ctypes.c_int), ("n_slots", ctypes.c_int),
                ("C", ctypes.c_int), ("W", ctypes.c_int), ("dtype", ctypes.c_int),
                ("act", ctypes.c_int), ("update", ctypes.c_int), ("x_stride", ctypes.c_longlong)]


class GatedNormShape(ctypes.Structure):
    _fields_ = [("N", ctypes.c_longlong), ("H", ctypes.c_int), ("D", ctypes.c_int),
                ("dtype", ctypes.c_int), ("act", ctypes.c_int), ("eps", ctypes.c_float),
                ("scale", ctypes.c_float), ("x_stride", ctypes.c_longlong),
                ("gate_stride", ctypes.c_longlong)]


class ResidualNormShape(ctypes.Structure):
    _fields_ = [("N", ctypes.c_longlong), ("C", ctypes.c_int), ("dtype", ctypes.c_int),
                ("eps", ctypes.c_float), ("scale", ctypes.c_float)]


class DecayShape(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int), ("n_tok", ctypes.c_int), ("Hk", ctypes.c_int),
                ("Hv", ctypes.c_int), ("Dk", ctypes.c_int), ("Dv", ctypes.c_int),
                ("dtype", ctypes.c_int), ("scale", ctypes.c_float),
                ("q_stride", ctypes.c_longlong), ("k_stride", ctypes.c_longlong),
                ("v_stride", ctypes.c_longlong)]


class DecayStepShape(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int), ("n_tok", ctypes.c_int), ("n_slots", ctypes.c_int),
                ("Hk", ctypes.c_int), ("Hv", ctypes.c_int), ("Dk", ctypes.c_int),
                ("Dv", ctypes.c_int), ("dtype", ctypes.c_int), ("update", ctypes.c_int),
                ("scale", ctypes.c_float), ("q_stride", ctypes.c_longlong),
                ("k_stride", ctypes.c_longlong), ("v_stride", ctypes.c_longlong)]


class RotaryShape(ctypes.Structure):
    _fields_ = [("N", ctypes.c_longlong), ("T", ctypes.c_longlong), ("Hq", ctypes.c_int),
                ("Hk", ctypes.c_int), ("D", ctypes.c_int), ("F", ctypes.c_int),
                ("dtype", ctypes.c_int), ("neighbours", ctypes.c_int), ("first", ctypes.c_int),
                ("eps", ctypes.c_float), ("q_scale", ctypes.c_float), ("k_scale", ctypes.c_float),
                ("q_stride", ctypes.c_longlong), ("k_stride", ctypes.c_longlong)]


SIGNATURES = {
    "sf_gdn_chunk_fwd_workspace_size": (ctypes.c_int, [ctypes.POINTER(Shape), ctypes.POINTER(_sz)]),
    "sf_gdn_chunk_bwd_workspace_size": (ctypes.c_int, [ctypes.POINTER(Shape), ctypes.POINTER(_sz)]),
    "sf_gdn_chunk_fwd": (ctypes.c_int, [ctypes.POINTER(Shape)] + [_vp] * 8 + [_vp, _sz, _vp]),
    "sf_gdn_chunk_bwd": (ctypes.c_int, [ctypes.POINTER(Shape)] + [_vp] * 14 + [_vp, _sz, _vp]),
    "sf_gdn_chunk_fwd_noalloc": (ctypes.c_int, [ctypes.POINTER(Shape)] + [_vp] * 8 + [_vp]),
    "sf_gdn_chunk_saved_size": (ctypes.c_int, [ctypes.POINTER(Shape), ctypes.POINTER(_sz)]),
    "sf_gdn_segment_plan": (ctypes.c_int, [ctypes.POINTER(Shape), ctypes.POINTER(ctypes.c_int),
                                           ctypes.POINTER(ctypes.c_int)]),
    "sf_gdn_chunk_fwd_save": (ctypes.c_int, [ctypes.POINTER(Shape)] + [_vp] * 9 + [_sz, _vp, _sz, _vp]),
    "sf_gdn_chunk_bwd_saved": (ctypes.c_int, [ctypes.POINTER(Shape)] + [_vp] * 6 + [_sz] + [_vp] * 8
                               + [_vp, _sz, _vp]),
    "sf_gdn_chunk_fwd_split": (ctypes.c_int, [ctypes.POINTER(Shape)] + [_vp] * 9
                               + [_sz, _vp, _sz, ctypes.c_int, _vp]),
    "sf_gdn_chunk_bwd_saved_split": (ctypes.c_int, [ctypes.POINTER(Shape)] + [_vp] * 6 + [_sz]
                                     + [_vp] * 8 + [_vp, _sz, ctypes.c_int, _vp]),
    "sf_gdn_shortconv_fwd": (ctypes.c_int, [ctypes.POINTER(ConvShape)] + [_vp] * 6),
    "sf_gdn_shortconv_bwd_workspace_size": (ctypes.c_int, [ctypes.POINTER(ConvShape),
                                                           ctypes.POINTER(_sz)]),
    "sf_gdn_shortconv_bwd": (ctypes.c_int, [ctypes.POINTER(ConvShape)] + [_vp] * 9 + [_sz, _vp]),
    "sf_gdn_recurrent_step": (ctypes.c_int, [ctypes.POINTER(StepShape)] + [_vp] * 10),
    "sf_gdn_shortconv_step": (ctypes.c_int, [ctypes.POINTER(ConvStepShape)] + [_vp] * 7),
    "sf_gdn_gated_norm_fwd": (ctypes.c_int, [ctypes.POINTER(GatedNormShape)] + [_vp] * 5),
    "sf_gdn_gated_norm_bwd_workspace_size": (ctypes.c_int, [ctypes.POINTER(GatedNormShape),
                                                            ctypes.POINTER(_sz)]),
    "sf_gdn_gated_norm_bwd": (ctypes.c_int, [ctypes.POINTER(GatedNormShape)] + [_vp] * 8
                              + [_sz, _vp]),
    "sf_gdn_residual_norm_fwd": (ctypes.c_int, [ctypes.POINTER(ResidualNormShape)] + [_vp] * 7),
    "sf_gdn_residual_norm_bwd_workspace_size": (ctypes.c_int, [ctypes.POINTER(ResidualNormShape),
                                                               ctypes.POINTER(_sz)]),
    "sf_gdn_residual_norm_bwd": (ctypes.c_int, [ctypes.POINTER(ResidualNormShape)] + [_vp] * 11
                                 + [_sz, _vp]),
    "sf_gdn_decay_chunk_fwd_workspace_size": (ctypes.c_int, [ctypes.POINTER(DecayShape),
                                                             ctypes.POINTER(_sz)]),
    "sf_gdn_decay_chunk_bwd_workspace_size": (ctypes.c_int, [ctypes.POINTER(DecayShape),
                                                             ctypes.POINTER(_sz)]),
    "sf_gdn_decay_chunk_fwd": (ctypes.c_int, [ctypes.POINTER(DecayShape)] + [_vp] * 9 + [_sz, _vp]),
    "sf_gdn_decay_chunk_bwd": (ctypes.c_int, [ctypes.POINTER(DecayShape)] + [_vp] * 13 + [_sz, _vp]),
    "sf_gdn_decay_step": (ctypes.c_int, [ctypes.POINTER(DecayStepShape)] + [_vp] * 9),
    "sf_gdn_qk_norm_rotary_fwd": (ctypes.c_int, [ctypes.POINTER(RotaryShape)] + [_vp] * 9),
    "sf_gdn_qk_norm_rotary_bwd_workspace_size": (ctypes.c_int, [ctypes.POINTER(RotaryShape),
                                                                ctypes.POINTER(_sz)]),
    "sf_gdn_qk_norm_rotary_bwd": (ctypes.c_int, [ctypes.POINTER(RotaryShape)] + [_vp] * 13
                                  + [_sz, _vp]),
    "sf_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "sf_last_error_message": (ctypes.c_char_p, []),
    "sf_gdn_version": (ctypes.c_char_p, []),
    "sf_gdn_profile_begin": (ctypes.c_int, [ctypes.c_int]),
    "sf_gdn_profile_end": (ctypes.c_int, []),
    "sf_gdn_profile_kernel_count": (ctypes.c_int, []),
    "sf_gdn_profile_kernel": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(ctypes.c_char_p),
                                             ctypes.POINTER(ctypes.c_longlong),
                                             ctypes.POINTER(ctypes.c_double)]),
}

_lib = None


# Launch groups of a chunk call (sf_gdn_chunk_fwd_split, sf_gdn_chunk_bwd_saved_split).
PHASE_ALL, PHASE_BEGIN, PHASE_END = 0, 1, 2


class GDNError(RuntimeError):
    def __init__(self, status, where, msg):
        super().__init__("%s: %s (%s)" % (where, msg, status_string(status)))
        self.status = status


def load():
    """Load the library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libsf_gdn.so is not built; run "
                           "`python -m linear_recurrence_chunked_gated_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_string(status):
    return load().sf_status_string(int(status)).decode()


def _check(status, where):
    if status != SF_OK:
        raise GDNError(status, where, load().sf_last_error_message().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def used_on(stream, *tensors):
    """Mark tensors that this package allocated on the current stream as in
    use by ``stream`` when kernels run there as well, so that the caching
    allocator does not hand their memory to current-stream work before those
    are done (tensor.record_stream).  No-op for the current stream."""
    if stream is None or stream == torch.cuda.current_stream(stream.device):
        return
    for t in tensors:
        if t is not None and t.numel() > 0:
            t.record_stream(stream)


def new_on(stream, make, *args, **kw):
    """make(*args, **kw), a new tensor (or None), for kernels on ``stream``
    (None: the current one).

    A block of the current stream's memory may have been freed with work of
    that stream on it still pending, which ``stream`` does not wait for, so the
    tensor is made with ``stream`` the current one (a fill then runs there
    too), and marked as used by the caller's current stream, where it may be
    read and freed as well."""
    if stream is None:
        return make(*args, **kw)
    here = torch.cuda.current_stream(stream.device)
    if stream == here:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        t = make(*args, **kw)
    if t is not None and t.numel() > 0:
        t.record_stream(here)
    return t


def make_shape(B, T, H, Dk, Dv, dtype, seg_blocks=0):
    if isinstance(dtype, torch.dtype):
        if dtype not in _DTYPES:
            raise TypeError("q/k/v must be bfloat16 or float32, got %s" % dtype)
        dtype = _DTYPES[dtype]
    return Shape(B, T, H, Dk, Dv, dtype, seg_blocks)


def workspace_bytes(shape, backward=False):
    n = ctypes.c_size_t(0)
    fn = load().sf_gdn_chunk_bwd_workspace_size if backward else load().sf_gdn_chunk_fwd_workspace_size
    _check(fn(ctypes.byref(shape), ctypes.byref(n)), "workspace_size")
    return n.value


def segment_plan(shape):
    """(blocks per segment, segments) of the in-chunk scan for `shape`."""
    L, P = ctypes.c_int(0), ctypes.c_int(0)
    _check(load().sf_gdn_segment_plan(ctypes.byref(shape), ctypes.byref(L), ctypes.byref(P)),
           "segment_plan")
    return L.value, P.value


def alloc_workspace(nbytes, device):
    """A 256-byte aligned uint8 view of at least nbytes (None when 0)."""
    if nbytes == 0:
        return None
    raw = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    off = (-raw.data_ptr()) % 256
    return raw[off:off + nbytes]


def _need(t, name, dtype, shape, device):
    if t is None:
        raise ValueError("%s is required" % name)
    if t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def saved_bytes(shape):
    n = ctypes.c_size_t(0)
    _check(load().sf_gdn_chunk_saved_size(ctypes.byref(shape), ctypes.byref(n)), "saved_size")
    return n.value


def chunk_fwd(q, k, v, alpha, beta, S_in=None, o=None, S_out=None, seg_blocks=0,
              workspace=None, stream=None, saved=None, phase=PHASE_ALL):
    """sf_gdn_chunk_fwd on torch tensors.  Returns (o, S_out).

    With ``saved`` (a uint8 tensor of at least ``saved_bytes`` bytes, 256-byte
    aligned, or True to allocate one) the saving forward runs and the return
    value is (o, S_out, saved).  ``phase`` selects one launch group
    (sf_gdn_chunk_fwd_split): PHASE_BEGIN then PHASE_END with the same
    arguments and workspace equals one PHASE_ALL call."""
    B, T, H, Dk = q.shape
    Dv = v.shape[3]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    _need(q, "q", q.dtype, (B, T, H, Dk), dev)
    _need(k, "k", q.dtype, (B, T, H, Dk), dev)
    _need(v, "v", q.dtype, (B, T, H, Dv), dev)
    _need(alpha, "alpha", torch.float32, (B, T, H), dev)
    _need(beta, "beta", torch.float32, (B, T, H), dev)
    if S_in is not None:
        _need(S_in, "S_in", torch.float32, (B, H, Dv, Dk), dev)
    if o is None:
        o = new_on(stream, torch.empty, (B, T, H, Dv), dtype=q.dtype, device=dev)
    _need(o, "o", q.dtype, (B, T, H, Dv), dev)
    if S_out is None:
        S_out = new_on(stream, torch.empty, (B, H, Dv, Dk), dtype=torch.float32, device=dev)
    _need(S_out, "S_out", torch.float32, (B, H, Dv, Dk), dev)
    shape = make_shape(B, T, H, Dk, Dv, q.dtype, seg_blocks)
    need = workspace_bytes(shape)
    if workspace is None or workspace.numel() < need:
        workspace = new_on(stream, alloc_workspace, need, dev)
    wsn = ctypes.c_size_t(0 if workspace is None else workspace.numel())
    if saved is True:
        n = saved_bytes(shape)
        saved = (new_on(stream, alloc_workspace, n, dev) if n else
                 torch.empty(0, dtype=torch.uint8, device=dev))
    if phase != PHASE_ALL:
        st = load().sf_gdn_chunk_fwd_split(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v),
                                           _ptr(alpha), _ptr(beta), _ptr(S_in), _ptr(o),
                                           _ptr(S_out), _ptr(saved),
                                           ctypes.c_size_t(0 if saved is None else saved.numel()),
                                           _ptr(workspace), wsn, int(phase), _stream(stream))
        _check(st, "sf_gdn_chunk_fwd_split")
        return (o, S_out) if saved is None else (o, S_out, saved)
    if saved is None:
        st = load().sf_gdn_chunk_fwd(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                                     _ptr(beta), _ptr(S_in), _ptr(o), _ptr(S_out),
                                     _ptr(workspace), wsn, _stream(stream))
        _check(st, "sf_gdn_chunk_fwd")
        return o, S_out
    st = load().sf_gdn_chunk_fwd_save(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                                      _ptr(beta), _ptr(S_in), _ptr(o), _ptr(S_out), _ptr(saved),
                                      ctypes.c_size_t(0 if saved is None else saved.numel()),
                                      _ptr(workspace), wsn, _stream(stream))
    _check(st, "sf_gdn_chunk_fwd_save")
    return o, S_out, saved


def chunk_fwd_noalloc(q, k, v, alpha, beta, S_in=None, o=None, S_out=None, seg_blocks=0,
                      stream=None):
    """sf_gdn_chunk_fwd_noalloc on torch tensors: the forward with the
    library's static workspace.  o and S_out must be preallocated by the
    caller when nothing may be allocated here.  Returns (o, S_out)."""
    B, T, H, Dk = q.shape
    Dv = v.shape[3]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    _need(q, "q", q.dtype, (B, T, H, Dk), dev)
    _need(k, "k", q.dtype, (B, T, H, Dk), dev)
    _need(v, "v", q.dtype, (B, T, H, Dv), dev)
    _need(alpha, "alpha", torch.float32, (B, T, H), dev)
    _need(beta, "beta", torch.float32, (B, T, H), dev)
    if S_in is not None:
        _need(S_in, "S_in", torch.float32, (B, H, Dv, Dk), dev)
    if o is None:
        o = new_on(stream, torch.empty, (B, T, H, Dv), dtype=q.dtype, device=dev)
    _need(o, "o", q.dtype, (B, T, H, Dv), dev)
    if S_out is None:
        S_out = new_on(stream, torch.empty, (B, H, Dv, Dk), dtype=torch.float32, device=dev)
    _need(S_out, "S_out", torch.float32, (B, H, Dv, Dk), dev)
    shape = make_shape(B, T, H, Dk, Dv, q.dtype, seg_blocks)
    st = load().sf_gdn_chunk_fwd_noalloc(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v),
                                         _ptr(alpha), _ptr(beta), _ptr(S_in), _ptr(o),
                                         _ptr(S_out), _stream(stream))
    _check(st, "sf_gdn_chunk_fwd_noalloc")
    return o, S_out


def chunk_bwd(q, k, v, alpha, beta, S_in, dO, dS_out=None, grads=None, seg_blocks=0,
              workspace=None, stream=None, saved=None, phase=PHASE_ALL):
    """sf_gdn_chunk_bwd on torch tensors (sf_gdn_chunk_bwd_saved when
    ``saved`` holds the buffer of a saving forward; S_in is then unused).
    ``phase`` selects one launch group of the saved backward
    (sf_gdn_chunk_bwd_saved_split).

    Returns (dq, dk, dv, dalpha, dbeta, dS_in).  ``grads`` may supply
    preallocated outputs in that order (dS_in may be None there)."""
    B, T, H, Dk = q.shape
    Dv = v.shape[3]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    for t, n, dt, shp in ((q, "q", q.dtype, (B, T, H, Dk)), (k, "k", q.dtype, (B, T, H, Dk)),
                          (v, "v", q.dtype, (B, T, H, Dv)), (dO, "dO", q.dtype, (B, T, H, Dv)),
                          (alpha, "alpha", torch.float32, (B, T, H)),
                          (beta, "beta", torch.float32, (B, T, H))):
        _need(t, n, dt, shp, dev)
    if S_in is not None and saved is None:
        _need(S_in, "S_in", torch.float32, (B, H, Dv, Dk), dev)
    if dS_out is not None:
        _need(dS_out, "dS_out", torch.float32, (B, H, Dv, Dk), dev)
    if grads is None:
        grads = [new_on(stream, torch.empty_like, t) for t in (q, k, v, alpha, beta)]
        grads.append(new_on(stream, torch.empty, (B, H, Dv, Dk), dtype=torch.float32, device=dev))
    dq, dk, dv, da, db, dS_in = grads
    shape = make_shape(B, T, H, Dk, Dv, q.dtype, seg_blocks)
    need = workspace_bytes(shape, backward=True)
    if workspace is None or workspace.numel() < need:
        workspace = new_on(stream, alloc_workspace, need, dev)
    wsn = ctypes.c_size_t(0 if workspace is None else workspace.numel())
    if phase != PHASE_ALL:
        if saved is None:
            raise ValueError("the split backward needs the saved buffer of a saving forward")
        st = load().sf_gdn_chunk_bwd_saved_split(
            ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(saved),
            ctypes.c_size_t(saved.numel()), _ptr(dO), _ptr(dS_out), _ptr(dq), _ptr(dk), _ptr(dv),
            _ptr(da), _ptr(db), _ptr(dS_in), _ptr(workspace), wsn, int(phase), _stream(stream))
        _check(st, "sf_gdn_chunk_bwd_saved_split")
    elif saved is None:
        st = load().sf_gdn_chunk_bwd(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                                     _ptr(beta), _ptr(S_in), _ptr(dO), _ptr(dS_out), _ptr(dq),
                                     _ptr(dk), _ptr(dv), _ptr(da), _ptr(db), _ptr(dS_in),
                                     _ptr(workspace), wsn, _stream(stream))
        _check(st, "sf_gdn_chunk_bwd")
    else:
        st = load().sf_gdn_chunk_bwd_saved(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v),
                                           _ptr(alpha), _ptr(beta), _ptr(saved),
                                           ctypes.c_size_t(saved.numel()), _ptr(dO), _ptr(dS_out),
                                           _ptr(dq), _ptr(dk), _ptr(dv), _ptr(da), _ptr(db),
                                           _ptr(dS_in), _ptr(workspace), wsn, _stream(stream))
        _check(st, "sf_gdn_chunk_bwd_saved")
    return dq, dk, dv, da, db, dS_in


def conv_shape(B, T, C, W, dtype, act=0):
    if isinstance(dtype, torch.dtype):
        if dtype not in _DTYPES:
            raise TypeError("x must be bfloat16 or float32, got %s" % dtype)
        dtype = _DTYPES[dtype]
    return ConvShape(B, T, C, W, dtype, int(act))


def shortconv_bwd_workspace_bytes(shape):
    n = ctypes.c_size_t(0)
    _check(load().sf_gdn_shortconv_bwd_workspace_size(ctypes.byref(shape), ctypes.byref(n)),
           "shortconv_bwd_workspace_size")
    return n.value


def shortconv_fwd(x, w, conv_in=None, act=0, y=None, conv_out=None, want_state=True,
                  stream=None):
    """sf_gdn_shortconv_fwd on torch tensors: x [B,T,C], w [C,W] fp32,
    conv_in [B,W-1,C] or None.  Returns (y, conv_out); conv_out is None when
    want_state is False."""
    B, T, C = x.shape
    W = w.shape[1]
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    _need(x, "x", x.dtype, (B, T, C), dev)
    _need(w, "w", torch.float32, (C, W), dev)
    if conv_in is not None:
        _need(conv_in, "conv_in", x.dtype, (B, W - 1, C), dev)
    if y is None:
        y = new_on(stream, torch.empty_like, x)
    _need(y, "y", x.dtype, (B, T, C), dev)
    if want_state and conv_out is None and W > 1:
        conv_out = new_on(stream, torch.empty, (B, W - 1, C), dtype=x.dtype, device=dev)
    shape = conv_shape(B, T, C, W, x.dtype, act)
    _check(load().sf_gdn_shortconv_fwd(ctypes.byref(shape), _ptr(x), _ptr(w), _ptr(conv_in),
                                       _ptr(y), _ptr(conv_out) if W > 1 else None,
                                       _stream(stream)), "sf_gdn_shortconv_fwd")
    return y, conv_out


def shortconv_bwd(x, w, conv_in, dy, dconv_out=None, act=0, dx=None, dw=None, want_state=True,
                  workspace=None, stream=None):
    """sf_gdn_shortconv_bwd on torch tensors.  Returns (dx, dw, dconv_in)."""
    B, T, C = x.shape
    W = w.shape[1]
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU device")
    _need(x, "x", x.dtype, (B, T, C), dev)
    _need(dy, "dy", x.dtype, (B, T, C), dev)
    _need(w, "w", torch.float32, (C, W), dev)
    for t, n in ((conv_in, "conv_in"), (dconv_out, "dconv_out")):
        if t is not None:
            _need(t, n, x.dtype, (B, W - 1, C), dev)
    if dx is None:
        dx = new_on(stream, torch.empty_like, x)
    if dw is None:
        dw = new_on(stream, torch.empty_like, w)
    dci = (new_on(stream, torch.empty, (B, W - 1, C), dtype=x.dtype, device=dev)
           if want_state and W > 1 else None)
    shape = conv_shape(B, T, C, W, x.dtype, act)
    need = shortconv_bwd_workspace_bytes(shape)
    if workspace is None or workspace.numel() < need:
        workspace = new_on(stream, alloc_workspace, need, dev)
    _check(load().sf_gdn_shortconv_bwd(ctypes.byref(shape), _ptr(x), _ptr(w), _ptr(conv_in),
                                       _ptr(dy), _ptr(dconv_out), _ptr(dx), _ptr(dw), _ptr(dci),
                                       _ptr(workspace),
                                       ctypes.c_size_t(0 if workspace is None else workspace.numel()),
                                       _stream(stream)), "sf_gdn_shortconv_bwd")
    return dx, dw, dci


# ---- decoding and norms: checks, allocation and call in the native module ----
_calls = None

# The C entry points that _calls takes, in its order.
_CALL_ENTRIES = ("sf_gdn_recurrent_step", "sf_gdn_shortconv_step", "sf_gdn_gated_norm_fwd",
                 "sf_gdn_gated_norm_bwd", "sf_gdn_gated_norm_bwd_workspace_size",
                 "sf_gdn_residual_norm_fwd", "sf_gdn_residual_norm_bwd",
                 "sf_gdn_residual_norm_bwd_workspace_size", "sf_gdn_decay_chunk_fwd",
                 "sf_gdn_decay_chunk_fwd_workspace_size", "sf_gdn_decay_chunk_bwd",
                 "sf_gdn_decay_chunk_bwd_workspace_size", "sf_gdn_decay_step",
                 "sf_gdn_qk_norm_rotary_fwd", "sf_gdn_qk_norm_rotary_bwd",
                 "sf_gdn_qk_norm_rotary_bwd_workspace_size")


def _raise(status, where):
    _check(status, where)


def load_calls():
    """The native module _calls, on the library's entry points (raises if
    either has not been built, or they come from different headers)."""
    global _calls
    if _calls is None:
        lib = load()
        try:
            from . import _calls as module
        except ImportError as e:
            raise RuntimeError("the native module _calls is not built; run "
                               "`python -m linear_recurrence_chunked_gated_amd.build`") from e
        version = lib.sf_gdn_version().decode()
        if not version.endswith("interface %s" % getattr(module, "INTERFACE", None)):
            raise RuntimeError("%s was not built with this library (%s); rebuild both with "
                               "`python -m linear_recurrence_chunked_gated_amd.build`"
                               % (module.__file__, version))
        module.bind(_raise, *(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
                              for n in _CALL_ENTRIES))
        _calls = module
    return _calls


def _raw_stream(t):
    """The handle of the current stream on t's device."""
    if not t.is_cuda:
        raise ValueError("tensors must be on a GPU device, got one on %s" % t.device)
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _none(got):  # no output was made
    return ()


def _call_on(stream, t, f, *args, made=None):
    """f(*args, handle) of the native module for work on ``stream``.

    What f allocates comes from the current stream's memory, and a block of
    that may have been freed with work of the current stream on it still
    pending, which ``stream`` does not wait for; so ``stream`` is made the
    current one for the call.  The outputs made here (made(result); None: all
    of them) are marked as used by the caller's current stream, where they may
    then be read and freed as well (after it has waited for ``stream``)."""
    if not t.is_cuda:
        raise ValueError("tensors must be on a GPU device, got one on %s" % t.device)
    if stream.device != t.device:
        raise ValueError("the stream is on %s, the tensors on %s" % (stream.device, t.device))
    here = torch.cuda.current_stream(stream.device)
    if stream == here:
        return f(*args, stream.cuda_stream)
    with torch.cuda.stream(stream):
        got = f(*args, stream.cuda_stream)
    for m in (got if isinstance(got, tuple) else (got,)) if made is None else made(got):
        if m is not None and m.numel() > 0:
            m.record_stream(here)
    return got


def recurrent_step(q, k, v, alpha, beta, state, slots=None, seq_start=None, o=None, update=True,
                   stream=None):
    """sf_gdn_recurrent_step on torch tensors: the gated delta rule token by
    token over a pool of sequence states, for decoding.

    q, k [n_tok, Hk, Dk], v [n_tok, Hv, Dv] (bf16 or fp32; token rows may be
    slices of wider rows), alpha, beta [n_tok, Hv] fp32, state [n_slots, Hv,
    Dv, Dk] fp32, advanced in place unless update is False.  slots [n_seq]
    int32 names each sequence's slot (None: sequence i has slot i, one for
    every slot; negative: padding; up to 65,536 of them with update), seq_start
    [n_seq + 1] int32 its token rows (None: n_tok / n_seq each).  Returns o
    [n_tok, Hv, Dv]; rows of padding and past the last sequence keep what o
    held (pass o to set it).

    For decoding only: the output carries no autograd graph, whatever its
    inputs require.  The pool counts as changed in place, so a graph that has
    kept its old values raises in its backward.

    With ``stream``, here and in the calls below, the kernels run there, in no
    order with the current stream's work but what the caller sets up; outputs
    that the call makes are the given stream's memory."""
    f = (_calls or load_calls()).recurrent_step
    args = q, k, v, alpha, beta, state, slots, seq_start, o, update
    if stream is None:
        return f(*args, _raw_stream(q))
    return _call_on(stream, q, f, *args, made=None if o is None else _none)


def shortconv_step(x, w, state, slots=None, seq_start=None, act=0, y=None, update=True,
                   stream=None):
    """sf_gdn_shortconv_step on torch tensors: the short convolution token by
    token over a pool of boundary states, for decoding.

    x [n_tok, C] (token rows may be slices of wider rows), w [C, W] fp32,
    state [n_slots, W-1, C] in x's dtype, advanced in place unless update is
    False; slots and seq_start, and what it means to autograd, as in
    recurrent_step.  Returns y [n_tok, C]."""
    f = (_calls or load_calls()).shortconv_step
    args = x, w, state, slots, seq_start, act, y, update
    if stream is None:
        return f(*args, _raw_stream(x))
    return _call_on(stream, x, f, *args, made=None if y is None else _none)


def gated_norm_bwd_workspace_bytes(shape):
    n = ctypes.c_size_t(0)
    _check(load().sf_gdn_gated_norm_bwd_workspace_size(ctypes.byref(shape), ctypes.byref(n)),
           "gated_norm_bwd_workspace_size")
    return n.value


def gated_norm_fwd(x, gate=None, w=None, eps=1e-6, scale=1.0, act=1, y=None, stream=None):
    """sf_gdn_gated_norm_fwd on torch tensors: y = scale * w * x / sqrt(mean(
    x^2) + eps) * act(gate) over the last dimension of x [..., H, D], with
    gate like x or None (factor 1) and w [D] fp32 or None (ones); act 1 for
    SiLU, 0 for the gate itself.  x and gate may be head slices of wider token
    rows."""
    f = (_calls or load_calls()).gated_norm_fwd
    args = x, gate, w, eps, scale, act, y
    if stream is None:
        return f(*args, _raw_stream(x))
    return _call_on(stream, x, f, *args, made=None if y is None else _none)


def gated_norm_bwd(x, gate, w, dy, eps=1e-6, scale=1.0, act=1, grads=None, want_dw=True,
                   workspace=None, stream=None):
    """sf_gdn_gated_norm_bwd on torch tensors.  Returns (dx, dgate, dw), with
    None for dgate without gate and for dw without w (or want_dw False).
    ``grads`` may supply preallocated outputs in that order."""
    f = (_calls or load_calls()).gated_norm_bwd
    args = x, gate, w, dy, eps, scale, act, grads, want_dw, workspace
    if stream is None:
        return f(*args, _raw_stream(x))[:3]
    return _call_on(stream, x, f, *args,
                    made=lambda got: got[:3] if grads is None else ())[:3]


def residual_norm_bwd_workspace_bytes(shape):
    n = ctypes.c_size_t(0)
    _check(load().sf_gdn_residual_norm_bwd_workspace_size(ctypes.byref(shape), ctypes.byref(n)),
           "residual_norm_bwd_workspace_size")
    return n.value


def residual_norm_fwd(x, r=None, w=None, s=None, scale=1.0, eps=1e-6, h=None, y=None,
                      stream=None):
    """sf_gdn_residual_norm_fwd on torch tensors: h = x + scale * s * r and
    y = w * h / sqrt(mean(h^2) + eps) over the last dimension of x [..., C],
    with r like x (None: h is x), s [C] fp32 (None: ones) and w [C] fp32
    (None: ones).  Returns (y, h)."""
    f = (_calls or load_calls()).residual_norm_fwd
    args = x, r, w, s, scale, eps, h, y
    if stream is None:
        return f(*args, _raw_stream(x))
    return _call_on(stream, x, f, *args,
                    made=lambda got: (None if y is not None else got[0],
                                      None if h is not None or r is None else got[1]))


def residual_norm_bwd(h, r, w, s, dy, dh=None, scale=1.0, eps=1e-6, grads=None, want_dr=True,
                      want_dw=True, want_ds=True, workspace=None, stream=None):
    """sf_gdn_residual_norm_bwd on torch tensors: h as the forward returned
    it, dy and dh (None: zeros) the gradients of y and h.  Returns (dx, dr, dw,
    ds): dr is None with want_dr False, dw without w, ds without s (r is read
    for ds only and may be None otherwise); ``grads`` may supply preallocated
    outputs in that order."""
    f = (_calls or load_calls()).residual_norm_bwd
    args = h, r, w, s, dy, dh, scale, eps, grads, want_dr, want_dw, want_ds, workspace
    if stream is None:
        return f(*args, _raw_stream(h))[:4]
    return _call_on(stream, h, f, *args,
                    made=lambda got: got[:4] if grads is None else ())[:4]


def decay_chunk_fwd(q, k, v, decay, S_in=None, seq_start=None, scale=1.0, o=None, S_out=None,
                    workspace=None, stream=None):
    """sf_gdn_decay_chunk_fwd on torch tensors: linear attention with a fixed
    decay for each head, S_t = decay S_{t-1} + v_t k_t^T and o_t = scale S_t
    q_t, over whole sequences.  Returns (o, S_out).

    q, k [B, T, Hk, Dk] and v [B, T, Hv, Dv], or packed sequences: [n_tok, Hk,
    Dk] and [n_tok, Hv, Dv] with seq_start [n_seq + 1] int32 offsets on the
    device (without it: one sequence).  bf16 or fp32; token rows may be slices
    of wider rows; value head h reads q and k of head h // (Hv // Hk).  decay
    [Hv] fp32; S_in (None: zeros) and S_out [B or n_seq, Hv, Dv, Dk] fp32, as
    in chunk_fwd and as the slots of decay_step's pool.  Rows of no sequence
    keep what o held (pass o to set it)."""
    f = (_calls or load_calls()).decay_chunk_fwd
    args = q, k, v, decay, S_in, seq_start, scale, o, S_out, workspace
    if stream is None:
        return f(*args, _raw_stream(q))[:2]
    return _call_on(stream, q, f, *args,
                    made=lambda got: (None if o is not None else got[0],
                                      None if S_out is not None else got[1]))[:2]


def decay_chunk_bwd(q, k, v, decay, S_in, dO, dS_out=None, seq_start=None, scale=1.0, grads=None,
                    want_dS_in=True, workspace=None, stream=None):
    """sf_gdn_decay_chunk_bwd on torch tensors: the gradients of <dO, o> +
    <dS_out, S_out> (dS_out None: zeros).  Returns (dq, dk, dv, dS_in); dS_in
    is None with want_dS_in False.  ``grads`` may supply preallocated outputs
    in that order.  The decay is a constant and gets no gradient; rows of no
    sequence keep what dq, dk and dv held."""
    f = (_calls or load_calls()).decay_chunk_bwd
    args = q, k, v, decay, S_in, dO, dS_out, seq_start, scale, grads, want_dS_in, workspace
    if stream is None:
        return f(*args, _raw_stream(q))[:4]
    return _call_on(stream, q, f, *args,
                    made=lambda got: got[:4] if grads is None else ())[:4]


def decay_step(q, k, v, decay, state, slots=None, seq_start=None, o=None, update=True, scale=1.0,
               stream=None):
    """sf_gdn_decay_step on torch tensors: the recurrence of decay_chunk_fwd
    token by token over a pool of states, for decoding.

    q, k [n_tok, Hk, Dk], v [n_tok, Hv, Dv] (bf16 or fp32), decay [Hv] fp32;
    state [n_slots, Hv, Dv, Dk] fp32, advanced in place unless update is False;
    slots, seq_start, o, padding, refused entries and what it means to autograd
    as in recurrent_step.  Returns o [n_tok, Hv, Dv]."""
    f = (_calls or load_calls()).decay_step
    args = q, k, v, decay, state, slots, seq_start, o, update, scale
    if stream is None:
        return f(*args, _raw_stream(q))
    return _call_on(stream, q, f, *args, made=None if o is None else _none)


_PAIRS = {"halves": False, "neighbours": True}


def _neighbours(pairs):
    if pairs not in _PAIRS:
        raise ValueError("pairs must be 'halves' or 'neighbours', got %r" % (pairs,))
    return _PAIRS[pairs]


def qk_norm_rotary_fwd(q, k, pos=None, freq=None, wq=None, wk=None, eps=1e-6, q_scale=1.0,
                       k_scale=1.0, pairs="halves", first=0, yq=None, yk=None, stream=None):
    """sf_gdn_qk_norm_rotary_fwd on torch tensors: every head of q [..., T, Hq,
    D] and k [..., T, Hk, D] as scale * w * x / sqrt(mean(x^2) + eps), its first
    2 F values turned in pairs by the angles pos * freq.  Returns (yq, yk).

    pos int32, the shape before the heads (None: first, first + 1, .. along T);
    freq [F] fp32 (None: no rotation); wq, wk [D] fp32 or None (ones); pairs
    "halves" (i with i + F) or "neighbours" (2 i with 2 i + 1).  q and k may be
    head slices of wider token rows."""
    f = (_calls or load_calls()).qk_norm_rotary_fwd
    args = q, k, pos, freq, wq, wk, eps, q_scale, k_scale, _neighbours(pairs), first, yq, yk
    if stream is None:
        return f(*args, _raw_stream(q))
    return _call_on(stream, q, f, *args,
                    made=lambda got: (None if yq is not None else got[0],
                                      None if yk is not None else got[1]))


def qk_norm_rotary_bwd(q, k, pos, freq, wq, wk, dyq, dyk, eps=1e-6, q_scale=1.0, k_scale=1.0,
                       pairs="halves", first=0, grads=None, want_dw=True, workspace=None,
                       stream=None):
    """sf_gdn_qk_norm_rotary_bwd on torch tensors.  Returns (dq, dk, dwq, dwk),
    with None for the gradient of a weight that is None (of both with want_dw
    False).  ``grads`` may supply preallocated outputs in that order."""
    f = (_calls or load_calls()).qk_norm_rotary_bwd
    args = (q, k, pos, freq, wq, wk, dyq, dyk, eps, q_scale, k_scale, _neighbours(pairs), first,
            grads, want_dw, workspace)
    if stream is None:
        return f(*args, _raw_stream(q))[:4]
    return _call_on(stream, q, f, *args,
                    made=lambda got: got[:4] if grads is None else ())[:4]


class profile:
    """Context manager: per-kernel HIP-event timing of the library's launches.

    After exit, ``.results`` maps kernel name -> (launches, total_ms)."""

    def __init__(self, capacity=65536):
        self.capacity = capacity
        self.results = {}

    def __enter__(self):
        _check(load().sf_gdn_profile_begin(int(self.capacity)), "sf_gdn_profile_begin")
        return self

    def __exit__(self, *exc):
        lib = load()
        _check(lib.sf_gdn_profile_end(), "sf_gdn_profile_end")
        for i in range(lib.sf_gdn_profile_kernel_count()):
            name = ctypes.c_char_p()
            n = ctypes.c_longlong()
            ms = ctypes.c_double()
            _check(lib.sf_gdn_profile_kernel(i, ctypes.byref(name), ctypes.byref(n), ctypes.byref(ms)),
                   "sf_gdn_profile_kernel")
            self.results[name.value.decode()] = (n.value, ms.value)
        return False
