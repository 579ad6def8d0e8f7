"""Host checks of linear attention with a decay (chunk and single tokens) and of
the norm with rotation: what they refuse, before anything is enqueued, and the
plan's sizes.  Placeholder addresses; no GPU call."""
import ctypes

import pytest
import torch

import linear_recurrence_chunked_gated_amd as gdn
from linear_recurrence_chunked_gated_amd import _lib

G = 1 << 36  # addresses far apart, never read
INV, UNS, WS = _lib.SF_ERR_INVALID_ARG, _lib.SF_ERR_UNSUPPORTED, _lib.SF_ERR_WORKSPACE


def vp(x):
    return None if x is None else ctypes.c_void_p(x)


def _shape(n_seq=2, n_tok=600, Hk=2, Hv=4, Dk=128, Dv=128, dtype=1, scale=1.0, qs=0, ks=0, vs=0):
    return _lib.DecayShape(n_seq, n_tok, Hk, Hv, Dk, Dv, dtype, scale, qs, ks, vs)


def _fwd(q=1 * G, k=2 * G, v=3 * G, decay=4 * G, start=None, S_in=5 * G, o=6 * G, S_out=7 * G,
         ws=8 * G, wsn=1 << 30, **kw):
    return _lib.load().sf_gdn_decay_chunk_fwd(ctypes.byref(_shape(**kw)), vp(q), vp(k), vp(v),
                                              vp(decay), vp(start), vp(S_in), vp(o), vp(S_out),
                                              vp(ws), ctypes.c_size_t(wsn), None)


def _bwd(q=1 * G, k=2 * G, v=3 * G, decay=4 * G, start=None, S_in=5 * G, dO=6 * G, dS_out=7 * G,
         dq=8 * G, dk=9 * G, dv=10 * G, dS_in=11 * G, ws=12 * G, wsn=1 << 30, **kw):
    return _lib.load().sf_gdn_decay_chunk_bwd(ctypes.byref(_shape(**kw)), vp(q), vp(k), vp(v),
                                              vp(decay), vp(start), vp(S_in), vp(dO), vp(dS_out),
                                              vp(dq), vp(dk), vp(dv), vp(dS_in), vp(ws),
                                              ctypes.c_size_t(wsn), None)


SHAPES = [
    (dict(dtype=2), INV), (dict(Hk=0), INV), (dict(Hv=3), INV), (dict(Dk=64), UNS),
    (dict(Dk=96, Dv=96), UNS), (dict(Dv=-1), INV), (dict(n_seq=-1), INV), (dict(n_tok=-1), INV),
    (dict(n_tok=601), INV),                        # not n_seq equal shares
    (dict(n_seq=0), INV),                          # tokens of no sequence
    (dict(qs=128), INV), (dict(ks=260), INV), (dict(vs=-512), INV),
    (dict(n_seq=1, n_tok=(1 << 30) + 1), UNS), (dict(n_seq=1 << 20, n_tok=1 << 20), UNS),
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(decay=None), INV),
    (dict(q=G + 8), INV), (dict(S_in=5 * G + 4), INV), (dict(decay=4 * G + 2), INV),
    (dict(start=13 * G + 2), INV), (dict(ws=None, n_seq=1), WS), (dict(wsn=256, n_seq=1), WS),
    (dict(start=13 * G, ws=None), WS),             # the table of a packed call
]


@pytest.mark.parametrize("kw,code", SHAPES + [
    (dict(o=None), INV), (dict(o=6 * G + 8), INV), (dict(o=1 * G + 64), INV),
    (dict(S_out=5 * G), INV), (dict(S_out=6 * G + 1024), INV), (dict(ws=3 * G), INV),
    (dict(ws=8 * G + 64), INV), (dict(decay=6 * G), INV), (dict(start=7 * G), INV),
    (dict(qs=1024, o=1 * G + 1024), INV),          # in the gaps of q's rows
])
def test_chunk_fwd_refuses(kw, code):
    assert _fwd(**kw) == code
    assert _lib.load().sf_last_error_message()


@pytest.mark.parametrize("kw,code", SHAPES + [
    (dict(dO=None), INV), (dict(dq=None), INV), (dict(dk=None), INV), (dict(dv=None), INV),
    (dict(dq=9 * G), INV), (dict(dv=6 * G), INV), (dict(dS_in=7 * G), INV), (dict(dk=2 * G), INV),
    (dict(ws=10 * G), INV), (dict(decay=8 * G), INV), (dict(dO=6 * G + 4), INV),
])
def test_chunk_bwd_refuses(kw, code):
    assert _bwd(**kw) == code


def test_empty_chunks_and_null_shapes():
    L = _lib.load()
    n = ctypes.c_size_t()
    assert L.sf_gdn_decay_chunk_fwd(None, *[None] * 9, 0, None) == INV
    assert L.sf_gdn_decay_chunk_bwd(None, *[None] * 13, 0, None) == INV
    assert L.sf_gdn_decay_chunk_fwd_workspace_size(None, ctypes.byref(n)) == INV
    assert L.sf_gdn_decay_chunk_bwd_workspace_size(ctypes.byref(_shape()), None) == INV
    none = dict(q=None, k=None, v=None, decay=None, S_in=None, ws=None, wsn=0, n_seq=0, n_tok=0)
    assert _fwd(o=None, S_out=None, **none) == _lib.SF_OK
    assert _bwd(dO=None, dS_out=None, dq=None, dk=None, dv=None, dS_in=None, **none) == _lib.SF_OK


def _bytes(bwd=False, **kw):
    n = ctypes.c_size_t()
    f = _lib.load()
    f = f.sf_gdn_decay_chunk_bwd_workspace_size if bwd else f.sf_gdn_decay_chunk_fwd_workspace_size
    assert f(ctypes.byref(_shape(**kw)), ctypes.byref(n)) == _lib.SF_OK
    return n.value


@pytest.mark.parametrize("kw", [
    dict(n_seq=1, n_tok=0), dict(n_seq=1, n_tok=1), dict(n_seq=3, n_tok=100), dict(),
    dict(n_seq=1, n_tok=65536, Hk=16, Hv=16), dict(n_seq=1, n_tok=1 << 30, Hk=1, Hv=1, Dk=64, Dv=64),
    dict(n_seq=32768, n_tok=32768, Hk=16, Hv=64), dict(n_seq=512, n_tok=512 * 40, Hk=1, Hv=1),
    dict(n_seq=1, n_tok=262144, Hk=32, Hv=32),
])
def test_workspace_sizes(kw):
    """Boundary states of all heads are some hundreds, and a backward in bf16
    has fewer, twice; the table is small, and up to 64 sequences need none."""
    s = _shape(**kw)
    states = (kw.get("n_seq", 2) + 3 * 512) * s.Dk * s.Dv * 4
    table = 4 * (16 + 9 * (s.n_seq + 3 * 512)) + 512
    fwd, bwd = _bytes(**kw), _bytes(True, **kw)
    assert (0 if s.n_seq <= 64 else 20 * s.n_seq) <= fwd <= states + table
    part = 2 * s.n_tok * s.Hv * s.Dv * 4 if s.Hv > s.Hk else 0
    assert part <= bwd <= 2 * states + table + part + 512


def test_rows_too_far_apart():
    """A block of 64 rows is addressed in 31 bits: strides up to 2^22."""
    ok, far = 1 << 22, (1 << 22) + 8
    for name in ("qs", "ks", "vs"):
        assert _fwd(wsn=0, ws=0, **{name: far}) == UNS
        assert _bwd(wsn=0, ws=0, **{name: far}) == UNS
        assert _fwd(wsn=0, ws=0, n_seq=1, n_tok=4096, **{name: ok}) == WS


def test_the_caller_may_give_more_workspace_but_not_less():
    need = _bytes(n_seq=1)
    assert _fwd(n_seq=1, start=13 * G, wsn=need - 1) == WS
    assert _bwd(n_seq=1, start=13 * G, wsn=_bytes(True, n_seq=1) - 1) == WS


def _step(n_seq=4, n_tok=4, n_slots=8, Hk=2, Hv=4, Dk=128, Dv=128, dtype=1, update=1, qs=0, ks=0,
          vs=0, q=1 * G, k=2 * G, v=3 * G, decay=4 * G, slots=6 * G, start=None, state=8 * G,
          o=16 * G):
    s = _lib.DecayStepShape(n_seq, n_tok, n_slots, Hk, Hv, Dk, Dv, dtype, update, 1.0, qs, ks, vs)
    return _lib.load().sf_gdn_decay_step(ctypes.byref(s), vp(q), vp(k), vp(v), vp(decay), vp(slots),
                                         vp(start), vp(state), vp(o), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), INV), (dict(Hk=0), INV), (dict(Hv=3), INV), (dict(Dk=64), UNS),
    (dict(Dk=96, Dv=96), UNS), (dict(update=2), INV), (dict(n_seq=-1), INV), (dict(n_tok=-4), INV),
    (dict(n_slots=-1), INV), (dict(n_tok=5), INV), (dict(n_seq=0), INV),
    (dict(slots=None, n_slots=3), INV), (dict(qs=64), INV), (dict(ks=260), INV), (dict(vs=511), INV),
    (dict(n_seq=1 << 20, n_tok=1 << 20, Hk=1, Hv=4), UNS), (dict(n_seq=1, n_tok=(1 << 30) + 1), UNS),
    (dict(n_seq=65537, n_tok=65537, n_slots=1 << 17), UNS),
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(decay=None), INV),
    (dict(state=None), INV), (dict(o=None), INV), (dict(q=G + 8), INV), (dict(state=8 * G + 4), INV),
    (dict(decay=4 * G + 2), INV), (dict(slots=6 * G + 2), INV), (dict(start=7 * G + 1), INV),
    (dict(o=1 * G + 64), INV), (dict(o=8 * G + 1024), INV), (dict(state=3 * G), INV),
    (dict(decay=8 * G + 4), INV), (dict(start=16 * G + 4), INV), (dict(qs=4096, o=1 * G + 1024), INV),
])
def test_step_refuses(kw, code):
    assert _step(**kw) == code


def test_empty_steps():
    assert _lib.load().sf_gdn_decay_step(None, *[None] * 8, None) == INV
    none = dict(q=None, k=None, v=None, decay=None, slots=None, state=None, o=None)
    assert _step(n_seq=0, n_tok=0, n_slots=0, **none) == _lib.SF_OK
    assert _step(n_tok=0, **none) == _lib.SF_OK


def _rshape(N=8, T=8, Hq=4, Hk=2, D=128, F=64, dtype=1, neighbours=0, first=0, eps=1e-6, qs=0, ks=0):
    return _lib.RotaryShape(N, T, Hq, Hk, D, F, dtype, neighbours, first, eps, 1.0, 1.0, qs, ks)


def _rfwd(q=1 * G, k=2 * G, pos=3 * G, freq=4 * G, wq=5 * G, wk=6 * G, yq=7 * G, yk=8 * G, **kw):
    return _lib.load().sf_gdn_qk_norm_rotary_fwd(ctypes.byref(_rshape(**kw)), vp(q), vp(k), vp(pos),
                                                 vp(freq), vp(wq), vp(wk), vp(yq), vp(yk), None)


def _rbwd(q=1 * G, k=2 * G, pos=3 * G, freq=4 * G, wq=5 * G, wk=6 * G, dyq=7 * G, dyk=8 * G,
          dq=9 * G, dk=10 * G, dwq=11 * G, dwk=12 * G, ws=13 * G, wsn=1 << 20, **kw):
    return _lib.load().sf_gdn_qk_norm_rotary_bwd(
        ctypes.byref(_rshape(**kw)), vp(q), vp(k), vp(pos), vp(freq), vp(wq), vp(wk), vp(dyq),
        vp(dyk), vp(dq), vp(dk), vp(dwq), vp(dwk), vp(ws), ctypes.c_size_t(wsn), None)


RSHAPES = [
    (dict(dtype=3), INV), (dict(N=-1), INV), (dict(Hq=0), INV), (dict(Hk=-1), INV), (dict(D=0), INV),
    (dict(D=12, F=0), UNS), (dict(D=520), UNS), (dict(neighbours=2), INV), (dict(F=-8), INV),
    (dict(F=72), INV), (dict(F=60), UNS), (dict(F=62, neighbours=1), UNS), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(qs=256), INV), (dict(ks=260), INV), (dict(N=1 << 40), UNS),
    (dict(pos=None, T=0), INV), (dict(pos=None, first=(1 << 31) - 4), UNS), (dict(freq=None), INV),
    (dict(q=None), INV), (dict(k=None), INV), (dict(q=G + 8), INV), (dict(wq=5 * G + 4), INV),
    (dict(pos=3 * G + 2), INV), (dict(freq=4 * G + 1), INV),
]


@pytest.mark.parametrize("kw,code", RSHAPES + [
    (dict(yq=None), INV), (dict(yk=None), INV), (dict(yq=1 * G + 64), INV), (dict(yk=7 * G), INV),
    (dict(yq=3 * G), INV), (dict(yk=4 * G), INV), (dict(qs=1024, yq=G + 1024), INV),
])
def test_rotary_fwd_refuses(kw, code):
    assert _rfwd(**kw) == code


@pytest.mark.parametrize("kw,code", RSHAPES + [
    (dict(dyq=None), INV), (dict(dyk=None), INV), (dict(dq=None), INV), (dict(dk=None), INV),
    (dict(wq=None), INV), (dict(wk=None), INV), (dict(dq=7 * G), INV), (dict(dk=9 * G), INV),
    (dict(dwq=12 * G), INV), (dict(ws=2 * G), INV), (dict(ws=None), WS), (dict(wsn=16), WS),
    (dict(ws=13 * G + 16), INV),
])
def test_rotary_bwd_refuses(kw, code):
    assert _rbwd(**kw) == code


def test_rotary_of_nothing():
    assert _rfwd(N=0, q=None, k=None, yq=None, yk=None, pos=None, T=0) == _lib.SF_OK
    assert _lib.load().sf_gdn_qk_norm_rotary_fwd(None, *[None] * 9) == INV


def test_calls_refuse_cpu_tensors():
    """The Python calls: a CPU tensor is refused before the library is asked."""
    x = torch.zeros(2, 1, 64)
    a = torch.ones(1)
    w = torch.ones(64)
    for f in (lambda: gdn.decay_chunk_fwd(x, x, x, a), lambda: gdn.decay_chunk(x, x, x, a),
              lambda: gdn.decay_chunk_bwd(x, x, x, a, None, x),
              lambda: gdn.decay_step(x, x, x, a, torch.zeros(2, 1, 64, 64)),
              lambda: gdn.qk_norm_rotary_fwd(x, x, None, None, w, w),
              lambda: gdn.qk_norm_rotary(x, x), lambda: gdn.qk_norm_rotary_bwd(x, x, None, None, w, w, x, x)):
        with pytest.raises(ValueError, match="GPU"):
            f()


@pytest.mark.parametrize("n_seq,n_tok,Hk,Hv,D,dtype", [
    (1, 1 << 30, 2048, 2048, 64, 1), (1, 1 << 28, 8192, 8192, 128, 1), (1, 1 << 30, 512, 512, 128, 1),
    (1, 1 << 30, 1, 1 << 16, 64, 0), (3, (1 << 30) - 1, 3, 48, 64, 1), (64, (1 << 30) - 37, 171, 513, 64, 0),
    (1 << 5, 1 << 30, 1 << 10, 1 << 16, 64, 1), (1 << 21, 1 << 30, 1, 1, 128, 0),
])
def test_plans_of_the_largest_batches(n_seq, n_tok, Hk, Hv, D, dtype):
    """Segments are no longer than the batch, whatever the limits allow: a
    segment's tokens stay in 32 bits and the boundaries some hundreds."""
    kw = dict(n_seq=n_seq, n_tok=n_tok, Hk=Hk, Hv=Hv, Dk=D, Dv=D, dtype=dtype)
    states = (n_seq + 3 * 512) * D * D * 4
    table = 4 * (16 + 9 * (n_seq + 3 * 512)) + 512
    part = 2 * n_tok * Hv * D * 4 if Hv > Hk else 0
    fwd, bwd = _bytes(**kw), _bytes(True, **kw)
    assert fwd <= states + table
    assert part <= bwd <= 2 * states + table + part + 512


@pytest.mark.parametrize("first,T", [((1 << 31) - 2, (1 << 63) - 1), (1, (1 << 63) - 1), (0, (1 << 31) + 1),
                                     ((1 << 31) - 8, 9), (-5, (1 << 31) + 6), (-(1 << 31), (1 << 63) - 1)])
def test_positions_past_32_bits_are_refused(first, T):
    """Without pos the last position is first + T - 1, whatever T's size."""
    assert _rfwd(pos=None, first=first, T=T) == UNS
    assert _rbwd(pos=None, first=first, T=T) == UNS
    ok = (1 << 31) - first  # the last position is 2^31 - 1: refused for its missing freq
    assert _rfwd(pos=None, first=first, T=ok, freq=None) == INV
