"""Host checks of the single-token calls and of the norms: what they refuse,
before anything is enqueued.  Placeholder addresses; no GPU call."""
import ctypes

import pytest
import torch

from linear_recurrence_chunked_gated_amd import _lib

G = 1 << 33  # addresses far apart, never read
INV, UNS, WS = _lib.SF_ERR_INVALID_ARG, _lib.SF_ERR_UNSUPPORTED, _lib.SF_ERR_WORKSPACE


def vp(x):
    return None if x is None else ctypes.c_void_p(x)


def _step(n_seq=4, n_tok=4, n_slots=8, Hk=2, Hv=4, Dk=128, Dv=128, dtype=1, update=1, qs=0, ks=0,
          vs=0, q=1 * G, k=2 * G, v=3 * G, alpha=4 * G, beta=5 * G, slots=6 * G, start=None,
          state=8 * G, o=16 * G):
    s = _lib.StepShape(n_seq, n_tok, n_slots, Hk, Hv, Dk, Dv, dtype, update, qs, ks, vs)
    return _lib.load().sf_gdn_recurrent_step(ctypes.byref(s), vp(q), vp(k), vp(v), vp(alpha),
                                             vp(beta), vp(slots), vp(start), vp(state), vp(o), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), INV), (dict(Hk=0), INV), (dict(Hv=3), INV), (dict(Dk=64), UNS),
    (dict(Dk=96, Dv=96), UNS), (dict(Dk=-1), INV), (dict(update=2), INV), (dict(n_seq=-1), INV),
    (dict(n_tok=-4), INV), (dict(n_slots=-1), INV),
    (dict(n_tok=5), INV),                           # not n_seq equal shares
    (dict(n_seq=0), INV),                           # tokens of no sequence
    (dict(slots=None, n_slots=3), INV),             # fewer slots than sequences
    (dict(qs=64), INV), (dict(ks=260), INV), (dict(vs=-512), INV), (dict(vs=511), INV),
    (dict(n_seq=1 << 20, n_tok=1 << 20, Hk=1, Hv=4), UNS),
    (dict(n_seq=1, n_tok=(1 << 30) + 1), UNS),
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(alpha=None), INV),
    (dict(beta=None), INV), (dict(state=None), INV), (dict(o=None), INV),
    (dict(q=G + 8), INV), (dict(state=8 * G + 4), INV), (dict(o=16 * G + 2), INV),
    (dict(alpha=4 * G + 2), INV), (dict(slots=6 * G + 2), INV), (dict(start=7 * G + 1), INV),
    (dict(o=1 * G + 64), INV), (dict(o=8 * G + 1024), INV), (dict(state=3 * G), INV),
    (dict(o=6 * G), INV), (dict(alpha=8 * G + 4), INV), (dict(start=16 * G + 4), INV),
    # o inside the gap between q's strided rows is inside q's range
    (dict(qs=4096, o=1 * G + 1024), INV),
])
def test_step_refuses(kw, code):
    assert _step(**kw) == code
    assert _lib.load().sf_last_error_message()


def test_step_null_shape_and_empty_batches():
    L = _lib.load()
    assert L.sf_gdn_recurrent_step(None, *[None] * 9, None) == INV
    assert L.sf_gdn_shortconv_step(None, *[None] * 6, None) == INV
    # nothing to do: no pointer is needed
    none = dict(q=None, k=None, v=None, alpha=None, beta=None, slots=None, state=None, o=None)
    assert _step(n_seq=0, n_tok=0, n_slots=0, **none) == _lib.SF_OK
    assert _step(n_seq=4, n_tok=0, **none) == _lib.SF_OK


def _conv(n_seq=4, n_tok=4, n_slots=8, C=64, W=4, dtype=1, act=1, update=1, xs=0, x=1 * G, w=2 * G,
          slots=3 * G, start=None, state=5 * G, y=6 * G):
    s = _lib.ConvStepShape(n_seq, n_tok, n_slots, C, W, dtype, act, update, xs)
    return _lib.load().sf_gdn_shortconv_step(ctypes.byref(s), vp(x), vp(w), vp(slots), vp(start),
                                             vp(state), vp(y), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=-1), INV), (dict(C=0), INV), (dict(C=12), UNS), (dict(W=0), UNS), (dict(W=9), UNS),
    (dict(act=2), INV), (dict(update=-1), INV), (dict(xs=32), INV), (dict(xs=68), INV),
    (dict(n_tok=6), INV), (dict(slots=None, n_slots=2), INV), (dict(x=None), INV),
    (dict(w=None), INV), (dict(state=None), INV), (dict(y=None), INV), (dict(x=G + 2), INV),
    (dict(y=G + 64), INV), (dict(state=6 * G + 16), INV), (dict(y=3 * G), INV),
    (dict(slots=5 * G + 64), INV),
    (dict(n_seq=1 << 20, n_tok=1 << 20, C=4096), UNS), (dict(n_seq=1, n_tok=(1 << 30) + 1), UNS),
])
def test_conv_step_refuses(kw, code):
    assert _conv(**kw) == code


def _gshape(N=8, H=4, D=128, dtype=1, act=1, eps=1e-6, scale=1.0, xs=0, gs=0):
    return _lib.GatedNormShape(N, H, D, dtype, act, eps, scale, xs, gs)


def _gfwd(x=1 * G, gate=2 * G, w=3 * G, y=4 * G, **kw):
    return _lib.load().sf_gdn_gated_norm_fwd(ctypes.byref(_gshape(**kw)), vp(x), vp(gate), vp(w),
                                             vp(y), None)


def _gbwd(x=1 * G, gate=2 * G, w=3 * G, dy=4 * G, dx=5 * G, dgate=6 * G, dw=7 * G, ws=8 * G,
          wsn=1 << 20, **kw):
    return _lib.load().sf_gdn_gated_norm_bwd(ctypes.byref(_gshape(**kw)), vp(x), vp(gate), vp(w),
                                             vp(dy), vp(dx), vp(dgate), vp(dw), vp(ws),
                                             ctypes.c_size_t(wsn), None)


SHAPES = [
    (dict(dtype=3), INV), (dict(N=-1), INV), (dict(H=0), INV), (dict(D=0), INV),
    (dict(D=12), UNS), (dict(D=520), UNS), (dict(act=2), INV), (dict(eps=-1e-6), INV),
    (dict(eps=float("nan")), INV), (dict(xs=256), INV), (dict(gs=516), INV), (dict(N=1 << 40), UNS),
]


@pytest.mark.parametrize("kw,code", SHAPES + [
    (dict(x=None), INV), (dict(y=None), INV), (dict(y=1 * G + 16), INV), (dict(x=G + 8), INV),
    (dict(w=3 * G + 4), INV), (dict(y=2 * G), INV), (dict(xs=1024, y=G + 1024), INV),
])
def test_gated_norm_fwd_refuses(kw, code):
    assert _gfwd(**kw) == code


@pytest.mark.parametrize("kw,code", SHAPES + [
    (dict(x=None), INV), (dict(dy=None), INV), (dict(dx=None), INV), (dict(gate=None), INV),
    (dict(dgate=None), INV), (dict(w=None), INV), (dict(dx=4 * G), INV), (dict(dgate=5 * G), INV),
    (dict(dw=8 * G), INV), (dict(ws=1 * G), INV), (dict(ws=None), WS), (dict(wsn=16), WS), (dict(ws=8 * G + 16), INV),
])
def test_gated_norm_bwd_refuses(kw, code):
    assert _gbwd(**kw) == code


def _rshape(N=8, C=2048, dtype=1, eps=1e-6, scale=1.0):
    return _lib.ResidualNormShape(N, C, dtype, eps, scale)


def _rfwd(x=1 * G, r=2 * G, s=3 * G, w=4 * G, h=5 * G, y=6 * G, **kw):
    return _lib.load().sf_gdn_residual_norm_fwd(ctypes.byref(_rshape(**kw)), vp(x), vp(r), vp(s),
                                                vp(w), vp(h), vp(y), None)


def _rbwd(h=1 * G, r=2 * G, s=3 * G, w=4 * G, dy=5 * G, dh=6 * G, dx=7 * G, dr=8 * G, dw=9 * G,
          ds=10 * G, ws=11 * G, wsn=1 << 20, **kw):
    return _lib.load().sf_gdn_residual_norm_bwd(ctypes.byref(_rshape(**kw)), vp(h), vp(r), vp(s),
                                                vp(w), vp(dy), vp(dh), vp(dx), vp(dr), vp(dw),
                                                vp(ds), vp(ws), ctypes.c_size_t(wsn), None)


RSHAPES = [
    (dict(dtype=3), INV), (dict(N=-1), INV), (dict(C=0), INV), (dict(C=20), UNS),
    (dict(C=16392), UNS), (dict(eps=-1.0), INV), (dict(N=1 << 40), UNS),
]


@pytest.mark.parametrize("kw,code", RSHAPES + [
    (dict(x=None), INV), (dict(y=None), INV), (dict(r=None), INV), (dict(h=None), INV),
    (dict(r=None, h=None), INV),                       # s without r
    (dict(h=G + 32), INV), (dict(y=5 * G), INV), (dict(x=G + 4), INV),
])
def test_residual_norm_fwd_refuses(kw, code):
    assert _rfwd(**kw) == code


@pytest.mark.parametrize("kw,code", RSHAPES + [
    (dict(h=None), INV), (dict(dy=None), INV), (dict(dx=None), INV), (dict(w=None), INV),
    (dict(s=None), INV), (dict(r=None), INV), (dict(dx=6 * G), INV), (dict(dr=7 * G + 16), INV),
    (dict(ds=11 * G), INV), (dict(ws=6 * G), INV), (dict(ws=None), WS), (dict(wsn=1 << 16), WS),
    (dict(ws=11 * G + 128), INV),
])
def test_residual_norm_bwd_refuses(kw, code):
    assert _rbwd(**kw) == code


def test_norm_workspaces_hold_a_row_per_workgroup():
    L = _lib.load()
    n = ctypes.c_size_t(0)
    assert L.sf_gdn_gated_norm_bwd_workspace_size(ctypes.byref(_gshape()), None) == INV
    assert L.sf_gdn_residual_norm_bwd_workspace_size(None, ctypes.byref(n)) == INV
    assert _lib.gated_norm_bwd_workspace_bytes(_gshape(N=0)) == 0
    small = _lib.gated_norm_bwd_workspace_bytes(_gshape(N=1))
    large = _lib.gated_norm_bwd_workspace_bytes(_gshape(N=1 << 20))
    assert 0 < small <= large < 64 << 20
    assert _lib.residual_norm_bwd_workspace_bytes(_rshape(N=0)) == 0
    assert 0 < _lib.residual_norm_bwd_workspace_bytes(_rshape(N=1 << 20)) < 512 << 20


def test_bindings_refuse_cpu_tensors():
    import linear_recurrence_chunked_gated_amd as gdn
    x = torch.zeros(4, 2, 64)
    for call in (lambda: gdn.recurrent_step(x, x, x, x[..., 0], x[..., 0], torch.zeros(4, 2, 64, 64)),
                 lambda: gdn.shortconv_step(x[:, 0], torch.zeros(64, 4), torch.zeros(4, 3, 64)),
                 lambda: gdn.gated_norm_fwd(x), lambda: gdn.gated_norm_bwd(x, None, None, x),
                 lambda: gdn.residual_norm_fwd(x), lambda: gdn.gated_norm(x),
                 lambda: gdn.residual_norm_bwd(x, None, None, None, x)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("call", [_step, _conv])
def test_checked_slots_are_bounded(call):
    """The check for repeated slots is quadratic in the sequences: past 65,536
    of them an updating call with slots is refused.  Without slots, or only
    reading, nothing is checked.  The output's odd address is refused after
    that, before any launch."""
    last = {"o" if call is _step else "y": (16 if call is _step else 6) * G + 2}
    n = 1 << 16
    small = dict(Hk=1, Hv=1, Dk=64, Dv=64) if call is _step else dict(C=8)
    kw = dict(small, n_slots=1 << 21, **last)
    assert call(n_seq=n + 1, n_tok=n + 1, **kw) == UNS
    assert "65536" in _lib.load().sf_last_error_message().decode()
    assert call(n_seq=n, n_tok=n, **kw) == INV
    assert call(n_seq=n + 1, n_tok=n + 1, update=0, **kw) == INV
    assert call(n_seq=n + 1, n_tok=n + 1, slots=None, **kw) == INV


def _residual_autograd(monkeypatch):
    """residual_norm's autograd over stand-ins for the two calls (h = x + r, y
    = h; gradients of ones), and what the backward call was given."""
    from linear_recurrence_chunked_gated_amd import autograd
    seen = []

    def fwd(x, r, w, s, scale, eps):
        h = x + r if r is not None else x
        return h.clone(), h

    def bwd(h, r, w, s, dy, dh, scale, eps, want_dr, want_dw, want_ds):
        seen.append(dict(r=r, dy=dy, dh=dh, want_ds=want_ds))
        return (torch.ones_like(h), torch.ones_like(h) if want_dr else None,
                torch.ones_like(w) if want_dw else None, torch.ones_like(s) if want_ds else None)

    monkeypatch.setattr(_lib, "residual_norm_fwd", fwd)
    monkeypatch.setattr(_lib, "residual_norm_bwd", bwd)
    return autograd.residual_norm, seen


def _leaves(s_grad=True):
    x, r = (torch.randn(4, 8).requires_grad_() for _ in range(2))
    return x, r, torch.ones(8).requires_grad_(), torch.ones(8).requires_grad_(s_grad)


def test_residual_norm_backward_of_an_unused_h(monkeypatch):
    """No tensor of zeros is made for the gradient of an h that nothing used."""
    norm, seen = _residual_autograd(monkeypatch)
    y, h = norm(*_leaves())
    y.sum().backward()
    assert seen[0]["dh"] is None and (seen[0]["dy"] == 1).all()
    y, h = norm(*_leaves())
    (y.sum() + 2 * h.sum()).backward()
    assert (seen[1]["dh"] == 2).all() and (seen[1]["dy"] == 1).all()
    # h alone: the norm's part is the gradient of zeros
    leaves = _leaves()
    norm(*leaves)[1].sum().backward()
    assert (seen[2]["dh"] == 1).all() and (seen[2]["dy"] == 0).all()
    assert seen[2]["dy"].shape == seen[2]["dh"].shape == (4, 8)
    assert all(t.grad is not None for t in leaves)


@pytest.mark.parametrize("s_grad", [True, False])
def test_residual_norm_keeps_r_for_the_gradient_of_s_only(monkeypatch, s_grad):
    norm, seen = _residual_autograd(monkeypatch)
    x, r, w, s = _leaves(s_grad)
    y, h = norm(x, r, w, s)
    assert any(t is r for t in y.grad_fn.saved_tensors) == s_grad
    y.sum().backward()
    assert seen[0]["want_ds"] == s_grad and (seen[0]["r"] is not None) == s_grad
    assert (s.grad is not None) == s_grad
