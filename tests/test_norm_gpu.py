"""The norms around the recurrence (gated_norm, residual_norm), forward and
backward, against their 64-bit forms and against differences; strides, empty
and single rows, NaN, determinism, autograd, graph replay, streams."""
import pytest
import torch

import linear_recurrence_chunked_gated_amd as gdn
from layer_testutil import (DT, U, check, gated_norm_bwd_ref, gated_norm_ref,
                            residual_norm_bwd_ref, residual_norm_ref)

pytestmark = pytest.mark.gpu


def _gated(N, H, D, dtype, gate, weight, seed, xstd=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    x = (xstd * r(N, H, D)).to(DT[dtype])
    return (x, 2 * r(N, H, D).to(DT[dtype]) if gate else None, 1 + 0.3 * r(D) if weight else None,
            r(N, H, D).to(DT[dtype]))


def _c(t):
    return None if t is None else t.cuda()


GATED = [
    # N, H, D, dtype, gate, weight, act, eps, scale, std of x
    (1, 1, 64, "f32", True, True, 1, 1e-6, 1.0, 1.0),
    (1, 16, 128, "bf16", True, True, 1, 1e-6, 1.0, 1.0),
    (37, 3, 128, "bf16", True, True, 1, 1e-5, 0.7, 1.0),
    (37, 3, 64, "f32", True, True, 0, 1e-5, -1.3, 1.0),
    (131, 2, 72, "f32", True, True, 1, 1e-6, 1.0, 1.0),     # lanes past the row's end
    (5, 5, 8, "bf16", True, True, 1, 1e-6, 1.0, 1.0),
    (65, 1, 256, "bf16", True, False, 1, 1e-6, 1.0, 1.0),
    (9, 2, 264, "f32", False, True, 1, 1e-6, 1.0, 1.0),
    (33, 1, 512, "f32", True, True, 1, 1e-6, 1.0, 1.0),
    (50, 4, 128, "f32", False, False, 1, 1e-12, 128 ** -0.5, 3.0),  # L2 norm
    (50, 4, 64, "bf16", False, False, 1, 0.0, 0.125, 1e-3),
    (1700, 16, 128, "bf16", True, True, 1, 1e-6, 1.0, 1.0),  # rows in more than one turn
]


@pytest.mark.parametrize("N,H,D,dtype,gate,weight,act,eps,scale,std", GATED)
def test_gated_norm_matches(N, H, D, dtype, gate, weight, act, eps, scale, std):
    x, g, w, dy = _gated(N, H, D, dtype, gate, weight, N + D, std)
    kw = dict(eps=eps, scale=scale, act=act)
    ref, bound = gated_norm_ref(x, g, w, **kw)
    y = gdn.gated_norm_fwd(_c(x), _c(g), _c(w), **kw)
    got = gdn.gated_norm_bwd(_c(x), _c(g), _c(w), _c(dy), **kw)
    torch.cuda.synchronize()
    check("y", y, ref, bound, dtype)
    # a partial's rows one after another, then the partials: no more adds than rows + 64
    refs, bounds = gated_norm_bwd_ref(x, g, w, dy, depth=N * H + 64, **kw)
    for name, a, b, e, t in zip(("dx", "dgate", "dw"), got, refs, bounds, (dtype, dtype, "f32")):
        if b is None:
            assert a is None
        else:
            check(name, a, b, e, t)


RES = [
    # N, C, dtype, r, w, s, dh, scale
    (1, 8, "f32", True, True, True, True, 1.0),
    (1, 2048, "bf16", True, True, False, True, 1.0),
    (3, 64, "bf16", True, True, True, True, 0.5),
    (7, 136, "f32", True, True, True, False, -0.5),
    (5, 512, "f32", False, True, False, True, 1.0),
    (5, 520, "bf16", True, False, True, True, 1.0),
    (33, 2048, "f32", True, True, True, True, 0.3),
    (6, 2056, "bf16", True, True, True, True, 1.0),
    (6, 4096, "f32", True, True, True, True, 1.0),
    (4, 8192, "bf16", True, True, True, True, 1.0),
    (3, 8200, "f32", True, True, True, True, 1.0),
    (3, 16384, "bf16", True, True, True, True, 1.0),
    (2500, 96, "bf16", True, True, True, True, 1.0),        # rows in more than one turn
]


@pytest.mark.parametrize("N,C,dtype,has_r,has_w,has_s,has_dh,scale", RES)
def test_residual_norm_matches(N, C, dtype, has_r, has_w, has_s, has_dh, scale):
    g = torch.Generator().manual_seed(N + C)
    rnd = lambda *s: torch.randn(s, generator=g)
    x = (2 * rnd(N, C)).to(DT[dtype])
    r = rnd(N, C).to(DT[dtype]) if has_r else None
    w = 1 + 0.3 * rnd(C) if has_w else None
    s = 1 + 0.3 * rnd(C) if has_s else None
    dy, dh = rnd(N, C).to(DT[dtype]), rnd(N, C).to(DT[dtype]) if has_dh else None
    (ry, rh), (by, bh) = residual_norm_ref(x, r, w, s, 1e-6, scale)
    y, h = gdn.residual_norm_fwd(_c(x), _c(r), _c(w), _c(s), scale=scale, eps=1e-6)
    torch.cuda.synchronize()
    check("y", y, ry, by, dtype)
    check("h", h, rh, bh, dtype)
    got = gdn.residual_norm_bwd(h, _c(r), _c(w), _c(s), _c(dy), _c(dh), scale=scale, eps=1e-6)
    torch.cuda.synchronize()
    refs, bounds = residual_norm_bwd_ref(h.cpu(), r, w, s, dy, dh, 1e-6, scale, depth=N + 64)
    for name, a, b, e, t, there in zip(("dx", "dr", "dw", "ds"), got, refs, bounds,
                                       (dtype, dtype, "f32", "f32"), (1, 1, has_w, has_s)):
        if not there:
            assert a is None
        else:
            check(name, a, b, e, t)


def test_gated_norm_backward_against_differences():
    """<grad, d> against central differences of the 64-bit forward along d:
    their error is of the step's square (third derivatives of order 10 give
    1e-8 at a step of 1e-5 over a loss of a few hundred terms)."""
    x, g, w, dy = _gated(6, 2, 64, "f32", True, True, 1)
    kw = dict(eps=1e-3, scale=0.8, act=1)
    grads = gdn.gated_norm_bwd(_c(x), _c(g), _c(w), _c(dy), **kw)
    _, bounds = gated_norm_bwd_ref(x, g, w, dy, depth=76, **kw)
    args = [t.double() for t in (x, g, w)]
    gen = torch.Generator().manual_seed(2)
    for i in range(3):
        d = torch.randn(args[i].shape, generator=gen, dtype=torch.float64)
        f = []
        for step in (1e-5, -1e-5):
            moved = [a + step * d if j == i else a for j, a in enumerate(args)]
            f.append((gated_norm_ref(*moved, **kw)[0] * dy.double()).sum())
        slope = (f[0] - f[1]) / 2e-5
        got = (grads[i].cpu().double() * d).sum()
        rounding = ((bounds[i] + grads[i].cpu().double().abs() * U) * d.abs()).sum()
        assert abs(got - slope) <= rounding + 1e-6, (i, got, slope)


def test_residual_norm_backward_against_differences():
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=gen)
    x, r, w, s = rnd(4, 72), rnd(4, 72), 1 + 0.3 * rnd(72), 1 + 0.3 * rnd(72)
    dy, dh = rnd(4, 72), rnd(4, 72)
    kw = dict(eps=1e-3, scale=0.7)
    _, h = gdn.residual_norm_fwd(_c(x), _c(r), _c(w), _c(s), **kw)
    dx, dr, dw, ds = gdn.residual_norm_bwd(h, _c(r), _c(w), _c(s), _c(dy), _c(dh), **kw)
    _, bounds = residual_norm_bwd_ref(h.cpu(), r, w, s, dy, dh, depth=68, **kw)
    args = [t.double() for t in (x, r, w, s)]
    for i, (grad, b) in enumerate(zip((dx, dr, dw, ds), bounds)):
        d = torch.randn(args[i].shape, generator=gen, dtype=torch.float64)
        f = []
        for step in (1e-5, -1e-5):
            moved = [a + step * d if j == i else a for j, a in enumerate(args)]
            (y, hh), _ = residual_norm_ref(*moved, **kw)
            f.append((y * dy.double()).sum() + (hh * dh.double()).sum())
        slope = (f[0] - f[1]) / 2e-5
        got = (grad.cpu().double() * d).sum()
        # the kernel's h is rounded to fp32: its gradients move by that relative error
        rounding = ((b + 8 * U * grad.cpu().double().abs() + 8 * U) * d.abs()).sum()
        assert abs(got - slope) <= rounding + 1e-6, (i, got, slope)


def test_gated_norm_slices_of_wider_rows():
    N, H, D = 41, 2, 64
    x, g, w, dy = _gated(N, H, D, "bf16", True, True, 4)
    y = gdn.gated_norm_fwd(_c(x), _c(g), _c(w))
    ref = gdn.gated_norm_bwd(_c(x), _c(g), _c(w), _c(dy))
    wide = torch.full((N, 3 * H, D), float("nan"), dtype=torch.bfloat16).cuda()
    wide[:, :H] = _c(x)
    wide[:, 2 * H:] = _c(g)
    y2 = gdn.gated_norm_fwd(wide[:, :H], wide[:, 2 * H:], _c(w))
    got = gdn.gated_norm_bwd(wide[:, :H], wide[:, 2 * H:], _c(w), _c(dy))
    torch.cuda.synchronize()
    assert torch.equal(y, y2)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    # [B, T, H, D] as the chunk gives it
    y4 = gdn.gated_norm_fwd(_c(x[:40]).view(2, 20, H, D), _c(g[:40]).view(2, 20, H, D), _c(w))
    assert y4.shape == (2, 20, H, D) and torch.equal(y4.view(40, H, D), y[:40])


@pytest.mark.parametrize("N,C", [(1, 72), (5, 8), (3, 512), (2, 640)])
def test_eps_zero_with_fewer_rows_than_a_workgroup_takes(N, C):
    """The workgroup's places without a row add nothing to the weight
    gradients, though 1 / sqrt(0 + 0) is infinite."""
    gen = torch.Generator().manual_seed(N + C)
    x, g, dy, dh = (torch.randn(N, C, generator=gen) for _ in range(4))
    w, s = 1 + 0.3 * torch.randn(C, generator=gen), 1 + 0.3 * torch.randn(C, generator=gen)
    if C <= 512:
        kw = dict(eps=0.0, scale=1.0, act=1)
        t = [v.view(N, 1, C) for v in (x, g, dy)]
        got = gdn.gated_norm_bwd(_c(t[0]), _c(t[1]), _c(w), _c(t[2]), **kw)
        refs, bounds = gated_norm_bwd_ref(t[0], t[1], w, t[2], depth=N + 64, **kw)
        for name, a, b, e in zip(("dx", "dgate", "dw"), got, refs, bounds):
            check(name, a, b, e, "f32")
    got = gdn.residual_norm_bwd(_c(x), _c(g), _c(w), _c(s), _c(dy), _c(dh), eps=0.0)
    refs, bounds = residual_norm_bwd_ref(x, g, w, s, dy, dh, 0.0, 1.0, depth=N + 64)
    for name, a, b, e in zip(("dx", "dr", "dw", "ds"), got, refs, bounds):
        check(name, a, b, e, "f32")


def test_offsets_past_32_bits():
    """Tensors of 2^31 elements and a little more: their last rows, beyond
    element 2^31, are those of a small call."""
    N, H, D = (1 << 20) + 40, 16, 128
    tail = 40
    xs, gs, w, ds = [_c(t) for t in _gated(tail, H, D, "bf16", True, True, 10)]
    big = []
    for t in (xs, gs, ds):
        b = torch.zeros(N, H, D, dtype=torch.bfloat16, device="cuda")
        b[N - tail:] = t
        big.append(b)
    x, g, dy = big
    assert (N - tail) * H * D >= 1 << 31
    y = gdn.gated_norm_fwd(x, g, w)
    dx, dg, dw = gdn.gated_norm_bwd(x, g, w, dy)
    ref = gdn.gated_norm_bwd(xs, gs, w, ds)
    torch.cuda.synchronize()
    assert torch.equal(y[N - tail:], gdn.gated_norm_fwd(xs, gs, w))
    assert torch.equal(dx[N - tail:], ref[0]) and torch.equal(dg[N - tail:], ref[1])
    assert torch.allclose(dw, ref[2], rtol=1e-4, atol=1e-4)  # other rows add zeros, in another order
    assert torch.count_nonzero(y[:1000]) == 0 and torch.count_nonzero(dx[N - 2000:N - tail]) == 0
    del y, dx, dg
    C = H * D
    X, R, DY = (t.view(N, C) for t in (x, g, dy))
    W = torch.linspace(0.5, 1.5, C, device="cuda")
    y, h = gdn.residual_norm_fwd(X, R, W, W)
    sy, sh = gdn.residual_norm_fwd(X[N - tail:], R[N - tail:], W, W)
    assert torch.equal(y[N - tail:], sy) and torch.equal(h[N - tail:], sh)
    del y
    got = gdn.residual_norm_bwd(h, R, W, W, DY, X)
    ref = gdn.residual_norm_bwd(sh, R[N - tail:], W, W, DY[N - tail:], X[N - tail:])
    torch.cuda.synchronize()
    assert torch.equal(got[0][N - tail:], ref[0]) and torch.equal(got[1][N - tail:], ref[1])
    assert torch.count_nonzero(got[0][:1000]) == 0


def test_more_rows_than_a_launch_holds():
    """Rows past the largest grid are taken in a second turn."""
    N, tail = (1 << 21) * 32 + 50, 60
    x, g, w, _ = [_c(t) for t in _gated(tail, 1, 8, "bf16", True, True, 11)]
    X = torch.zeros(N, 1, 8, dtype=torch.bfloat16, device="cuda")
    X[N - tail:] = x
    G = torch.zeros_like(X)
    G[N - tail:] = g
    y = gdn.gated_norm_fwd(X, G, w)
    torch.cuda.synchronize()
    assert torch.equal(y[N - tail:], gdn.gated_norm_fwd(x, g, w))
    assert torch.count_nonzero(y[:N - tail]) == 0
    X, G, y = X.view(-1, 8), G.view(-1, 8), None
    y, h = gdn.residual_norm_fwd(X, G, w)
    sy, sh = gdn.residual_norm_fwd(x.view(-1, 8), g.view(-1, 8), w)
    torch.cuda.synchronize()
    assert torch.equal(y[N - tail:], sy) and torch.equal(h[N - tail:], sh)
    assert torch.count_nonzero(y[:N - tail]) == 0


def test_no_rows():
    x = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    assert gdn.gated_norm_fwd(x, x, w).shape == x.shape
    dx, dg, dw = gdn.gated_norm_bwd(x, x, w, x)
    assert dx.shape == x.shape and torch.count_nonzero(dw) == 0
    x = torch.empty(0, 64, device="cuda")
    y, h = gdn.residual_norm_fwd(x, x, w, w)
    dx, dr, dw, ds = gdn.residual_norm_bwd(h, x, w, w, x, x)
    torch.cuda.synchronize()
    assert y.shape == x.shape and torch.count_nonzero(dw) == 0 and torch.count_nonzero(ds) == 0


def test_rows_keep_their_nan_and_zero_rows_their_zeros():
    x, g, w, dy = _gated(20, 1, 128, "f32", True, True, 6)
    y = gdn.gated_norm_fwd(_c(x), _c(g), _c(w))
    dx, dg, _ = gdn.gated_norm_bwd(_c(x), _c(g), _c(w), _c(dy))
    x2, g2 = x.clone(), g.clone()
    x2[3, 0, 5] = float("nan")
    x2[7] = 0.0
    g2[11, 0, 9] = float("inf")
    g2[12, 0, 9] = -100.0  # the exponential overflows: act is 0
    y2 = gdn.gated_norm_fwd(_c(x2), _c(g2), _c(w))
    dx2, dg2, _ = gdn.gated_norm_bwd(_c(x2), _c(g2), _c(w), _c(dy))
    torch.cuda.synchronize()
    same = [i for i in range(20) if i not in (3, 7, 11, 12)]
    for a, b in ((y, y2), (dx, dx2), (dg, dg2)):
        assert torch.equal(a[same], b[same])
    assert torch.isnan(y2[3]).all() and torch.isnan(dx2[3]).all()
    assert (y2[7] == 0).all() and (dg2[7] == 0).all() and torch.isfinite(dx2[7]).all()
    assert torch.isinf(y2[11, 0, 9]) and torch.isfinite(y2[11, 0, :9]).all()
    assert y2[12, 0, 9].abs() < 1e-30 and torch.isfinite(dx2[12]).all()
    r = torch.zeros(3, 640, device="cuda")
    r[1, 600] = float("nan")
    y, h = gdn.residual_norm_fwd(r, r)
    assert torch.isnan(y[1]).all() and (y[[0, 2]] == 0).all() and torch.isnan(h[1, 600])


def test_deterministic_and_workspace_reuse():
    x, g, w, dy = [_c(t) for t in _gated(3000, 8, 128, "bf16", True, True, 7)]
    ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN patterns
    a = gdn.gated_norm_bwd(x, g, w, dy)
    b = gdn.gated_norm_bwd(x, g, w, dy, workspace=ws)
    c = gdn.gated_norm_bwd(x[:5], g[:5], w, dy[:5], workspace=ws)
    c2 = gdn.gated_norm_bwd(x[:5], g[:5], w, dy[:5])
    r = [t.view(3000, 1024) for t in (x, g, dy)]
    v = torch.ones(1024, device="cuda")
    p = gdn.residual_norm_bwd(r[0], r[1], v, v, r[2], r[1])
    q = gdn.residual_norm_bwd(r[0], r[1], v, v, r[2], r[1], workspace=ws)
    torch.cuda.synchronize()
    for m, n in zip(a + c + p, b + c2 + q):
        assert torch.equal(m, n)


def test_autograd_equals_direct_calls():
    x, g, w, dy = [_c(t) for t in _gated(40, 3, 64, "bf16", True, True, 8)]
    kw = dict(eps=1e-5, scale=0.9, act=1)
    leaves = [t.clone().requires_grad_() for t in (x, g, w)]
    y = gdn.gated_norm(*leaves, **kw)
    y.backward(dy)
    for leaf, ref in zip(leaves, gdn.gated_norm_bwd(x, g, w, dy, **kw)):
        assert torch.equal(leaf.grad, ref)
    # without gate and weight; a gradient that is one value broadcast
    leaf = x.clone().requires_grad_()
    gdn.gated_norm(leaf, scale=0.125).sum().backward()
    assert torch.equal(leaf.grad, gdn.gated_norm_bwd(x, None, None, torch.ones_like(x),
                                                     scale=0.125)[0])
    # a frozen weight
    leaf = x.clone().requires_grad_()
    gdn.gated_norm(leaf, g, w, **kw).backward(dy)
    assert torch.equal(leaf.grad, gdn.gated_norm_bwd(x, g, w, dy, **kw)[0])

    X, R, DY, DH = (t.reshape(40, 192).contiguous() for t in (x, g, dy, dy.flip(0)))
    W, S = (torch.linspace(0.5, 1.5, 192, device="cuda") for _ in range(2))
    leaves = [t.clone().requires_grad_() for t in (X, R, W, S)]
    y, h = gdn.residual_norm(*leaves, scale=0.5)
    torch.autograd.backward((y, h), (DY, DH))
    _, hh = gdn.residual_norm_fwd(X, R, W, S, scale=0.5)
    ref = gdn.residual_norm_bwd(hh, R, W, S, DY, DH, scale=0.5)
    for leaf, b in zip(leaves, ref):
        assert torch.equal(leaf.grad, b)
    # h unused: its gradient is zero
    leaves = [t.clone().requires_grad_() for t in (X, R, W, S)]
    gdn.residual_norm(*leaves, scale=0.5)[0].backward(DY)
    ref = gdn.residual_norm_bwd(hh, R, W, S, DY, None, scale=0.5)
    for leaf, b in zip(leaves, ref):
        assert torch.equal(leaf.grad, b)
    # the norm alone: h is x, whose gradients add up
    leaf = X.clone().requires_grad_()
    y, h = gdn.residual_norm(leaf, None, W)
    assert h is leaf
    y.backward(DY)
    assert torch.equal(leaf.grad, gdn.residual_norm_bwd(X, None, W, None, DY)[0])


def test_norms_replay_from_a_graph_and_on_a_side_stream():
    x, g, w, dy = [_c(t) for t in _gated(300, 4, 128, "bf16", True, True, 9)]
    X, R = x.view(300, 512), g.view(300, 512)
    W = torch.linspace(0.5, 1.5, 512, device="cuda")
    S = W.flip(0).contiguous()

    def work():
        y = gdn.gated_norm_fwd(x, g, w)
        n, h = gdn.residual_norm_fwd(X, R, W, S)
        return (y, n, h) + gdn.gated_norm_bwd(x, g, w, dy) + \
            gdn.residual_norm_bwd(h, R, W, S, dy.view(300, 512), X)

    ref = work()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for rep in range(4):
        for t in out:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, ref):
            assert torch.equal(a, b), rep
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = gdn.gated_norm_fwd(x, g, w, stream=side)
    grads = gdn.gated_norm_bwd(x, g, w, dy, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip((y,) + grads, (ref[0],) + ref[3:6]):
        assert torch.equal(a, b)


def test_binding_refusals():
    x = torch.zeros(4, 2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    for exc, call in (
            (TypeError, lambda: gdn.gated_norm_fwd(x.half())),
            (TypeError, lambda: gdn.gated_norm_fwd(x, x.bfloat16())),
            (ValueError, lambda: gdn.gated_norm_fwd(x, x[:2])),
            (ValueError, lambda: gdn.gated_norm_fwd(x, None, w[:32])),
            (ValueError, lambda: gdn.gated_norm_fwd(x.view(2, 2, 2, 64), x)),
            (ValueError, lambda: gdn.gated_norm_fwd(x.view(2, 2, 2, 64).transpose(0, 1))),
            (ValueError, lambda: gdn.gated_norm_fwd(x.view(2, 2, 2, 64)[:, :1].expand(2, 2, 2, 64))),
            (ValueError, lambda: gdn.gated_norm_fwd(x[:1].expand(4, 2, 64))),
            (TypeError, lambda: gdn.gated_norm_fwd(x, 3.0)),
            (TypeError, lambda: gdn.gated_norm_bwd(x, None, w, x, grads=(x, None))),
            (ValueError, lambda: gdn.gated_norm_bwd(x, None, w, x, grads=(None, None, None))),
            (ValueError, lambda: gdn.gated_norm_bwd(x, None, w, x, workspace=torch.empty(1 << 20))),
            (ValueError, lambda: gdn.gated_norm_fwd(x.transpose(0, 1))),
            (ValueError, lambda: gdn.gated_norm_fwd(w)),
            (ValueError, lambda: gdn.gated_norm_bwd(x, None, w, x[:, :1])),
            (gdn.GDNError, lambda: gdn.gated_norm_fwd(x[..., :4].contiguous())),
            (gdn.GDNError, lambda: gdn.gated_norm_fwd(x, y=x)),
            (gdn.GDNError, lambda: gdn.gated_norm_fwd(x, eps=-1.0)),
            (gdn.GDNError, lambda: gdn.gated_norm_fwd(x, x, act=3)),
            (ValueError, lambda: gdn.residual_norm_fwd(x, None, None, w)),
            (ValueError, lambda: gdn.residual_norm_fwd(x, x[:2])),
            (ValueError, lambda: gdn.residual_norm_fwd(x.transpose(0, 1))),
            (gdn.GDNError, lambda: gdn.residual_norm_fwd(x, x, h=x)),
            (ValueError, lambda: gdn.residual_norm_bwd(x, None, w, w, x)),
            (ValueError, lambda: gdn.residual_norm(x, None, w, w))):
        with pytest.raises(exc):
            call()
