"""The norm and rotation of queries and keys (qk_norm_rotary_fwd, _bwd) against
their 64-bit form: token types, head layouts, sizes, both kinds of pairs,
partial and no rotation, far and negative positions, slices, graphs, streams,
autograd."""
import pytest
import torch

import linear_recurrence_chunked_gated_amd as gdn
from decay_testutil import rotary_bwd_ref, rotary_ref
from layer_testutil import DT, check

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _inputs(N, Hq, Hk, D, F, dtype, seed, far=1 << 18):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g)
    d = dict(q=rnd(N, Hq, D).to(DT[dtype]), k=(2 * rnd(N, Hk, D)).to(DT[dtype]),
             pos=torch.randint(0, far, (N,), generator=g).to(torch.int32),
             freq=10000.0 ** (-torch.arange(F).float() / max(F, 1)) if F else None,
             wq=1 + 0.3 * rnd(D), wk=1 + 0.3 * rnd(D), dyq=rnd(N, Hq, D).to(DT[dtype]),
             dyk=rnd(N, Hk, D).to(DT[dtype]))
    return d


def _cuda(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def _fwd(c, **kw):
    r = gdn.qk_norm_rotary_fwd(c["q"], c["k"], c["pos"], c["freq"], c["wq"], c["wk"], eps=EPS, **kw)
    torch.cuda.synchronize()
    return r


def _bwd(c, **kw):
    r = gdn.qk_norm_rotary_bwd(c["q"], c["k"], c["pos"], c["freq"], c["wq"], c["wk"], c["dyq"],
                               c["dyk"], eps=EPS, **kw)
    torch.cuda.synchronize()
    return r


# a wave's tokens in one lane's registers, 8 rows of a wave, 4 waves, 512 groups in a tree
def _depth(N, H):
    return (N // 2048 + 1) * (H + 1) + 64 + 10


CASES = [
    (1, 16, 16, 128, 64, "halves", "bf16"),
    (1, 1, 1, 64, 32, "neighbours", "f32"),
    (3, 3, 1, 64, 16, "halves", "f32"),
    (5, 2, 2, 72, 32, "halves", "bf16"),         # 9 of 16 lanes
    (5, 2, 2, 72, 36, "neighbours", "f32"),      # all of an odd number of lanes
    (7, 4, 2, 8, 4, "neighbours", "f32"),
    (9, 6, 2, 256, 128, "halves", "bf16"),
    (2, 5, 1, 512, 8, "halves", "f32"),
    (33, 1, 7, 128, 0, "halves", "bf16"),        # no rotation
    (131, 33, 2, 128, 64, "neighbours", "bf16"),  # heads that no wave divides
    (4099, 2, 1, 64, 32, "halves", "f32"),
]


@pytest.mark.parametrize("N,Hq,Hk,D,F,pairs,dtype", CASES)
def test_forward_and_backward_match(N, Hq, Hk, D, F, pairs, dtype):
    d = _inputs(N, Hq, Hk, D, F, dtype, seed=N + D + F)
    c = _cuda(d)
    opts = dict(q_scale=0.3, k_scale=1.7, pairs=pairs)
    for name, y, x, w, s in zip(("yq", "yk"), _fwd(c, **opts), (d["q"], d["k"]), (d["wq"], d["wk"]),
                                (0.3, 1.7)):
        ref, b = rotary_ref(x, d["pos"], d["freq"], w, EPS, s, pairs)
        check(name, y, ref, b, dtype)
    dq, dk, dwq, dwk = _bwd(c, **opts)
    for name, dx, dw, x, w, dy, s in (("q", dq, dwq, d["q"], d["wq"], d["dyq"], 0.3),
                                      ("k", dk, dwk, d["k"], d["wk"], d["dyk"], 1.7)):
        (rx, rw), (bx, bw) = rotary_bwd_ref(x, d["pos"], d["freq"], w, dy, EPS, s, pairs,
                                            _depth(N, x.shape[1]))
        check("d" + name, dx, rx, bx, dtype)
        check("dw" + name, dw, rw, bw, None)


@pytest.mark.parametrize("wq,wk", [(False, False), (True, False), (False, True)])
def test_without_weights(wq, wk):
    d = _inputs(50, 3, 2, 64, 32, "f32", seed=7)
    if not wq:
        d["wq"] = None
    if not wk:
        d["wk"] = None
    c = _cuda(d)
    got = _bwd(c)
    for i, (n, y) in enumerate(zip("qk", _fwd(c))):
        ref, b = rotary_ref(d[n], d["pos"], d["freq"], d["w" + n], EPS, 1.0, "halves")
        check("y" + n, y, ref, b, "f32")
        (rx, rw), (bx, bw) = rotary_bwd_ref(d[n], d["pos"], d["freq"], d["w" + n], d["dy" + n], EPS,
                                            1.0, "halves", _depth(50, 3))
        check("d" + n, got[i], rx, bx, "f32")
        if d["w" + n] is None:
            assert got[2 + i] is None
        else:
            check("dw" + n, got[2 + i], rw, bw, None)
    a = _bwd(c, want_dw=False)
    assert a[2] is None and a[3] is None and torch.equal(a[0], got[0])


def test_far_and_negative_positions():
    """Angles of the first and last int32 positions; equal positions turn alike."""
    d = _inputs(6, 1, 1, 64, 32, "f32", seed=9)
    d["pos"] = torch.tensor([0, -1, 2 ** 31 - 1, -2 ** 31, 123456789, 1], dtype=torch.int32)
    yq, yk = _fwd(_cuda(d))
    ref, b = rotary_ref(d["q"], d["pos"], d["freq"], d["wq"], EPS, 1.0, "halves")
    check("yq", yq, ref, b, "f32")
    ref, b = rotary_ref(d["k"], d["pos"], d["freq"], d["wk"], EPS, 1.0, "halves")
    check("yk", yk, ref, b, "f32")


@pytest.mark.parametrize("first", [0, 1000, -3])
def test_positions_by_the_row(first):
    """[B, T, H, D] without positions: first, first + 1, .. along T."""
    d = _inputs(2 * 37, 2, 1, 64, 32, "bf16", seed=11)
    c = _cuda(d)
    c["pos"] = (torch.arange(37, dtype=torch.int32) + first).repeat(2).cuda()
    want = _fwd(c) + _bwd(c)
    for n in ("q", "k", "dyq", "dyk"):
        c[n] = c[n].unflatten(0, (2, 37))
    c["pos"] = None
    got = _fwd(c, first=first) + _bwd(c, first=first)
    for x, y in zip(got, want):
        assert torch.equal(x.reshape(y.shape), y)


def test_slices_of_wider_rows():
    d = _inputs(70, 4, 2, 128, 64, "bf16", seed=13)
    c = _cuda(d)
    want = _fwd(c) + _bwd(c)
    wide = torch.cat([c["q"], c["k"], c["k"]], 1)
    c.update(q=wide[:, :4], k=wide[:, 4:6])
    assert not c["q"].is_contiguous()
    for x, y in zip(_fwd(c) + _bwd(c), want):
        assert torch.equal(x, y)


def test_zero_rows_empty_batches_and_eps_zero():
    """A row of zeros at eps = 0 is NaN itself and nothing beside it, dw aside;
    no tokens: dw is zeros."""
    d = _inputs(9, 3, 1, 64, 32, "f32", seed=15)
    c = _cuda(d)
    e = {n: None if t is None else t[:0] if n in ("q", "k", "pos", "dyq", "dyk") else t
         for n, t in c.items()}
    assert all(t.shape[0] == 0 for t in _fwd(e))
    g = _bwd(e)
    assert (g[2] == 0).all() and (g[3] == 0).all()
    args = (c["q"], c["k"], c["pos"], c["freq"], c["wq"], c["wk"])
    got = gdn.qk_norm_rotary_bwd(*args, c["dyq"], c["dyk"], eps=0.0)
    assert all(torch.isfinite(t).all() for t in got)
    c["q"][4, 1] = 0
    y = gdn.qk_norm_rotary_fwd(*args, eps=0.0)[0]
    bad = torch.isnan(y).any(-1)
    assert bad[4, 1] and bad.sum() == 1


def test_large_tensors_past_the_caches_and_their_bits():
    """Over 256 MB in all (the streamed forms), heads spread over the waves of
    one token in a small call: the same bits as the same rows in a large one."""
    N, Hq, Hk, D = 33000, 16, 16, 128
    g = torch.Generator(device="cuda").manual_seed(17)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    q, k, dyq, dyk = (r(N, Hq, D) for _ in range(4))
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    freq = (10000.0 ** (-torch.arange(64).float() / 64)).cuda()
    w = (1 + 0.1 * torch.randn(D, generator=g, device="cuda"))
    yq, yk = gdn.qk_norm_rotary_fwd(q, k, pos, freq, w, w)
    dq, dk, dwq, dwk = gdn.qk_norm_rotary_bwd(q, k, pos, freq, w, w, dyq, dyk)
    for sl in (slice(0, 1), slice(32990, 33000), slice(100, 400)):
        y1 = gdn.qk_norm_rotary_fwd(q[sl], k[sl], pos[sl], freq, w, w)
        assert torch.equal(y1[0], yq[sl]) and torch.equal(y1[1], yk[sl])
        d1 = gdn.qk_norm_rotary_bwd(q[sl], k[sl], pos[sl], freq, w, w, dyq[sl], dyk[sl])
        assert torch.equal(d1[0], dq[sl]) and torch.equal(d1[1], dk[sl])
    again = gdn.qk_norm_rotary_bwd(q, k, pos, freq, w, w, dyq, dyk)
    assert torch.equal(again[2], dwq) and torch.equal(again[3], dwk)
    xd, gd = q.double(), dyq.double()
    n = xd / (xd.square().mean(-1, keepdim=True) + EPS).sqrt()
    ang = pos.double()[:, None] * freq.double()
    cs, sn = ang.cos()[:, None], ang.sin()[:, None]
    back = torch.cat([gd[..., :64] * cs + gd[..., 64:] * sn, gd[..., 64:] * cs - gd[..., :64] * sn], -1)
    want = (back * n).sum((0, 1))
    assert float((dwq.double() - want).norm() / want.norm()) < 5e-6


def test_offsets_past_32_bits():
    """Rows past 2^31 elements of a strided tensor."""
    N, D, wide = 140_000, 128, 16384
    x = torch.empty(N, wide // D, D, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(19)
    x[-5:].normal_(generator=g)
    q, k = x[-3:, :2], x[-3:, 2:3]
    freq = (10000.0 ** (-torch.arange(64).float() / 64)).cuda()
    want = gdn.qk_norm_rotary_fwd(q.clone(), k.clone(), None, freq, first=N - 3)
    x[:-5] = 1.0
    got = gdn.qk_norm_rotary_fwd(x[:, :2], x[:, 2:3], None, freq)
    assert torch.equal(got[0][-3:], want[0]) and torch.equal(got[1][-3:], want[1])


def test_given_stream_and_outputs():
    d = _inputs(300, 4, 2, 128, 64, "bf16", seed=21)
    c = _cuda(d)
    want = _fwd(c) + _bwd(c)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = (torch.zeros_like(c["q"]), torch.zeros_like(c["k"]))
    g = (torch.zeros_like(c["q"]), torch.zeros_like(c["k"]), torch.zeros_like(c["wq"]),
         torch.zeros_like(c["wk"]))
    torch.cuda.synchronize()
    got = _fwd(c, stream=side, yq=y[0], yk=y[1]) + _bwd(c, stream=side, grads=g)
    assert got[0].data_ptr() == y[0].data_ptr() and got[4].data_ptr() == g[2].data_ptr()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    got = _fwd(c, stream=side) + _bwd(c, stream=side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_captured_and_replayed():
    d = _inputs(40, 4, 2, 64, 32, "bf16", seed=23)
    c = _cuda(d)
    f = lambda: (gdn.qk_norm_rotary_fwd(c["q"], c["k"], c["pos"], c["freq"], c["wq"], c["wk"])
                 + gdn.qk_norm_rotary_bwd(c["q"], c["k"], c["pos"], c["freq"], c["wq"], c["wk"],
                                          c["dyq"], c["dyk"]))
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    for rep in range(3):
        e = _cuda(_inputs(40, 4, 2, 64, 32, "bf16", seed=30 + rep))
        for n in c:
            c[n].copy_(e[n])
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for x, y in zip(got, f()):
            assert torch.equal(x, y), rep


@pytest.mark.parametrize("use", [(1, 1), (1, 0), (0, 1)])
def test_autograd_against_64_bits(use):
    """Both outputs and each alone; a key broadcast over the batch."""
    d = _inputs(2 * 20, 4, 2, 64, 16, "f32", seed=41)
    g = torch.Generator().manual_seed(42)
    up = torch.randn(2, 20, 4, 64, generator=g), torch.randn(2, 20, 2, 64, generator=g)

    def run(dev, dt, f):
        leaves = [d["q"].unflatten(0, (2, 20)), d["k"][:20].unflatten(0, (1, 20)), d["wq"], d["wk"]]
        q, k, wq, wk = x = [t.to(dev, dt).clone().requires_grad_() for t in leaves]
        yq, yk = f(q, k.expand(2, -1, -1, -1).contiguous(), wq, wk)
        sum((y * u.to(dev, dt)).sum() for y, u, on in zip((yq, yk), up, use) if on).backward()
        return [None if t.grad is None else t.grad.cpu().double() for t in x]

    def plain(q, k, wq, wk):
        pos = torch.arange(20) + 5
        return [rotary_plain(x, pos, d["freq"], w, s) for x, w, s in ((q, wq, 0.5), (k, wk, 1.0))]

    def rotary_plain(x, pos, freq, w, s):
        z = s * w * x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        F = freq.numel()
        a = (pos.double()[:, None] * freq.double())[:, None]
        z1, z2 = z[..., 0:2 * F:2], z[..., 1:2 * F:2]
        t = torch.stack([z1 * a.cos() - z2 * a.sin(), z2 * a.cos() + z1 * a.sin()], -1).flatten(-2)
        return torch.cat([t, z[..., 2 * F:]], -1)

    got = run("cuda", torch.float32, lambda q, k, wq, wk: gdn.qk_norm_rotary(
        q, k, None, d["freq"].cuda(), wq, wk, eps=EPS, q_scale=0.5, pairs="neighbours", first=5))
    ref = run("cpu", torch.float64, plain)
    for name, x, r in zip(("q", "k", "wq", "wk"), got, ref):
        if r is None or not r.abs().max():
            assert x is None or not x.abs().max()
        else:
            assert (x - r).norm() <= 2e-6 * r.norm(), (name, float((x - r).norm() / r.norm()))


def test_frequencies_that_want_a_gradient_are_refused():
    q = torch.randn(2, 1, 64, device="cuda")
    with pytest.raises(ValueError, match="no gradient"):
        gdn.qk_norm_rotary(q, q, None, torch.ones(8, device="cuda", requires_grad=True))
    with pytest.raises(ValueError, match="pairs"):
        gdn.qk_norm_rotary_fwd(q, q, pairs="other")
