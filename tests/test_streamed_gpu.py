"""Calls large enough that their kernels go past the caches (bf16 norms over
more than 256 MB, steps over 128 MiB of states): one case at least for each
form of such a kernel.  Rows are independent, so outputs equal, bit for bit,
those of the same rows in calls too small for that; the sums over rows are
checked against 64 bits."""
import pytest
import torch

import linear_recurrence_chunked_gated_amd as gdn
from layer_testutil import DT, check, gated_norm_bwd_ref, residual_norm_bwd_ref

pytestmark = pytest.mark.gpu

EDGE = 256 << 20  # bytes of all token tensors


def _rnd(g, *s):
    return torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)


def _parts(N, bytes_a_row):
    """Row ranges whose calls stay below the edge."""
    step = EDGE // bytes_a_row - 1
    return [slice(i, min(N, i + step)) for i in range(0, N, step)]


def _same(whole, parts, fn):
    """Each of whole's tensors equals fn's on the parts, to the bit."""
    for p in parts:
        for a, b in zip(whole, fn(p)):
            assert (a is None) == (b is None)
            if a is not None:
                assert torch.equal(a[p], b)


def _depth(rows, groups, rows_a_group):
    """Adds on the longest path of a sum over rows: a lane's turns, the
    workgroup's rows, then the partials on 128 sets and a tree."""
    return -(-rows // (groups * rows_a_group)) + rows_a_group + -(-groups // 128) + 8


@pytest.mark.parametrize("H,D,gate,weight,sliced,act", [
    (4, 64, True, True, False, 1),      # 8 lanes a head row
    (2, 72, True, True, True, 1),       # 16, some past the row's end; slices of wider rows
    (8, 128, False, False, False, 1),   # the L2 norm
    (2, 256, True, True, True, 0),      # 32
    (1, 264, False, True, False, 1),    # 64, some past the row's end
    (1, 512, True, True, False, 1),
])
def test_gated_norm(H, D, gate, weight, sliced, act):
    g = torch.Generator(device="cuda").manual_seed(D + H)
    N = EDGE // (2 * (3 if gate else 2) * H * D) + 37
    head = lambda: _rnd(g, N, 3 * H, D)[:, H:2 * H] if sliced else _rnd(g, N, H, D)
    x, gt, dy = head(), head() if gate else None, _rnd(g, N, H, D)
    w = torch.linspace(0.5, 1.5, D, device="cuda") if weight else None
    kw = dict(eps=1e-6, scale=1.0 if weight else D ** -0.5, act=act)
    cut = lambda t, p: None if t is None else t[p]
    y = gdn.gated_norm_fwd(x, gt, w, **kw)
    _same((y,), _parts(N, 2 * 3 * H * D), lambda p: (gdn.gated_norm_fwd(x[p], cut(gt, p), w, **kw),))
    del y
    dx, dg, dw = gdn.gated_norm_bwd(x, gt, w, dy, **kw)
    _same((dx, dg), _parts(N, 2 * 5 * H * D),
          lambda p: gdn.gated_norm_bwd(x[p], cut(gt, p), w, dy[p], **kw)[:2])
    if weight:
        lanes = next(n for n in (8, 16, 32, 64) if 8 * n >= D)
        refs, bounds = gated_norm_bwd_ref(x, gt, w, dy, depth=_depth(N * H, 512, 256 // lanes), **kw)
        check("dw", dw, refs[2].cpu(), bounds[2].cpu(), "f32")


@pytest.mark.parametrize("C,r,s,dh", [
    (72, True, True, True),        # 16 lanes a row
    (512, True, True, False),      # 64
    (1288, False, False, False),   # 256: the norm alone
    (2056, True, True, True),      # 512
    (8192, True, False, True),     # 1024
    (8200, True, True, True),      # two pieces a lane
    (16384, True, True, False),
])
def test_residual_norm(C, r, s, dh):
    g = torch.Generator(device="cuda").manual_seed(C)
    N = EDGE // (2 * (4 if r else 2) * C) + 5
    x, dy = _rnd(g, N, C), _rnd(g, N, C)
    rr, hh = _rnd(g, N, C) if r else None, _rnd(g, N, C) if dh else None
    w = torch.linspace(0.5, 1.5, C, device="cuda")
    sv = w.flip(0).contiguous() if s else None
    kw = dict(scale=0.5, eps=1e-6)
    cut = lambda t, p: None if t is None else t[p]
    y, h = gdn.residual_norm_fwd(x, rr, w, sv, **kw)
    _same((y, h), _parts(N, 2 * 4 * C), lambda p: gdn.residual_norm_fwd(x[p], cut(rr, p), w, sv, **kw))
    del y
    N = min(N, EDGE // (2 * (4 + dh + s) * C) + 5)  # the backward's edge
    h, dy, rr, hh = h[:N], dy[:N], cut(rr, slice(N)), cut(hh, slice(N))
    got = gdn.residual_norm_bwd(h, rr, w, sv, dy, hh, **kw)
    _same(got[:2], _parts(N, 2 * 6 * C),
          lambda p: gdn.residual_norm_bwd(h[p], cut(rr, p), w, sv, dy[p], cut(hh, p), **kw)[:2])
    rows = 16 if C <= 128 else 4 if C <= 512 else 1
    groups = 256 if C > 2048 else 512
    one = torch.ones(C, device="cuda")
    refs, bounds = residual_norm_bwd_ref(h, rr, w, one if sv is None else sv, dy, hh, 1e-6, 0.5,
                                         depth=_depth(N, groups, rows))
    check("dw", got[2], refs[2].cpu(), bounds[2].cpu(), "f32")
    if s:
        check("ds", got[3], refs[3].cpu(), bounds[3].cpu(), "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 9])
def test_step_of_64_wide_states(T, dtype):
    """A sequence alone, in a batch of 40, and in one of 520 (136 MB of
    states): the same outputs and state, to the bit."""
    n, H, D = 520, 16, 64
    g = torch.Generator(device="cuda").manual_seed(82)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    q, k = (torch.nn.functional.normalize(rnd(n, T, H, D), dim=-1).to(DT[dtype]) for _ in range(2))
    v, al, be = rnd(n, T, H, D).to(DT[dtype]), rnd(n, T, H).sigmoid(), rnd(n, T, H).sigmoid()
    pool = rnd(n, H, D, D)
    flat = lambda t, m: t[:m].reshape(m * T, *t.shape[2:]).contiguous()
    out = []
    for m in (1, 40, n):
        S = pool[:m].clone()
        out.append((gdn.recurrent_step(*(flat(t, m) for t in (q, k, v, al, be)), S), S))
    torch.cuda.synchronize()
    (o1, s1), (o40, s40), (on, sn) = out
    assert torch.equal(on[:40 * T], o40) and torch.equal(sn[:40], s40)
    assert torch.equal(o40[:T], o1) and torch.equal(s40[:1], s1)
