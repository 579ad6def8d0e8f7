"""The operators together, as a layer uses them: one training layer through
the chunk and its gradients, and the same layer decoding token by token from
the states that a prompt's chunk left."""
import pytest
import torch

import linear_recurrence_chunked_gated_amd as gdn
from gdn_testutil import TOL, assert_close, f64

pytestmark = pytest.mark.gpu

H, D, W, EPS = 2, 64, 4, 1e-6
C = H * D


def _weights():
    g = torch.Generator().manual_seed(11)
    r = lambda *s: torch.randn(s, generator=g)
    p = dict(norm=1 + 0.1 * r(C), conv=r(3 * C, W) / W, onorm=1 + 0.1 * r(D), s=1 + 0.1 * r(C),
             out=r(C, C) / C ** 0.5, qkv=r(C, 3 * C) / C ** 0.5, gate=r(C, C) / C ** 0.5,
             ab=r(C, 2 * H) / C ** 0.5)
    return p


def _acc(x):
    return x.to(torch.promote_types(x.dtype, torch.float32))


def _gates(h, p):
    z = _acc(h) @ p["ab"]
    return torch.exp(-0.1 * torch.nn.functional.softplus(z[..., :H])), torch.sigmoid(z[..., H:])


def _mm(x, w):
    return (_acc(x) @ w).to(x.dtype)


def _train(x, p, ops):
    """One layer over x [B, T, C]; ops: the five operators."""
    norm, conv, l2, chunk, onorm = ops
    n = norm(x, None, p["norm"], None)[0]
    u = conv(_mm(n, p["qkv"]), p["conv"])
    q, k, v = (t.reshape(*t.shape[:2], H, D) for t in u.split(C, -1))
    al, be = _gates(n, p)
    o = chunk(l2(q), l2(k), v, al, be)
    y = onorm(o, _mm(n, p["gate"]).view(o.shape), p["onorm"])
    r = _mm(y.reshape(x.shape), p["out"])
    return norm(x, r, p["norm"], p["s"])  # the sum, and the next block's norm


def _ours():
    return (lambda x, r, w, s: gdn.residual_norm(x, r, w, s, eps=EPS),
            lambda x, w: gdn.short_conv(x.contiguous(), w, None, 1)[0],
            lambda x: gdn.gated_norm(x, scale=D ** -0.5, eps=EPS / D),
            lambda q, k, v, a, b: gdn.gated_delta_chunk(q, k, v.contiguous(), a.contiguous(),
                                                        b.contiguous())[0],
            lambda o, g, w: gdn.gated_norm(o, g, w, eps=EPS))


def _plain():
    def norm(x, r, w, s):
        h = x if r is None else x + s * r
        return h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * w, h

    def conv(x, w):
        e = torch.nn.functional.pad(x, (0, 0, W - 1, 0))
        return torch.nn.functional.silu(sum(e[:, W - 1 - j:e.shape[1] - j] * w[:, j]
                                            for j in range(W)))

    def chunk(q, k, v, a, b):
        S = torch.zeros(q.shape[0], H, D, D, dtype=q.dtype)
        out = []
        for t in range(q.shape[1]):
            kt, bt, at = k[:, t], b[:, t, :, None], a[:, t, :, None]
            u = bt * (v[:, t] - at * (S * kt[:, :, None]).sum(-1))
            S = at[..., None] * S + u[..., None] * kt[:, :, None]
            out.append((S * q[:, t, :, None]).sum(-1))
        return torch.stack(out, 1)

    return (norm, conv, lambda x: x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS), chunk,
            lambda o, g, w: o * torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS) * w
            * torch.nn.functional.silu(g))


def test_training_layer_and_its_gradients():
    """fp32 against the same layer in 64 bits (torch autograd on the CPU), at
    the bar that the chunk's fp32 outputs are held to."""
    p = _weights()
    g = torch.Generator().manual_seed(12)
    x, dy, dh = (torch.randn(2, 75, C, generator=g) for _ in range(3))

    def run(dev, dt, ops):
        leaves = {n: t.to(dev, dt).requires_grad_() for n, t in p.items()}
        xx = x.to(dev, dt).requires_grad_()
        y, h = _train(xx, leaves, ops)
        torch.autograd.backward((y, h), (dy.to(dev, dt), dh.to(dev, dt)))
        return [y, h, xx.grad] + [leaves[n].grad for n in sorted(leaves)]

    got = run("cuda", torch.float32, _ours())
    torch.cuda.synchronize()
    ref = run("cpu", torch.float64, _plain())
    for name, a, b in zip(["y", "h", "dx"] + sorted(p), got, ref):
        assert_close(name, f64(a), f64(b), TOL["f32"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decoding_continues_the_chunk(dtype):
    """Two prompts of 70 and 70 tokens through the chunk calls, then three
    tokens one at a time over the pools: the rows that the chunk calls give
    over all 73."""
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    p = {n: t.cuda() for n, t in _weights().items()}
    x = torch.randn(2, 73, C, generator=torch.Generator().manual_seed(13)).to(dt).cuda()
    y_all, h_all = _train(x, p, _ours())

    T = 70
    pool, cpool = torch.zeros(5, H, D, D).cuda(), torch.zeros(5, W - 1, 3 * C, dtype=dt).cuda()
    slots = torch.tensor([4, 1], dtype=torch.int32).cuda()
    n = gdn.residual_norm_fwd(x[:, :T].contiguous(), None, p["norm"], eps=EPS)[0]
    u, cs = gdn.shortconv_fwd(_mm(n, p["qkv"]), p["conv"], None, 1)
    q, k, v = (t.reshape(2, T, H, D).contiguous() for t in u.split(C, -1))
    al, be = _gates(n, p)
    l2 = lambda t: gdn.gated_norm_fwd(t, scale=D ** -0.5, eps=EPS / D)
    _, S = gdn.chunk_fwd(l2(q), l2(k), v, al.contiguous(), be.contiguous())
    pool[slots.long()], cpool[slots.long()] = S, cs

    for t in range(T, 73):
        xt = x[:, t].contiguous()
        n = gdn.residual_norm_fwd(xt, None, p["norm"], eps=EPS)[0]
        u = gdn.shortconv_step(_mm(n, p["qkv"]), p["conv"], cpool, slots, act=1)
        q, k, v = (u[:, i * C:(i + 1) * C].view(2, H, D) for i in range(3))
        al, be = _gates(n, p)
        o = gdn.recurrent_step(l2(q), l2(k), v, al.contiguous(), be.contiguous(), pool, slots)
        y = gdn.gated_norm_fwd(o, _mm(n, p["gate"]).view(2, H, D), p["onorm"], eps=EPS)
        y, h = gdn.residual_norm_fwd(xt, _mm(y.view(2, C), p["out"]), p["norm"], p["s"], eps=EPS)
        assert_close("y%d" % t, f64(y), f64(y_all[:, t]), TOL[dtype])
        assert_close("h%d" % t, f64(h), f64(h_all[:, t]), TOL[dtype])
    assert torch.count_nonzero(pool[[0, 2, 3]]) == 0
