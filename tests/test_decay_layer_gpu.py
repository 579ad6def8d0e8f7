"""The operators of a layer of linear attention with a decay together: one
training layer (norm and rotation of q and k, the chunk, the gated norm of its
outputs) and its gradients, and a packed batch of prompts that goes on token by
token from the states the chunk left."""
import pytest
import torch

import linear_recurrence_chunked_gated_amd as gdn
from gdn_testutil import TOL, assert_close, f64

pytestmark = pytest.mark.gpu

HK, HV, D, EPS = 2, 4, 64, 1e-6
C = HV * D
FREQ = 10000.0 ** (-torch.arange(D // 2).float() / (D // 2))
DECAY = 1 - 2.0 ** -torch.linspace(2, 8, HV)


def _weights():
    g = torch.Generator().manual_seed(21)
    r = lambda *s: torch.randn(s, generator=g)
    return dict(norm=1 + 0.1 * r(C), qkv=r(C, (2 * HK + HV) * D) / C ** 0.5, wq=1 + 0.1 * r(D),
                wk=1 + 0.1 * r(D), gate=r(C, C) / C ** 0.5, onorm=1 + 0.1 * r(D),
                out=r(C, C) / C ** 0.5)


def _mm(x, w):
    acc = torch.promote_types(x.dtype, torch.float32)
    return (x.to(acc) @ w).to(x.dtype)


def _project(n, p):
    """q, k and v as slices of one projection's rows."""
    u = _mm(n, p["qkv"])
    u = u.view(*u.shape[:-1], 2 * HK + HV, D)
    return u[..., :HK, :], u[..., HK:2 * HK, :], u[..., 2 * HK:, :]


def _train(x, p, ops):
    norm, turn, chunk, onorm = ops
    n = norm(x, p["norm"])
    q, k, v = _project(n, p)
    q, k = turn(q, k, p["wq"], p["wk"])
    o = chunk(q, k, v)
    y = onorm(o, _mm(n, p["gate"]).view(o.shape), p["onorm"])
    return x + _mm(y.reshape(x.shape), p["out"])


def _ours():
    return (lambda x, w: gdn.residual_norm(x, None, w, None, eps=EPS)[0],
            lambda q, k, wq, wk: gdn.qk_norm_rotary(q, k, None, FREQ.cuda(), wq, wk, eps=EPS,
                                                    q_scale=D ** -0.5, k_scale=D ** -0.5),
            lambda q, k, v: gdn.decay_chunk(q, k, v, DECAY.cuda())[0],
            lambda o, g, w: gdn.gated_norm(o, g, w, eps=EPS))


def _plain():
    rms = lambda x: x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)

    def turn(q, k, wq, wk):
        a = (torch.arange(q.shape[1]).double()[:, None] * FREQ.double())[:, None]
        out = []
        for x, w in ((q, wq), (k, wk)):
            z = D ** -0.5 * w * rms(x)
            z1, z2 = z[..., :D // 2], z[..., D // 2:]
            out.append(torch.cat([z1 * a.cos() - z2 * a.sin(), z2 * a.cos() + z1 * a.sin()], -1))
        return out

    def chunk(q, k, v):
        q, k = q.repeat_interleave(HV // HK, 2), k.repeat_interleave(HV // HK, 2)
        t = torch.arange(q.shape[1])
        gap = t[:, None] - t
        M = torch.where(gap >= 0, DECAY.double()[:, None, None] ** gap.clamp(min=0).double(), 0.0)
        q, k, v = (z.transpose(1, 2) for z in (q, k, v))
        return (((q @ k.transpose(2, 3)) * M) @ v).transpose(1, 2)

    return (lambda x, w: rms(x) * w, turn, chunk,
            lambda o, g, w: rms(o) * w * torch.nn.functional.silu(g))


def test_training_layer_and_its_gradients():
    """fp32 against the same layer in 64 bits (torch autograd on the CPU), at
    the bar that the chunk's fp32 outputs are held to."""
    p = _weights()
    g = torch.Generator().manual_seed(22)
    x, dy = (torch.randn(2, 290, C, generator=g) for _ in range(2))

    def run(dev, dt, ops):
        leaves = {n: t.to(dev, dt).requires_grad_() for n, t in p.items()}
        xx = x.to(dev, dt).requires_grad_()
        y = _train(xx, leaves, ops)
        y.backward(dy.to(dev, dt))
        return [y, xx.grad] + [leaves[n].grad for n in sorted(leaves)]

    got = run("cuda", torch.float32, _ours())
    torch.cuda.synchronize()
    ref = run("cpu", torch.float64, _plain())
    for name, a, b in zip(["y", "dx"] + sorted(p), got, ref):
        assert_close(name, f64(a), f64(b), TOL["f32"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prompts_go_on_by_single_tokens(dtype):
    """Three packed prompts through the chunk, then four tokens one at a time
    over the pool: the rows that the chunk gives over all of them."""
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    p = {n: t.cuda() for n, t in _weights().items()}
    lens = [70, 5, 260]
    xs = [torch.randn(n + 4, C, generator=torch.Generator().manual_seed(30 + n)).to(dt).cuda()
          for n in lens]
    want = [_train(x[None], p, _ours())[0] for x in xs]
    freq, decay = FREQ.cuda(), DECAY.cuda()

    def layer(x, pos, attend):
        n = gdn.residual_norm_fwd(x, None, p["norm"], eps=EPS)[0]
        q, k, v = _project(n, p)
        q, k = gdn.qk_norm_rotary_fwd(q, k, pos, freq, p["wq"], p["wk"], eps=EPS,
                                      q_scale=D ** -0.5, k_scale=D ** -0.5)
        o = attend(q, k, v)
        y = gdn.gated_norm_fwd(o, _mm(n, p["gate"]).view(o.shape), p["onorm"], eps=EPS)
        return x + _mm(y.view(x.shape), p["out"])

    start = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()
    pool = torch.zeros(5, HV, D, D, device="cuda")
    slots = torch.tensor([4, 1, 2], dtype=torch.int32).cuda()

    def prompt(q, k, v):
        o, S = gdn.decay_chunk_fwd(q, k, v, decay, seq_start=start)
        pool[slots.long()] = S
        return o

    y = layer(torch.cat([x[:n] for x, n in zip(xs, lens)]), pos, prompt)
    for i, n in enumerate(lens):
        assert_close("prompt%d" % i, f64(y[start[i]:start[i + 1]]), f64(want[i][:n]), TOL[dtype])
    for t in range(4):
        x = torch.stack([x[n + t] for x, n in zip(xs, lens)])
        at = torch.tensor([n + t for n in lens], dtype=torch.int32).cuda()
        y = layer(x, at, lambda q, k, v: gdn.decay_step(q, k, v, decay, pool, slots))
        for i, n in enumerate(lens):
            assert_close("token%d.%d" % (i, t), f64(y[i]), f64(want[i][n + t]), TOL[dtype])
    assert torch.count_nonzero(pool[[0, 3]]) == 0
