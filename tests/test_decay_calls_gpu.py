"""Calls of linear attention with a decay and of the norm with rotation as a
user may make them: two at once, captured with their backward pass, with views
that are refused, with decays outside 0 .. 1 and values that are not finite."""
import pytest
import torch

import linear_recurrence_chunked_gated_amd as gdn
from decay_testutil import chunk_bwd_ref, chunk_inputs, chunk_ref
from layer_testutil import check

pytestmark = pytest.mark.gpu


def _cuda(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def _both(c, **kw):
    return (gdn.decay_chunk_fwd(c["q"], c["k"], c["v"], c["decay"], c["S_in"], c["seq_start"], **kw)
            + gdn.decay_chunk_bwd(c["q"], c["k"], c["v"], c["decay"], c["S_in"], c["dO"], c["dS_out"],
                                  c["seq_start"], **kw))


@pytest.mark.parametrize("lens", [[900, 100, 3], [40] * 70 + [500]])
def test_two_calls_at_once(lens):
    """Eager calls on two streams that do not wait for each other, each with
    its own workspace (both plans of packed sequences)."""
    cs = [_cuda(chunk_inputs(lens, 1, 2, 64, "bf16", seed=201 + i, grads=True)) for i in range(2)]
    want = [_both(c) for c in cs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for rep in range(3):
        for c, s, out in zip(cs, streams, got):
            out.append(_both(c, stream=s))
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        for o in outs:
            assert all(torch.equal(x, y) for x, y in zip(w, o))


def test_captured_training_step():
    """Norm, rotation and chunk with their backward pass in one graph, replayed
    for other values with the program's own eager steps between."""
    g = torch.Generator().manual_seed(211)
    r = lambda *s: torch.randn(*s, generator=g).cuda()
    freq = (10000.0 ** (-torch.arange(32) / 32)).cuda()
    decay = (1 - 2.0 ** -torch.linspace(2, 8, 4)).cuda()
    start = torch.tensor([0, 150, 151, 400], dtype=torch.int32, device="cuda")
    leaves = [r(400, 2, 64).bfloat16(), r(400, 2, 64).bfloat16(), r(400, 4, 64).bfloat16(), 1 + 0.1 * r(64),
              1 + 0.1 * r(64), r(3, 4, 64, 64)]
    up = r(400, 4, 64).bfloat16()

    def step(x):
        q, k = gdn.qk_norm_rotary(x[0], x[1], None, freq, x[3], x[4], q_scale=0.125)
        o, S = gdn.decay_chunk(q, k, x[2], decay, x[5], start)
        return (o, S) + torch.autograd.grad([o, S], x, [up, torch.ones_like(S)])

    def eager(values):
        return [t.detach().clone() for t in step([t.clone().requires_grad_() for t in values])]

    static = [t.clone().requires_grad_() for t in leaves]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = eager(leaves)  # on leaves of its own, gone before the capture
        del warm
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(static)
    for rep in range(3):
        values = [r(*t.shape).to(t.dtype) for t in leaves]
        with torch.no_grad():
            for s, v in zip(static, values):
                s.copy_(v)
        for t in out:
            t.detach().fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.detach().clone() for t in out]
        for x, y in zip(got, eager(values)):
            assert torch.equal(x, y), rep


@pytest.mark.parametrize("decay", [-0.75, 1.02, -1.0])
def test_decays_outside_the_usual_range(decay):
    d = chunk_inputs([200, 30], 1, 2, 64, "f32", seed=221, decay=decay, grads=True)
    (ro, rS), (ob, Sb) = chunk_ref(d)
    ref, bnd = chunk_bwd_ref(d)
    for name, x, r, b, t in zip(("o", "S", "dq", "dk", "dv", "dS"), _both(_cuda(d)), (ro, rS) + ref,
                                (ob, Sb) + bnd, ("f32", None, "f32", "f32", "f32", None)):
        check(name, x, r, b, t)


def test_a_head_whose_decay_is_not_finite():
    """It spoils its own head's outputs (and the shared heads' gradients), no
    other head's."""
    d = chunk_inputs([300, 40], 2, 2, 64, "bf16", seed=231, grads=True)
    c = _cuda(d)
    want = _both(c)
    got = _both(dict(c, decay=torch.tensor([float("nan"), float(c["decay"][1])], device="cuda")))
    for x, y in zip(want, got):
        assert torch.equal(x[:, 1], y[:, 1])


def test_one_tensor_as_all_inputs():
    """q, k, v and dO may be the same memory."""
    d = chunk_inputs([130], 2, 2, 64, "f32", seed=241, grads=True)
    d.update(k=d["q"], v=d["q"], dO=d["q"])
    c = _cuda(d)
    c.update(k=c["q"], v=c["q"], dO=c["q"])
    (ro, rS), (ob, Sb) = chunk_ref(d)
    ref, bnd = chunk_bwd_ref(d)
    for name, x, r, b, t in zip(("o", "S", "dq", "dk", "dv", "dS"), _both(c), (ro, rS) + ref, (ob, Sb) + bnd,
                                ("f32", None, "f32", "f32", "f32", None)):
        check(name, x, r, b, t)


def test_a_workspace_too_small():
    """The Python calls take one of their own instead, as the other calls do."""
    c = _cuda(chunk_inputs([700, 200], 1, 2, 64, "bf16", seed=246, grads=True))
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    for x, y in zip(_both(c), _both(c, workspace=small)):
        assert torch.equal(x, y)


def test_gradients_of_any_layout():
    """o's and S_out's gradients as expanded and transposed views."""
    d = chunk_inputs([70], 2, 2, 64, "f32", seed=251)
    c = _cuda(d)

    def run(views):
        x = [c[n].clone().requires_grad_() for n in ("q", "k", "v", "S_in")]
        o, S = gdn.decay_chunk(*x[:3], c["decay"], x[3])
        gen = torch.Generator().manual_seed(252)
        go = torch.randn(2, 70, 1, generator=gen).cuda().transpose(0, 1).expand(70, 2, 64)
        gS = torch.randn(1, 2, 64, 64, generator=gen).cuda().transpose(2, 3)
        if not views:
            go, gS = go.contiguous(), gS.contiguous()
        return torch.autograd.grad([o, S], x, [go, gS])

    for x, y in zip(run(True), run(False)):
        assert torch.equal(x, y)


def _refused():
    x = torch.zeros(6, 2, 64, device="cuda")
    v = torch.zeros(6, 4, 64, device="cuda")
    a, S = torch.ones(4, device="cuda"), torch.zeros(2, 4, 64, 64, device="cuda")
    st = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    f, b, t = gdn.decay_chunk_fwd, gdn.decay_chunk_bwd, gdn.decay_step
    fr = torch.ones(32, device="cuda")
    return {
        "offsets on the host": lambda: f(x, x, v, a, S, st.cpu()),
        "offsets of 64 bits": lambda: f(x, x, v, a, S, st.long()),
        "decay on the host": lambda: f(x, x, v, a.cpu(), S, st),
        "decay of 64 bits": lambda: f(x, x, v, a.double(), S, st),
        "decays for other heads": lambda: f(x, x, v, a[:2], S, st),
        "states for other sequences": lambda: f(x, x, v, a, S[:1], st),
        "states in bf16": lambda: f(x, x, v, a, S.bfloat16(), st),
        "k of another type": lambda: f(x, x.bfloat16(), v, a, S, st),
        "k of other rows": lambda: f(x, x[:5], v, a, S, st),
        "offsets for rows by the batch": lambda: f(x[None], x[None], v[None], a, S, st),
        "v without heads": lambda: f(x, x, v[:, 0], a, S, st),
        "heads that no group divides": lambda: f(x, x, v[:, :3].contiguous(), a[:3], S[:, :3].contiguous(), st),
        "half precision": lambda: f(x.half(), x.half(), v.half(), a, S, st),
        "transposed rows": lambda: f(x.transpose(1, 2).contiguous().transpose(1, 2), x, v, a, S, st),
        "a broadcast batch": lambda: f(x[None].expand(2, -1, -1, -1), x[None].expand(2, -1, -1, -1),
                                       v[None].expand(2, -1, -1, -1), a),
        "o on its input": lambda: f(v, v, v, a, S, st, o=v),
        "S_out on S_in": lambda: f(x, x, v, a, S, st, S_out=S),
        "a gradient of other rows": lambda: b(x, x, v, a, S, v[:5], None, st),
        "a transposed gradient": lambda: b(x, x, v, a, S, v.transpose(0, 1).contiguous().transpose(0, 1),
                                           None, st),
        "gradients on an input": lambda: b(x, x, v, a, S, v.clone(), None, st,
                                           grads=(x, x.clone(), v.clone(), S.clone())),
        "too few gradients": lambda: b(x, x, v, a, S, v.clone(), None, st, grads=(x.clone(), x.clone())),
        "a pool of other heads": lambda: t(x, x, v, a, S[:, :2].contiguous(), None, st),
        "slots for other sequences": lambda: t(x, x, v, a, S, torch.zeros(3, dtype=torch.int32, device="cuda"), st),
        "pairs of another kind": lambda: gdn.qk_norm_rotary_fwd(x, x, None, fr, pairs="both"),
        "more frequencies than pairs": lambda: gdn.qk_norm_rotary_fwd(x, x, None, torch.ones(40, device="cuda")),
        "positions of 64 bits": lambda: gdn.qk_norm_rotary_fwd(x, x, torch.zeros(6, dtype=torch.int64, device="cuda"), fr),
        "a weight of another size": lambda: gdn.qk_norm_rotary_fwd(x, x, None, fr, torch.ones(32, device="cuda")),
        "positions past 32 bits": lambda: gdn.qk_norm_rotary_fwd(x, x, None, fr, first=2 ** 31 - 2),
        "a negative epsilon": lambda: gdn.qk_norm_rotary_fwd(x, x, None, fr, eps=-1.0),
    }


@pytest.mark.parametrize("what", ["offsets on the host", "offsets of 64 bits", "decay on the host",
                                  "decay of 64 bits", "decays for other heads", "states for other sequences",
                                  "states in bf16", "k of another type", "k of other rows",
                                  "offsets for rows by the batch", "v without heads",
                                  "heads that no group divides", "half precision", "transposed rows",
                                  "a broadcast batch", "o on its input", "S_out on S_in",
                                  "a gradient of other rows", "a transposed gradient", "gradients on an input",
                                  "too few gradients", "a pool of other heads", "slots for other sequences",
                                  "pairs of another kind", "more frequencies than pairs", "positions of 64 bits",
                                  "a weight of another size", "positions past 32 bits", "a negative epsilon"])
def test_refused(what):
    with pytest.raises((ValueError, RuntimeError, TypeError)):
        _refused()[what]()


@pytest.mark.parametrize("lens,Hk,Hv,D,dtype", [
    ([130], 1, 1, 128, "bf16"), ([70, 1, 90], 2, 4, 64, "f32"), ([300, 0, 257], 1, 2, 128, "f32"),
    ([7000, 300, 9, 1003], 4, 16, 64, "bf16"),  # backward: 10 boundaries, segments of 13 blocks
    ([1, 5, 16990, 4], 8, 32, 64, "bf16"),      # forward: one sequence has nearly all of them
    ([4000, 3900, 4100, 3], 16, 32, 128, "bf16"),
])
def test_boundaries_joined_by_the_items_and_by_the_chain(lens, Hk, Hv, D, dtype):
    """Few boundaries are joined by every item for itself, more (and those of
    more than 64 sequences, most of them empty here) by a kernel: one result."""
    d = chunk_inputs(lens, Hk, Hv, D, dtype, seed=261 + sum(lens), grads=True)
    c, n = _cuda(d), len(lens)
    more = 65 - n
    ext = lambda x: torch.cat([x, x.new_zeros(more, *x.shape[1:])])
    m = dict(c, seq_start=torch.cat([c["seq_start"], c["seq_start"][-1:].expand(more)]),
             S_in=ext(c["S_in"]), dS_out=ext(c["dS_out"]))

    def run(x):
        o, S = gdn.decay_chunk_fwd(x["q"], x["k"], x["v"], x["decay"], x["S_in"], x["seq_start"])
        g = gdn.decay_chunk_bwd(x["q"], x["k"], x["v"], x["decay"], x["S_in"], x["dO"],
                                x["dS_out"], x["seq_start"])
        torch.cuda.synchronize()
        return (o, S[:n]) + tuple(g[:3]) + (g[3][:n],)

    for x, y in zip(run(c), run(m)):
        assert torch.isfinite(x).all() and torch.equal(x, y)
