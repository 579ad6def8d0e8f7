"""decay_step (single tokens over a pool of states) against its 64-bit form:
token types, head layouts, ragged and empty sequences, strided rows, padding,
refused entries, read-only calls, graph replay, other streams, offsets past 32
bits, and beside the chunk form."""
import pytest
import torch

import linear_recurrence_chunked_gated_amd as gdn
from decay_testutil import chunk_inputs, chunk_ref, step_ref
from layer_testutil import DT, U, check

pytestmark = pytest.mark.gpu


def _inputs(lens, Hk, Hv, D, dtype, n_slots, seed, extra=0):
    g = torch.Generator().manual_seed(seed)
    N = sum(lens) + extra
    rnd = lambda *s: torch.randn(s, generator=g)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    return dict(q=unit(rnd(N, Hk, D)).to(DT[dtype]), k=unit(rnd(N, Hk, D)).to(DT[dtype]),
                v=rnd(N, Hv, D).to(DT[dtype]), decay=1 - 2.0 ** -torch.linspace(1, 9, Hv),
                state=rnd(n_slots, Hv, D, D) * 0.3,
                slots=torch.randperm(n_slots, generator=g)[:len(lens)].to(torch.int32),
                seq_start=torch.tensor([0] + lens).cumsum(0).to(torch.int32))


def _cuda(d):
    return {k: v.cuda() for k, v in d.items()}


def _run(c, **kw):
    o = gdn.decay_step(c["q"], c["k"], c["v"], c["decay"], c["state"], c["slots"], c["seq_start"],
                       **kw)
    torch.cuda.synchronize()
    return o


@pytest.mark.parametrize("lens,Hk,Hv,D,dtype", [
    ([1], 1, 1, 64, "f32"),
    ([1], 16, 16, 128, "bf16"),
    ([1, 1, 1], 2, 2, 128, "f32"),
    ([1] * 7, 3, 6, 64, "bf16"),
    ([2, 1, 5, 3], 2, 4, 128, "bf16"),
    ([0, 3, 0, 1, 0], 2, 2, 64, "f32"),
    ([65, 1, 30], 2, 2, 128, "f32"),
    ([130], 1, 2, 64, "bf16"),
    ([1] * 70, 1, 1, 64, "bf16"),
])
def test_step_matches(lens, Hk, Hv, D, dtype):
    d = _inputs(lens, Hk, Hv, D, dtype, len(lens) + 3, seed=sum(lens) + D + Hv)
    (ro, rs), (ob, sb) = step_ref(d, lens, 0.7)
    c = _cuda(d)
    o = _run(c, scale=0.7)
    check("o", o, ro, ob, dtype)
    check("state", c["state"], rs, sb, None)
    used = d["slots"].tolist()
    idle = [i for i in range(len(lens) + 3) if i not in used or lens[used.index(i)] == 0]
    assert torch.equal(c["state"].cpu()[idle], d["state"][idle])


@pytest.mark.parametrize("decay", [0.0, 1.0])
def test_decays_at_their_ends(decay):
    d = _inputs([3, 20], 1, 2, 64, "f32", 3, seed=5)
    d["decay"].fill_(decay)
    (ro, rs), (ob, sb) = step_ref(d, [3, 20])
    c = _cuda(d)
    check("o", _run(c), ro, ob, "f32")
    check("state", c["state"], rs, sb, None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bits_do_not_depend_on_the_batch_or_the_call(dtype):
    """Nine tokens at once, one by one, and in a batch whose 147 MB of states
    go past the caches: the same bits; a read-only call leaves the pool."""
    n, T, Hh, D = 140, 9, 16, 128
    d = _inputs([T] * n, Hh, Hh, D, dtype, n, seed=81)
    c = _cuda(d)
    big = dict(c, state=c["state"].clone())
    o = _run(big)
    peek = dict(c, state=c["state"].clone())
    assert torch.equal(_run(peek, update=False), o) and torch.equal(peek["state"], c["state"])
    i = 77
    sl = slice(i * T, (i + 1) * T)
    one = dict(q=c["q"][sl], k=c["k"][sl], v=c["v"][sl], decay=c["decay"], state=c["state"].clone(),
               slots=c["slots"][i:i + 1], seq_start=None)
    assert torch.equal(_run(one), o[sl])
    s = int(d["slots"][i])
    assert torch.equal(one["state"][s], big["state"][s])
    st = c["state"].clone()
    for t in range(T):
        r = slice(i * T + t, i * T + t + 1)
        y = gdn.decay_step(c["q"][r], c["k"][r], c["v"][r], c["decay"], st, c["slots"][i:i + 1])
        assert torch.equal(y, o[r]), t
    assert torch.equal(st, one["state"])


def test_without_slots_and_offsets():
    d = _inputs([3] * 5, 2, 4, 64, "bf16", 5, seed=3)
    d["slots"] = torch.arange(5, dtype=torch.int32)
    a, b = _cuda(d), _cuda(d)
    o = _run(a)
    p = gdn.decay_step(b["q"], b["k"], b["v"], b["decay"], b["state"])
    torch.cuda.synchronize()
    assert torch.equal(o, p) and torch.equal(a["state"], b["state"])


def test_padding_refused_entries_and_rows_of_no_sequence():
    """Negative slots, slots past the pool, a repeated slot, rows behind the
    last sequence; offsets past the rows."""
    lens = [2, 3, 1, 2, 1]
    d = _inputs(lens, 1, 2, 64, "f32", 6, seed=13, extra=4)
    d["slots"] = torch.tensor([4, -1, 6, 4, 2], dtype=torch.int32)
    c = _cuda(d)
    o = torch.full_like(c["v"], 7)
    before = c["state"].clone()
    _run(c, o=o)
    o = o.cpu()
    assert (o[2:5] == 7).all() and (o[9:] == 7).all()          # padding, no sequence
    assert torch.isnan(o[5:6]).all() and torch.isnan(o[6:8]).all()  # past the pool, repeated
    keep = [0, 1, 3, 5]
    assert torch.equal(c["state"][keep], before[keep])
    e = dict(d, slots=torch.tensor([4, 2], dtype=torch.int32))
    rows = torch.tensor([0, 1, 8])
    for n in ("q", "k", "v"):
        e[n] = d[n][rows]
    e["seq_start"] = torch.tensor([0, 2, 3], dtype=torch.int32)
    (ro, rs), (ob, sb) = step_ref(e, [2, 1])
    check("o", o[rows], ro, ob, "f32")
    check("state", c["state"], rs, sb, None)
    c = _cuda(d)
    c["seq_start"] = torch.tensor([-9, 2, 1, 99, 99, 99], dtype=torch.int32).cuda()
    o = torch.full_like(c["v"], 7)
    _run(c, o=o)                                                # clamped: within the rows
    assert (c["state"][keep] == before[keep]).all()


def test_strided_rows_and_other_streams():
    d = _inputs([2, 1, 3], 2, 4, 64, "bf16", 4, seed=23)
    a, b, e = _cuda(d), _cuda(d), _cuda(d)
    o = _run(a)
    wide = torch.cat([b["q"], b["k"], b["v"]], 1)
    b.update(q=wide[:, :2], k=wide[:, 2:4], v=wide[:, 4:])
    assert torch.equal(_run(b), o) and torch.equal(a["state"], b["state"])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert torch.equal(_run(e, stream=side), o) and torch.equal(a["state"], e["state"])


def test_captured_and_replayed_for_other_batches():
    d = _inputs([1] * 6, 2, 2, 64, "bf16", 8, seed=33)
    c = _cuda(d)
    f = lambda: gdn.decay_step(c["q"], c["k"], c["v"], c["decay"], c["state"], c["slots"],
                               c["seq_start"])
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f()
    for rep, (lens, slots) in enumerate((([1] * 6, [0, 1, 2, 3, 4, 5]), ([0, 2, 1, 1, 0, 2], [7, 5, -1, 2, 0, 1]))):
        e = _cuda(_inputs(lens, 2, 2, 64, "bf16", 8, seed=40 + rep))
        e["slots"] = torch.tensor(slots, dtype=torch.int32).cuda()
        for n in c:
            c[n].copy_(e[n])
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        o = torch.full_like(out, 7)
        _run(e, o=o)
        assert torch.equal(out, o) and torch.equal(c["state"], e["state"]), rep


def test_offsets_past_32_bits():
    """A pool of 4.3e9 values and more: its last slot and its first."""
    Hh, D, n = 64, 128, 4200
    state = torch.zeros(n, Hh, D, D, device="cuda")
    d = _inputs([1, 1], Hh, Hh, D, "bf16", 2, seed=43)
    c = _cuda(d)
    state[[0, n - 1]] = c["state"]
    d["slots"] = torch.tensor([0, 1], dtype=torch.int32)
    (ro, rs), (ob, sb) = step_ref(d, [1, 1])
    c.update(state=state, slots=torch.tensor([0, n - 1], dtype=torch.int32).cuda())
    check("o", _run(c), ro, ob, "bf16")
    check("state", state[[0, n - 1]], rs, sb, None)
    assert torch.count_nonzero(state[1]) == 0 and torch.count_nonzero(state[n - 2]) == 0


def test_the_pool_counts_as_changed():
    d = _cuda(_inputs([1], 1, 1, 64, "f32", 1, seed=53))
    v = d["state"]._version
    _run(d, update=False)
    assert d["state"]._version == v
    _run(d)
    assert d["state"]._version > v


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_continue_a_chunk(dtype):
    """A prompt's chunk leaves its state in the pool; 20 steps on equal the
    chunk over all tokens, within the rounding of the chunk's operands."""
    d = chunk_inputs([90], 1, 2, 64, dtype, seed=63)
    (ro, rS), (ob, Sb) = chunk_ref(d)
    c = _cuda(d)
    cut = lambda sl: [c[n][sl] for n in ("q", "k", "v")]
    _, S = gdn.decay_chunk_fwd(*cut(slice(0, 70)), c["decay"], c["S_in"])
    pool = torch.zeros(3, 2, 64, 64, device="cuda")
    pool[1] = S[0]
    slot = torch.tensor([1], dtype=torch.int32).cuda()
    o = gdn.decay_step(*cut(slice(70, 90)), c["decay"], pool, slot)
    torch.cuda.synchronize()
    # the step rounds o alone; S's error (Sb at most) meets |q|, and 20 steps of fp32
    more = torch.einsum("nk,hvk->nhv", d["q"][70:, 0].double().abs(), Sb[0] + 40 * U * rS[0].abs() + 1e-6)
    check("o", o, ro[70:], more, dtype)
    check("S", pool[1], rS[0], Sb[0] + 40 * U * rS[0].abs() + 1e-6, None)
