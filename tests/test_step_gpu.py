"""The single-token calls over a pool of states (recurrent_step,
shortconv_step) against their 64-bit forms: token types, head layouts, ragged
and empty sequences, strided rows, padding, refused entries, read-only calls,
offsets past 32 bits, streams, graph replay."""
import pytest
import torch

import linear_recurrence_chunked_gated_amd as gdn
from gdn_testutil import TOL, assert_close, f64, inputs, to_dev
from layer_testutil import DT, check, conv_step_ref, step_inputs, step_ref

pytestmark = pytest.mark.gpu


def _cuda(d):
    return {k: v.cuda() for k, v in d.items()}


def _run(d, **kw):
    c = _cuda(d)
    o = gdn.recurrent_step(c["q"], c["k"], c["v"], c["alpha"], c["beta"], c["state"], c["slots"],
                           c["seq_start"], **kw)
    torch.cuda.synchronize()
    return o, c["state"]


@pytest.mark.parametrize("lens,Hk,Hv,D,dtype", [
    ([1], 1, 1, 64, "f32"),
    ([1], 16, 16, 128, "bf16"),
    ([1, 1, 1], 2, 2, 128, "f32"),
    ([1] * 7, 3, 6, 64, "bf16"),
    ([2, 1, 5, 3], 2, 4, 128, "bf16"),
    ([0, 3, 0, 1, 0], 2, 2, 64, "f32"),      # empty sequences keep their states
    ([4, 4, 4], 1, 3, 128, "f32"),
    ([65, 1, 30], 2, 2, 128, "f32"),
    ([130], 1, 2, 64, "bf16"),
    ([1] * 70, 1, 1, 64, "bf16"),            # more sequences than a wave has lanes
])
def test_step_matches(lens, Hk, Hv, D, dtype):
    d = step_inputs(lens, Hk, Hv, D, dtype, len(lens) + 3, seed=sum(lens) + D + Hv)
    ref_o, ob, ref_s, sb = step_ref(d, lens, D)
    o, state = _run(d)
    check("o", o, ref_o, ob, dtype)
    check("state", state, ref_s, sb, None)
    # slots of no sequence, and of empty ones, to the bit
    idle = [i for i in range(len(lens) + 3)
            if i not in d["slots"].tolist() or lens[d["slots"].tolist().index(i)] == 0]
    assert torch.equal(state.cpu()[idle], d["state"][idle])


@pytest.mark.parametrize("decay,beta", [(0.0, 1.0), (30.0, 0.5), (0.1, 0.0)])
def test_step_at_the_ends_of_the_gates(decay, beta):
    """No decay with full writes, near-total decay, no writes."""
    lens = [3, 40]
    d = step_inputs(lens, 2, 2, 64, "f32", 4, seed=77, decay=decay)
    d["beta"].fill_(beta)
    ref_o, ob, ref_s, sb = step_ref(d, lens, 64)
    o, state = _run(d)
    check("o", o, ref_o, ob, "f32")
    check("state", state, ref_s, sb, None)


def test_step_without_offsets_and_slots():
    """No seq_start: equal shares of the rows; no slots: sequence i has slot i."""
    lens = [3] * 5
    d = step_inputs(lens, 2, 4, 64, "bf16", 5, seed=3)
    a, sa = _run(d)
    c = _cuda(d)
    b = gdn.recurrent_step(c["q"], c["k"], c["v"], c["alpha"], c["beta"], c["state"], c["slots"])
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(sa, c["state"])
    d["slots"] = torch.arange(5, dtype=torch.int32)
    a, sa = _run(d)
    c = _cuda(d)
    b = gdn.recurrent_step(c["q"], c["k"], c["v"], c["alpha"], c["beta"], c["state"])
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(sa, c["state"])


def test_step_token_by_token_equals_one_call():
    """Five tokens in one call and in five calls: the same bits, and a
    read-only call gives the same outputs and leaves the pool."""
    lens = [5, 5, 5]
    d = step_inputs(lens, 2, 2, 128, "bf16", 4, seed=9)
    o, state = _run(d)
    c = _cuda(d)
    peek = gdn.recurrent_step(c["q"], c["k"], c["v"], c["alpha"], c["beta"], c["state"],
                              c["slots"], c["seq_start"], update=False)
    assert torch.equal(peek, o) and torch.equal(c["state"].cpu(), d["state"])
    outs = []
    for t in range(5):
        rows = torch.tensor([t, 5 + t, 10 + t]).cuda()
        outs.append(gdn.recurrent_step(*(c[n][rows] for n in ("q", "k", "v", "alpha", "beta")),
                                       c["state"], c["slots"]))
    torch.cuda.synchronize()
    assert torch.equal(torch.stack(outs, 1).reshape(o.shape), o)
    assert torch.equal(c["state"], state)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 9])
def test_step_bits_do_not_depend_on_the_batch(T, dtype):
    """A sequence alone, in a batch of 40, and in one of 140 (whose 147 MB of
    states go past the caches): the same outputs and state, to the bit."""
    H, D = 16, 128
    g = torch.Generator(device="cuda").manual_seed(81)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    n = 140
    q, k = (torch.nn.functional.normalize(rnd(n, T, H, D), dim=-1).to(DT[dtype]) for _ in range(2))
    v, al, be = rnd(n, T, H, D).to(DT[dtype]), rnd(n, T, H).sigmoid(), rnd(n, T, H).sigmoid()
    pool = rnd(n, H, D, D)
    flat = lambda t, m: t[:m].reshape(m * T, *t.shape[2:]).contiguous()
    out = []
    for m in (1, 40, n):
        S = pool[:m].clone()
        o = gdn.recurrent_step(*(flat(t, m) for t in (q, k, v, al, be)), S)
        out.append((o[:T], S[0]))
    torch.cuda.synchronize()
    for o, S in out[1:]:
        assert torch.equal(o, out[0][0]) and torch.equal(S, out[0][1])


@pytest.mark.parametrize("n", [3, 300, 700])
def test_repeated_slots_in_large_batches(n):
    """The last entry repeats the first one's slot, one in the middle its
    neighbour's: refused, and the others as without them."""
    H, D, C = 1, 64, 64
    lens = [1] * n
    d = step_inputs(lens, H, H, D, "f32", n, seed=n)
    ok, state_ok = _run(d)
    cg = torch.Generator().manual_seed(n)
    x, w = torch.randn(n, C, generator=cg).cuda(), torch.randn(C, 4, generator=cg).cuda()
    cst = torch.randn(n, 3, C, generator=cg)
    y_ok = gdn.shortconv_step(x, w, cst.cuda(), d["slots"].cuda())
    keep = d["slots"].clone()
    twice = {n - 1: 0, n // 2: n // 2 - 1}
    for i, j in twice.items():
        d["slots"][i] = keep[j]
    o, state = _run(d)
    pool = cst.cuda()
    y = gdn.shortconv_step(x, w, pool, d["slots"].cuda())
    torch.cuda.synchronize()
    good = [i for i in range(n) if i not in twice]
    assert torch.equal(o[good], ok[good]) and torch.equal(y[good], y_ok[good])
    assert torch.isnan(o[list(twice)]).all() and torch.isnan(y[list(twice)]).all()
    at = keep[good].long()
    assert torch.equal(state[at], state_ok[at])
    left = keep[list(twice)].long()  # slots that no entry names any more
    assert torch.equal(state.cpu()[left], d["state"][left])
    assert torch.equal(pool.cpu()[left], cst[left])


def test_two_calls_at_once():
    """Two streams, two pools, at the same time: as one after the other."""
    a = _cuda(step_inputs([3] * 30, 4, 4, 128, "bf16", 30, seed=91))
    b = _cuda(step_inputs([2] * 50, 4, 4, 128, "bf16", 50, seed=92))
    call = lambda c, s, st: gdn.recurrent_step(c["q"], c["k"], c["v"], c["alpha"], c["beta"], s,
                                               c["slots"], c["seq_start"], stream=st)
    want = []
    for c in (a, b):
        s = c["state"].clone()
        want += [call(c, s, None), s]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for c, st in zip((a, b), streams):
        s = c["state"].clone()
        st.wait_stream(torch.cuda.current_stream())
        got += [call(c, s, st), s]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_threads_on_streams_of_their_own():
    """Two host threads, each decoding 20 steps on its own stream and pool."""
    import threading
    batches = [_cuda(step_inputs([1] * n, 2, 2, 64, "bf16", n, seed=95 + n)) for n in (9, 33)]

    def decode(c, stream, out):
        with torch.cuda.stream(stream):
            s = c["state"].clone()
            for _ in range(20):
                o = gdn.recurrent_step(c["q"], c["k"], c["v"], c["alpha"], c["beta"], s, c["slots"])
                gdn.gated_norm_fwd(o, o)
            out.append((o, s))

    want, got = [], [[], []]
    for c in batches:
        decode(c, torch.cuda.current_stream(), want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    threads = [threading.Thread(target=decode, args=(c, st, out))
               for c, st, out in zip(batches, streams, got)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for (o, s), ((ro, rs),) in zip(want, got):
        assert torch.equal(o, ro) and torch.equal(s, rs)


def test_step_strided_rows():
    """q, k and v as slices of one projection's rows."""
    lens = [2, 7, 1]
    N, Hk, Hv, D = 10, 2, 4, 64
    d = step_inputs(lens, Hk, Hv, D, "bf16", 5, seed=21)
    o, state = _run(d)
    c = _cuda(d)
    wide = torch.full((N, (2 * Hk + Hv) * D + 40), float("nan"), dtype=torch.bfloat16).cuda()
    q = wide[:, 8:8 + Hk * D].view(N, Hk, D)
    k = wide[:, 8 + Hk * D:8 + 2 * Hk * D].view(N, Hk, D)
    v = wide[:, 16 + 2 * Hk * D:16 + (2 * Hk + Hv) * D].view(N, Hv, D)
    for view, n in ((q, "q"), (k, "k"), (v, "v")):
        view.copy_(c[n])
    o2 = gdn.recurrent_step(q, k, v, c["alpha"], c["beta"], c["state"], c["slots"], c["seq_start"])
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(state, c["state"])


def test_step_padding_and_refused_entries():
    """Negative slots, slots past the pool, a repeated slot, offsets outside
    the rows, rows after the last sequence; infinities and NaN in what is not
    to be read."""
    lens = [2, 1, 2, 3, 1, 2]
    D, N = 64, 14
    d = step_inputs(lens, 2, 2, D, "f32", 5, seed=33, extra_rows=3)
    slots = [3, -1, 5, 1, 3, -7]  # 5: past the pool; the second 3: a repeat
    d["slots"] = torch.tensor(slots, dtype=torch.int32)
    good = [0, 3]
    bounds = d["seq_start"].tolist()
    for i in range(6):
        if i not in good:
            for n in ("q", "k", "v", "alpha"):
                d[n][bounds[i]:bounds[i + 1]] = float("nan") if i % 2 else float("inf")
    d["q"][11:] = float("nan")
    one = {n: (d[n] if n == "state" else torch.cat([d[n][bounds[i]:bounds[i + 1]] for i in good]))
           for n in ("q", "k", "v", "alpha", "beta", "state")}
    one["slots"] = torch.tensor([3, 1])
    ref_o, ob, ref_s, sb = step_ref(one, [2, 3], D)
    mark = torch.full((N, 2, D), 7.0).cuda()
    o, state = _run(d, o=mark)
    rows = [0, 1, 5, 6, 7]
    check("o", o[rows], ref_o, ob, "f32")
    check("state", state, ref_s, sb, None)
    assert torch.isnan(o[[3, 4, 8]]).all()                 # the refused entries' rows
    assert (o[[2, 9, 10, 11, 12, 13]] == 7.0).all()        # padding and no sequence
    # only read, the pool may be shared by entries
    d["slots"] = torch.tensor([3, -1, 5, 1, 3, -7], dtype=torch.int32)
    for n in ("q", "k", "v", "alpha"):
        d[n][8] = d[n][0]
    d["beta"][8] = d["beta"][0]
    o, state = _run(d, o=torch.full((N, 2, D), 7.0).cuda(), update=False)
    assert torch.equal(o[8], o[0]) and torch.equal(state.cpu(), d["state"])
    # offsets that leave the rows, or run backwards, stay inside them
    d2 = step_inputs([2, 2], 2, 2, D, "f32", 4, seed=34)
    d2["seq_start"] = torch.tensor([-5, 2, 900], dtype=torch.int32)
    o, state = _run(d2)
    ref_o, ob, ref_s, sb = step_ref(d2, [2, 2], D)
    check("o", o, ref_o, ob, "f32")
    check("state", state, ref_s, sb, None)
    d2["seq_start"] = torch.tensor([4, 2, 1], dtype=torch.int32)
    o, state = _run(d2, o=torch.full((4, 2, D), 7.0).cuda())
    assert (o == 7.0).all() and torch.equal(state.cpu(), d2["state"])


def test_step_nan_and_inf_stay_in_their_sequence():
    lens = [2, 2, 2]
    d = step_inputs(lens, 2, 2, 64, "bf16", 3, seed=35)
    o, state = _run(d)
    d["v"][2] = float("nan")
    d["state"][d["slots"][2].long()] = float("inf")
    o2, state2 = _run(d)
    s0 = int(d["slots"][0])
    assert torch.equal(o2[:2], o[:2]) and torch.equal(state2[s0], state[s0])
    assert torch.isnan(o2[2:4]).all() and not torch.isfinite(o2[4:]).any()


def test_step_pool_past_32_bit_offsets():
    """A pool of 8.6 GB: the last slot's element offset passes 2^31, its byte
    offset 2^33."""
    H, D = 16, 128
    n_slots = (1 << 31) // (H * D * D) + 2
    d = step_inputs([2, 1], H, H, D, "bf16", 4, seed=41)
    ref_o, ob, ref_s, sb = step_ref(d, [2, 1], D)
    c = _cuda(d)
    pool = torch.zeros((n_slots, H, D, D), device="cuda")
    pool[n_slots - 4:] = c["state"]
    slots = c["slots"] + (n_slots - 4)
    o = gdn.recurrent_step(c["q"], c["k"], c["v"], c["alpha"], c["beta"], pool,
                           slots.to(torch.int32), c["seq_start"])
    torch.cuda.synchronize()
    check("o", o, ref_o, ob, "bf16")
    check("state", pool[n_slots - 4:], ref_s, sb, None)
    assert torch.count_nonzero(pool[:4]) == 0


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
def test_step_continues_a_chunk(dtype, D):
    """A prompt of 192 tokens through the chunk call, whose exit state is a
    pool slot, then 5 tokens through the step: the chunk over all 197."""
    H, T = 3, 197
    d = to_dev(inputs(1, T, H, D, dtype, seed=51, s_in_std=0.1, decay=0.05))
    fa = [d[n] for n in ("q", "k", "v", "alpha", "beta")]
    o_all, S_all = gdn.chunk_fwd(*fa, d["S_in"])
    pool = torch.zeros(4, H, D, D, device="cuda")
    cut = [t[:, :192].contiguous() for t in fa]
    gdn.chunk_fwd(*cut, d["S_in"], S_out=pool[2:3])
    o = gdn.recurrent_step(*(t[0, 192:].contiguous() for t in fa), pool,
                           torch.tensor([2], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert_close("o", f64(o), f64(o_all[0, 192:]), TOL[dtype], head_axis=1)
    assert_close("S", f64(pool[2]), f64(S_all[0]), TOL[dtype], head_axis=0)
    assert torch.count_nonzero(pool[[0, 1, 3]]) == 0


@pytest.mark.parametrize("lens,C,W,dtype,act", [
    ([1], 64, 4, "f32", 0),
    ([1] * 5, 6144, 4, "bf16", 1),
    ([0, 1, 2, 3, 4, 5, 9], 136, 4, "bf16", 1),
    ([3, 1, 20], 520, 8, "f32", 1),
    ([2, 1, 4], 72, 2, "f32", 0),
    ([2, 3], 8, 3, "bf16", 0),
    ([1, 2], 64, 1, "f32", 1),               # one tap: no state
    ([1] * 67, 40, 4, "f32", 1),
    ([1] * 300, 64, 4, "bf16", 1),
])
def test_conv_step_matches(lens, C, W, dtype, act):
    g = torch.Generator().manual_seed(C + W + len(lens))
    N, n_slots = sum(lens), len(lens) + 2
    x = torch.randn(N, C, generator=g).to(DT[dtype])
    w = torch.randn(C, W, generator=g) / W
    state = torch.randn(n_slots, W - 1, C, generator=g).to(DT[dtype])
    slots = torch.randperm(n_slots, generator=g)[:len(lens)].to(torch.int32)
    start = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    ref, bound, ref_s = conv_step_ref(x, w, state, slots, lens, act)
    pool = state.cuda()
    y = gdn.shortconv_step(x.cuda(), w.cuda(), pool, slots.cuda(), start.cuda(), act=act)
    torch.cuda.synchronize()
    check("y", y, ref, bound, dtype)
    assert torch.equal(pool.cpu(), ref_s)
    # only read: the same outputs, the pool as it was; and rows out of wider ones
    pool = state.cuda()
    wide = torch.full((N, C + 24), float("nan"), dtype=DT[dtype]).cuda()
    wide[:, 8:8 + C] = x.cuda()
    y2 = gdn.shortconv_step(wide[:, 8:8 + C], w.cuda(), pool, slots.cuda(), start.cuda(), act=act,
                            update=False)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(pool.cpu(), state)


def test_conv_step_continues_a_chunk():
    """A chunk's conv_out is a pool slot: the step continues it to the bit."""
    C, W, T = 128, 4, 37
    g = torch.Generator().manual_seed(8)
    x = torch.randn(1, T, C, generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn(C, W, generator=g) / W).cuda()
    y, cout = gdn.shortconv_fwd(x, w, None, 1)
    pool = torch.zeros(3, W - 1, C, dtype=torch.bfloat16, device="cuda")
    gdn.shortconv_fwd(x[:, :33].contiguous(), w, None, 1, conv_out=pool[1:2])
    y2 = gdn.shortconv_step(x[0, 33:], w, pool, torch.tensor([1], dtype=torch.int32).cuda(), act=1)
    torch.cuda.synchronize()
    assert torch.equal(y[0, 33:], y2) and torch.equal(pool[1:2], cout)


def test_conv_step_padding_and_refused_entries():
    C, W = 64, 4
    g = torch.Generator().manual_seed(9)
    lens = [2, 1, 2, 1, 2]
    x = torch.randn(10, C, generator=g)
    w = torch.randn(C, W, generator=g) / W
    state = torch.randn(4, W - 1, C, generator=g)
    slots = torch.tensor([2, -1, 4, 0, 2], dtype=torch.int32)
    start = torch.tensor([0, 2, 3, 5, 6, 8], dtype=torch.int32)
    ref, bound, ref_s = conv_step_ref(x[[0, 1, 5]], w, state, [2, 0], [2, 1], 1)
    pool = state.cuda()
    y = gdn.shortconv_step(x.cuda(), w.cuda(), pool, slots.cuda(), start.cuda(), act=1,
                           y=torch.full((10, C), 7.0).cuda())
    torch.cuda.synchronize()
    check("y", y[[0, 1, 5]], ref, bound, "f32")
    assert torch.equal(pool.cpu(), ref_s)
    assert torch.isnan(y[[3, 4, 6, 7]]).all() and (y[[2, 8, 9]] == 7.0).all()


def _decode(d, c, pool, cpool, x, w, o, y):
    gdn.shortconv_step(x, w, cpool, c["slots"], c["seq_start"], act=1, y=y)
    gdn.recurrent_step(c["q"], c["k"], c["v"], c["alpha"], c["beta"], pool, c["slots"],
                       c["seq_start"], o=o)


def test_steps_replay_from_a_graph_and_on_a_side_stream():
    lens = [1, 2, 1, 3]
    d = step_inputs(lens, 2, 2, 128, "bf16", 6, seed=61)
    c = _cuda(d)
    g = torch.Generator().manual_seed(5)
    x = torch.randn(7, 256, generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn(256, 4, generator=g) / 4).cuda()
    cstate = torch.randn(6, 3, 256, generator=g).to(torch.bfloat16).cuda()
    want, pool, cpool = [], c["state"].clone(), cstate.clone()
    for _ in range(4):
        o, y = torch.empty_like(c["v"]), torch.empty_like(x)
        _decode(d, c, pool, cpool, x, w, o, y)
        want.append((o, y, pool.clone(), cpool.clone()))
    torch.cuda.synchronize()

    o, y = torch.empty_like(c["v"]), torch.empty_like(x)
    pool, cpool = c["state"].clone(), cstate.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _decode(d, c, pool, cpool, x, w, o, y)
    torch.cuda.synchronize()
    assert torch.equal(pool, c["state"])  # capturing ran nothing
    for rep in range(4):
        o.fill_(float("nan"))
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((o, y, pool, cpool), want[rep]):
            assert torch.equal(got, ref), rep

    # another batch by writing its arrays: other slots, other lengths, padding
    c2 = {n: t.clone() for n, t in c.items()}
    c2["slots"] = torch.tensor([5, -1, 0, 2], dtype=torch.int32).cuda()
    c2["seq_start"] = torch.tensor([0, 3, 3, 5, 6], dtype=torch.int32).cuda()
    mark = lambda t: t.fill_(3.0)
    o2, y2, pool2, cpool2 = mark(torch.empty_like(o)), mark(torch.empty_like(y)), pool.clone(), \
        cpool.clone()
    _decode(d, c2, pool2, cpool2, x, w, o2, y2)
    c["slots"].copy_(c2["slots"])
    old = c["seq_start"].clone()
    c["seq_start"].copy_(c2["seq_start"])
    mark(o), mark(y)
    graph.replay()
    torch.cuda.synchronize()
    for got, ref in zip((o, y, pool, cpool), (o2, y2, pool2, cpool2)):
        assert torch.equal(got, ref)
    assert (o[6] == 3.0).all() and (y[6] == 3.0).all()  # a row of no sequence
    c["slots"].copy_(d["slots"])
    c["seq_start"].copy_(old)

    side = torch.cuda.Stream()
    pool = c["state"].clone()
    side.wait_stream(torch.cuda.current_stream())
    o2 = gdn.recurrent_step(c["q"], c["k"], c["v"], c["alpha"], c["beta"], pool, c["slots"],
                            c["seq_start"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o2, want[0][0]) and torch.equal(pool, want[0][2])


def test_binding_refusals():
    d = _cuda(step_inputs([1, 1], 2, 2, 64, "bf16", 3, seed=71))
    good = [d["q"], d["k"], d["v"], d["alpha"], d["beta"], d["state"], d["slots"]]

    def bad(exc, i, t):
        a = list(good)
        a[i] = t
        with pytest.raises(exc):
            gdn.recurrent_step(*a)

    bad(TypeError, 0, d["q"].half())
    bad(TypeError, 1, d["k"].float())
    bad(ValueError, 2, d["v"][:1])
    bad(ValueError, 3, d["alpha"].t())
    bad(TypeError, 3, d["alpha"].to(torch.bfloat16))
    bad(ValueError, 5, d["state"][:, :1])
    bad(ValueError, 5, d["state"].transpose(2, 3))
    bad(TypeError, 6, d["slots"].long())
    bad(ValueError, 6, d["slots"].cpu())
    bad(ValueError, 0, d["q"].transpose(1, 2).contiguous().transpose(1, 2))  # columns apart
    bad(ValueError, 0, d["q"][:1].expand(2, 2, 64))                           # rows on one another
    bad(gdn.GDNError, 6, d["slots"][:0])                                      # rows of no sequence
    with pytest.raises(ValueError):
        gdn.recurrent_step(*good, torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(gdn.GDNError):
        gdn.recurrent_step(*good, o=d["q"])  # o on q
    with pytest.raises(ValueError):
        gdn.shortconv_step(d["q"].view(2, 128), torch.zeros(128, 4, device="cuda"),
                           torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda"))


def test_autograd_notices_a_written_pool_and_outputs():
    """What a call writes counts as written in place: autograd refuses to use a
    value that it kept of it, and a read-only call does not touch the count."""
    d = _cuda(step_inputs([1, 1], 2, 2, 64, "bf16", 3, seed=73))
    args = [d[n] for n in ("q", "k", "v", "alpha", "beta", "state", "slots")]
    scale = torch.ones_like(d["state"]).requires_grad_()
    kept = (scale * d["state"]).sum()
    gdn.recurrent_step(*args, update=False)
    kept.backward(retain_graph=True)  # the pool as it was
    gdn.recurrent_step(*args)
    with pytest.raises(RuntimeError, match="inplace"):
        kept.backward()

    x, w = torch.randn(3, 64, device="cuda"), torch.randn(64, 4, device="cuda")
    pool, y = torch.zeros(3, 3, 64, device="cuda"), torch.zeros(3, 64, device="cuda")
    g = x.view(3, 1, 64)
    outs = [torch.empty_like(x) for _ in range(5)] + [torch.empty(64, device="cuda")
                                                      for _ in range(2)]
    dx, n = torch.empty_like(g), torch.empty_like(g)
    before = [t._version for t in [pool, y, dx, n] + outs]
    gdn.shortconv_step(x, w, pool, y=y, update=False)
    assert pool._version == before[0]
    gdn.shortconv_step(x, w, pool)
    gdn.gated_norm_fwd(g, y=n)
    gdn.gated_norm_bwd(g, None, None, g, grads=(dx, None, None))
    gdn.residual_norm_fwd(x, x, h=outs[0], y=outs[1])
    gdn.residual_norm_bwd(x, x, w[:, 0].contiguous(), w[:, 1].contiguous(), x,
                          grads=(outs[2], outs[3], outs[5], outs[6]))
    now = [t._version for t in [pool, y, dx, n] + outs]
    assert all((b > a) == (i != 8) for i, (a, b) in enumerate(zip(before, now)))  # 8: outs[4]

    # a pool made in inference mode has no count, in and out of the mode
    with torch.inference_mode():
        pool = d["state"].clone()
        a = gdn.recurrent_step(*args[:5], pool, d["slots"])
    want = d["state"].clone()
    assert torch.equal(a, gdn.recurrent_step(*args[:5], want, d["slots"]))
    gdn.recurrent_step(*args[:5], pool, d["slots"])
    gdn.recurrent_step(*args[:5], want, d["slots"])
    torch.cuda.synchronize()
    assert torch.equal(pool, want)


def test_step_makes_no_graph():
    d = _cuda(step_inputs([1, 1], 2, 2, 64, "bf16", 3, seed=74))
    d["v"].requires_grad_()
    o = gdn.recurrent_step(*(d[n] for n in ("q", "k", "v", "alpha", "beta", "state", "slots")))
    w = torch.ones(256, 4, device="cuda").requires_grad_()
    y = gdn.shortconv_step(torch.ones(3, 256, device="cuda"), w,
                           torch.zeros(3, 3, 256, device="cuda"))
    assert not o.requires_grad and not y.requires_grad
