"""Linear attention with a decay for each head (decay_chunk_fwd, _bwd) against
its 64-bit form: token types, head layouts, packed and empty sequences, lengths
from one token over several segments, strided rows, decays at their ends,
offsets that are out of order, graphs, streams, autograd."""
import pytest
import torch

import linear_recurrence_chunked_gated_amd as gdn
from decay_testutil import chunk_bwd_ref, chunk_inputs, chunk_ref
from layer_testutil import DT, check

pytestmark = pytest.mark.gpu


def _cuda(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def _fwd(c, **kw):
    r = gdn.decay_chunk_fwd(c["q"], c["k"], c["v"], c["decay"], c["S_in"], c["seq_start"], **kw)
    torch.cuda.synchronize()
    return r


def _bwd(c, **kw):
    r = gdn.decay_chunk_bwd(c["q"], c["k"], c["v"], c["decay"], c["S_in"], c["dO"], c["dS_out"],
                            c["seq_start"], **kw)
    torch.cuda.synchronize()
    return r


LENS = [
    ([1], 1, 1, 64, "f32"),
    ([1], 2, 2, 128, "bf16"),
    ([64], 2, 2, 64, "bf16"),
    ([65], 1, 2, 128, "f32"),
    ([63, 1, 2, 64, 130], 2, 4, 128, "bf16"),
    ([0, 5, 0, 0, 70, 0], 1, 3, 64, "f32"),       # empty ones pass their state through
    ([300], 2, 2, 64, "f32"),                     # two segments
    ([700, 257, 256, 1, 513], 1, 2, 128, "bf16"),  # several, whole and ragged
    ([520, 3, 1030], 3, 6, 64, "bf16"),
    ([7] * 41, 1, 1, 64, "bf16"),
]


@pytest.mark.parametrize("lens,Hk,Hv,D,dtype", LENS)
def test_forward_matches(lens, Hk, Hv, D, dtype):
    d = chunk_inputs(lens, Hk, Hv, D, dtype, seed=sum(lens) + D + Hv)
    (ro, rS), (ob, Sb) = chunk_ref(d, 0.7)
    o, S = _fwd(_cuda(d), scale=0.7)
    check("o", o, ro, ob, dtype)
    check("S_out", S, rS, Sb, None)


@pytest.mark.parametrize("lens,Hk,Hv,D,dtype", LENS)
def test_backward_matches(lens, Hk, Hv, D, dtype):
    d = chunk_inputs(lens, Hk, Hv, D, dtype, seed=sum(lens) + D + Hv + 1, grads=True)
    ref, bnd = chunk_bwd_ref(d, 0.7)
    got = _bwd(_cuda(d), scale=0.7)
    for name, x, r, b in zip(("dq", "dk", "dv"), got, ref, bnd):
        check(name, x, r, b, dtype)
    check("dS_in", got[3], ref[3], bnd[3], None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_entry_state_and_exit_gradient(dtype):
    d = chunk_inputs([270, 33], 2, 2, 64, dtype, seed=5, state=False, grads=True)
    (ro, rS), (ob, Sb) = chunk_ref(d)
    o, S = _fwd(_cuda(d))
    check("o", o, ro, ob, dtype)
    check("S_out", S, rS, Sb, None)
    d["dS_out"].zero_()
    ref, bnd = chunk_bwd_ref(d)
    c = _cuda(d)
    c["dS_out"] = None
    got = _bwd(c)
    for name, x, r, b in zip(("dq", "dk", "dv"), got, ref, bnd):
        check(name, x, r, b, dtype)
    check("dS_in", got[3], ref[3], bnd[3], None)
    assert _bwd(c, want_dS_in=False)[3] is None


@pytest.mark.parametrize("B,T,dtype", [(3, 150, "bf16"), (2, 600, "f32"), (1, 64, "bf16"), (2, 0, "f32"),
                                       (0, 7, "f32")])
def test_one_length(B, T, dtype):
    """[B, T, H, D] without offsets (cut into other segments than packed rows);
    [T, H, D] without offsets is one sequence, to the bit."""
    d = chunk_inputs([T] * B, 2, 4, 64, dtype, seed=B + T, grads=True)
    c = _cuda(d)
    (ro, rS), (ob, Sb) = chunk_ref(d)
    ref, bnd = chunk_bwd_ref(d)
    e = dict(c, seq_start=None)
    for n in ("q", "k", "v", "dO"):
        e[n] = c[n].reshape(B, T, *c[n].shape[1:])
    o, S = _fwd(e)
    assert o.shape == (B, T, 4, 64)
    check("o", o.reshape(ro.shape), ro, ob, dtype) if o.numel() else None
    check("S_out", S, rS, Sb, None) if B else None
    got = _bwd(e)
    for name, x, r, b in zip(("dq", "dk", "dv", "dS"), got, ref, bnd):
        assert x.shape == {"dq": e["q"], "dk": e["k"], "dv": e["v"], "dS": S}[name].shape
        if x.numel():
            check(name, x.reshape(r.shape), r, b, None if name == "dS" else dtype)
    if B == 1:
        flat = dict(c, seq_start=None)
        for x, y in zip(_fwd(flat) + _bwd(flat), (o, S) + got):
            assert torch.equal(x, y.reshape(x.shape))


def test_many_sequences_of_one_length_are_not_cut():
    """600 heads of their own fill the GPU: one segment each, no boundaries."""
    d = chunk_inputs([333] * 2, 2, 2, 64, "bf16", seed=9, grads=True)
    c = _cuda(d)
    rep = lambda t: t.reshape(2, 333, 2, 64).repeat(150, 1, 1, 1)
    q, k, v, dO = (rep(c[n]) for n in ("q", "k", "v", "dO"))
    S_in, dS = c["S_in"].repeat(150, 1, 1, 1), c["dS_out"].repeat(150, 1, 1, 1)
    (ro, rS), (ob, Sb) = chunk_ref(d)
    o, S = gdn.decay_chunk_fwd(q, k, v, c["decay"], S_in)
    check("o", o[:2].reshape(ro.shape), ro, ob, "bf16")
    check("S", S[:2], rS, Sb, None)
    assert torch.equal(o[2:], o[:-2]) and torch.equal(S[2:], S[:-2])
    ref, bnd = chunk_bwd_ref(d)
    got = gdn.decay_chunk_bwd(q, k, v, c["decay"], S_in, dO, dS)
    for x, r, b, t in zip(got, ref, bnd, ("bf16", "bf16", "bf16", None)):
        check("grad", x[:2].reshape(r.shape), r, b, t)
        assert torch.equal(x[2:], x[:-2])


@pytest.mark.parametrize("decay", [0.0, 1.0, 1e-3, 0.5, 1 - 2.0 ** -20])
def test_decays_at_their_ends(decay):
    """None at all, total, and near both: a = 0 keeps each token's own term."""
    d = chunk_inputs([280, 3], 1, 2, 64, "f32", seed=31, decay=decay, grads=True)
    (ro, rS), (ob, Sb) = chunk_ref(d)
    o, S = _fwd(_cuda(d))
    check("o", o, ro, ob, "f32")
    check("S_out", S, rS, Sb, None)
    ref, bnd = chunk_bwd_ref(d)
    for name, x, r, b in zip(("dq", "dk", "dv", "dS"), _bwd(_cuda(d)), ref, bnd):
        check(name, x, r, b, "f32")


def test_strided_rows():
    """q, k and v as slices of one projection's rows: the bits of copies."""
    d = chunk_inputs([100, 290], 2, 4, 64, "bf16", seed=41, grads=True)
    c = _cuda(d)
    want = _fwd(c) + _bwd(c)
    wide = torch.cat([c["q"], c["k"], c["v"]], 1)
    s = dict(c, q=wide[:, :2], k=wide[:, 2:4], v=wide[:, 4:])
    assert not s["q"].is_contiguous()
    for x, y in zip(_fwd(s) + _bwd(s), want):
        assert torch.equal(x, y)


def test_rows_of_no_sequence_are_left():
    """Rows before the first and behind the last sequence: not read (NaN in
    them), and their outputs left, also where shared heads are summed."""
    lens, before, after = [70, 0, 300], 5, 9
    d = chunk_inputs(lens, 1, 2, 64, "bf16", seed=51, before=before, after=after, grads=True)
    rest = torch.ones(d["q"].shape[0], dtype=torch.bool)
    rest[before:-after] = False
    for n in ("q", "k", "v", "dO"):
        d[n][rest] = float("nan")
    c = _cuda(d)
    o = torch.full_like(c["v"], 7)
    _, S = _fwd(c, o=o)
    assert (o[rest] == 7).all() and not torch.isnan(o).any() and not torch.isnan(S).any()
    g = tuple(torch.full_like(c[n], 7) for n in ("q", "k", "v", "S_in"))
    _bwd(c, grads=g)
    for x in g[:3]:
        assert (x[rest] == 7).all() and not torch.isnan(x).any()
    m = {n: c[n][~rest].contiguous() for n in ("q", "k", "v", "dO")}
    m = dict(c, **m, seq_start=c["seq_start"] - before)
    o2, S2 = _fwd(m)
    assert torch.equal(o2, o[~rest]) and torch.equal(S2, S)
    for x, y in zip(_bwd(m), (g[0][~rest], g[1][~rest], g[2][~rest], g[3])):
        assert torch.equal(x, y)


@pytest.mark.parametrize("given,taken", [
    ([0, 90, 40, 200], [0, 90, 90, 200]),          # a step back: the sequence is empty
    ([-5, 90, 150, 9999], [0, 90, 150, 200]),      # clamped to the rows
    ([300, 400, 10, 20], [200, 200, 200, 200]),    # nothing left
    ([0, 200, 0, 200], [0, 200, 200, 200]),        # the same rows twice: once
])
def test_offsets_out_of_order(given, taken):
    """Offsets are clamped and taken as their running maximum."""
    d = chunk_inputs([200, 0, 0], 1, 2, 64, "f32", seed=61, grads=True)
    c = _cuda(d)
    a = dict(c, seq_start=torch.tensor(given, dtype=torch.int32).cuda())
    b = dict(c, seq_start=torch.tensor(taken, dtype=torch.int32).cuda())
    outs = []
    for s in (a, b):
        o = torch.zeros_like(c["v"])
        g = tuple(torch.zeros_like(c[n]) for n in ("q", "k", "v", "S_in"))
        outs.append((o, _fwd(s, o=o)[1]) + tuple(_bwd(s, grads=g)))
    for x, y in zip(*outs):
        assert torch.equal(x, y)


def test_more_sequences_than_the_plan_takes_at_once():
    """2500 short sequences (the table is made 1024 at a time), two of them
    cut: each has the bits of itself alone."""
    g = torch.Generator().manual_seed(71)
    lens = torch.randint(0, 4, (2500,), generator=g).tolist()
    lens[1023], lens[2047] = 700, 300
    d = chunk_inputs(lens, 1, 1, 64, "f32", seed=72)
    c = _cuda(d)
    o, S = _fwd(c)
    st = d["seq_start"].tolist()
    for i in (0, 1, 1022, 1023, 1024, 1025, 2046, 2047, 2048, 2499):
        sl = slice(st[i], st[i + 1])
        one = dict(q=c["q"][sl], k=c["k"][sl], v=c["v"][sl], decay=c["decay"],
                   S_in=c["S_in"][i:i + 1],
                   seq_start=torch.tensor([0, lens[i]], dtype=torch.int32).cuda())
        o1, S1 = _fwd(one)
        assert torch.equal(o1, o[sl]) and torch.equal(S1[0], S[i]), i


@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("f32", 64), ("bf16", 128)])
def test_planned_by_waves_and_by_a_table(dtype, D):
    """Up to 64 sequences are planned by each wave, more by a table.  Empty
    sequences behind the others change nothing but that."""
    lens = [0, 700, 1, 0, 64, 65, 600, 128, 3, 0] + [17] * 40 + [0, 400, 129, 0]
    n = len(lens)
    d = chunk_inputs(lens, 1, 2, D, dtype, seed=77, grads=True)
    c = _cuda(d)
    (ro, rS), (ob, Sb) = chunk_ref(d)
    ref, bnd = chunk_bwd_ref(d)
    outs = []
    for more in (0, 64 - n, 65 - n, 1100 - n):
        st = torch.cat([c["seq_start"], c["seq_start"][-1:].expand(more)])
        ext = lambda x: torch.cat([x, x.new_zeros(more, *x.shape[1:])])
        m = dict(c, seq_start=st, S_in=ext(c["S_in"]), dS_out=ext(c["dS_out"]))
        o, S = _fwd(m)
        g = _bwd(m)
        outs.append((o, S[:n]) + tuple(g[:3]) + (g[3][:n],))
        assert not S[n:].any() and not g[3][n:].any()
    for x, r, b, t in zip(outs[0], (ro, rS) + tuple(ref), (ob, Sb) + tuple(bnd),
                          (dtype, None, dtype, dtype, dtype, None)):
        check("packed", x, r, b, t)
    for other in outs[1:]:
        for x, y in zip(outs[0], other):
            assert torch.equal(x, y)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
def test_long_sequences_and_large_batches(dtype, D):
    """Segments of more than the least four blocks: 20,011 tokens of 16 heads,
    packed with short ones, against a 64-bit scan on the GPU."""
    lens, Hh = [20011, 1, 640, 5], 16
    d = chunk_inputs(lens, 8, Hh, D, dtype, seed=81, grads=True)
    c = _cuda(d)
    o, S = _fwd(c)
    got = _bwd(c)
    f = {n: t.double() for n, t in c.items() if t is not None and t.is_floating_point()}
    st = d["seq_start"].tolist()
    tol = 5e-3 if dtype == "bf16" else 1e-5  # of the norm: half a step of the type and the operands'

    def near(name, x, r, t=tol):
        e = float((x.double() - r).norm() / r.norm())
        assert e <= t, (name, e)

    for i, h in ((0, 0), (0, 15), (1, 3), (2, 7), (3, 12)):
        sl, k2 = slice(st[i], st[i + 1]), h // 2
        T = lens[i]
        pw = f["decay"][h] ** torch.arange(T + 1, device="cuda").double()
        r = torch.arange(T, device="cuda")

        def scan(x, u, w):  # every pair, 2048 rows at a time
            y = torch.zeros_like(w)
            for t in range(0, T, 2048):
                gap = r[t:t + 2048, None] - r
                M = torch.where(gap >= 0, pw[gap.clamp(min=0)], 0.0)
                y[t:t + 2048] = (M * (x[t:t + 2048] @ u.t())) @ w
            return y

        q, k, v, do = f["q"][sl, k2], f["k"][sl, k2], f["v"][sl, h], f["dO"][sl, h]
        E, G = f["S_in"][i, h], f["dS_out"][i, h]
        near("o", o[sl, h], scan(q, k, v) + pw[1:, None] * (q @ E.t()))
        near("S", S[i, h], (pw[:T].flip(0)[:, None] * v).t() @ k + pw[T] * E, 1e-5)
        last = pw[:T].flip(0)[:, None]
        rev = lambda *a: scan(*(t.flip(0) for t in a)).flip(0)
        near("dv", got[2][sl, h], rev(k, q, do) + last * (k @ G.t()))
        near("dS", got[3][i, h], (pw[1:, None] * do).t() @ q + pw[T] * G, 1e-5)
        dq, dk = 0.0, 0.0
        for g in (2 * k2, 2 * k2 + 1):
            pw = f["decay"][g] ** torch.arange(T + 1, device="cuda").double()
            w, y, S1, G1 = f["v"][sl, g], f["dO"][sl, g], f["S_in"][i, g], f["dS_out"][i, g]
            dq = dq + scan(y, w, k) + pw[1:, None] * (y @ S1)
            dk = dk + rev(w, y, q) + pw[:T].flip(0)[:, None] * (w @ G1)
        near("dq", got[0][sl, k2], dq)
        near("dk", got[1][sl, k2], dk)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chunks_chain(dtype):
    """Two chunks through S_out -> S_in, and their gradients through dS_in ->
    dS_out, against one: within both results' bounds."""
    d = chunk_inputs([400], 2, 2, 64, dtype, seed=91, grads=True)
    (ro, rS), (ob, Sb) = chunk_ref(d)
    ref, bnd = chunk_bwd_ref(d)
    c = _cuda(d)
    cut = 150
    part = lambda sl: {n: c[n][sl] for n in ("q", "k", "v", "dO")}
    one = dict(c, **part(slice(0, cut)), seq_start=None)
    two = dict(c, **part(slice(cut, None)), seq_start=None)
    o1, S1 = _fwd(one)
    two["S_in"] = S1
    o2, S2 = _fwd(two)
    # the cut moves the blocks, and S1's error (Sb at most) meets |q|
    q = d["q"].double().repeat_interleave(1, 1).abs()
    more = torch.einsum("nhk,hvk->nhv", q, Sb[0])
    check("o", torch.cat([o1, o2]), ro, 2 * ob + more, dtype)
    check("S", S2, rS, 2 * Sb, None)
    g2 = _bwd(two)
    one["dS_out"] = g2[3]
    g1 = _bwd(one)
    for name, a, b, r, bb, x in zip(("dq", "dk", "dv"), g1, g2, ref, bnd, ("dO", "v", "k")):
        side = d[x].double().abs()
        e = Sb[0] if name == "dq" else bnd[3][0]
        more = torch.einsum("nhv,hvk->nhk" if name != "dv" else "nhk,hvk->nhv", side, e)
        check(name, torch.cat([a, b]), r, 2 * bb + more, dtype)


def test_values_that_are_not_finite_stay_in_their_sequence():
    """NaN and infinities in one sequence of a packed batch, and the rest of
    the batch has the bits that it has without them; earlier blocks of that
    sequence's outputs too."""
    d = chunk_inputs([300, 200, 100], 1, 2, 64, "bf16", seed=95, grads=True)
    c = _cuda(d)
    clean = _fwd(c) + _bwd(c)
    for n, x in (("q", float("inf")), ("k", float("nan")), ("v", float("-inf")), ("dO", float("nan"))):
        c[n][300 + 150] = x
    dirty = _fwd(c) + _bwd(c)
    rows = torch.ones(600, dtype=torch.bool)
    rows[300:500] = False
    for i, (x, y) in enumerate(zip(clean, dirty)):
        if i in (1, 5):
            assert torch.equal(x[[0, 2]], y[[0, 2]])
        else:
            assert torch.equal(x[rows], y[rows])
    assert torch.equal(clean[0][300:428], dirty[0][300:428])       # o before the block
    assert torch.equal(clean[3][492:500], dirty[3][492:500])       # dk behind it
    assert torch.isnan(dirty[0][300 + 150].float()).any()


def test_captured_and_replayed_for_other_batches():
    """A captured forward and backward, the offsets and tensors rewritten
    between replays: every replay has the bits of an eager call, with eager
    calls between."""
    d = chunk_inputs([200, 313, 7], 1, 2, 64, "bf16", seed=101, grads=True)
    c = _cuda(d)
    call = lambda: _fwd_nosync(c) + _bwd_nosync(c)

    def _fwd_nosync(c):
        return gdn.decay_chunk_fwd(c["q"], c["k"], c["v"], c["decay"], c["S_in"], c["seq_start"])

    def _bwd_nosync(c):
        return gdn.decay_chunk_bwd(c["q"], c["k"], c["v"], c["decay"], c["S_in"], c["dO"],
                                   c["dS_out"], c["seq_start"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for rep, lens in enumerate(([200, 313, 7], [0, 1, 519], [520, 0, 0], [64, 300, 156])):
        e = _cuda(chunk_inputs(lens, 1, 2, 64, "bf16", seed=110 + rep, grads=True))
        for n in c:
            c[n].copy_(e[n])
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for x, y in zip(got, call()):
            assert torch.equal(x, y), (rep, lens)


def test_two_graphs_with_a_workspace_each():
    """Two captured calls replayed on two streams at once: each has its own
    workspace out of its graph's memory."""
    cs = [_cuda(chunk_inputs([900, 100], 2, 2, 64, "bf16", seed=121 + i)) for i in range(2)]
    want = [_fwd(c) for c in cs]
    graphs, outs, streams = [], [], []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(gdn.decay_chunk_fwd(c["q"], c["k"], c["v"], c["decay"], c["S_in"],
                                            c["seq_start"]))
        graphs.append(g)
        streams.append(torch.cuda.Stream())
    for rep in range(3):
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            assert all(torch.equal(x, y) for x, y in zip(w, o)), rep


def test_given_stream_outputs_and_workspace():
    """On another stream, with the caller's outputs and workspace."""
    d = chunk_inputs([600, 20], 1, 2, 64, "bf16", seed=131, grads=True)
    c = _cuda(d)
    want = _fwd(c) + _bwd(c)
    side = torch.cuda.Stream()
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    o, S = torch.zeros_like(c["v"]), torch.zeros_like(c["S_in"])
    side.wait_stream(torch.cuda.current_stream())
    got = _fwd(c, stream=side, o=o, S_out=S, workspace=ws) + _bwd(c, stream=side, workspace=ws)
    assert got[0].data_ptr() == o.data_ptr() and got[1].data_ptr() == S.data_ptr()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_memory_of_the_current_streams_pending_work():
    """Blocks freed with work of the current stream pending on them are not
    what a call on another stream writes to."""
    c = _cuda(chunk_inputs([600, 20], 1, 2, 64, "bf16", seed=141, grads=True))
    want = _fwd(c) + _bwd(c)
    side = torch.cuda.Stream()
    a = torch.randn(4096, 4096, device="cuda")
    sizes = [t.numel() * t.element_size() for t in want] + [1 << 20, 4 << 20]
    old = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    copies = [torch.empty_like(t) for t in old]
    torch.cuda.synchronize()
    for _ in range(10):
        a = a @ a * 1e-3
    for t, p in zip(old, copies):
        p.copy_(t)
    del old, t
    got = (gdn.decay_chunk_fwd(c["q"], c["k"], c["v"], c["decay"], c["S_in"], c["seq_start"],
                               stream=side)
           + gdn.decay_chunk_bwd(c["q"], c["k"], c["v"], c["decay"], c["S_in"], c["dO"], c["dS_out"],
                                 c["seq_start"], stream=side))
    torch.cuda.synchronize()
    assert all((p == 7).all() for p in copies)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def _plain(q, k, v, a, S, scale):
    """Token by token over [B, T, H, D] in the type given."""
    rep = v.shape[2] // q.shape[2]
    q, k = q.repeat_interleave(rep, 2), k.repeat_interleave(rep, 2)
    out = []
    for t in range(q.shape[1]):
        S = a[:, None, None] * S + v[:, t, :, :, None] * k[:, t, :, None, :]
        out.append(scale * (S * q[:, t, :, None, :]).sum(-1))
    return torch.stack(out, 1), S


def test_autograd_against_64_bits():
    """Gradients through decay_chunk, two chunks chained, shared heads and
    broadcast inputs, against torch's own of the token-by-token form; o's and
    S_out's gradients together and each alone."""
    d = chunk_inputs([90, 90], 2, 4, 64, "f32", seed=151)
    shape = lambda t: t.reshape(2, 90, *t.shape[1:])
    base = [shape(d["q"]), shape(d["k"]), shape(d["v"])[:1], d["S_in"]]  # v shared by the batch
    g = torch.Generator().manual_seed(152)
    up = [torch.randn(2, 90, 4, 64, generator=g), torch.randn(2, 4, 64, 64, generator=g)]

    def run(dev, dt, chunk, use):
        x = [t.to(dev, dt).clone().requires_grad_() for t in base]
        a = d["decay"].to(dev, dt)
        v = x[2].expand(2, -1, -1, -1).contiguous()
        o1, S1 = chunk(x[0][:, :40].contiguous(), x[1][:, :40].contiguous(), v[:, :40].contiguous(), a, x[3])
        o2, S2 = chunk(x[0][:, 40:].contiguous(), x[1][:, 40:].contiguous(), v[:, 40:].contiguous(), a, S1)
        loss = 0
        if use[0]:
            loss = loss + (torch.cat([o1, o2], 1) * up[0].to(dev, dt)).sum()
        if use[1]:
            loss = loss + (S2 * up[1].to(dev, dt)).sum()
        loss.backward()
        # the loss of S_out alone does not reach q: none, or zeros
        return [torch.zeros(t.shape).double() if t.grad is None else t.grad.cpu().double() for t in x]

    for use in ((1, 1), (1, 0), (0, 1)):
        got = run("cuda", torch.float32, lambda *a: gdn.decay_chunk(*a, scale=0.5), use)
        ref = run("cpu", torch.float64, lambda *a: _plain(*a, 0.5), use)
        for name, x, r in zip("qkvS", got, ref):
            # (72 + 90) U = 1e-5 of the terms bounds a chunk's; two are chained
            assert (x - r).norm() <= 2e-5 * r.norm(), (use, name, float((x - r).norm() / r.norm()))


def test_gradients_against_differences():
    """The loss is linear in v and in S_in and quadratic in nothing else that
    moves here: central differences of it along random directions of q and of k."""
    d = chunk_inputs([140], 1, 2, 64, "f32", seed=161, grads=True)
    c = _cuda(d)
    dq, dk, dv, dS = _bwd(c)

    def loss(**moved):
        (o, S), _ = chunk_ref(dict(d, **moved))
        return float((o * d["dO"].double()).sum() + (S * d["dS_out"].double()).sum())

    g = torch.Generator().manual_seed(162)
    for name, grad in (("q", dq), ("k", dk), ("v", dv), ("S_in", dS)):
        dirn = torch.randn(d[name].shape, generator=g).double()
        e = 2.0 ** -10
        # the loss is linear in each of them alone, so a difference is exact but
        # for the last bits of a sum of about 1e4 in 64
        up, down = (loss(**{name: (d[name].double() + s * e * dirn)}) for s in (1, -1))
        num = (up - down) / (2 * e)
        got = float((grad.cpu().double() * dirn).sum())
        size = float((grad.cpu().double() * dirn).norm())
        assert abs(got - num) <= 2e-5 * size * 8, (name, got, num)


def test_autograd_of_packed_rows_and_unused_outputs():
    """Rows of no sequence: zeros in o and in the gradients.  A decay that wants
    a gradient is refused."""
    d = chunk_inputs([50, 20], 1, 2, 64, "bf16", seed=171, before=3, after=4)
    c = _cuda(d)
    x = [c[n].clone().requires_grad_() for n in ("q", "k", "v")]
    junk = [torch.full((1 << 16,), float("nan"), device="cuda") for _ in range(20)]
    del junk
    o, S = gdn.decay_chunk(*x, c["decay"], c["S_in"], c["seq_start"])
    o.float().sum().backward()
    rest = torch.tensor([0, 1, 2, 73, 74, 75, 76])
    assert (o[rest] == 0).all()
    for t in x:
        assert (t.grad[rest] == 0).all() and torch.isfinite(t.grad).all()
    with pytest.raises(ValueError, match="no gradient"):
        gdn.decay_chunk(*x, c["decay"].clone().requires_grad_(), c["S_in"])


def test_offsets_past_32_bits():
    """Token rows whose byte and element offsets pass 2^32 and 2^31: the last
    sequence of 2.2e9 elements, against itself alone."""
    N, Hh, D = 1_050_000, 16, 128
    g = torch.Generator(device="cuda").manual_seed(181)
    q = torch.empty(N, Hh, D, dtype=torch.bfloat16, device="cuda")
    for t in range(0, N, 1 << 16):
        q[t:t + (1 << 16)].normal_(generator=g)
    q *= D ** -0.5
    decay = (1 - 2.0 ** -torch.linspace(2, 9, Hh)).cuda()
    start = torch.tensor([0, N - 400, N], dtype=torch.int32, device="cuda")
    o, S = gdn.decay_chunk_fwd(q, q, q, decay, None, start)
    e = q[N - 400:].clone()
    # the long one's segments are 32,832 tokens, these 400 one segment either way
    one = torch.tensor([0, 0, 400], dtype=torch.int32, device="cuda")
    o1, S1 = gdn.decay_chunk_fwd(e, e, e, decay, None, one)
    f = e.double()
    r = torch.arange(400, device="cuda")
    for h in (0, 15):
        gap = r[:, None] - r
        M = torch.where(gap >= 0, decay[h].double() ** gap.clamp(min=0).double(), 0.0)
        want = (M * (f[:, h] @ f[:, h].t())) @ f[:, h]
        for x in (o[N - 400:, h], o1[:, h]):
            assert float((x.double() - want).norm() / want.norm()) < 5e-3
    assert float((S[1] - S1[1]).norm() / S1[1].norm()) < 1e-5
    dq, dk, dv, dS = gdn.decay_chunk_bwd(q, q, q, decay, None, q, None, start)
    h1 = gdn.decay_chunk_bwd(e, e, e, decay, None, e, None, one)
    for x, y in zip((dq, dk, dv), h1):
        assert float((x[N - 400:].double() - y.double()).norm() / y.double().norm()) < 1e-2
