"""Calls on a stream that has not waited for the current one, while memory that
the current stream has just given up is still being read there: the calls'
outputs and workspaces must come from elsewhere."""
import pytest
import torch

import linear_recurrence_chunked_gated_amd as gdn

pytestmark = pytest.mark.gpu


def rnd(*s, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + sum(s))
    return torch.randn(*s, generator=g, device="cuda").to(dtype)


def _recurrent_step(stream):
    n, H, D = 300, 16, 64
    q, k = (torch.nn.functional.normalize(rnd(n, H, D, seed=i), dim=-1) for i in (1, 2))
    v, al, be = rnd(n, H, D, seed=3), rnd(n, H, seed=4).sigmoid(), rnd(n, H, seed=5).sigmoid()
    state = rnd(n, H, D, D, seed=6)
    return lambda: (gdn.recurrent_step(q, k, v, al, be, state, update=False, stream=stream),)


def _shortconv_step(stream):
    x, w, state = rnd(300, 1024, seed=1), rnd(1024, 4, seed=2), rnd(300, 3, 1024, seed=3)
    return lambda: (gdn.shortconv_step(x, w, state, update=False, stream=stream),)


def _gated_norm_fwd(stream):
    x, g, w = rnd(1200, 4, 64, seed=1), rnd(1200, 4, 64, seed=2), rnd(64, seed=3)
    return lambda: (gdn.gated_norm_fwd(x, g, w, stream=stream),)


def _gated_norm_bwd(stream):
    x, g, dy = (rnd(2400, 4, 64, seed=i) for i in (1, 2, 3))
    w = rnd(64, seed=4)
    return lambda: gdn.gated_norm_bwd(x, g, w, dy, stream=stream)


def _residual_norm_fwd(stream):
    x, r, w = rnd(600, 512, seed=1), rnd(600, 512, seed=2), rnd(512, seed=3)
    return lambda: gdn.residual_norm_fwd(x, r, w, w, stream=stream)


def _residual_norm_bwd(stream):
    h, r, dy, dh = (rnd(600, 512, seed=i) for i in (1, 2, 3, 4))
    w = rnd(512, seed=5)
    return lambda: gdn.residual_norm_bwd(h, r, w, w, dy, dh, stream=stream)


def _chunk(T=200, H=4, D=64):
    q, k = (torch.nn.functional.normalize(rnd(1, T, H, D, seed=i), dim=-1) for i in (1, 2))
    return (q, k, rnd(1, T, H, D, seed=3), rnd(1, T, H, seed=4).sigmoid(),
            rnd(1, T, H, seed=5).sigmoid())


def _chunk_fwd(stream):
    x = _chunk()
    return lambda: gdn.chunk_fwd(*x, stream=stream, saved=True)[:2]


def _chunk_bwd(stream):
    x, dO, dS = _chunk(), rnd(1, 200, 4, 64, seed=6), rnd(1, 4, 64, 64, seed=7)
    return lambda: gdn.chunk_bwd(*x, None, dO, dS, stream=stream)


def _shortconv_fwd(stream):
    x, w = rnd(2, 300, 512, seed=1), rnd(512, 4, seed=2)
    return lambda: gdn.shortconv_fwd(x, w, stream=stream)


def _shortconv_bwd(stream):
    x, w, dy = rnd(2, 300, 512, seed=1), rnd(512, 4, seed=2), rnd(2, 300, 512, seed=3)
    return lambda: gdn.shortconv_bwd(x, w, None, dy, stream=stream)


def _chain(stream, overlap):
    x, dO, dS = _chunk(), rnd(1, 200, 4, 64, seed=6), rnd(1, 4, 64, 64, seed=7)
    lens = [64, 100, 36]

    def call():
        o, states, saved = gdn.chain_fwd(*x, None, lens, stream=stream, save=True, overlap=overlap)
        grads = gdn.chain_bwd(*x, dO, dS, lens, states, stream=stream, saved=saved,
                              overlap=overlap)
        return (o, *states, *grads)
    return call


def _chain_plain(stream):
    return _chain(stream, False)


def _chain_overlapped(stream):
    return _chain(stream, True)


CALLS = [_recurrent_step, _shortconv_step, _gated_norm_fwd, _gated_norm_bwd, _residual_norm_fwd,
         _residual_norm_bwd, _chunk_fwd, _chunk_bwd, _shortconv_fwd, _shortconv_bwd, _chain_plain,
         _chain_overlapped]


@pytest.mark.parametrize("make", CALLS, ids=lambda f: f.__name__.strip("_"))
def test_memory_of_the_current_streams_pending_work(make):
    """Blocks of every size the call allocates are freed with a copy out of
    them still waiting behind some milliseconds of products; the call on the
    other stream must leave them alone."""
    want = [t for t in make(None)() if t is not None]
    side = torch.cuda.Stream()
    call = make(side)
    a = rnd(4096, 4096)
    sizes = [t.numel() * t.element_size() for t in want] + [1 << 20]  # the last: a workspace
    old = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    copies = [torch.empty_like(t) for t in old]
    where = {t.data_ptr() for t in old}
    torch.cuda.synchronize()
    for _ in range(10):
        a = a @ a * 1e-3
    for t, c in zip(old, copies):
        c.copy_(t)
    del old, t
    got = [t for t in call() if t is not None]
    assert not where & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all((c == 7).all() for c in copies)
    assert len(got) == len(want) and all(torch.equal(x, y) for x, y in zip(got, want))


def test_side_stream_inside_a_captured_graph():
    """A captured step that forks to a side stream and joins it again: outputs
    made there belong to the graph's memory, replay after replay."""
    x, g, dy = (rnd(200, 4, 64, seed=i) for i in (1, 2, 3))
    w = rnd(64, seed=5)

    def work(side):
        y = gdn.gated_norm_fwd(x, g, w)
        if side is not None:
            side.wait_stream(torch.cuda.current_stream())
        grads = gdn.gated_norm_bwd(x, y, w, dy, stream=side)
        z = gdn.gated_norm_fwd(grads[0], g, w, stream=side)
        if side is not None:
            torch.cuda.current_stream().wait_stream(side)
        return (y, z) + tuple(grads)

    want = work(None)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        out = work(side)
    for rep in range(4):
        for t in out:
            t.fill_(float("nan"))
        spill = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), rep
        del spill
