"""Linear attention with a decay where its documented range ends: decays far
past 1, and plans that the other tests do not reach."""
import pytest
import torch

import linear_recurrence_chunked_gated_amd as gdn
from decay_testutil import chunk_bwd_ref, chunk_inputs, chunk_ref
from layer_testutil import check

pytestmark = pytest.mark.gpu

NAMES = ("o", "S_out", "dq", "dk", "dv", "dS_in")


def _cuda(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def _both(c, **kw):
    return (gdn.decay_chunk_fwd(c["q"], c["k"], c["v"], c["decay"], c["S_in"], c["seq_start"], **kw)
            + gdn.decay_chunk_bwd(c["q"], c["k"], c["v"], c["decay"], c["S_in"], c["dO"], c["dS_out"],
                                  c["seq_start"], **kw))


def _check_both(d, dtype, c=None):
    (ro, rS), (ob, Sb) = chunk_ref(d)
    ref, bnd = chunk_bwd_ref(d)
    types = (dtype, None, dtype, dtype, dtype, None)
    for name, x, r, b, t in zip(NAMES, _both(c or _cuda(d)), (ro, rS) + ref, (ob, Sb) + bnd, types):
        check(name, x.reshape(r.shape), r, b, t)


@pytest.mark.parametrize("decay", [50.0, -50.0])
@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 64), ("bf16", 128), ("f32", 128)])
def test_decays_far_past_one_in_short_sequences(dtype, D, decay):
    """Powers of the decay up to a sequence's length are within range (50^17 <
    2^97), those of a whole block are not, and nothing of them shows."""
    _check_both(chunk_inputs([17, 3, 0, 1], 1, 2, D, dtype, seed=401, decay=decay, grads=True), dtype)


# sequences of one length: (B, T, Hk, Hv, D), and how their boundaries are joined
UNIFORM = [
    ((4, 1600, 8, 16, 128), "items"),   # up to three boundaries: by the items
    ((4, 1600, 8, 16, 64), "items"),
    ((1, 700, 1, 2, 128), "chain"),     # a block a segment, ragged
    ((1, 17000, 8, 16, 128), "chain"),  # bf16: a last segment shorter than the others
    ((1, 17000, 8, 16, 64), "chain"),
    ((12, 450, 8, 16, 128), "whole"),   # not cut: the heads fill the GPU
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size,joined", UNIFORM)
def test_plans_of_sequences_of_one_length(size, joined, dtype):
    """Every plan of a batch without offsets, forward and backward, at both head
    sizes: the first and last sequence's first and last key head against 64
    bits, and the kernels that ran."""
    B, T, Hk, Hv, D = size
    d = chunk_inputs([T] * B, Hk, Hv, D, dtype, seed=411 + T + D, grads=True)
    c = _cuda(d)
    for n in ("q", "k", "v", "dO"):
        c[n] = c[n].unflatten(0, (B, T))
    c["seq_start"] = None
    with gdn.profile() as p:
        o, S, dq, dk, dv, dS = _both(c)
        torch.cuda.synchronize()
    for call in ("", "_bwd"):
        assert ("decay_sum" + call in p.results) == (joined != "whole")
    assert p.results.get("decay_chain", (0,))[0] == (2 if joined == "chain" else 0)
    G = Hv // Hk
    for i, g in ((0, 0), (B - 1, Hk - 1)):
        t, h = slice(i * T, (i + 1) * T), slice(g * G, (g + 1) * G)
        part = dict(q=d["q"][t, g:g + 1], k=d["k"][t, g:g + 1], v=d["v"][t, h], dO=d["dO"][t, h],
                    decay=d["decay"][h], S_in=d["S_in"][i:i + 1, h], dS_out=d["dS_out"][i:i + 1, h],
                    seq_start=torch.tensor([0, T]))
        (ro, rS), (ob, Sb) = chunk_ref(part)
        ref, bnd = chunk_bwd_ref(part)
        got = (o[i, :, h], S[i:i + 1, h], dq[i, :, g:g + 1], dk[i, :, g:g + 1], dv[i, :, h], dS[i:i + 1, h])
        types = (dtype, None, dtype, dtype, dtype, None)
        for name, x, r, b, ty in zip(NAMES, got, (ro, rS) + ref, (ob, Sb) + bnd, types):
            check(name, x, r, b, ty)
