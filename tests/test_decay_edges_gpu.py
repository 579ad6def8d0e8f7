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
