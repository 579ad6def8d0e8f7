"""How close the chunk form of linear attention with a decay is to 64 bits: bf16
outputs are off by their own rounding and what two bf16 planes of an operand
leave, no more."""
import pytest
import torch

import linear_recurrence_chunked_gated_amd as gdn
from decay_testutil import H, chunk_bwd_ref, chunk_inputs, chunk_ref
from layer_testutil import U, check

pytestmark = pytest.mark.gpu


def _cuda(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


@pytest.mark.parametrize("T,Hk,Hv,D", [(130, 1, 2, 128), (333, 2, 2, 64), (700, 1, 1, 128)])
def test_bf16_outputs_are_off_by_their_own_rounding(T, Hk, Hv, D):
    """The operands rounded on the way (the masked scores, the state's copy,
    the state's terms) keep two planes: H^2 of each term, of all terms' absolute
    values at most 4 H^2 (the factors of two compound), and a U of them for each
    of T + 64 additions.  chunk_ref's bound for fp32 tensors is (T + 72) U of
    the same terms."""
    d = chunk_inputs([T], Hk, Hv, D, "bf16", seed=301 + T, grads=True)
    f = {k: t.float() if t is not None and t.is_floating_point() else t for k, t in d.items()}
    (ro, _), (ob, _) = chunk_ref(f, 0.7)
    ref, bnd = chunk_bwd_ref(f, 0.7)
    c = _cuda(d)
    o, _ = gdn.decay_chunk_fwd(c["q"], c["k"], c["v"], c["decay"], c["S_in"], c["seq_start"], scale=0.7)
    got = gdn.decay_chunk_bwd(c["q"], c["k"], c["v"], c["decay"], c["S_in"], c["dO"], c["dS_out"],
                              c["seq_start"], scale=0.7)
    for name, x, r, b in zip(("o", "dq", "dk", "dv"), (o,) + got[:3], (ro,) + ref, (ob,) + bnd):
        terms = b / ((T + 72) * U)
        check(name, x, r, (4 * H * H + (T + 64) * U) * terms, "bf16")
