"""How close the chunk form of linear attention with a decay is to 64 bits: bf16
outputs are off by their own rounding and what two bf16 planes of an operand
leave, no more."""
import pytest
import torch

import linear_recurrence_chunked_gated_amd as gdn
from decay_testutil import H, chunk_bwd_ref, chunk_inputs, chunk_ref
from layer_testutil import DT, U, check

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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_states_decay_over_many_blocks(dtype):
    """192 heads of 8192 tokens (not cut: 128 or 256 blocks each) that add
    nothing to the state: S_out = a^T S_in, and dS_in = a^T dS_out.  The blocks'
    decays are taken together in 48 bits at least, so the result has a rounding
    of the decay and one of the product whenever it is taken into the state,
    which is for every 2^-20 of it and at the end: (2 folds + 2) U, however
    many blocks there are.  (Blocks' decays rounded to fp32 are off by up to
    154 U and 92 U here.)"""
    T, H, B = 8192, 24, 8
    dt = DT[dtype]
    decay = (1 - 2.0 ** -torch.linspace(7, 14, H)).cuda()
    S = torch.randn(B, H, 64, 64, generator=torch.Generator().manual_seed(311)).cuda()
    q = torch.ones(B, T, 1, 64, dtype=dt, device="cuda")
    none, v = torch.zeros_like(q), torch.zeros(B, T, H, 64, dtype=dt, device="cuda")
    aT = decay.double() ** T
    folds = torch.floor(-torch.log2(aT) / 20) + 1
    want = aT[:, None, None] * S.double()
    lim = ((2 * folds + 2) * U + 2.0 ** -40)[:, None, None] * want.abs()
    _, S_out = gdn.decay_chunk_fwd(q, none, v, decay, S)
    assert ((S_out.double() - want).abs() <= lim).all()
    dS = gdn.decay_chunk_bwd(none, q, v, decay, None, v, S)[3]
    assert ((dS.double() - want).abs() <= lim).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_states_decay_over_many_boundaries(dtype):
    """One sequence cut into more than a hundred segments that add nothing to
    the state: S_out = a^T S_in, and dS_in = a^T dS_out.  Every boundary rounds
    the state once (its factor has 48 bits), the last segment its factor and the
    product: at most a U each of 130 for every value.  The roundings of the
    products go either way, and in the mean over a head's 4096 values are within
    6 U sqrt(130 / 3) / 64 < U: with the last factor's, 2 U.  (A factor rounded to
    fp32 shifts all of a head's values, here by up to 90 U in fp32 and 54 in bf16.)"""
    T, dt = 65536, DT[dtype]
    decay = (1 - 2.0 ** -torch.linspace(9, 16, 16)[[2, 3, 10, 14]]).cuda()
    S = torch.randn(1, 4, 64, 64, generator=torch.Generator().manual_seed(321)).cuda()
    q = torch.ones(1, T, 1, 64, dtype=dt, device="cuda")
    none, v = torch.zeros_like(q), torch.zeros(1, T, 4, 64, dtype=dt, device="cuda")
    want = decay.double()[:, None, None] ** T * S.double()
    for x in (gdn.decay_chunk_fwd(q, none, v, decay, S)[1],
              gdn.decay_chunk_bwd(none, q, v, decay, None, v, S)[3]):
        off = (x.double() - want) / want
        assert (off.abs() <= 130 * U).all()
        assert (off.mean((0, 2, 3)).abs() <= 2 * U).all(), off.mean((0, 2, 3)) / U
