"""The norm and rotation of queries and keys where its documented range ends:
values that are not finite beside the turned ones."""
import pytest
import torch

import linear_recurrence_chunked_gated_amd as gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_values_past_the_turned_ones_stay_by_themselves(pairs, dtype):
    """Values past the pairs are not turned: one that is not finite is as it
    would be without a rotation, and its neighbour too, in the outputs and in
    the weights' gradients."""
    g = torch.Generator().manual_seed(501)
    r = lambda *s: torch.randn(*s, generator=g).cuda()
    q, k, dy = r(5, 3, 64).to(dtype), r(5, 2, 64).to(dtype), r(5, 3, 64).to(dtype)
    freq = torch.full((16,), 0.3, device="cuda")
    w = 1 + 0.1 * r(64)
    w[40], w[63] = float("inf"), float("nan")
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    none = gdn.qk_norm_rotary_fwd(q, k, None, None, w, w)
    got = gdn.qk_norm_rotary_fwd(q, k, pos, freq, w, w, pairs=pairs)
    for x, y in zip(got, none):
        assert torch.equal(x[..., 32:].nan_to_num(7.0), y[..., 32:].nan_to_num(7.0))
        assert torch.isinf(x[..., 40].float()).all() and torch.isnan(x[..., 63].float()).all()
        assert torch.isfinite(x[..., :32].float()).all()

    w = 1 + 0.1 * r(64)
    dy[2, 1, 40], dy[3, 0, 63] = float("inf"), float("nan")
    dk = torch.zeros_like(k)
    none = gdn.qk_norm_rotary_bwd(q, k, None, None, w, w, dy, dk)[2]
    got = gdn.qk_norm_rotary_bwd(q, k, pos, freq, w, w, dy, dk, pairs=pairs)[2]
    bad = torch.zeros(64, dtype=torch.bool, device="cuda")
    bad[40] = bad[63] = True
    assert torch.equal(torch.isfinite(got), ~bad)
    assert torch.equal(got[32:].nan_to_num(7.0), none[32:].nan_to_num(7.0))
