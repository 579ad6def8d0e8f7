"""Refusals of the Python calls of linear attention with a decay and of the norm
with rotation: each by its own error, with the tensors and arguments made before
the call that is refused."""
import pytest
import torch

import linear_recurrence_chunked_gated_amd as gdn
from linear_recurrence_chunked_gated_amd import GDNError

pytestmark = pytest.mark.gpu


class _T:
    """Tensors of a call that is taken: 6 rows, 2 key heads, 4 value heads, two
    sequences."""

    def __init__(self):
        z = lambda *s: torch.zeros(*s, device="cuda")
        self.x, self.y, self.v, self.dO = z(6, 2, 64), z(6, 2, 64), z(6, 4, 64), z(6, 4, 64)
        self.a, self.S, self.fr = torch.ones(4, device="cuda"), z(2, 4, 64, 64), torch.ones(32, device="cuda")
        self.st = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
        self.grads = z(6, 2, 64), z(6, 2, 64), z(6, 4, 64), z(2, 4, 64, 64)

    def fwd(self, **kw):
        a = dict(q=self.x, k=self.y, v=self.v, decay=self.a, S_in=self.S, seq_start=self.st)
        return gdn.decay_chunk_fwd, dict(a, **kw)

    def bwd(self, **kw):
        a = dict(q=self.x, k=self.y, v=self.v, decay=self.a, S_in=self.S, dO=self.dO, seq_start=self.st)
        return gdn.decay_chunk_bwd, dict(a, **kw)

    def step(self, **kw):
        a = dict(q=self.x, k=self.y, v=self.v, decay=self.a, state=self.S, seq_start=self.st)
        return gdn.decay_step, dict(a, **kw)

    def qk(self, **kw):
        return gdn.qk_norm_rotary_fwd, dict(dict(q=self.x, k=self.y, freq=self.fr), **kw)


def _turned(x):
    return x.transpose(0, 1).contiguous().transpose(0, 1)


def _batch(x):
    return x[None].expand(2, -1, -1, -1)


CASES = {
    "offsets on the host": (lambda t: t.fwd(seq_start=t.st.cpu()), ValueError, "seq_start is on cpu"),
    "offsets of 64 bits": (lambda t: t.fwd(seq_start=t.st.long()), TypeError, "seq_start has dtype torch.int64"),
    "decay on the host": (lambda t: t.fwd(decay=t.a.cpu()), ValueError, "decay is on cpu"),
    "decay of 64 bits": (lambda t: t.fwd(decay=t.a.double()), TypeError, "decay has dtype torch.float64"),
    "decays for other heads": (lambda t: t.fwd(decay=t.a[:2]), ValueError, r"decay has shape \(2,\), expected \(4,\)"),
    "states for other sequences": (lambda t: t.fwd(S_in=t.S[:1]), ValueError, r"S_in has shape \(1, 4, 64, 64\)"),
    "states in bf16": (lambda t: t.fwd(S_in=t.S.bfloat16()), TypeError, "S_in has dtype torch.bfloat16"),
    "k of another type": (lambda t: t.fwd(k=t.y.bfloat16()), TypeError, "k has dtype torch.bfloat16"),
    "k of other rows": (lambda t: t.fwd(k=t.y[:5]), ValueError, r"k has shape \(5, 2, 64\), expected \(6, 2, 64\)"),
    "offsets for rows by the batch": (lambda t: t.fwd(q=t.x[None], k=t.y[None], v=t.v[None]), ValueError,
                                      "packed sequences"),
    "v without heads": (lambda t: t.fwd(v=t.v[:, 0]), ValueError, "q and v must be"),
    "heads that no group divides": (lambda t: t.fwd(v=t.v[:, :3].contiguous(), decay=t.a[:3],
                                                    S_in=t.S[:, :3].contiguous()),
                                    GDNError, "Hv must be a multiple of Hk"),
    "half precision": (lambda t: t.fwd(q=t.x.half(), k=t.y.half(), v=t.v.half()), TypeError,
                       "q must be bfloat16 or float32"),
    "transposed rows": (lambda t: t.fwd(q=t.x.transpose(1, 2).contiguous().transpose(1, 2)), ValueError,
                        "q: each token's row must be contiguous"),
    "a broadcast batch": (lambda t: t.fwd(q=_batch(t.x), k=_batch(t.y), v=_batch(t.v), seq_start=None),
                          ValueError, "q: the rows of all leading dimensions must lie at one stride"),
    "o on its input": (lambda t: t.fwd(o=t.v), GDNError, "o overlaps input v"),
    "S_out on S_in": (lambda t: t.fwd(S_out=t.S), GDNError, "S_out overlaps input S_in"),
    "o of another type": (lambda t: t.fwd(o=t.dO.bfloat16()), TypeError, "o has dtype torch.bfloat16"),
    "a gradient of other rows": (lambda t: t.bwd(dO=t.dO[:5]), ValueError, r"dO has shape \(5, 4, 64\)"),
    "a transposed gradient": (lambda t: t.bwd(dO=_turned(t.dO)), ValueError, "dO must be contiguous"),
    "a state's gradient of other sequences": (lambda t: t.bwd(dS_out=t.S[:1]), ValueError,
                                              r"dS_out has shape \(1, 4, 64, 64\)"),
    "gradients on an input": (lambda t: t.bwd(grads=(t.x,) + t.grads[1:]), GDNError, "dq overlaps input q"),
    "gradients on each other": (lambda t: t.bwd(grads=(t.grads[0], t.grads[0]) + t.grads[2:]), GDNError,
                                "overlap"),
    "too few gradients": (lambda t: t.bwd(grads=t.grads[:2]), TypeError, "grads must be a tuple of 4 outputs"),
    "a pool of other heads": (lambda t: t.step(state=t.S[:, :2].contiguous()), ValueError,
                              r"state has shape \(2, 2, 64, 64\)"),
    "slots for other sequences": (lambda t: t.step(slots=torch.zeros(3, dtype=torch.int32, device="cuda")),
                                  ValueError, r"seq_start has shape \(3,\), expected \(4,\)"),
    "pairs of another kind": (lambda t: t.qk(pairs="both"), ValueError, "pairs must be 'halves' or 'neighbours'"),
    "more frequencies than pairs": (lambda t: t.qk(freq=torch.ones(40, device="cuda")), GDNError,
                                    "F must be in 0 .. D / 2"),
    "positions of 64 bits": (lambda t: t.qk(pos=torch.zeros(6, dtype=torch.int64, device="cuda")), TypeError,
                             "pos has dtype torch.int64"),
    "positions of other rows": (lambda t: t.qk(pos=torch.zeros(5, dtype=torch.int32, device="cuda")), ValueError,
                                r"pos has shape \(5,\), expected \(6,\)"),
    "a weight of another size": (lambda t: t.qk(wq=torch.ones(32, device="cuda")), ValueError,
                                 r"wq has shape \(32,\), expected \(64,\)"),
    "positions past 32 bits": (lambda t: t.qk(first=2 ** 31 - 2), GDNError, r"positions past 2\^31 - 1"),
    "a negative epsilon": (lambda t: t.qk(eps=-1.0), GDNError, "eps must be >= 0"),
}


@pytest.mark.parametrize("what", list(CASES))
def test_refused_by_its_own_error(what):
    make, kind, message = CASES[what]
    call, args = make(_T())
    with pytest.raises(kind, match=message) as e:
        call(**args)
    assert type(e.value) is kind


def test_the_calls_are_taken_without_the_fault():
    t = _T()
    for call, args in (t.fwd(), t.bwd(grads=t.grads), t.step(), t.qk()):
        call(**args)
    torch.cuda.synchronize()
