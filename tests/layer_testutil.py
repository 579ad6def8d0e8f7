"""Plain 64-bit forms of the operators around the chunk, with error bounds of
fp32 kernels beside their values (not a test module).

U = 2^-24 is half a step of fp32.  A sum of n products whose terms are added
one after another in lanes and in a tree across lanes is off by at most
(adds on the longest path + 1) U times the sum of the terms' absolute values;
a value stored in type t by at most finfo(t).eps / 2 times itself.
"""
import torch

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def half_step(dtype):
    return torch.finfo(DT[dtype]).eps / 2


def check(name, got, ref, bound, dtype):
    """|got - ref| <= bound + the rounding of a value within bound of ref."""
    got, ref, bound = got.detach().cpu().double(), ref.double(), bound.double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    hs = half_step(dtype) if dtype else 0.0
    lim = bound + hs * (ref.abs() + bound) + 1e-38
    over = (got - ref).abs() - lim
    assert not torch.isnan(got).any(), "%s: NaN" % name
    assert (over <= 0).all(), "%s: off by %.3e where %.3e is allowed" % (
        name, (got - ref).abs().flatten()[over.argmax()], lim.flatten()[over.argmax()])


# ------------------------------------------------------------ the recurrence
def step_inputs(lens, Hk, Hv, D, dtype, n_slots, seed, decay=0.1, extra_rows=0):
    """A ragged batch on the CPU: every sequence's rows one after another,
    then extra_rows of no sequence."""
    g = torch.Generator().manual_seed(seed)
    N = sum(lens) + extra_rows

    def normal(*s):
        return torch.randn(s, generator=g)

    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    slots = torch.randperm(n_slots, generator=g)[:len(lens)].to(torch.int32)
    start = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    return dict(q=unit(normal(N, Hk, D)).to(DT[dtype]), k=unit(normal(N, Hk, D)).to(DT[dtype]),
                v=normal(N, Hv, D).to(DT[dtype]),
                alpha=torch.exp(-decay * torch.nn.functional.softplus(normal(N, Hv))),
                beta=torch.sigmoid(normal(N, Hv)), state=0.3 * normal(n_slots, Hv, D, D),
                slots=slots, seq_start=start)


def step_ref(d, lens, D):
    """(o, its bound, state, its bound): the recurrence in 64 bits.

    Each token adds, to a row r of the state, the errors of p = S k (two
    products a term, D/8 + 3 adds deep), of u and of the update's two
    roundings: at most (D/8 + 12) U (2 |S_r| + |v_r|) with |k|, |q| <= 1.01 and
    alpha, beta <= 1, and the exact update does not increase an error already
    there by more than |k|^2's excess over 1 (under 1.02 per token in bf16,
    taken as 1.05 to the number of tokens)."""
    q, k, v = d["q"].double(), d["k"].double(), d["v"].double()
    al, be, st = d["alpha"].double(), d["beta"].double(), d["state"].double().clone()
    Hv, rep = v.shape[1], v.shape[1] // q.shape[1]
    o, ob = torch.zeros(v.shape, dtype=torch.float64), torch.zeros(v.shape, dtype=torch.float64)
    sb = torch.zeros_like(st)
    t = 0
    for i, n in enumerate(lens):
        S = st[d["slots"][i]].clone()
        err = torch.zeros(Hv, D, dtype=torch.float64)  # per state row
        for _ in range(n):
            kt, qt = k[t].repeat_interleave(rep, 0), q[t].repeat_interleave(rep, 0)
            a, b = al[t][:, None], be[t][:, None]
            mag = 2 * S.norm(dim=-1) + v[t].abs()
            u = b * (v[t] - a * (S * kt[:, None]).sum(-1))
            S = a[..., None] * S + u[..., None] * kt[:, None]
            o[t] = (S * qt[:, None]).sum(-1)
            err = 1.05 * err + (D / 8 + 12) * U * (mag + u.abs())
            ob[t] = 1.05 * err
            t += 1
        st[d["slots"][i]] = S
        sb[d["slots"][i]] = err[..., None]
    return o, ob, st, sb


# -------------------------------------------------------------- the convolution
def conv_step_ref(x, w, state, slots, lens, act):
    """(y, its bound, state): the fp32 sum of W products is W deep; SiLU with
    an exponential whose argument is rounded once."""
    xd, wd, st = x.double(), w.double(), state.clone()
    W = w.shape[1]
    y, b = torch.zeros(x.shape, dtype=torch.float64), torch.zeros(x.shape, dtype=torch.float64)
    t = 0
    for i, n in enumerate(lens):
        ext = torch.cat([state[slots[i]], x[t:t + n]])
        e = ext.double()
        z = sum(wd[:, j] * e[W - 1 - j:W - 1 - j + n] for j in range(W))
        za = sum((wd[:, j] * e[W - 1 - j:W - 1 - j + n]).abs() for j in range(W))
        zb = (W + 1) * U * za
        if act:
            s = torch.sigmoid(z)
            y[t:t + n] = z * s
            # |d silu| <= 1.1; exp's relative error 2 (|z| + 2) U, the divide and 1 + e 4 U
            b[t:t + n] = 1.1 * zb + (z * s).abs() * (2 * z.abs() + 8) * U
        else:
            y[t:t + n], b[t:t + n] = z, zb
        st[slots[i]] = ext[n:]
        t += n
    return y, b, st


# ------------------------------------------------------------------- the norms
def _act(g, act):
    """act(g), act'(g), and the relative error of the kernel's act and the
    absolute one of its derivative: the exponential's 2 (|g| + 2) U, and 6 U of
    the operations after it."""
    if g is None:
        return None
    if not act:
        return g, torch.ones_like(g), torch.zeros_like(g), torch.zeros_like(g)
    s = torch.sigmoid(g)
    e = (2 * g.abs() + 10) * U
    return g * s, s * (1 + g * (1 - s)), e, 2 * e * s * (1 + g.abs())


# Adds on the longest path of a row's sum: 16 in a lane, 6 across a wave's
# lanes, 16 across waves; a mean's relative error is that plus its own ops.
DEEP = 16 + 6 + 16 + 4


def gated_norm_ref(x, gate, w, eps, scale, act):
    x = x.double()
    rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    y = scale * x * rstd * (1 if w is None else w.double())
    rel = torch.full_like(y, (DEEP / 2 + 8) * U)
    if gate is not None:
        a, _, ea, _ = _act(gate.double(), act)
        y = y * a
        rel = rel + ea
    return y, y.abs() * rel


def gated_norm_bwd_ref(x, gate, w, dy, eps, scale, act, depth):
    """((dx, dgate, dw), their bounds); depth: adds on dw's longest path."""
    x, e = x.double(), scale * dy.double()
    D = x.shape[-1]
    rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * rstd
    wd = torch.ones(D, dtype=torch.float64) if w is None else w.double()
    a, da, ea, eda = (torch.ones_like(x), None, 0.0, None) if gate is None else _act(gate.double(), act)
    base = (DEEP / 2 + 10) * U
    dn = e * wd * a
    m = (dn * n).mean(-1, keepdim=True)
    mabs = (dn * n).abs().mean(-1, keepdim=True)
    # with act's error taken at the row's largest gate
    worst = ea if gate is None else ea.amax(-1, keepdim=True)
    dx = rstd * (dn - n * m)
    dxb = rstd * ((dn.abs() + n.abs() * m.abs()) * (2 * base + ea)
                  + n.abs() * mabs * (DEEP * U + 2 * base + worst))
    dg = dgb = dw = dwb = None
    if gate is not None:
        dg = e * wd * n * da
        dgb = dg.abs() * 2 * base + (e * wd * n).abs() * eda
    if w is not None:
        t = e * n * a
        dw = t.reshape(-1, D).sum(0)
        dwb = (t.abs() * (base + ea + depth * U)).reshape(-1, D).sum(0)
    return (dx, dg, dw), (dxb, dgb, dwb)


def residual_norm_ref(x, r, w, s, eps, scale):
    """((y, h), bounds)."""
    h = x.double()
    hb = torch.zeros_like(h)
    if r is not None:
        add = scale * (1.0 if s is None else s.double()) * r.double()
        h = h + add
        hb = (2 * add.abs() + h.abs()) * U
    rms = torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    wd = 1.0 if w is None else w.double()
    y = wd * h / rms
    # h's error moves h itself and, through the mean, rstd
    hrel = torch.sqrt((hb * hb).mean(-1, keepdim=True)) / rms
    wa = 1.0 if w is None else w.double().abs()
    yb = wa * hb / rms + y.abs() * (hrel + (DEEP / 2 + 8) * U)
    return (y, h), (yb, hb)


def residual_norm_bwd_ref(h, r, w, s, dy, dh, eps, scale, depth):
    """((dx, dr, dw, ds), bounds); depth: adds on dw's and ds's longest path."""
    h, dy = h.double(), dy.double()
    C = h.shape[-1]
    rstd = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    n = h * rstd
    wd = torch.ones(C, dtype=torch.float64) if w is None else w.double()
    f = scale * (torch.ones(C, dtype=torch.float64) if s is None else s.double())
    dn = dy * wd
    m = (dn * n).mean(-1, keepdim=True)
    mabs = (dn * n).abs().mean(-1, keepdim=True)
    base = (DEEP / 2 + 8) * U
    g = rstd * (dn - n * m)
    gb = rstd * ((dn.abs() + n.abs() * m.abs()) * 2 * base + n.abs() * mabs * (DEEP * U + 2 * base))
    d = torch.zeros_like(h) if dh is None else dh.double()
    dx = d + g
    dxb = gb + (dx.abs() + gb) * U
    dr, drb = f * dx, f.abs() * dxb + (f * dx).abs() * 3 * U
    dw = (dy * n).reshape(-1, C).sum(0)
    dwb = ((dy * n).abs() * (base + depth * U)).reshape(-1, C).sum(0)
    ds = dsb = None
    if r is not None:
        t = dx * r.double()
        ds = scale * t.reshape(-1, C).sum(0)
        dsb = abs(scale) * (dxb * r.double().abs() + t.abs() * (4 + depth) * U).reshape(-1, C).sum(0)
    return (dx, dr, dw, ds), (dxb, drb, dwb, dsb)
