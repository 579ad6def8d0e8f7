"""Plain 64-bit forms of linear attention with a decay and of the norm with
rotation, with error bounds of their kernels beside the values (not a test
module).

The chunk kernels work in blocks of 64 (fp32: 32) tokens:
    y_r = sum_{s <= r} P_rs w_s + a^(r+first) E x_r,   P_rs = a^(r-s) x_r . u_s
with the state E at the block's start.  H = 2^-8 is half a step of bf16, H^2
what two bf16 planes of an fp32 value leave of it, and three leave nothing.

 bf16 tensors: P and E are rounded to bf16 on the way to y, H of each term; E's
   own sums have w times its decay in two planes, H^2 of each term (the factors
   of the two compound: 4 H^2 in all), and in three where E ends as an output.
 fp32 tensors: every operand in three planes, and of the products of planes
   those down to H^2: the others are 2 H^3 and less.  P, P w, E and E x have
   one such product each: at most 8 H^3 of the sum of all terms' absolute values
   (H^3 = 2^-24 = U, what a sum in fp32 rounds to).
 fp32 sums: one U of the terms' absolute values for each of at most T + 64
   additions, and a few for the decays' factors.
"""
import torch

from layer_testutil import DT, U

H = 2.0 ** -8


def chunk_inputs(lens, Hk, Hv, D, dtype, seed, state=True, before=0, after=0, grads=False,
                 decay=None):
    """Packed sequences on the CPU, `before` rows ahead of the first and
    `after` behind the last."""
    g = torch.Generator().manual_seed(seed)
    N, n = sum(lens) + before + after, len(lens)
    rnd = lambda *s: torch.randn(s, generator=g)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    dt = DT[dtype]
    d = dict(q=unit(rnd(N, Hk, D)).to(dt), k=unit(rnd(N, Hk, D)).to(dt), v=rnd(N, Hv, D).to(dt),
             decay=1 - 2.0 ** -torch.linspace(1, 9, Hv) if decay is None
             else torch.full((Hv,), float(decay)),
             S_in=rnd(n, Hv, D, D) * 0.3 if state else None,
             seq_start=(torch.tensor([0] + lens).cumsum(0) + before).to(torch.int32))
    if grads:
        d.update(dO=rnd(N, Hv, D).to(dt), dS_out=rnd(n, Hv, D, D) * 0.3)
    return d


def _blocks(x, u, w, a, E, first, cuts, exact):
    """(y, bound, exit state, bound) of one head; cuts: tokens of each block;
    exact: fp32 tensors."""
    T, D = x.shape
    y, b = torch.zeros_like(w), torch.zeros_like(w)
    E = torch.zeros(D, D, dtype=torch.float64) if E is None else E.double()
    A = E.abs()  # the terms' absolute values
    t = 0
    for n in cuts:
        X, V, W = x[t:t + n], u[t:t + n], w[t:t + n]
        r = torch.arange(n)
        gap = r[:, None] - r
        M = torch.where(gap >= 0, a ** gap.clamp(min=0).double(), 0.0)
        P = (X @ V.t()) * M
        f = (a ** (r + first).double())[:, None]
        y[t:t + n] = P @ W + f * (X @ E.t())
        terms = ((X.abs() @ V.abs().t()) * M.abs()) @ W.abs() + f.abs() * (X.abs() @ A.t())
        b[t:t + n] = (8 * U if exact else 4 * H * H) * terms + (T + 64) * U * terms
        if not exact:
            b[t:t + n] += H * (P.abs() @ W.abs() + f.abs() * (X.abs() @ E.abs().t()))
        dec = (a ** (n - r - first).double())[:, None]
        E = a ** n * E + (dec * W).t() @ V
        A = abs(a) ** n * A + (dec.abs() * W.abs()).t() @ V.abs()
        t += n
    return y, b, E, (T + 72) * U * A


def _cuts(T):
    return [min(64, T - t) for t in range(0, T, 64)]


def chunk_ref(d, scale=1.0):
    """((o, S_out), bounds); rows of no sequence 0."""
    Hk, Hv, n = d["q"].shape[1], d["v"].shape[1], d["seq_start"].numel() - 1
    exact = d["q"].dtype == torch.float32
    q, k, v = (d[x].double() for x in ("q", "k", "v"))
    o, ob = torch.zeros_like(v), torch.zeros_like(v)
    D = v.shape[-1]
    S, Sb = torch.zeros(n, Hv, D, D).double(), torch.zeros(n, Hv, D, D).double()
    st = d["seq_start"].tolist()
    for i in range(n):
        sl = slice(st[i], st[i + 1])
        for h in range(Hv):
            g = h * Hk // Hv
            y, b, S[i, h], Sb[i, h] = _blocks(
                q[sl, g], k[sl, g], v[sl, h], float(d["decay"][h].double()),
                None if d["S_in"] is None else d["S_in"][i, h], 1, _cuts(st[i + 1] - st[i]), exact)
            o[sl, h], ob[sl, h] = scale * y, abs(scale) * b
    return (o, S), (ob, Sb)


def chunk_bwd_ref(d, scale=1.0):
    """((dq, dk, dv, dS_in), bounds)."""
    Hk, Hv, n = d["q"].shape[1], d["v"].shape[1], d["seq_start"].numel() - 1
    exact = d["q"].dtype == torch.float32
    q, k, v, do = (d[x].double() for x in ("q", "k", "v", "dO"))
    out = [torch.zeros_like(t) for t in (q, k, v)]
    bnd = [torch.zeros_like(t) for t in (q, k, v)]
    dS, dSb = torch.zeros_like(d["dS_out"]).double(), torch.zeros_like(d["dS_out"]).double()
    st = d["seq_start"].tolist()
    for i in range(n):
        sl, cuts = slice(st[i], st[i + 1]), _cuts(st[i + 1] - st[i])
        for h in range(Hv):
            g, a = h * Hk // Hv, float(d["decay"][h].double())
            x, u, w, y = q[sl, g], k[sl, g], v[sl, h], do[sl, h]
            S = None if d["S_in"] is None else d["S_in"][i, h].t()
            G = d["dS_out"][i, h]
            dq, b, _, _ = _blocks(y, w, u, a, S, 1, cuts, exact)
            out[0][sl, g] += scale * dq
            bnd[0][sl, g] += abs(scale) * b
            r = lambda t: t.flip(0)
            dv, b, dS[i, h], dSb[i, h] = _blocks(r(u), r(x), scale * r(y), a, G, 0, cuts[::-1], exact)
            out[2][sl, h], bnd[2][sl, h] = r(dv), r(b)
            dk, b, _, _ = _blocks(r(w), scale * r(y), r(x), a, G.t(), 0, cuts[::-1], exact)
            out[1][sl, g] += r(dk)
            bnd[1][sl, g] += r(b)
    return tuple(out) + (dS,), tuple(bnd) + (dSb,)


def step_ref(d, lens, scale=1.0):
    """((o, state), bounds) of the single-token form: fp32 throughout, one
    rounding for each of the update's two operations on every token, D + 8
    adds and products of the output's sum."""
    Hk, Hv, D = d["q"].shape[1], d["v"].shape[1], d["v"].shape[2]
    o, ob = torch.zeros(d["v"].shape).double(), torch.zeros(d["v"].shape).double()
    st, sb = d["state"].double(), torch.zeros(d["state"].shape).double()
    a = d["decay"].double()[:, None, None]
    rep = lambda x: x.double().repeat_interleave(Hv // Hk, 0)
    t = 0
    for i, n in enumerate(lens):
        s = int(d["slots"][i])
        S, B = st[s].clone(), sb[s].clone()
        for j in range(t, t + n):
            q, k, v = rep(d["q"][j]), rep(d["k"][j]), d["v"][j].double()
            S = a * S + v[:, :, None] * k[:, None, :]
            B = a.abs() * B + ((a * S).abs() + S.abs() + (v[:, :, None] * k[:, None, :]).abs()) * 2 * U
            o[j] = scale * (S @ q[:, :, None])[..., 0]
            ob[j] = abs(scale) * ((B + (D / 8 + 12) * U * S.abs()) @ q.abs()[:, :, None])[..., 0]
        st[s], sb[s] = S, B
        t += n
    return (o, st), (ob, sb)


# ---------------------------------------------------------------- the rotation
# A row's mean is summed over at most 512 values, 8 in a lane, 6 across lanes.
DEEP = 8 + 6 + 4


def turn(z, pos, freq, pairs, back=False):
    """z [N, H, D] turned; the pair's length beside it, which bounds either
    value."""
    if freq is None:
        return z, z.abs()
    F = freq.numel()
    ang = pos.double()[:, None] * freq.double()
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None] * (-1 if back else 1)
    i = torch.arange(F)
    x, y = (i, i + F) if pairs == "halves" else (2 * i, 2 * i + 1)
    out, size = z.clone(), z.abs()
    out[..., x], out[..., y] = z[..., x] * c - z[..., y] * s, z[..., y] * c + z[..., x] * s
    size[..., x] = size[..., y] = z[..., x].abs() + z[..., y].abs()
    return out, size


# The angle's fraction of a turn is rounded once to fp32 (pi 2^-25 of a radian),
# its sine and cosine are within 4 U, and the turn takes two products.
TURN = (3.2 / 2 + 4 + 2) * U


def rotary_ref(x, pos, freq, w, eps, scale, pairs):
    x = x.double()
    rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    z = scale * x * rstd * (1.0 if w is None else w.double())
    y, size = turn(z, pos, freq, pairs)
    return y, size * ((DEEP / 2 + 8) * U + TURN)


def rotary_bwd_ref(x, pos, freq, w, dy, eps, scale, pairs, depth):
    """((dx, dw), bounds); depth: adds on dw's longest path."""
    x = x.double()
    D = x.shape[-1]
    rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * rstd
    g, size = turn(scale * dy.double(), pos, freq, pairs, back=True)
    gb = size * (TURN + 2 * U)
    wd = torch.ones(D, dtype=torch.float64) if w is None else w.double()
    t, tb = g * wd, gb * wd.abs()
    base = (DEEP / 2 + 10) * U
    m = (t * n).mean(-1, keepdim=True)
    mb = ((tb + t.abs() * (2 * base + DEEP * U)) * n.abs()).mean(-1, keepdim=True)
    dx = rstd * (t - n * m)
    dxb = rstd * (tb + (t.abs() + n.abs() * m.abs()) * 2 * base + n.abs() * mb)
    dw = (g * n).reshape(-1, D).sum(0)
    dwb = (n.abs() * (gb + g.abs() * (base + depth * U))).reshape(-1, D).sum(0)
    return (dx, dw), (dxb, dwb)
