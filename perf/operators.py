"""The operators around the gated delta-rule chunk, as measured work.

A Gated DeltaNet layer needs more than its chunk: norms before and after it
(training and serving), and forms of the recurrence and of the short
convolution that advance a pool of sequences by single tokens (serving).

  step           recurrent_step: every sequence's state in a pool advances by
                 its new tokens, in place
                     S <- alpha S (I - beta k k^T) + beta v k^T,   o = S q
  conv_step      shortconv_step: the W-tap causal convolution of the same new
                 tokens over a pool of the last W-1 inputs, in place
  gated_norm     y = scale * w * x rsqrt(mean(x^2) + eps) * act(gate) per head;
                 without gate and weight, the L2 norm of q and k
  residual_norm  h = x + scale * s * r;  y = w * h rsqrt(mean(h^2) + eps)

Where ``own`` is false, run() computes them from elementary torch operations in
32 bits, rounded once at the end; where it is true it calls the package.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------- cases
def _step(n_seq, max_len, ragged, Hk, Hv, D, dtype, update=True):
    return dict(op="step", n_seq=n_seq, max_len=max_len, ragged=ragged, Hk=Hk, Hv=Hv, D=D,
                dtype=dtype, update=update)


def _conv(n_seq, max_len, ragged, C, W, dtype, act=1):
    return dict(op="conv_step", n_seq=n_seq, max_len=max_len, ragged=ragged, C=C, W=W,
                dtype=dtype, act=act)


def _gated(rows, H, D, dtype, bwd, gate=True, weight=True, sliced=False):
    return dict(op="gated_norm", rows=rows, H=H, D=D, dtype=dtype, bwd=bwd, gate=gate,
                weight=weight, sliced=sliced)


def _residual(rows, C, dtype, bwd, vector=True):
    return dict(op="residual_norm", rows=rows, C=C, dtype=dtype, bwd=bwd, vector=vector)


def listed():
    return [
        # one user decoding: a single token of a single sequence, latency alone
        dict(_step(1, 1, False, 16, 16, 128, "bf16"), name="step_1seq_h16_d128"),
        # a full decoding batch, two value heads to a key head: the states' traffic
        dict(_step(256, 1, False, 16, 32, 128, "bf16"), name="step_256seq_h16x32_d128"),
        # checking drafted tokens: 1 to 8 of them for each sequence
        dict(_step(64, 8, True, 16, 16, 128, "bf16"), name="step_64seq_draft8_h16_d128"),
        # a small fp32 model, an odd batch, short prompts of one length
        dict(_step(7, 33, False, 2, 6, 64, "f32"), name="step_7seq_len33_h2x6_d64_f32"),
        # the convolution over q, k and v of 16 heads for one user's token
        dict(_conv(1, 1, False, 6144, 4, "bf16"), name="conv_step_1seq_c6144"),
        # the same for a batch with 1 to 4 new tokens each
        dict(_conv(256, 4, True, 6144, 4, "bf16"), name="conv_step_256seq_draft4_c6144"),
        # the output norm and gate of one training chunk (262,144 tokens in 8)
        dict(_gated(32768, 16, 128, "bf16", False), name="gated_norm_fwd_32768x16x128"),
        # its backward on the longest chunk of the skewed partition
        dict(_gated(62720, 16, 128, "bf16", True), name="gated_norm_bwd_62720x16x128"),
        # L2 norm of q out of the convolution's [tokens, q k v] rows, fp32, a ragged chunk
        dict(_gated(4099, 2, 64, "f32", False, gate=False, weight=False, sliced=True),
             name="qk_norm_fwd_4099x2x64_f32"),
        # the norm before the next block with the residual sum, one training chunk
        dict(_residual(32768, 2048, "bf16", False), name="residual_norm_fwd_32768x2048"),
        # its backward: both residual branches, the weight and the residual scale
        dict(_residual(32768, 2048, "bf16", True), name="residual_norm_bwd_32768x2048"),
        # the same norm while decoding one token: latency alone
        dict(_residual(1, 2048, "bf16", False, vector=False), name="residual_norm_fwd_1x2048"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["step", "conv_step", "gated_norm", "residual_norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "step":
        Hk, D = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([64, 128])
        Hv = Hk * rng.choice([1, 1, 2, 3][:4 if Hk <= 8 else 3])
        max_len = rng.choice([1, 1, 2, 3, 5, 8, 17, 40, 129])
        most = 2_500_000_000 // (7 * D * D * Hv * max_len)  # no more than the longest listed work
        n_seq = _log_int(rng, 1, max(1, min(256, most)))
        return _step(n_seq, max_len, max_len > 1 and rng.random() < 0.6, Hk, Hv, D, dtype,
                     update=rng.random() < 0.85)
    if op == "conv_step":
        max_len = rng.choice([1, 1, 2, 4, 7, 30])
        return _conv(_log_int(rng, 1, 400 if max_len < 8 else 60), max_len,
                     max_len > 1 and rng.random() < 0.6, 8 * _log_int(rng, 8, 1024),
                     rng.choice([2, 3, 4, 4, 8]), dtype, act=rng.choice([0, 1, 1]))
    if op == "gated_norm":
        H, D = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([64, 72, 128, 128, 256, 512])
        gate = rng.random() < 0.75
        rows = _log_int(rng, 1, max(2, 60_000_000 // (H * D * (2 if dtype == "f32" else 1))))
        return _gated(min(rows, 65537), H, D, dtype, rng.random() < 0.5, gate=gate,
                      weight=gate or rng.random() < 0.5, sliced=rng.random() < 0.4)
    C = 8 * _log_int(rng, 8, 1024)
    rows = _log_int(rng, 1, max(2, 60_000_000 // (C * (2 if dtype == "f32" else 1))))
    return _residual(min(rows, 65537), C, dtype, rng.random() < 0.5, vector=rng.random() < 0.6)


def _lengths(case):
    """New tokens of each sequence, by the case alone (prepare shuffles them)."""
    m = case["max_len"]
    return [1 + (5 * i + m - 1) % m if case["ragged"] else m for i in range(case["n_seq"])]


# ------------------------------------------------------------------ inputs
def _pool_plan(case, gen, dev):
    """The batch's plan, which a server keeps: pool slots and token offsets."""
    n = case["n_seq"]
    n_slots = n + n // 4 + 1
    slots = torch.randperm(n_slots, generator=gen, device=dev)[:n].to(torch.int32)
    order = torch.randperm(n, generator=gen, device=dev)
    lens = torch.tensor(_lengths(case), device=dev)[order]
    start = torch.zeros(n + 1, dtype=torch.int32, device=dev)
    start[1:] = torch.cumsum(lens, 0).to(torch.int32)
    return n_slots, slots, start


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device=dev) * std

    s = {"case": dict(case)}
    if case["op"] == "step":
        n_slots, slots, start = _pool_plan(case, gen, dev)
        N, Hk, Hv, D = sum(_lengths(case)), case["Hk"], case["Hv"], case["D"]
        q, k = normal(N, Hk, D), normal(N, Hk, D)
        s.update(q=(q / q.norm(dim=-1, keepdim=True)).to(dt),
                 k=(k / k.norm(dim=-1, keepdim=True)).to(dt), v=normal(N, Hv, D).to(dt),
                 alpha=torch.exp(-0.1 * torch.nn.functional.softplus(normal(N, Hv))),
                 beta=torch.sigmoid(normal(N, Hv)),
                 state=normal(n_slots, Hv, D, D, std=0.1), slots=slots,
                 seq_start=start if case["ragged"] else None)
    elif case["op"] == "conv_step":
        n_slots, slots, start = _pool_plan(case, gen, dev)
        N, C, W = sum(_lengths(case)), case["C"], case["W"]
        s.update(x=normal(N, C).to(dt), w=normal(C, W) / W,
                 state=normal(n_slots, W - 1, C).to(dt), slots=slots,
                 seq_start=start if case["ragged"] else None)
    elif case["op"] == "gated_norm":
        N, H, D = case["rows"], case["H"], case["D"]

        def heads():
            if not case["sliced"]:
                return normal(N, H, D).to(dt)
            # the middle third of wider token rows, as out of one projection
            return normal(N, 3 * H, D).to(dt)[:, H:2 * H]

        s.update(x=heads(), gate=heads() if case["gate"] else None,
                 w=1.0 + normal(D, std=0.1) if case["weight"] else None,
                 scale=1.0 if case["weight"] else D ** -0.5)
        if case["bwd"]:
            s["dy"] = normal(N, H, D).to(dt)
    else:
        N, C = case["rows"], case["C"]
        s.update(r=normal(N, C).to(dt), w=1.0 + normal(C, std=0.1),
                 s=1.0 + normal(C, std=0.1) if case["vector"] else None, scale=0.5)
        if case["bwd"]:
            s.update(h=normal(N, C, std=2.0).to(dt), dy=normal(N, C).to(dt), dh=normal(N, C).to(dt))
        else:
            s["x"] = normal(N, C, std=2.0).to(dt)
    return s


# --------------------------------------------------------------- the passes
def run(s):
    return _RUN_OWN[s["case"]["op"]](s) if own else _RUN_PLAIN[s["case"]["op"]](s)


def _own_step(s):
    import linear_recurrence_chunked_gated_amd as gdn
    o = gdn.recurrent_step(s["q"], s["k"], s["v"], s["alpha"], s["beta"], s["state"], s["slots"],
                           s["seq_start"], update=s["case"]["update"])
    return {"o": o, "state": s["state"]}


def _own_conv_step(s):
    import linear_recurrence_chunked_gated_amd as gdn
    y = gdn.shortconv_step(s["x"], s["w"], s["state"], s["slots"], s["seq_start"],
                           act=s["case"]["act"])
    return {"y": y, "state": s["state"]}


def _own_gated_norm(s):
    import linear_recurrence_chunked_gated_amd as gdn
    if not s["case"]["bwd"]:
        return {"y": gdn.gated_norm_fwd(s["x"], s["gate"], s["w"], eps=EPS, scale=s["scale"])}
    dx, dgate, dw = gdn.gated_norm_bwd(s["x"], s["gate"], s["w"], s["dy"], eps=EPS,
                                       scale=s["scale"])
    return {"dx": dx, "dgate": dgate, "dw": dw}


def _own_residual_norm(s):
    import linear_recurrence_chunked_gated_amd as gdn
    if not s["case"]["bwd"]:
        y, h = gdn.residual_norm_fwd(s["x"], s["r"], s["w"], s["s"], scale=s["scale"], eps=EPS)
        return {"y": y, "h": h}
    dx, dr, dw, ds = gdn.residual_norm_bwd(s["h"], s["r"], s["w"], s["s"], s["dy"], s["dh"],
                                           scale=s["scale"], eps=EPS)
    return {"dx": dx, "dr": dr, "dw": dw, "ds": ds}


_RUN_OWN = {"step": _own_step, "conv_step": _own_conv_step, "gated_norm": _own_gated_norm,
            "residual_norm": _own_residual_norm}


def _plain_step(s):
    c, dt = s["case"], s["q"].dtype
    rep, n, N = c["Hv"] // c["Hk"], c["n_seq"], s["q"].shape[0]
    dev = s["q"].device
    q = s["q"].float().repeat_interleave(rep, 1)
    k = s["k"].float().repeat_interleave(rep, 1)
    v, alpha, beta = s["v"].float(), s["alpha"], s["beta"]
    slots = s["slots"].long()
    S = s["state"][slots]
    o = torch.empty((N + 1, c["Hv"], c["D"]), device=dev)  # one row more, for what is past an end
    if c["ragged"]:
        first, last = s["seq_start"][:-1].long(), s["seq_start"][1:].long()
    else:
        first = torch.arange(n, device=dev) * c["max_len"]
    for t in range(c["max_len"]):  # the recurrence itself: one token after another
        row = first + t
        live = row < last if c["ragged"] else None
        src = row.clamp(max=N - 1) if c["ragged"] else row
        kt, a, b = k[src], alpha[src, :, None, None], beta[src, :, None]
        S1 = a * S
        u = b * (v[src] - (S1 * kt[:, :, None, :]).sum(-1))
        S1 = S1 + u[..., None] * kt[:, :, None, :]
        out = (S1 * q[src][:, :, None, :]).sum(-1)
        if c["ragged"]:
            S = torch.where(live[:, None, None, None], S1, S)
            o[torch.where(live, row, N)] = out
        else:
            S = S1
            o[row] = out
    if c["update"]:
        s["state"].index_copy_(0, slots, S)
    return {"o": o[:N].to(dt), "state": s["state"]}


def _plain_conv_step(s):
    c, x = s["case"], s["x"]
    n, N, W = c["n_seq"], x.shape[0], c["W"]
    dev = x.device
    slots = s["slots"].long()
    if c["ragged"]:
        start = s["seq_start"].long()
    else:
        start = torch.arange(n + 1, device=dev) * c["max_len"]
    # rows of [the n sequences' states; x], W-1 rows of state before each sequence's tokens
    rows = torch.cat([s["state"][slots].reshape(n * (W - 1), c["C"]), x])
    seq = torch.searchsorted(start, torch.arange(N, device=dev), right=True) - 1

    def at(seq, first, i):  # index into rows of the i-th token of a sequence, i >= -(W-1)
        return torch.where(i >= 0, n * (W - 1) + first + i, seq * (W - 1) + (W - 1) + i)

    pos = torch.arange(N, device=dev) - start[seq]
    tap = torch.arange(W, device=dev)
    idx = at(seq[:, None], start[seq][:, None], pos[:, None] - tap)
    z = (rows[idx].float() * s["w"].t()).sum(1)
    y = z / (1.0 + torch.exp(-z)) if c["act"] else z
    each = torch.arange(n, device=dev)[:, None]
    keep = (start[1:] - start[:-1])[:, None] - (W - 1) + torch.arange(W - 1, device=dev)
    s["state"].index_copy_(0, slots, rows[at(each, start[:-1][:, None], keep)])
    return {"y": y.to(x.dtype), "state": s["state"]}


def _plain_gated_norm(s):
    c, dt = s["case"], s["x"].dtype
    x, scale = s["x"].float(), s["scale"]
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * rstd
    w = s["w"] if s["w"] is not None else 1.0
    if s["gate"] is not None:
        g = s["gate"].float()
        sig = 1.0 / (1.0 + torch.exp(-g))
        a = g * sig
    else:
        a = 1.0
    if not c["bwd"]:
        return {"y": (n * (scale * w) * a).to(dt)}
    dy = s["dy"].float() * scale
    dn = dy * w * a
    out = {"dx": (rstd * (dn - n * (dn * n).mean(-1, keepdim=True))).to(dt), "dgate": None,
           "dw": None}
    if s["gate"] is not None:
        out["dgate"] = (dy * w * n * (sig * (1.0 + g * (1.0 - sig)))).to(dt)
    if s["w"] is not None:
        out["dw"] = (dy * n * a).sum((0, 1))
    return out


def _plain_residual_norm(s):
    c, dt = s["case"], s["r"].dtype
    f = s["scale"] * s["s"] if s["s"] is not None else s["scale"]
    r = s["r"].float()
    if not c["bwd"]:
        h = s["x"].float() + f * r
        y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"]
        return {"y": y.to(dt), "h": h.to(dt)}
    h, dy = s["h"].float(), s["dy"].float()
    rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    n = h * rstd
    dn = dy * s["w"]
    dx = s["dh"].float() + rstd * (dn - n * (dn * n).mean(-1, keepdim=True))
    return {"dx": dx.to(dt), "dr": (f * dx).to(dt), "dw": (dy * n).sum(0),
            "ds": (s["scale"] * dx * r).sum(0) if s["s"] is not None else None}


_RUN_PLAIN = {"step": _plain_step, "conv_step": _plain_conv_step,
              "gated_norm": _plain_gated_norm, "residual_norm": _plain_residual_norm}


# ------------------------------------------------------------- what it costs
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "step":
        N, Hk, Hv, D = sum(_lengths(case)), case["Hk"], case["Hv"], case["D"]
        states = case["n_seq"] * Hv * D * D * 4 * (2 if case["update"] else 1)
        return {"bytes": states + N * (2 * Hk + 2 * Hv) * D * e + N * Hv * 8 + case["n_seq"] * 8,
                "flops": N * Hv * 7 * D * D}
    if case["op"] == "conv_step":
        N, C, W = sum(_lengths(case)), case["C"], case["W"]
        return {"bytes": case["n_seq"] * ((W - 1) * C * e * 2 + 8) + 2 * N * C * e + C * W * 4,
                "flops": N * C * (2 * W + (4 if case["act"] else 0))}
    if case["op"] == "gated_norm":
        n = case["rows"] * case["H"] * case["D"]
        tensors = (3 if case["bwd"] else 2) + (2 if case["bwd"] else 1) * case["gate"]
        return {"bytes": n * e * tensors + case["weight"] * case["D"] * 4 * (1 + case["bwd"]),
                "flops": n * (20 if case["bwd"] else 10)}
    n = case["rows"] * case["C"]
    # forward x, r, h, y; backward h, dy, dh, dx, dr, and r where the residual scale is learned
    tensors = (6 if case["vector"] else 5) if case["bwd"] else 4
    vectors = (1 + case["vector"]) * (1 + case["bwd"])
    return {"bytes": n * e * tensors + vectors * case["C"] * 4,
            "flops": n * (16 if case["bwd"] else 7)}


# ----------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = {key: (t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t)
         for key, t in s.items()}
    return _EXACT[case["op"]](case, d)


def _exact_step(case, d):
    N, G = d["q"].shape[0], case["Hv"] // case["Hk"]
    dev = d["q"].device
    lens = _lengths(case)
    bounds = (d["seq_start"].tolist() if case["ragged"] else
              [i * case["max_len"] for i in range(len(lens) + 1)])
    longest = max(lens)
    slots = d["slots"].long()
    head = torch.arange(case["Hv"], device=dev) // G
    S = d["state"][slots].clone()
    eye = torch.eye(case["D"], dtype=torch.float64, device=dev)
    o = torch.zeros((N, case["Hv"], case["D"]), dtype=torch.float64, device=dev)
    for t in range(longest):
        which = [i for i in range(len(lens)) if bounds[i] + t < bounds[i + 1]]
        i = torch.tensor(which, device=dev)
        row = torch.tensor([bounds[j] + t for j in which], device=dev)
        # a few sequences at a time: the transition matrix I - beta k k^T is formed as written
        for part in range(0, len(which), 32):
            ii, rr = i[part:part + 32], row[part:part + 32]
            k, q = d["k"][rr][:, head], d["q"][rr][:, head]
            a, b = d["alpha"][rr][..., None, None], d["beta"][rr][..., None, None]
            M = a * (eye - b * (k[..., :, None] * k[..., None, :]))
            Sn = torch.matmul(S[ii], M) + b * (d["v"][rr][..., :, None] * k[..., None, :])
            S[ii] = Sn
            o[rr] = torch.matmul(Sn, q[..., None])[..., 0]
    if case["update"]:
        d["state"][slots] = S
    return {"o": o, "state": d["state"]}


def _exact_conv_step(case, d):
    W, lens = case["W"], _lengths(case)
    bounds = (d["seq_start"].tolist() if case["ragged"] else
              [i * case["max_len"] for i in range(len(lens) + 1)])
    y, state, slots = torch.empty_like(d["x"]), d["state"], d["slots"].tolist()
    for i, slot in enumerate(slots):
        b, e = bounds[i], bounds[i + 1]
        ext = torch.cat([state[slot], d["x"][b:e]])
        z = sum(d["w"][:, j] * ext[W - 1 - j:W - 1 - j + e - b] for j in range(W))
        y[b:e] = z * torch.sigmoid(z) if case["act"] else z
        state[slot] = ext[e - b:]
    return {"y": y, "state": state}


def _exact_gated_norm(case, d):
    x, D = d["x"], case["D"]
    w = d["w"] if d["w"] is not None else torch.ones(D, dtype=torch.float64, device=x.device)
    g = d["gate"]
    act = torch.nn.functional.silu(g) if g is not None else torch.ones_like(x)
    root = (x.square().sum(-1, keepdim=True) / D + EPS).sqrt()
    if not case["bwd"]:
        return {"y": d["scale"] * w * (x / root) * act}
    up = d["scale"] * d["dy"]
    t = up * w * act  # the gradient of x / root
    dx = t / root - x * (t * x).sum(-1, keepdim=True) / (D * root ** 3)
    dgate = None
    if g is not None:
        sig = torch.sigmoid(g)
        dgate = up * w * (x / root) * (sig + g * sig * torch.sigmoid(-g))
    dw = (up * act * (x / root)).reshape(-1, D).sum(0) if d["w"] is not None else None
    return {"dx": dx, "dgate": dgate, "dw": dw}


def _exact_residual_norm(case, d):
    C, scale = case["C"], d["scale"]
    f = scale * (d["s"] if d["s"] is not None else torch.ones(C, dtype=torch.float64,
                                                               device=d["r"].device))
    if not case["bwd"]:
        h = torch.addcmul(d["x"], f.expand_as(d["r"]), d["r"])
        return {"y": d["w"] * h / (h.square().sum(-1, keepdim=True) / C + EPS).sqrt(), "h": h}
    h = d["h"]
    root = (h.square().sum(-1, keepdim=True) / C + EPS).sqrt()
    t = d["dy"] * d["w"]
    dx = d["dh"] + t / root - h * (t * h).sum(-1, keepdim=True) / (C * root ** 3)
    return {"dx": dx, "dr": f * dx, "dw": (d["dy"] * (h / root)).sum(0),
            "ds": scale * (dx * d["r"]).sum(0) if d["s"] is not None else None}


_EXACT = {"step": _exact_step, "conv_step": _exact_conv_step, "gated_norm": _exact_gated_norm,
          "residual_norm": _exact_residual_norm}
