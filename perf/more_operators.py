"""Linear attention with a decay for each head, and the norm and rotation of
queries and keys before it, as measured work.

  decay_fwd    decay_chunk_fwd: prompts or training chunks, packed or of one
               length, value head h with decay a_h, q and k of head h / (Hv/Hk)
                   S_t = a S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t
               from a state for each sequence to the next one
  decay_bwd    decay_chunk_bwd: its gradients in q, k, v and the entry state
  decay_step   decay_step: the same recurrence over a pool of states by single
               tokens, in place
  qk_fwd       qk_norm_rotary_fwd: per head of q and of k
                   z = scale w x rsqrt(mean(x^2) + eps),   y = R(pos) z
               with R turning pairs of z's first values by pos * freq
  qk_bwd       qk_norm_rotary_bwd: its gradients in q, k and both weights

Where ``own`` is false, run() computes them from elementary torch operations in
32 bits (powers of a decay and angles in 64), rounded once at the end; where it
is true it calls the package.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------- cases
def _chunk(op, n_seq, tokens, packed, Hk, Hv, D, dtype, state=True):
    return dict(op=op, n_seq=n_seq, tokens=tokens, packed=packed, Hk=Hk, Hv=Hv, D=D, dtype=dtype,
                state=state)


def _step(n_seq, max_len, ragged, Hk, Hv, D, dtype):
    return dict(op="decay_step", n_seq=n_seq, max_len=max_len, ragged=ragged, Hk=Hk, Hv=Hv, D=D,
                dtype=dtype)


def _qk(op, rows, Hq, Hk, D, rot, pairs, dtype, sliced=False):
    return dict(op=op, rows=rows, Hq=Hq, Hk=Hk, D=D, rot=rot, pairs=pairs, dtype=dtype,
                sliced=sliced)


def listed():
    return [
        # the longest forward chunk: 65,536 tokens of one sequence, 16 heads
        dict(_chunk("decay_fwd", 1, 65536, False, 16, 16, 128, "bf16"),
             name="decay_fwd_65536_h16_d128"),
        # a serving batch: 24 prompts of different lengths packed, two value heads to a key head
        dict(_chunk("decay_fwd", 24, 16411, True, 16, 32, 128, "bf16", state=False),
             name="decay_fwd_24packed_h16x32_d128"),
        # a small fp32 model's chunk of 256 tokens: latency counts
        dict(_chunk("decay_fwd", 1, 256, False, 2, 2, 64, "f32"), name="decay_fwd_256_h2_d64_f32"),
        # the backward of one training chunk (262,144 tokens in 8), one sequence
        dict(_chunk("decay_bwd", 1, 32768, False, 16, 16, 128, "bf16"),
             name="decay_bwd_32768_h16_d128"),
        # the same for a training batch of documents packed, shared key heads, fp32, odd lengths
        dict(_chunk("decay_bwd", 9, 4099, True, 2, 6, 64, "f32"), name="decay_bwd_9packed_h2x6_d64_f32"),
        # one user decoding: a token of one sequence, latency alone
        dict(_step(1, 1, False, 16, 16, 128, "bf16"), name="decay_step_1seq_h16_d128"),
        # a full decoding batch, two value heads to a key head: the states' traffic
        dict(_step(256, 1, False, 16, 32, 128, "bf16"), name="decay_step_256seq_h16x32_d128"),
        # drafted tokens to check, 1 to 5 for each of an odd number of sequences
        dict(_step(37, 5, True, 4, 8, 64, "f32"), name="decay_step_37seq_draft5_h4x8_d64_f32"),
        # q and k of one training chunk, out of one projection's rows
        dict(_qk("qk_fwd", 32768, 16, 16, 128, 128, "halves", "bf16", sliced=True),
             name="qk_fwd_32768_h16_d128"),
        # the backward on the longest chunk of the skewed partition
        dict(_qk("qk_bwd", 62720, 16, 16, 128, 128, "halves", "bf16"),
             name="qk_bwd_62720_h16_d128"),
        # one decoded token: latency alone
        dict(_qk("qk_fwd", 1, 16, 16, 128, 128, "halves", "bf16"), name="qk_fwd_1_h16_d128"),
        # an odd fp32 batch, half of each head rotated, neighbouring values as pairs, fewer key heads
        dict(_qk("qk_bwd", 4099, 6, 2, 64, 32, "neighbours", "f32"), name="qk_bwd_4099_h6x2_d64_f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["decay_fwd", "decay_bwd", "decay_step", "qk_fwd", "qk_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("decay_fwd", "decay_bwd"):
        Hk, D = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([64, 128, 128])
        Hv = Hk * rng.choice([1, 1, 2, 3] if Hk <= 8 else [1, 1, 2])
        # no more than the longest listed one of its direction, in fp32 a quarter of it
        most = (65536 if op == "decay_fwd" else 32768) * 16 * 128 // (Hv * D)
        packed = rng.random() < 0.5
        most = min(65536, most // (4 if dtype == "f32" else 1)) // (2 if packed else 1)
        tokens = _log_int(rng, 1, most)
        n_seq = _log_int(rng, 1, max(1, min(40, tokens // 8)))
        if not packed:
            n_seq = min(n_seq, 8)
            tokens = max(1, tokens // n_seq) * n_seq
        return _chunk(op, n_seq, tokens, packed, Hk, Hv, D, dtype, state=rng.random() < 0.6)
    if op == "decay_step":
        Hk, D = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([64, 128])
        Hv = Hk * rng.choice([1, 1, 2, 3] if Hk <= 8 else [1, 1, 2])
        max_len = rng.choice([1, 1, 2, 3, 5, 8, 17, 33])
        most = 256 * 32 * 128 * 128 // (D * D * Hv * max(1, max_len // 4))
        return _step(_log_int(rng, 1, max(1, min(256, most))), max_len,
                     max_len > 1 and rng.random() < 0.6, Hk, Hv, D, dtype)
    D = rng.choice([64, 72, 128, 128, 256])
    pairs = rng.choice(["halves", "halves", "neighbours"])
    rot = rng.choice([16, 32, 64, D // 16 * 16])
    Hk = rng.choice([1, 2, 4, 8, 16])
    Hq = Hk * rng.choice([1, 1, 2, 3, 4] if Hk <= 8 else [1, 2])
    most = 62720 * 32 * 128 // ((Hq + Hk) * D * (2 if dtype == "f32" else 1))
    return _qk(op, _log_int(rng, 1, min(65537, most)), Hq, Hk, D, rot, pairs, dtype,
               sliced=rng.random() < 0.4)


def _lengths(case):
    """Tokens of each sequence, by the case alone (prepare shuffles them)."""
    n = case["n_seq"]
    if case["op"] == "decay_step":
        m = case["max_len"]
        return [1 + (7 * i + m - 1) % m if case["ragged"] else m for i in range(n)]
    total = case["tokens"]
    if not case["packed"]:
        return [total // n] * n
    parts = [1 + (7 * i + 3) % 16 for i in range(n)]
    lens = [1 + i % 3 if i % 5 == 4 else max(1, total * p // sum(parts))
            for i, p in enumerate(parts)]
    lens[0] += total - sum(lens)
    return lens


# ------------------------------------------------------------------ inputs
def _decays(H, dev):
    """1 - 2^-5 for the shortest memory to 1 - 2^-12 for the longest."""
    return 1.0 - torch.exp2(-torch.linspace(5.0, 12.0, H, device=dev))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device=dev) * std

    s = {"case": dict(case)}
    if case["op"] in ("qk_fwd", "qk_bwd"):
        N, Hq, Hk, D = case["rows"], case["Hq"], case["Hk"], case["D"]
        q, k = normal(N, Hq, D).to(dt), normal(N, Hk, D).to(dt)
        if case["sliced"]:  # rows of one projection to q, k and as many v heads as k's
            qkv = torch.cat([q, k, k], 1)
            q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        # positions anywhere in a long context
        pos = torch.randint(0, 1 << 18, (N,), generator=gen, device=dev, dtype=torch.int32)
        freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=dev) / case["rot"])
        s.update(q=q, k=k, pos=pos, freq=freq, wq=1.0 + normal(D, std=0.1),
                 wk=1.0 + normal(D, std=0.1), q_scale=D ** -0.5, k_scale=1.0)
        if case["op"] == "qk_bwd":
            s.update(dyq=normal(N, Hq, D).to(dt), dyk=normal(N, Hk, D).to(dt))
        return s
    n, Hk, Hv, D = case["n_seq"], case["Hk"], case["Hv"], case["D"]
    order = torch.randperm(n, generator=gen, device=dev)
    lens = torch.tensor(_lengths(case), device=dev)[order]
    start = torch.zeros(n + 1, dtype=torch.int32, device=dev)
    start[1:] = torch.cumsum(lens, 0).to(torch.int32)
    N = sum(_lengths(case))

    def unit(x):
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    s.update(q=unit(normal(N, Hk, D)), k=unit(normal(N, Hk, D)), v=normal(N, Hv, D).to(dt),
             decay=_decays(Hv, dev), scale=1.0)
    if case["op"] == "decay_step":
        n_slots = n + n // 4 + 1
        slots = torch.randperm(n_slots, generator=gen, device=dev)[:n].to(torch.int32)
        s.update(state=normal(n_slots, Hv, D, D, std=0.5), slots=slots,
                 seq_start=start if case["ragged"] else None)
        return s
    s["S_in"] = normal(n, Hv, D, D, std=0.5) if case["state"] else None
    s["seq_start"] = start if case["packed"] else None
    if not case["packed"]:
        for name in ("q", "k", "v"):
            s[name] = s[name].unflatten(0, (n, N // n))
    if case["op"] == "decay_bwd":
        s.update(dO=normal(*s["v"].shape).to(dt), dS_out=normal(n, Hv, D, D, std=0.1))
    return s


# --------------------------------------------------------------- the passes
def run(s):
    return _RUN_OWN[s["case"]["op"]](s) if own else _RUN_PLAIN[s["case"]["op"]](s)


def _own_fwd(s):
    import linear_recurrence_chunked_gated_amd as gdn
    o, S_out = gdn.decay_chunk_fwd(s["q"], s["k"], s["v"], s["decay"], s["S_in"],
                                   seq_start=s["seq_start"], scale=s["scale"])
    return {"o": o, "S_out": S_out}


def _own_bwd(s):
    import linear_recurrence_chunked_gated_amd as gdn
    dq, dk, dv, dS_in = gdn.decay_chunk_bwd(s["q"], s["k"], s["v"], s["decay"], s["S_in"], s["dO"],
                                            s["dS_out"], seq_start=s["seq_start"],
                                            scale=s["scale"])
    return {"dq": dq, "dk": dk, "dv": dv, "dS_in": dS_in}


def _own_step(s):
    import linear_recurrence_chunked_gated_amd as gdn
    o = gdn.decay_step(s["q"], s["k"], s["v"], s["decay"], s["state"], s["slots"], s["seq_start"],
                       scale=s["scale"])
    return {"o": o, "state": s["state"]}


def _own_qk_fwd(s):
    import linear_recurrence_chunked_gated_amd as gdn
    yq, yk = gdn.qk_norm_rotary_fwd(s["q"], s["k"], s["pos"], s["freq"], s["wq"], s["wk"], eps=EPS,
                                    q_scale=s["q_scale"], k_scale=s["k_scale"],
                                    pairs=s["case"]["pairs"])
    return {"yq": yq, "yk": yk}


def _own_qk_bwd(s):
    import linear_recurrence_chunked_gated_amd as gdn
    dq, dk, dwq, dwk = gdn.qk_norm_rotary_bwd(s["q"], s["k"], s["pos"], s["freq"], s["wq"],
                                              s["wk"], s["dyq"], s["dyk"], eps=EPS,
                                              q_scale=s["q_scale"], k_scale=s["k_scale"],
                                              pairs=s["case"]["pairs"])
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


_RUN_OWN = {"decay_fwd": _own_fwd, "decay_bwd": _own_bwd, "decay_step": _own_step,
            "qk_fwd": _own_qk_fwd, "qk_bwd": _own_qk_bwd}


def _rows(s, reverse=False):
    """Token rows [n, L] of the sequences, padded at the end to one length (the
    pad points past the tokens), each in order or from its last token on; and
    the lengths [n]."""
    lens, dev = _lengths(s["case"]), s["q"].device
    n = len(lens)
    L, N = max(lens), sum(lens)
    if s["seq_start"] is not None:
        first, last = s["seq_start"][:-1].long(), s["seq_start"][1:].long()
    else:
        first = torch.arange(n, device=dev) * L
        last = first + L
    t = torch.arange(L, device=dev)
    row = last[:, None] - 1 - t if reverse else first[:, None] + t
    return torch.where(t < (last - first)[:, None], row, N), last - first


def _padded(x, rows, rep):
    """Tokens x [.., H, D] as [n, H * rep, L, D] in 32 bits, zeros in the pad."""
    x = x.reshape(-1, x.shape[-2], x.shape[-1]).float()
    x = torch.cat([x, x.new_zeros((1, x.shape[1], x.shape[2]))])
    x = x[rows].transpose(1, 2)
    return x.repeat_interleave(rep, 1) if rep > 1 else x


def _powers(a, e):
    """a^e of decays a [H] and whole exponents e >= 0, in 64 bits, rounded."""
    return (a.double().reshape(-1, *[1] * e.dim()) ** e.double()).float()


def _scan(x, u, w, a, E, first):
    """y_t = sum_{s <= t} a^(t-s) (x_t . u_s) w_s + a^(t+first) E x_t over
    [n, H, L, D], by blocks: within a block through the products of all its
    pairs, across blocks through the sums of w u^T before it."""
    n, H, L, D = x.shape
    C = min(128, L)
    nb = -(-L // C)
    dev = x.device
    pad = nb * C - L
    if pad:
        x, u, w = (torch.nn.functional.pad(t, (0, 0, 0, pad)) for t in (x, u, w))
    xb, ub, wb = (t.reshape(n, H, nb, C, D) for t in (x, u, w))
    r = torch.arange(C, device=dev)
    gap = r[:, None] - r
    M = torch.where(gap >= 0, _powers(a, gap.clamp(min=0)), 0.0)
    y = ((xb @ ub.transpose(-1, -2)) * M[:, None]) @ wb
    late = (wb * _powers(a, C - 1 - r)[:, None, :, None]).transpose(-1, -2) @ ub
    b = torch.arange(nb, device=dev)
    gap = b[:, None] - b - 1
    W = torch.where(gap >= 0, _powers(a, C * gap.clamp(min=0)), 0.0)
    entry = (W @ late.reshape(n, H, nb, D * D)).reshape(n, H, nb, D, D)
    y = y + (xb * _powers(a, r + 1)[:, None, :, None]) @ entry.transpose(-1, -2)
    y = y.reshape(n, H, nb * C, D)[:, :, :L]
    if E is not None:
        t = torch.arange(L, device=dev)
        y = y + (x[:, :, :L] * _powers(a, t + first)[:, :, None]) @ E.transpose(-1, -2)
    return y


def _exit_state(u, w, a, E, lens, more):
    """sum_t a^(len-1-t+more) w_t u_t^T + a^len E over [n, H, L, D]."""
    t = torch.arange(u.shape[2], device=u.device)
    e = (lens[:, None] - 1 - t + more).clamp(min=0)
    out = (w * _powers(a, e).transpose(0, 1)[..., None]).transpose(-1, -2) @ u
    return out if E is None else out + _powers(a, lens).t()[..., None, None] * E


def _unpadded(y, rows, like):
    """[n, H, L, D] back to token rows, in the type and shape of `like`."""
    H, D = y.shape[1], y.shape[3]
    N = like.numel() // (like.shape[-1] * like.shape[-2])
    out = y.new_zeros((N + 1, H, D))
    out[rows] = y.transpose(1, 2)
    return out[:N].reshape(*like.shape[:-2], H, D).to(like.dtype)


def _grouped(y, Hk):
    """The sum over the value heads of each key head."""
    n, H, L, D = y.shape
    return y.reshape(n, Hk, H // Hk, L, D).sum(2) if H > Hk else y


def _plain_fwd(s):
    rep = s["case"]["Hv"] // s["case"]["Hk"]
    rows, lens = _rows(s)
    q, k, v = _padded(s["q"], rows, rep), _padded(s["k"], rows, rep), _padded(s["v"], rows, 1)
    o = s["scale"] * _scan(q, k, v, s["decay"], s["S_in"], 1)
    return {"o": _unpadded(o, rows, s["v"]),
            "S_out": _exit_state(k, v, s["decay"], s["S_in"], lens, 0)}


def _plain_bwd(s):
    Hk = s["case"]["Hk"]
    rep = s["case"]["Hv"] // Hk
    a, S, G = s["decay"], s["S_in"], s["dS_out"]
    rows, lens = _rows(s)
    k, v = _padded(s["k"], rows, rep), _padded(s["v"], rows, 1)
    do = s["scale"] * _padded(s["dO"], rows, 1)
    dq = _grouped(_scan(do, v, k, a, None if S is None else S.transpose(-1, -2), 1), Hk)
    out = {"dq": _unpadded(dq, rows, s["q"])}
    rows, _ = _rows(s, reverse=True)
    q, k = _padded(s["q"], rows, rep), _padded(s["k"], rows, rep)
    v, do = _padded(s["v"], rows, 1), s["scale"] * _padded(s["dO"], rows, 1)
    out["dk"] = _unpadded(_grouped(_scan(v, do, q, a, G.transpose(-1, -2), 0), Hk), rows, s["k"])
    out["dv"] = _unpadded(_scan(k, q, do, a, G, 0), rows, s["v"])
    out["dS_in"] = _exit_state(q, do, a, G, lens, 1)
    return out


def _plain_step(s):
    rep = s["case"]["Hv"] // s["case"]["Hk"]
    slots = s["slots"].long()
    rows, lens = _rows(s)
    q, k, v = _padded(s["q"], rows, rep), _padded(s["k"], rows, rep), _padded(s["v"], rows, 1)
    S = s["state"][slots]
    o = s["scale"] * _scan(q, k, v, s["decay"], S, 1)
    s["state"].index_copy_(0, slots, _exit_state(k, v, s["decay"], S, lens, 0))
    return {"o": _unpadded(o, rows, s["v"]), "state": s["state"]}


def _turn(z, s, back=False):
    """z with its pairs turned by pos * freq (back: by the opposite angle)."""
    angle = s["pos"].double()[:, None] * s["freq"].double()
    c, sn = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    if back:
        sn = -sn
    R = 2 * s["freq"].numel()
    if s["case"]["pairs"] == "halves":
        x, y = z[..., :R // 2], z[..., R // 2:R]
        turned = torch.cat([x * c - y * sn, y * c + x * sn], -1)
    else:
        x, y = z[..., 0:R:2], z[..., 1:R:2]
        turned = torch.stack([x * c - y * sn, y * c + x * sn], -1).flatten(-2)
    return torch.cat([turned, z[..., R:]], -1)


def _plain_qk_fwd(s):
    def one(x, w, scale):
        f = x.float()
        n = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
        return _turn(n * (scale * w), s).to(x.dtype)

    return {"yq": one(s["q"], s["wq"], s["q_scale"]), "yk": one(s["k"], s["wk"], s["k_scale"])}


def _plain_qk_bwd(s):
    def one(x, w, scale, dy):
        f = x.float()
        rstd = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
        n = f * rstd
        g = scale * _turn(dy.float(), s, back=True)
        t = g * w
        dx = rstd * (t - n * (t * n).mean(-1, keepdim=True))
        return dx.to(x.dtype), (g * n).sum((0, 1))

    dq, dwq = one(s["q"], s["wq"], s["q_scale"], s["dyq"])
    dk, dwk = one(s["k"], s["wk"], s["k_scale"], s["dyk"])
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


_RUN_PLAIN = {"decay_fwd": _plain_fwd, "decay_bwd": _plain_bwd, "decay_step": _plain_step,
              "qk_fwd": _plain_qk_fwd, "qk_bwd": _plain_qk_bwd}


# ------------------------------------------------------------- what it costs
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("qk_fwd", "qk_bwd"):
        bwd = case["op"] == "qk_bwd"
        n = case["rows"] * (case["Hq"] + case["Hk"]) * case["D"]
        return {"bytes": n * e * (3 if bwd else 2) + case["rows"] * 4 + case["rot"] * 2
                + 2 * case["D"] * 4 * (2 if bwd else 1),
                "flops": n * (14 if bwd else 8)}
    lens, Hk, Hv, D = _lengths(case), case["Hk"], case["Hv"], case["D"]
    N, n = sum(lens), len(lens)
    state = n * Hv * D * D * 4
    if case["op"] == "decay_step":
        return {"bytes": 2 * state + N * (2 * Hk + 2 * Hv) * D * e + n * 4 + Hv * 4,
                "flops": N * Hv * 5 * D * D}
    # a product with the state and the state's own update for every token, or,
    # where that is less, the products of a sequence's pairs of tokens
    pairs = sum(min(4 * D * D * t, 2 * D * t * (t + 1)) for t in lens) * Hv
    if case["op"] == "decay_fwd":
        return {"bytes": N * (2 * Hk + 2 * Hv) * D * e + state * (1 + case["state"]) + Hv * 4,
                "flops": pairs}
    return {"bytes": N * (4 * Hk + 3 * Hv) * D * e + state * (2 + case["state"]) + Hv * 4,
            "flops": 3 * pairs}


# ----------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = {key: (t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t)
         for key, t in s.items()}
    return _EXACT[case["op"]](case, d)


def _sequences(case, d):
    """Each sequence's token rows, as slices of the flattened token tensors."""
    if d["seq_start"] is not None:
        b = d["seq_start"].tolist()
    else:
        b = [0]
        for t in _lengths(case):
            b.append(b[-1] + t)
    return [slice(b[i], b[i + 1]) for i in range(len(b) - 1)]


TILE = 2048


def _weighed(x, u, w, pw):
    """sum_{s <= t} a^(t-s) (x_t . u_s) w_s, every pair of tokens of a sequence
    by itself, [T, D]; pw = the powers of the decay."""
    T, out = x.shape[0], torch.zeros_like(w)
    i = torch.arange(T, device=x.device)
    for t in range(0, T, TILE):
        for b in range(0, t + 1, TILE):
            gap = i[t:t + TILE, None] - i[None, b:b + TILE]
            A = pw[gap.clamp(min=0)] * (gap >= 0)
            out[t:t + TILE] += (A * (x[t:t + TILE] @ u[b:b + TILE].t())) @ w[b:b + TILE]
    return out


def _pw(a, T):
    return a ** torch.arange(T + 1, device=a.device, dtype=torch.float64)


def _exact_fwd(case, d, S_in=None):
    q, k, v = (d[x].flatten(0, -3) for x in ("q", "k", "v"))
    G = case["Hv"] // case["Hk"]
    S_in = d["S_in"] if S_in is None else S_in
    o = torch.zeros_like(v)
    S_out = torch.zeros((case["n_seq"], case["Hv"], case["D"], case["D"]), dtype=torch.float64,
                        device=v.device)
    for i, sl in enumerate(_sequences(case, d)):
        for h in range(case["Hv"]):
            x, u, w, T = q[sl, h // G], k[sl, h // G], v[sl, h], sl.stop - sl.start
            pw = _pw(d["decay"][h], T)
            y = _weighed(x, u, w, pw)
            S_out[i, h] = (pw[:T].flip(0)[:, None] * w).t() @ u
            if S_in is not None:
                y += pw[1:, None] * (x @ S_in[i, h].t())
                S_out[i, h] += pw[T] * S_in[i, h]
            o[sl, h] = d["scale"] * y
    return {"o": o.reshape(d["v"].shape), "S_out": S_out}


def _exact_bwd(case, d):
    q, k, v, do = (d[x].flatten(0, -3) for x in ("q", "k", "v", "dO"))
    G = case["Hv"] // case["Hk"]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dS_in = torch.zeros_like(d["dS_out"])
    for i, sl in enumerate(_sequences(case, d)):
        for h in range(case["Hv"]):
            T, g = sl.stop - sl.start, h // G
            x, u, w, y = q[sl, g], k[sl, g], v[sl, h], d["scale"] * do[sl, h]
            a, S1 = d["decay"][h], d["dS_out"][i, h]
            pw = _pw(a, T)
            last = pw[:T].flip(0)[:, None]  # a^(T-1-t)
            # o_t = sum_{s<=t} a^(t-s) (q_t . k_s) v_s: the pairs' gradients
            dq[sl, g] += _weighed(y, w, u, pw)
            dk[sl, g] += _weighed(w.flip(0), y.flip(0), x.flip(0), pw).flip(0) + last * (w @ S1)
            dv[sl, h] = _weighed(u.flip(0), x.flip(0), y.flip(0), pw).flip(0) + last * (u @ S1.t())
            if d["S_in"] is not None:
                dq[sl, g] += pw[1:, None] * (y @ d["S_in"][i, h])
            dS_in[i, h] = (pw[1:, None] * y).t() @ x + pw[T] * S1
    return {"dq": dq.reshape(d["q"].shape), "dk": dk.reshape(d["k"].shape),
            "dv": dv.reshape(d["v"].shape), "dS_in": dS_in}


def _exact_step(case, d):
    G, slots = case["Hv"] // case["Hk"], d["slots"].long()
    a = d["decay"][:, None, None]
    o = torch.zeros_like(d["v"])
    seqs = _sequences(case, d)
    first = torch.tensor([sl.start for sl in seqs], device=o.device)
    lens = torch.tensor([sl.stop - sl.start for sl in seqs], device=o.device)
    head = torch.arange(case["Hv"], device=o.device) // G
    for t in range(int(lens.max())):  # one token after another
        live = (t < lens).nonzero()[:, 0]
        row, sl = first[live] + t, slots[live]
        k, q = d["k"][row][:, head], d["q"][row][:, head]
        S = a * d["state"][sl] + d["v"][row][..., :, None] * k[..., None, :]
        d["state"][sl] = S
        o[row] = d["scale"] * torch.matmul(S, q[..., None])[..., 0]
    return {"o": o, "state": d["state"]}


def _rotation(case, d):
    """The rotation of every token as a matrix on the first values, [N, R, R]."""
    F = d["freq"].numel()
    angle = d["pos"].double()[:, None] * d["freq"]
    i = torch.arange(F, device=angle.device)
    x, y = (i, i + F) if case["pairs"] == "halves" else (2 * i, 2 * i + 1)
    M = torch.zeros((angle.shape[0], 2 * F, 2 * F), dtype=torch.float64, device=angle.device)
    M[:, x, x] = torch.cos(angle)
    M[:, y, y] = torch.cos(angle)
    M[:, x, y] = -torch.sin(angle)
    M[:, y, x] = torch.sin(angle)
    return M


def _exact_qk(case, d):
    D, N, R = case["D"], case["rows"], 2 * d["freq"].numel()
    bwd = case["op"] == "qk_bwd"
    out = {}
    for x, w, scale, dy, names in ((d["q"], d["wq"], d["q_scale"], d.get("dyq"), ("yq", "dq", "dwq")),
                                   (d["k"], d["wk"], d["k_scale"], d.get("dyk"), ("yk", "dk", "dwk"))):
        root = (x.square().sum(-1, keepdim=True) / D + EPS).sqrt()
        y = (scale * w * (x / root)) if not bwd else scale * dy
        for t in range(0, N, 4096):  # a few tokens' matrices at a time
            part = {**d, "pos": d["pos"][t:t + 4096]}
            M = _rotation(case, part)
            y[t:t + 4096, :, :R] = y[t:t + 4096, :, :R] @ (M if bwd else M.transpose(1, 2)).contiguous()
        if not bwd:
            out[names[0]] = y
            continue
        g = y * w
        out[names[1]] = g / root - x * (g * x).sum(-1, keepdim=True) / (D * root ** 3)
        out[names[2]] = (y * (x / root)).reshape(-1, D).sum(0)
    return out


_EXACT = {"decay_fwd": _exact_fwd, "decay_bwd": _exact_bwd, "decay_step": _exact_step,
          "qk_fwd": _exact_qk, "qk_bwd": _exact_qk}
