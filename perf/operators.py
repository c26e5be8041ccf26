"""The operators of the 8-bit KV cache: cases, plain forms and their work.

A cache row (b, h) holds rotated keys and values in 8 bits ("e4m3" or
"int8") with one fp32 scale per block of 128 tokens and head, for K and for
V, and per block the channel-wise bounds of its keys as int8 in units of
(block scale * Q / 127), Q = 448 (e4m3) or 127 (int8). Four operators:

* write: rotate (RoPE) and quantise new tokens into the cache, raising a
  partly filled block's scale (and re-rounding what it holds) when needed;
  what was written is read back as bf16, as chunked prefill does;
* read: a range of the cache as bf16 [B, T, H, 128];
* select: per (row, KV head) the K blocks whose bounds admit the largest
  scores for the query, the first and the last visible block always kept;
* decode: one query token per head against the visible tokens of the cache,
  of all its blocks or of a list of blocks.

Scores and out come from the codes as they are, so both sides see the same
inputs; the quantiser is defined operation by operation in fp32 (no fused
multiply-add) and the selection's query codes and scores are rounded from
fp64, so codes and lists are equal and not merely near.
"""

import math

import torch

own = False

D = 128           # head dim
BLK = 128         # tokens per block
QMAX = {"e4m3": 448.0, "int8": 127.0}    # largest code
RQMAX = {k: 1.0 / q for k, q in QMAX.items()}        # factors in fp32
UNIT = {k: 127.0 / q for k, q in QMAX.items()}       # codes to bound units
TINY = 2.0 ** -126
THETA = 1e7


# ------------------------------------------------------------------ cases
def listed():
    c = lambda name, op, **kw: dict(name=name, op=op, **kw)  # noqa: E731
    return [
        # one sequence decoding: the step's token enters the cache
        c("append_1x32", "write", kind="e4m3", layout="interleaved", B=1,
          H=32, T=1, L=4096),
        # a serving batch of grouped-head rows at ragged lengths
        c("append_64x8", "write", kind="int8", layout="half", B=64, H=8, T=1,
          L=4096),
        # a 32K prompt written in one call behind a cached prefix
        c("write_32k", "write", kind="e4m3", layout="interleaved", B=1, H=32,
          T=32768, L=36864),
        # a short cached prefix read back to attend over it in bf16
        c("read_2x2111", "read", kind="int8", B=2, H=8, T=2111, L=8192),
        # a 128K prefix read back for the next prompt chunk
        c("read_128k", "read", kind="e4m3", B=1, H=32, T=131072, L=131072),
        # decode, short cache: latency
        c("decode_2k", "decode", kind="e4m3", layout="interleaved", B=1,
          H=32, G=1, L=2048, ragged=False),
        # decode, a ragged batch with grouped heads and packed starts
        c("decode_16x32k", "decode", kind="int8", layout="half", B=16, H=8,
          G=4, L=32768, ragged=True),
        # decode against a 1M-token cache
        c("decode_1m", "decode", kind="e4m3", layout="interleaved", B=1,
          H=32, G=1, L=1 << 20, ragged=False),
        # block selection for a small batch, grouped heads
        c("select_4x32k", "select", kind="int8", layout="half", B=4, H=8,
          G=4, L=32768, K=64, ragged=True),
        # block selection over a 1M-token cache
        c("select_1m", "select", kind="e4m3", layout="interleaved", B=1,
          H=32, G=1, L=1 << 20, K=512, ragged=False),
        # attention over 64 of up to 1024 blocks per head
        c("sparse_8x128k", "sparse", kind="int8", layout="half", B=8, H=8,
          G=4, L=131072, K=64, ragged=True),
        # attention over 512 of 8192 blocks per head
        c("sparse_1m", "sparse", kind="e4m3", layout="interleaved", B=1,
          H=32, G=1, L=1 << 20, K=512, ragged=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "select", "sparse"])
    c = {"op": op, "kind": rng.choice(["e4m3", "int8"]),
         "layout": rng.choice(["interleaved", "half"]),
         "B": _log_int(rng, 1, 64), "H": rng.choice([1, 2, 4, 5, 8, 16, 32])}
    # tokens x heads of the whole batch: at most half the 1M-token case
    cap = max(1, (1 << 24) // (c["B"] * c["H"]))
    if op in ("write", "read"):
        cap = max(1, (1 << 20) // (c["B"] * c["H"]))
        c["T"] = min(cap, _log_int(rng, 1, 32768))
        c["L"] = c["T"] + rng.randint(1, 4096)
        if op == "read":
            del c["layout"]
        return c
    c["G"] = rng.choice([1, 1, 2, 3, 4, 7, 8, 16])
    c["L"] = min(cap, _log_int(rng, 1 if op == "decode" else 300, 1 << 19))
    c["ragged"] = rng.random() < 0.7
    if op != "decode":
        nblk = -(-c["L"] // BLK)
        c["K"] = max(2, min(_log_int(rng, 2, 1024), nblk))
    return c


def _ranges(case):
    """Visible range (start, length) of each row: the same for every seed."""
    B, L = case["B"], case["L"]
    if not case["ragged"]:
        return [0] * B, [L] * B
    length = [max(1, L - (b * 7919 * (L // 8 + 1)) % max(1, (7 * L) // 8))
              for b in range(B)]
    start = [0 if b % 3 == 0 else (n // 5) * (b % 3) // 2
             for b, n in enumerate(length)]
    return start, length


def _starts(case):
    """First new slot of each row of a write, behind a cached prefix."""
    room = case["L"] - case["T"]
    return [(room * 5 // 8 + b * 337) % (room + 1) for b in range(case["B"])]


# ------------------------------------------------------------- inputs
def _encode(x, kind):
    if kind == "int8":
        return torch.clamp(torch.round(x), -127, 127).to(torch.int8)
    return torch.clamp(x, -448, 448).to(torch.float8_e4m3fn)


def _bounds_of(codes, kind):
    """[..., n, BLK, D] codes as floats -> int8 [..., n, 2, D] (lo, hi)."""
    u = UNIT[kind]
    lo = torch.floor(codes.amin(-2) * u).clamp(-127, 127)
    hi = torch.ceil(codes.amax(-2) * u).clamp(-127, 127)
    return torch.stack([lo, hi], -2).to(torch.int8)


def _cache(case, gen):
    """A filled cache: keys whose blocks lean in directions of their own
    with a few strong channels, values N(0, 1)."""
    B, H, L, kind = case["B"], case["H"], case["L"], case["kind"]
    n = -(-L // BLK)
    dev = "cuda"
    dt = torch.int8 if kind == "int8" else torch.float8_e4m3fn
    k = torch.empty((B, H, L, D), dtype=dt, device=dev)
    v = torch.empty((B, H, L, D), dtype=dt, device=dev)
    ks = torch.empty((B, H, n), device=dev)
    vs = torch.empty((B, H, n), device=dev)
    kb = torch.empty((B, H, n, 2, D), dtype=torch.int8, device=dev)
    chan = torch.where(torch.arange(D, device=dev) % 31 == 3, 3.0, 0.8)
    step = max(1, (1 << 19) // (n * BLK))      # heads per pass
    rows = B * H
    for r in range(0, rows, step):
        e = min(rows, r + step)
        for codes, scale, is_key in ((k, ks, True), (v, vs, False)):
            x = torch.randn((e - r, n, BLK, D), generator=gen, device=dev)
            if is_key:
                x += torch.randn((e - r, n, 1, D), generator=gen, device=dev)
                x *= chan
            s = x.abs().amax((-2, -1)) * RQMAX[kind]
            c = _encode(x / s[..., None, None], kind)
            if is_key:
                kb.view(rows, n, 2, D)[r:e] = _bounds_of(c.float(), kind)
            codes.view(rows, L, D)[r:e] = c.view(e - r, n * BLK, D)[:, :L]
            scale.view(rows, n)[r:e] = s
    return k, v, ks, vs, kb


def _table(max_pos):
    """(cos, sin) of position * theta^(-2k/D): angles in fp64, [max_pos, D/2, 2]
    fp32, as the framework's rotations take it."""
    inv = THETA ** (-torch.arange(D // 2, dtype=torch.float64,
                                  device="cuda") * 2 / D)
    out = torch.empty((max_pos, D // 2, 2), device="cuda")
    for p in range(0, max_pos, 1 << 18):
        a = torch.arange(p, min(max_pos, p + (1 << 18)), dtype=torch.float64,
                         device="cuda")[:, None] * inv
        out[p:p + (1 << 18)] = torch.stack([a.cos(), a.sin()], -1).float()
    return out


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    B, H, L = case["B"], case["H"], case["L"]
    st = {"case": dict(case), "cache": _cache(case, gen)}
    if case["op"] == "write":
        T, start = case["T"], _starts(case)
        st["start"] = _i32(start)
        # a touch larger than the prefix in places, so some scales rise
        st["k"] = (rand(B, T, H, D) * 1.2).bfloat16()
        st["v"] = (rand(B, T, H, D) * 1.1).bfloat16()
        st["positions"] = _i32([[s + t for t in range(T)] for s in start]) \
            if B * T < 4096 else (
                st["start"][:, None]
                + torch.arange(T, dtype=torch.int32, device="cuda"))
        st["table"] = _table(L)
        st["back"] = st["start"] - (BLK - 1)
        return st
    if case["op"] == "read":
        room = L - case["T"]
        st["start"] = _i32([(room * 3 // 7 + b * 101) % (room + 1)
                            for b in range(B)])
        return st
    s, n = _ranges(case)
    st["q"] = rand(B, H * case["G"], D).bfloat16()
    st["kv_start"], st["kv_len"] = _i32(s), _i32(n)
    st["q_pos"] = _i32([b - a - 1 for a, b in zip(s, n)])
    st["table"] = _table(L)
    if case["op"] == "sparse":
        K, nblk = case["K"], -(-L // BLK)
        # K distinct blocks in ascending order among the visible ones of
        # each row (fewer where fewer are visible: -1 at the end)
        first, last = st["kv_start"] // BLK, (st["kv_len"] - 1) // BLK
        j = torch.arange(nblk, device="cuda")
        seen = (j >= first[:, None]) & (j <= last[:, None])
        key = torch.rand((B, H, nblk), generator=gen, device="cuda")
        key = torch.where(seen[:, None], key, 2.0)
        pick = key.argsort(-1)[..., :K]
        pick = torch.where(key.gather(-1, pick) < 1.5, pick, nblk)
        pick = pick.sort(-1).values
        st["blocks"] = torch.where(pick < nblk, pick, -1).to(torch.int32)
    return st


# ------------------------------------------------------------ plain forms
def _rotate(x, cs, layout):
    """R(pos) x in fp32; cs [..., D/2, 2] broadcast against x's heads. Every
    product and sum is rounded on its own."""
    c, s = cs[..., 0], cs[..., 1]
    if layout == "half":
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * c - b * s, a * s + b * c], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)


def _plain_write_one(x, codes, scale, bounds, start, n_blocks, kind):
    """x [B, T, H, D] fp32 (rotated already) into codes [B, H, L, D]."""
    B, T, H, _ = x.shape
    L = codes.shape[2]
    dev = x.device
    start = start.long()
    slot = (start // BLK * BLK)[:, None] + torch.arange(n_blocks * BLK,
                                                        device=dev)  # [B, S]
    t = slot - start[:, None]
    new = (t >= 0) & (t < T) & (slot < L)
    old = (t < 0)
    rows = torch.arange(B, device=dev)[:, None]
    xs = x[rows, t.clamp(0, T - 1)].transpose(1, 2)        # [B, H, S, D]
    at = slot.clamp(0, L - 1)
    had = codes.transpose(1, 2)[rows, at].transpose(1, 2).float()
    split = lambda y: y.reshape(B, H, n_blocks, BLK, D)    # noqa: E731
    newm = new[:, None, :, None]
    amax = split(torch.where(newm, xs.abs(), 0.0)).amax((-2, -1))
    blk = (start // BLK)[:, None] + torch.arange(n_blocks, device=dev)
    nblk = scale.shape[2]
    held = scale.transpose(1, 2)[rows, blk.clamp(0, nblk - 1)].transpose(1, 2)
    has_old = (old.view(B, n_blocks, BLK).any(-1))[:, None]
    s_old = torch.where(has_old, held, 0.0)
    s = torch.maximum(s_old, amax * RQMAX[kind])
    s = torch.where(s < TINY, 0.0, s)
    inv = torch.where(s > 0, 1.0 / s, 0.0)[..., None, None]
    ratio = torch.where(s > 0, s_old / s, 0.0)[..., None, None]
    c_new = _encode(split(xs) * inv, kind).float()
    c_old = split(had)
    c_old = torch.where(ratio == 1.0, c_old,
                        _encode(c_old * ratio, kind).float())
    keep_new = split(newm.expand(B, H, n_blocks * BLK, D))
    keep_old = split(old[:, None, :, None].expand(B, H, n_blocks * BLK, D))
    c = torch.where(keep_new, c_new, c_old)
    # write back the slots of old and new tokens of touched blocks
    touched = new.view(B, n_blocks, BLK).any(-1)
    on = ((new | old) & touched[..., None].expand(B, n_blocks, BLK)
          .reshape(B, -1))
    bi, si = on.nonzero(as_tuple=True)
    codes[bi, :, slot[bi, si]] = c.view(B, H, n_blocks * BLK, D)[
        bi, :, si].to(codes.dtype)
    bi, ji = touched.nonzero(as_tuple=True)
    scale[bi, :, blk[bi, ji]] = s[bi, :, ji]
    if bounds is not None:
        # a block that grew is summarised anew, else the older tokens'
        # bounds are kept and widened
        grew = (s > s_old)[..., None, None]
        live = keep_new | (keep_old & grew)
        u = UNIT[kind]
        lo = torch.where(live, c, math.inf).amin(-2)
        hi = torch.where(live, c, -math.inf).amax(-2)
        bb = torch.stack([torch.floor(lo * u), torch.ceil(hi * u)],
                         -2).clamp(-127, 127)
        was = bounds.transpose(1, 2)[rows, blk.clamp(0, nblk - 1)] \
            .transpose(1, 2).float()
        both = torch.stack([torch.minimum(bb[..., 0, :], was[..., 0, :]),
                            torch.maximum(bb[..., 1, :], was[..., 1, :])], -2)
        bb = torch.where(has_old[..., None, None] & ~grew, both, bb)
        bounds[bi, :, blk[bi, ji]] = bb[bi, :, ji].to(torch.int8)


def _plain_read(codes, scale, start, T):
    """bf16 [B, T, H, D] of slots start[b] + t; zeros outside the cache."""
    B, H, L, _ = codes.shape
    slot = start.long()[:, None] + torch.arange(T, device=codes.device)
    rows = torch.arange(B, device=codes.device)[:, None]
    at = slot.clamp(0, L - 1)
    x = codes.transpose(1, 2)[rows, at].float()
    x = x * scale.transpose(1, 2)[rows, at // BLK][..., None]
    inside = (slot >= 0) & (slot < L)
    return torch.where(inside[..., None, None], x, 0.0).bfloat16()


def _plain_query(st, x):
    """Rotated queries [B, H, G, D] in the type of x."""
    c = st["case"]
    cs = st["table"][st["q_pos"].long()][:, None].to(x.dtype)
    r = _rotate(x, cs, c["layout"])
    return r.view(c["B"], c["H"], c["G"], D)


def _plain_attend(qr, k, v, ks, vs, seen):
    """qr [B, H, G, D]; codes [B, H, S, D]; scales [B, H, S]; seen [B, *, S]."""
    x = k.float()
    x *= ks[..., None]
    s = qr @ x.transpose(-1, -2) / math.sqrt(D)
    del x
    s = torch.where(seen[:, :, None], s, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    x = v.float()
    x *= vs[..., None]
    o = p @ x
    out = torch.where(total > 0, o / total, 0.0)
    lse = (m + torch.log(total))[..., 0]
    B, H, G, _ = qr.shape
    return {"out": out.bfloat16().view(B, H * G, D), "lse": lse.view(B, H * G)}


def _plain_decode(st):
    c = st["case"]
    k, v, ks, vs, _ = st["cache"]
    j = torch.arange(c["L"], device=k.device)
    seen = (j >= st["kv_start"][:, None]) & (j < st["kv_len"][:, None])
    return _plain_attend(_plain_query(st, st["q"].float()), k, v, ks[..., j // BLK],
                         vs[..., j // BLK], seen[:, None])


def _plain_sparse(st):
    c = st["case"]
    k, v, ks, vs, _ = st["cache"]
    blocks = st["blocks"].long()
    B, H, K = blocks.shape
    slot = (blocks[..., None] * BLK
            + torch.arange(BLK, device=k.device)).reshape(B, H, K * BLK)
    seen = (slot >= st["kv_start"][:, None, None]) & \
        (slot < st["kv_len"][:, None, None]) & (slot >= 0)
    at = slot.clamp(0, c["L"] - 1)
    bi = torch.arange(B, device=k.device)[:, None, None]
    hi = torch.arange(H, device=k.device)[:, None]
    return _plain_attend(_plain_query(st, st["q"].float()), k[bi, hi, at], v[bi, hi, at],
                         ks[bi, hi, at // BLK], vs[bi, hi, at // BLK], seen)


def _plain_select(st):
    """Blocks [B, H, K] int32, ascending, -1 behind the last, and their
    scores. The query's codes are rounded from 64 bits, and the score of
    whole numbers and scales is too: a list hangs on either."""
    c = st["case"]
    _, _, ks, _, kb = st["cache"]
    K = c["K"]
    n = ks.shape[2]
    qr = _plain_query(st, st["q"].double())
    amax = qr.abs().amax(-1, keepdim=True)
    qi = torch.where(amax > 0, torch.round(
        qr * (torch.full_like(amax, 127.0) / amax)), 0.0).float()
    # whole numbers below 2^24: the sums are exact in fp32
    dots = qi.clamp(min=0) @ kb[..., 1, :].float().transpose(-1, -2) + \
        qi.clamp(max=0) @ kb[..., 0, :].float().transpose(-1, -2)
    score = dots.double() * ks[:, :, None].double() * (amax * (1.0 / 127.0))
    score = score.float().amax(2)                          # [B, H, n]
    first = (st["kv_start"] // BLK)[:, None]
    last = ((st["kv_len"] - 1) // BLK)[:, None]
    j = torch.arange(n, device=ks.device)
    seen = ((j >= first) & (j <= last))[:, None]
    kept = ((j == first) | (j == last))[:, None]
    rank = torch.where(kept, math.inf, score)
    rank = torch.where(seen, rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    order = order[..., :K]
    order = torch.where(rank.gather(-1, order) > -math.inf, order, n)
    order = order.sort(-1).values
    took = order < n
    score = score.gather(-1, order.clamp(max=n - 1))
    return {"blocks": torch.where(took, order, -1).to(torch.int32),
            "scores": torch.where(took, score, -math.inf)}


def _plain_write(st):
    c = st["case"]
    k, v, ks, vs, kb = st["cache"]
    T = c["T"]
    n_blocks = (T + BLK - 1) // BLK + 1
    cs = st["table"][st["positions"].long()][:, :, None]
    kr = _rotate(st["k"].float(), cs, c["layout"])
    _plain_write_one(kr, k, ks, kb, st["start"], n_blocks, c["kind"])
    _plain_write_one(st["v"].float(), v, vs, None, st["start"], n_blocks,
                     c["kind"])
    return {"k": _plain_read(k, ks, st["back"], T + BLK - 1),
            "v": _plain_read(v, vs, st["back"], T + BLK - 1),
            "k_scale": ks, "v_scale": vs, "k_bounds": kb}


def run(state):
    op, c = state["case"]["op"], state["case"]
    if not own:
        if op == "write":
            return _plain_write(state)
        if op == "read":
            k, v, ks, vs, _ = state["cache"]
            return {"k": _plain_read(k, ks, state["start"], c["T"]),
                    "v": _plain_read(v, vs, state["start"], c["T"])}
        if op == "select":
            return _plain_select(state)
        return _plain_decode(state) if op == "decode" else \
            _plain_sparse(state)
    from long_context_blockwise_causal_b200 import ops
    cache = ops.Kv8Cache(*state["cache"])
    if op == "write":
        ops.kv8_write(cache, state["k"], state["v"], state["positions"],
                      state["start"], state["table"], rope_layout=c["layout"])
        k, v = ops.kv8_read(cache, state["back"], c["T"] + BLK - 1)
        return {"k": k, "v": v, "k_scale": cache.k_scale,
                "v_scale": cache.v_scale, "k_bounds": cache.k_bounds}
    if op == "read":
        k, v = ops.kv8_read(cache, state["start"], c["T"])
        return {"k": k, "v": v}
    if op == "select":
        blocks, scores = ops.kv8_select(
            state["q"], cache, state["kv_start"], state["kv_len"],
            state["q_pos"], state["table"], c["K"], rope_layout=c["layout"])
        return {"blocks": blocks, "scores": scores}
    out, lse = ops.kv8_decode(
        state["q"], cache, state["kv_start"], state["kv_len"],
        state["q_pos"], state["table"], blocks=state.get("blocks"),
        rope_layout=c["layout"])
    return {"out": out, "lse": lse}


# ----------------------------------------------------------------- work
def work(case):
    B, H, L = case["B"], case["H"], case["L"]
    if case["op"] == "write":
        T, back = case["T"], case["T"] + BLK - 1
        tok = B * H * D
        # bf16 k, v in, codes out; then the codes read and bf16 k, v out
        return {"bytes": tok * T * (4 + 2) + tok * back * (2 + 4)
                + B * T * D * 4,
                "flops": tok * T * 12 + tok * back * 2}
    if case["op"] == "read":
        n = B * H * case["T"] * D
        return {"bytes": n * (2 + 4), "flops": n * 2}
    s, n = _ranges(case)
    q = B * H * case["G"]
    io = q * D * 2 + B * D * 4
    if case["op"] == "select":
        blocks = sum((b + BLK - 1) // BLK - a // BLK for a, b in zip(s, n))
        return {"bytes": H * blocks * (2 * D + 4) + io + B * H * case["K"] * 8,
                "flops": 4 * D * H * case["G"] * blocks}
    if case["op"] == "decode":
        tokens = H * sum(b - a for a, b in zip(s, n))
    else:
        seen = [min(case["K"] * BLK, b - a) for a, b in zip(s, n)]
        tokens = H * sum(seen)
    return {"bytes": tokens * 2 * D + tokens // BLK * 8 + io
            + q * (D * 2 + 4), "flops": 4 * D * tokens * case["G"]}


# ---------------------------------------------------- the definition, fp64
def _turn(x, pos, layout):
    """RoPE from its angles, fp64: x [..., D], pos broadcastable to x[..., 0]."""
    f = torch.pow(torch.tensor(THETA, dtype=torch.float64, device=x.device),
                  torch.arange(0, D, 2, dtype=torch.float64,
                               device=x.device) / -D)
    w = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                    pos.double()[..., None] * f)
    pair = x.unflatten(-1, (2, D // 2)).transpose(-1, -2) \
        if layout == "half" else x.unflatten(-1, (D // 2, 2))
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * w)
    return (z.transpose(-1, -2) if layout == "half" else z).flatten(-2)


def _exact_attend(st, rows_of):
    c = st["case"]
    B, H, G = c["B"], c["H"], c["G"]
    k, v, ks, vs, _ = st["cache"]
    out = torch.zeros((B, H, G, D), dtype=torch.float64, device=k.device)
    lse = torch.full((B, H, G), -math.inf, dtype=torch.float64,
                     device=k.device)
    q = _turn(st["q"].double().view(B, H, G, D),
              st["q_pos"][:, None, None].expand(B, H, G), c["layout"])
    for b in range(B):
        for h in range(H):
            at = rows_of(b, h)
            if at.numel() == 0:
                continue
            s = ks[b, h].double()[at // BLK] * (
                k[b, h, at].double() @ q[b, h].T / math.sqrt(D)).T
            lse[b, h] = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[b, h, :, None])
            out[b, h] = (p * vs[b, h].double()[at // BLK]) @ \
                v[b, h, at].double()
    return {"out": out.view(B, H * G, D), "lse": lse.view(B, H * G)}


def _exact_select(st):
    """Scores of the K best blocks of each (row, head), one head at a time:
    the largest of qi . lo and qi . hi channel by channel, summed."""
    c = st["case"]
    B, H, G, K = c["B"], c["H"], c["G"], c["K"]
    _, _, ks, _, kb = st["cache"]
    s, n = st["kv_start"].tolist(), st["kv_len"].tolist()
    cs = torch.view_as_complex(st["table"][st["q_pos"].long()].double())
    q = st["q"].double().view(B, H, G, D)
    pair = q.unflatten(-1, (2, D // 2)).transpose(-1, -2) \
        if c["layout"] == "half" else q.unflatten(-1, (D // 2, 2))
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous())
                           * cs[:, None, None])
    q = (z.transpose(-1, -2) if c["layout"] == "half" else z).flatten(-2)
    out = torch.full((B, H, K), -math.inf, dtype=torch.float64,
                     device=q.device)
    for b in range(B):
        j0, j1 = s[b] // BLK, (n[b] - 1) // BLK + 1
        for h in range(H):
            best = None
            lo, hi = kb[b, h, j0:j1].double().unbind(1)
            for g in range(G):
                unit = q[b, h, g].abs().max() / 127.0
                code = torch.round(q[b, h, g] / unit) if unit > 0 else \
                    torch.zeros_like(q[b, h, g])
                one = torch.maximum(code * lo, code * hi).sum(-1) \
                    * ks[b, h, j0:j1].double() * unit
                best = one if best is None else torch.maximum(best, one)
            rank = best.float().tolist()      # the ranking is of fp32 scores
            rank[0] = rank[-1] = math.inf
            took = sorted(sorted(range(j1 - j0),
                                 key=lambda i: (-rank[i], i))[:K])
            out[b, h, :len(took)] = best[torch.tensor(took, device=q.device)]
    return {"blocks": None, "scores": out}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "select":
        return _exact_select(st)
    k, v, ks, vs, _ = st["cache"]
    B, H, L, _ = k.shape
    if case["op"] in ("decode", "sparse"):
        s, n = st["kv_start"].tolist(), st["kv_len"].tolist()

        def rows_of(b, h):
            if case["op"] == "decode":
                return torch.arange(s[b], n[b], device=k.device)
            j = st["blocks"][b, h].long()
            at = (j[j >= 0, None] * BLK
                  + torch.arange(BLK, device=k.device)).flatten()
            return at[(at >= s[b]) & (at < n[b])]
        return _exact_attend(st, rows_of)
    T = case["T"]
    if case["op"] == "read":
        at = [torch.arange(a, a + T, device=k.device)
              for a in st["start"].tolist()]
        val = lambda x, s: torch.stack([                     # noqa: E731
            (x[b][:, at[b]].double() * s[b].double()[:, at[b] // BLK, None])
            .transpose(0, 1) for b in range(B)])
        return {"k": val(k, ks), "v": val(v, vs)}
    # write: row by row, block by block of the touched range
    res = {"k_bounds": None}
    x = {"k": _turn(st["k"].double(), st["positions"][:, :, None],
                    case["layout"]), "v": st["v"].double()}
    q = QMAX[case["kind"]]
    for name, codes, scale in (("k", k, ks), ("v", v, vs)):
        scale = scale.double()
        span = torch.zeros((B, T + BLK - 1, H, D), dtype=torch.float64,
                           device=k.device)
        for b, a in enumerate(st["start"].tolist()):
            lo, j0 = a - (BLK - 1), a // BLK
            j1 = (a + T - 1) // BLK + 1
            # the blocks j0 .. j1 - 1 as [H, j1 - j0, BLK, D]
            new = torch.zeros((H, (j1 - j0) * BLK, D), dtype=torch.float64,
                              device=k.device)
            new[:, a - j0 * BLK:a - j0 * BLK + T] = x[name][b].transpose(0, 1)
            s = new.view(H, j1 - j0, -1).abs().amax(-1) / q
            if a % BLK:
                s[:, 0] = torch.maximum(s[:, 0], scale[b, :, j0])
            old = codes[b, :, j0 * BLK:a].double() * \
                scale[b, :, j0, None, None]
            new[:, :a - j0 * BLK] = old
            y = new.view(H, j1 - j0, BLK, D) / s[..., None, None]
            y = (_encode(y, case["kind"]).double()
                 * s[..., None, None]).view(H, -1, D)
            if lo < j0 * BLK:                # tokens of the block before
                e = max(lo, 0)
                prev = codes[b, :, e:j0 * BLK].double()
                if prev.shape[1]:
                    prev = prev * scale[b, :, j0 - 1, None, None]
                    span[b, e - lo:j0 * BLK - lo] = prev.transpose(0, 1)
            f = max(lo, j0 * BLK)
            span[b, f - lo:] = y[:, f - j0 * BLK:a + T - j0 * BLK] \
                .transpose(0, 1)
            scale[b, :, j0:j1] = s
        res[name], res[name + "_scale"] = span, scale
    return res
