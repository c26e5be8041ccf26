"""The 8-bit KV cache in fp64 (oracle; test infrastructure only).

Readings taken here (the pages have no 8-bit cache): a block is 128
consecutive slots of one (row, head); a code c stands for c * scale; the
codes are OCP e4m3 (largest 448, smallest step 2^-9) or integers in
[-127, 127], rounded to nearest even; a block's scale is the largest
magnitude it has met, divided by the largest code.
"""

import numpy as np

from .rope import rope_rotate, rope_rotate_half

KV8_BLOCK = 128
KV8_QMAX = {"e4m3": 448.0, "int8": 127.0}


def kv8_half_step(y, kind):
    """Half the distance between neighbouring codes around y."""
    y = np.abs(np.asarray(y, dtype=np.float64))
    if kind == "int8":
        return np.full_like(y, 0.5)
    _, e = np.frexp(np.maximum(y, 2.0 ** -6))     # y in [2^(e-1), 2^e)
    return np.ldexp(1.0, e - 1 - 3) / 2


def kv8_encode(y, kind):
    """The code values nearest to y (ties to even), saturating."""
    y = np.asarray(y, dtype=np.float64)
    step = 2 * kv8_half_step(y, kind)
    q = KV8_QMAX[kind]
    return np.clip(np.round(y / step) * step, -q, q)


def kv8_rotate(x, positions, theta, layout):
    """R(pos) x for x [T, D] or [T, H, D] with positions [T]."""
    rot = rope_rotate_half if layout == "half" else rope_rotate
    x = np.asarray(x, dtype=np.float64)
    if x.ndim == 2:
        return rot(x, positions, theta)
    return np.stack([rot(x[:, h], positions, theta)
                     for h in range(x.shape[1])], 1)


def kv8_block_scale(x_new, s_old, kind):
    """Scale of a block that meets x_new; s_old: of its older tokens or 0."""
    return max(float(s_old), float(np.abs(x_new).max()) / KV8_QMAX[kind])


def kv8_attend(q_rot, k, v, ks, vs, slots):
    """One rotated query [D] against code values k, v [L, D] at `slots` (a
    list of slot indices, repeats count), with per-block scales ks, vs.
    Returns (out [D], lse, sum of p |v| per channel)."""
    slots = np.asarray(slots, dtype=np.int64)
    d = k.shape[1]
    if slots.size == 0:
        return np.zeros(d), -np.inf, np.zeros(d)
    kk = k[slots] * ks[slots // KV8_BLOCK, None]
    vv = v[slots] * vs[slots // KV8_BLOCK, None]
    s = kk @ np.asarray(q_rot, dtype=np.float64) / np.sqrt(d)
    m = s.max()
    p = np.exp(s - m)
    z = p.sum()
    return p @ vv / z, m + np.log(z), p @ np.abs(vv) / z


def kv8_block_scores(q_rot, bounds, ks):
    """fp32 scores of blocks with bounds [n, 2, D] and scales ks [n] for the
    rotated queries q_rot [G, D] that share them (fp64)."""
    best = None
    for x in np.asarray(q_rot, dtype=np.float64):
        a = np.abs(x).max()
        qi = np.round(x * (127.0 / a)) if a > 0 else np.zeros_like(x)
        dot = np.maximum(qi * bounds[:, 0].astype(np.float64),
                         qi * bounds[:, 1].astype(np.float64)).sum(-1)
        s = (dot * ks.astype(np.float64) * (a * (1.0 / 127.0))) \
            .astype(np.float32)
        best = s if best is None else np.maximum(best, s)   # keeps a NaN
    return best


def kv8_pick(scores, first, last, n_select, n_sink, n_recent):
    """Blocks of [first, last) by score: forced ones, NaN, then the best,
    ties to the lowest index; ascending."""
    def rank(j):
        if j - first < n_sink or last - 1 - j < n_recent:
            return (0, 0.0, j)
        s = scores[j]
        return (1, 0.0, j) if np.isnan(s) else (2, -float(s), j)
    return sorted(sorted(range(first, last), key=rank)[:n_select])
