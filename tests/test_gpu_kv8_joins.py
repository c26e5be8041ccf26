"""Decode over the 8-bit cache where parts are joined, NaN in and beside the
visible slots for every way the query heads are grouped, and inputs written on
the stream just before the calls (needs a B200). Tolerances and helpers:
test_gpu_kv8.py."""

import numpy as np
import pytest
import torch

from long_context_blockwise_causal_b200 import ops
from test_gpu_kv8 import KINDS, check_decode, filled, i32, queries, tokens

pytestmark = pytest.mark.gpu

THETA = 1e6
GROUPS = [1, 2, 5, 8, 12, 16]


def ragged(B, L, seed):
    """Rows of every kind: empty ones, one slot, part of a block, all."""
    rng = np.random.default_rng(seed)
    n = rng.integers(0, L + 1, B)
    s = (n * rng.random(B) * 1.1).astype(int)
    for b, length in enumerate((L, 1, 0)[:B]):
        n[b], s[b] = length, 0
    return s.tolist(), n.tolist()


# more (row, cache head) pairs than CTAs: the cut ones are joined, a warp per
# query head, in two turns above 8
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G", GROUPS[1:])
def test_cut_pairs_of_grouped_heads(cuda_dev, kind, G):
    B, H, L = 80, 4, 420
    c = filled(B, L, H, kind, seed=40)
    q, pos, table = queries(B, H * G, L, 41)
    s, n = ragged(B, L, 42)
    check_decode(c, q, pos, table, s, n, "half" if G % 2 else "interleaved")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G", [1, 4, 16])
def test_cut_pairs_of_lists(cuda_dev, kind, G):
    B, H, L, K = 80, 4, 1100, 4
    c = filled(B, L, H, kind, seed=43)
    q, pos, table = queries(B, H * G, L, 44)
    s, n = ragged(B, L, 45)
    rng = np.random.default_rng(46)
    bl = np.full((B, H, K), -1)
    for b in range(B):
        for h in range(H):
            m = rng.integers(0, K + 1)       # short and empty lists too
            bl[b, h, :m] = np.sort(rng.choice(9, m, replace=False))
    check_decode(c, q, pos, table, s, n, "interleaved", blocks=i32(bl))


# B, H: a few pairs cut over many CTAs, and more pairs than CTAs
@pytest.mark.parametrize("B,H", [(2, 2), (80, 4)])
@pytest.mark.parametrize("G", GROUPS)
@pytest.mark.parametrize("kind", KINDS)
def test_unseen_slots_hold_anything(cuda_dev, kind, G, B, H):
    L = 700
    c = filled(B, L, H, kind, seed=50)
    q, pos, table = queries(B, H * G, L, 51)
    s = [(200, 0, 128, 37)[b % 4] for b in range(B)]
    n = [(430, 129, 256, 41)[b % 4] for b in range(B)]
    call = lambda **kw: ops.kv8_decode(q, c, i32(s), i32(n), pos, table,
                                       rope_layout="half", **kw)
    bl = i32(np.broadcast_to(np.arange(6), (B, H, 6)).copy())
    want = [*call(), *call(blocks=bl)]
    assert all(torch.isfinite(x.float()).all() for x in want)
    for b in range(B):
        for lo, hi in ((0, s[b]), (n[b], L)):
            if kind == "e4m3":                  # NaN codes
                c.k.view(torch.uint8)[b, :, lo:hi] = 0x7F
                c.v.view(torch.uint8)[b, :, lo:hi] = 0xFF
            else:
                c.k[b, :, lo:hi] = -128
                c.v[b, :, lo:hi] = 127
        for j in range(c.k_scale.shape[-1]):
            if j * 128 + 128 <= s[b] or j * 128 >= n[b]:
                c.k_scale[b, :, j] = float("nan")
                c.v_scale[b, :, j] = float("inf")
    got = [*call(), *call(blocks=bl)]
    torch.cuda.synchronize()
    assert ops.last_status() == ops.OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("B,H", [(2, 2), (80, 4)])
@pytest.mark.parametrize("G", GROUPS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("which", ["k_scale", "v_scale", "q"])
def test_visible_nan_stays_with_its_heads(cuda_dev, which, kind, G, B, H):
    L = 600
    c = filled(B, L, H, kind, seed=52)
    q, pos, table = queries(B, H * G, L, 53)
    s, n = i32([0] * B), i32([L - b % 70 for b in range(B)])
    call = lambda: ops.kv8_decode(q, c, s, n, pos, table)
    clean, clean_lse = call()
    row = B - 1
    hit = torch.zeros((B, H * G), dtype=torch.bool, device="cuda")
    if which == "q":
        q[row, H * G - 1, 5] = float("nan")
        hit[row, H * G - 1] = True
    else:
        getattr(c, which)[row, 1, 2] = float("nan")
        hit[row, G:2 * G] = True
    out, lse = call()
    torch.cuda.synchronize()
    assert torch.isnan(out[hit]).all()
    assert torch.equal(out[~hit], clean[~hit])
    assert torch.equal(lse[~hit], clean_lse[~hit])
    if which == "v_scale":          # the weights do not see the values
        assert torch.equal(lse, clean_lse)
    else:
        assert torch.isnan(lse[hit]).all()


@pytest.mark.parametrize("B,H,G,L", [(2, 4, 2, 5000), (1, 2, 16, 3000),
                                     (90, 4, 2, 500)])
def test_calls_see_inputs_written_just_before_them(cuda_dev, B, H, G, L):
    """Lengths, starts, lists, tokens and scales rewritten on the stream by a
    torch kernel right before each call, and results read right after it, give
    what calls on settled inputs give. (The join reads the rows' lengths while
    the kernel before it still runs.)"""
    q, pos, table = queries(B, H * G, L, 60)
    k, v = tokens(B, 1, H, 61)
    steps = []
    for i in range(6):
        s, n = ragged(B, L - 1, 62 + i)
        steps.append((i32(s), i32(n), 1.0 + 0.25 * i))
    n_blocks = 4

    def run(settle):
        wait = torch.cuda.synchronize if settle else lambda: None
        c = filled(B, L, H, "e4m3", seed=63)
        scale = c.k_scale.clone()
        start, length = i32([0] * B), i32([L] * B)
        token = torch.empty_like(k)
        res = []
        torch.cuda.synchronize()
        for s, n, f in steps:
            start.copy_(s)
            length.copy_(n)
            torch.mul(k, f, out=token)
            torch.mul(scale, f, out=c.k_scale)
            wait()
            ops.kv8_write(c, token, v, pos[:, None].contiguous(), length,
                          table)
            length.add_(1)
            wait()
            bl, sc = ops.kv8_select(q, c, start, length, pos, table,
                                    n_blocks, 1, 1)
            wait()
            one = ops.kv8_decode(q, c, start, length, pos, table, blocks=bl)
            wait()
            bl2 = torch.where(bl >= 0, bl, -1)
            bl2[:, :, 0] = -1
            wait()
            two = ops.kv8_decode(q, c, start, length, pos, table, blocks=bl2)
            length.sub_(1)                   # another range, at once
            wait()
            all_ = ops.kv8_decode(q, c, start, length, pos, table)
            start.zero_()
            length.fill_(L)
            wait()
            back = ops.kv8_read(c, start, 200, kv_len=length)
            res += [bl, sc, *one, *two, *all_, *back]
            res += [x.float().sum() for x in (one[0], all_[0], back[0])]
        torch.cuda.synchronize()
        assert ops.last_status() == ops.OK
        return res + [c.k.view(torch.uint8), c.k_scale, c.k_bounds]

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)
