"""The 8-bit KV cache against the fp64 oracle (needs a B200).

Tolerances, from the roundings that the calls make (bf16 is off by at most
2^-8 of a value, fp32 by 2^-24):

* a code may be either neighbour of a tie: |code - x / s| is at most half a
  step, plus the fp32 error of x / s. The rotation rounds cos, sin, two
  products and a sum, at most 2^-22 of the pair's length, which is at most
  sqrt(2) Q in codes; 1 / s and the product with it add 2^-23 of the code.
* scores: the query is rounded to 2^-20 of each channel (int8: 2^-22 of the
  largest) and rotated with 2^-22, products are exact and sums fp32, so a
  score is off by at most DS = 2^-18 sum (|q_d| + max|q| / 16) |k_d| /
  sqrt(D); weights are then off by 2 DS and by the 2^-12 to which they enter
  the second product.
* a weight below 2^-13 of the largest one of its block enters the second
  product as a multiple of a fixed fraction of that one: int8 codes hold
  p 127 in three parts 1/254 apart, a last step of 1 / (127 254^2) < 2^-22.9
  and half of it at most 2^-23.9; e4m3 codes hold p 256 in three parts 1/16
  apart with a smallest step of 2^-9, 2^-9 / 256 / 256 = 2^-25 and half of
  it 2^-26. So each value may be off by 2^-23 |v_t| times the largest weight
  of its block, whatever its own weight is.
"""

import numpy as np
import pytest
import torch

import oracle
from long_context_blockwise_causal_b200 import ops
from long_context_blockwise_causal_b200 import workloads as wl

pytestmark = pytest.mark.gpu

THETA = 1e6
DT = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
KINDS = ["e4m3", "int8"]
LAYOUTS = ["interleaved", "half"]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def val(t):
    """Tensor -> fp64 numpy (codes as the numbers they are)."""
    return t.float().cpu().numpy().astype(np.float64)


def snap(cache):
    return [val(x) for x in cache]


def filled(B, L, H, kind, seed=0, scale=1.0):
    """A cache with every slot holding N(0, 1) keys and values."""
    c = ops.kv8_cache(B, L, H, dtype=DT[kind])
    n = -(-L // 128)
    k = wl.random_tensor((B, n * 128, H, 128), seed * 16 + 2, scale,
                         torch.float32, "cuda").transpose(1, 2)
    v = wl.random_tensor((B, n * 128, H, 128), seed * 16 + 3, 1.0,
                         torch.float32, "cuda").transpose(1, 2)
    q = oracle.KV8_QMAX[kind]
    for x, codes, sc in ((k, c.k, c.k_scale), (v, c.v, c.v_scale)):
        x = x.reshape(B, H, n, 128, 128)
        s = x.abs().amax((-2, -1)) / q
        y = x / s[..., None, None]
        y = y.round() if kind == "int8" else y.clamp(-q, q)
        codes.copy_(y.reshape(B, H, n * 128, 128)[:, :, :L].to(DT[kind]))
        sc.copy_(s)
        if codes is c.k:
            live = y.to(DT[kind]).float()
            live = torch.where((torch.arange(n * 128, device="cuda") < L)
                               .view(n, 128, 1), live, live[..., :1, :])
            u = 127.0 / q
            c.k_bounds[..., 0, :] = (live.amin(-2) * u).floor().clamp(
                -127, 127).to(torch.int8)
            c.k_bounds[..., 1, :] = (live.amax(-2) * u).ceil().clamp(
                -127, 127).to(torch.int8)
    return c


def tokens(B, T, H, seed, scale=1.0):
    d = lambda k: wl.random_tensor((B, T, H, 128), seed * 16 + k, scale,
                                   torch.bfloat16, "cuda")
    return d(5), d(6)


def check_write(c, kind, layout, T, start, n_new=None, seed=3, scale=1.0):
    """One write against the definition, block by block; what lies outside
    keeps its bits. Returns the fp64 views after it."""
    B, H, L, D = c.k.shape
    k, v = tokens(B, T, H, seed, scale)
    max_pos = 5000
    pos = torch.randint(0, max_pos, (B, T), dtype=torch.int32, device="cuda",
                        generator=torch.Generator("cuda").manual_seed(seed))
    table = ops.rope_table(THETA, max_pos)
    before = snap(c)
    ops.kv8_write(c, k, v, pos, i32(start), table,
                  n_new=None if n_new is None else i32(n_new),
                  rope_layout=layout)
    torch.cuda.synchronize()
    assert ops.last_status() == ops.OK
    after = snap(c)
    q = oracle.KV8_QMAX[kind]
    kb0, kb1 = before[4], after[4]
    kn, vn, pn = val(k), val(v), pos.cpu().numpy()
    for b in range(B):
        m = T if n_new is None else max(0, min(n_new[b], T))
        lo, hi = max(start[b], 0), min(start[b] + m, L)
        xk = oracle.kv8_rotate(kn[b], pn[b], THETA, layout)
        for which, x in ((0, xk), (1, vn[b])):
            c0, c1 = before[which][b], after[which][b]
            s0, s1 = before[2 + which][b], after[2 + which][b]
            seen = set()
            for j in range(lo // 128, (hi - 1) // 128 + 1 if hi > lo else 0):
                seen.add(j)
                a, z = max(lo, j * 128), min(hi, j * 128 + 128)
                for h in range(H):
                    new = x[a - start[b]:z - start[b], h]
                    old = c0[h, j * 128:a]
                    s_old = s0[h, j] if len(old) else 0.0
                    want = oracle.kv8_block_scale(new, s_old, kind)
                    s = s1[h, j]
                    assert abs(s - want) <= 2 ** -21 * want
                    y = new / s if s else np.zeros_like(new)
                    tol = oracle.kv8_half_step(y, kind) + \
                        2 ** -22 * (1.5 * q + np.abs(y))
                    assert (np.abs(c1[h, a:z] - y) <= tol).all()
                    if s == s_old:
                        assert np.array_equal(c1[h, j * 128:a], old)
                    else:
                        y = old * s_old / s if s else old * 0
                        tol = oracle.kv8_half_step(y, kind) + 2 ** -22 * q
                        assert (np.abs(c1[h, j * 128:a] - y) <= tol).all()
                    # slots behind the last new one keep their bits
                    assert np.array_equal(c1[h, z:j * 128 + 128],
                                          c0[h, z:j * 128 + 128])
                    if which == 0:
                        u = np.float32(127.0 / q)
                        live = c1[h, a:z] if len(old) and s == s_old else \
                            c1[h, j * 128:z]
                        f = live.astype(np.float32)
                        bl = np.clip(np.floor(f.min(0) * u), -127, 127)
                        bh = np.clip(np.ceil(f.max(0) * u), -127, 127)
                        if len(old) and s == s_old:
                            bl = np.minimum(bl, kb0[b, h, j, 0])
                            bh = np.maximum(bh, kb0[b, h, j, 1])
                        assert np.array_equal(kb1[b, h, j, 0], bl)
                        assert np.array_equal(kb1[b, h, j, 1], bh)
            for j in range(s0.shape[1]):            # untouched blocks
                if j not in seen:
                    sl = slice(j * 128, j * 128 + 128)
                    assert np.array_equal(c1[:, sl], c0[:, sl])
                    assert np.array_equal(s1[:, j], s0[:, j])
                    if which == 0:
                        assert np.array_equal(kb1[b, :, j], kb0[b, :, j])
    return after


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("L,T,start,n_new", [
    (256, 1, [0, 1, 127, 128, 255], None),
    (300, 1, [299, 300, -1, 200, 64], None),         # ragged last block
    (700, 300, [77, 0, 401, 690, -40], None),
    (515, 130, [0, 126, 3, 380, 500], [130, 0, 1, 77, 500]),
    (300, 12, [120, 0, 117, 290, -9], [12, 3, 12, 12, 12]),
    (300, 13, [120, 0, 116, 290, -9], [13, 1, 13, 12, 13]),
    (2000, 900, [1000, 5, 640, 1100, 127], [900, 899, 256, 900, -3]),
])
def test_write_matches_the_definition(cuda_dev, kind, layout, L, T, start,
                                      n_new):
    c = filled(5, L, 2, kind, seed=1)
    check_write(c, kind, layout, T, start, n_new)


@pytest.mark.parametrize("H,T,start", [(5, 4500, [130, 0]), (3, 9000, [61, 0]),
                                       (1, 14000, [0, 500])])
@pytest.mark.parametrize("kind,layout", [("e4m3", "half"),
                                         ("int8", "interleaved")])
def test_long_writes_match_the_definition(cuda_dev, kind, layout, H, T, start):
    # several blocks per CTA, runs of one and of several heads
    c = filled(2, 14600, H, kind, seed=1)
    check_write(c, kind, layout, T, start, [T, T - 131])


@pytest.mark.parametrize("T,H", [(150, 7), (32, 8), (33, 8)])
@pytest.mark.parametrize("kind,layout", [("e4m3", "interleaved"),
                                         ("int8", "half")])
def test_writes_of_many_uneven_rows(cuda_dev, kind, layout, T, H):
    # more rows than a warp takes at once, runs of rows without a new token,
    # shares that are cut between the heads of a block
    B, L = 75, 400
    rng = np.random.default_rng(11)
    start = rng.integers(-20, L, B)
    n_new = rng.integers(0, T + 1, B)
    n_new[3:6] = 0
    n_new[20:60] = 0
    start[62], start[63] = L, -T
    c = filled(B, L, H, kind, seed=1)
    check_write(c, kind, layout, T, start.tolist(), n_new.tolist())


@pytest.mark.parametrize("kind", KINDS)
def test_append_raises_a_blocks_scale(cuda_dev, kind):
    # larger tokens each time: the older codes are rounded again
    c = ops.kv8_cache(2, 384, 3, dtype=DT[kind])
    for step, scale in enumerate((0.1, 1.0, 0.5, 7.0)):
        check_write(c, kind, "half", 3, [100 + 3 * step, 3 * step],
                    seed=10 + step, scale=scale)


@pytest.mark.parametrize("kind", KINDS)
def test_write_in_pieces_is_one_write_when_scales_agree(cuda_dev, kind):
    B, T, H = 1, 700, 2
    k, v = tokens(B, T, H, 4)
    # the largest magnitude of every block comes first: no later growth
    v[:, ::128] = 9.0
    pos = torch.arange(T, dtype=torch.int32, device="cuda")[None].contiguous()
    table = ops.rope_table(THETA, T)
    a = ops.kv8_cache(B, T, H, dtype=DT[kind])
    b = ops.kv8_cache(B, T, H, dtype=DT[kind])
    ops.kv8_write(a, k, v, pos, i32([0]), table)
    at = 0
    for n in (1, 200, 55, 128, 1, 315):
        sl = slice(at, at + n)
        ops.kv8_write(b, k[:, sl].contiguous(), v[:, sl].contiguous(),
                      pos[:, sl].contiguous(), i32([at]), table)
        at += n
    torch.cuda.synchronize()
    assert torch.equal(a.v_scale, b.v_scale)
    assert np.array_equal(val(a.v), val(b.v))
    # keys: scales only grow, and end up equal
    assert torch.equal(a.k_scale, b.k_scale)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_values_make_their_block_nan(cuda_dev, kind, bad):
    c = filled(1, 512, 2, kind, seed=2)
    before = snap(c)
    k, v = tokens(1, 140, 2, 5)
    v[0, 3, 1, 17] = bad           # slot 203: block 1 of head 1
    pos = torch.arange(140, dtype=torch.int32, device="cuda")[None] \
        .contiguous()
    ops.kv8_write(c, k, v, pos, i32([200]), ops.rope_table(THETA, 512))
    torch.cuda.synchronize()
    s = c.v_scale.cpu()
    assert torch.isnan(s[0, 1, 1]) and torch.isnan(s).sum() == 1
    assert not torch.isnan(c.k_scale).any()
    # older codes of the block keep their bits
    assert np.array_equal(val(c.v)[0, 1, 128:200], before[1][0, 1, 128:200])
    _, vr = ops.kv8_read(c, i32([0]), 512)
    assert torch.isnan(vr[0, 128:256, 1]).all()
    assert torch.isfinite(vr[0, :128]).all()
    assert torch.isfinite(vr[0, 256:]).all()


@pytest.mark.parametrize("kind", KINDS)
def test_zero_and_tiny_blocks(cuda_dev, kind):
    c = filled(1, 256, 1, kind, seed=3)
    z = torch.zeros((1, 256, 1, 128), dtype=torch.bfloat16, device="cuda")
    t = z.clone()
    t[0, :128] = 2.0 ** -126      # a scale below the smallest normal: 0
    t[0, 128:] = 2.0 ** -100
    pos = torch.zeros((1, 256), dtype=torch.int32, device="cuda")
    table = ops.rope_table(THETA, 4)
    ops.kv8_write(c, z, t, pos, i32([0]), table)
    kr, vr = ops.kv8_read(c, i32([0]), 256)
    torch.cuda.synchronize()
    assert (c.k_scale == 0).all() and (kr == 0).all()
    assert (vr[0, :128] == 0).all()
    assert torch.equal(vr[0, 128:], t[0, 128:])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("L,T,start,kv_len", [
    (300, 300, [0, 0], None), (300, 1, [299, 17], None),
    (1000, 333, [-5, 900], None), (1000, 257, [700, 3], [800, 0]),
    (513, 600, [-50, 510], [2000, -1]),
])
def test_read_is_code_times_scale(cuda_dev, kind, L, T, start, kv_len):
    B, H = 2, 3
    c = filled(B, L, H, kind, seed=4)
    out = ops.kv8_read(c, i32(start), T,
                       kv_len=None if kv_len is None else i32(kv_len))
    torch.cuda.synchronize()
    for codes, scale, got in ((c.k, c.k_scale, out[0]),
                              (c.v, c.v_scale, out[1])):
        assert got.shape == (B, T, H, 128)
        full = codes.float() * scale.repeat_interleave(128, -1)[
            ..., :L, None]
        for b in range(B):
            end = L if kv_len is None else max(0, min(kv_len[b], L))
            want = torch.zeros((T, H, 128), device="cuda")
            a, z = max(start[b], 0), min(start[b] + T, end)
            if z > a:
                want[a - start[b]:z - start[b]] = full[b, :, a:z].transpose(
                    0, 1)
            assert torch.equal(got[b], want.bfloat16())


# ------------------------------------------------------------- attention
def queries(B, Hq, L, seed, scale=1.0):
    q = wl.random_tensor((B, Hq, 128), seed * 16 + 1, scale, torch.bfloat16,
                         "cuda")
    g = torch.Generator("cuda").manual_seed(seed)
    pos = torch.randint(0, L, (B,), dtype=torch.int32, device="cuda",
                        generator=g)
    return q, pos, ops.rope_table(THETA, L)


def check_decode(c, q, pos, table, start, length, layout, blocks=None,
                 **kw):
    out, lse = ops.kv8_decode(q, c, i32(start), i32(length), pos, table,
                              blocks=blocks, rope_layout=layout, **kw)
    torch.cuda.synchronize()
    assert ops.last_status() == ops.OK
    B, H, L, D = c.k.shape
    G = q.shape[1] // H
    go, gl = val(out), val(lse)
    k, v, ks, vs, _ = snap(c)
    qn, pn = val(q), pos.cpu().numpy()
    bl = None if blocks is None else blocks.cpu().numpy()
    for b in range(B):
        qr = oracle.kv8_rotate(qn[b][None], pn[b:b + 1], THETA, layout)[0]
        s, n = max(0, start[b]), max(0, min(length[b], L))
        for h in range(H):
            if bl is None:
                slots = np.arange(s, n)
            else:
                row = bl[b, h]
                keep = [j for i, j in enumerate(row)
                        if j >= 0 and (i == 0 or j > row[i - 1])]
                slots = np.array([t for j in keep
                                  for t in range(j * 128, j * 128 + 128)
                                  if s <= t < n], dtype=np.int64)
            for g in range(G):
                i = h * G + g
                o, l, w = oracle.kv8_attend(qr[i], k[b, h], v[b, h],
                                            ks[b, h], vs[b, h], slots)
                if slots.size == 0:
                    assert (go[b, i] == 0).all() and gl[b, i] == -np.inf
                    continue
                ds = 2 ** -18 * float(
                    (np.abs(k[b, h][slots]) @ (np.abs(qr[i])
                                               + np.abs(qr[i]).max() / 16)
                     * ks[b, h][slots // 128]).max()) / np.sqrt(D)
                assert abs(gl[b, i] - l) <= ds + 2 ** -20 * (1 + abs(l))
                floor = sum(np.abs(v[b, h][slots[slots // 128 == j]]).sum(0)
                            * vs[b, h][j] * np.exp(oracle.kv8_attend(
                                qr[i], k[b, h], v[b, h], ks[b, h], vs[b, h],
                                slots[slots // 128 == j])[1] - l)
                            for j in np.unique(slots // 128))
                tol = 2 ** -8 * np.abs(o) + (2 ** -11 + 4 * ds) * w + \
                    2 ** -23 * floor
                assert (np.abs(go[b, i] - o) <= tol).all(), \
                    (b, i, np.abs(go[b, i] - o).max())
    return out, lse


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H,G,layout", [
    (4, 1, "interleaved"), (2, 2, "half"), (1, 3, "interleaved"),
    (2, 4, "half"), (1, 7, "interleaved"), (2, 8, "interleaved"),
    (1, 12, "half"), (1, 16, "interleaved")])
def test_decode_head_groups(cuda_dev, kind, H, G, layout):
    L = 1337
    c = filled(3, L, H, kind, seed=6)
    q, pos, table = queries(3, H * G, L, 7)
    check_decode(c, q, pos, table, [0, 130, 700], [L, 131, 900], layout)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("L,start,length", [
    (1, [0, 0], [1, 0]), (127, [0, 126], [127, 127]),
    (128, [0, 0], [128, 1]), (129, [128, 0], [129, 129]),
    (640, [5, 300], [640, 300]),                # one row sees nothing
    (640, [-7, 9], [10 ** 9, 2]),               # clamped, and start > length
    (5000, [0, 4999], [4097, 5000]),
])
def test_decode_ranges(cuda_dev, kind, L, start, length):
    c = filled(2, L, 2, kind, seed=8)
    q, pos, table = queries(2, 4, max(L, 4), 9)
    check_decode(c, q, pos, table, start, length, "interleaved")


@pytest.mark.parametrize("kind", KINDS)
def test_decode_many_short_rows(cuda_dev, kind):
    # shares of one CTA cross many (row, head) pairs, empty rows among them
    B, L, H = 150, 260, 3
    c = filled(B, L, H, kind, seed=10)
    q, pos, table = queries(B, H, L, 11)
    rng = np.random.default_rng(5)
    n = rng.integers(0, L + 1, B)
    s = (n * rng.random(B) * 1.2).astype(int)
    check_decode(c, q, pos, table, s.tolist(), n.tolist(), "half")


@pytest.mark.parametrize("B", [1, 400])
def test_decode_of_rows_that_all_see_nothing(cuda_dev, B):
    c = filled(B, 130, 2, "e4m3", seed=11)
    q, pos, table = queries(B, 4, 130, 11)
    z = torch.zeros((B,), dtype=torch.int32, device="cuda")
    for kw in ({}, {"blocks": torch.empty((B, 2, 0), dtype=torch.int32,
                                          device="cuda")}):
        # (the list is empty though the range is not)
        end = z + 130 if kw else z
        out = torch.full_like(q, float("nan"))
        lse = torch.full((B, 4), float("nan"), device="cuda")
        ops.kv8_decode(q, c, z, end, pos, table, out=out, lse=lse, **kw)
        torch.cuda.synchronize()
        assert (out == 0).all() and (lse == -float("inf")).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [8.0, 60.0])
def test_decode_peaked_softmax(cuda_dev, kind, scale):
    # scores of tens to hundreds: few keys carry the weight, and the running
    # maximum rises late
    L = 3000
    c = filled(1, L, 2, kind, seed=12)
    c.k_scale.mul_(torch.linspace(0.2, 1, c.k_scale.shape[-1],
                                  device="cuda"))
    q, pos, table = queries(1, 4, L, 13, scale=scale)
    check_decode(c, q, pos, table, [3], [L], "interleaved")


@pytest.mark.parametrize("kind", KINDS)
def test_decode_ignores_what_it_cannot_see(cuda_dev, kind):
    L = 700
    c = filled(2, L, 2, kind, seed=14)
    q, pos, table = queries(2, 4, L, 15)
    s, n = [200, 0], [430, 129]
    want = check_decode(c, q, pos, table, s, n, "half")
    for b in range(2):
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
    got = ops.kv8_decode(q, c, i32(s), i32(n), pos, table,
                         rope_layout="half")
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("which", ["k_scale", "v_scale", "q"])
def test_decode_carries_visible_nan(cuda_dev, kind, which):
    L = 600
    c = filled(1, L, 2, kind, seed=16)
    q, pos, table = queries(1, 4, L, 17)
    clean, clean_lse = ops.kv8_decode(q, c, i32([0]), i32([L]), pos, table)
    if which == "q":
        q[0, 2, 5] = float("nan")
    else:
        getattr(c, which)[0, 1, 2] = float("nan")
    out, lse = ops.kv8_decode(q, c, i32([0]), i32([L]), pos, table)
    torch.cuda.synchronize()
    hit = [2] if which == "q" else [2, 3]       # heads of cache head 1
    for i in range(4):
        if i in hit:
            assert torch.isnan(out[0, i]).all()
        else:
            assert torch.equal(out[0, i], clean[0, i])
            assert torch.equal(lse[0, i], clean_lse[0, i])


def test_decode_of_a_blocks_list(cuda_dev):
    B, L, H, G = 3, 2000, 2, 2
    for kind in KINDS:
        c = filled(B, L, H, kind, seed=18)
        q, pos, table = queries(B, H * G, L, 19)
        bl = torch.tensor([
            [[0, 3, 4, 15], [1, 2, -1, -1]],
            # beside the range, twice the same, out of order, out of range
            [[0, 1, 1, 9], [5, 2, 3, 9999]],
            [[-1, -1, -1, -1], [15, 15, 15, 15]]], dtype=torch.int32,
            device="cuda")
        check_decode(c, q, pos, table, [0, 140, 0], [L, 1200, 1999],
                     "interleaved", blocks=bl)
        empty = torch.empty((B, H, 0), dtype=torch.int32, device="cuda")
        check_decode(c, q, pos, table, [0, 140, 0], [L, 1200, 1999],
                     "interleaved", blocks=empty)


@pytest.mark.parametrize("kind", KINDS)
def test_a_list_of_every_block_is_the_dense_result(cuda_dev, kind):
    B, L, H = 2, 9000, 4
    c = filled(B, L, H, kind, seed=20)
    q, pos, table = queries(B, H, L, 21)
    n = -(-L // 128)
    bl = torch.arange(n, dtype=torch.int32, device="cuda") \
        .expand(B, H, n).contiguous()
    a = ops.kv8_decode(q, c, i32([0, 0]), i32([L, L]), pos, table)
    b = ops.kv8_decode(q, c, i32([0, 0]), i32([L, L]), pos, table, blocks=bl)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------- selection
def check_select(c, q, pos, table, start, length, K, layout, n_sink=1,
                 n_recent=1):
    blocks, scores = ops.kv8_select(q, c, i32(start), i32(length), pos,
                                    table, K, n_sink=n_sink,
                                    n_recent=n_recent, rope_layout=layout)
    torch.cuda.synchronize()
    B, H, L, _ = c.k.shape
    G = q.shape[1] // H
    gb, gs = blocks.cpu().numpy(), scores.cpu().numpy()
    kb = c.k_bounds.cpu().numpy()
    ks = c.k_scale.cpu().numpy()
    tab = table.double().cpu().numpy()
    qn, pn = val(q), pos.cpu().numpy()
    for b in range(B):
        # the rotation by the table's own angles, in fp64
        cs, sn = tab[pn[b], :, 0], tab[pn[b], :, 1]
        x = qn[b]
        qr = np.empty_like(x)
        if layout == "half":
            qr[:, :64] = x[:, :64] * cs - x[:, 64:] * sn
            qr[:, 64:] = x[:, :64] * sn + x[:, 64:] * cs
        else:
            qr[:, 0::2] = x[:, 0::2] * cs - x[:, 1::2] * sn
            qr[:, 1::2] = x[:, 0::2] * sn + x[:, 1::2] * cs
        s, n = max(0, start[b]), max(0, min(length[b], L))
        first, last = s // 128, -(-n // 128) if n > s else s // 128
        for h in range(H):
            sc = oracle.kv8_block_scores(qr[h * G:h * G + G], kb[b, h],
                                         ks[b, h])
            want = oracle.kv8_pick(sc, first, last, K, n_sink, n_recent)
            m = len(want)
            assert gb[b, h, :m].tolist() == want
            assert (gb[b, h, m:] == -1).all()
            assert (gs[b, h, m:] == -np.inf).all()
            assert np.array_equal(gs[b, h, :m], sc[want], equal_nan=True)
    return blocks


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H,G,layout", [(4, 1, "interleaved"), (2, 4, "half"),
                                        (1, 7, "half"),
                                        (1, 16, "interleaved")])
@pytest.mark.parametrize("L,K", [(700, 3), (20000, 16), (70000, 100),
                                 (140000, 600)])
def test_select_matches_the_definition(cuda_dev, kind, H, G, layout, L, K):
    c = filled(2, L, H, kind, seed=22)
    c.k_scale.mul_(torch.rand(c.k_scale.shape, device="cuda",
                              generator=torch.Generator("cuda")
                              .manual_seed(3)) + 0.5)
    q, pos, table = queries(2, H * G, 4000, 23)
    check_select(c, q, pos, table, [0, L // 3 + 1], [L, L - 77], K, layout)


def test_select_of_the_longest_row(cuda_dev):
    L = 1 << 22
    n = L // 128
    g = torch.Generator("cuda").manual_seed(9)
    c = ops.kv8_cache(1, L, 1, dtype=torch.int8)
    b = torch.randint(-127, 128, c.k_bounds.shape, dtype=torch.int8,
                      device="cuda", generator=g)
    c.k_bounds.copy_(torch.sort(b, dim=-2).values)
    c.k_scale.copy_(torch.rand((1, 1, n), device="cuda", generator=g))
    q, pos, table = queries(1, 3, 4000, 39)
    check_select(c, q, pos, table, [1000], [L - 1], 3000, "half", 4, 100)


@pytest.mark.parametrize("start,length,K,sink,recent", [
    ([0, 0], [0, 1], 2, 1, 1), ([500, 127], [500, 129], 2, 1, 1),
    ([0, 300], [3000, 301], 64, 4, 8),          # fewer blocks than K
    ([0, 0], [3000, 2900], 5, 0, 0), ([0, 0], [3000, 2999], 6, 3, 3),
    ([10, -5], [10 ** 9, 2000], 1, 0, 1),
])
def test_select_ranges_and_forced_blocks(cuda_dev, start, length, K, sink,
                                         recent):
    c = filled(2, 3000, 2, "e4m3", seed=24)
    q, pos, table = queries(2, 2, 4000, 25)
    check_select(c, q, pos, table, start, length, K, "interleaved", sink,
                 recent)


@pytest.mark.parametrize("L", [128 * 100, 128 * 1500])
def test_select_ties_nan_and_odd_queries(cuda_dev, L):
    # equal scores everywhere, then NaN scales and a query of zeros
    c = filled(1, L, 2, "int8", seed=26)
    c.k_bounds.copy_(c.k_bounds[:, :, :1])
    c.k_scale.fill_(0.25)
    q, pos, table = queries(1, 4, 4000, 27)
    b = check_select(c, q, pos, table, [0], [L], 40, "interleaved")
    assert b[0, 0].tolist() == list(range(39)) + [L // 128 - 1]
    c.k_scale[0, 0, [7, 50, 99]] = float("nan")
    c.k_scale[0, 1] = 0.0
    check_select(c, q, pos, table, [0], [L], 40, "interleaved")
    q[0, 0] = 0
    check_select(c, q, pos, table, [0], [L], 40, "interleaved")
    q[0, 2, 3] = float("inf")       # scores of 0: still a list in range
    blocks, _ = ops.kv8_select(q, c, i32([0]), i32([L]), pos, table, 40)
    torch.cuda.synchronize()
    assert blocks[0, 1].tolist() == list(range(39)) + [L // 128 - 1]


# ----------------------------------------------------- all of it together
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout", LAYOUTS)
def test_serving_steps(cuda_dev, kind, layout):
    """A prompt enters the cache, tokens are appended one by one; each step
    selects blocks and attends over them. Against fp64 attention over the
    codes, and against the bf16 cache's decode within the cache's rounding."""
    B, H, G, T, L = 2, 2, 2, 900, 1024
    c = ops.kv8_cache(B, L, H, dtype=DT[kind])
    k, v = tokens(B, T + 6, H, 30)
    pos = torch.arange(T + 6, dtype=torch.int32, device="cuda") \
        .expand(B, -1).contiguous()
    q, _, table = queries(B, H * G, L, 31)
    n0 = [T, 651]
    ops.kv8_write(c, k[:, :T].contiguous(), v[:, :T].contiguous(),
                  pos[:, :T].contiguous(), i32([0, 0]), table,
                  n_new=i32(n0), rope_layout=layout)
    for step in range(6):
        n = [x + step for x in n0]
        kt = torch.stack([k[b, n[b]] for b in range(B)])[:, None]
        vt = torch.stack([v[b, n[b]] for b in range(B)])[:, None]
        ops.kv8_write(c, kt.contiguous(), vt.contiguous(),
                      i32([[x] for x in n]), i32(n), table,
                      rope_layout=layout)
        length = [x + 1 for x in n]
        blocks, _ = ops.kv8_select(q, c, i32([0, 0]), i32(length), i32(n),
                                   table, 3, rope_layout=layout)
        check_decode(c, q, i32(n), table, [0, 0], length, layout,
                     blocks=blocks)
    out, lse = check_decode(c, q, i32(n), table, [0, 0], length, layout)
    kr = ops.rope_apply(k, pos, table, rope_layout=layout)
    kx = kr.repeat_interleave(G, 2).contiguous()
    vx = v.repeat_interleave(G, 2).contiguous()
    ref, ref_lse = ops.decode(q, kx, vx, i32([0, 0]), i32(length), i32(n),
                              table, rope_layout=layout)
    # codes are off by at most 2^-4 (e4m3) or amax / 254 (int8); averaged
    # over hundreds of keys a tenth of |v| is ample
    assert (out.float() - ref.float()).abs().max() <= 0.1
    assert (lse - ref_lse).abs().max() <= 0.1


@pytest.mark.parametrize("kind", KINDS)
def test_read_back_feeds_a_prompt_chunk(cuda_dev, kind):
    """Chunked prefill: the cached prefix, read back as bf16, is a key chunk
    of fwd_block; its last query row is a decode over the same codes."""
    B, H, Np = 1, 2, 640
    c = filled(B, Np, H, kind, seed=32)
    k_rot, v = ops.kv8_read(c, i32([0]), Np)
    Nq = 128
    q = wl.random_tensor((B, Nq, H, 128), 33, 1.0, torch.bfloat16, "cuda")
    pos = torch.arange(Np, Np + Nq, dtype=torch.int32, device="cuda")[None] \
        .contiguous()
    zq = torch.zeros((B, Nq), dtype=torch.int32, device="cuda")
    zk = torch.zeros((B, Np), dtype=torch.int32, device="cuda")
    o, l = ops.fwd_block(q, k_rot, v, zq, pos, zk, Np, 0, THETA, 1024)
    table = ops.rope_table(THETA, 1024)
    od, ld = ops.kv8_decode(q[:, -1].contiguous(), c, i32([0]), i32([Np]),
                            pos[:, -1].contiguous(), table)
    torch.cuda.synchronize()
    # fwd_block rounds rotated q, k (2^-8 each) and P to bf16
    assert (o[:, -1].float() - od.float()).abs().max() <= 2e-2
    assert (l[:, :, -1] - ld).abs().max() <= 2e-2


def test_graph_replay_and_another_stream(cuda_dev):
    """One serving step captured twice (each graph with its own workspace)
    and replayed gives the eager results; so does another stream."""
    B, H, G, L = 2, 4, 2, 20000
    c = filled(B, L, H, "e4m3", seed=34)
    q, pos, table = queries(B, H * G, L, 35)
    k, v = tokens(B, 1, H, 36)
    at, n = i32([19000, 777]), i32([19001, 778])
    z = i32([0, 0])

    def step(res):
        ops.kv8_write(c, k, v, pos[:, None].contiguous(), at, table)
        bl, _ = ops.kv8_select(q, c, z, n, pos, table, 8)
        res["blocks"] = bl
        res["sparse"] = ops.kv8_decode(q, c, z, n, pos, table, blocks=bl)
        res["dense"] = ops.kv8_decode(q, c, z, n, pos, table)

    want, got, other = {}, {}, {}
    step(want)
    step(want)          # the write is idempotent from here on
    torch.cuda.synchronize()
    flat = lambda r: [r["blocks"], *r["sparse"], *r["dense"]]
    keep = [x.clone() for x in flat(want)]
    graphs = []
    for res in (got, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(res)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for res in (got, other):
        assert all(torch.equal(a, b) for a, b in zip(flat(res), keep))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    res = {}
    with torch.cuda.stream(side):
        step(res)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(flat(res), keep))
    # the stream given to the calls instead
    ops.kv8_write(c, k, v, pos[:, None].contiguous(), at, table, stream=side)
    bl, _ = ops.kv8_select(q, c, z, n, pos, table, 8, stream=side)
    res = {"blocks": bl, "sparse": ops.kv8_decode(q, c, z, n, pos, table,
                                                  blocks=bl, stream=side),
           "dense": ops.kv8_decode(q, c, z, n, pos, table, stream=side)}
    kr, _ = ops.kv8_read(c, at, 1, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(flat(res), keep))
    assert torch.equal(kr, ops.kv8_read(c, at, 1)[0])


def test_offsets_past_32_bits(cuda_dev):
    """Codes beyond the first 4 GiB: the last head of a 1M-slot cache."""
    L, H = 1 << 20, 34
    c = ops.kv8_cache(1, L, H, dtype=torch.int8)
    T, at = 300, L - 300
    k, v = tokens(1, T, H, 37)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")[None].contiguous()
    q, qp, table = queries(1, H, 4000, 38)
    ops.kv8_write(c, k, v, pos, i32([at]), table)
    kr, vr = ops.kv8_read(c, i32([at]), T)
    out, lse = ops.kv8_decode(q, c, i32([at]), i32([L]), qp, table)
    bl, _ = ops.kv8_select(q, c, i32([at]), i32([L]), qp, table, 2)
    torch.cuda.synchronize()
    assert ops.last_status() == ops.OK
    assert bl[0, H - 1].tolist() == [L // 128 - 3, L // 128 - 1]
    h = H - 1
    s = val(kr[0, :, h]) @ oracle.kv8_rotate(
        val(q[0, h])[None], qp.cpu().numpy(), THETA, "interleaved")[0] \
        / np.sqrt(128)
    p = np.exp(s - s.max())
    # codes read back through bf16: 2^-8 of each key and value
    assert abs(float(lse[0, h]) - (s.max() + np.log(p.sum()))) <= 2 ** -6
    o = p @ val(vr[0, :, h]) / p.sum()
    assert np.abs(val(out[0, h]) - o).max() <= 2 ** -5


def test_a_small_workspace_is_refused(cuda_dev):
    c = filled(2, 640, 2, "e4m3")
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    table = ops.rope_table(THETA, 64)
    need = ops.kv8_decode_workspace_size(2, 640, 4, 2)
    assert need > 0
    out, lse = torch.full_like(q, 7.0), torch.full((2, 4), 7.0, device="cuda")
    for at, size in ((0, need - 1), (8, need)):       # too short, misaligned
        ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
        with pytest.raises(ops.LwmError):
            ops.kv8_decode(q, c, i32([0, 0]), i32([640, 5]), i32([1, 2]),
                           table, out=out, lse=lse,
                           workspace=ws[at:at + size])
    torch.cuda.synchronize()
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all())


def test_two_streams_at_once(cuda_dev):
    """Prompts written, blocks chosen and tokens decoded on two streams at
    the same time, each with its cache, give what they give alone."""
    B, H, G, L, T = 3, 8, 2, 4000, 3000
    kinds = ("e4m3", "int8")
    made = []
    for i, kind in enumerate(kinds):
        k, v = tokens(B, T, H, 50 + i)
        q, pos, table = queries(B, H * G, L, 60 + i)
        made.append((kind, k, v, q, pos, table))
    at = i32([0, 77, 900])
    n, z = at + T, i32([0, 0, 0])
    where = torch.arange(T, dtype=torch.int32, device="cuda").expand(B, T)
    where = where.contiguous()

    def run(kind, k, v, q, pos, table):
        c = ops.kv8_cache(B, L, H, dtype=DT[kind])
        ops.kv8_write(c, k, v, where, at, table)
        bl, sc = ops.kv8_select(q, c, z, n, pos, table, 6)
        return [*c, bl, sc, *ops.kv8_decode(q, c, z, n, pos, table),
                *ops.kv8_decode(q, c, z, n, pos, table, blocks=bl)]

    alone = [run(*m) for m in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in kinds]
    for _ in range(4):
        got = []
        for st, m in zip(streams, made):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append(run(*m))
        torch.cuda.synchronize()
        assert ops.last_status() == ops.OK
        for a, b in zip(alone, got):
            for x, y in zip(a, b):
                x, y = ((t.view(torch.int8) if t.dtype.itemsize == 1 else t)
                        for t in (x, y))
                assert torch.equal(x, y)
