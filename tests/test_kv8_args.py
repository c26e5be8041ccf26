"""Host-side checks of the 8-bit cache's entry points and oracle (no GPU):
refusals come back as status codes before anything is launched."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from long_context_blockwise_causal_b200 import ops

P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 4)      # not for 16-byte loads
OFF = ctypes.c_void_p((1 << 20) + 2)      # not for 4-byte words
BIG = 1 << 40


def write(k=P, v=P, pos=P, start=P, n_new=None, table=P, max_pos=64, B=1, T=4,
          L=256, H=2, D=128, dtype=0, kind=0, layout=0, kc=P, vc=P, ks=P,
          vs=P, kb=P):
    return ops.lib().lwm_kv8_write(k, v, pos, start, n_new, table, max_pos, B,
                                   T, L, H, D, dtype, kind, layout, kc, vc,
                                   ks, vs, kb, None)


def read(kc=P, vc=P, ks=P, vs=P, start=P, kv_len=None, B=1, T=4, L=256, H=2,
         D=128, dtype=0, kind=0, k=P, v=P):
    return ops.lib().lwm_kv8_read(kc, vc, ks, vs, start, kv_len, B, T, L, H,
                                  D, dtype, kind, k, v, None)


def select(q=P, kb=P, ks=P, s=P, n=P, pos=P, table=P, max_pos=64, B=1, L=256,
           Hq=4, H=2, D=128, dtype=0, layout=0, K=2, sink=1, recent=1,
           blocks=P, scores=P):
    return ops.lib().lwm_kv8_select(q, kb, ks, s, n, pos, table, max_pos, B,
                                    L, Hq, H, D, dtype, layout, K, sink,
                                    recent, blocks, scores, None)


def decode(q=P, kc=P, vc=P, ks=P, vs=P, s=P, n=P, pos=P, blocks=None, K=-1,
           table=P, max_pos=64, B=1, L=256, Hq=4, H=2, D=128, dtype=0, kind=0,
           layout=0, out=P, lse=P, ws=P, wsb=BIG):
    return ops.lib().lwm_kv8_decode(q, kc, vc, ks, vs, s, n, pos, blocks, K,
                                    table, max_pos, B, L, Hq, H, D, dtype,
                                    kind, layout, out, lse, ws, wsb, None)


INV, UNS, WSP = ops.ERR_INVALID_ARG, ops.ERR_UNSUPPORTED, ops.ERR_WORKSPACE


@pytest.mark.parametrize("call,kw,status", [
    (write, {"k": None}, INV), (write, {"kb": None}, INV),
    (write, {"ks": OFF}, INV), (write, {"n_new": OFF}, INV),
    (write, {"k": ODD}, INV), (write, {"pos": OFF}, INV),
    (write, {"T": -1}, INV), (write, {"L": -1}, INV),
    (write, {"max_pos": 0}, INV), (write, {"kind": 2}, INV),
    (write, {"layout": 2}, INV), (write, {"D": 64}, UNS),
    (write, {"dtype": 1}, UNS),
    (write, {"B": 4, "L": 1 << 30}, INV),           # B * L in 32 bits
    (write, {"B": 1 << 20, "H": 256}, INV),         # B * H
    (write, {"H": 1 << 20, "T": 1 << 20}, UNS),     # too many CTAs
    (write, {"T": 0, "k": None}, ops.OK), (write, {"H": 0}, ops.OK),
    (write, {"L": 0, "kc": None}, ops.OK),
    (read, {"kc": None}, INV), (read, {"start": OFF}, INV),
    (read, {"kv_len": OFF}, INV), (read, {"T": -4}, INV),
    (read, {"k": None}, INV), (read, {"kind": -1}, INV),
    (read, {"H": 1 << 18, "T": 1 << 18}, UNS),      # too many CTAs
    (read, {"D": 256}, UNS), (read, {"dtype": 1}, UNS),
    (read, {"T": 0, "k": None}, ops.OK), (read, {"B": 0}, ops.OK),
    (select, {"kb": None}, INV), (select, {"scores": OFF}, INV),
    (select, {"H": 0}, INV), (decode, {"H": 0}, INV),   # heads over none
    (select, {"Hq": 5}, INV), (select, {"Hq": -2}, INV),
    (select, {"K": 0}, INV), (select, {"sink": -1}, INV),
    (select, {"sink": 2, "recent": 1}, INV),        # more than K
    (write, {"L": 2 ** 31 - 1, "H": 1}, INV), (write, {"T": 2 ** 31 - 1}, INV),
    (read, {"L": 2 ** 31 - 127, "H": 1}, INV), (read, {"T": 2 ** 31 - 1}, INV),
    (decode, {"L": 2 ** 31 - 1, "H": 1}, INV),
    (decode, {"B": 1 << 12, "L": 128, "H": 1, "Hq": 1, "K": 1 << 19}, UNS),
    (read, {"B": 1 << 20, "H": 1 << 7, "L": 128}, UNS),
    (select, {"sink": 2 ** 31 - 1, "recent": 2 ** 31 - 1}, INV),
    (select, {"max_pos": 0}, INV), (select, {"layout": 7}, INV),
    (select, {"Hq": 34}, UNS), (select, {"D": 64}, UNS),
    (select, {"L": (1 << 22) + 1}, UNS), (select, {"dtype": 1}, UNS),
    (select, {"B": 0, "q": None}, ops.OK), (select, {"Hq": 0}, ops.OK),
    (decode, {"q": None}, INV), (decode, {"vc": ODD}, INV),
    (decode, {"ws": None}, INV), (decode, {"blocks": OFF, "K": 1}, INV),
    (decode, {"blocks": None, "K": 1}, INV), (decode, {"Hq": 3}, INV),
    (decode, {"kind": 3}, INV), (decode, {"max_pos": 0}, INV),
    (decode, {"B": -1}, INV), (decode, {"Hq": 34}, UNS),
    (decode, {"K": 1 << 30, "blocks": P}, UNS),     # tiles in 32 bits
    (decode, {"D": 96}, UNS), (decode, {"dtype": 1}, UNS),
    (decode, {"wsb": 64}, WSP),
    (decode, {"wsb": 64, "blocks": P, "K": 3}, WSP), (decode, {"B": 0, "q": None}, ops.OK),
    (decode, {"H": 0, "Hq": 0, "q": None}, ops.OK),
])
def test_bad_arguments_are_refused_before_launch(call, kw, status):
    assert call(**kw) == status


def test_workspace_size_counts_partial_results():
    size = lambda *a: ops.lib().lwm_kv8_decode_workspace_size(*a)
    assert size(1, 4096, 8, 2, 128, -1) >= 130 * 4 * 4
    assert size(1, 4096, 8, 2, 128, 4) > 0
    assert size(1, 1 << 20, 8, 8, 128, -1) > size(1, 128, 8, 8, 128, -1)
    assert size(1, 4096, 7, 2, 128, -1) == 0          # Hq over H
    assert size(1, 4096, 8, 2, 64, -1) == 0
    assert size(-1, 4096, 8, 2, 128, -1) == 0
    assert size(0, 4096, 8, 2, 128, -1) == 0
    assert size(1, 4096, 8, 0, 128, -1) == 0


def _refused(fn, *a, **kw):
    with pytest.raises(ops.LwmError) as e:
        fn(*a, **kw)
    assert e.value.status == ops.ERR_INVALID_ARG


def test_bindings_check_tensors_before_the_library():
    B, L, H, T = 2, 300, 2, 5
    c = ops.kv8_cache(B, L, H, device="cpu")
    assert c.k_scale.shape == (B, H, 3) and c.k_bounds.shape == (B, H, 3, 2,
                                                                 128)
    k = torch.zeros(B, T, H, 128, dtype=torch.bfloat16)
    pos = torch.zeros(B, T, dtype=torch.int32)
    i32 = torch.zeros(B, dtype=torch.int32)
    table = torch.zeros(L, 64, 2)
    w = lambda **kw: ops.kv8_write(**{**dict(
        cache=c, k=k, v=k, positions=pos, start=i32, table=table), **kw})
    _refused(w, k=k.float())
    _refused(w, v=k[:, :3])
    _refused(w, positions=pos.long())
    _refused(w, start=i32[:1])
    _refused(w, n_new=i32.float())
    _refused(w, table=table.double())
    _refused(w, cache=c._replace(v=c.v.float()))
    _refused(w, cache=c._replace(k=c.k.float(), v=c.v.float()))
    _refused(w, cache=c._replace(k_scale=c.k_scale[..., :2]))
    _refused(w, cache=c._replace(k_bounds=c.k_bounds[..., 0, :]))
    _refused(ops.kv8_read, c, i32.long(), 4)
    _refused(ops.kv8_read, c, i32, -1)
    _refused(ops.kv8_read, c, i32, 4, k_rot=k)
    q = torch.zeros(B, 2 * H, 128, dtype=torch.bfloat16)
    _refused(ops.kv8_select, q[:, :3].contiguous(), c, i32, i32, i32, table, 4)
    _refused(ops.kv8_select, q, c, i32, i32, i32, table, 0)
    _refused(ops.kv8_select, q, c, i32, i32, i32.long(), table, 4)
    _refused(ops.kv8_decode, q.float(), c, i32, i32, i32, table)
    _refused(ops.kv8_decode, q, c, i32, i32, i32, table,
             blocks=torch.zeros(B, 2 * H, 3, dtype=torch.int32))
    _refused(ops.kv8_decode, q, c, i32, i32, i32, table,
             blocks=torch.zeros(B, H, 3, dtype=torch.int64))
    _refused(ops.kv8_decode, q, c, i32, i32, i32, table, out=q[:, :2])
    with pytest.raises(TypeError):
        ops.kv8_cache(1, 8, 1, dtype=torch.float16, device="cpu")
    # consistent tensors: only the device check is left
    for call in (lambda: w(), lambda: ops.kv8_read(c, i32, 4),
                 lambda: ops.kv8_select(q, c, i32, i32, i32, table, 2),
                 lambda: ops.kv8_decode(q, c, i32, i32, i32, table)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


# ---------------------------------------------------------- oracle pins
def test_oracle_codes_are_the_nearest():
    grid = np.array([float(torch.tensor(i, dtype=torch.uint8).view(
        torch.float8_e4m3fn).float()) for i in range(127)])
    assert grid.max() == oracle.KV8_QMAX["e4m3"]
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.normal(size=2000) * s for s in (1e-3, 1, 300)])
    c = oracle.kv8_encode(y, "e4m3")
    near = np.abs(np.abs(y)[:, None] - grid).min(1)
    assert np.allclose(np.abs(np.abs(c) - np.abs(y)), near, rtol=0, atol=0)
    assert set(np.abs(c)) <= set(grid)
    mids = (grid[1:] + grid[:-1]) / 2               # ties: the even code
    got = oracle.kv8_encode(mids, "e4m3")
    want = np.where(np.arange(126) % 2 == 0, grid[:-1], grid[1:])
    assert np.array_equal(got, want)
    assert np.array_equal(oracle.kv8_encode([0.5, 1.5, -2.5, 500], "int8"),
                          [0, 2, -2, 127])


def test_oracle_scores_bound_the_keys():
    rng = np.random.default_rng(1)
    c = oracle.kv8_encode(rng.normal(size=(3, 128, 128)) * 40, "int8")
    b = np.stack([c.min(1), c.max(1)], 1)
    q = rng.normal(size=(2, 128))
    s = oracle.kv8_block_scores(q, b, np.ones(3))
    for g in range(2):
        a = np.abs(q[g]).max()
        qi = np.round(q[g] * (127 / a)) * a / 127
        assert (s >= (c @ qi).max(1) * (1 - 1e-6)).all()
    assert oracle.kv8_pick(np.array([1., 5., 5., np.nan, 0.]), 0, 5, 3, 0,
                           1) == [1, 3, 4]
