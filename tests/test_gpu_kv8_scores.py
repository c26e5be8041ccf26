"""Units of the block scores (needs a B200): times (Q / 127) / sqrt(D), and
with what the rounding of the query's codes may take, they bound the scores of
every key of the block; where all keys of a block are one and the same, they
are its score, but for that rounding and the bounds' (outwards, by less than
one unit of k_scale Q / 127 a channel)."""

import numpy as np
import pytest
import torch

import oracle
from long_context_blockwise_causal_b200 import ops
from test_gpu_kv8 import KINDS, THETA, filled, i32, queries, val

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("alike", [False, True])
def test_scores_bound_the_keys_in_units_of_lse(cuda_dev, kind, layout, alike):
    B, H, G, L = 2, 2, 3, 128 * 12
    n = L // 128
    c = filled(B, L, H, kind, seed=70)
    if alike:
        one = c.k.view(torch.uint8).view(B, H, n, 128, 128)
        one.copy_(one[:, :, :, :1].clone())
        u = c.k.view(B, H, n, 128, 128)[:, :, :, 0].float() * (
            127 / oracle.KV8_QMAX[kind])
        c.k_bounds[..., 0, :] = u.floor().to(torch.int8)
        c.k_bounds[..., 1, :] = u.ceil().to(torch.int8)
    q, pos, table = queries(B, H * G, L, 71)
    bl, sc = ops.kv8_select(q, c, i32([0] * B), i32([L] * B), pos, table, n,
                            rope_layout=layout)
    torch.cuda.synchronize()
    assert torch.equal(bl, i32(np.broadcast_to(np.arange(n), (B, H, n))
                               .copy()))
    k, _, ks, _, kb = (val(x) for x in c)
    factor = oracle.KV8_QMAX[kind] / 127 / np.sqrt(128)
    for b in range(B):
        qr = np.stack([oracle.kv8_rotate(val(q[b, i])[None],
                                         pos[b:b + 1].cpu().numpy(), THETA,
                                         layout)[0] for i in range(H * G)])
        for h in range(H):
            mine = qr[h * G:h * G + G]
            s = (k[b, h] @ mine.T).reshape(n, 128, G) * ks[b, h][:, None,
                                                               None]
            most = s.max((1, 2)) / np.sqrt(128)
            slack = np.abs(kb[b, h]).max(1).sum(-1) * ks[b, h] * \
                np.abs(mine).max() / 254
            bound = (val(sc[b, h]) + slack) * factor
            # (scores are fp32, the table's angles too: 2^-22 of |q| |k|)
            room = 2 ** -20 * np.abs(bound)
            assert (most <= bound + room).all()
            if alike:
                wide = np.abs(mine).sum(-1).max() * ks[b, h] * factor
                assert (bound - 2 * slack * factor <= most + wide
                        + room).all()
