"""Decode of rows with very many heads (needs a B200): 2^25 query heads a row,
whose channels are counted past 32 bits (2^25 heads x 64 pairs of channels are
2^31, a negative number in 32 bits, with which a row that sees nothing kept
what was in `out`). About 40 GB on the device."""

import pytest
import torch

from long_context_blockwise_causal_b200 import ops

pytestmark = pytest.mark.gpu


def test_rows_of_many_heads(cuda_dev):
    H, G = 1 << 21, 16
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    c = ops.kv8_cache(2, 1, H)
    c.v.view(torch.uint8).random_(0, 120)            # finite codes
    c.v_scale.uniform_(0.5, 2.0)
    q = torch.zeros((2, H * G, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    lse = torch.full((2, H * G), 7.0, device="cuda")
    ops.kv8_decode(q, c, i32(0, 0), i32(0, 1), i32(0, 0),
                   ops.rope_table(1e4, 4), out=out, lse=lse)
    torch.cuda.synchronize()
    assert ops.last_status() == ops.OK
    del q
    # the first row sees nothing, the second one slot with a weight of 1
    assert bool((lse[0] == -float("inf")).all())
    assert bool((lse[1] == 0).all())
    step = 1 << 17
    for h in range(0, H, step):
        at = slice(h * G, (h + step) * G)
        assert bool((out[0, at] == 0).all())
        want = (c.v[1, h:h + step, 0].float()
                * c.v_scale[1, h:h + step]).bfloat16()
        got = out[1, at].view(step, G, 128)
        assert bool((got == want[:, None]).all())
