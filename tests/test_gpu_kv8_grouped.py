"""Read-back of a grouped 8-bit cache for a prompt chunk (needs a B200): the
heads are repeated first, and fwd_block refuses them where they are not."""

import pytest
import torch

from long_context_blockwise_causal_b200 import ops
from long_context_blockwise_causal_b200 import workloads as wl

pytestmark = pytest.mark.gpu

THETA = 1e6


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("H,G,layout", [(2, 4, "half"), (1, 16, "interleaved"),
                                        (3, 2, "interleaved")])
def test_grouped_prefix_feeds_a_prompt_chunk(cuda_dev, dtype, H, G, layout):
    B, Np, Nq = 1, 20, 4
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    rand = lambda s, *n: wl.random_tensor(n, s, 1.0, torch.bfloat16, "cuda")
    table = ops.rope_table(THETA, 64)
    c = ops.kv8_cache(B, 300, H, dtype=dtype)
    ops.kv8_write(c, rand(1, B, Np, H, 128), rand(2, B, Np, H, 128),
                  i32([list(range(Np))]), i32([0]), table, rope_layout=layout)
    k_rot, v = ops.kv8_read(c, i32([0]), Np)
    q = rand(3, B, Nq, H * G, 128)
    pos = i32([list(range(Np, Np + Nq))])
    segs = torch.zeros((B, Nq), dtype=torch.int32, device="cuda")
    segk = torch.zeros((B, Np), dtype=torch.int32, device="cuda")
    call = lambda a, b: ops.fwd_block(q, a, b, segs, pos, segk, Np, 0, THETA,
                                      64, rope_layout=layout)
    kx, vx = (x.repeat_interleave(G, 2) for x in (k_rot, v))
    for a, b in ((k_rot, v), (kx, v), (k_rot, vx)):
        with pytest.raises(ops.LwmError) as e:
            call(a, b)
        assert e.value.status == ops.ERR_INVALID_ARG
    o, l = call(kx, vx)
    for t in range(Nq):        # no query of the chunk sees another's key here
        od, ld = ops.kv8_decode(q[:, t].contiguous(), c, i32([0]), i32([Np]),
                                pos[:, t].contiguous(), table,
                                rope_layout=layout)
        torch.cuda.synchronize()
        # fwd_block's rotated q and the keys read back are bf16, 2^-8 each, so
        # scores are off by DS; P, v and both outputs are bf16 too
        s = (q[0, t].abs().float()[:, None] * kx[0].transpose(0, 1).abs()
             .float()).sum(-1).amax() / 128 ** 0.5
        # (rotated, a pair's channels are at most sqrt(2) of its largest)
        ds = 2 * 2 ** -8 * 2 ** 0.5 * float(s)
        big = float(vx.abs().amax())
        assert (l[:, :, t] - ld).abs().max() <= ds
        assert (o[:, t].float() - od.float()).abs().max() <= \
            big * (2 * ds + 4 * 2 ** -8)
        assert ds < 0.15 and float(od.float().std()) > 0.1
