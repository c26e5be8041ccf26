"""Tensors that ops.fwd_block refuses before any pointer reaches the library
(no GPU): the C call takes its sizes from q and trusts every other buffer."""

import pytest
import torch

from long_context_blockwise_causal_b200 import ops

B, NQ, NK, H = 2, 5, 7, 4
BF, I32 = torch.bfloat16, torch.int32


def call(**kw):
    z = lambda *s, dt=BF: torch.zeros(s, dtype=dt)
    a = dict(q=z(B, NQ, H, 128), k_rot=z(B, NK, H, 128), v=z(B, NK, H, 128),
             seg_q=z(B, NQ, dt=I32), pos_q=z(B, NQ, dt=I32),
             seg_k=z(B, NK, dt=I32), q_off=NK, k_off=0, theta=1e4, max_pos=16)
    return ops.fwd_block(**{**a, **kw})


def z(*s, dt=BF):
    return torch.zeros(s, dtype=dt)


@pytest.mark.parametrize("kw", [
    # a cache of fewer heads than the queries, read back as it is
    {"k_rot": z(B, NK, 1, 128), "v": z(B, NK, 1, 128)},
    {"k_rot": z(B, NK, H, 128), "v": z(B, NK, 2, 128)},
    {"v": z(B, NK - 1, H, 128)}, {"v": z(B - 1, NK, H, 128)},
    {"k_rot": z(B - 1, NK, H, 128)}, {"k_rot": z(B, NK, H * 128)},
    {"k_rot": z(B, NK, H, 64)}, {"q": z(B, NQ * H, 128)},
    {"q": z(B, NQ, H, 128, dt=torch.float32)},
    {"k_rot": z(B, NK, H, 128, dt=torch.int8)},
    {"v": z(B, NK, H, 128, dt=torch.float16)},
    {"seg_q": z(B, NQ - 1, dt=I32)}, {"seg_k": z(B, NQ, dt=I32)},
    {"pos_q": z(B, NQ, dt=torch.int64)}, {"pos_q": z(NQ, dt=I32)},
    {"out": z(B, NQ, 1, 128)}, {"out": z(B, NQ, H, 128, dt=torch.float32)},
    {"lse": z(B, NQ, H, dt=torch.float32)}, {"lse": z(B, H, NQ)},
    {"table": z(16, 64, 2)}, {"table": z(16, 128, dt=torch.float32)},
])
def test_fwd_block_refuses_tensors_that_do_not_match(kw):
    with pytest.raises(ops.LwmError) as e:
        call(**kw)
    assert e.value.status == ops.ERR_INVALID_ARG


def test_matching_tensors_only_lack_the_device():
    for kw in ({}, {"k_rot": z(B, 0, H, 128), "v": z(B, 0, H, 128),
                    "seg_k": z(B, 0, dt=I32)},
               {"table": z(16, 64, 2, dt=torch.float32)}):
        with pytest.raises(ValueError, match="CUDA"):
            call(**kw)
