"""A stream of another device than the cache's is refused (no GPU): the calls
run on a stream of the cache's device, and would have run on its current one."""

from types import SimpleNamespace

import pytest
import torch

from long_context_blockwise_causal_b200 import ops


@pytest.mark.parametrize("call", [
    lambda c, i, q, t, s: ops.kv8_write(c, q[:, None], q[:, None], i[:, None],
                                        i, t, stream=s),
    lambda c, i, q, t, s: ops.kv8_read(c, i, 3, stream=s),
    lambda c, i, q, t, s: ops.kv8_select(q, c, i, i, i, t, 2, stream=s),
    lambda c, i, q, t, s: ops.kv8_decode(q, c, i, i, i, t, stream=s),
])
def test_a_stream_of_another_device_is_refused(call):
    c = ops.kv8_cache(2, 300, 2, device="cpu")
    other = SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0)
    with pytest.raises(ops.LwmError) as e:
        call(c, torch.zeros(2, dtype=torch.int32),
             torch.zeros(2, 2, 128, dtype=torch.bfloat16),
             torch.zeros(8, 64, 2), other)
    assert e.value.status == ops.ERR_INVALID_ARG
