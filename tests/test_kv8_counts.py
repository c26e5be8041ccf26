"""Counts given to the 8-bit cache's bindings that do not fit a C int: refused,
not cut to their low 32 bits (no GPU)."""

import pytest
import torch

from long_context_blockwise_causal_b200 import ops

WRAP = 1 << 32                      # low 32 bits: 0
B, L, H = 2, 300, 2


def call(**kw):
    c = ops.kv8_cache(B, L, H, device="cpu")
    q = torch.zeros(B, H, 128, dtype=torch.bfloat16)
    i32 = torch.zeros(B, dtype=torch.int32)
    return ops.kv8_select(q, c, i32, i32, i32, torch.zeros(L, 64, 2),
                          **{**dict(n_select=4), **kw})


@pytest.mark.parametrize("kw", [
    {"n_select": WRAP + 4}, {"n_select": 1 << 31}, {"n_select": -WRAP + 4},
    {"n_sink": WRAP}, {"n_sink": -1}, {"n_recent": WRAP + 1},
    {"n_recent": -1}])
def test_select_counts(kw):
    with pytest.raises(ops.LwmError) as e:
        call(**kw)
    assert e.value.status == ops.ERR_INVALID_ARG
    with pytest.raises(ValueError, match="CUDA"):
        call(n_select=4, n_sink=2, n_recent=2)


def test_read_count():
    c = ops.kv8_cache(0, L, H, device="cpu")       # no row: nothing to hold
    i32 = torch.zeros(0, dtype=torch.int32)
    for T in (WRAP + 1, -1, 1 << 31):
        with pytest.raises(ops.LwmError) as e:
            ops.kv8_read(c, i32, T)
        assert e.value.status == ops.ERR_INVALID_ARG


def test_workspace_counts():
    size = ops.kv8_decode_workspace_size
    assert size(1, 4096, 8, 2) > 0 and size(1, 4096, 8, 2, 4) > 0
    for args in ((WRAP + 1, 4096, 8, 2), (1, WRAP + 4096, 8, 2),
                 (1, 4096, WRAP + 8, 2), (1, 4096, 8, WRAP + 2),
                 (1 - WRAP, 4096, 8, 2), (1, 4096, 8, 2, WRAP + 4)):
        assert size(*args) == 0
