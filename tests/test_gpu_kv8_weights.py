"""Precision of the softmax weights in the 8-bit cache's decode (needs a
B200).

Values that cancel make the weights' rounding visible beside the rounding of
`out` to bf16: each channel's values are chosen so that the exact sum of one
query head is less than 2^-9 of the sum of magnitudes W = sum p |v|. The
queries hold one power of two, at position 0, and the scales are 1, so that
scores, at most 2 in magnitude, are exact but for fp32: the factor log2(e) /
sqrt(D) and its two products, at most 2^-22 of a score (3 in units of log 2),
the difference from the maximum 2^-24 of 6, the exponential 2^-22, the sums
2^-22: together below 2^-17.5 W. The weights themselves enter the second
product as codes: e4m3 to 2^-4 of what is left four times over, 2^-16 of each;
int8 in three parts, 2^-23 of the block's largest weight, which is less than
2^6 times any other, so 2^-17 W. All of it is less than 2^-15.5 W, and `out` is
rounded by 2^-8 of itself.
"""

import numpy as np
import pytest
import torch

import oracle
from long_context_blockwise_causal_b200 import ops

pytestmark = pytest.mark.gpu

DT = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
SLOTS = 5


def code_values(kind):
    """The positive codes of a type, from 1/16 of the largest on."""
    if kind == "int8":
        return np.arange(8.0, 128.0)
    e = np.arange(32, 449, 0.5)
    return np.unique(oracle.kv8_encode(e, kind))


def cancelling(p, kind, rng, tries=6000):
    """[SLOTS] codes whose sum under the weights p nearly cancels."""
    c = code_values(kind)
    v = rng.choice(c, (tries, SLOTS)) * rng.choice([-1.0, 1.0],
                                                   (tries, SLOTS))
    return v[np.argmin(np.abs(v @ p) / (np.abs(v) @ p))]


def setting(kind, H, G, seed=0):
    """Codes k, v [H, SLOTS, 128] and queries [H * G, 128] in fp64."""
    rng = np.random.default_rng(seed)
    k = np.zeros((H, SLOTS, 128))
    v = np.zeros((H, SLOTS, 128))
    q = np.zeros((H * G, 128))
    big = oracle.KV8_QMAX[kind]
    for h in range(H):
        k[h, :, 0] = rng.choice(code_values(kind), SLOTS) * \
            rng.choice([-1.0, 1.0], SLOTS)
        for g in range(G):
            # scores of at most 2 (so 4 apart): |q| big / sqrt(128) <= 2
            top = np.floor(np.log2(2 * np.sqrt(128) / big))
            q[h * G + g, 0] = 2.0 ** (top - g % 4)
        for d in range(128):
            s = k[h, :, 0] * q[h * G + d % G, 0] / np.sqrt(128)
            v[h, :, d] = cancelling(np.exp(s), kind, rng)
    return k, v, q


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("H,G", [(12, 1), (6, 2), (3, 4), (2, 8), (2, 16),
                                 (2, 11)])
def test_weights_are_not_rounded_to_few_bits(cuda_dev, kind, H, G):
    k, v, q = setting(kind, H, G)
    L = 128
    c = ops.kv8_cache(1, L, H, dtype=DT[kind])
    for codes, x in ((c.k, k), (c.v, v)):
        codes[0, :, :SLOTS] = torch.tensor(x, device="cuda").to(DT[kind])
        assert np.array_equal(codes[0, :, :SLOTS].double().cpu().numpy(), x)
    c.k_scale.fill_(1.0)
    c.v_scale.fill_(1.0)
    i32 = lambda n: torch.tensor([n], dtype=torch.int32, device="cuda")
    qt = torch.tensor(q, device="cuda").bfloat16()[None].contiguous()
    out, lse = ops.kv8_decode(qt, c, i32(0), i32(SLOTS), i32(0),
                              ops.rope_table(1e4, 4))
    torch.cuda.synchronize()
    assert ops.last_status() == ops.OK
    got = out[0].double().cpu().numpy()
    near = 0
    for i in range(H * G):
        h = i // G
        o, l, w = oracle.kv8_attend(q[i], k[h], v[h], np.ones(1), np.ones(1),
                                    np.arange(SLOTS))
        near += (np.abs(o) < 2 ** -9 * w).sum()
        assert abs(lse[0, i].item() - l) <= 2 ** -20 * (1 + abs(l))
        tol = 2 ** -8 * np.abs(o) + 2 ** -15.5 * w
        assert (np.abs(got[i] - o) <= tol).all(), \
            (i, (np.abs(got[i] - o) / tol).max())
    assert near >= 64 * H       # the sums do cancel
