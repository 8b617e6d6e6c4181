"""Decode over the quantised cache at the ends of the numbers' range, where every input is finite and so is the result:
huge and tiny values, queries, scales and scores. Oracle, cases and tolerances of the parity tests (their first lines
derive the tolerances; what is added to them is derived at the test)."""
import numpy as np
import pytest
import torch

import causal_self_attention_bf16_b200 as attn
from test_kvq_parity import BITS_GROUPS, check_decode, clean, cpu, ints, randn

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


def decode_of(k, v, q, bits, group, lens, scale=SCALE, window=None):
    """Rows k, v (on the CPU) written, attended to by q, and checked."""
    B, Tk, Hkv, _ = k.shape
    cache = attn.kvq_cache(B, Hkv, Tk, bits, group)
    attn.kvq_write(cache, k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), ints([Tk] * B))
    q = q.to(torch.bfloat16).cuda()
    o, lse = attn.attn_decode_kvq(q, cache, ints(lens), scale, window=window)
    clean()
    check_decode(q, cache, lens, scale, window, o, lse, f"{bits, group, tuple(k.shape), lens, scale, window}")
    return cache, q, o, lse


@pytest.mark.parametrize("size,Tk", [(1e33, 120), (1e35, 120), (4e33, 5000), (1e37, 5)])
@pytest.mark.parametrize("bits,group", BITS_GROUPS)
def test_huge_values(bits, group, size, Tk):
    """In one warp's unit, in one that a CTA's warps join, and merged from several CTAs. The weighted sums before they
    are divided (weights of at most 2^4, 1 where the keys are one tile's) stay below fp32's largest number."""
    k, v = randn((2, Tk, 2, 128), 1, 0.2), randn((2, Tk, 2, 128), 2, 0.0).float() * size
    decode_of(k, v, randn((2, 1, 4, 128), 3, 0.2), bits, group, [Tk, Tk // 2])
