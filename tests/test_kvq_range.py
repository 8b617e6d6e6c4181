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


@pytest.mark.parametrize("size", [2.0 ** 20, 1e10, 1e25, 1e35, 1e37])
@pytest.mark.parametrize("Tk,Tq", [(20, 1), (700, 3), (6000, 1)])
@pytest.mark.parametrize("bits,group", [(4, 64), (8, 32)])
def test_huge_scores(bits, group, Tk, Tq, size):
    """Scores far past 2^24: of each row's keys the largest one takes all the weight, or those that tie for it do in
    equal parts. A row's scores are its size times the first dim's code, so they are known: lse is the largest and the
    logarithm of how many have it (the rounding of the score and of the base-2 scale: under 2^-20 together), o the mean
    of their values (2^-8 of itself for bf16, 2^-11 * 2^bits * s for the weights)."""
    B, H, Hkv = 2, 6, 2
    g = torch.Generator().manual_seed(bits + Tk)
    cache = attn.kvq_cache(B, Hkv, Tk, bits, group)
    attn.kvq_write(cache, torch.zeros(B, Tk, Hkv, 128, dtype=torch.bfloat16, device="cuda"),
                   randn((B, Tk, Hkv, 128), 5, 0.0).cuda(), ints([Tk] * B))
    n = torch.randint(0, 15, (B, Hkv, Tk), generator=g)
    for at in ((Tk - Tq) // 3, (Tk - Tq) // 2, Tk - Tq):          # seen by every query: the largest, three times
        n[:, :, at] = 15
    cache.k_codes[..., 0] = n.to(torch.uint8).cuda()              # (4 bits: dim 1's code, the high half, is 0)
    cache.k_params[..., 0] = 1
    q = torch.zeros(B, Tq, H, 128)
    q[..., 0] = size * torch.linspace(0.7, 1.3, H)
    q = q.to(torch.bfloat16).cuda()
    o, lse = attn.attn_decode_kvq(q, cache, ints([Tk] * B), 0.0883)
    clean()
    top = 15 * np.float64(np.float32(0.0883)) * cpu(q)[..., 0].transpose(0, 2, 1)
    assert (np.abs(cpu(lse) - top - np.log(3)) <= 2.0 ** -20 * top + 2.0 ** -20).all()
    codes = cache.v_codes
    if bits == 4:
        codes = (codes[..., None] >> torch.tensor([0, 4], device="cuda") & 15).flatten(-2)
    step = cpu(cache.v_params[..., 0].repeat_interleave(group, -1))
    values = cpu(codes) * step + cpu(cache.v_params[..., 1].repeat_interleave(group, -1))
    for b in range(B):
        for h in range(Hkv):
            keys = (n[b, h] == 15).numpy()
            mean = values[b, h, keys].mean(0)
            size_of = (np.abs(values[b, h, keys]) + 2 * 2 ** bits * step[b, h, keys]).mean(0)
            tol = 2.0 ** -8 * np.abs(mean) + (2.0 ** -11 + 2.0 ** -14) * size_of
            assert (np.abs(cpu(o)[b, :, 3 * h:3 * h + 3] - mean) <= tol).all()


@pytest.mark.parametrize("size_q,size_k,scale", [
    (1e37, 2.0 ** -122, SCALE),               # the largest queries, the smallest keys
    (1.0, 2.0 ** -112, 2.0 ** 112 * SCALE),   # the softmax scale in their place
    (2.0 ** 60, 2.0 ** -122, 2.0 ** 62 * SCALE),
    (2.0 ** 100, 2.0 ** -118, 2.0 ** 18 * SCALE),
    (2.0 ** -118, 2.0 ** 100, 2.0 ** 18 * SCALE),
    (2.0 ** -112, 1.0, 2.0 ** 112 * SCALE)])
@pytest.mark.parametrize("bits,group", BITS_GROUPS)
def test_queries_and_scales_of_any_size(bits, group, size_q, size_k, scale):
    """Ordinary scores from queries, keys and a softmax scale whose sizes cancel. Every other head's query is smaller by
    2^12, and one of them 0: their scores are small or 0, not lost to the others' range."""
    B, Tq, H, Hkv, Tk = 2, 2, 8, 2, 300
    q = randn((B, Tq, H, 128), 7, 0.2).double() * size_q
    q[:, :, 1::2] *= 2.0 ** -12
    q[:, :, 3] = 0
    k = randn((B, Tk, Hkv, 128), 8, 0.2).double() * size_k
    decode_of(k, randn((B, Tk, Hkv, 128), 9), q, bits, group, [Tk, 33], scale)
    decode_of(k, randn((B, Tk, Hkv, 128), 9), q, bits, group, [Tk, 33], scale, window=40)


@pytest.mark.parametrize("Tk", [5, 300, 6000])
def test_the_lowest_scores(Tk):
    """Every score -2.22e38 (in base 2 -3.203e38, fp32's end is -3.403e38): keys that are seen and weigh alike, so o is
    the values' mean and lse the score."""
    cache = attn.kvq_cache(1, 1, Tk, 8, 64)
    v = randn((1, Tk, 1, 128), 5, 0.0)
    k = torch.full((1, Tk, 1, 128), -2.609375 * 2.0 ** 59, dtype=torch.bfloat16, device="cuda")
    attn.kvq_write(cache, k, v.cuda(), ints([Tk]))
    q = torch.full((1, 1, 2, 128), 2.0 ** 60, dtype=torch.bfloat16, device="cuda")
    o, lse = attn.attn_decode_kvq(q, cache, ints([Tk]), 1.0)
    clean()
    assert np.allclose(cpu(lse), -2.609375 * 2.0 ** 126, rtol=2.0 ** -20, atol=0)
    step = cpu(cache.v_params[0, 0, :, :, 0]).repeat(64, -1)
    values = cpu(cache.v_codes[0, 0]) * step + cpu(cache.v_params[0, 0, :, :, 1]).repeat(64, -1)
    mean, size = values.mean(0), (np.abs(values) + 2 * 256 * step).mean(0)
    assert (np.abs(cpu(o)[0, 0] - mean) <= 2.0 ** -8 * np.abs(mean) + (2.0 ** -11 + 2.0 ** -14) * size).all()


def test_a_sequence_without_keys_under_the_most_heads():
    """2^27 query heads (o is 32 GiB, 2^31 parts of 16 bytes) over one empty sequence: every row is 0 and -inf."""
    H, Hkv = 1 << 27, 1 << 22
    if torch.cuda.mem_get_info()[0] < (70 << 30):
        pytest.skip("not enough free device memory")
    cache = attn.kvq_cache(1, Hkv, 1, 4, 128)
    q = torch.empty(1, 1, H, 128, dtype=torch.bfloat16, device="cuda")
    o = torch.full_like(q, float("nan"))
    lse = torch.full((1, H, 1), float("nan"), device="cuda")
    attn.attn_decode_kvq(q, cache, ints([0]), o=o, lse=lse)
    clean()
    assert all((part == 0).all() for part in o.view(64, -1)) and (lse == -float("inf")).all()
    del cache, q, o, lse
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["null", "small", "often"])
@pytest.mark.parametrize("bits,group", BITS_GROUPS)
def test_a_heavy_key_of_little_value(bits, group, kind):
    """A key that all rows weigh 2^12 to 2^20 times as much as any other, whose value is 0 (scale 0), or in steps 2^-12 of
    the others' (once, or at every 61st key)."""
    B, H, Hkv, Tk = 2, 4, 2, 3000
    k = randn((B, Tk, Hkv, 128), 11, 0.0).float() * 0.1
    v = randn((B, Tk, Hkv, 128), 12, 0.0).float()
    at = slice(0, None, 61) if kind == "often" else 3
    k[:, at] = 1.0
    v[:, at] *= 0.0 if kind == "null" else 2.0 ** -12
    decode_of(k, v, 1 + 0.1 * randn((B, 1, H, 128), 13, 0.0).float(), bits, group, [Tk, 2000])


@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -112, 2.0 ** -120])
@pytest.mark.parametrize("Tk", [40, 3000])
@pytest.mark.parametrize("bits,group", BITS_GROUPS)
def test_tiny_values(bits, group, Tk, size):
    """Values whose scales are near fp32's smallest normal number keep as many bits as others. (bf16 outputs below
    2^-126 are rounded to 2^-134, which the weights' 2^-14 of 2 * 2^bits s covers.)"""
    k, v = randn((2, Tk, 2, 128), 14, 0.2), randn((2, Tk, 2, 128), 15, 0.2).float() * size
    decode_of(k, v, randn((2, 1, 4, 128), 16, 0.2), bits, group, [Tk, Tk // 3])


@pytest.mark.parametrize("heavy_code,z", [("middle", -1.546875), ("lowest", -1.1015625)])
@pytest.mark.parametrize("bits", [4, 8])
def test_many_light_keys_behind_a_heavy_one(bits, heavy_code, z):
    """A key with most of the weight and 2^17 - 1 keys behind it, of 2^-25.2 or 2^-18 of it each, in one warp's stretch
    (32 rows to a head: 148 x 3 stretches for as many units). The heavy key's value is 0, so they are all of the output.
    A weight is rounded to 2^-11 of itself or 2^-33 of the heaviest and multiplies at most 2^(bits - 1) steps of its
    scale. In each of 8192 matrix products the 16 products and the sum so far, at most the heavy key's code less the
    middle one and all of the light keys' together, are cut off at 2^-23 of the largest. The fp32 sums of the weights
    times the values' middle take 2^14 terms a lane, each rounded by 2^-24 of the sum; the sums of the weights 2^13 (8
    bits) or 2^12 tiles' sums. o is bf16."""
    Hkv, Tk, scale, middle = 148 * 3, 1 << 17, 128 ** -0.5, 2 ** (bits - 1)
    if torch.cuda.mem_get_info()[0] < 2.5 * Hkv * Tk * (32 * bits + 8):
        pytest.skip("not enough free device memory")
    cache = attn.kvq_cache(1, Hkv, Tk, bits, 128)
    code = middle if heavy_code == "middle" else 0
    cache.v_codes.fill_(255)
    cache.v_codes[:, :, 0] = 17 * code if bits == 4 else code
    cache.v_params[..., 0] = 1
    cache.v_params[..., 1] = -code
    cache.k_params[..., 1] = z
    cache.k_params[:, :, 0] = 0
    q = torch.ones(1, 1, 32 * Hkv, 128, dtype=torch.bfloat16, device="cuda")
    o, lse = attn.attn_decode_kvq(q, cache, ints([Tk]), scale)
    clean()
    light = (Tk - 1) * np.exp(z * 128 * np.float64(np.float32(scale)))
    top, total = 2 ** bits - 1, 1 + light
    want = (top - code) * light / total
    sums = max(middle - code, middle * light)
    tol = (2.0 ** -11 * light + 2.0 ** -33 * Tk) * middle + 17 * 8192 * 2.0 ** -23 * sums
    tol += 2.0 ** -10 * ((middle - code) * total + want)
    assert np.abs(cpu(lse) - np.log(total)).max() <= 2.0 ** -11 + 2.0 ** -20
    assert np.abs(cpu(o) - want).max() <= 2.0 ** -8 * want + tol / total, (np.abs(cpu(o) - want).max(), tol, want)
    del cache
    torch.cuda.empty_cache()
