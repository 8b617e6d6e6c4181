"""The quantised key/value cache on the GPU, through the binding and the C ABI, against the float64 oracle.

Tolerances, derived from the arithmetic:
  codes, params : the device rounds max - z, x - z and both quotients to fp32. Params are equal to the oracle's. A
            quotient below 256 is off by at most 256 * 3 * 2^-24 < 2^-14 (three roundings), so codes are equal
            wherever the oracle's quotient is further than 2^-14 from a tie, and off by one at most elsewhere.
  read    : bf16(fp32(n s + z)): n s is exact in fp32, one fp32 rounding (2^-24 of |n s| + |z|), one bf16 (2^-8 of the
            value).
  lse     : scores are fp32 sums of under 160 products (128 dims, the groups' terms), in any order and with each
            partial sum rounded or truncated at 2^-23: off by at most dS = 160 * 2^-23 * A with A the sum of the
            terms' sizes, scale * sum_d |q_d| (|z| + c s), where c = 2 * 2^bits covers codes that are carried with
            an offset of up to 2^bits + 16. lse is off by the largest dS of its keys, plus the fp32 rounding of
            the running max and sum (2^-20, and 2^-22 of its value).
  o       : one bf16 rounding, 2^-8 |o|; each weight is off by 2 dS + 2^-14 of itself (exp2 and the running sums in
            fp32), counted against sum_j p_j (|z| + c s); and the product of a weight and a scale is rounded to fp16,
            2^-11 of itself, before it multiplies a code, centred or not, of at most 2^bits: 2^-11 sum_j p_j 2^bits s.
            (One below 2^-14 of the largest of its row and group is off by up to 2^-25 of that largest: of 2^12 keys
            together within the 2^-14 sum_j p_j 2 * 2^bits s above.)
"""
import numpy as np
import pytest
import torch

import causal_self_attention_bf16_b200 as attn
from oracle import decode_forward_kvq, dequantize, quantize, unpack_codes

pytestmark = pytest.mark.gpu

BITS_GROUPS = [(b, g) for b in (4, 8) for g in (32, 64, 128)]


def cpu(t):
    return t.detach().to("cpu", torch.float64).numpy()


def randn(shape, seed, rows=0.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    return (x * torch.exp(rows * torch.randn((*shape[:-1], 1), generator=g))).to(torch.bfloat16)


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def clean():
    torch.cuda.synchronize()
    assert attn.get_device_error() == 0


def poisoned(B, Hkv, Tk, bits, group, seed=0):
    """A cache whose rows hold arbitrary codes and NaN params, as memory that was never written may."""
    c = attn.kvq_cache(B, Hkv, Tk, bits, group)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in (c.k_codes, c.v_codes):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    c.k_params.fill_(float("nan"))
    c.v_params.fill_(float("nan"))
    return c


def check_row(x, codes, params, bits, group, what):
    """Rows x [..., 128] against their codes and params."""
    n, s, z, tie = quantize(x, bits, group)
    got = unpack_codes(codes.cpu().numpy(), bits)
    p = cpu(params)
    assert np.array_equal(p[..., 0], s, equal_nan=True) and np.array_equal(p[..., 1], z, equal_nan=True), what
    off = np.abs(got - n)
    assert (off <= 1).all() and (off[tie > 2.0 ** -14] == 0).all(), f"{what}: codes off by {off.max()}"


# ---------------------------------------------------------------------------------------------- write

@pytest.mark.parametrize("bits,group", BITS_GROUPS)
@pytest.mark.parametrize("B,T,Hkv,Tk,lens", [
    (1, 1, 1, 1, [1]),                       # the smallest call
    (3, 1, 2, 40, [1, 17, 40]),              # one new token each
    (2, 37, 3, 100, [37, 99]),               # a prompt, and tokens after others
    (4, 9, 5, 9, [9, 4, 0, 1]),              # left padding, an empty sequence
    (3, 20, 1, 12, [12, 40, -3]),            # more tokens than positions, lengths outside [0, Tk]
])
def test_write_matches_the_format(bits, group, B, T, Hkv, Tk, lens):
    k, v = randn((B, T, Hkv, 128), 1).cuda(), randn((B, T, Hkv, 128), 2).cuda()
    cache = poisoned(B, Hkv, Tk, bits, group)
    before = [t.clone() for t in cache]
    attn.kvq_write(cache, k, v, ints(lens))
    clean()
    written = torch.zeros((B, Hkv, Tk), dtype=torch.bool)
    for b, L in enumerate(min(max(L, 0), Tk) for L in lens):
        i0 = max(0, T - L)
        written[b, :, L - T + i0:L] = True
        for x, codes, params, name in ((k, *cache[:2], "k"), (v, *cache[2:], "v")):
            check_row(x[b, i0:].cpu(), codes[b, :, L - T + i0:L].transpose(0, 1),
                      params[b, :, L - T + i0:L].transpose(0, 1), bits, group, f"{name} b={b}")
    for t, old in zip(cache, before):        # every other row is left as it was (bit for bit: NaN params too)
        flat = lambda x: x.view(torch.uint8).cpu().reshape(B, Hkv, Tk, -1)[~written]  # noqa: E731
        assert torch.equal(flat(t), flat(old))


@pytest.mark.parametrize("bits,group", [(4, 32), (8, 128)])
def test_write_unusual_rows(bits, group):
    """Constant rows, grids that come back exactly, ties, NaN and infinities, overflowing and subnormal ranges."""
    x = torch.zeros(12, 128)
    x[1] = 3.5
    x[2] = torch.arange(128).remainder(16) * 0.25 - 2
    x[3] = torch.arange(128).remainder(31) * 0.5            # halves of the 4-bit step: ties
    x[4, 7], x[5, 7], x[6, 7] = float("nan"), float("inf"), -float("inf")
    x[7, 3], x[7, 4] = 3e38, -3e38
    x[8, 0] = 1e-40
    x[9] = torch.linspace(-1, 1, 128) * 1e-38
    x[10] = torch.linspace(1, 2, 128) * 1e38
    x[11, 64] = -1e-3
    x = x.to(torch.bfloat16).reshape(1, 12, 1, 128).cuda()
    cache = attn.kvq_cache(1, 1, 12, bits, group)
    attn.kvq_write(cache, x, -x, ints([12]))
    clean()
    check_row(x[0, :, 0].cpu(), cache.k_codes[0, 0], cache.k_params[0, 0], bits, group, "k")
    check_row(-x[0, :, 0].cpu(), cache.v_codes[0, 0], cache.v_params[0, 0], bits, group, "v")


@pytest.mark.parametrize("bits,group", BITS_GROUPS)
def test_write_codes_are_the_formula_bit_for_bit(bits, group):
    """Codes and params equal the format's fp32 operations made one by one on the CPU (IEEE divisions), ties included:
    rows of every size (2^-90 to 2^90), on coarse grids where ties are common, and each of the 128 scale mantissas."""
    g = torch.Generator().manual_seed(100 * bits + group)
    x = torch.randn(4000, 128, generator=g) * torch.exp2(torch.randint(-90, 91, (4000, 1), generator=g).float())
    grid = torch.randint(-300, 300, (3000, 128), generator=g).float()
    grid *= torch.exp2(torch.randint(-20, 20, (3000, 1), generator=g).float())
    # a span of m * 2^k * levels has the scale m * 2^k: m in [1, 2) in steps of 2^-7, the rest of the group on halves
    m = 1 + torch.arange(128).float() / 128
    lanes = torch.arange(128) % group
    steps = torch.where(lanes == 0, torch.tensor(0.0), torch.where(lanes == 1, torch.tensor(float(2 ** bits - 1)),
                                                                  (lanes % (2 ** bits - 1)).float() + 0.5))
    halves = (m[:, None] * steps[None, :])
    x = torch.cat([x, grid, halves, x[:500] + 1000 * x[:500, :1]]).to(torch.bfloat16)
    levels = float(2 ** bits - 1)
    r = x.float().reshape(-1, 128 // group, group)
    z = r.amin(-1, keepdim=True)
    span = r.amax(-1, keepdim=True) - z
    s = ((span / torch.full_like(span, levels)).view(torch.int32) + 0xFFFF & -65536).view(torch.float32)
    n = torch.where(s > 0, torch.round((r - z) / s), torch.zeros_like(r)).clamp(max=levels).reshape(-1, 128).long()
    rows = x.shape[0]
    cache = attn.kvq_cache(1, 1, rows, bits, group)
    attn.kvq_write(cache, x.reshape(1, rows, 1, 128).cuda(), (-x).reshape(1, rows, 1, 128).cuda(), ints([rows]))
    clean()
    assert np.array_equal(unpack_codes(cache.k_codes[0, 0].cpu().numpy(), bits), n.numpy())
    assert torch.equal(cache.k_params[0, 0].cpu().float(), torch.cat([s, z], -1))


@pytest.mark.parametrize("T", [701, 4503])
def test_write_many_rows(T):
    """Enough rows for many blocks (T = 4503: for some that take several sets of rows), checked against the oracle on a
    sample and for every row's error bound."""
    B, Hkv, bits, group, lens = 3, 10, 4, 64, (T, T + 99, T + 199)
    k, v = randn((B, T, Hkv, 128), 5).cuda(), randn((B, T, Hkv, 128), 6).cuda()
    cache = attn.kvq_cache(B, Hkv, T + 199, bits, group)
    attn.kvq_write(cache, k, v, ints(lens))
    rk, rv = attn.kvq_read(cache, T, ints(lens))
    clean()
    for b, L in enumerate(lens):
        for h in (0, 7):
            check_row(k[b, :, h].cpu(), cache.k_codes[b, h, L - T:L], cache.k_params[b, h, L - T:L], bits, group, "k")
    for x, y, p in ((k, rk, cache.k_params), (v, rv, cache.v_params)):
        step = torch.stack([p[b, :, L - T:L, :, 0] for b, L in enumerate(lens)]).transpose(1, 2).float()
        bound = step.repeat_interleave(group, -1) / 2 + 2.0 ** -7 * x.float().abs() + 2.0 ** -8 * step.amax(-1, True)
        assert ((x.float() - y.float()).abs() <= bound).all()


# ---------------------------------------------------------------------------------------------- read

@pytest.mark.parametrize("bits,group", BITS_GROUPS)
@pytest.mark.parametrize("B,T,Hkv,Tk,lens", [
    (1, 1, 1, 1, [1]), (1, 1, 1, 1, None), (3, 5, 2, 40, [5, 2, 40]), (2, 33, 3, 33, None), (2, 7, 5, 33, None),
    (4, 50, 3, 20, [20, 0, -1, 99])])
def test_read_matches_the_values(bits, group, B, T, Hkv, Tk, lens):
    cache = poisoned(B, Hkv, Tk, bits, group, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    for t in (cache.k_params, cache.v_params):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        t[..., 0].abs_()
    out = [torch.full((B, T, Hkv, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    attn.kvq_read(cache, T, None if lens is None else ints(lens), *out)
    clean()
    for y, codes, params in ((out[0], *cache[:2]), (out[1], *cache[2:])):
        ref = dequantize(codes.cpu().numpy(), params.cpu(), bits).transpose(0, 2, 1, 3)
        size = (dequantize(codes.cpu().numpy(), params.cpu().abs(), bits)).transpose(0, 2, 1, 3)
        for b in range(B):
            L = T if lens is None else min(max(lens[b], 0), Tk)
            i0 = max(0, T - L)
            assert (cpu(y[b, :i0]) == 0).all()
            r, z = ref[b, L - T + i0:L], size[b, L - T + i0:L]
            assert (np.abs(cpu(y[b, i0:]) - r) <= 2.0 ** -8 * np.abs(r) + 2.0 ** -23 * z).all()


def test_read_whole_cache_by_default():
    cache = attn.kvq_cache(2, 3, 11, 8, 64)
    k = randn((2, 11, 3, 128), 8).cuda()
    attn.kvq_write(cache, k, k, ints([11, 11]))
    a, b = attn.kvq_read(cache), attn.kvq_read(cache, 11, ints([11, 11]))
    clean()
    assert a[0].shape == (2, 11, 3, 128) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------------------------------------- decode

def filled(B, Hkv, Tk, bits, group, lens, seed, tail_nan=True):
    """A cache holding random rows; past each sequence's length, rows of NaN params (never to be used)."""
    cache = attn.kvq_cache(B, Hkv, Tk, bits, group)
    attn.kvq_write(cache, randn((B, Tk, Hkv, 128), seed, 0.2).cuda(), randn((B, Tk, Hkv, 128), seed + 1).cuda(),
                   ints([Tk] * B))
    if tail_nan:
        for b, L in enumerate(lens):
            L = min(max(L, 0), Tk)
            cache.k_params[b, :, L:] = float("nan")
            cache.v_params[b, :, L:] = float("nan")
            cache.k_codes[b, :, L:] = 255
            cache.v_codes[b, :, L:] = 255
    return cache


def check_decode(q, cache, lens, scale, window, o, lse, what):
    q64, (kc, kp, vc, vp) = cpu(q), [t.cpu() for t in cache]
    B, Tq, H, D = q64.shape
    Hkv, Tk, bits = kc.shape[1], kc.shape[2], kc.shape[3] * 8 // D
    G = H // Hkv
    o, lse = cpu(o), cpu(lse)
    O, LSE = decode_forward_kvq(q64, (kc.numpy(), kp, vc.numpy(), vp), lens, scale, window)
    c = 2.0 * 2 ** bits
    for b, L in enumerate(min(max(L, 0), Tk) for L in lens):
        for h in range(H):
            k, v = (dequantize(t[b, h // G, :L].numpy(), p[b, h // G, :L], bits) for t, p in ((kc, kp), (vc, vp)))
            ks, vs = (np.repeat(np.abs(cpu(p[b, h // G, :L, :, 1])) + c * np.abs(cpu(p[b, h // G, :L, :, 0])),
                                D // p.shape[3], -1) for p in (kp, vp))
            vstep = np.repeat(np.abs(cpu(vp[b, h // G, :L, :, 0])), D // vp.shape[3], -1)
            for i in range(Tq):
                last = L - Tq + i
                w = f"{what} b={b} h={h} i={i}"
                if last < 0:
                    assert (o[b, i, h] == 0).all() and lse[b, h, i] == -np.inf, w
                    continue
                first = 0 if window is None else max(0, last - window)
                dS = 160 * 2.0 ** -23 * scale * (ks[first:last + 1] @ np.abs(q64[b, i, h])).max()
                assert abs(lse[b, h, i] - LSE[b, h, i]) <= dS + 2.0 ** -20 + 2.0 ** -22 * abs(LSE[b, h, i]), w
                p = np.exp(scale * (k[first:last + 1] @ q64[b, i, h]) - LSE[b, h, i])
                tol = 2.0 ** -8 * np.abs(O[b, i, h]) + (2 * dS + 2.0 ** -14) * (p @ vs[first:last + 1])
                tol += 2.0 ** -11 * 2 ** bits * (p @ vstep[first:last + 1])
                err = np.abs(o[b, i, h] - O[b, i, h])
                assert (err <= tol).all(), f"{w}: {(err / tol).max():.2f} of the tolerance"


def run_decode(B, H, Hkv, Tq, Tk, bits, group, lens, window=None, scale=128 ** -0.5, seed=10):
    cache = filled(B, Hkv, Tk, bits, group, lens, seed)
    q = randn((B, Tq, H, 128), seed + 2, 0.2).cuda()
    o = torch.full_like(q, float("nan"))
    lse = torch.full((B, H, Tq), float("nan"), device="cuda")
    attn.attn_decode_kvq(q, cache, ints(lens), scale, o, lse, window=window)
    clean()
    check_decode(q, cache, lens, scale, window, o, lse, f"{B, H, Hkv, Tq, Tk, bits, group, lens, window}")
    return q, cache, o, lse


@pytest.mark.parametrize("bits,group", BITS_GROUPS)
@pytest.mark.parametrize("B,H,Hkv,Tq,Tk,lens", [
    (1, 1, 1, 1, 1, [1]),                                # one key
    (3, 4, 2, 2, 300, [300, 1, 77]),                     # grouped heads, two tokens, one below position 0
    (4, 3, 3, 1, 130, [0, 16, 17, 129]),                 # an empty sequence, lengths around a tile's ends
    (2, 10, 2, 1, 999, [999, 640]),                      # five rows
    (2, 8, 1, 4, 515, [515, 3]),                         # 32 rows
    (1, 6, 2, 3, 64, [70]),                              # nine rows, a length past the capacity
])
def test_decode_matches_oracle(bits, group, B, H, Hkv, Tq, Tk, lens):
    run_decode(B, H, Hkv, Tq, Tk, bits, group, lens)


@pytest.mark.parametrize("R", [1, 2, 3, 4, 5, 7, 8, 9, 12, 15, 16, 17, 24, 25, 31, 32])
@pytest.mark.parametrize("bits", [4, 8])
def test_decode_every_row_count(R, bits):
    run_decode(2, R, 1, 1, 200, bits, 64, [200, 33], seed=R)


@pytest.mark.parametrize("window", [0, 1, 15, 16, 100, 699, 700, 5000, 2 ** 31 - 1])
@pytest.mark.parametrize("bits,group", [(4, 64), (8, 32)])
def test_decode_window(window, bits, group):
    run_decode(3, 4, 2, 3, 700, bits, group, [700, 2, 333], window=window)


@pytest.mark.parametrize("Tq", [2, 5, 16, 32])
def test_decode_several_tokens(Tq):
    run_decode(3, 2, 2, Tq, 100, 4, 32, [100, Tq, Tq // 2])


@pytest.mark.parametrize("bits,group,Hkv,window", [(4, 32, 1, None), (8, 128, 2, None), (4, 64, 1, 3000)])
def test_decode_long_cache(bits, group, Hkv, window):
    """Few heads over a long cache: the work is split along it."""
    run_decode(1, 2, Hkv, 1, 20011, bits, group, [19997], window=window)
    run_decode(2, 2 * Hkv, Hkv, 2, 9000, bits, group, [9000, 1], window=window)


def test_decode_ragged_batch():
    """Many sequences of very different lengths: each must be seen whole, once."""
    lens = [(37 * i * i) % 501 for i in range(60)]
    run_decode(60, 2, 2, 1, 500, 4, 64, lens)


@pytest.mark.parametrize("bits,group,Tk", [(4, 64, 20), (4, 32, 70), (8, 128, 33), (8, 64, 700)])
def test_decode_many_short_sequences(bits, group, Tk):
    """Hundreds of sequences of 0 to Tk keys: several units to a warp, and sequences without keys between them."""
    lens = [(13 * i * i + i) % (Tk + 1) if i % 7 else 0 for i in range(400)]
    run_decode(400, 2, 1, 1, Tk, bits, group, lens)


@pytest.mark.parametrize("Tk", [768, 769])
@pytest.mark.parametrize("H,Tq", [(1, 1), (3, 4), (8, 4)])
def test_decode_on_both_sides_of_the_split_rule(Tk, H, Tq):
    """The same keys in whole units and split over CTAs (a capacity past the rule's limit): the oracle's result, and
    each other's up to the rounding of the joined sums."""
    lens = [700, 31]
    q, cache, o, lse = run_decode(2, H, 1, Tq, Tk, 4, 64, lens)
    wide = attn.kvq_cache(2, 1, 4000, 4, 64)
    for a, b in zip(wide, cache):
        a[:, :, :Tk] = b
    o2, lse2 = attn.attn_decode_kvq(q, wide, ints(lens))
    clean()
    check_decode(q, wide, lens, 128 ** -0.5, None, o2, lse2, "wide")
    assert torch.allclose(lse, lse2, rtol=2 ** -20, atol=2 ** -18)


@pytest.mark.parametrize("T", [1, 3, 64])
def test_more_tokens_than_keys(T):
    """Sequences shorter than the call's tokens, through all three calls."""
    B, Hkv = 3, 2
    lens = [2, 0, 1]
    cache = poisoned(B, Hkv, 5, 8, 32)
    k, v = randn((B, T, Hkv, 128), 200).cuda(), randn((B, T, Hkv, 128), 201).cuda()
    attn.kvq_write(cache, k, v, ints(lens))
    rk, rv = attn.kvq_read(cache, T, ints(lens))
    q = randn((B, min(T, 32), Hkv, 128), 202).cuda()
    o, lse = attn.attn_decode_kvq(q, cache, ints([min(L, T) for L in lens]))
    clean()
    for b, L in enumerate(lens):
        n = min(L, T)
        assert (rk[b, :T - n] == 0).all() and (rv[b, :T - n] == 0).all()
        check_row(k[b, T - n:].cpu(), cache.k_codes[b, :, L - n:L].transpose(0, 1),
                  cache.k_params[b, :, L - n:L].transpose(0, 1), 8, 32, "k")
    if T > 1:  # (with one token only sequence 0's second key is written: its first row is still NaN)
        check_decode(q, cache, lens, 128 ** -0.5, None, o, lse, "short")
    assert (o[1] == 0).all() and (lse[1] == -float("inf")).all()


def test_refusals_on_the_device():
    """What the binding refuses with CUDA tensors in hand; nothing is launched and the cache stays."""
    cache = attn.kvq_cache(2, 3, 8)
    before = [t.clone() for t in cache]
    k = torch.ones(2, 4, 3, 128, dtype=torch.bfloat16, device="cuda")
    q = torch.ones(2, 1, 6, 128, dtype=torch.bfloat16, device="cuda")
    lens = ints([4, 4])
    for call in (lambda: attn.kvq_write(cache, k.half(), k, lens), lambda: attn.kvq_write(cache, k, k[:, :3], lens),
                 lambda: attn.kvq_write(cache, k[:, :, :2].contiguous(), k[:, :, :2].contiguous(), lens),
                 lambda: attn.kvq_write(cache, k[:1], k[:1], lens), lambda: attn.kvq_write(cache, k, k, lens.long()),
                 lambda: attn.kvq_write(cache, k, k, lens.cpu()),
                 lambda: attn.kvq_write(cache, k.transpose(1, 2), k, lens),
                 lambda: attn.kvq_read(cache, 0), lambda: attn.kvq_read(cache, 9),
                 lambda: attn.kvq_read(cache, 4, lens[:1]), lambda: attn.kvq_read(cache, 4, lens, k.float(), k),
                 lambda: attn.kvq_read(cache, 4, lens, k[:, :3], k),
                 lambda: attn.attn_decode_kvq(q.float(), cache, lens), lambda: attn.attn_decode_kvq(q[:1], cache, lens),
                 lambda: attn.attn_decode_kvq(q, cache, lens, window=-1),
                 lambda: attn.attn_decode_kvq(q, cache, lens, o=q[:, :, :3]),
                 lambda: attn.attn_decode_kvq(q, cache, lens, lse=torch.empty(2, 6, 2, device="cuda")),
                 lambda: attn.attn_decode_kvq(q, cache, lens, workspace=torch.empty(64))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: attn.attn_decode_kvq(q[:, :, :5].contiguous(), cache, lens),             # 5 heads over 3
                 lambda: attn.attn_decode_kvq(q.repeat(1, 17, 1, 1), cache, lens),                # 34 rows
                 lambda: attn.attn_decode_kvq(q, cache, lens, 0.0), lambda: attn.attn_decode_kvq(q, cache, lens, o=q),
                 lambda: attn.kvq_read(cache, 4, lens, k, k)):                                    # one output twice
        with pytest.raises(attn.AttnError):
            call()
    clean()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(cache, before))


def test_decode_large_scores():
    """Scores in the hundreds: one key takes all the weight, nothing overflows."""
    run_decode(2, 2, 1, 1, 300, 8, 64, [300, 299], scale=5.0)
    run_decode(2, 2, 1, 1, 300, 4, 32, [300, 299], scale=1e-6)


def test_decode_nan_reaches_only_the_rows_that_see_it():
    B, H, Hkv, Tq, Tk = 2, 4, 2, 2, 90
    lens = [90, 50]
    cache = filled(B, Hkv, Tk, 4, 64, lens, 20)
    q = randn((B, Tq, H, 128), 21).cuda()
    good, good_lse = attn.attn_decode_kvq(q, cache, ints(lens))
    cache.k_params[0, 0, 89] = float("nan")              # the newest key of sequence 0, head 0: only token 1 sees it
    cache.v_params[1, 1, 10, 1] = float("nan")           # dims 64.. of a value of sequence 1, head 1
    o, lse = attn.attn_decode_kvq(q, cache, ints(lens))
    clean()
    bad_o = torch.zeros_like(o, dtype=torch.bool)
    bad_o[0, 1, 0:2] = True
    bad_o[1, :, 2:4, 64:] = True
    bad_l = torch.zeros_like(lse, dtype=torch.bool)
    bad_l[0, 0:2, 1] = True
    assert torch.equal(o.isnan(), bad_o) and torch.equal(lse.isnan(), bad_l)
    assert torch.equal(o[~bad_o], good[~bad_o]) and torch.equal(lse[~bad_l], good_lse[~bad_l])


def test_decode_extreme_scales():
    """Groups whose scales differ by many orders of magnitude, and tiny and huge values."""
    B, H, Hkv, Tk = 1, 2, 1, 120
    k, v = randn((B, Tk, Hkv, 128), 30).cuda(), randn((B, Tk, Hkv, 128), 31).float().cuda()
    v[..., :32] *= 1e30
    v[..., 32:64] *= 1e-30
    v[..., 64:96] += 1000
    for bits in (4, 8):
        cache = attn.kvq_cache(B, Hkv, Tk, bits, 32)
        attn.kvq_write(cache, k, v.to(torch.bfloat16), ints([Tk]))
        q = randn((B, 1, H, 128), 32).cuda()
        o, lse = attn.attn_decode_kvq(q, cache, ints([Tk]))
        clean()
        check_decode(q, cache, [Tk], 128 ** -0.5, None, o, lse, f"extreme scales {bits}")


@pytest.mark.parametrize("bits,group", BITS_GROUPS)
def test_decode_of_a_cache_filled_by_others(bits, group):
    """Any codes and params are n * s + z: scales of both signs, all negative, and groups of sizes far apart."""
    B, H, Hkv, Tq, Tk, lens = 3, 4, 2, 2, 200, [200, 37, 133]
    cache = attn.kvq_cache(B, Hkv, Tk, bits, group)
    g = torch.Generator(device="cuda").manual_seed(bits + group)
    for codes, params in ((cache.k_codes, cache.k_params), (cache.v_codes, cache.v_params)):
        codes.copy_(torch.randint(0, 256, codes.shape, generator=g, device="cuda", dtype=torch.uint8))
        params.copy_(torch.randn(params.shape, generator=g, device="cuda") * 2.0 ** (1 - bits))
    cache.k_params[1, ..., 0].abs_().neg_()
    cache.v_params[1, ..., 0].abs_().neg_()
    cache.v_params[2, :, 50:90] *= 2.0 ** 20
    cache.v_params[2, :, 90:] *= -2.0 ** 40
    q = randn((B, Tq, H, 128), 33).cuda()
    o, lse = attn.attn_decode_kvq(q, cache, ints(lens))
    clean()
    check_decode(q, cache, lens, 128 ** -0.5, None, o, lse, f"by others {bits} {group}")


@pytest.mark.parametrize("bits,group", BITS_GROUPS)
def test_decode_values_of_other_sizes_where_they_do_not_count(bits, group):
    """Values of very different sizes: at a key that only some rows see, at one that some rows hardly weigh, and at keys
    that later ones leave far behind. Each row's result holds to its own weights."""
    B, H, Hkv, Tq, Tk, lens = 3, 4, 2, 2, 300, [300, 290, 300]
    cache = filled(B, Hkv, Tk, bits, group, lens, 140)
    cache.v_params[0, :, 299] *= 2.0 ** 40               # the newest key: token 0 does not see it
    cache.v_params[1, :, 7] *= 2.0 ** 30                 # heads 0 and 2 weigh it by about 2^-100, the others like any
    q = randn((B, Tq, H, 128), 142).cuda()
    q[1, :, 0::2], q[1, :, 1::2] = 1, 0
    cache.k_params[1, :, 7, :, 0], cache.k_params[1, :, 7, :, 1] = 0, -6
    cache.k_params[1, 1, 8:280, :, 1] += 0.01
    q[2] = 1                                             # scores that rise by about 2^100 from end to end
    cache.k_params[2, ..., 0] *= 0.01
    cache.k_params[2, ..., 1] = torch.linspace(-3, 3, Tk, device="cuda")[None, :, None]
    cache.v_params[2, 0, :40] *= 2.0 ** 40
    cache.v_params[2, 1, 100] *= -2.0 ** 24
    o, lse = attn.attn_decode_kvq(q, cache, ints(lens))
    clean()
    check_decode(q, cache, lens, 128 ** -0.5, None, o, lse, f"sizes {bits} {group}")


def test_decode_is_repeatable_and_leaves_its_inputs():
    q, cache, o, lse = run_decode(5, 4, 2, 1, 3000, 4, 32, [3000, 10, 1500, 2999, 64])
    before = [t.clone() for t in cache]
    ws = torch.full((attn.load_library().attn_decode_kvq_workspace_bytes(5, 4, 2, 1, 3000, 128),), 255,
                    dtype=torch.uint8, device="cuda")    # NaN as fp32: its contents must not matter
    for _ in range(3):
        o2, lse2 = attn.attn_decode_kvq(q, cache, ints([3000, 10, 1500, 2999, 64]), workspace=ws)
        clean()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(cache, before))


def test_decode_workspace_and_neighbours_are_not_overrun():
    """Outputs and workspace in the middle of larger buffers: the bytes around them stay."""
    B, H, Hkv, Tq, Tk, lens = 2, 6, 3, 2, 5000, [4999, 700]
    cache = filled(B, Hkv, Tk, 4, 64, lens, 40)
    q = randn((B, Tq, H, 128), 41).cuda()
    n = int(attn.load_library().attn_decode_kvq_workspace_bytes(B, H, Hkv, Tq, Tk, 128))
    ws = torch.full((n + 512,), 77, dtype=torch.uint8, device="cuda")
    ob = torch.full((q.numel() + 256,), 7.0, dtype=torch.bfloat16, device="cuda")
    lb = torch.full((B * H * Tq + 64,), 7.0, device="cuda")
    o, lse = ob[128:-128].view_as(q), lb[32:-32].view(B, H, Tq)
    attn.attn_decode_kvq(q, cache, ints(lens), None, o, lse, ws[256:256 + n])
    clean()
    check_decode(q, cache, lens, 128 ** -0.5, None, o, lse, "middle")
    assert (ws[:256] == 77).all() and (ws[256 + n:] == 77).all()
    assert (ob[:128] == 7).all() and (ob[-128:] == 7).all() and (lb[:32] == 7).all() and (lb[-32:] == 7).all()


# ---------------------------------------------------------------------------------------------- together, as used

def test_prompt_then_steps():
    """A prompt written, then token by token: prologue, write, decode. Each step against the float64 oracle on the
    codes the cache holds, and the codes against the rows that the prologue gave."""
    B, H, Hkv, bits, group, Tk = 3, 4, 2, 4, 32, 64
    lens = torch.tensor([20, 7, 1], dtype=torch.int32, device="cuda")
    P = 20                                               # left-padded prompts
    raw_q, raw_k, v = (randn((B, P, h, 128), 50 + h + j).cuda() for j, h in enumerate((H, Hkv, Hkv)))
    cache = poisoned(B, Hkv, Tk, bits, group)
    _, k = attn.qk_norm_rope(raw_q, raw_k, pos_offsets=lens - P)
    attn.kvq_write(cache, k, v, lens)
    for step in range(4):
        lens = lens + 1
        rq, rk, v = (randn((B, 1, h, 128), 60 + 10 * step + j).cuda() for j, h in enumerate((H, Hkv, Hkv)))
        q, k = attn.qk_norm_rope(rq, rk, pos_offsets=lens - 1)
        attn.kvq_write(cache, k, v, lens)
        o, lse = attn.attn_decode_kvq(q, cache, lens)
        clean()
        L = lens.tolist()
        for b in range(B):
            check_row(k[b, 0].cpu(), cache.k_codes[b, :, L[b] - 1], cache.k_params[b, :, L[b] - 1], bits, group, "step")
        check_decode(q, cache, L, 128 ** -0.5, None, o, lse, f"step {step}")
    # the bf16 decode over the cache read back: the same values up to their rounding to bf16
    kb, vb = attn.kvq_read(cache)
    o_b, _ = attn.attn_decode(q, kb, vb, lens)
    clean()
    assert (o_b.float() - o.float()).norm() <= 2.0 ** -6 * o.float().norm()


def test_steps_captured_in_a_graph():
    """A captured step (lengths + 1, write, decode) replayed against the same steps run one by one."""
    B, H, Hkv, Tk = 2, 4, 2, 300
    def state():
        lens = ints([250, 3])
        return lens, filled(B, Hkv, Tk, 4, 64, [250, 3], 70)
    ks, vs, qs = (randn((5, B, 1, h, 128), 71 + h + j).cuda() for j, h in enumerate((Hkv, Hkv, H)))
    lens, cache = state()
    ref = []
    for i in range(5):
        lens += 1
        attn.kvq_write(cache, ks[i], vs[i], lens)
        ref.append([t.clone() for t in attn.attn_decode_kvq(qs[i], cache, lens)])
    lens, cache = state()
    k, v, q = ks[0].clone(), vs[0].clone(), qs[0].clone()
    o, lse = torch.empty_like(q), torch.empty((B, H, 1), device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens += 1
        attn.kvq_write(cache, k, v, lens)
        attn.attn_decode_kvq(q, cache, lens, None, o, lse)
    for i in range(5):
        for dst, src in ((k, ks), (v, vs), (q, qs)):
            dst.copy_(src[i])
        graph.replay()
        clean()
        assert torch.equal(o, ref[i][0]) and torch.equal(lse, ref[i][1]), f"step {i}"


def test_capture_of_a_forked_step_and_of_two_graphs():
    """A captured step whose calls follow copies, a memset and another stream's kernels: the write on a side stream that
    joins before the decode, default workspace and outputs. Two such graphs replayed in turn keep their results apart."""
    B, H, Hkv, Tk, lens0 = 3, 4, 2, 3000, [2000, 5, 2999]
    k, v, q = (randn((2, B, 1, h, 128), 100 + j).cuda() for j, h in enumerate((Hkv, Hkv, H)))
    caches = [filled(B, Hkv, Tk, bits, 64, lens0, 110 + bits) for bits in (4, 8)]
    ref = []
    for i, cache in enumerate(caches):
        copy = tuple(t.clone() for t in cache)
        attn.kvq_write(copy, k[i], v[i], ints(lens0) + 1)
        ref.append((*attn.attn_decode_kvq(q[i], copy, ints(lens0) + 1), *attn.kvq_read(copy, 3, ints(lens0))))
    lens_in, lens, qs, side = ints(lens0), ints([0] * B), torch.empty_like(q[0]), torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i, cache in enumerate(caches):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lens.copy_(lens_in)
            lens += 1
            side.wait_stream(torch.cuda.current_stream())
            attn.kvq_write(cache, k[i], v[i], lens, stream=side)
            qs.zero_()
            qs.copy_(q[i])
            torch.cuda.current_stream().wait_stream(side)
            o, lse = attn.attn_decode_kvq(qs, cache, lens)
            lens -= 1
            outs.append((o, lse, *attn.kvq_read(cache, 3, lens)))
        graphs.append(graph)
    for _ in range(3):
        for graph, out, want in zip(graphs, outs, ref):
            graph.replay()
            clean()
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_calls_on_another_stream():
    """Every call with stream=: ordered on that stream, outputs made there belong to it."""
    B, H, Hkv, Tk = 2, 4, 2, 4000
    k, v, q = (randn((B, n, h, 128), 80 + j).cuda() for j, (n, h) in enumerate(((Tk, Hkv), (Tk, Hkv), (1, H))))
    lens = ints([Tk, 1234])
    cache = attn.kvq_cache(B, Hkv, Tk)
    attn.kvq_write(cache, k, v, ints([Tk, Tk]))
    ref = [*attn.attn_decode_kvq(q, cache, lens), *attn.kvq_read(cache, 7, lens)]
    side = torch.cuda.Stream()
    cache2 = attn.kvq_cache(B, Hkv, Tk)
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        attn.kvq_write(cache2, k, v, ints([Tk, Tk]), stream=side)
        got.append([*attn.attn_decode_kvq(q, cache2, lens, stream=side), *attn.kvq_read(cache2, 7, lens, stream=side)])
    torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")   # memory that the calls let go must not be theirs
    clean()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(ref, g))


def test_two_streams_at_once():
    """Two decodes in flight, each with its own workspace (the binding's default)."""
    a = (randn((1, 1, 8, 128), 90).cuda(), filled(1, 4, 8000, 4, 64, [8000], 91), ints([8000]))
    b = (randn((3, 2, 4, 128), 92).cuda(), filled(3, 4, 2500, 8, 32, [2500, 9, 700], 94), ints([2500, 9, 700]))
    ref = [attn.attn_decode_kvq(*x) for x in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[attn.attn_decode_kvq(*x, stream=s) for x, s in zip((a, b), streams)] for _ in range(10)]
    clean()
    for pair in got:
        for r, g in zip(ref, pair):
            assert torch.equal(r[0], g[0]) and torch.equal(r[1], g[1])


def test_offsets_past_32_bits():
    """A cache whose codes pass 4 GiB a tensor: the last sequence's rows are written, read and attended to."""
    B, Hkv, Tk = 2, 2, (1 << 32) // (128 * 4) + 333       # 8-bit codes: B * Hkv * Tk * 128 bytes > 2^32
    cache = attn.kvq_cache(B, Hkv, Tk, 8, 128)
    lens = ints([5, Tk])
    k, v = randn((B, 40, Hkv, 128), 95).cuda(), randn((B, 40, Hkv, 128), 96).cuda()
    attn.kvq_write(cache, k, v, lens)
    check_row(k[1].cpu(), cache.k_codes[1, :, Tk - 40:].transpose(0, 1), cache.k_params[1, :, Tk - 40:].transpose(0, 1),
              8, 128, "k")
    rk, rv = attn.kvq_read(cache, 40, lens)
    for x, y, p in ((k, rk, cache.k_params), (v, rv, cache.v_params)):
        step = p[1, :, Tk - 40:, :, 0].transpose(0, 1).float()
        assert ((x[1].float() - y[1].float()).abs() <= step / 2 * 1.02 + 2.0 ** -7 * x[1].float().abs()).all()
        assert (y[0, :35] == 0).all()
    q = randn((B, 1, 2, 128), 97).cuda()
    o, lse = attn.attn_decode_kvq(q, cache, lens, window=39)
    clean()
    tail = tuple(torch.stack([t[0, :, :40], t[1, :, Tk - 40:]]) for t in cache)
    check_decode(q, tail, [5, 40], 128 ** -0.5, 39, o, lse, "past 32 bits")
    # every key 0 and every value 1.5: lse is the logarithm of the length, o is 1.5
    cache.k_params.zero_()
    cache.v_params[..., 0] = 0
    cache.v_params[..., 1] = 1.5
    o, lse = attn.attn_decode_kvq(q, cache, lens)
    clean()
    assert (o == 1.5).all()
    assert np.abs(cpu(lse) - np.log([[[5], [5]], [[Tk], [Tk]]])).max() <= 2.0 ** -18
    # the whole cache read back, 8.6 GB a tensor: first, middle and last rows of each sequence
    cache.v_params[1, 1, Tk - 1] = 7
    rk, rv = attn.kvq_read(cache)
    clean()
    assert (rk[:, ::100001] == 0).all() and (rv[:, :-1:100001] == 1.5).all()
    assert (rv[0, -1] == 1.5).all() and (rv[1, -1, 0] == 1.5).all() and (rv[1, -1, 1] >= 7).all()
    del cache, rk, rv
    torch.cuda.empty_cache()
