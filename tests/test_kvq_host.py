"""The quantised key/value cache without a GPU: the float64 oracle against its closed forms, the C ABI's and the
binding's argument checks (all before any CUDA call), and the sizes the host computes."""
import numpy as np
import pytest
import torch

import causal_self_attention_bf16_b200 as attn
from causal_self_attention_bf16_b200 import build as attn_build
from oracle import decode_forward, decode_forward_kvq, dequantize, quantize, round_up_bf16, unpack_codes
from test_abi import fake_ptrs

BITS_GROUPS = [(b, g) for b in (4, 8) for g in (32, 64, 128)]


@pytest.fixture(scope="module")
def lib():
    attn_build.build()
    return attn.load_library()


# ---------------------------------------------------------------------------------------------- the oracle

def test_round_up_bf16_against_torch():
    """Not below its argument, a bf16 number, and the one below it is smaller than the argument."""
    x = np.abs(np.random.default_rng(0).standard_normal(2000)) * np.exp(np.random.default_rng(1).uniform(-80, 80, 2000))
    x = np.concatenate([x, [0.0, 1.0, 1.0 + 2.0 ** -8, 255 / 128, 2.0 ** -133, 1.5 * 2.0 ** -133, 3e-40]])
    up = round_up_bf16(x)
    assert np.array_equal(torch.tensor(up).to(torch.bfloat16).double().numpy(), up)
    assert (up >= x).all()
    bits = torch.tensor(up).to(torch.bfloat16).view(torch.int16)
    below = (bits - 1).view(torch.bfloat16).double().numpy()
    assert (below[up > 0] < x[up > 0]).all()


@pytest.mark.parametrize("bits,group", BITS_GROUPS)
def test_oracle_quantizes_within_half_a_step(bits, group):
    x = torch.randn(50, 128, generator=torch.Generator().manual_seed(bits + group)).to(torch.bfloat16)
    n, s, z, _ = quantize(x, bits, group)
    assert n.min() >= 0 and n.max() <= 2 ** bits - 1
    step = np.repeat(s, group, -1)
    back = n * step + np.repeat(z, group, -1)
    assert (np.abs(back - x.double().numpy()) <= step / 2 * (1 + 1e-12)).all()
    # the least value of a group is held exactly
    low = x.double().numpy().reshape(50, -1, group).min(-1)
    assert np.array_equal(z, low)


def test_oracle_exact_steps_and_constant_groups():
    """Numbers already on a grid of 16 steps come back exactly; a constant group has s = 0."""
    x = torch.arange(128).remainder(16).float().mul(0.25).sub(2).to(torch.bfloat16)[None]
    n, s, z, _ = quantize(x, 4, 64)
    assert np.array_equal(n[0], np.arange(128) % 16) and (s == 0.25).all() and (z == -2).all()
    n, s, z, _ = quantize(torch.full((1, 128), 3.5), 8, 32)
    assert (n == 0).all() and (s == 0).all() and (z == 3.5).all()


def test_oracle_bad_groups_are_nan():
    x = torch.zeros(4, 128)
    x[0, 5], x[1, 40], x[2, 127] = float("nan"), float("inf"), -float("inf")
    x[3, 0], x[3, 1] = 3e38, -3e38                       # max - min overflows fp32
    _, s, z, _ = quantize(x.to(torch.bfloat16), 4, 32)
    bad = np.zeros((4, 4), bool)
    bad[0, 0] = bad[1, 1] = bad[2, 3] = bad[3, 0] = True
    assert np.array_equal(np.isnan(s), bad) and np.array_equal(np.isnan(z), bad)


def test_oracle_code_order():
    assert unpack_codes(np.array([[0x21, 0x43]], np.uint8), 4).tolist() == [[1, 2, 3, 4]]
    assert unpack_codes(np.array([[0x21, 0x43]], np.uint8), 8).tolist() == [[0x21, 0x43]]


def test_oracle_decode_equals_decode_of_the_values():
    """With every code 0 the values are the zeros, constant per group: the bf16 oracle's result on them."""
    rng = np.random.default_rng(3)
    kc = np.zeros((2, 2, 9, 64), np.uint8)
    kp, vp = (np.stack([np.ones((2, 2, 9, 4)), rng.standard_normal((2, 2, 9, 4))], -1) for _ in range(2))
    q = rng.standard_normal((2, 1, 4, 128))
    k, v = (np.repeat(p[..., 1], 32, -1).transpose(0, 2, 1, 3) for p in (kp, vp))
    assert np.array_equal(dequantize(kc, kp, 4).transpose(0, 2, 1, 3), k)
    got, ref = decode_forward_kvq(q, (kc, kp, kc, vp), [9, 3], 0.1), decode_forward(q, k, v, [9, 3], 0.1)
    assert all(np.array_equal(a, b) for a, b in zip(got, ref))


# ---------------------------------------------------------------------------------------------- refusals of the C ABI

B, T, HKV, TK = 2, 5, 3, 40


def write_call(lib, ptrs, **kw):
    names = ["k", "v", "kc", "kp", "vc", "vp", "lens"]
    a = dict(zip(names, ptrs), B=B, T=T, hkv=HKV, Tk=TK, D=128, bits=4, group=32)
    a.update(kw)
    return lib.attn_kvq_write(*[a[n] for n in (*names, "B", "T", "hkv", "Tk", "D", "bits", "group")], None)


def read_call(lib, ptrs, **kw):
    names = ["kc", "kp", "vc", "vp", "lens", "k", "v"]
    a = dict(zip(names, ptrs), B=B, T=T, hkv=HKV, Tk=TK, D=128, bits=4, group=32)
    a.update(kw)
    return lib.attn_kvq_read(*[a[n] for n in (*names, "B", "T", "hkv", "Tk", "D", "bits", "group")], None)


def test_write_and_read_argument_errors(lib):
    for call in (write_call, read_call):
        names = ["k", "v", "kc", "kp", "vc", "vp"]
        p = fake_ptrs(7, 1 << 20)
        for n in names:
            assert call(lib, p, **{n: None}) == 1
        for n in ("B", "T", "hkv", "Tk"):
            assert call(lib, p, **{n: 0}) == 1 and call(lib, p, **{n: -1}) == 1
        assert call(lib, p, D=64) == 2
        for bits in (0, 2, 5, 16):
            assert call(lib, p, bits=bits) == 2
        for group in (0, 16, 48, 256):
            assert call(lib, p, group=group) == 2
        for i in range(7):                               # every buffer on 16 bytes, the lengths on 4
            q = list(p)
            q[i] += 2 if q[i] == p[6 if call is write_call else 4] else 8
            assert call(lib, q) == 3
        assert call(lib, p, B=1 << 20, T=1 << 12) == 2   # more rows than 31 bits count
        assert call(lib, p, B=1 << 20, Tk=1 << 20, hkv=8) == 2
    assert write_call(lib, fake_ptrs(7, 1 << 20), lens=None) == 1
    p = fake_ptrs(7, 1 << 20)
    assert write_call(lib, p, kc=p[0]) == 1              # codes over the new keys
    assert write_call(lib, p, vp=p[1] + 16) == 1         # params inside the new values
    assert write_call(lib, p, vc=p[2]) == 1              # both codes in one place
    assert write_call(lib, p, kp=p[6]) == 1              # params over the lengths
    assert read_call(lib, p, k=p[0]) == 1                # output over codes
    assert read_call(lib, p, v=p[5]) == 1                # output over output
    assert read_call(lib, p, k=p[4]) == 1                # output over the lengths
    assert read_call(lib, p, lens=None, T=TK + 1) == 1   # past the end of the cache


def decode_call(lib, ptrs, wb, **kw):
    names = ["q", "kc", "kp", "vc", "vp", "lens", "o", "lse", "w"]
    a = dict(zip(names, ptrs), wb=wb, B=2, H=8, hkv=2, Tq=2, Tk=1000, D=128, bits=4, group=64, scale=0.088, window=-1)
    a.update(kw)
    return lib.attn_decode_kvq(*[a[n] for n in (*names, "wb", "B", "H", "hkv", "Tq", "Tk", "D", "bits", "group",
                                                "scale", "window")], None)


def test_decode_argument_errors(lib):
    wb = lib.attn_decode_kvq_workspace_bytes(2, 8, 2, 2, 1000, 128)
    assert wb > 0
    p = fake_ptrs(9, max(wb, 1 << 22))
    for n in ("q", "kc", "kp", "vc", "vp", "lens", "o", "lse"):
        assert decode_call(lib, p, wb, **{n: None}) == 1
    for n in ("B", "H", "hkv", "Tq", "Tk"):
        assert decode_call(lib, p, wb, **{n: 0}) == 1
    assert decode_call(lib, p, wb, hkv=3) == 1
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert decode_call(lib, p, wb, scale=scale) == 1
    assert decode_call(lib, p, wb, window=-2) == 1
    assert decode_call(lib, p, wb, D=64) == 2
    assert decode_call(lib, p, wb, bits=3) == 2 and decode_call(lib, p, wb, group=16) == 2
    assert decode_call(lib, p, wb, Tq=9) == 2            # 36 rows to a key/value head
    assert decode_call(lib, p, wb - 1) == 6 and decode_call(lib, p, wb, w=None) == 6
    for i in range(9):
        q = list(p)
        q[i] += 2 if i in (5, 7) else 8                  # the lengths and lse on 4 bytes, the rest on 16
        assert decode_call(lib, q, wb) == 3
    for out in ("o", "lse", "w"):
        for i in (0, 1, 2, 3, 4, 5):
            assert decode_call(lib, p, wb, **{out: p[i]}) == 1
    assert decode_call(lib, p, wb, lse=p[6] + 64) == 1


def test_decode_sizes_refused_by_the_host_queries(lib):
    ws, kern = lib.attn_decode_kvq_workspace_bytes, lib.attn_decode_kvq_kernels
    assert ws(2, 8, 3, 1, 1000, 128) == 0 and ws(2, 64, 1, 1, 1000, 128) == 0 and ws(0, 8, 2, 1, 10, 128) == 0
    assert kern(2, 8, 3, 1, 1000, 128, -1) == 0 and kern(2, 8, 2, 1, 1000, 128, -2) == 0


def test_decode_split_rule(lib):
    """Small calls are whole units, one kernel without a workspace: up to 8 tiles of 16 keys for each of a CTA's 12
    warps where the units fill three quarters of 148 CTAs, else 4 (the warps shared by the row tiles of 8 query rows).
    Others are split over up to 148 CTAs: a span (16 bytes) per CTA, and two pieces of 130 floats per CTA and row."""
    ws, kern = lib.attn_decode_kvq_workspace_bytes, lib.attn_decode_kvq_kernels
    for B, H, hkv, Tq, Tk, whole in ((3, 4, 2, 2, 300, True),      # 6 units of 19 tiles
                                     (1, 10, 10, 1, 768, True),    # 10 units of 48 tiles: 4 a warp
                                     (1, 10, 10, 1, 769, False),
                                     (14, 10, 10, 1, 1536, True),  # 140 units of 96 tiles: 8 a warp
                                     (14, 10, 10, 1, 1537, False),
                                     (64, 10, 10, 1, 300, True),   # 5 units to a CTA, 19 tiles each
                                     (64, 10, 10, 1, 320, False),  # 20 tiles each
                                     (16, 12, 3, 8, 128, True),    # 32 rows: three stretches of 8 tiles
                                     (16, 12, 3, 8, 193, False),
                                     (5000, 1, 1, 1, 16, False)):  # 34 units to a CTA: more than its warps look at
        assert kern(B, H, hkv, Tq, Tk, 128, -1) == (1 if whole else 2), (B, H, hkv, Tq, Tk)
        if whole:
            assert ws(B, H, hkv, Tq, Tk, 128) == 0
        else:
            R = H // hkv * Tq
            slices = 12 // ((R + 7) // 8)
            ctas = min(148, (B * hkv * ((Tk + 15) // 16) + slices - 1) // slices)
            assert ws(B, H, hkv, Tq, Tk, 128) == ctas * 16 + ctas * 2 * R * 130 * 4
    assert kern(64, 10, 10, 1, 2048, 128, -1) == 2 and kern(64, 10, 10, 1, 2048, 128, 300) == 1  # a window's few keys


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU behaviour")
def test_no_cpu_fallback_without_gpu(lib):
    p = fake_ptrs(9, 1 << 22)
    assert write_call(lib, p[:7]) == 4 and lib.attn_last_cuda_error().decode() != ""
    assert read_call(lib, p[:7]) == 4
    assert read_call(lib, p[:7], lens=None) == 4
    assert decode_call(lib, p, 1 << 22) == 4


# ---------------------------------------------------------------------------------------------- the binding

@pytest.mark.parametrize("bits,group", BITS_GROUPS)
def test_cache_shapes(bits, group):
    c = attn.kvq_cache(2, 3, 7, bits, group, device="cpu")
    assert c.k_codes.shape == (2, 3, 7, 16 * bits) and c.v_codes.dtype == torch.uint8
    assert c.v_params.shape == (2, 3, 7, 128 // group, 2) and c.k_params.dtype == torch.bfloat16
    assert (c.bits, c.group) == (bits, group)
    assert attn._check_kvq(c)[1:6] == (2, 3, 7, bits, group)


def test_cache_refusals():
    for bad in (dict(bits=2), dict(group=16), dict(D=64), dict(B=0), dict(Tk=0), dict(H_kv=0)):
        with pytest.raises(ValueError):
            attn.kvq_cache(**{**dict(B=1, H_kv=1, Tk=4, device="cpu"), **bad})
    kc, kp, vc, vp = attn.kvq_cache(2, 3, 8, 4, 32, device="cpu")
    for bad in (None, kc, (kc, kp, vc), (kc, kp, vc, None),
                (kc.to(torch.int8), kp, vc, vp), (kc, kp.float(), vc, vp),
                (kc[..., :32].contiguous(), kp, vc, vp), (kc, kp[:, :, :, :3].contiguous(), vc, vp),
                (kc, kp, vc[:, :, :7].contiguous(), vp), (kc, kp, vc, vp[:1]),
                (kc[:, :, :4], kp[:, :, :4], vc[:, :, :4], vp[:, :, :4]),         # not contiguous
                (kc, kp, vc.to("meta"), vp)):
        with pytest.raises(ValueError):
            attn._check_kvq(bad)


def test_calls_reject_cpu_tensors(lib):
    c = attn.kvq_cache(1, 2, 8, device="cpu")
    k = torch.zeros(1, 1, 2, 128, dtype=torch.bfloat16)
    lens = torch.ones(1, dtype=torch.int32)
    for call in (lambda: attn.kvq_write(c, k, k, lens), lambda: attn.kvq_read(c),
                 lambda: attn.attn_decode_kvq(k, c, lens)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_lengths_are_checked():
    dev = torch.device("cpu")
    for bad in (None, [1, 2], torch.ones(2, dtype=torch.int64), torch.ones(3, dtype=torch.int32),
                torch.ones(2, 1, dtype=torch.int32), torch.ones(4, dtype=torch.int32)[::2],
                torch.ones(2, dtype=torch.int32, device="meta")):
        with pytest.raises(ValueError):
            attn._check_seqlens(bad, 2, dev)


def test_a_stream_of_another_device_is_refused():
    """Before anything is changed: the current device and stream stay."""
    class Other:
        device = torch.device("cuda", 1)

    with pytest.raises(ValueError, match="stream is on cuda:1"):
        with attn._on(torch.device("cuda", 0), Other()):
            pass


def test_what_is_no_cache_is_refused():
    c = attn.kvq_cache(1, 1, 4, device="cpu")
    for bad in (iter(c), dict(zip("abcd", c)), "abcd", [1, 2, 3, 4], torch.zeros(4, 1, 1, 4, 64, dtype=torch.uint8), None,
                c[:3], (*c, c[0]), (*c[:3], c[3].to("meta")), (c[0], c[1][..., 0], c[2], c[3])):
        with pytest.raises(ValueError, match="cache must|is on meta|k_params has shape"):
            attn._check_kvq(bad)
    assert attn._check_kvq(list(c))[1:6] == (1, 1, 4, 4, 64)
