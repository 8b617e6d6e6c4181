"""Float64 CPU oracle of the quantised key/value cache (test infrastructure only; never on the product path).

Format, per head vector x of D dims, in groups of `group` dims, with `bits`-bit codes n standing for n * s + z:
  z = min(x),   s = least bf16 number that is not below the fp32 quotient (max(x) - z) / (2^bits - 1),
  n = (x - z) / s rounded to the nearest integer, ties to even (0 when s = 0).
The device computes max - z, x - z and both quotients in fp32; here only the first quotient is rounded to fp32 (the
format says so), the rest is float64, so a code may differ by one where the float64 quotient lies within fp32 rounding
of a tie: ``quantize`` returns its distance from the nearest tie as well. Groups with a NaN or an infinity, or whose
range overflows fp32, have s = z = NaN.

The cache is head-major, [B, H_kv, Tk, ...]; token i of the T newest of a sequence of length L has position L - T + i.
"""
from __future__ import annotations

from typing import Tuple

import numpy as np

from .attn_ref import _as_f64, decode_forward


def round_up_bf16(x: np.ndarray) -> np.ndarray:
    """The least bf16 number >= x (x >= 0, float64; 8 significant bits, subnormal spacing 2^-133)."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - 8, -133))
    return np.ceil(x / step) * step


def quantize(x, bits: int, group: int) -> Tuple[np.ndarray, np.ndarray, np.ndarray, np.ndarray]:
    """x [..., D] -> codes int64 [..., D], scale and zero float64 [..., D / group], and each code's quotient's
    distance from the nearest tie [..., D]."""
    x = _as_f64(x)
    levels = 2 ** bits - 1
    g = x.reshape(*x.shape[:-1], x.shape[-1] // group, group)
    with np.errstate(all="ignore"):
        z, top = g.min(-1, keepdims=True), g.max(-1, keepdims=True)      # (numpy's min and max pass NaN on)
        span = (top - z).astype(np.float32)
        bad = ~np.isfinite(span)
        quotient = (np.where(bad, np.float32(0), span) / np.float32(levels)).astype(np.float64)
        s = round_up_bf16(quotient)
        r = np.where(s > 0, (g - z) / np.where(s > 0, s, 1.0), 0.0)
        r = np.where(bad, 0.0, r)
        n = np.minimum(np.rint(r), levels)
    tie = np.abs(r - np.floor(r) - 0.5)
    s, z = np.where(bad, np.nan, s)[..., 0], np.where(bad, np.nan, z)[..., 0]
    return n.astype(np.int64).reshape(x.shape), s, z, tie.reshape(x.shape)


def unpack_codes(codes, bits: int) -> np.ndarray:
    """uint8 [..., D * bits / 8] -> int64 [..., D]: dims in order, 4 bits: the even dim in the low half."""
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    if bits == 8:
        return c
    return np.stack([c & 15, c >> 4], axis=-1).reshape(*c.shape[:-1], 2 * c.shape[-1])


def dequantize(codes, params, bits: int) -> np.ndarray:
    """codes uint8 [..., D * bits / 8], params [..., D / group, 2] -> float64 n * s + z [..., D]."""
    n = unpack_codes(codes, bits).astype(np.float64)
    p = _as_f64(params)
    group = n.shape[-1] // p.shape[-2]
    return n * np.repeat(p[..., 0], group, -1) + np.repeat(p[..., 1], group, -1)


def decode_forward_kvq(q, cache, cache_seqlens, scale: float, window=None):
    """``decode_forward`` of q [B, Tq, H, D] over a quantised cache (k_codes, k_params, v_codes, v_params). Rows past
    a sequence's length are not looked at."""
    kc, kp, vc, vp = cache
    bits = kc.shape[-1] * 8 // q.shape[-1]
    lens = np.clip(np.asarray(cache_seqlens, dtype=np.int64), 0, kc.shape[2])
    with np.errstate(invalid="ignore"):
        k, v = (dequantize(c, p, bits).transpose(0, 2, 1, 3) for c, p in ((kc, kp), (vc, vp)))
    return decode_forward(q, k, v, lens, scale, window=window)
