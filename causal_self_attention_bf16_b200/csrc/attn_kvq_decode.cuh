// Attention of a few new queries over the quantised key/value cache (include/attn.h, attn_decode_kvq): the cached
// decode of attn_decode with keys and values held as 4- or 8-bit codes that stand for n * s + z per group of dims.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "sm100.cuh"

namespace attn {

// This unit's device error word (kind 2 = an address check of the debug build failed, site in the higher bits).
__device__ uint32_t g_kvq_error;

constexpr int kKvqMaxRows = 32;  // (H / H_kv) * Tq query rows per key/value head, at most

enum : uint32_t {
  kSiteKvqDecQ = 0xa4, kSiteKvqDecCodes = 0xa5, kSiteKvqDecParams = 0xa6, kSiteKvqDecO = 0xa7, kSiteKvqDecLse = 0xa8
};

struct KvqDecodeParams {
  const __nv_bfloat16* q;        // [B, Tq, H, 128]
  const uint8_t* k_codes;        // [B, H_kv, Tk, 128 * bits / 8]
  const uint8_t* v_codes;
  const uint32_t* k_params;      // [B, H_kv, Tk, 128 / group] words: s in the low half, z in the high half
  const uint32_t* v_params;
  const int* seqlens;            // [B]
  __nv_bfloat16* o;              // [B, Tq, H, 128]
  float* lse;                    // [B, H, Tq]
  int B, H, Hkv, Tq, Tk;
  int window;                    // sliding window: the query at position p sees keys p - window .. p; -1: none
  float scale_log2;              // scale * log2(e)
};

template <int kBits>
__device__ __forceinline__ float kvq_code(const uint8_t* row, int d) {
  if constexpr (kBits == 4) return static_cast<float>((row[d / 2] >> (4 * (d & 1))) & 15);
  else return static_cast<float>(row[d]);
}

// One CTA of 128 threads per output row (b, i, h), over its visible keys in blocks of 128: thread j scores key j,
// the block takes its maximum (online softmax in base 2, fp32), then thread d sums dim d over the block's keys.
template <int kBits, int kGroup>
__global__ void __launch_bounds__(128) kvq_decode_rows_kernel(const KvqDecodeParams p) {
  constexpr int kRowBytes = 16 * kBits, kGroups = 128 / kGroup;
  __shared__ float qs[128], ps[128], red[4];
  const int t = threadIdx.x;
  const int h = blockIdx.x % p.H, i = (blockIdx.x / p.H) % p.Tq, b = blockIdx.x / p.H / p.Tq;
  const int hk = h / (p.H / p.Hkv);
  const int L = min(max(p.seqlens[b], 0), p.Tk);
  const int last = L - p.Tq + i;
  const int first = p.window < 0 ? 0 : max(0, last - p.window);
  const size_t q_off = ((static_cast<size_t>(b) * p.Tq + i) * p.H + h) * 128 + t;
  const size_t row0 = (static_cast<size_t>(b) * p.Hkv + hk) * p.Tk;
  const size_t n_rows = static_cast<size_t>(p.B) * p.Hkv * p.Tk;
  (void)n_rows;
  qs[t] = ATTN_IN_RANGE(q_off, 1, static_cast<size_t>(p.B) * p.Tq * p.H * 128, kSiteKvqDecQ, &g_kvq_error)
              ? __bfloat162float(p.q[q_off]) * p.scale_log2 : 0.f;
  __syncthreads();
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int kb = first; kb <= last; kb += 128) {
    const int n = min(128, last + 1 - kb);
    float s = -INFINITY;
    if (t < n && ATTN_IN_RANGE(row0 + kb + t, 1, n_rows, kSiteKvqDecCodes, &g_kvq_error)) {
      const uint8_t* c = p.k_codes + (row0 + kb + t) * kRowBytes;
      const uint32_t* w = p.k_params + (row0 + kb + t) * kGroups;
      s = 0.f;
      for (int g = 0; g < kGroups; ++g) {
        const float sc = __uint_as_float(w[g] << 16), z = __uint_as_float(w[g] & 0xffff0000u);
        for (int d = g * kGroup; d < (g + 1) * kGroup; ++d) s = fmaf(qs[d], fmaf(kvq_code<kBits>(c, d), sc, z), s);
      }
    }
    float mx = s;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (t % 32 == 0) red[t / 32] = mx;
    __syncthreads();
    const float m_new = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float a = m == m_new ? 1.f : exp2f(m - m_new);
    ps[t] = s == -INFINITY ? 0.f : exp2f(s - m_new);  // (a NaN score makes its row NaN)
    __syncthreads();
    acc *= a, l *= a, m = m_new;
    for (int j = 0; j < n; ++j) {
      if (!ATTN_IN_RANGE(row0 + kb + j, 1, n_rows, kSiteKvqDecCodes, &g_kvq_error)) break;
      const uint32_t w = p.v_params[(row0 + kb + j) * kGroups + t / kGroup];
      const float v = fmaf(kvq_code<kBits>(p.v_codes + (row0 + kb + j) * kRowBytes, t), __uint_as_float(w << 16),
                           __uint_as_float(w & 0xffff0000u));
      acc = fmaf(ps[j], v, acc);
      l += ps[j];
    }
    __syncthreads();
  }
  const size_t n_out = static_cast<size_t>(p.B) * p.H * p.Tq;
  if (ATTN_IN_RANGE(q_off, 1, n_out * 128, kSiteKvqDecO, &g_kvq_error))
    p.o[q_off] = __float2bfloat16_rn(l == 0.f ? 0.f : acc / l);
  const size_t lse_i = (static_cast<size_t>(b) * p.H + h) * p.Tq + i;
  if (t == 0 && ATTN_IN_RANGE(lse_i, 1, n_out, kSiteKvqDecLse, &g_kvq_error))
    p.lse[lse_i] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace attn
