// The quantised key/value cache: new rows written as 4- or 8-bit codes (attn_kvq_write), rows read back as bf16
// (attn_kvq_read), and cached decode over it (attn_decode_kvq, attn_kvq_decode.cuh). The format is in
// include/attn.h: per group of `group` dims of a head vector, codes n, a bf16 scale s and a bf16 zero z stand for
// n * s + z, with
//   z = min(x),   s = fp32 quotient (max(x) - z) / (2^bits - 1), rounded up to bf16,   n = rint((x - z) / s).
// The minimum of bf16 numbers is one of them, so z is exact; s is rounded up so that no code needs clamping below
// its value (|n s + z - x| <= s / 2). Every step is one correctly rounded fp32 operation, so the codes are defined
// bit for bit. A group that holds a NaN or an infinity, or whose max - min overflows fp32, gets s = z = NaN.
//
// Write and read are HBM-bound copies with a few operations per value. A thread owns some of a row's 128 dims, of the
// key and the value row alike: 16 of them in write, whose work per group (minimum, scale, inverse) is then shared by
// twice as many values as with 8, and 8 in read. Rows are taken in the cache's order, the tokens of one head next to
// each other, so that a warp's codes and params are one stretch of the cache.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <type_traits>

#include "attn.h"
#include "attn_errors.h"
#include "attn_kvq_decode.cuh"

using attn::add2;
using attn::F2;
using attn::f2;
using attn::fma2;
using attn::g_kvq_error;
using attn::mul2;

namespace {

using attn::g_cuda_error;

// Threads per block: 256 made write 3 to 5 % slower (its registers leave no whole number of such blocks on an SM), 128
// made read 9 to 36 % slower.
constexpr int kReadThreads = 256, kWriteThreads = 128;
constexpr int kReadLanes = 16, kWriteLanes = 8;  // threads per row
// Blocks of write, at most: six times the nine that an SM holds. Blocks with one set of rows each were slower in
// batches of padded prompts, where many have nothing to do (32 prompts of up to 2,048 tokens, 10 heads, 4 bits in
// groups of 32: 51 us against 47), and a single wave of them in full ones (102 us against 86).
constexpr unsigned kWriteBlocks = 148 * 54;
enum : uint32_t {
  kSiteKvqNew = 0xa0, kSiteKvqCodes = 0xa1, kSiteKvqParams = 0xa2, kSiteKvqOut = 0xa3
};

// Division by a number known on the host: n / d for n < 2^31 (the high half of n times 2^32 (2^shift / d - 1), rounded
// up, plus n, shifted: Granlund and Montgomery, "Division by invariant integers using multiplication", 1994).
struct FastDiv {
  uint32_t d, mul, shift;
  FastDiv(uint32_t d_ = 1) : d(d_), mul(0), shift(0) {
    while ((1ull << shift) < d) ++shift;
    mul = static_cast<uint32_t>((((1ull << shift) - d) << 32) / d + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

struct CopyParams {
  const __nv_bfloat16* x[2];  // write: new key and value rows [B, T, H_kv, 128]
  __nv_bfloat16* y[2];        // read: key and value rows [B, T, H_kv, 128]
  uint8_t* codes[2];          // [B, H_kv, Tk, 128 * bits / 8]
  uint32_t* params[2];        // [B, H_kv, Tk, 128 / group] words: s in the low half, z in the high half
  const int* seqlens;         // [B]; read: null for rows from position 0 on
  int B, T, Hkv, Tk;
  FastDiv by_T, by_Hkv;  // by T and by H_kv
};

// A kernel launched by launch_early: wait for the grid before it, and let the next one start up.
__device__ __forceinline__ void begin_early() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Row r in the order [B, H_kv, T]: its row of [B, T, H_kv], its cache row, and whether the token has a position (both
// counted in 31 bits).
struct CopyRow {
  uint32_t dense, cache;
  bool there;
};
__device__ __forceinline__ CopyRow copy_row(const CopyParams& p, uint32_t r) {
  const uint32_t bh = p.by_T.div(r), i = r - bh * p.T, b = p.by_Hkv.div(bh), h = bh - b * p.Hkv;
  int pos = static_cast<int>(i);
  if (p.seqlens) pos += min(max(p.seqlens[b], 0), p.Tk) - p.T;
  return {(b * p.T + i) * p.Hkv + h, bh * p.Tk + pos, pos >= 0};
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Quantise this thread's 16 dims (bf16 pairs w), in a group that spans kGroup / 16 neighbouring threads: their codes,
// packed in dim order, and the group's (s, z) word.
template <int kBits, int kGroup>
__device__ __forceinline__ void quantise16(const uint32_t (&w)[8], uint32_t (&codes)[kBits / 2], uint32_t* sz) {
  constexpr float kLevels = kBits == 4 ? 15.f : 255.f;
  // min and max of bf16 pairs; a NaN anywhere in the group wins
  __nv_bfloat162 mn = as_bf162(w[0]), mx = as_bf162(w[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) mn = __hmin2_nan(mn, as_bf162(w[i])), mx = __hmax2_nan(mx, as_bf162(w[i]));
#pragma unroll
  for (int m = 1; m < kGroup / 16; m <<= 1) {
    mn = __hmin2_nan(mn, as_bf162(__shfl_xor_sync(0xffffffffu, as_u32(mn), m)));
    mx = __hmax2_nan(mx, as_bf162(__shfl_xor_sync(0xffffffffu, as_u32(mx), m)));
  }
  const __nv_bfloat16 zb = __hmin_nan(__low2bfloat16(mn), __high2bfloat16(mn));
  const float z = __bfloat162float(zb);
  const float span = __bfloat162float(__hmax_nan(__low2bfloat16(mx), __high2bfloat16(mx))) - z;
  // Quotients by Markstein's method (IBM J. Res. Dev. 34, 1990): with y = 1 / b rounded to nearest and q = a y, the
  // sum q + (a - q b) y, the remainder exact, is a / b rounded to nearest. Nothing less will do: bf16 numbers over a
  // bf16 scale lie on ties often (one in 50 at 4 bits). The compiler's divisions took 2.6 times as long (226 us
  // against 86 for 32 x 2048 tokens of 10 heads at 4 bits, groups of 32). Added to 1.5 * 2^23 a quotient is rounded
  // to an integer in the sum's low bits.
  constexpr float kMagic = 12582912.f, kInverse = 1.f / kLevels;
  uint32_t t[16];
  if (span >= 0x1p-80f && span <= 0x1p100f) {
    float quotient = span * kInverse;
    quotient = fmaf(fmaf(-quotient, kLevels, span), kInverse, quotient);
    const uint32_t sbits = (__float_as_uint(quotient) + 0xffffu) & 0xffff0000u;  // up to bf16
    const float s = __uint_as_float(sbits), y = __frcp_rn(s);
    const F2 y2 = f2(y, y), minus_s = f2(-s, -s), minus_z = f2(-z, -z), magic = f2(kMagic, kMagic);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const F2 a = add2(f2(lo_f32(w[i]), hi_f32(w[i])), minus_z), q = mul2(a, y2);
      const F2 n = add2(fma2(fma2(q, minus_s, a), y2, q), magic);
      t[2 * i] = static_cast<uint32_t>(n.v), t[2 * i + 1] = static_cast<uint32_t>(n.v >> 32);
    }
    *sz = (sbits >> 16) | (static_cast<uint32_t>(__bfloat16_as_ushort(zb)) << 16);
  } else if (span < INFINITY) {  // an inverse or a remainder may not be a normal number; constant group: s = n = 0
    const uint32_t sbits = (__float_as_uint(__fdiv_rn(span, kLevels)) + 0xffffu) & 0xffff0000u;
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] = __float_as_uint(kMagic);
    if (sbits) {
#pragma unroll 1
      for (int i = 0; i < 16; ++i) {
        uint32_t word = w[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) word = i / 2 == j ? w[j] : word;
        const float a = ((i & 1) ? hi_f32(word) : lo_f32(word)) - z;
        const uint32_t n = __float_as_uint(fminf(__fdiv_rn(a, __uint_as_float(sbits)), kLevels) + kMagic);
#pragma unroll
        for (int j = 0; j < 16; ++j) t[j] = i == j ? n : t[j];
      }
    }
    *sz = (sbits >> 16) | (static_cast<uint32_t>(__bfloat16_as_ushort(zb)) << 16);
  } else {  // a NaN or an infinity in the group, or a range past fp32: NaN throughout
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] = __float_as_uint(kMagic);
    *sz = 0x7fff7fffu;
  }
  // t = 0x4b400000 + n, of which only the low bits are wanted
#pragma unroll
  for (int i = 0; i < kBits / 2; ++i) {
    if constexpr (kBits == 4) {
      uint32_t u = t[8 * i + 7];
#pragma unroll
      for (int j = 6; j >= 0; --j) u = (u << 4) + t[8 * i + j];
      codes[i] = u - 0x4b400000u * 0x11111111u;
    } else {
      codes[i] = __byte_perm(__byte_perm(t[4 * i], t[4 * i + 1], 0x0040),
                             __byte_perm(t[4 * i + 2], t[4 * i + 3], 0x0040), 0x5410);
    }
  }
}

template <int kBits, int kGroup>
__global__ void __launch_bounds__(kWriteThreads) kvq_write_kernel(const CopyParams p) {
  begin_early();
  constexpr int kRowBytes = 16 * kBits, kGroups = 128 / kGroup;
  const uint32_t c = threadIdx.x % kWriteLanes;
  constexpr uint32_t kRows = kWriteThreads / kWriteLanes;
  const uint32_t rows = static_cast<uint32_t>(p.B) * p.T * p.Hkv;
  const size_t n_new = static_cast<size_t>(rows) * 128, n_cache = static_cast<size_t>(p.B) * p.Hkv * p.Tk;
  (void)n_new, (void)n_cache;
  for (uint32_t r0 = blockIdx.x * kRows; r0 < rows; r0 += gridDim.x * kRows) {
    const uint32_t r = r0 + threadIdx.x / kWriteLanes;
    const bool live = r < rows;  // (every lane stays for the shuffles)
    const CopyRow at = copy_row(p, live ? r : 0u);
    // A warp whose tokens have no position reads nothing: half of a batch of left-padded prompts may be such (47 us
    // against 80 for 32 prompts of up to 2,048 tokens; with none of them loads that wait for the lengths cost 1 to 4 %).
    if (!__any_sync(0xffffffffu, live && at.there)) continue;
    const size_t from = at.dense * size_t{128} + 16 * c;
    const bool in = ATTN_IN_RANGE(from, 16, n_new, kSiteKvqNew, &g_kvq_error);
    uint32_t raw[2][8];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 u = in ? reinterpret_cast<const uint4*>(p.x[t] + from)[i] : make_uint4(0u, 0u, 0u, 0u);
        raw[t][4 * i] = u.x, raw[t][4 * i + 1] = u.y, raw[t][4 * i + 2] = u.z, raw[t][4 * i + 3] = u.w;
      }
    }
    const size_t to = at.cache * static_cast<size_t>(kRowBytes) + c * (2 * kBits);
    const size_t sz_to = at.cache * static_cast<size_t>(kGroups) + 16 * c / kGroup;
    const bool write = live && at.there && in &&
                       ATTN_IN_RANGE(to, 2 * kBits, n_cache * kRowBytes, kSiteKvqCodes, &g_kvq_error) &&
                       ATTN_IN_RANGE(sz_to, 1, n_cache * kGroups, kSiteKvqParams, &g_kvq_error);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint32_t sz, codes[kBits / 2];
      quantise16<kBits, kGroup>(raw[t], codes, &sz);
      if (!write) continue;
      if constexpr (kBits == 4) *reinterpret_cast<uint2*>(p.codes[t] + to) = make_uint2(codes[0], codes[1]);
      else *reinterpret_cast<uint4*>(p.codes[t] + to) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
      if ((16 * c) % kGroup == 0) p.params[t][sz_to] = sz;
    }
  }
}

template <int kBits, int kGroup>
__global__ void __launch_bounds__(kReadThreads) kvq_read_kernel(const CopyParams p) {
  begin_early();
  constexpr int kRowBytes = 16 * kBits, kGroups = 128 / kGroup;
  const uint32_t c = threadIdx.x % kReadLanes, r = blockIdx.x * (kReadThreads / kReadLanes) + threadIdx.x / kReadLanes;
  const uint32_t rows = static_cast<uint32_t>(p.B) * p.T * p.Hkv;
  const size_t n_out = static_cast<size_t>(rows) * 128, n_cache = static_cast<size_t>(p.B) * p.Hkv * p.Tk;
  (void)n_out, (void)n_cache;
  if (r >= rows) return;
  const CopyRow at = copy_row(p, r);
  uint2 codes[2] = {make_uint2(0u, 0u), make_uint2(0u, 0u)};
  uint32_t sz[2] = {0u, 0u};  // s = z = 0: rows without a position read as 0
  const size_t from = at.cache * static_cast<size_t>(kRowBytes) + c * kBits;
  const size_t sz_from = at.cache * static_cast<size_t>(kGroups) + 8 * c / kGroup;
  if (at.there && ATTN_IN_RANGE(from, kBits, n_cache * kRowBytes, kSiteKvqCodes, &g_kvq_error) &&
      ATTN_IN_RANGE(sz_from, 1, n_cache * kGroups, kSiteKvqParams, &g_kvq_error)) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if constexpr (kBits == 4) codes[t].x = *reinterpret_cast<const uint32_t*>(p.codes[t] + from);
      else codes[t] = *reinterpret_cast<const uint2*>(p.codes[t] + from);
      sz[t] = p.params[t][sz_from];
    }
  }
  const size_t to = at.dense * size_t{128} + 8 * c;
  if (!ATTN_IN_RANGE(to, 8, n_out, kSiteKvqOut, &g_kvq_error)) return;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const float s = lo_f32(sz[t]), z = hi_f32(sz[t]);
    // Byte b of a word as the bits of 2^23 + b, less 2^23: full-rate operations, where the integer conversions are
    // made at a quarter of the rate.
    auto number = [](uint32_t bytes, int i) {
      return __uint_as_float(__byte_perm(bytes, 0x4b000000u, 0x7440 + i)) - 8388608.f;
    };
    uint32_t even = 0, odd = 0;  // 4 bits: the even and the odd dims' codes, a byte each
    if constexpr (kBits == 4) even = codes[t].x & 0x0f0f0f0fu, odd = (codes[t].x >> 4) & 0x0f0f0f0fu;
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // dims 2 i and 2 i + 1
      float n0, n1;
      if constexpr (kBits == 4) {
        n0 = number(even, i), n1 = number(odd, i);
      } else {
        const uint32_t w = i < 2 ? codes[t].x : codes[t].y;
        n0 = number(w, 2 * (i % 2)), n1 = number(w, 2 * (i % 2) + 1);
      }
      out[i] = as_u32(__floats2bfloat162_rn(fmaf(n0, s, z), fmaf(n1, s, z)));
    }
    *reinterpret_cast<uint4*>(p.y[t] + to) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

// ---------------------------------------------------------------------------------------------- host side

attn_status cuda_fail(cudaError_t e, const char* what) {
  std::snprintf(g_cuda_error, attn::kErrorTextBytes, "%s: %s", what, cudaGetErrorString(e));
  return ATTN_ERR_CUDA;
}

struct Range {
  uintptr_t lo, hi;
};
Range span(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, a + bytes};
}
bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }
bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// No output may overlap an input or another output.
template <int kIns, int kOuts>
bool any_overlap(const Range (&ins)[kIns], const Range (&outs)[kOuts]) {
  for (int i = 0; i < kOuts; ++i) {
    for (int j = 0; j < kIns; ++j)
      if (overlap(outs[i], ins[j])) return true;
    for (int j = i + 1; j < kOuts; ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}

attn_status check_format(int D, int bits, int group) {
  if (D != 128) return ATTN_ERR_UNSUPPORTED;
  if (bits != 4 && bits != 8) return ATTN_ERR_UNSUPPORTED;
  if (group != 32 && group != 64 && group != 128) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

attn_status check_copy(int B, int T, int H_kv, int Tk, int D, int bits, int group) {
  if (B < 1 || T < 1 || H_kv < 1 || Tk < 1) return ATTN_ERR_INVALID_ARG;
  const attn_status st = check_format(D, bits, group);
  if (st != ATTN_OK) return st;
  // rows and cache rows are counted in 31 bits, byte offsets in 64
  if (static_cast<long long>(B) * T > 0x7fffffffLL / H_kv) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * H_kv > 0x7fffffffLL / Tk) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

size_t codes_bytes(int B, int H_kv, int Tk, int bits) { return static_cast<size_t>(B) * H_kv * Tk * 16 * bits; }
size_t params_bytes(int B, int H_kv, int Tk, int group) { return static_cast<size_t>(B) * H_kv * Tk * (512 / group); }

// Calls f with the format as compile-time constants.
template <typename F>
void with_format(int bits, int group, F&& f) {
  using std::integral_constant;
  auto by_group = [&](auto b) {
    if (group == 32) f(b, integral_constant<int, 32>());
    else if (group == 64) f(b, integral_constant<int, 64>());
    else f(b, integral_constant<int, 128>());
  };
  if (bits == 4) by_group(integral_constant<int, 4>());
  else by_group(integral_constant<int, 8>());
}

// Launches a kernel that may start while the one before it in the stream still runs: each of this file's kernels waits
// for that one's end (griddepcontrol.wait) before it touches memory, so only its start-up overlaps.
template <typename P>
cudaError_t launch_early(void (*kernel)(P), dim3 grid, int threads, size_t smem, cudaStream_t s, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

attn_status launch_copy(bool write, const CopyParams& p, int bits, int group, void* stream) {
  const long long rows = static_cast<long long>(p.B) * p.T * p.Hkv;
  const int threads = write ? kWriteThreads : kReadThreads, per_block = threads / (write ? kWriteLanes : kReadLanes);
  unsigned grid = static_cast<unsigned>((rows + per_block - 1) / per_block);
  if (write) grid = std::min(grid, kWriteBlocks);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  with_format(bits, group, [&](auto b, auto g) {
    e = launch_early(write ? kvq_write_kernel<b.value, g.value> : kvq_read_kernel<b.value, g.value>, dim3(grid),
                     threads, 0, s, p);
  });
  if (e != cudaSuccess) return cuda_fail(e, write ? "kvq_write_kernel launch" : "kvq_read_kernel launch");
  return ATTN_OK;
}

attn_status check_decode(int B, int H, int Hkv, int Tq, int Tk, int D, int bits, int group, float scale) {
  if (B < 1 || H < 1 || Tq < 1 || Tk < 1) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (Hkv < 1 || Hkv > H || H % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  const attn_status st = check_format(D, bits, group);
  if (st != ATTN_OK) return st;
  if ((H / Hkv) * static_cast<long long>(Tq) > attn::kKvqMaxRows) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * H * Tq > 0x7fffffffLL / 8) return ATTN_ERR_UNSUPPORTED;
  // cache rows are counted in 31 bits, the row of all places (a unit's tiles, 16 keys or more each, and a few) in 30
  if (static_cast<long long>(B) * Hkv > 0x7fffffffLL / Tk) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * Hkv > (1LL << 30) / (Tk / 16 + 1 + attn::kKvqUnitCost)) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

// Keys a sequence's rows can see: the whole cache, or with a sliding window the Tq + window before its end.
int decode_span(int Tq, int Tk, int window) {
  return window < 0 ? Tk : static_cast<int>(std::min<long long>(Tk, static_cast<long long>(Tq) + window));
}

// How a decode call is split: the split kernel's CTAs, one per SM or fewer where there is not a 16-key tile for every
// warp, and whether each of them has whole units. That spares the merge kernel but leaves CTAs uneven, or idle where
// there are fewer units, so it is for small calls: up to 8 tiles of 16 keys a warp where there are units for (nearly)
// all CTAs, else up to 4. Measured, whole / split: 640 units of 200 keys 11.4 / 13.8 us, of 1 to 200 keys 11.8 /
// 12.6; 140 units of 192 keys 6.9 / 9.2, of 1,500 keys 12.6 / 13.8, of 1 to 2,000 keys (over the limit) 14.2 / 12.4;
// 10 units of 384 keys 7.3 / 8.8, of 1,500 keys (over it) 12.0 / 9.1.
struct DecodeSplit {
  unsigned ctas;
  bool whole;
};
DecodeSplit decode_split(int B, int H, int Hkv, int Tq, int span) {
  const int R = (H / Hkv) * Tq, n_rt = (R + 7) / 8, slices = attn::kKvqWarps / n_rt;
  const long long units = static_cast<long long>(B) * Hkv, each = (span + 15) / 16;
  const long long per_cta = (units + attn::kKvqCtas - 1) / attn::kKvqCtas;
  if (per_cta * each <= (4 * units >= 3 * attn::kKvqCtas ? 8 : 4) * slices && per_cta <= 32)
    return {static_cast<unsigned>(std::min<long long>(attn::kKvqCtas, units)), true};
  return {static_cast<unsigned>(std::min<long long>(attn::kKvqCtas, (units * each + slices - 1) / slices)), false};
}

// Room for the pieces of the most CTAs that any window makes (fewer keys are never split over more of them).
size_t decode_pieces(int B, int H, int Hkv, int Tq, int Tk) {
  const int R = (H / Hkv) * Tq, slices = attn::kKvqWarps / ((R + 7) / 8);
  const long long tiles = static_cast<long long>(B) * Hkv * ((Tk + 15) / 16);
  return static_cast<size_t>(std::min<long long>(attn::kKvqCtas, (tiles + slices - 1) / slices));
}
size_t decode_workspace(int B, int H, int Hkv, int Tq, int Tk) {
  if (decode_split(B, H, Hkv, Tq, Tk).whole) return 0;  // (and so with any window, which only leaves fewer keys)
  const size_t pieces = decode_pieces(B, H, Hkv, Tq, Tk), rows = pieces * 2 * ((H / Hkv) * Tq);
  return pieces * sizeof(attn::KvqSpan) + rows * (128 + 2) * 4;
}

template <int kBits, int kGroup>
cudaError_t launch_split(const attn::KvqDecodeParams& p, unsigned ctas, cudaStream_t s) {
  auto kernel = attn::kvq_decode_split_kernel<kBits, kGroup>;
  constexpr int kSmem = attn::KvqShape<kBits, kGroup>::kSmem;
  static_assert(kSmem + 1024 <= 227 * 1024, "one CTA per SM");
  static std::atomic<uint64_t> done{0};  // devices (by number, below 64) whose opt-in is made
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (!(done.load(std::memory_order_relaxed) & bit)) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_early(kernel, dim3(ctas), attn::kKvqThreads, kSmem, s, p);
}

}  // namespace

extern "C" {

attn_status attn_kvq_write(const void* k, const void* v, void* k_codes, void* k_params, void* v_codes,
                           void* v_params, const int* cache_seqlens, int B, int T, int H_kv, int Tk, int D, int bits,
                           int group, void* stream) {
  if (!k || !v || !k_codes || !k_params || !v_codes || !v_params || !cache_seqlens) return ATTN_ERR_INVALID_ARG;
  const attn_status st = check_copy(B, T, H_kv, Tk, D, bits, group);
  if (st != ATTN_OK) return st;
  for (const void* ptr : {k, v, static_cast<const void*>(k_codes), static_cast<const void*>(k_params),
                          static_cast<const void*>(v_codes), static_cast<const void*>(v_params)})
    if (!aligned(ptr, 16)) return ATTN_ERR_MISALIGNED;
  if (!aligned(cache_seqlens, 4)) return ATTN_ERR_MISALIGNED;
  const size_t xb = static_cast<size_t>(B) * T * H_kv * 256;
  const size_t cb = codes_bytes(B, H_kv, Tk, bits), pb = params_bytes(B, H_kv, Tk, group);
  const Range ins[3] = {span(k, xb), span(v, xb), span(cache_seqlens, static_cast<size_t>(B) * 4)};
  const Range outs[4] = {span(k_codes, cb), span(k_params, pb), span(v_codes, cb), span(v_params, pb)};
  if (any_overlap(ins, outs)) return ATTN_ERR_INVALID_ARG;
  CopyParams p{};
  p.x[0] = static_cast<const __nv_bfloat16*>(k);
  p.x[1] = static_cast<const __nv_bfloat16*>(v);
  p.codes[0] = static_cast<uint8_t*>(k_codes);
  p.codes[1] = static_cast<uint8_t*>(v_codes);
  p.params[0] = static_cast<uint32_t*>(k_params);
  p.params[1] = static_cast<uint32_t*>(v_params);
  p.seqlens = cache_seqlens;
  p.B = B, p.T = T, p.Hkv = H_kv, p.Tk = Tk;
  p.by_T = FastDiv(T), p.by_Hkv = FastDiv(H_kv);
  return launch_copy(true, p, bits, group, stream);
}

attn_status attn_kvq_read(const void* k_codes, const void* k_params, const void* v_codes, const void* v_params,
                          const int* cache_seqlens, void* k, void* v, int B, int T, int H_kv, int Tk, int D,
                          int bits, int group, void* stream) {
  if (!k || !v || !k_codes || !k_params || !v_codes || !v_params) return ATTN_ERR_INVALID_ARG;
  const attn_status st = check_copy(B, T, H_kv, Tk, D, bits, group);
  if (st != ATTN_OK) return st;
  if (!cache_seqlens && T > Tk) return ATTN_ERR_INVALID_ARG;
  for (const void* ptr : {k_codes, k_params, v_codes, v_params, static_cast<const void*>(k),
                          static_cast<const void*>(v)})
    if (!aligned(ptr, 16)) return ATTN_ERR_MISALIGNED;
  if (!aligned(cache_seqlens, 4)) return ATTN_ERR_MISALIGNED;
  const size_t xb = static_cast<size_t>(B) * T * H_kv * 256;
  const size_t cb = codes_bytes(B, H_kv, Tk, bits), pb = params_bytes(B, H_kv, Tk, group);
  const Range ins[5] = {span(k_codes, cb), span(k_params, pb), span(v_codes, cb), span(v_params, pb),
                        span(cache_seqlens, cache_seqlens ? static_cast<size_t>(B) * 4 : 0)};
  const Range outs[2] = {span(k, xb), span(v, xb)};
  if (any_overlap(ins, outs)) return ATTN_ERR_INVALID_ARG;
  CopyParams p{};
  p.y[0] = static_cast<__nv_bfloat16*>(k);
  p.y[1] = static_cast<__nv_bfloat16*>(v);
  p.codes[0] = const_cast<uint8_t*>(static_cast<const uint8_t*>(k_codes));
  p.codes[1] = const_cast<uint8_t*>(static_cast<const uint8_t*>(v_codes));
  p.params[0] = const_cast<uint32_t*>(static_cast<const uint32_t*>(k_params));
  p.params[1] = const_cast<uint32_t*>(static_cast<const uint32_t*>(v_params));
  p.seqlens = cache_seqlens;
  p.B = B, p.T = T, p.Hkv = H_kv, p.Tk = Tk;
  p.by_T = FastDiv(T), p.by_Hkv = FastDiv(H_kv);
  return launch_copy(false, p, bits, group, stream);
}

size_t attn_decode_kvq_workspace_bytes(int B, int H, int H_kv, int Tq, int Tk, int D) {
  if (check_decode(B, H, H_kv, Tq, Tk, D, 4, 128, 1.0f) != ATTN_OK) return 0;
  return decode_workspace(B, H, H_kv, Tq, Tk);
}

int attn_decode_kvq_kernels(int B, int H, int H_kv, int Tq, int Tk, int D, int window) {
  if (check_decode(B, H, H_kv, Tq, Tk, D, 4, 128, 1.0f) != ATTN_OK || window < -1) return 0;
  const DecodeSplit split = decode_split(B, H, H_kv, Tq, decode_span(Tq, Tk, window));
  return split.whole || split.ctas == 1 ? 1 : 2;
}

attn_status attn_decode_kvq(const void* q, const void* k_codes, const void* k_params, const void* v_codes,
                            const void* v_params, const int* cache_seqlens, void* o, float* lse, void* workspace,
                            size_t workspace_bytes, int B, int H, int H_kv, int Tq, int Tk, int D, int bits,
                            int group, float scale, int window, void* stream) {
  if (!q || !k_codes || !k_params || !v_codes || !v_params || !cache_seqlens || !o || !lse)
    return ATTN_ERR_INVALID_ARG;
  const attn_status st = check_decode(B, H, H_kv, Tq, Tk, D, bits, group, scale);
  if (st != ATTN_OK) return st;
  if (window < -1) return ATTN_ERR_INVALID_ARG;
  const size_t need = attn_decode_kvq_workspace_bytes(B, H, H_kv, Tq, Tk, D);
  if (need && (!workspace || workspace_bytes < need)) return ATTN_ERR_WORKSPACE;
  for (const void* ptr : {q, k_codes, k_params, v_codes, v_params, static_cast<const void*>(o),
                          static_cast<const void*>(workspace)})
    if (!aligned(ptr, 16)) return ATTN_ERR_MISALIGNED;
  if (!aligned(lse, 4) || !aligned(cache_seqlens, 4)) return ATTN_ERR_MISALIGNED;
  const size_t qb = static_cast<size_t>(B) * Tq * H * 256;
  const size_t cb = codes_bytes(B, H_kv, Tk, bits), pb = params_bytes(B, H_kv, Tk, group);
  const Range ins[6] = {span(q, qb), span(k_codes, cb), span(k_params, pb), span(v_codes, cb), span(v_params, pb),
                        span(cache_seqlens, static_cast<size_t>(B) * 4)};
  const Range outs[3] = {span(o, qb), span(lse, static_cast<size_t>(B) * H * Tq * 4), span(workspace, need)};
  if (any_overlap(ins, outs)) return ATTN_ERR_INVALID_ARG;
  attn::KvqDecodeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_codes = static_cast<const uint8_t*>(k_codes);
  p.v_codes = static_cast<const uint8_t*>(v_codes);
  p.k_params = static_cast<const uint32_t*>(k_params);
  p.v_params = static_cast<const uint32_t*>(v_params);
  p.seqlens = cache_seqlens;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.B = B, p.H = H, p.Hkv = H_kv, p.Tq = Tq, p.Tk = Tk;
  p.window = window < Tk ? window : -1;  // (a window of the capacity hides nothing)
  p.half_scale_log2 = scale * (0.5f * 1.4426950408889634f);
  const int R = p.R = (H / H_kv) * Tq;
  for (int r = 0; r < attn::kKvqMaxRows; ++r) p.row_i[r] = r < R ? r % Tq : 0, p.row_g[r] = r < R ? r / Tq : 0;
  const DecodeSplit split = decode_split(B, H, H_kv, Tq, decode_span(Tq, Tk, window));
  const unsigned ctas = split.ctas;
  p.whole = split.whole;
  p.per_stretch = 1.0 / ((split.whole ? 1.0 : ctas) * (attn::kKvqWarps / ((R + 7) / 8)));
  const size_t most = decode_pieces(B, H, H_kv, Tq, Tk);
  p.spans = static_cast<attn::KvqSpan*>(workspace);
  p.part_o = reinterpret_cast<float*>(p.spans + most);
  p.part_ml = p.part_o + most * 2 * R * 128;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  with_format(bits, group, [&](auto b, auto g) {
    e = launch_split<b.value, g.value>(p, ctas, s);
  });
  if (e != cudaSuccess) return cuda_fail(e, "kvq_decode_split_kernel launch");
  if (!split.whole && ctas > 1) {
    // A unit spans about ctas / (B * H_kv) CTAs: with many pieces to a unit a block takes one row, with few up to 8.
    if (R == 1 || static_cast<long long>(B) * H_kv * 8 < ctas)
      e = launch_early(attn::kvq_decode_merge_kernel<1>, dim3(ctas, R), 256, 0, s, p);
    else if (R == 2)
      e = launch_early(attn::kvq_decode_merge_kernel<2>, dim3(ctas), 256, 0, s, p);
    else if (R <= 4)
      e = launch_early(attn::kvq_decode_merge_kernel<4>, dim3(ctas), 256, 0, s, p);
    else
      e = launch_early(attn::kvq_decode_merge_kernel<8>, dim3(ctas, (R + 7) / 8), 256, 0, s, p);
    if (e != cudaSuccess) return cuda_fail(e, "kvq_decode_merge_kernel launch");
  }
  return ATTN_OK;
}

}  // extern "C"

namespace attn {
// Read and clear this unit's device error word (synchronous; the caller has synchronised the device).
int kvq_error_word(uint32_t* word) {
  return static_cast<int>(cudaMemcpyFromSymbol(word, g_kvq_error, sizeof(uint32_t)));
}
int kvq_error_clear() {
  const uint32_t zero = 0;
  return static_cast<int>(cudaMemcpyToSymbol(g_kvq_error, &zero, sizeof(uint32_t)));
}
}  // namespace attn
