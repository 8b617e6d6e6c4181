// Attention of a few new queries over the quantised key/value cache (include/attn.h, attn_decode_kvq): the cached
// decode of attn_decode with keys and values held as 4- or 8-bit codes n that stand for n * s + z per group of dims.
//
// The cache is read once and bounds the call: a key and its value are 2 * (16 * bits + 512 / group) bytes, 136 to 160
// at 4 bits, and at the 6.56 TB/s of an HBM copy an SM gets about 23 bytes per clock, a 16-key tile every 105 clocks.
// CUDA cores alone cannot turn 4,096 codes into products in that time (two operations a code are 64 clocks of every
// lane), so the codes go to the matrix unit, as A fragments of mma.m16n8k16 (fp16 in, fp32 sums) made in registers.
// tcgen05 would need them widened in shared or tensor memory first, four bytes written for every byte read, to fill
// 128-row tiles with 1 to 32 queries. What bounds the loop at 4 bits is the memory and the widening together, so that
// is kept to few operations. 256 sequences of 1,024 to 2,048 keys with 10 heads, groups of 64: 112 us, 5.1 TB/s (77 %
// of the copy) in a graph of a few calls; 95 us with the arithmetic taken out. A loop of calls meets the power cap: 117
// to 125 us.
//
//   Codes. A small integer in the low bits of an fp16 number is that number: n * 2^-24, a subnormal, which the matrix
//   unit multiplies exactly. So one logical operation makes two numbers of a 32-bit word's low nibbles (n * 2^-24), of
//   its second nibbles (n * 2^-20, without a shift), and after one shift of the third and fourth; 8-bit codes take a
//   byte permutation a pair. The powers of two go into the queries' numbers and, for values, into the result's.
//   Scores. For key j and query row r, with the sums taken group by group of dims:
//     q . k = sum_g s_g (sum_d q_d n_d) + z_g (sum_d q_d).     The first sum is the matrix product, the last is made
//   once per query row. A query row is scaled by a power of two that puts its largest dim into [2^14, 2^15), so that
//   its bf16 numbers are fp16 numbers (exactly down to 2^-27 of the largest, below that to 2^-35 of it); the power
//   goes off with the softmax scale. The unit aligns products by their factors' exponent fields, so a subnormal
//   factor's leading zeros are bits that small products of a sum lose: with the codes lse stays within 5e-7 of
//   itself, but the queries' sums, whose other factor could be as small as 2^-24, are made with 1 (lse was off by
//   2e-6 otherwise).
//   Values. o = sum_j p_j s_g (n - c) + sum_j p_j (z_g + c s_g), c = 8 or 128: one packed addition centres the codes,
//   so that the fp32 accumulators hold sums of both signs: they are cut off, not rounded (1 + 1.5 * 2^-24 stays 1),
//   which sums of one sign over a whole cache would show. p_j s_g is the B fragment, rounded to fp16: 2^-11 of itself
//   at most against the output's own 2^-8. So that it is in fp16's range whatever the scales, it is carried in units
//   of a power of two per query row and group of dims, in which the largest so far is 2^8 or more: light keys behind a
//   heavy one keep 2^-11 of themselves down to 2^-22 of it, and are lost below 2^-33 only. (The matrix unit cuts each
//   product off at about 2^-24 of the sum it joins, so that this much counts where the heavy key's code is near the
//   middle.) Per row, since a row must not lose its weights to the scale of a key that it does not see or
//   hardly weighs (one unit for all rows was 0.5 % faster, 3 % in groups of 32). The second sum is fp32 throughout.
//   Softmax in base 2 and fp32. The running max is only raised when a score passes it by more than 4 (then p <= 2^4
//   and the sums stay far from overflow) or a weight times a scale its unit by 2^15: one vote a tile in place of the
//   reduction and the rescaling. The vote takes a lane's largest weight times its largest scale. With the scales alone
//   a heavy key without a value, whose unit the other keys' small weights set, made every tile after it raise (64
//   sequences of 1,024 to 2,048 keys, 10 heads: 38.9 us against 35.5 at 4 bits, 52.0 against 44.3 in groups of 32).
//
// Work split. A unit is one (sequence, key/value head); its visible keys, tiles of 32 (8 bits: 16). All units' tiles
// in a row, with two places more for each unit's own cost, are dealt to the warps in equal stretches, found on the
// device from the lengths, so that every warp has the same work however ragged the batch, through a ring of tiles in
// shared memory that it fills for itself (cp.async; no barrier in the loop). A unit that begins and ends in one
// warp's stretch is finished there; the pieces of one that spans warps are joined by the CTA at its end, and the
// CTAs' pieces by kvq_decode_merge_kernel.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "sm100.cuh"

namespace attn {

// This unit's device error word (kind 2 = an address check of the debug build failed, site in the higher bits).
__device__ uint32_t g_kvq_error;

constexpr int kKvqMaxRows = 32;   // (H / H_kv) * Tq query rows per key/value head, at most
constexpr int kKvqWarps = 12;     // warps per CTA (divides by 1, 2, 3 and 4 row tiles)
constexpr int kKvqThreads = kKvqWarps * 32;
constexpr int kKvqCtas = 148;     // CTAs of the split kernel, at most: one per SM of a 148-SM part

// Running max of a row before its first key: fp32's lowest number, below which there is no score.
constexpr float kKvqNone = -3.402823466e38f;

// Places of a unit in the row beside its tiles: its queries, its first maximum and its result take a warp about as long
// as two tiles do (one or none measured 3 and 20 % slower on decode_d20, whose batch holds short sequences).
constexpr int kKvqUnitCost = 2;

enum : uint32_t {
  kSiteKvqDecQ = 0xa4, kSiteKvqDecCodes = 0xa5, kSiteKvqDecParams = 0xa6, kSiteKvqDecO = 0xa7, kSiteKvqDecLse = 0xa8,
  kSiteKvqDecPart = 0xa9
};

// What a CTA of the split kernel leaves for the merge kernel: the unit that begins in it and goes on past it.
struct KvqSpan {
  int unit;      // b * H_kv + hk, or -1: none
  int last_cta;  // the CTA it ends in
  int slot;      // this CTA's piece of it: 0 if that has the CTA's first tile, else 1
  int pad;
};

// A warp's piece of a unit that does not both begin and end with it: its first one (slot 0) or its last (slot 1).
struct KvqPiece {
  int unit;    // b * H_kv + hk, or -1: none
  int begins;  // the unit's first tile is the piece's
  int end;     // the unit's end in the row of all places
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
  KvqSpan* spans;                // [grid]
  float* part_ml;                // [grid, 2, R, 2]: a piece's max (log2 units) and sum per row
  float* part_o;                 // [grid, 2, R, 128]: its unnormalised output
  int B, H, Hkv, Tq, Tk, R;
  int window;                    // sliding window: the query at position p sees keys p - window .. p; -1: none
  int whole;                     // 1: every CTA has whole units (at most 32 of them): no piece is left to merge
  float half_scale_log2;         // scale * log2(e) / 2 (finite for any finite scale)
  double per_stretch;            // 1 / the warps' stretches of the row of all places (of the CTA's with `whole`)
  uint8_t row_i[kKvqMaxRows], row_g[kKvqMaxRows];  // row r is token r % Tq of query head r / Tq of the group
};

// ------------------------------------------------------------------------------------------------ fragments

// c += 16 x 16 (A, row-major) times 16 x 8 (B): c[0..1] = A row lane / 4, columns 2 (lane % 4) + 0..1; c[2..3] = A row
// lane / 4 + 8.
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with c = 0 before.
__device__ __forceinline__ void mma_16x8x16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                  uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
               "{%10,%10,%10,%10};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Transpose of an 8 x 8 matrix of 16-bit numbers held two to a lane.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// lse of a row from its max m and sum l (log2 units), o's factor from its sum; a row that saw no key has l = 0.
__device__ __forceinline__ float kvq_lse(float m, float l) {
  return l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
}
__device__ __forceinline__ float kvq_factor(float l) { return l == 0.f ? 0.f : rcp(l); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t c;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}

// Two fp32 operations in one instruction, each rounded to nearest.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ float lo_of(F2 a) { return __uint_as_float(static_cast<uint32_t>(a.v)); }
__device__ __forceinline__ float hi_of(F2 a) { return __uint_as_float(static_cast<uint32_t>(a.v >> 32)); }

// Nibbles 0..3 of the low and of the high half of w as fp16 numbers n * 2^-24 (x[0], x[2]) and n * 2^-20 (x[1], x[3]);
// centred: n - 8.
template <bool kCentred>
__device__ __forceinline__ void widen4(uint32_t (&x)[4], uint32_t w) {
  const uint32_t v = w >> 8;
  x[0] = w & 0x000f000fu;
  x[1] = w & 0x00f000f0u;
  x[2] = v & 0x000f000fu;
  x[3] = v & 0x00f000f0u;
  if constexpr (kCentred) {
    x[0] = hadd2(x[0], 0x80088008u), x[1] = hadd2(x[1], 0x80808080u);
    x[2] = hadd2(x[2], 0x80088008u), x[3] = hadd2(x[3], 0x80808080u);
  }
}
// The bytes of w that kSel names (its nibbles 0 and 2) as fp16 numbers n * 2^-24; centred: n - 128.
template <bool kCentred, uint32_t kSel>
__device__ __forceinline__ uint32_t widen8(uint32_t w) {
  const uint32_t x = __byte_perm(w, 0u, kSel | 0x4040u);
  return kCentred ? hadd2(x, 0x80808080u) : x;
}

template <int kBytes>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes) : "memory");
}
template <int kBytes>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool valid) {  // 0 where not valid
  const int n = valid ? kBytes : 0;
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int kWords>
__device__ __forceinline__ void lds(uint32_t (&w)[kWords], uint32_t addr) {
  static_assert(kWords == 1 || kWords == 2 || kWords % 4 == 0, "32, 64 or a multiple of 128 bits");
  if constexpr (kWords == 1) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
  } else if constexpr (kWords == 2) {
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  } else {
#pragma unroll
    for (int i = 0; i < kWords; i += 4)
      asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]) : "r"(addr + 4 * i));
  }
}

// 2^e of e in [-126, 127].
__device__ __forceinline__ float kvq_power(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
// 1 / x of a power of two in [2^-126, 2^126].
__device__ __forceinline__ float kvq_inverse(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }

// ------------------------------------------------------------------------------------------------ layout

// A tile in shared memory: its key rows of codes, its value rows, then a row of key and of value params each. Chunk c
// (16 bytes) of row r sits at chunk c ^ kvq_swizzle(r). A score tile's row g is key kvq_key(g) (rows 8-15: + 8). With
// these two every read below, 4 to 16 bytes a lane, meets each bank once: the eight keys of a row set, and the four
// that a half (or quarter) warp reads together, fall into different banks.
template <int kBits>
__device__ __forceinline__ int kvq_swizzle(int r) {
  if constexpr (kBits == 4) return (r & 2) | ((r >> 2) & 1);
  else return ((r & 3) << 1) | ((r >> 2) & 1);
}
__device__ __forceinline__ int kvq_key(int g) { return ((g >> 1) & 1) | (((g ^ (g >> 2)) & 1) << 1) | (g & 4); }

template <int kBits, int kGroup>
struct KvqShape {
  static constexpr int kRowBytes = 16 * kBits, kGroups = 128 / kGroup;
  static constexpr int kHalves = kBits == 4 ? 2 : 1, kTile = 16 * kHalves;  // keys per tile, 16 to a product
  static constexpr int kCodeBytes = kTile * kRowBytes, kParamBytes = kTile * kGroups * 4;
  static constexpr int kStageBytes = 2 * kCodeBytes + 2 * kParamBytes;
  // Tiles per warp in the ring: one in use, the others in flight (4-5 KB a tile). A third made 8 bits, which the memory
  // bounds, 2 % faster and 4 bits up to 3 % slower.
  static constexpr int kStages = kBits == 8 ? 3 : 2;
  static constexpr int kRing = kKvqWarps * kStages * kStageBytes;
  // Pieces to be joined: 8 rows a warp. The first is kept beside the ring, the last one takes its warp's ring over.
  static constexpr int kPiece = 8 * 128 * 4;
  static_assert(kPiece <= kStages * kStageBytes, "a piece fits a warp's ring");
  static constexpr int kMerge = kKvqWarps * kPiece + 2 * kKvqWarps * 8 * 2 * 4;
  static constexpr int kSmem = kRing + kMerge;
};

// A sequence's keys that any of its queries sees, [start, L), and how many tiles they are.
struct KvqSeq {
  int L, start, tiles;
};
template <int kTile>
__device__ __forceinline__ KvqSeq kvq_seq(const KvqDecodeParams& p, int b) {
  KvqSeq s;
  s.L = min(max(p.seqlens[b], 0), p.Tk);  // lengths outside [0, Tk] are clamped
  s.start = p.window < 0 ? 0 : max(0, s.L - p.Tq - p.window);
  s.tiles = (s.L - s.start + kTile - 1) / kTile;
  return s;
}

// A tile of a unit, and the unit's end in the row of all places.
struct KvqCursor {
  int b, hk, tile, end;
  KvqSeq s;
};
// The first tile of the next unit; the end of all places where there is none.
template <int kTile>
__device__ __forceinline__ void kvq_next_unit(const KvqDecodeParams& p, KvqCursor& c) {
  c.tile = 0;
  if (++c.hk == p.Hkv) {
    c.hk = 0;
    do {
      if (++c.b >= p.B) {
        c.end = 0x7fffffff;
        return;
      }
      c.s = kvq_seq<kTile>(p, c.b);
    } while (c.s.tiles == 0);
  }
  c.end += kKvqUnitCost + c.s.tiles;
}

// ------------------------------------------------------------------------------------------------ split kernel

// A warp takes up to 8 query rows; with more, n_rt = ceil(R / 8) warps take a stretch's tiles together, each for itself
// (32 rows: 24 us where the bytes would take 2.3). 12 warps of 168 registers an SM: 16 of 128 took half as many
// instructions again. Groups of 32 dims do not quite fit: at 4 bits some 170 bytes a thread are spilled, at 8 bits 8.
template <int kBits, int kGroup>
__global__ void __launch_bounds__(kKvqThreads, 1) kvq_decode_split_kernel(const KvqDecodeParams p) {
  using Shape = KvqShape<kBits, kGroup>;
  constexpr int kGroups = Shape::kGroups, kRowBytes = Shape::kRowBytes, kStages = Shape::kStages;
  constexpr int kHalves = Shape::kHalves, kTile = Shape::kTile;
  constexpr int kWords = kGroup * kBits / 128;   // 32-bit words of a key row and group that a lane scores
  constexpr int kVWords = kGroup * kBits / 256;  // of a value row and group that a lane multiplies (0: half a word)
  constexpr float kCentre = kBits == 4 ? 8.f : 128.f;
  constexpr int kLift = 120;
  // A weight is at most kLazy, and with its scale and unit kMostWeight, without a raise: in fp16's range. A raise puts
  // a tile's largest into [2^kAim, 2^(kAim + 1)): near the range's upper end, with room for 2^6 before the next raise.
  // A unit is at most 2^kMostUnit, so that no product passes fp32's range before the scale comes to it; the weights of
  // subnormal scales, down to 2^-133, are normal fp16 numbers still.
  constexpr float kLazy = 16.f, kMostWeight = 32768.f;
  constexpr int kAim = 8, kMostUnit = 122;
  extern __shared__ __align__(128) uint8_t kvq_smem[];
  __shared__ KvqPiece sh_piece[2 * kKvqWarps];  // stretch i's slots at 2 i, 2 i + 1
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  const int R = p.R, G = p.H / p.Hkv;
  const int n_rt = (R + 7) / 8;
  const int slices = kKvqWarps / n_rt;  // stretches per CTA, each for the n_rt warps of its row tiles
  const int rt = warp % n_rt, slice = warp / n_rt;
  if (rt == 0 && lane < 2) sh_piece[2 * slice + lane].unit = -1;  // (this warp's to write; read after the barrier)

  // Every warp looks for itself where its stretch of the row of all places begins, 32 items at a time. An item is a
  // sequence with its H_kv units, or with p.whole one of the units that this CTA has to itself (the row is then the
  // CTA's). A unit without tiles has no places; otherwise it has kKvqUnitCost, then its tiles'.
  const int n_units = p.B * p.Hkv;
  const int u0 = p.whole ? static_cast<int>(static_cast<long long>(blockIdx.x) * n_units / gridDim.x) : 0;
  const int u1 = p.whole ? static_cast<int>(static_cast<long long>(blockIdx.x + 1) * n_units / gridDim.x) : n_units;
  const int each_item = p.whole ? 1 : p.Hkv, items = p.whole ? u1 - u0 : p.B;
  auto places = [&](int i) {
    const int n = i < items ? kvq_seq<kTile>(p, p.whole ? (u0 + i) / p.Hkv : i).tiles : 0;
    return n ? (n + kKvqUnitCost) * each_item : 0;
  };
  // This grid may be launched before the one it follows ends; the merge kernel in turn waits for this grid's end. (What
  // needs no memory is above: 1 % on decode_d20, 6 % on the smallest calls.)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0 && !p.whole) p.spans[blockIdx.x].unit = -1;
  int total = 0;
  bool empty = p.whole;  // whether there may be sequences without keys
  for (int i = lane; i < items; i += 32) {
    const int n = places(i);
    total += n;
    empty |= n == 0;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
  const int stretches = (p.whole ? 1 : static_cast<int>(gridDim.x)) * slices;
  const int stretch0 = p.whole ? 0 : blockIdx.x * slices;
  // Stretch i of all begins at place i * total / stretches, rounded down (the half place keeps the product's rounding
  // away from whole numbers), so that every CTA has the same number of places, to one; with fewer places than
  // stretches the first ones have one each. No stretch before another's end is empty. A stretch's tiles are those
  // whose places it has.
  auto begin_of = [&](int i) {
    if (total <= stretches || i >= stretches) return min(i < stretches ? i : total, total);
    return static_cast<int>((static_cast<double>(static_cast<long long>(i) * total) + 0.5) * p.per_stretch);
  };
  auto start_of = [&](int i) { return begin_of(stretch0 + i); };  // the CTA's i-th
  const int first = start_of(slice), last = start_of(slice + 1);
  KvqCursor cur = {};  // the unit being computed, from its tile cur.tile on
  cur.end = total;
  if (first < last) {
    for (int i0 = 0, before = 0;; i0 += 32) {
      const int n = places(i0 + lane);
      int incl = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
      }
      const unsigned past = __ballot_sync(0xffffffffu, before + incl > first);
      if (past) {  // (some item ends past it: first < total)
        const int l = __ffs(past) - 1, start = before + __shfl_sync(0xffffffffu, incl - n, l);
        cur.b = p.whole ? (u0 + l) / p.Hkv : i0 + l;
        cur.s = kvq_seq<kTile>(p, cur.b);
        const int each = cur.s.tiles + kKvqUnitCost, at = (first - start) / each;
        cur.hk = p.whole ? u0 + l - cur.b * p.Hkv : at;
        cur.end = start + (at + 1) * each;
        cur.tile = max(first - (cur.end - cur.s.tiles), 0);
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }

  // --- the ring
  const uint32_t ring = sm100::smem_u32(kvq_smem) + warp * kStages * Shape::kStageBytes;
  constexpr int kChunks = kRowBytes / 16, kRowsAtOnce = 32 / kChunks;  // 16-byte chunks of a row; rows a copy covers
  const int c_row = lane / kChunks, p_row = lane % 16;  // (params: key rows by the lower lanes, else value rows)
  // (a copy's rows are a multiple of 4 apart, and of 8 where the swizzle looks at bit 2)
  uint32_t code_at[kTile / kRowsAtOnce];
#pragma unroll
  for (int i = 0; i < kTile / kRowsAtOnce; ++i) {
    const int r = c_row + i * kRowsAtOnce;
    code_at[i] = r * kRowBytes + (((lane % kChunks) ^ kvq_swizzle<kBits>(r)) << 4);
  }
  const size_t n_rows = static_cast<size_t>(p.B) * p.Hkv * p.Tk;
  (void)n_rows;
  KvqCursor pre = cur;  // the next tile this warp fetches
  int pre_left = cur.s.tiles - cur.tile;  // its unit's tiles from it on that the stretch has
  pre_left = min(pre_left, last - (cur.end - pre_left));
  // its first row's codes at this lane's chunk, and its params (the lower half warp fetches the keys', the upper the
  // values')
  const uint8_t *k_from, *v_from, *p_from;
  size_t pre_row;
  auto aim = [&]() {
    pre_row = (static_cast<size_t>(pre.b) * p.Hkv + pre.hk) * p.Tk + (pre.s.start + pre.tile * kTile);
    k_from = p.k_codes + pre_row * kRowBytes + lane * 16;
    v_from = p.v_codes + pre_row * kRowBytes + lane * 16;
    p_from = reinterpret_cast<const uint8_t*>(lane < 16 ? p.k_params : p.v_params) +
             (pre_row + p_row) * (kGroups * 4);
  };
  auto fetch = [&](int stage) {  // copies (or nothing) and one commit
    if (pre_left > 0) {
      const int n = pre.s.L - (pre.s.start + pre.tile * kTile);  // valid rows (at least one)
      const uint32_t to = ring + stage * Shape::kStageBytes;
      const uint32_t p_to = to + 2 * Shape::kCodeBytes + (lane < 16 ? 0 : Shape::kParamBytes) + p_row * kGroups * 4;
      if (n >= kTile && ATTN_IN_RANGE(pre_row, kTile, n_rows, kSiteKvqDecCodes, &g_kvq_error)) {
#pragma unroll
        for (int i = 0; i < kTile / kRowsAtOnce; ++i) {
          cp_async<16>(to + code_at[i], k_from + i * 512);
          cp_async<16>(to + code_at[i] + Shape::kCodeBytes, v_from + i * 512);
        }
#pragma unroll
        for (int i = 0; i < kHalves; ++i) cp_async<kGroups * 4>(p_to + i * 64 * kGroups, p_from + i * 64 * kGroups);
      } else {  // rows past the sequence's end are zeros, and not read
#pragma unroll
        for (int i = 0; i < kTile / kRowsAtOnce; ++i) {
          const int r = c_row + i * kRowsAtOnce;
          const bool in = r < n && ATTN_IN_RANGE(pre_row + r, 1, n_rows, kSiteKvqDecCodes, &g_kvq_error);
          cp_async<16>(to + code_at[i], in ? k_from + i * 512 : p.k_codes, in);
          cp_async<16>(to + code_at[i] + Shape::kCodeBytes, in ? v_from + i * 512 : p.v_codes, in);
        }
#pragma unroll
        for (int i = 0; i < kHalves; ++i) {
          const int r = p_row + 16 * i;
          const bool in = r < n && ATTN_IN_RANGE(pre_row + r, 1, n_rows, kSiteKvqDecParams, &g_kvq_error);
          cp_async<kGroups * 4>(p_to + i * 64 * kGroups,
                                in ? p_from + i * 64 * kGroups : reinterpret_cast<const uint8_t*>(p.k_params), in);
        }
      }
      ++pre.tile;
      pre_row += kTile;
      k_from += kTile * kRowBytes;
      v_from += kTile * kRowBytes;
      p_from += kTile * kGroups * 4;
      if (--pre_left == 0) {
        kvq_next_unit<kTile>(p, pre);
        pre_left = min(pre.s.tiles, last - (pre.end - pre.s.tiles));
        if (pre_left > 0) aim();
      }
    }
    cp_async_commit();
  };
  aim();
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i);

  // Where this lane reads a tile. Keys: row kg (and kg + 8), its words of each group. Values: rows vk0, vk1 (and + 8),
  // which are the columns 2 t, 2 t + 1 (and + 8) of the value fragments.
  const int kg = kvq_key(g), vk0 = kvq_key(2 * t), vk1 = kvq_key(2 * t + 1);
  const int v_byte = kVWords < 1 ? (g >> 1) * 4 : g * kVWords * 4;
  auto at_byte = [](int row, int byte) {
    return row * kRowBytes + (((byte >> 4) ^ kvq_swizzle<kBits>(row)) << 4) + (byte & 15);
  };
  const uint32_t k_lds = at_byte(kg, t * kWords * 4), kp_lds = kg * kGroups * 4;
  const uint32_t v0_lds = Shape::kCodeBytes + at_byte(vk0, v_byte), v1_lds = Shape::kCodeBytes + at_byte(vk1, v_byte);

  auto piece_o = [&](int slot, int w) {  // [8][128]
    return reinterpret_cast<float*>(
        kvq_smem + (slot ? w * kStages * Shape::kStageBytes : Shape::kRing + w * Shape::kPiece));
  };
  auto piece_ml = [&](int slot, int w) {  // [8][2]
    return reinterpret_cast<float*>(kvq_smem + Shape::kRing + kKvqWarps * Shape::kPiece) + (slot * kKvqWarps + w) * 16;
  };
  const size_t n_q = static_cast<size_t>(p.B) * p.Tq * p.H * 128;
  (void)n_q;

  int stage = 0;
  for (int slot = 0; ; slot = 1) {
    // --- one piece: n_tiles tiles of unit (cur.b, cur.hk), from its tile cur.tile on
    const int n_tiles = min(cur.s.tiles - cur.tile, last - (cur.end - cur.s.tiles + cur.tile));
    if (n_tiles <= 0) break;  // (no stretch, or one that ends in a unit's own places)
    const bool whole = n_tiles == cur.s.tiles;
    // The unit's queries as B fragments: column g is row rt * 8 + g; the lane holds its dims that meet the words of a
    // key row that it reads, paired as the codes are, in units of 2^-up (4 bits: second and fourth nibbles 2^(4 - up),
    // as their codes are 2^4 larger).
    uint32_t qb[16];
    float qsum[kGroups][2];  // a group's sum of q over its dims, units of 2^(24 - up), of columns 2 t and 2 t + 1
    // softmax scale (log2 units) times 2^(24 - up) of columns 2 t and 2 t + 1; where that is past fp32's range (queries
    // of 2^121 or more at the default scale, whose scores tiny keys may bring back into it), less 2^kLift, and negative
    float down[2];
    {
      const int row = rt * 8 + g, i = p.row_i[row], h = cur.hk * G + p.row_g[row];
      const size_t off = ((static_cast<size_t>(cur.b) * p.Tq + i) * p.H + h) * 128;
      const bool live = row < R && ATTN_IN_RANGE(off, 128, n_q, kSiteKvqDecQ, &g_kvq_error);
      uint4 u[4];
      float qs[kGroups][4];
      uint32_t top = 0;  // the largest exponent, bf16 bits 7-14 of a half
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        u[x] = make_uint4(0u, 0u, 0u, 0u);
        const int j = x / (kGroup / 32), e = x % (kGroup / 32);  // 8 dims of group j
        if (live) u[x] = *reinterpret_cast<const uint4*>(p.q + off + j * kGroup + t * (kGroup / 4) + 8 * e);
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(u[x].x & 0x7f807f80u, u[x].y & 0x7f807f80u),
                                     __vmaxu2(u[x].z & 0x7f807f80u, u[x].w & 0x7f807f80u)));
      }
      top = max(top & 0xffffu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^up brings exponent `top` to 2^14 (an infinity or NaN stays one); 2^up and 2^-up are normal numbers
      const int up = min(14 + 127 - static_cast<int>(top >> 7), 126);
      const float mul = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint32_t w[4] = {u[x].x, u[x].y, u[x].z, u[x].w};
        uint32_t f[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          f[y] = pack_f16x2(__uint_as_float(w[y] << 16) * mul,
                            __uint_as_float(w[y] & 0xffff0000u) * (kBits == 4 ? mul * 0.0625f : mul));
        if constexpr (kBits == 4) {  // dims (0,4) (1,5) (2,6) (3,7) of a word's eight
          qb[4 * x] = __byte_perm(f[0], f[2], 0x5410);
          qb[4 * x + 1] = __byte_perm(f[0], f[2], 0x7632);
          qb[4 * x + 2] = __byte_perm(f[1], f[3], 0x5410);
          qb[4 * x + 3] = __byte_perm(f[1], f[3], 0x7632);
        } else {  // dims (0,1) (2,3) of each word's four
#pragma unroll
          for (int y = 0; y < 4; ++y) qb[4 * x + y] = f[y];
        }
        // the sums of q over a group's dims: products with 1 (16 for the numbers that are 2^4 smaller)
        constexpr uint32_t kOne = 0x3c003c00u, kSecond = kBits == 4 ? 0x4c004c00u : kOne;
        const int j = x / (kGroup / 32);
        if (x % (kGroup / 32) == 0) mma_16x8x16_first(qs[j], kOne, kOne, kSecond, kSecond, qb[4 * x], qb[4 * x + 1]);
        else mma_16x8x16(qs[j], kOne, kOne, kSecond, kSecond, qb[4 * x], qb[4 * x + 1]);
        mma_16x8x16(qs[j], kOne, kOne, kSecond, kSecond, qb[4 * x + 2], qb[4 * x + 3]);
        qsum[j][0] = qs[j][0] * 0x1p-24f, qsum[j][1] = qs[j][1] * 0x1p-24f;
      }
      const int e = 25 - up;  // in [-101, 139]
      float back = p.half_scale_log2 * kvq_power(min(e, 127)) * kvq_power(max(e - 127, 0));
      if (back == INFINITY)
        back = -fminf(p.half_scale_log2 * kvq_power(-kLift / 2) * kvq_power(e - kLift / 2), -kKvqNone);
      down[0] = __shfl_sync(0xffffffffu, back, 8 * t);
      down[1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
    }
    // the last tile that needs no mask begins here, if any (none where a score has two factors: those are the masked
    // tiles', so that the others do without; a flag of its own was 1 % slower)
    const int plain_to = __any_sync(0xffffffffu, down[0] < 0.f || down[1] < 0.f) ? -1 : cur.s.L - p.Tq - (kTile - 1);
    float acc[8][4], corr[kGroups][2], m[2] = {kKvqNone, kKvqNone}, l[2] = {0.f, 0.f};
    float unit[kGroups][2];  // the weights p s of columns 2 t, 2 t + 1 are in units of 1 / unit, a power of two
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll
    for (int j = 0; j < kGroups; ++j) corr[j][0] = corr[j][1] = 0.f, unit[j][0] = unit[j][1] = kvq_power(kMostUnit);

    // The tile of codes at `at` and params at `ap`: n_halves times 16 keys, from key0 on.
    auto tile = [&](const uint32_t at, const uint32_t ap, const int key0, auto masked, auto n_halves) {
      constexpr int kN = n_halves.value;
      // --- scores: rows g and g + 8 of half y are keys kg + 16 y and kg + 16 y + 8
      float s[4 * kN];
#pragma unroll
      for (int y = 0; y < kN; ++y) {
        uint32_t sz[2][kGroups];
        lds(sz[0], ap + kp_lds + 16 * y * kGroups * 4);
        lds(sz[1], ap + kp_lds + (16 * y + 8) * kGroups * 4);
        float* sy = s + 4 * y;
        sy[0] = sy[1] = sy[2] = sy[3] = 0.f;
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
          float c[4];
          constexpr int kPart = kWords < 4 ? kWords : 4;  // words read at once
#pragma unroll
          for (int w0 = 0; w0 < kWords; w0 += kPart) {
            const uint32_t a = ((at + k_lds) ^ (j * (kGroup * kBits / 8) + w0 * 4)) + 16 * y * kRowBytes;
            uint32_t ka[kPart], kb[kPart];
            lds(ka, a);
            lds(kb, a + 8 * kRowBytes);
#pragma unroll
            for (int w = 0; w < kPart; ++w) {
              if constexpr (kBits == 4) {
                const uint32_t* b = qb + 4 * (j * kWords + w0 + w);
                uint32_t xa[4], xb[4];
                widen4<false>(xa, ka[w]);
                widen4<false>(xb, kb[w]);
                if (w0 + w == 0) mma_16x8x16_first(c, xa[0], xb[0], xa[1], xb[1], b[0], b[1]);
                else mma_16x8x16(c, xa[0], xb[0], xa[1], xb[1], b[0], b[1]);
                mma_16x8x16(c, xa[2], xb[2], xa[3], xb[3], b[2], b[3]);
              } else {
                const uint32_t* b = qb + 2 * (j * kWords + w0 + w);
                const uint32_t a0 = widen8<false, 0x0100>(ka[w]), a1 = widen8<false, 0x0100>(kb[w]);
                const uint32_t a2 = widen8<false, 0x0302>(ka[w]), a3 = widen8<false, 0x0302>(kb[w]);
                if (w0 + w == 0) mma_16x8x16_first(c, a0, a1, a2, a3, b[0], b[1]);
                else mma_16x8x16(c, a0, a1, a2, a3, b[0], b[1]);
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sy[e] = fmaf(__uint_as_float(sz[e / 2][j] << 16), c[e],
                         fmaf(__uint_as_float(sz[e / 2][j] & 0xffff0000u), qsum[j][e & 1], sy[e]));
        }
      }
      // --- softmax: keys past a row's last (or before its window) have weight 0, whatever they hold
      bool seen[4 * kN];
#pragma unroll
      for (int e = 0; e < 4 * kN; ++e) {
        seen[e] = true;
        if constexpr (masked.value) {
          const int key = key0 + kg + 8 * (e / 2), hi = cur.s.L - p.Tq + p.row_i[rt * 8 + 2 * t + (e & 1)];
          seen[e] = key <= hi && (p.window < 0 || key >= hi - p.window);
        }
      }
      // In log2 units a score is rounded before the max, one of them, comes off: the largest one then weighs 1 however
      // large it is. (An unrounded product less the max left it half a unit in the last place, 2^7 at 2^31.)
      float x[4 * kN], most_x[2] = {0.f, 0.f};  // the weights, and the lane's largest of each column
#pragma unroll
      for (int e = 0; e < 4 * kN; e += 2) {
        F2 score = f2(s[e], s[e + 1]), factor = f2(down[0], down[1]);
        if constexpr (masked.value) {
          score = mul2(score, f2(down[0] < 0.f ? kvq_power(kLift) : 1.f, down[1] < 0.f ? kvq_power(kLift) : 1.f));
          factor = f2(fabsf(down[0]), fabsf(down[1]));
        }
        score = mul2(score, factor);
        const F2 less = add2(score, f2(-m[0], -m[1]));
        s[e] = lo_of(score), s[e + 1] = hi_of(score);
        x[e] = seen[e] ? ex2(lo_of(less)) : 0.f, x[e + 1] = seen[e + 1] ? ex2(hi_of(less)) : 0.f;
        most_x[0] = fmaxf(most_x[0], x[e]), most_x[1] = fmaxf(most_x[1], x[e + 1]);
      }
      bool raise = most_x[0] > kLazy || most_x[1] > kLazy;
      uint32_t vsz[2 * kN][kGroups];
#pragma unroll
      for (int y = 0; y < 2 * kN; ++y) lds(vsz[y], ap + kp_lds + Shape::kParamBytes + 8 * y * kGroups * 4);
      float top[kGroups];  // the largest scale of this lane's keys (a cache filled by others may hold negative ones)
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        top[j] = fabsf(__uint_as_float(vsz[0][j] << 16));
#pragma unroll
        for (int y = 1; y < 2 * kN; ++y) top[j] = fmaxf(top[j], fabsf(__uint_as_float(vsz[y][j] << 16)));
#pragma unroll
        for (int c = 0; c < 2; ++c) raise |= most_x[c] * unit[j][c] * top[j] > kMostWeight;
      }
      if (__any_sync(0xffffffffu, raise)) {
        // A column's max becomes a whole number, so that the old weights' factor is a power of two, which their sums
        // in acc take up as their unit's.
        int up[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float y = m[c];  // the new max
#pragma unroll
          for (int e = c; e < 4 * kN; e += 2)
            if (seen[e]) y = fmaxf(y, s[e]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
          y = ceilf(y);
          up[c] = static_cast<int>(fminf(y - m[c], 1000.f));
          const float f = ex2(m[c] - y);
          m[c] = y;
#pragma unroll
          for (int e = c; e < 4 * kN; e += 2)
            if (seen[e]) x[e] = ex2(s[e] - y);
          l[c] *= f;
#pragma unroll
          for (int j = 0; j < kGroups; ++j) corr[j][c] *= f;
        }
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
          uint32_t most = 0;  // the tile's largest p |s|, the upper half of the fp32 number: column 2 t, 2 t + 1
#pragma unroll
          for (int y = 0; y < 2 * kN; ++y) {
            const float sc = fabsf(__uint_as_float(vsz[y][j] << 16));
            const float w0 = seen[2 * y] ? x[2 * y] * sc : 0.f;
            const float w1 = seen[2 * y + 1] ? x[2 * y + 1] * sc : 0.f;
            most = __vmaxu2(most, __byte_perm(__float_as_uint(w0), __float_as_uint(w1), 0x7632));
          }
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, o));
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            // in exponent fields: the unit that the sums have now, and the one from here on
            const int at = static_cast<int>(__float_as_uint(unit[j][c]) >> 23) + up[c];
            const int aim = 2 * 127 + kAim - static_cast<int>((most >> (16 * c + 7)) & 0xffu);
            const int to = min(min(at, 127 + kMostUnit), aim);
            unit[j][c] = __uint_as_float(static_cast<uint32_t>(to) << 23);
            const float f = to - at < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 + to - at) << 23);
#pragma unroll
            for (int i = j * (kGroup / 16); i < (j + 1) * (kGroup / 16); ++i) acc[i][c] *= f, acc[i][c + 2] *= f;
          }
        }
      }
      F2 sum = f2(x[0], x[1]);  // (the tile's by themselves first: a light key may be lost to what a heavy one left)
#pragma unroll
      for (int e = 2; e < 4 * kN; e += 2) sum = add2(sum, f2(x[e], x[e + 1]));
      l[0] += lo_of(sum), l[1] += hi_of(sum);
      // --- values
#pragma unroll
      for (int y = 0; y < kN; ++y) {
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
          uint32_t b[2];  // the weights of keys kg (+ 8) and columns 2 t, 2 t + 1, then transposed
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const int e = 4 * y + 2 * z;
            const uint32_t w = vsz[2 * y + z][j];
            const float sc = __uint_as_float(w << 16), zc = fmaf(kCentre, sc, __uint_as_float(w & 0xffff0000u));
            float w0 = x[e] * unit[j][0] * sc, w1 = x[e + 1] * unit[j][1] * sc;
            if constexpr (masked.value) {  // (a NaN in a key that a row does not see stays out of it)
              if (!seen[e]) w0 = 0.f;
              if (!seen[e + 1]) w1 = 0.f;
              if (seen[e]) corr[j][0] = fmaf(x[e], zc, corr[j][0]);
              if (seen[e + 1]) corr[j][1] = fmaf(x[e + 1], zc, corr[j][1]);
            } else {
              corr[j][0] = fmaf(x[e], zc, corr[j][0]);
              corr[j][1] = fmaf(x[e + 1], zc, corr[j][1]);
            }
            b[z] = movmatrix(pack_f16x2(w0, w1));
          }
          // The lane's dims j * kGroup + g * (kGroup / 8) + ... of its four keys: eight dims a word (4 bits) or four (8
          // bits); with 4 bits and groups of 32 the lane's four dims are half a word.
          constexpr int kRead = kVWords < 1 ? 1 : kVWords;
          const uint32_t a0 = ((at + v0_lds) ^ (j * (kGroup * kBits / 8))) + 16 * y * kRowBytes;
          const uint32_t a1 = ((at + v1_lds) ^ (j * (kGroup * kBits / 8))) + 16 * y * kRowBytes;
          uint32_t va[kRead], vb[kRead], vc[kRead], vd[kRead];
          lds(va, a0);
          lds(vb, a1);
          lds(vc, a0 + 8 * kRowBytes);
          lds(vd, a1 + 8 * kRowBytes);
          constexpr int kTiles = kGroup / 16;  // tiles of 16 dims in the group
#pragma unroll
          for (int r = 0; r < kGroup / 32; ++r) {  // four dims at a time
            if constexpr (kBits == 4) {
              const uint32_t sel = (kVWords < 1 ? g & 1 : r & 1) ? 0x7632u : 0x5410u;
              uint32_t u[4], v[4];
              widen4<true>(u, __byte_perm(va[r / 2], vb[r / 2], sel));
              widen4<true>(v, __byte_perm(vc[r / 2], vd[r / 2], sel));
              mma_16x8x16(acc[j * kTiles + 2 * r], u[0], u[1], v[0], v[1], b[0], b[1]);
              mma_16x8x16(acc[j * kTiles + 2 * r + 1], u[2], u[3], v[2], v[3], b[0], b[1]);
            } else {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t sel = h ? 0x7632u : 0x5410u;
                const uint32_t u = __byte_perm(va[r], vb[r], sel), v = __byte_perm(vc[r], vd[r], sel);
                mma_16x8x16(acc[j * kTiles + 2 * r + h], widen8<true, 0x0200>(u), widen8<true, 0x0301>(u),
                            widen8<true, 0x0200>(v), widen8<true, 0x0301>(v), b[0], b[1]);
              }
            }
          }
        }
      }
    };

    int key0 = cur.s.start + cur.tile * kTile;
    for (int n = n_tiles; n > 0; --n, key0 += kTile) {
      cp_async_wait<kStages - 2>();
      __syncwarp();  // this tile is in, and every lane has read the one before it
      fetch(stage == 0 ? kStages - 1 : stage - 1);
      const uint32_t at = ring + stage * Shape::kStageBytes;
      if (key0 <= plain_to && (p.window < 0 || key0 >= cur.s.L - 1 - p.window))
        tile(at, at + 2 * Shape::kCodeBytes, key0, std::false_type(), std::integral_constant<int, kHalves>());
      else  // some row does not see some key, or a score has two factors: rare in long caches, and kept small
#pragma unroll 1
        for (int y = 0; y < kHalves; ++y)
          tile(at + 16 * y * kRowBytes, at + 2 * Shape::kCodeBytes + 16 * y * kGroups * 4, key0 + 16 * y,
               std::true_type(), std::integral_constant<int, 1>());
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }

    // --- the piece's result
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        l[c] += __shfl_xor_sync(0xffffffffu, l[c], o);
#pragma unroll
        for (int j = 0; j < kGroups; ++j) corr[j][c] += __shfl_xor_sync(0xffffffffu, corr[j][c], o);
      }
    }
    constexpr float kSecond = kBits == 4 ? 0.0625f : 1.f;  // rows g + 8 of a tile: second (fourth) nibbles
    if (!whole && slot) __syncwarp();  // (every lane has read the last tile, which the piece overwrites)
    float* to_o = piece_o(slot, warp);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = rt * 8 + 2 * t + c;
      if (r >= R) continue;
      const int i = p.row_i[r], h = cur.hk * G + p.row_g[r];
      const float inv = kvq_factor(l[c]);
      const size_t off = ((static_cast<size_t>(cur.b) * p.Tq + i) * p.H + h) * 128;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int j = x / (kGroup / 16), dim = j * kGroup + g * (kGroup / 8) + 2 * (x % (kGroup / 16));
        // 2^24 of the codes, then what a weight's unit is: their product may pass fp32's range where the result does not
        const float inverse = kvq_inverse(unit[j][c]);
        const float a = fmaf(acc[x][c] * 0x1p24f, inverse, corr[j][c]);
        const float b = fmaf(acc[x][c + 2] * (0x1p24f * kSecond), inverse, corr[j][c]);
        if (!whole)
          *reinterpret_cast<float2*>(to_o + (2 * t + c) * 128 + dim) = make_float2(a, b);
        else if (ATTN_IN_RANGE(off + dim, 2, n_q, kSiteKvqDecO, &g_kvq_error))
          *reinterpret_cast<uint32_t*>(p.o + off + dim) = sm100::pack_bf16x2(a * inv, b * inv);
      }
      if (g) continue;
      const size_t lse_i = (static_cast<size_t>(cur.b) * p.H + h) * p.Tq + i;
      if (!whole)
        *reinterpret_cast<float2*>(piece_ml(slot, warp) + (2 * t + c) * 2) = make_float2(m[c], l[c]);
      else if (ATTN_IN_RANGE(lse_i, 1, n_q / 128, kSiteKvqDecLse, &g_kvq_error))
        p.lse[lse_i] = kvq_lse(m[c], l[c]);
    }
    if (!whole && lane == 0 && rt == 0)
      sh_piece[2 * slice + slot] = KvqPiece{cur.b * p.Hkv + cur.hk, cur.tile == 0, cur.end};
    kvq_next_unit<kTile>(p, cur);
  }
  // Sequences without keys: o = 0, lse = -inf, shared out over the CTAs.
  for (int b = __any_sync(0xffffffffu, empty) ? blockIdx.x : p.B; b < p.B; b += gridDim.x) {
    if (kvq_seq<kTile>(p, b).tiles > 0) continue;
    const size_t rows = static_cast<size_t>(p.Tq) * p.H;  // (counted in 28 bits, their 16-byte parts are not)
    for (size_t i = tid + b * rows * 16; i < (b + 1) * rows * 16; i += kKvqThreads)
      if (ATTN_IN_RANGE(i * 8, 8, n_q, kSiteKvqDecO, &g_kvq_error))
        reinterpret_cast<uint4*>(p.o)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (size_t i = tid + b * rows; i < (b + 1) * rows; i += kKvqThreads)
      if (ATTN_IN_RANGE(i, 1, n_q / 128, kSiteKvqDecLse, &g_kvq_error)) p.lse[i] = -INFINITY;
  }
  cp_async_wait<0>();
  __syncthreads();

  // --- the CTA's pieces of one unit, joined by their maxima: a chain begins with a stretch's last piece, or with its
  // first where the unit begins there (or the CTA does), and goes on through the first pieces of the stretches after
  // it. Lane i looks at piece i; a chain's pieces are then the lanes from its head up to the next head.
  static_assert(2 * kKvqWarps <= 32, "a lane per piece");
  const int cta_end = start_of(slices);
  KvqPiece pc = {-1, 0, 0};
  if (lane < 2 * slices) pc = sh_piece[lane];
  const unsigned have = __ballot_sync(0xffffffffu, pc.unit >= 0);
  unsigned heads = __ballot_sync(0xffffffffu, pc.unit >= 0 && ((lane & 1) || pc.begins || lane == 0));
  for (int n = 0; heads; ++n) {
    const int i0 = __ffs(heads) - 1;
    heads &= heads - 1;
    int r = (warp + 64 * kKvqWarps - n * R) % kKvqWarps;  // the chains' rows are the warps' in turn
    if (r >= R) continue;
    const unsigned chain = have & (0xffffffffu << i0) & (heads ? (1u << (__ffs(heads) - 1)) - 1u : 0xffffffffu);
    const int pieces = __popc(chain);  // the head, then the first pieces of the stretches after it
    const int unit = __shfl_sync(0xffffffffu, pc.unit, i0), end = __shfl_sync(0xffffffffu, pc.end, i0);
    const bool begins = __shfl_sync(0xffffffffu, pc.begins, i0), ends = end <= cta_end;
    const int b = unit / p.Hkv, hk = unit - b * p.Hkv;
    for (; r < R; r += kKvqWarps) {
      auto slot_of = [&](int s) { return s ? 0 : i0 & 1; };
      auto warp_of = [&](int s) { return (i0 / 2 + s) * n_rt + r / 8; };  // piece s: its stretch's warp that had row r
      float2 ml = make_float2(kKvqNone, 0.f);
      if (lane < pieces) ml = *reinterpret_cast<const float2*>(piece_ml(slot_of(lane), warp_of(lane)) + (r % 8) * 2);
      float M = ml.x;
#pragma unroll
      for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float f = ex2(ml.x - M);
      float L = ml.y * f;
#pragma unroll
      for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
      float4 o4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int s = 0; s < pieces; ++s) {
        const float fs = __shfl_sync(0xffffffffu, f, s);
        const float4 x = *reinterpret_cast<const float4*>(piece_o(slot_of(s), warp_of(s)) + (r % 8) * 128 + lane * 4);
        o4.x = fmaf(x.x, fs, o4.x), o4.y = fmaf(x.y, fs, o4.y), o4.z = fmaf(x.z, fs, o4.z), o4.w = fmaf(x.w, fs, o4.w);
      }
      if (begins && ends) {
        const int q = p.row_i[r], h = hk * G + p.row_g[r];
        const float inv = kvq_factor(L);
        const size_t off = ((static_cast<size_t>(b) * p.Tq + q) * p.H + h) * 128 + lane * 4;
        if (ATTN_IN_RANGE(off, 4, n_q, kSiteKvqDecO, &g_kvq_error))
          *reinterpret_cast<uint2*>(p.o + off) =
              make_uint2(sm100::pack_bf16x2(o4.x * inv, o4.y * inv), sm100::pack_bf16x2(o4.z * inv, o4.w * inv));
        const size_t lse_i = (static_cast<size_t>(b) * p.H + h) * p.Tq + q;
        if (lane == 0 && ATTN_IN_RANGE(lse_i, 1, n_q / 128, kSiteKvqDecLse, &g_kvq_error)) p.lse[lse_i] = kvq_lse(M, L);
      } else {
        const int slot = i0 == 0 ? 0 : 1;
        const size_t part = (static_cast<size_t>(blockIdx.x) * 2 + slot) * R + r;
        if (ATTN_IN_RANGE(part, 1, static_cast<size_t>(gridDim.x) * 2 * R, kSiteKvqDecPart, &g_kvq_error)) {
          *reinterpret_cast<float4*>(p.part_o + part * 128 + lane * 4) = o4;
          if (lane == 0) *reinterpret_cast<float2*>(p.part_ml + part * 2) = make_float2(M, L);
        }
        if (r == 0 && lane == 0 && begins)  // it begins here and goes on past this CTA
        {
          // the CTA of its last place, to one
          int c = static_cast<int>(static_cast<long long>(end - 1) * gridDim.x / total);
          while (c > 0 && begin_of(c * slices) >= end) --c;
          while (begin_of((c + 1) * slices) < end) ++c;  // (ends: begin_of(gridDim.x * slices) is the row's end)
          p.spans[blockIdx.x] = KvqSpan{unit, c, slot, 0};
        }
      }
    }
  }
}

// ------------------------------------------------------------------------------------------------ merge kernel

// Block (x, y): rows kRows y .. kRows (y + 1) - 1 of the unit that begins in the split kernel's CTA x and goes on
// past it, if there is one: O = sum_s O_s 2^(m_s - M) / sum_s l_s 2^(m_s - M) over its pieces, M = max_s m_s. The
// block's 8 warps share the rows and, where there are fewer rows, each row's pieces; a lane takes four dims. A
// running maximum as in the split kernel, so that a piece is read once, with its maximum and sum.
template <int kRows>
__global__ void __launch_bounds__(256) kvq_decode_merge_kernel(const KvqDecodeParams p) {
  constexpr int kSlices = 8 / kRows;  // warps that share a row's pieces
  __shared__ float2 sh_ml[8];
  __shared__ float4 sh_o[8][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the split kernel's results
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int x = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32, R = p.R;
  const KvqSpan span = p.spans[x];
  if (span.unit < 0) return;
  const int n = span.last_cta - x + 1;  // pieces: this CTA's slot, then the first slot of each CTA after it
  if (!ATTN_IN_RANGE(span.last_cta, 1, gridDim.x, kSiteKvqDecPart, &g_kvq_error)) return;
  const int r = blockIdx.y * kRows + warp / kSlices;
  float M = kKvqNone, l = 0.f;
  float4 o4 = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r < R) {
    constexpr int kAtOnce = 4;
    for (int s0 = warp % kSlices; s0 < n; s0 += kAtOnce * kSlices) {
      float2 ml[kAtOnce];
      float4 v[kAtOnce];
      float top = M;
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int s = s0 + u * kSlices;
        ml[u] = make_float2(-INFINITY, 0.f), v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s < n) {
          const size_t part = (static_cast<size_t>(x + s) * 2 + (s == 0 ? span.slot : 0)) * R + r;
          ml[u] = *reinterpret_cast<const float2*>(p.part_ml + part * 2);
          v[u] = reinterpret_cast<const float4*>(p.part_o + part * 128)[lane];
        }
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) top = fmaxf(top, ml[u].x);
      const float down = ex2(M - top);
      M = top;
      l *= down, o4.x *= down, o4.y *= down, o4.z *= down, o4.w *= down;
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const float f = ex2(ml[u].x - M);
        l = fmaf(ml[u].y, f, l);
        o4.x = fmaf(v[u].x, f, o4.x), o4.y = fmaf(v[u].y, f, o4.y);
        o4.z = fmaf(v[u].z, f, o4.z), o4.w = fmaf(v[u].w, f, o4.w);
      }
    }
  }
  if constexpr (kSlices > 1) {  // the row's first warp adds up the others' sums
    sh_o[warp][lane] = o4;
    if (lane == 0) sh_ml[warp] = make_float2(M, l);
    __syncthreads();
    if (warp % kSlices) return;
    float top = M;
#pragma unroll
    for (int w = 1; w < kSlices; ++w) top = fmaxf(top, sh_ml[warp + w].x);
    const float down = ex2(M - top);
    M = top;
    l *= down, o4.x *= down, o4.y *= down, o4.z *= down, o4.w *= down;
#pragma unroll
    for (int w = 1; w < kSlices; ++w) {
      const float2 ml = sh_ml[warp + w];
      const float4 v = sh_o[warp + w][lane];
      const float f = ex2(ml.x - M);
      l = fmaf(ml.y, f, l);
      o4.x = fmaf(v.x, f, o4.x), o4.y = fmaf(v.y, f, o4.y), o4.z = fmaf(v.z, f, o4.z), o4.w = fmaf(v.w, f, o4.w);
    }
  }
  if (r >= R) return;
  const int b = span.unit / p.Hkv, hk = span.unit % p.Hkv, i = p.row_i[r], h = hk * (p.H / p.Hkv) + p.row_g[r];
  const float inv = kvq_factor(l);
  const size_t n_out = static_cast<size_t>(p.B) * p.Tq * p.H;
  (void)n_out;
  const size_t off = (static_cast<size_t>(b) * p.Tq + i) * p.H + h;
  if (ATTN_IN_RANGE(off, 1, n_out, kSiteKvqDecO, &g_kvq_error))
    reinterpret_cast<uint2*>(p.o + off * 128)[lane] =
        make_uint2(sm100::pack_bf16x2(o4.x * inv, o4.y * inv), sm100::pack_bf16x2(o4.z * inv, o4.w * inv));
  const size_t lse_i = (static_cast<size_t>(b) * p.H + h) * p.Tq + i;
  if (lane == 0 && ATTN_IN_RANGE(lse_i, 1, n_out, kSiteKvqDecLse, &g_kvq_error)) p.lse[lse_i] = kvq_lse(M, l);
}

}  // namespace attn
