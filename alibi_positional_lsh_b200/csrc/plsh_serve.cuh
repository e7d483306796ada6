// What the serving kernels share: packed sequences, pages, and the e4m3 rows of a quantised cache.
//
// A call works on S sequences whose new tokens are packed one after another, without padding:
// tokens [cu[s], cu[s + 1]) belong to sequence s, and token t sits at position
// start[s] + t - cu[s] of it (start NULL: every sequence begins at position 0). The lengths live on
// the device only, so a launch covers an upper bound of tiles ("slots") and every slot finds its
// sequence itself.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "plsh_binid.cuh"
#include "plsh_internal.h"

namespace plsh {
namespace serve {

// One sequence of a call. ok is false for an entry that breaks the contract (the sequence is then skipped).
struct Seq {
  int s, c0, len, pos0;
  bool ok;
};

__device__ __forceinline__ Seq load_seq(const SeqArgs& a, int s) {
  Seq q;
  q.s = s;
  q.c0 = a.cu[s];
  const int c1 = a.cu[s + 1];
  q.pos0 = a.start ? a.start[s] : 0;
  q.ok = q.c0 >= 0 && c1 >= q.c0 && c1 <= a.T && q.pos0 >= 0 && q.pos0 <= a.max_len && c1 - q.c0 <= a.max_len - q.pos0 &&
         c1 - q.c0 <= a.max_new;
  q.len = q.ok ? c1 - q.c0 : 0;
  if (!q.ok) q.c0 = q.pos0 = 0;
  return q;
}

// Sets PLSH_DEVERR_SEQUENCE if any sequence of the call is malformed (called by one block).
__device__ __forceinline__ void check_seqs(const SeqArgs& a, uint32_t* err) {
  bool bad = false;
#pragma unroll 1
  for (int s = threadIdx.x; s < a.S; s += blockDim.x) bad |= !load_seq(a, s).ok;
  if (bad) atomicOr(err, PLSH_DEVERR_SEQUENCE);
}

// Tiles of `tile` rows on the grid of absolute positions: a sequence of len tokens from pos0 on touches
// at most floor((c0 + len) / tile) - floor(c0 / tile) + k of them, k = 1 when pos0 is a multiple of
// the tile and 2 else, so slots k s + floor(cu[s] / tile) .. hold them all. Returns the last sequence whose
// first slot is at most x: each step of the search looks at 32 entries, one per lane.
__device__ __forceinline__ int warp_find(const int32_t* cu, int S, int lg_tile, int k, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = S;
#pragma unroll 1
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step;
    const bool at_or_before = lane == 0 || (lane * step < n && (cu[i] >> lg_tile) + k * i <= x);
    const int c = __popc(__ballot_sync(0xffffffffu, at_or_before));
    lo += (c - 1) * step;
    n = min(step, n - (c - 1) * step);
  }
  return lo;
}

// ---------------------------------------------------------------- pages

// The page of position p, or -1 where the page table has none.
__device__ __forceinline__ int find_page(const PageArgs& g, int s, int p) {
  const int slot = p >> g.lg_page;
  const int page = slot < g.width ? g.table[static_cast<long long>(s) * g.width + slot] : -1;
  return page >= 0 && page < g.num_pages ? page : -1;
}

// The row (page, head, place in the page) of position p, or -1.
__device__ __forceinline__ long long find_row(const PageArgs& g, int s, int p, int kvh) {
  const int page = find_page(g, s, p);
  if (page < 0) return -1;
  return ((static_cast<long long>(page) * g.H_kv + kvh) << g.lg_page) + (p & ((1 << g.lg_page) - 1));
}

// The same of a position that the call needs: PLSH_DEVERR_PAGE where there is none.
__device__ __forceinline__ long long page_row(const PageArgs& g, int s, int p, int kvh, uint32_t* err) {
  const long long row = find_row(g, s, p, kvh);
  if (row < 0) atomicOr(err, PLSH_DEVERR_PAGE);
  return row;
}

// The first position of the block of hash `b` that holds p.
__device__ __forceinline__ int block_begin(const Binning& b, int p) {
  if (!b.ok) return 0;
  const int32_t id = b.at(p);
  const double x = ceil((static_cast<double>(id) + b.base) * b.delta - b.u);  // at most a rounding away
  const int guess = x <= 0.0 ? 0 : x >= static_cast<double>(p) ? p : static_cast<int>(x);
  if (b.at(guess) == id && (guess == 0 || b.at(guess - 1) != id)) return guess;
  int good = p, bad = -1;  // ids do not decrease
  while (good - bad > 1) {
    const int mid = bad + (good - bad) / 2;
    if (b.at(mid) == id) good = mid;
    else bad = mid;
  }
  return good;
}

// 2^e as a float, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// The scale of a row with largest finite magnitude m: the least e >= -126 with m <= 448 * 2^e. With
// m = f * 2^x, 1 <= f < 2, and 448 = 1.75 * 2^8 that is x - 8, and one more where f > 1.75. A power of two costs an
// e4m3 value no bits (its own exponent absorbs the scale), makes x * 2^-e exact, so the result
// depends on one rounding only, and makes every dequantised value exact in bf16 (down to its smallest subnormal).
__device__ __forceinline__ int e4m3_exponent(float m) {
  const uint32_t b = __float_as_uint(m);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(e, -126);
}

// Four values, already scaled, as e4m3 bytes (ties to even). NaN and infinities become NaN: the format has no infinity, and
// a saturated one would pass for a number.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Four e4m3 bytes as floats (exact).
__device__ __forceinline__ void e4m3_to_float4(uint32_t w, float (&f)[4]) {
  uint32_t h0, h1;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h0) : "h"(static_cast<uint16_t>(w)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h1) : "h"(static_cast<uint16_t>(w >> 16)));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h0));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h1));
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

// Four consecutive elements as floats.
__device__ __forceinline__ void load4f(const float* p, float (&f)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
}
__device__ __forceinline__ void load4f(const __nv_bfloat16* p, float (&f)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  f[0] = __uint_as_float(v.x << 16);
  f[1] = __uint_as_float(v.x & 0xFFFF0000u);
  f[2] = __uint_as_float(v.y << 16);
  f[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
__device__ __forceinline__ void store4f(float* p, const float (&f)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store4f(__nv_bfloat16* p, const float (&f)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

template <typename MaskT>
__device__ __forceinline__ int popc_mask(MaskT m) {
  if constexpr (sizeof(MaskT) == 8) return __popcll(static_cast<unsigned long long>(m));
  else return __popc(static_cast<unsigned>(m));
}

}  // namespace serve
}  // namespace plsh
