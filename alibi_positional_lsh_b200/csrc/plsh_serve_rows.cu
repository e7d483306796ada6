// T~ of a few new tokens of each sequence (one when decoding) against the paged cache, bf16.
//
// Rows are the (token, query head) pairs that share a KV head, up to 16 in a block; their keys are the
// window below them, so the work is reading K and V once: 2 (d + 1) bytes a key and KV head when the pages
// hold e4m3. One to eight blocks share a window, by its width, four warps a block, each taking steps of 16 keys on its own:
//   S[16 rows][16 keys] = Q K^T   d/16 x 2 products mma.m16n8k16 per step, fp32 accumulation
//   P = c 2^(S sc - m), against the warp's own running maximum m over keys with c > 0
//   O[16 rows][d] += P V
// and the partial rows (m, l, O) meet at the end, the warps' in shared memory and the blocks' across it (eight blocks
// are a cluster: one wide window's, or two, four or eight narrower ones'): one launch, no scratch, and always
// joined in the same order, so results do not depend on timing.
//
// K and V go from the pages to registers, 16 bytes at a time, and are not staged: a dot product may take its d in any order, so
// lane (g, t) of a warp takes bytes 16 t .. 16 t + 15 of each 64 of key g's row as its operand of four products, and Q is
// loaded in the same order. For P V it takes columns (d/8) g .. of four keys and pairs them up by key.
// e4m3 values become f16 exactly (one conversion per pair) for S, with each row of Q scaled by a power of two into f16's range,
// and bf16 exactly for P V; the rows' exponents multiply S and P, in fp32.
//
// Counts: blocks are contiguous, so hash k puts key j with row i >= j exactly if i's block begins at or below j. With p0 the
// block's first token, the beginning b_k of p0's own block follows from the table in closed form (no mask is read for the window, whose
// load would be one more trip to memory before K and V), the lowest of them is the window's exact end, and
//   c_ij = popcount({k : b_k <= j} without the hashes that open a block in (p0, i]),
// one word per key and head and one word per row. The up to 15 keys above p0 are a step of their own,
// counted from the masks.
//
// What bounds it: a few tokens read so little that the time is the chain of trips to memory (lengths and table; pages;
// exponents, K and V; the cluster's exchange); a batch reads each window once, 16 keys a step with the next step's rows on their way.
#include <cooperative_groups.h>

#include "plsh_binid.cuh"
#include "plsh_serve.cuh"

namespace plsh {
namespace {

namespace cg = cooperative_groups;
using namespace serve;

constexpr int kThreads = 128, kWarps = 4, kRowsMax = 16, kStep = 16;
constexpr int kCluster = 8;
constexpr int kChunkSteps = 64;  // steps whose pages a block holds at a time
constexpr int kMaxSplitHeads = 64;
constexpr int kMaxGroup = 16;    // query heads of a block (a larger group takes several blocks)

// How a launch's windows are dealt out: 2^lg[kv head] blocks of each (with more KV heads, lg_all), kv heads from the last.
struct Split {
  int tokens, heads, row_blocks, head_blocks;  // of a block; blocks of a sequence's rows and of a group's heads
  int per_head;                                // windows of a KV head: sequences x row blocks x head blocks
  int lg_all;
  uint8_t lg[kMaxSplitHeads];
};

// Shared memory of a block for `heads` query heads and `rows` rows.
template <int D, typename MaskT>
struct Layout {
  int o, ml, begin, keep, row_off, tail, page, row, ks, vs, total;
  __host__ __device__ Layout(int heads, int rows) {
    int at = 0;
    auto take = [&](int bytes) {
      const int here = at;
      at += (bytes + 15) / 16 * 16;
      return here;
    };
    o = take(kWarps * rows * (D + 4) * 4);         // [warp][row][D + 4]: the warps' rows of O
    ml = take(2 * kWarps * rows * 4);              // [2][warp][row]: their m and l
    begin = take(heads * PLSH_MAX_S * 4);          // [head][hash]: where p0's block begins
    keep = take(kWarps * heads * kStep * (int)sizeof(MaskT));  // [warp][head][key]: hashes whose block reaches the key
    row_off = take(rows * (int)sizeof(MaskT));     // [row]: hashes that open a block in (p0, i]
    tail = take(heads * kStep * (int)sizeof(MaskT));    // [head][k]: masks of positions p0 + 1 + k
    page = take((kChunkSteps + 2) * 4);            // pages of the chunk's positions (they hold 16 and more)
    row = take(2 * kWarps * kStep * 8);            // [stage][warp][key]: its row in the pages (-1: none)
    ks = take(2 * kWarps * kStep * 4);             // the same: 2^exponent of K and of V
    vs = take(2 * kWarps * kStep * 4);
    total = at;
  }
};

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

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Two e4m3 bytes as f16 and as bf16, both exact.
__device__ __forceinline__ uint32_t e4m3_f16x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return h;
}
__device__ __forceinline__ uint32_t e4m3_bf16x2(uint32_t two) {
  const uint32_t h = e4m3_f16x2(two);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return bf16x2(f.x, f.y);
}
__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

template <int D, typename MaskT, bool kQuant>
__global__ void __launch_bounds__(kThreads, D == 128 && !kQuant ? 2 : 3)
serve_rows_kernel(ServeArgs a, Split sp) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  if (blockIdx.x == 0) check_seqs(a.sq, a.err);

  // KV heads from the last (with the usual slopes, the widest windows first), a KV head's windows 8 / C to a cluster
  const int cl = blockIdx.x / kCluster, in_cl = blockIdx.x % kCluster;
  int kvh, lg = sp.lg_all, x;
  if (a.H_kv > kMaxSplitHeads) {
    const int per = (sp.per_head << lg) / kCluster + ((sp.per_head << lg) % kCluster != 0);
    kvh = a.H_kv - 1 - cl / per;
    x = cl % per;
  } else {
    x = cl;
    for (kvh = a.H_kv - 1; kvh > 0; --kvh) {
      lg = sp.lg[kvh];
      const int per = ((sp.per_head << lg) + kCluster - 1) / kCluster;
      if (x < per) break;
      x -= per;
    }
    lg = sp.lg[kvh];
  }
  const int C = 1 << lg, rank = in_cl & (C - 1), rank0 = in_cl - rank;  // the window's blocks are rank0 .. rank0 + C - 1 of the cluster
  x = (x << (3 - lg)) + (in_cl >> lg);                                  // the window's number within the KV head
  const int tokens = sp.tokens, heads = sp.heads;
  const int hb = x % sp.head_blocks;
  x /= sp.head_blocks;
  const int rb = x % sp.row_blocks, sid = x / sp.row_blocks;
  const int G = a.H / a.H_kv, h0 = kvh * G + hb * heads, nh = min(heads, G - hb * heads);
  Seq sq{};
  if (sid < a.sq.S) sq = load_seq(a.sq, sid);
  const int first = rb * tokens;                              // the block's first token in the sequence
  const int nt = min(tokens, sq.len - first);
  // nothing here (or a longer sequence, the tile kernel's): the cluster's barriers do not wait for a block that has ended, and
  // nobody reads its memory
  if (sid >= a.sq.S || nt <= 0 || sq.len > a.few) return;
  const int rows = nt * nh, p0 = sq.pos0 + first, c0 = sq.c0 + first;
  const MaskT* bmask = static_cast<const MaskT*>(a.bmask);
  const int max_rows = tokens * heads;  // of any block of the launch, alike for the whole cluster
  const Layout<D, MaskT> at_(heads, max_rows);
  float* const s_o = reinterpret_cast<float*>(smem_raw + at_.o);
  float* const s_ml = reinterpret_cast<float*>(smem_raw + at_.ml);
  int* const s_begin = reinterpret_cast<int*>(smem_raw + at_.begin);
  MaskT* const s_keep = reinterpret_cast<MaskT*>(smem_raw + at_.keep);
  MaskT* const s_row_off = reinterpret_cast<MaskT*>(smem_raw + at_.row_off);
  MaskT* const s_tail = reinterpret_cast<MaskT*>(smem_raw + at_.tail);
  long long* const s_row = reinterpret_cast<long long*>(smem_raw + at_.row);
  float* const s_ks = reinterpret_cast<float*>(smem_raw + at_.ks);
  float* const s_vs = reinterpret_cast<float*>(smem_raw + at_.vs);
  int* const s_page = reinterpret_cast<int*>(smem_raw + at_.page);

  // where the blocks of p0 begin, and so the window; masks above p0
  int lo = p0;
  for (int e = tid; e < nh * PLSH_MAX_S; e += kThreads) s_begin[e] = 0x7fffffff;
  __syncthreads();
  for (int e = tid; e < nh * a.s; e += kThreads) {
    const int h = e / a.s, k = e % a.s;
    const int b = block_begin(Binning::from_table(a.table + (static_cast<size_t>(h0 + h) * a.s + k) * 2), p0);
    s_begin[h * PLSH_MAX_S + k] = b;
    lo = min(lo, b);
  }
  for (int e = tid; e < nh * kStep; e += kThreads) {
    const int h = e / kStep, k = e % kStep;
    s_tail[e] = k + 1 < nt ? bmask[static_cast<size_t>(h0 + h) * a.sq.max_len + p0 + 1 + k] : static_cast<MaskT>(0);
  }
  __shared__ int s_lo[kWarps];
  lo = __reduce_min_sync(0xffffffffu, lo);
  if (lane == 0) s_lo[warp] = lo;

  // Q: lane (g, t) holds rows g and g + 8, in K's order of d
  float inv_scale[2] = {1.0f, 1.0f};
  uint32_t q[D / 16][4];
  {
    float amax[2] = {0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = g + 8 * u;
      const bool on = r < rows;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.Q) +
          (on ? static_cast<long long>(c0 + r / nh) * a.qs.token + (h0 + r % nh) * a.qs.head : 0);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (on) {
          w[0] = *reinterpret_cast<const uint4*>(src + 64 * c + 16 * t);
          w[1] = *reinterpret_cast<const uint4*>(src + 64 * c + 16 * t + 8);
        }
        const uint32_t ws[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          q[4 * c + k][u] = ws[2 * k];
          q[4 * c + k][u + 2] = ws[2 * k + 1];
        }
        if (kQuant) {
#pragma unroll
          for (int k = 0; k < 8; ++k) amax[u] = fmaxf(amax[u], fmaxf(fabsf(bf16_lo(ws[k])), fabsf(bf16_hi(ws[k]))));
        }
      }
    }
    if (kQuant) {  // rows scaled to a largest magnitude in [1, 2): f16 then holds bf16's eight bits down to 2^-14 of it
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        amax[u] = fmaxf(amax[u], __shfl_xor_sync(0xffffffffu, amax[u], 1));
        amax[u] = fmaxf(amax[u], __shfl_xor_sync(0xffffffffu, amax[u], 2));
        const int e = min(126, max(-126, static_cast<int>(__float_as_uint(amax[u]) >> 23) - 127));
        inv_scale[u] = pow2(e);
        const float sc = pow2(-e);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          q[k][u] = f16x2(bf16_lo(q[k][u]) * sc, bf16_hi(q[k][u]) * sc);
          q[k][u + 2] = f16x2(bf16_lo(q[k][u + 2]) * sc, bf16_hi(q[k][u + 2]) * sc);
        }
      }
    }
  }
  const float sc0 = 1.4426950408889634f / sqrtf(static_cast<float>(D));
  const float sc[2] = {sc0 * inv_scale[0], sc0 * inv_scale[1]};

  __syncthreads();
  lo = min(min(s_lo[0], s_lo[1]), min(s_lo[2], s_lo[3]));
  // this block's keys: steps of 16 down from p0, dealt out to the cluster in runs; step i: keys p0 - 16 i - 15 .. p0 - 16 i
  const int steps = (p0 - lo + kStep) / kStep;
  const int per = (steps + C - 1) / C;
  const int s0 = rank * per, s1 = min(steps, s0 + per);
  if (tid < rows) {
    MaskT v = 0;
    for (int k = 0; k < tid / nh; ++k) v |= s_tail[tid % nh * kStep + k];
    s_row_off[tid] = v;
  }

  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  MaskT mine[2] = {0, 0};  // of rows g and g + 8: the hashes that may count, and the row's head in the group
  int hh[2] = {0, 0};

  // places of this warp's step in flight
  auto place = [&](int stage) { return (stage * kWarps + warp) * kStep; };
  // one step: 16 keys at places at .. of sm.row;
  // byte n of c4[u]: the count of row g + 8 u with key 2 t, 2 t + 1, 2 t + 8 or 2 t + 9
  auto load_k = [&](int at, uint4 (&kr)[2][D / 64][kQuant ? 1 : 2]) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const long long row = s_row[at + 8 * n + g];
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        if constexpr (kQuant) {
          kr[n][c][0] = row >= 0 ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.pg.k) + row * D + 64 * c + 16 * t))
                                 : make_uint4(0, 0, 0, 0);
        } else {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.pg.k) + row * D + 64 * c + 16 * t);
          kr[n][c][0] = row >= 0 ? __ldg(src) : make_uint4(0, 0, 0, 0);
          kr[n][c][1] = row >= 0 ? __ldg(src + 1) : make_uint4(0, 0, 0, 0);
        }
      }
    }
  };
  // V's columns (D/8) g .. of keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9: D/8 values each
  constexpr int kVWords = kQuant ? D / 32 : D / 16;  // 32-bit words
  auto load_v = [&](int at, uint32_t (&vr)[4][kVWords]) {
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const long long row = s_row[at + 2 * t + (n & 1) + 8 * (n >> 1)];
      const uint8_t* src = static_cast<const uint8_t*>(a.pg.v) + row * (kQuant ? D : 2 * D) + (kQuant ? 1 : 2) * (D / 8) * g;
      if constexpr (kVWords % 4 == 0) {
#pragma unroll
        for (int i = 0; i < kVWords / 4; ++i) {
          const uint4 w = row >= 0 ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
          vr[n][4 * i] = w.x; vr[n][4 * i + 1] = w.y; vr[n][4 * i + 2] = w.z; vr[n][4 * i + 3] = w.w;
        }
      } else {
        const uint2 w = row >= 0 ? __ldg(reinterpret_cast<const uint2*>(src)) : make_uint2(0, 0);
        vr[n][0] = w.x; vr[n][1] = w.y;
      }
    }
  };
  auto step = [&](int at, const uint4 (&kr)[2][D / 64][kQuant ? 1 : 2], const uint32_t (&vr)[4][kVWords], const uint32_t (&c4)[2]) {
    float x[2][4];
    auto count = [&](int u, int n) { return (c4[u] >> (8 * n)) & 0xFFu; };
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int cc = 0; cc < D / 64; ++cc) {
        if constexpr (kQuant) {
          const uint32_t w[4] = {kr[n][cc][0].x, kr[n][cc][0].y, kr[n][cc][0].z, kr[n][cc][0].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_f16(acc, q[4 * cc + k], e4m3_f16x2(w[k]), e4m3_f16x2(w[k] >> 16));
        } else {
          const uint32_t w[8] = {kr[n][cc][0].x, kr[n][cc][0].y, kr[n][cc][0].z, kr[n][cc][0].w,
                                 kr[n][cc][1].x, kr[n][cc][1].y, kr[n][cc][1].z, kr[n][cc][1].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_bf16(acc, q[4 * cc + k], w[2 * k], w[2 * k + 1]);
        }
      }
      // acc: rows g (0, 1) and g + 8 (2, 3), keys 8 n + 2 t, + 1
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ks = kQuant ? s_ks[at + 8 * n + 2 * t + e] : 1.0f;
        x[0][2 * n + e] = acc[e] * ks * sc[0];
        x[1][2 * n + e] = acc[2 + e] * ks * sc[1];
      }
    }
    uint32_t p[4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float top = m[u];
#pragma unroll
      for (int n = 0; n < 4; ++n) top = count(u, n) > 0 ? fmaxf(top, x[u][n]) : top;
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      if (top > m[u]) {
        const float alpha = exp2f(m[u] - top);  // 0 the first time
        l[u] *= alpha;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][2 * u] *= alpha;
          o[i][2 * u + 1] *= alpha;
        }
        m[u] = top;
      }
      float w[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        w[n] = count(u, n) > 0 ? static_cast<float>(count(u, n)) * exp2f(x[u][n] - m[u]) : 0.0f;
        l[u] += w[n];
        if (kQuant) w[n] *= count(u, n) > 0 ? s_vs[at + 2 * t + (n & 1) + 8 * (n >> 1)] : 0.0f;
      }
      p[u] = bf16x2(w[0], w[1]);
      p[u + 2] = bf16x2(w[2], w[3]);
    }
    // O += P V: column (D/8) g + i of V is n = g of product i
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      uint32_t b0, b1;
      if constexpr (kQuant) {
        const uint32_t sel = 0x0040u + 0x0011u * (i & 3);  // byte i & 3 of both
        b0 = e4m3_bf16x2(__byte_perm(vr[0][i >> 2], vr[1][i >> 2], sel));
        b1 = e4m3_bf16x2(__byte_perm(vr[2][i >> 2], vr[3][i >> 2], sel));
      } else {
        const uint32_t sel = (i & 1) ? 0x7632u : 0x5410u;
        b0 = __byte_perm(vr[0][i >> 1], vr[1][i >> 1], sel);
        b1 = __byte_perm(vr[2][i >> 1], vr[3][i >> 1], sel);
      }
      mma_bf16(o[i], p, b0, b1);
    }
  };

  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = g + 8 * u;
    if (r < rows) {
      mine[u] = static_cast<MaskT>(~s_row_off[r]);
      hh[u] = r % nh;
    }
  }
  // exponents of the rows at places at ..: lanes 0 .. 15 K's, 16 .. 31 V's
  auto exponents = [&](int at) {
    if (kQuant) {
      const long long row = s_row[at + (lane & 15)];
      return row >= 0 ? pow2((lane < 16 ? a.pg.k_exp : a.pg.v_exp)[row]) : 0.0f;
    }
    return 0.0f;
  };
  auto put_exponents = [&](int at, float e) {
    if (kQuant) (lane < 16 ? s_ks : s_vs)[at + (lane & 15)] = e;
  };

  // ---- the keys above p0, one step of the first block's first warp
  if (rank == 0 && warp == 0 && nt > 1) {
    const int at = place(0);
    if (lane < kStep) s_row[at + lane] = lane + 1 < nt ? page_row(a.pg, sid, p0 + 1 + lane, kvh, a.err) : -1;
    __syncwarp();
    uint4 kr[2][D / 64][kQuant ? 1 : 2];
    uint32_t vr[4][kVWords];
    load_k(at, kr);
    load_v(at, vr);
    put_exponents(at, exponents(at));
    __syncwarp();
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = g + 8 * u, tok = r / nh;  // the row's token: position p0 + tok
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int k = 2 * t + (n & 1) + 8 * (n >> 1);  // key p0 + 1 + k
        if (r < rows && k + 1 <= tok) {
          MaskT v = 0;
          for (int y = k + 1; y < tok; ++y) v |= s_tail[hh[u] * kStep + y];
          c[u] |= static_cast<uint32_t>(a.s - popc_mask<MaskT>(v)) << (8 * n);
        }
      }
    }
    step(at, kr, vr, c);
    __syncwarp();
  }

  // ---- the window
  MaskT* const keep = s_keep + warp * heads * kStep;
  for (int b = s0; b < s1; b += kChunkSteps) {
    const int ns = min(kChunkSteps, s1 - b);
    const int slot0 = max(lo, p0 - kStep * (b + ns) + 1) >> a.pg.lg_page, slots = ((p0 - kStep * b) >> a.pg.lg_page) - slot0 + 1;
    __syncthreads();
    for (int k = tid; k < slots; k += kThreads) {
      int page = slot0 + k < a.pg.width ? a.pg.table[static_cast<long long>(sid) * a.pg.width + slot0 + k] : -1;
      if (page < 0 || page >= a.pg.num_pages) {
        atomicOr(a.err, PLSH_DEVERR_PAGE);
        page = -1;
      }
      s_page[k] = page;
    }
    __syncthreads();
    // Step i of the chunk: rows and counts of its keys into the stage's places. False: nothing has weight there. Key k of
    // the step is p0 - 16 (b + i) - k; a lane per hash says which hashes' blocks reach it.
    auto describe = [&](int i, int stage, uint32_t (&c)[2]) {
      const int at = place(stage), j0 = p0 - kStep * (b + i);
      __syncwarp();
      if (lane < kStep) {
        const int j = j0 - lane;
        long long row = -1;
        if (j >= lo) {
          const int page = s_page[(j >> a.pg.lg_page) - slot0];
          if (page >= 0)
            row = ((static_cast<long long>(page) * a.pg.H_kv + kvh) << a.pg.lg_page) + (j & ((1 << a.pg.lg_page) - 1));
        }
        s_row[at + lane] = row;
      }
      for (int h = 0; h < nh; ++h) {
        const int b0 = s_begin[h * PLSH_MAX_S + lane];
        const int b1 = sizeof(MaskT) == 8 ? s_begin[h * PLSH_MAX_S + 32 + lane] : 0;
        MaskT v = 0;
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
          MaskT m = static_cast<MaskT>(__ballot_sync(0xffffffffu, b0 <= j0 - k));
          if (sizeof(MaskT) == 8) m |= static_cast<MaskT>(static_cast<unsigned long long>(__ballot_sync(0xffffffffu, b1 <= j0 - k)) << 32);
          if (lane == k) v = m;
        }
        if (lane < kStep) keep[h * kStep + lane] = v;
      }
      __syncwarp();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        c[u] = 0;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int k = 2 * t + (n & 1) + 8 * (n >> 1);
          if (s_row[at + k] >= 0) c[u] |= static_cast<uint32_t>(popc_mask<MaskT>(static_cast<MaskT>(keep[hh[u] * kStep + k] & mine[u]))) << (8 * n);
        }
      }
      return __any_sync(0xffffffffu, (c[0] | c[1]) != 0) != 0;
    };
    // a warp's steps, the next one's K on its way while this one is computed
    uint4 kr[2][D / 64][kQuant ? 1 : 2];
    uint32_t c[2];
    int i = warp, stage = 0;
    while (i < ns && !describe(i, stage, c)) i += kWarps;
    float ex = 0.0f;
    if (i < ns) {
      load_k(place(stage), kr);
      ex = exponents(place(stage));
    }
    while (i < ns) {
      uint32_t vr[4][kVWords];
      load_v(place(stage), vr);
      put_exponents(place(stage), ex);
      int nx = i + kWarps;
      uint32_t cn[2];
      while (nx < ns && !describe(nx, stage ^ 1, cn)) nx += kWarps;
      uint4 kn[2][D / 64][kQuant ? 1 : 2];
      if (kQuant && nx < ns) {
        load_k(place(stage ^ 1), kn);
        ex = exponents(place(stage ^ 1));
      }
      __syncwarp();
      step(place(stage), kr, vr, c);
      if (!kQuant && nx < ns) load_k(place(stage ^ 1), kn);  // (rows of bf16 take twice the registers)
      i = nx;
      stage ^= 1;
      c[0] = cn[0];
      c[1] = cn[1];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int cc = 0; cc < D / 64; ++cc)
#pragma unroll
          for (int y = 0; y < (kQuant ? 1 : 2); ++y) kr[n][cc][y] = kn[n][cc][y];
    }
  }

  // ---- join: the warps' rows of every block of the cluster
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
    l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
    const int r = g + 8 * u;
    if (r >= rows) continue;
    if (t == 0) {
      s_ml[warp * max_rows + r] = m[u];
      s_ml[(kWarps + warp) * max_rows + r] = l[u];
    }
    // product i's columns n = 2 t, 2 t + 1: V's columns (D/8) (2 t) + i and (D/8) (2 t + 1) + i
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      s_o[(warp * max_rows + r) * (D + 4) + (D / 8) * (2 * t) + i] = o[i][2 * u];
      s_o[(warp * max_rows + r) * (D + 4) + (D / 8) * (2 * t + 1) + i] = o[i][2 * u + 1];
    }
  }
  __syncthreads();
  // the block's warps, into the first one's place
  for (int e = tid; e < rows * (D / 4); e += kThreads) {
    const int r = e / (D / 4), col = e % (D / 4) * 4;
    float top = -INFINITY, total = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w * max_rows + r]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = s_ml[w * max_rows + r];
      const float f = mw == -INFINITY ? 0.0f : exp2f(mw - top);  // -inf: a warp without keys
      const float4 v = *reinterpret_cast<const float4*>(s_o + (w * max_rows + r) * (D + 4) + col);
      total += s_ml[(kWarps + w) * max_rows + r] * f;
      acc[0] += v.x * f;
      acc[1] += v.y * f;
      acc[2] += v.z * f;
      acc[3] += v.w * f;
    }
    *reinterpret_cast<float4*>(s_o + r * (D + 4) + col) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    if (col == 0) *reinterpret_cast<float2*>(s_o + r * (D + 4) + D) = make_float2(top, total);  // behind the row
  }
  auto finish = [&](int r, int col, float top, float total, const float (&acc)[4]) {
    const float inv = 1.0f / total;
    const size_t at = static_cast<size_t>(c0 + r / nh) * a.H + h0 + r % nh;
    const float out[4] = {acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv};
    store4f(static_cast<__nv_bfloat16*>(a.O) + at * D + col, out);
    if (col == 0) a.row_sum[at] = (log2f(total) + top) * 0.6931471805599453f - logf(static_cast<float>(a.s));
  };
  cluster.sync();
  // the window's blocks, each joining its share of the elements
  for (int e = rank + C * tid; e < rows * (D / 4); e += C * kThreads) {
    const int r = e / (D / 4), col = e % (D / 4) * 4;
    float2 ml[kCluster];
    float4 v[kCluster];
    float top = -INFINITY, total = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int b = 0; b < kCluster; ++b) {
      if (b >= C) break;
      const float* ro = cluster.map_shared_rank(s_o, rank0 + b) + r * (D + 4);
      ml[b] = *reinterpret_cast<const float2*>(ro + D);
      v[b] = *reinterpret_cast<const float4*>(ro + col);
      top = fmaxf(top, ml[b].x);
    }
#pragma unroll
    for (int b = 0; b < kCluster; ++b) {
      if (b >= C) break;
      const float f = ml[b].x == -INFINITY ? 0.0f : exp2f(ml[b].x - top);
      total += ml[b].y * f;
      acc[0] += v[b].x * f;
      acc[1] += v[b].y * f;
      acc[2] += v[b].z * f;
      acc[3] += v[b].w * f;
    }
    finish(r, col, top, total, acc);
  }
  cluster.sync();  // the others have read this block's rows
}

template <int D, typename MaskT, bool kQuant>
int launch(const ServeArgs& a, cudaStream_t st) {
  const int G = a.H / a.H_kv;
  const int most = a.sq.max_new < a.few ? a.sq.max_new : a.few;
  Split sp{};
  sp.heads = G < kMaxGroup ? G : kMaxGroup;
  sp.head_blocks = ceil_div(G, sp.heads);
  sp.tokens = most < kRowsMax / sp.heads ? most : kRowsMax / sp.heads;
  sp.row_blocks = ceil_div(most, sp.tokens);
  const long long per_head = static_cast<long long>(a.sq.S) * sp.row_blocks * sp.head_blocks;
  if (per_head * kCluster * a.H_kv > 0x7fffffffLL) return fail(PLSH_ERR_RANGE, "plsh_paged_fwd: too many rows");
  sp.per_head = static_cast<int>(per_head);
  // Blocks of a window: one for each `keys` keys of the widest head's longest block, 64 (a step a warp) while the launch then has
  // up to four blocks an SM, else the fewest doublings that come near it.
  long long clusters = 0;
  for (int keys = kWarps * kStep; keys <= 4096; keys *= 2) {
    clusters = 0;
    long long blocks = 0;
    for (int k = 0; k < a.H_kv; ++k) {
      int w = 1;
      for (int h = 0; h < G; ++h) {
        const int x = a.windows_host ? a.windows_host[k * G + h] : a.max_window;
        w = x > w ? x : w;
      }
      int lg = 0;
      while (lg < 3 && (static_cast<long long>(keys) << lg) < w) ++lg;
      if (a.H_kv > kMaxSplitHeads) lg = sp.lg_all = lg > sp.lg_all && k > 0 ? lg : k > 0 ? sp.lg_all : lg;
      else sp.lg[k] = static_cast<uint8_t>(lg);
      blocks += per_head << lg;
      clusters += ((per_head << lg) + kCluster - 1) / kCluster;
    }
    if (a.H_kv > kMaxSplitHeads) clusters = a.H_kv * (((per_head << sp.lg_all) + kCluster - 1) / kCluster);
    if (blocks <= 4 * 148) break;
  }
  auto kern = serve_rows_kernel<D, MaskT, kQuant>;
  const int smem = Layout<D, MaskT>(sp.heads, sp.tokens * sp.heads).total;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(serve_rows_kernel)");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * kCluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kCluster;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, a, sp);
  return e == cudaSuccess ? PLSH_OK : cuda_fail(e, "serve_rows_kernel launch");
}

template <int D, typename MaskT>
int launch_src(const ServeArgs& a, cudaStream_t st) {
  return a.pg.k_exp ? launch<D, MaskT, true>(a, st) : launch<D, MaskT, false>(a, st);
}

}  // namespace

int launch_serve_rows(const ServeArgs& a, cudaStream_t st) {
  if (a.d == 128) return a.s <= 32 ? launch_src<128, uint32_t>(a, st) : launch_src<128, unsigned long long>(a, st);
  return a.s <= 32 ? launch_src<64, uint32_t>(a, st) : launch_src<64, unsigned long long>(a, st);
}

}  // namespace plsh
