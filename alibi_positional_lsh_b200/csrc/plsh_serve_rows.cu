// T~ of a few new tokens of each sequence (one when decoding) against the paged cache, bf16.
//
// Rows are the (token, query head) pairs that share a KV head, up to 8 in a block; their keys are the
// window below them, so the work is reading K and V once: 2 (d + 1) bytes a key and KV head when the pages
// hold e4m3. A team of 1 to 64 warps shares a window, by its width: some of the eight of a block, or up to eight whole blocks (a
// cluster). A warp takes 32 keys at a time, two steps of 16:
//   S^T[16 keys][8 rows] = K Q^T   d/16 products mma.m16n8k16, fp32 accumulation
//   P = c 2^(S sc - m), against the warp's own running maximum m over keys with c > 0
//   O^T[d][8 rows] += V^T P^T      d/16 products
// O is divided by the sum of the P that it was made with, rounded to bf16 (a row's only key then gives its V exactly; with few
// keys it takes back most of that rounding); row_sum is of P itself.
// The partial rows (m, the sums, O) meet at the end, the warps' in shared memory and the blocks' across it (distributed shared
// memory): one launch, no scratch, and always joined in the same order, so results do not depend on timing. Teams are
// sized so that the launch fits the machine at once: narrow windows with a block each left a second wave of blocks whose
// time is all trips to memory. 64 sequences of 443 to 15,566 tokens, 16/8 heads, d 128, e4m3: 36.9 us; one of 4,096 tokens, 32/8
// heads: 20 us (16 us with a warm L2).
//
// The rows are the products' narrow side: with them on the wide one (16), half of the products, of O's registers and of
// the exponentials were padding. K and V go from the pages to registers, 16 bytes at a time, and are not staged: a dot product may
// take its d in any order, so lane (g, t) of a warp takes bytes 16 t .. 16 t + 15 of each 64 of key g's (and g + 8's) row as
// its operand of four products, and Q is loaded in the same order. For P V it takes columns (d/8) g .. of four keys and pairs
// them up by key; P is turned round by a matrix transpose in registers.
// e4m3 values become f16 exactly (one conversion per pair) for S, with each row of Q scaled by a power of two into f16's range,
// and bf16 exactly for P V; the rows' exponents multiply S and P, in fp32.
//
// Counts: blocks are contiguous, so hash k puts key j with row i >= j exactly if i's block begins at or below j. With p0 the
// block's first token, the beginning b_k of p0's own block follows from the table in closed form (no mask is read for the window, whose
// load would be one more trip to memory before K and V), the lowest of them is the window's exact end, and
//   c_ij = popcount({k : b_k <= j} without the hashes that open a block in (p0, i]),
// one word per key and head and one word per row. The up to 7 keys above p0 are a step of their own,
// counted from the masks.
//
// What bounds it: a few tokens read so little that the time is the chain of trips to memory (lengths and table; pages;
// exponents, K and V; the cluster's exchange); a batch reads each window once, 16 keys a step with the next step's rows on their way
// (32 MB in 32 us, a quarter of the issue slots: what the warps wait for is the first keys and each other).
#include <cooperative_groups.h>

#include "plsh_serve.cuh"
#include "plsh_tile_common.cuh"

namespace plsh {
namespace {

namespace cg = cooperative_groups;
using namespace serve;

constexpr int kThreads = 256, kWarps = 8, kRowsMax = 8, kStep = 32;
constexpr int kCluster = 8;
constexpr int kTail = kRowsMax;  // places above p0 (of which a block's up to 8 tokens use 7)
constexpr int kChunkSteps = 32;  // steps of 32 keys whose pages a block holds at a time
constexpr int kMaxSplitHeads = 64;
constexpr int kMaxGroup = 8;     // query heads of a block (a larger group takes several blocks)

// How a launch's windows are dealt out: 2^lg warps to each (with more KV heads, lg_all), KV heads from the last.
struct Split {
  int tokens, heads, row_blocks, head_blocks;  // of a team; teams of a sequence's rows and of a group's heads
  int per_head;                                // windows of a KV head: sequences x row blocks x head blocks
  int lg_all, window_all;
  int window[kMaxSplitHeads];  // the longest block of a KV head's heads
  uint8_t lg[kMaxSplitHeads];
};
// Clusters of eight blocks (64 warps) for `windows` windows of 2^lg warps.
__host__ __device__ inline int clusters_of(int windows, int lg) { return static_cast<int>(((static_cast<long long>(windows) << lg) + 63) >> 6); }

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
    ml = take(3 * kWarps * rows * 4);              // [3][warp][row]: their m, l and lr
    begin = take(kWarps * heads * PLSH_MAX_S * 4); // [team, at its first warp][head][hash]: where p0's block begins
    keep = take(2 * kWarps * heads * kStep * (int)sizeof(MaskT));  // [stage][warp][head][key]: hashes whose block reaches the key
    row_off = take(kWarps * rows * (int)sizeof(MaskT));  // [team][row]: hashes that open a block in (p0, i]
    tail = take(kWarps * heads * kTail * (int)sizeof(MaskT));  // [team][head][k]: masks of positions p0 + 1 + k
    page = take(kWarps * (2 * kChunkSteps + 4) * 4);   // [team]: pages of the chunk's positions (they hold 16 and more)
    row = take(2 * kWarps * kStep * 8);            // [stage][warp][key]: its row in the pages (-1: none)
    ks = take(2 * kWarps * kStep * 4);             // the same: 2^exponent of K and of V
    vs = take(2 * kWarps * kStep * 4);
    total = at;
  }
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// A 32 x 32 matrix of bits, lane i holding row i, transposed: blocks of 16, 8, .. change places across the diagonal.
__device__ __forceinline__ uint32_t transpose_bits(uint32_t x, int lane) {
  uint32_t m = 0x0000FFFFu;
#pragma unroll
  for (int j = 16; j >= 1; j >>= 1) {
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, j);
    x = lane & j ? (x & ~m) | ((y >> j) & m) : (x & m) | ((y & m) << j);
    m ^= m << (j >> 1);
  }
  return x;
}
// An 8 x 8 matrix of 16-bit values, lane (g, t) holding row g's columns 2 t, 2 t + 1, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
__global__ void __launch_bounds__(kThreads, D == 128 && !kQuant ? 1 : 2)
serve_rows_kernel(ServeArgs a, Split sp) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  if (blockIdx.x == 0) check_seqs(a.sq, a.err);

  // KV heads from the last (with the usual slopes, the widest windows first)
  int x = blockIdx.x / kCluster, kvh, lg = sp.lg_all;  // x: the cluster's number within the KV head
  if (a.H_kv > kMaxSplitHeads) {
    const int per = clusters_of(sp.per_head, lg);
    kvh = a.H_kv - 1 - x / per;
    x %= per;
  } else {
    for (kvh = a.H_kv - 1; kvh > 0; --kvh) {
      const int per = clusters_of(sp.per_head, sp.lg[kvh]);
      if (x < per) break;
      x -= per;
    }
    lg = sp.lg[kvh];
  }
  const int window = a.H_kv > kMaxSplitHeads ? sp.window_all : sp.window[kvh];
  // the team: W warps of each of C blocks; this block's part is warps w0 .. w0 + W - 1
  const int W = min(kWarps, 1 << lg), C = max(1, (1 << lg) / kWarps), in_cl = blockIdx.x % kCluster;
  const int rank = in_cl & (C - 1), rank0 = in_cl - rank;  // blocks rank0 .. rank0 + C - 1 of the cluster
  const int w0 = warp & ~(W - 1), team_tid = tid - 32 * w0, team_threads = 32 * W;
  auto team_sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + w0), "r"(team_threads) : "memory"); };
  x = ((x * kCluster + in_cl) * kWarps + warp) >> lg;      // the window's number within the KV head
  const int tokens = sp.tokens, heads = sp.heads;
  const int hb = x % sp.head_blocks;
  x /= sp.head_blocks;
  const int rb = x % sp.row_blocks, sid = x / sp.row_blocks;
  const int G = a.H / a.H_kv, h0 = kvh * G + hb * heads, nh = min(heads, G - hb * heads);
  Seq sq{};
  if (sid < a.sq.S) sq = load_seq(a.sq, sid);
  const int first = rb * tokens;                              // the block's first token in the sequence
  const int nt = min(tokens, sq.len - first);
  // nothing here (or a longer sequence, the tile kernel's): the cluster's barriers do not wait for warps that have ended, and
  // nobody reads their memory
  if (sid >= a.sq.S || nt <= 0 || sq.len > a.few) return;
  const int rows = nt * nh, p0 = sq.pos0 + first, c0 = sq.c0 + first;
  const MaskT* bmask = static_cast<const MaskT*>(a.bmask);
  const int max_rows = tokens * heads;  // of any block of the launch, alike for the whole cluster
  const Layout<D, MaskT> at_(heads, max_rows);
  float* const s_o = reinterpret_cast<float*>(smem_raw + at_.o);
  float* const s_ml = reinterpret_cast<float*>(smem_raw + at_.ml);
  int* const s_begin = reinterpret_cast<int*>(smem_raw + at_.begin) + w0 * heads * PLSH_MAX_S;
  MaskT* const s_keep = reinterpret_cast<MaskT*>(smem_raw + at_.keep);
  MaskT* const s_row_off = reinterpret_cast<MaskT*>(smem_raw + at_.row_off) + w0 * max_rows;
  MaskT* const s_tail = reinterpret_cast<MaskT*>(smem_raw + at_.tail) + w0 * heads * kTail;
  long long* const s_row = reinterpret_cast<long long*>(smem_raw + at_.row);
  float* const s_ks = reinterpret_cast<float*>(smem_raw + at_.ks);
  float* const s_vs = reinterpret_cast<float*>(smem_raw + at_.vs);
  int* const s_page = reinterpret_cast<int*>(smem_raw + at_.page) + w0 * (2 * kChunkSteps + 4);

  // This block's keys: steps of 32 down from p0, as many as the longest block can reach, dealt out to the window's blocks in runs (step i:
  // keys p0 - 32 i - 31 .. p0 - 32 i). Their first pages are looked up before anything else is known.
  const int steps = (min(window, p0 + 1) + kStep - 1) / kStep;
  const int per = (steps + C - 1) / C;
  const int s0 = rank * per;
  int s1 = min(steps, s0 + per);
  auto find_pages = [&](int b, int ns) {
    const int slot0 = max(0, p0 - kStep * (b + ns) + 1) >> a.pg.lg_page, slots = ((p0 - kStep * b) >> a.pg.lg_page) - slot0 + 1;
    for (int k = team_tid; k < slots; k += team_threads)
      s_page[k] = slot0 + k < a.pg.width ? a.pg.table[static_cast<long long>(sid) * a.pg.width + slot0 + k] : -1;
    return slot0;
  };
  int slot0 = s0 < s1 ? find_pages(s0, min(kChunkSteps, s1 - s0)) : 0;
  // where the blocks of p0 begin, and so the window; masks above p0
  int lo = p0;
  for (int e = team_tid; e < nh * PLSH_MAX_S; e += team_threads)
    if (e % PLSH_MAX_S >= a.s) s_begin[e] = 0x7fffffff;
  for (int e = team_tid; e < nh * a.s; e += team_threads) {
    const int h = e / a.s, k = e % a.s;
    const int b = block_begin(Binning::from_table(a.table + (static_cast<size_t>(h0 + h) * a.s + k) * 2), p0);
    s_begin[h * PLSH_MAX_S + k] = b;
    lo = min(lo, b);
  }
  for (int e = team_tid; e < nh * kTail; e += team_threads) {
    const int h = e / kTail, k = e % kTail;
    s_tail[e] = k + 1 < nt ? bmask[static_cast<size_t>(h0 + h) * a.sq.max_len + p0 + 1 + k] : static_cast<MaskT>(0);
  }
  __shared__ int s_lo[kWarps];
  lo = __reduce_min_sync(0xffffffffu, lo);
  if (lane == 0) s_lo[warp] = lo;

  // Q: lane (g, t) holds row g, in K's order of d
  uint32_t q[D / 16][2];
  float scale_g = 1.4426950408889634f / sqrtf(static_cast<float>(D));  // of row g: S to the exponent of 2
  {
    const bool on = g < rows;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.Q) +
        (on ? static_cast<long long>(c0 + g / nh) * a.qs.token + (h0 + g % nh) * a.qs.head : 0);
    float amax = 0.0f;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
      if (on) {
        w[0] = *reinterpret_cast<const uint4*>(src + 64 * c + 16 * t);
        w[1] = *reinterpret_cast<const uint4*>(src + 64 * c + 16 * t + 8);
      }
      const uint32_t ws[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        q[4 * c + k / 2][k & 1] = ws[k];
        if (kQuant) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(ws[k])), fabsf(bf16_hi(ws[k]))));
      }
    }
    if (kQuant) {  // rows scaled to a largest magnitude in [1, 2): f16 then holds bf16's eight bits down to 2^-17
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int e = min(126, max(-126, static_cast<int>(__float_as_uint(amax) >> 23) - 127));
      scale_g *= pow2(e);
      const float sc = pow2(-e);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        q[k][0] = f16x2(bf16_lo(q[k][0]) * sc, bf16_hi(q[k][0]) * sc);
        q[k][1] = f16x2(bf16_lo(q[k][1]) * sc, bf16_hi(q[k][1]) * sc);
      }
    }
  }
  // of rows 2 t and 2 t + 1, whose columns of S^T the lane has
  const float sc[2] = {__shfl_sync(0xffffffffu, scale_g, 8 * t), __shfl_sync(0xffffffffu, scale_g, 8 * t + 4)};

  team_sync();
  for (int w = 0; w < W; ++w) lo = min(lo, s_lo[w0 + w]);
  s1 = min(s1, (p0 - lo + kStep) / kStep);  // the window's exact end
  if (team_tid < rows) {
    MaskT v = 0;
    for (int k = 0; k < team_tid / nh; ++k) v |= s_tail[team_tid % nh * kTail + k];
    s_row_off[team_tid] = v;
  }

  // O^T: product i has columns (d/8) g + 2 i (0, 1) and (d/8) g + 2 i + 1 (2, 3) of rows 2 t (0, 2) and 2 t + 1 (1, 3)
  float o[D / 16][4];
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, lr[2] = {0.0f, 0.0f};  // of rows 2 t and 2 t + 1; l, and lr of the rounded weights: this lane's keys only
  team_sync();
  MaskT mine[2] = {0, 0};  // the hashes that may count for the two rows, and the rows' heads in the group
  int hh[2] = {0, 0};
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (2 * t + u < rows) {
      mine[u] = static_cast<MaskT>(~s_row_off[2 * t + u]);
      hh[u] = (2 * t + u) % nh;
    }

  // places of this warp's keys in flight
  auto place = [&](int stage) { return (stage * kWarps + warp) * kStep; };
  // K of the 16 keys at places at ..: keys g and g + 8
  constexpr int kKWords = D / 64 * (kQuant ? 4 : 8);
  auto load_k = [&](int at, uint32_t (&kr)[2][kKWords]) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const long long row = s_row[at + 8 * n + g];
#pragma unroll
      for (int i = 0; i < kKWords / 4; ++i) {
        const uint8_t* src = static_cast<const uint8_t*>(a.pg.k) + row * (kQuant ? D : 2 * D) +
                             (kQuant ? 64 * i + 16 * t : 128 * (i >> 1) + 32 * t + 16 * (i & 1));
        const uint4 w = row >= 0 ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
        kr[n][4 * i] = w.x; kr[n][4 * i + 1] = w.y; kr[n][4 * i + 2] = w.z; kr[n][4 * i + 3] = w.w;
      }
    }
  };
  // V's columns (d/8) g .. of keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
  constexpr int kVWords = kQuant ? D / 32 : D / 16;
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
  // The 16 keys at places at ..; byte 2 n + u of c4: the count of key g + 8 n with row 2 t + u.
  auto step = [&](int at, const uint32_t (&kr)[2][kKWords], uint32_t c4) {
    uint32_t vr[4][kVWords];
    load_v(at, vr);  // lands while S is computed
    float acc[2][4] = {};  // two chains of products
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      if constexpr (kQuant)
        mma_f16(acc[k & 1], e4m3_f16x2(kr[0][k]), e4m3_f16x2(kr[1][k]), e4m3_f16x2(kr[0][k] >> 16), e4m3_f16x2(kr[1][k] >> 16), q[k][0], q[k][1]);
      else
        mma_bf16(acc[k & 1], kr[0][2 * k], kr[1][2 * k], kr[0][2 * k + 1], kr[1][2 * k + 1], q[k][0], q[k][1]);
    }
    float x[2][2], top[2] = {-INFINITY, -INFINITY};  // [key][row]
    uint32_t c[2][2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const float ks = kQuant ? s_ks[at + 8 * n + g] : 1.0f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        c[n][u] = (c4 >> (8 * (2 * n + u))) & 0xFFu;
        x[n][u] = (acc[0][2 * n + u] + acc[1][2 * n + u]) * ks * sc[u];
        if (c[n][u]) top[u] = fmaxf(top[u], x[n][u]);
      }
    }
    if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int s = 4; s <= 16; s <<= 1) top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], s));
        const float now = fmaxf(m[u], top[u]);
        const float alpha = now == -INFINITY ? 1.0f : ex2(m[u] - now);  // 0 the first time
        m[u] = now;
        l[u] *= alpha;
        lr[u] *= alpha;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[i][u] *= alpha;
          o[i][2 + u] *= alpha;
        }
      }
    }
    uint32_t b[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      float w[2];
      const float vs = kQuant ? s_vs[at + 8 * n + g] : 1.0f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        w[u] = c[n][u] ? static_cast<float>(c[n][u]) * ex2(x[n][u] - m[u]) : 0.0f;
        l[u] += w[u];
      }
      const uint32_t wr = bf16x2(w[0], w[1]);
      lr[0] += bf16_lo(wr);
      lr[1] += bf16_hi(wr);
      if (kQuant) {
#pragma unroll
        for (int u = 0; u < 2; ++u) w[u] = c[n][u] ? w[u] * vs : 0.0f;
      }
      b[n] = transpose8(bf16x2(w[0], w[1]));  // row g, keys 8 n + 2 t, + 1
    }
    // column (d/8) g + j of keys 2 t, 2 t + 1 (n = 0) and 2 t + 8, 2 t + 9 (n = 1)
    auto pair = [&](int j, int n) {
      if constexpr (kQuant) return e4m3_bf16x2(__byte_perm(vr[2 * n][j >> 2], vr[2 * n + 1][j >> 2], 0x0040u + 0x0011u * (j & 3)));
      else return __byte_perm(vr[2 * n][j >> 1], vr[2 * n + 1][j >> 1], (j & 1) ? 0x7632u : 0x5410u);
    };
#pragma unroll
    for (int i = 0; i < D / 16; ++i) mma_bf16(o[i], pair(2 * i, 0), pair(2 * i + 1, 0), pair(2 * i, 1), pair(2 * i + 1, 1), b[0], b[1]);
  };

  // ---- the keys above p0, one step of the first block's first warp
  if (rank == 0 && warp == w0 && nt > 1) {
    const int at = place(0);
    if (lane < 16) {
      const long long row = lane + 1 < nt ? page_row(a.pg, sid, p0 + 1 + lane, kvh, a.err) : -1;
      s_row[at + lane] = row;
      if (kQuant) {
        s_ks[at + lane] = row >= 0 ? pow2(a.pg.k_exp[row]) : 0.0f;
        s_vs[at + lane] = row >= 0 ? pow2(a.pg.v_exp[row]) : 0.0f;
      }
    }
    __syncwarp();
    uint32_t kr[2][kKWords];
    load_k(at, kr);
    uint32_t c4 = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = 2 * t + u, tok = r / nh;  // the row's token: position p0 + tok
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int k = g + 8 * n;              // key p0 + 1 + k
        if (r < rows && k + 1 <= tok) {
          MaskT v = 0;
          for (int y = k + 1; y < tok; ++y) v |= s_tail[hh[u] * kTail + y];
          c4 |= static_cast<uint32_t>(a.s - popc_mask<MaskT>(v)) << (8 * (2 * n + u));
        }
      }
    }
    step(at, kr, c4);
    __syncwarp();
  }

  // ---- the window
  for (int b = s0; b < s1; b += kChunkSteps) {
    const int ns = min(kChunkSteps, s1 - b);
    if (b > s0) {
      team_sync();
      slot0 = find_pages(b, ns);
      team_sync();
    }
    // Step i of the chunk, a lane per key (lane k: key p0 - 32 (b + i) - k): its row, exponents and the hashes whose blocks
    // reach it, into the stage's places. Returns which keys have weight for some row.
    int8_t ek = 0, ev = 0;
    auto put_exponents = [&](int stage) {
      if (kQuant) {
        s_ks[place(stage) + lane] = pow2(ek);
        s_vs[place(stage) + lane] = pow2(ev);
        __syncwarp();
      }
    };
    auto describe = [&](int i, int stage) -> uint32_t {
      const int at = place(stage), j = p0 - kStep * (b + i) - lane;
      MaskT* const keep = s_keep + (stage * kWarps + warp) * heads * kStep;
      __syncwarp();  // the stage's last reader is done
      long long row = -1;
      if (i < ns && j >= lo) {
        const int page = s_page[(j >> a.pg.lg_page) - slot0];
        if (page < 0 || page >= a.pg.num_pages) atomicOr(a.err, PLSH_DEVERR_PAGE);
        else row = ((static_cast<long long>(page) * a.pg.H_kv + kvh) << a.pg.lg_page) + (j & ((1 << a.pg.lg_page) - 1));
      }
      if (kQuant && row >= 0) {  // stored when they have come, before the step
        ek = a.pg.k_exp[row];
        ev = a.pg.v_exp[row];
      }
      // A lane takes one hash (or two) and finds which of the step's keys its block reaches: all, none, or those from its
      // beginning on; where some block begins within the step, these words of keys are turned round into the keys' words of hashes.
      // (Every hash compared with every key: 108 sequences of one to four tokens, 40/8 heads, 64 hashes, 346 us; so 238 us.)
      const int top = p0 - kStep * (b + i), bottom = top - (kStep - 1);
      auto reached = [&](int first) -> uint32_t {
        const uint32_t whole = __ballot_sync(0xffffffffu, first <= bottom);
        if (!(__ballot_sync(0xffffffffu, first <= top) & ~whole)) return whole;
        return transpose_bits(first <= bottom ? 0xffffffffu : first > top ? 0u : (2u << (top - first)) - 1u, lane);
      };
      MaskT all = 0;
      for (int h = 0; h < nh; ++h) {
        const int* const begin = s_begin + h * PLSH_MAX_S;  // places past the last hash hold the largest position
        MaskT v = reached(begin[lane]);
        if constexpr (sizeof(MaskT) == 8) v |= static_cast<MaskT>(reached(begin[32 + lane])) << 32;
        keep[h * kStep + lane] = v;
        all |= v;
      }
      s_row[at + lane] = row;
      const uint32_t live = __ballot_sync(0xffffffffu, row >= 0 && all != 0);
      __syncwarp();
      return live;
    };
    // the counts of half h's keys g and g + 8 with rows 2 t and 2 t + 1
    auto counts = [&](int stage, int h) -> uint32_t {
      const MaskT* const keep = s_keep + (stage * kWarps + warp) * heads * kStep + 16 * h;
      const long long* const row = s_row + place(stage) + 16 * h;
      uint32_t c4 = 0;
#pragma unroll
      for (int n = 0; n < 2; ++n)
        if (row[g + 8 * n] >= 0) {
#pragma unroll
          for (int u = 0; u < 2; ++u)
            c4 |= static_cast<uint32_t>(popc_mask<MaskT>(static_cast<MaskT>(keep[hh[u] * kStep + g + 8 * n] & mine[u]))) << (8 * (2 * n + u));
        }
      return c4;
    };
    // a warp's steps; the next half's K is on its way while one is computed
    int stage = 0;
    uint32_t live = describe(warp - w0, 0);
    uint32_t ka[2][kKWords], kb[2][kKWords];
    if (live & 0xFFFFu) load_k(place(0), ka);
    put_exponents(0);
    for (int i = warp - w0; i < ns; i += W) {
      if (live >> 16) load_k(place(stage) + 16, kb);
      if (live & 0xFFFFu) step(place(stage), ka, counts(stage, 0));
      const uint32_t next = describe(i + W, stage ^ 1);
      if (next & 0xFFFFu) load_k(place(stage ^ 1), ka);
      if (live >> 16) step(place(stage) + 16, kb, counts(stage, 1));
      put_exponents(stage ^ 1);
      live = next;
      stage ^= 1;
    }
  }

  // ---- join: the warps' rows of every block of the cluster
#pragma unroll
  for (int u = 0; u < 2; ++u) {
#pragma unroll
    for (int s = 4; s <= 16; s <<= 1) {
      l[u] += __shfl_xor_sync(0xffffffffu, l[u], s);
      lr[u] += __shfl_xor_sync(0xffffffffu, lr[u], s);
    }
    const int r = 2 * t + u;
    if (r >= rows) continue;
    if (g == 0) {
      s_ml[warp * max_rows + r] = m[u];
      s_ml[(kWarps + warp) * max_rows + r] = l[u];
      s_ml[(2 * kWarps + warp) * max_rows + r] = lr[u];
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
      *reinterpret_cast<float2*>(s_o + (warp * max_rows + r) * (D + 4) + (D / 8) * g + 2 * i) = make_float2(o[i][u], o[i][2 + u]);
  }
  team_sync();
  auto finish = [&](int r, int col, float top, float total, float norm, const float (&acc)[4]) {
    const float inv = 1.0f / norm;
    const size_t at = static_cast<size_t>(c0 + r / nh) * a.H + h0 + r % nh;
    const float out[4] = {acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv};
    store4f(static_cast<__nv_bfloat16*>(a.O) + at * D + col, out);
    if (col == 0) a.row_sum[at] = (log2f(total) + top) * 0.6931471805599453f - logf(static_cast<float>(a.s));
  };
  // the block's warps, into the first one's place, or straight into the result
  float* const o0 = s_o + w0 * max_rows * (D + 4);
  for (int e = team_tid; e < rows * (D / 4); e += team_threads) {
    const int r = e / (D / 4), col = e % (D / 4) * 4;
    float top = -INFINITY, total = 0.0f, norm = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int w = w0; w < w0 + W; ++w) top = fmaxf(top, s_ml[w * max_rows + r]);
#pragma unroll 4
    for (int w = w0; w < w0 + W; ++w) {
      const float mw = s_ml[w * max_rows + r];
      const float f = mw == -INFINITY ? 0.0f : ex2(mw - top);  // -inf: a warp without keys
      const float4 v = *reinterpret_cast<const float4*>(s_o + (w * max_rows + r) * (D + 4) + col);
      total += s_ml[(kWarps + w) * max_rows + r] * f;
      norm += s_ml[(2 * kWarps + w) * max_rows + r] * f;
      acc[0] += v.x * f;
      acc[1] += v.y * f;
      acc[2] += v.z * f;
      acc[3] += v.w * f;
    }
    if (C == 1) {
      finish(r, col, top, total, norm, acc);
    } else {
      *reinterpret_cast<float4*>(o0 + r * (D + 4) + col) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      if (col == 0) *reinterpret_cast<float4*>(o0 + r * (D + 4) + D) = make_float4(top, total, norm, 0.0f);  // behind the row
    }
  }
  if (C == 1) return;  // (alike for the whole cluster)
  cluster.sync();
  // the window's blocks, each joining its share of the elements
  for (int e = rank + C * tid; e < rows * (D / 4); e += C * kThreads) {
    const int r = e / (D / 4), col = e % (D / 4) * 4;
    float4 ml[kCluster];
    float4 v[kCluster];
    float top = -INFINITY, total = 0.0f, norm = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int b = 0; b < kCluster; ++b) {
      const float* ro = cluster.map_shared_rank(s_o, rank0 + (b & (C - 1))) + r * (D + 4);
      ml[b] = *reinterpret_cast<const float4*>(ro + D);
      v[b] = *reinterpret_cast<const float4*>(ro + col);
      if (b >= C) ml[b].x = -INFINITY;
      top = fmaxf(top, ml[b].x);
    }
#pragma unroll
    for (int b = 0; b < kCluster; ++b) {
      const float f = ml[b].x == -INFINITY ? 0.0f : ex2(ml[b].x - top);
      total += ml[b].y * f;
      norm += ml[b].z * f;
      acc[0] += v[b].x * f;
      acc[1] += v[b].y * f;
      acc[2] += v[b].z * f;
      acc[3] += v[b].w * f;
    }
    finish(r, col, top, total, norm, acc);
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
  if (per_head > 0x7fffffffLL / 64) return fail(PLSH_ERR_RANGE, "plsh_paged_fwd: too many rows");
  sp.per_head = static_cast<int>(per_head);
  // Warps of a window: enough that each has `each` turns of 32 keys of its heads' longest block, the fewest turns with which the
  // launch's blocks are on the machine at once.
  const int room = tiles::sm_count() * (D == 128 && !kQuant ? 1 : 2);
  long long clusters = 0;
  for (int each = 1; each <= 1 << 20; each += each < 8 ? 1 : each / 2) {
    long long blocks = 0;
    clusters = 0;
    sp.lg_all = 0;
    for (int k = 0; k < a.H_kv; ++k) {
      int w = 1, lg = 0;
      for (int h = 0; h < G; ++h) w = a.windows_host[k * G + h] > w ? a.windows_host[k * G + h] : w;
      while (lg < 6 && (static_cast<long long>(kStep) * each << lg) < w) ++lg;
      if (a.H_kv > kMaxSplitHeads) {
        sp.window_all = sp.window_all > w ? sp.window_all : w;
        sp.lg_all = sp.lg_all > lg ? sp.lg_all : lg;
        continue;
      }
      sp.window[k] = w;
      sp.lg[k] = static_cast<uint8_t>(lg);
      blocks += ((per_head << lg) + kWarps - 1) / kWarps;
      clusters += clusters_of(sp.per_head, lg);
    }
    if (a.H_kv > kMaxSplitHeads) {
      blocks = a.H_kv * (((per_head << sp.lg_all) + kWarps - 1) / kWarps);
      clusters = static_cast<long long>(a.H_kv) * clusters_of(sp.per_head, sp.lg_all);
    }
    if (blocks <= room) break;
  }
  if (clusters * kCluster > 0x7fffffffLL) return fail(PLSH_ERR_RANGE, "plsh_paged_fwd: too many rows");
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

// Tokens of one block of rows. Where this kernel shares a call with the tile kernel, it takes the sequences that fit one: room
// for 16 tokens a sequence would leave most of the launch without rows (ten chunks of 1 to 2,048 tokens: 98 us, so 84).
int rows_block_tokens(int group) { return group < kRowsMax ? kRowsMax / group : 1; }

int launch_serve_rows(const ServeArgs& a, cudaStream_t st) {
  if (a.d == 128) return a.s <= 32 ? launch_src<128, uint32_t>(a, st) : launch_src<128, unsigned long long>(a, st);
  return a.s <= 32 ? launch_src<64, uint32_t>(a, st) : launch_src<64, unsigned long long>(a, st);
}

}  // namespace plsh
