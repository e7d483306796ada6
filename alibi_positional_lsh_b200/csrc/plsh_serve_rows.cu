// T~ of a few new tokens of each sequence (one when decoding) against the paged cache, bf16.
//
// Rows are the (token, query head) pairs that share a KV head, up to 16 in a block; their keys are the
// window below them, so the work is reading K and V once: 2 (d + 1) bytes a key and KV head when the pages
// hold e4m3. A cluster of blocks shares one window, four warps a block, each taking steps of 16 keys:
//   S[16 rows][16 keys] = Q K^T   8 d/16 x 2 products mma.m16n8k16 per step, fp32 accumulation
//   P = c 2^(S sc - m), against the warp's own running maximum m over keys with c > 0
//   O[16 rows][d] += P V
// and the partial rows (m, l, O) meet in shared memory at the end, each block of the cluster joining its share
// of the rows from all blocks' (distributed shared memory): one launch, no scratch, and always in the
// same order, so results do not depend on timing.
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
constexpr int kChunk = 256;      // keys whose rows, exponents and counts a block holds at a time
constexpr int kMaxGroup = 16;    // query heads of a block (a larger group takes several blocks)

// Shared memory of a block for `heads` query heads and `rows` rows.
template <int D, typename MaskT>
struct Layout {
  int o, ml, begin, keep, row_off, tail, row, ks, vs, total;
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
    keep = take(heads * kChunk * (int)sizeof(MaskT));   // [head][key]: hashes whose block reaches the key
    row_off = take(rows * (int)sizeof(MaskT));     // [row]: hashes that open a block in (p0, i]
    tail = take(heads * kStep * (int)sizeof(MaskT));    // [head][k]: masks of positions p0 + 1 + k
    row = take((kChunk + kStep) * 8);              // [key]: its row in the pages (-1: none)
    ks = take((kChunk + kStep) * 4);               // [key]: 2^exponent of K and of V
    vs = take((kChunk + kStep) * 4);
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
serve_rows_kernel(ServeArgs a, int tokens, int heads, int row_blocks, int head_blocks) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  if (blockIdx.x == 0) check_seqs(a.sq, a.err);

  // KV heads from the last (with the usual slopes, the widest windows first), then sequences, then row blocks
  int x = blockIdx.x / C;
  const int hb = x % head_blocks;
  x /= head_blocks;
  const int rb = x % row_blocks;
  x /= row_blocks;
  const int sid = x % a.sq.S, kvh = a.H_kv - 1 - x / a.sq.S;
  const int G = a.H / a.H_kv, h0 = kvh * G + hb * heads, nh = min(heads, G - hb * heads);
  const Seq sq = load_seq(a.sq, sid);
  const int first = rb * tokens;                              // the block's first token in the sequence
  const int nt = min(tokens, sq.len - first);
  // (longer sequences are the tile kernel's)
  if (nt <= 0 || sq.len > a.few) return;                      // the whole cluster returns
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

  // where the blocks of p0 begin, and so the window; masks above p0
  int lo = p0;
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

  // rows, exponents of keys j(k), k = 0 .. n - 1, into places at ..
  auto describe = [&](int at, int k, int j, bool on) {
    long long row = -1;
    if (on) row = page_row(a.pg, sid, j, kvh, a.err);
    s_row[at + k] = row;
    if (kQuant) {
      s_ks[at + k] = row >= 0 ? pow2(a.pg.k_exp[row]) : 0.0f;
      s_vs[at + k] = row >= 0 ? pow2(a.pg.v_exp[row]) : 0.0f;
    }
  };

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

  // ---- the keys above p0, one step of block 0's first warp
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = g + 8 * u;
    if (r < rows) {
      mine[u] = static_cast<MaskT>(~s_row_off[r]);
      hh[u] = r % nh;
    }
  }
  if (rank == 0 && warp == 0 && nt > 1) {
    if (lane < kStep) describe(kChunk, lane, p0 + 1 + lane, lane + 1 < nt);
    __syncwarp();
    uint4 kr[2][D / 64][kQuant ? 1 : 2];
    uint32_t vr[4][kVWords];
    load_k(kChunk, kr);
    load_v(kChunk, vr);
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
    step(kChunk, kr, vr, c);
  }

  // ---- the window, kChunk keys at a time
  for (int b = s0; b < s1; b += kChunk / kStep) {
    const int ns = min(kChunk / kStep, s1 - b);
    __syncthreads();
    // key at place k of the chunk: p0 - 16 b - k, steps downward; within a step of 16 places ascending order does not matter
    for (int k = tid; k < ns * kStep; k += kThreads) {
      const int j = p0 - kStep * b - k;
      describe(0, k, j, j >= lo);
    }
    // the hashes whose block reaches the key, per head
    for (int k = tid; k < ns * kStep; k += kThreads) {
      const int j = p0 - kStep * b - k;
      for (int h = 0; h < nh; ++h) {
        MaskT v = 0;
        const int* begin = s_begin + h * PLSH_MAX_S;
#pragma unroll 4
        for (int i = 0; i < a.s; ++i) v |= static_cast<MaskT>(begin[i] <= j) << i;
        s_keep[h * kChunk + k] = v;
      }
    }
    __syncthreads();
    // a warp's steps, the next one's rows on their way while this one is computed
    auto counts = [&](int i, uint32_t (&c)[2]) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        c[u] = 0;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int k = kStep * i + 2 * t + (n & 1) + 8 * (n >> 1);
          if (s_row[k] >= 0) c[u] |= static_cast<uint32_t>(popc_mask<MaskT>(static_cast<MaskT>(s_keep[hh[u] * kChunk + k] & mine[u]))) << (8 * n);
        }
      }
      return __any_sync(0xffffffffu, (c[0] | c[1]) != 0) != 0;  // else nothing has weight there
    };
    uint4 kr[2][D / 64][kQuant ? 1 : 2];
    uint32_t c[2];
    int i = warp;
    while (i < ns && !counts(i, c)) i += kWarps;
    if (i < ns) load_k(kStep * i, kr);
    while (i < ns) {
      uint32_t vr[4][kVWords];
      load_v(kStep * i, vr);
      int nx = i + kWarps;
      uint32_t cn[2];
      while (nx < ns && !counts(nx, cn)) nx += kWarps;
      uint4 kn[2][D / 64][kQuant ? 1 : 2];
      if (kQuant && nx < ns) load_k(kStep * nx, kn);
      step(kStep * i, kr, vr, c);
      if (!kQuant && nx < ns) load_k(kStep * nx, kn);  // (rows of bf16 take twice the registers)
      i = nx;
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
  cluster.sync();
  for (int e = rank * kThreads + tid; e < rows * (D / 4); e += C * kThreads) {
    const int r = e / (D / 4), col = e % (D / 4) * 4;
    float top = -INFINITY;
    for (int b = 0; b < C; ++b) {
      const float* ml = cluster.map_shared_rank(s_ml, b);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * max_rows + r]);
    }
    float total = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int b = 0; b < C; ++b) {
      const float* ml = cluster.map_shared_rank(s_ml, b);
      const float* ro = cluster.map_shared_rank(s_o, b);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(ml[w * max_rows + r] - top);  // 0 for a warp without keys
        if (f > 0.0f) {
          total += ml[(kWarps + w) * max_rows + r] * f;
          const float4 v = *reinterpret_cast<const float4*>(ro + (w * max_rows + r) * (D + 4) + col);
          acc[0] += v.x * f;
          acc[1] += v.y * f;
          acc[2] += v.z * f;
          acc[3] += v.w * f;
        }
      }
    }
    const float inv = 1.0f / total;
    const size_t at = static_cast<size_t>(c0 + r / nh) * a.H + h0 + r % nh;
    const float out[4] = {acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv};
    store4f(static_cast<__nv_bfloat16*>(a.O) + at * D + col, out);
    if (col == 0) a.row_sum[at] = (log2f(total) + top) * 0.6931471805599453f - logf(static_cast<float>(a.s));
  }
  cluster.sync();  // the others have read this block's rows
}

template <int D, typename MaskT, bool kQuant>
int launch(const ServeArgs& a, cudaStream_t st) {
  const int G = a.H / a.H_kv;
  const int heads = G < kMaxGroup ? G : kMaxGroup, head_blocks = ceil_div(G, heads);
  const int most = a.sq.max_new < a.few ? a.sq.max_new : a.few;
  const int tokens = most < kRowsMax / heads ? most : kRowsMax / heads;
  const int row_blocks = ceil_div(most, tokens);
  const long long items = static_cast<long long>(a.sq.S) * a.H_kv * head_blocks * row_blocks;
  // blocks of a window: up to the portable eight, as long as the machine has room for more, and no more than two steps a warp
  int C = 1;
  while (C < 8 && items * C < 4 * 148 && 2 * C * kWarps * kStep < a.max_window) C *= 2;
  if (items * C > 0x7fffffffLL) return fail(PLSH_ERR_RANGE, "plsh_paged_fwd: too many rows");
  auto kern = serve_rows_kernel<D, MaskT, kQuant>;
  const int smem = Layout<D, MaskT>(heads, tokens * heads).total;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(serve_rows_kernel)");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(items * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = C;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, a, tokens, heads, row_blocks, head_blocks);
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
