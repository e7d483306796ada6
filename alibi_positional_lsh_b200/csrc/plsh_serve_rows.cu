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
// Counts: c_ij = s - popcount(OR of the masks over (j, i]). With p0 the block's first token, the OR splits into
// (j, p0], which the block holds per key and head of the group, and (p0, i], one word per row. The up to 15 keys
// above p0 are a last step, counted from the masks directly.
#include <cooperative_groups.h>

#include "plsh_serve.cuh"

namespace plsh {
namespace {

namespace cg = cooperative_groups;
using namespace serve;

constexpr int kThreads = 128, kWarps = 4, kRowsMax = 16, kStep = 16;
constexpr int kChunk = 256;      // keys whose rows, exponents and counts a block holds at a time
constexpr int kMaxGroup = 16;    // query heads of a block (a larger group takes several blocks)

template <int D, typename MaskT>
struct RowsSmem {
  float o[kWarps][kRowsMax][D + 4];
  float m[kWarps][kRowsMax], l[kWarps][kRowsMax];
  MaskT suf[kMaxGroup][kChunk];   // OR of the masks over (j, p0], per head and key
  MaskT carry[kMaxGroup];         // of the keys above the chunk
  MaskT row_or[kRowsMax];         // OR of the masks over (p0, i]
  MaskT tail[kMaxGroup][kStep];   // masks of positions p0 + 1 ..
  long long row[kChunk + kStep];  // the keys' rows in the pages (-1: none)
  float ks[kChunk + kStep], vs[kChunk + kStep];
};

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
__global__ void __launch_bounds__(kThreads) serve_rows_kernel(ServeArgs a, int tokens, int heads, int row_blocks, int head_blocks) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  auto& sm = *reinterpret_cast<RowsSmem<D, MaskT>*>(smem_raw);
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

  // the window: the lowest key with weight for one of the block's rows is in no lower a place than its row tile's
  const int T128 = (a.sq.max_len + PLSH_TILE - 1) / PLSH_TILE;
  int lo = p0;
  for (int h = lane; h < nh; h += 32) lo = min(lo, a.spans[(static_cast<size_t>(h0 + h) * T128 + (p0 >> 7)) * 2]);
  lo = max(0, __reduce_min_sync(0xffffffffu, lo));
  // this block's keys: steps of 16 down from p0, dealt out to the cluster in runs
  const int steps = (p0 - lo + kStep) / kStep;
  const int per = (steps + C - 1) / C;
  const int s0 = rank * per, s1 = min(steps, s0 + per);       // step i: keys p0 - 16 i - 15 .. p0 - 16 i

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

  // masks above p0, and per row the OR over (p0, i]
  for (int e = tid; e < nh * kStep; e += kThreads) {
    const int h = e / kStep, k = e % kStep;
    sm.tail[h][k] = k + 1 < nt ? bmask[static_cast<size_t>(h0 + h) * a.sq.max_len + p0 + 1 + k] : static_cast<MaskT>(0);
  }
  // the OR over the keys between p0 and this block's first step, per head: a warp takes heads in turn
  for (int h = warp; h < nh; h += kWarps) {
    const MaskT* bm = bmask + static_cast<size_t>(h0 + h) * a.sq.max_len;
    MaskT v = 0;
    for (int j = p0 - lane; j > p0 - kStep * s0; j -= 32) v |= bm[j];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v |= __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0) sm.carry[h] = v;
  }
  __syncthreads();
  if (tid < kRowsMax) {
    MaskT v = 0;
    if (tid < rows)
      for (int k = 0; k < tid / nh; ++k) v |= sm.tail[tid % nh][k];
    sm.row_or[tid] = v;
  }

  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  MaskT mine[2] = {0, 0};
  int hh[2] = {0, 0};

  // rows, exponents of keys j(k), k = 0 .. n - 1, into places at ..
  auto describe = [&](int at, int k, int j, bool on) {
    long long row = -1;
    if (on) row = page_row(a.pg, sid, j, kvh, a.err);
    sm.row[at + k] = row;
    if (kQuant) {
      sm.ks[at + k] = row >= 0 ? pow2(a.pg.k_exp[row]) : 0.0f;
      sm.vs[at + k] = row >= 0 ? pow2(a.pg.v_exp[row]) : 0.0f;
    }
  };

  // one step: 16 keys at places at .. of sm.row; c[u][n] their counts for rows g and g + 8, keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
  auto load_k = [&](int at, uint4 (&kr)[2][D / 64][kQuant ? 1 : 2]) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const long long row = sm.row[at + 8 * n + g];
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
      const long long row = sm.row[at + 2 * t + (n & 1) + 8 * (n >> 1)];
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
  auto step = [&](int at, const uint4 (&kr)[2][D / 64][kQuant ? 1 : 2], const uint32_t (&vr)[4][kVWords], const int (&c)[2][4]) {
    float x[2][4];
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
        const float ks = kQuant ? sm.ks[at + 8 * n + 2 * t + e] : 1.0f;
        x[0][2 * n + e] = acc[e] * ks * sc[0];
        x[1][2 * n + e] = acc[2 + e] * ks * sc[1];
      }
    }
    uint32_t p[4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float top = m[u];
#pragma unroll
      for (int n = 0; n < 4; ++n) top = c[u][n] > 0 ? fmaxf(top, x[u][n]) : top;
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
        w[n] = c[u][n] > 0 ? static_cast<float>(c[u][n]) * exp2f(x[u][n] - m[u]) : 0.0f;
        l[u] += w[n];
        if (kQuant) w[n] *= c[u][n] > 0 ? sm.vs[at + 2 * t + (n & 1) + 8 * (n >> 1)] : 0.0f;
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
    mine[u] = sm.row_or[r];
    hh[u] = r < rows ? r % nh : 0;
  }
  if (rank == 0 && warp == 0 && nt > 1) {
    if (lane < kStep) describe(kChunk, lane, p0 + 1 + lane, lane + 1 < nt);
    __syncwarp();
    uint4 kr[2][D / 64][kQuant ? 1 : 2];
    uint32_t vr[4][kVWords];
    load_k(kChunk, kr);
    load_v(kChunk, vr);
    int c[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = g + 8 * u, tok = r / nh;  // the row's token: position p0 + tok
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int k = 2 * t + (n & 1) + 8 * (n >> 1);  // key p0 + 1 + k
        c[u][n] = 0;
        if (r < rows && k + 1 <= tok) {
          MaskT v = 0;
          for (int y = k + 1; y < tok; ++y) v |= sm.tail[hh[u]][y];
          c[u][n] = a.s - popc_mask<MaskT>(v);
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
    // OR over (j, p0]: an inclusive scan over the masks of j + 1 .. downward, per head
    for (int h = warp; h < nh; h += kWarps) {
      const MaskT* bm = bmask + static_cast<size_t>(h0 + h) * a.sq.max_len;
      MaskT run = sm.carry[h];
      for (int k0 = 0; k0 < ns * kStep; k0 += 32) {
        const int k = k0 + lane, j = p0 - kStep * b - k;
        MaskT v = j >= lo ? bm[j] : static_cast<MaskT>(0);   // of key j: joins the OR below j
        MaskT inc = v;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
          const MaskT y = __shfl_up_sync(0xffffffffu, inc, s);
          if (lane >= s) inc |= y;
        }
        MaskT exc = __shfl_up_sync(0xffffffffu, inc, 1);
        if (lane == 0) exc = 0;
        if (k < ns * kStep) sm.suf[h][k] = static_cast<MaskT>(run | exc);
        run |= __shfl_sync(0xffffffffu, inc, 31);
      }
      __syncwarp();
      if (lane == 0) sm.carry[h] = run;
    }
    __syncthreads();
    for (int i = warp; i < ns; i += kWarps) {
      const int at = kStep * i;
      uint4 kr[2][D / 64][kQuant ? 1 : 2];
      uint32_t vr[4][kVWords];
      int c[2][4];
      bool any = false;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int k = at + 2 * t + (n & 1) + 8 * (n >> 1);
          c[u][n] = g + 8 * u < rows && sm.row[k] >= 0 ? a.s - popc_mask<MaskT>(static_cast<MaskT>(sm.suf[hh[u]][k] | mine[u])) : 0;
          any |= c[u][n] > 0;
        }
      if (!__any_sync(0xffffffffu, any)) continue;  // nothing has weight here
      load_k(at, kr);
      load_v(at, vr);
      step(at, kr, vr, c);
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
      sm.m[warp][r] = m[u];
      sm.l[warp][r] = l[u];
    }
    // product i's columns n = 2 t, 2 t + 1: V's columns (D/8) (2 t) + i and (D/8) (2 t + 1) + i
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      sm.o[warp][r][(D / 8) * (2 * t) + i] = o[i][2 * u];
      sm.o[warp][r][(D / 8) * (2 * t + 1) + i] = o[i][2 * u + 1];
    }
  }
  cluster.sync();
  for (int e = rank * kThreads + tid; e < rows * (D / 4); e += C * kThreads) {
    const int r = e / (D / 4), col = e % (D / 4) * 4;
    float top = -INFINITY;
    for (int b = 0; b < C; ++b) {
      const float* pm = &cluster.map_shared_rank(&sm, b)->m[0][0];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, pm[w * kRowsMax + r]);
    }
    float total = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int b = 0; b < C; ++b) {
      const auto* rs = cluster.map_shared_rank(&sm, b);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(rs->m[w][r] - top);  // 0 for a warp without keys
        if (f > 0.0f) {
          total += rs->l[w][r] * f;
          const float4 v = *reinterpret_cast<const float4*>(&rs->o[w][r][col]);
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
  const int tokens = kRowsMax / heads;
  const int most = a.sq.max_new < a.few ? a.sq.max_new : a.few;
  const int row_blocks = ceil_div(most, tokens);
  const long long items = static_cast<long long>(a.sq.S) * a.H_kv * head_blocks * row_blocks;
  // blocks of a window: as many as fill the machine about twice over, up to the portable eight
  int C = 1;
  while (C < 8 && items * C < 2 * 148) C *= 2;
  if (C < 4) C = 4;
  if (items * C > 0x7fffffffLL) return fail(PLSH_ERR_RANGE, "plsh_paged_fwd: too many rows");
  auto kern = serve_rows_kernel<D, MaskT, kQuant>;
  const int smem = static_cast<int>(sizeof(RowsSmem<D, MaskT>));
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
