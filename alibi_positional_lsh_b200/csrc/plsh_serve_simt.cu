// T~ for packed prompts and against the paged cache, fp32: on the CUDA cores, because its tolerance rules the tensor
// cores out.
//
//   O_i = sum_{j <= i} c_ij e^{S_ij} V_j / sum_{j <= i} c_ij e^{S_ij},  row_sum_i = ln sum_{j <= i} (c_ij / s) e^{S_ij},
// with c_ij = s - popcount(OR of the boundary masks over (j, i]) (blocks are contiguous).
//
// A cluster of one to four blocks takes a tile of 32 positions of one query head, each block a run of the window's
// 64-key tiles, from the diagonal down, with a running maximum and sum; the blocks' rows then meet across their shared
// memory, each block joining a share of the elements, always in the same order. Tiles lie on the grid of absolute
// positions, so that the counts need one word per row (the OR from the key tile's end to the row) and one suffix OR per
// key; those of the row's own key tile are the plan's near counts (scanned here, they were a chain of up to 64 dependent
// steps a block). A warp has 4 rows, each lane 2 keys of S and d/32 columns of O: rows are then
// broadcast, and the lanes' own loads all differ (2 rows x 4 keys a lane, two lanes sharing each key: 51 us in the case below).
//
// What bounds it: operands come from shared memory, 12 passes of it for 32 multiply-adds of a warp, key tiles follow one
// another in a block (four for the widest windows), and some 5 us go before the first and after the last. Three prompts of
// 1,024, 301 and 699 tokens, 4/2 heads, d 64: 48 us (one block a tile of 64 rows 110 us; 64 rows, 4 x 4 a thread: 55 us in
// clusters of four, 100 us in clusters of eight; K and V loaded before their tile's arithmetic: 49 us).
#include <cooperative_groups.h>

#include "plsh_serve.cuh"
#include "plsh_tile_common.cuh"

namespace plsh {
namespace {

namespace cg = cooperative_groups;
using namespace serve;

constexpr int kRows = 32, kKeys = 64, kThreads = 256, kCluster = 4;
constexpr int kR = kRows / (kThreads / 32);  // rows of a warp

template <int D, typename MaskT>
struct SimtSmem {
  float q[kRows][D + 4];
  float k[kKeys][D + 4];  // in the end the block's rows, with m and l behind each
  float v[kKeys][D];
  float p[kRows][kKeys + 4];
  MaskT suf[kKeys];       // OR of the masks after key c, up to the key tile's last
  MaskT own[kRows];       // OR of the masks from the row's own key tile's first key to the row
  MaskT gap[kThreads / 32];
  alignas(16) uint8_t c[kRows][kKeys];
  int sid;
};

template <int D, typename MaskT, bool kPaged, bool kQuant>
__global__ void __launch_bounds__(kThreads) serve_simt_kernel(ServeArgs a, int C) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  auto& sm = *reinterpret_cast<SimtSmem<D, MaskT>*>(smem_raw);
  cg::cluster_group cluster = cg::this_cluster();  // heads from the last: with the usual slopes, the widest windows first
  if (blockIdx.x == 0 && blockIdx.y == 0) check_seqs(a.sq, a.err);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int mult = a.sq.start ? 2 : 1, slot = blockIdx.x / C, rank = blockIdx.x % C;
  if (warp == 0) {
    const int s = warp_find(a.sq.cu, a.sq.S, 5, mult, slot);
    if (lane == 0) sm.sid = s;
  }
  __syncthreads();
  const Seq sq = load_seq(a.sq, sm.sid);
  const int tile = (sq.pos0 / kRows) + slot - ((a.sq.cu[sm.sid] / kRows) + mult * sm.sid);
  const int end = sq.pos0 + sq.len;
  const int i0 = tile * kRows;
  if (tile < 0 || sq.len == 0 || i0 >= end) return;  // the whole cluster
  const int h = a.H - 1 - blockIdx.y, kvh = h / (a.H / a.pg.H_kv);
  const MaskT* bm = static_cast<const MaskT*>(a.bmask) + static_cast<size_t>(h) * a.sq.max_len;
  const float sc = 1.4426950408889634f / sqrtf(static_cast<float>(D));

  const int T128 = (a.sq.max_len + PLSH_TILE - 1) / PLSH_TILE;
  int lo = a.spans[(static_cast<size_t>(h) * T128 + (i0 >> 7)) * 2];
  if (lo < 0 || lo > i0) {
    if (tid == 0) atomicOr(a.err, PLSH_DEVERR_WINDOW);
    lo = i0;
  }
  // key tiles diag, diag - 1, ..; this block's run of them
  const int diag = i0 >> 6, tiles = diag - (lo >> 6) + 1;
  const int per = (tiles + C - 1) / C, t0 = min(tiles, rank * per), t1 = min(tiles, t0 + per);
  // the row of the packed token at a position, or -1 where the position holds none of the new tokens
  auto token = [&](int p) { return (p >= sq.pos0 && p < end) ? sq.c0 + p - sq.pos0 : -1; };
  for (int e = tid; e < kRows * (D / 4); e += kThreads) {
    const int r = e / (D / 4), c = e % (D / 4) * 4;
    const int t = token(i0 + r);
    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (t >= 0) load4f(static_cast<const float*>(a.Q) + t * a.qs.token + h * a.qs.head + c, x);
    store4f(&sm.q[r][c], x);
  }

  // the OR of the tiles between the diagonal one and the run
  MaskT gap = 0;
  for (int j = kKeys * (diag - t0 + 1) + tid; j < kKeys * diag; j += kThreads) gap |= bm[j];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) gap |= __shfl_xor_sync(0xffffffffu, gap, o);
  if (lane == 0) sm.gap[warp] = gap;
  if (warp == 0) {  // ORs from the diagonal tile's first key to each row
    const MaskT b0 = kKeys * diag + lane < end ? bm[kKeys * diag + lane] : static_cast<MaskT>(0);
    const MaskT b1 = kKeys * diag + 32 + lane < end ? bm[kKeys * diag + 32 + lane] : static_cast<MaskT>(0);
    const MaskT u = tiles::warp_prefix_or<MaskT>(b0, lane), v = tiles::warp_prefix_or<MaskT>(b1, lane);
    const MaskT w = static_cast<MaskT>(__shfl_sync(0xffffffffu, u, 31) | v);
    sm.own[lane] = i0 & 32 ? w : u;
  }
  if (t0 == 0)  // the counts in the diagonal tile are the plan's
    for (int e = tid; e < kRows * (kKeys / 16); e += kThreads) {
      const int r = e / (kKeys / 16), p = i0 + r;
      reinterpret_cast<uint4*>(sm.c[r])[e % (kKeys / 16)] =
          p < end ? __ldg(reinterpret_cast<const uint4*>(a.near + (static_cast<size_t>(h) * a.sq.max_len + p) * kKeys) + e % (kKeys / 16))
                  : make_uint4(0, 0, 0, 0);
    }
  __syncthreads();
  gap = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) gap |= sm.gap[w];
  constexpr int kCols = D / 32;  // columns of O of a lane, kCols * lane ..
  float m[kR], l[kR], acc[kR][kCols];
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.0f;
#pragma unroll
    for (int e = 0; e < kCols; ++e) acc[r][e] = 0.0f;
  }

  // K or V of a key tile into shared memory, rows past the end or without a page as zeros. fp32 rows are copied behind the arithmetic: V
  // under S, the next tile's K under P V; e4m3 rows go through registers. Returns the last of this thread's rows without a page.
  auto load_tile = [&](bool value, int j0) {
    int missing = -1;
#pragma unroll (D == 64 ? 4 : 2)
    for (int e = tid; e < kKeys * (D / 4); e += kThreads) {
      const int r = e / (D / 4), c = e % (D / 4) * 4, p = j0 + r;
      float* const dst = value ? &sm.v[r][c] : &sm.k[r][c];
      long long row = -1;
      if (p < end) row = kPaged ? find_row(a.pg, sq.s, p, kvh) : sq.c0 + p;
      if (kPaged && p < end && row < 0) missing = r;
      if constexpr (kQuant) {
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (row >= 0) {
          e4m3_to_float4(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(value ? a.pg.v : a.pg.k) + row * D + c), x);
          const float s = pow2((value ? a.pg.v_exp : a.pg.k_exp)[row]);
#pragma unroll
          for (int u = 0; u < 4; ++u) x[u] *= s;
        }
        store4f(dst, x);
      } else {
        const float* src = static_cast<const float*>(a.Q);  // any address: nothing is read where there is no row
        if (row >= 0) {
          if constexpr (kPaged) src = static_cast<const float*>(value ? a.pg.v : a.pg.k) + row * D + c;
          else src = static_cast<const float*>(value ? a.V : a.K) + row * (value ? a.vs.token : a.ks.token) + kvh * (value ? a.vs.head : a.ks.head) + c;
        }
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))), "l"(src), "r"(row >= 0 ? 16 : 0)
                     : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return missing;
  };
  // A tile's first key that the call's first row reaches (kKeys: none): in pages, what lies before it is no longer the sequence's own
  // and may be anything, not finite or not there.
  const int r0 = max(0, sq.pos0 - i0);
  auto lowest = [](uint32_t even, uint32_t odd) {  // of keys 2 i and 2 i + 1
    return min(even ? 2 * (__ffs(even) - 1) : kKeys, odd ? 2 * (__ffs(odd) - 1) + 1 : kKeys);
  };
  if (t0 < t1) load_tile(false, kKeys * (diag - t0));
  for (int t = t0; t < t1; ++t) {
    const int j0 = kKeys * (diag - t);
    __syncthreads();  // V of the tile before has been read
    const int missing = load_tile(true, j0);
    int reach = 0;
    if (kPaged && t == 0) {
      auto reached = [&](int key) { return __ballot_sync(0xffffffffu, j0 + key >= i0 + r0 || sm.c[r0][key] > 0); };
      const uint32_t even = reached(2 * lane), odd = reached(2 * lane + 1);
      reach = lowest(even, odd);
    }
    MaskT all = 0;  // every mask of the tile (a later tile's gap)
    if (t > 0) {    // suffix ORs over the tile's keys, two a lane; every warp for itself, the first one for all
      const MaskT b0 = bm[j0 + 2 * lane], b1 = bm[j0 + 2 * lane + 1];
      const MaskT inc = tiles::warp_suffix_or<MaskT>(static_cast<MaskT>(b0 | b1), lane);
      MaskT after = __shfl_down_sync(0xffffffffu, inc, 1);
      if (lane == 31) after = 0;
      all = __shfl_sync(0xffffffffu, inc, 0);
      if (kPaged) {
        auto reached = [&](MaskT between) { return __ballot_sync(0xffffffffu, popc_mask<MaskT>(static_cast<MaskT>(sm.own[r0] | between | gap)) < a.s); };
        const uint32_t even = reached(static_cast<MaskT>(after | b1)), odd = reached(after);
        reach = lowest(even, odd);
      }
      if (warp == 0) {
        sm.suf[2 * lane] = static_cast<MaskT>(after | b1 | gap);
        sm.suf[2 * lane + 1] = static_cast<MaskT>(after | gap);
      }
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");  // K
    __syncthreads();

    float x[kR][2];
#pragma unroll
    for (int r = 0; r < kR; ++r) x[r][0] = x[r][1] = 0.0f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      float4 qa[kR], ka[2];
#pragma unroll
      for (int r = 0; r < kR; ++r) qa[r] = *reinterpret_cast<const float4*>(&sm.q[kR * warp + r][c]);
#pragma unroll
      for (int e = 0; e < 2; ++e) ka[e] = *reinterpret_cast<const float4*>(&sm.k[lane + 32 * e][c]);
#pragma unroll
      for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          x[r][e] = fmaf(qa[r].x, ka[e].x, fmaf(qa[r].y, ka[e].y, fmaf(qa[r].z, ka[e].z, fmaf(qa[r].w, ka[e].w, x[r][e]))));
    }
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int row = kR * warp + r;
      int cn[2];
      float top = m[r];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = lane + 32 * e;
        cn[e] = t == 0 ? sm.c[row][key] : a.s - popc_mask<MaskT>(static_cast<MaskT>(sm.own[row] | sm.suf[key]));
        x[r][e] *= sc;
        if (cn[e] > 0) top = fmaxf(top, x[r][e]);
      }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float alpha = top == -INFINITY ? 1.0f : exp2f(m[r] - top);
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float p = cn[e] > 0 ? static_cast<float>(cn[e]) * exp2f(x[r][e] - top) : 0.0f;
        sum += p;
        sm.p[row][lane + 32 * e] = p;
      }
      l[r] = l[r] * alpha + sum;
      m[r] = top;
#pragma unroll
      for (int e = 0; e < kCols; ++e) acc[r][e] *= alpha;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (kPaged) {
      if (missing >= reach) atomicOr(a.err, PLSH_DEVERR_PAGE);
      // V there meets weights of zero, which a NaN would not leave: the thread that copied it clears it (K's scores are not taken)
      for (int e = tid; e < reach * (D / 4); e += kThreads) *reinterpret_cast<float4*>(&sm.v[e / (D / 4)][e % (D / 4) * 4]) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    __syncthreads();  // V is there, K has been read (a warp's rows of P are its own)
    if (t + 1 < t1) load_tile(false, j0 - kKeys);
    gap = static_cast<MaskT>(gap | all);
#pragma unroll 4
    for (int k = 0; k < kKeys; k += 4) {
      float4 pr[kR];
#pragma unroll
      for (int r = 0; r < kR; ++r) pr[r] = *reinterpret_cast<const float4*>(&sm.p[kR * warp + r][k]);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        float vv[kCols];
        if constexpr (kCols == 4) {
          load4f(&sm.v[k + kk][4 * lane], vv);
        } else {
          const float2 v2 = *reinterpret_cast<const float2*>(&sm.v[k + kk][2 * lane]);
          vv[0] = v2.x; vv[1] = v2.y;
        }
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          const float p = kk == 0 ? pr[r].x : kk == 1 ? pr[r].y : kk == 2 ? pr[r].z : pr[r].w;
#pragma unroll
          for (int e = 0; e < kCols; ++e) acc[r][e] = fmaf(p, vv[e], acc[r][e]);
        }
      }
    }
  }

  auto finish = [&](int t, int col, float top, float total, const float (&o)[4]) {
    const float inv = 1.0f / total;
    const float out[4] = {o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv};
    store4f(static_cast<float*>(a.O) + (static_cast<size_t>(t) * a.H + h) * D + col, out);
    if (col == 0)
      a.row_sum[static_cast<size_t>(t) * a.H + h] = (log2f(total) + top) * 0.6931471805599453f - logf(static_cast<float>(a.s));
  };
  __syncthreads();  // K has been read
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    float total = l[r];
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const int row = kR * warp + r;
    if constexpr (kCols == 4) store4f(&sm.k[row][4 * lane], acc[r]);
    else *reinterpret_cast<float2*>(&sm.k[row][2 * lane]) = make_float2(acc[r][0], acc[r][1]);
    if (lane == 0) {
      sm.k[row][D] = m[r];
      sm.k[row][D + 1] = total;
    }
  }
  cluster.sync();
  for (int e = rank + C * tid; e < kRows * (D / 4); e += C * kThreads) {
    const int row = e / (D / 4), col = e % (D / 4) * 4, t = token(i0 + row);
    if (t < 0) continue;
    float top = -INFINITY, total = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int b = 0; b < C; ++b) top = fmaxf(top, cluster.map_shared_rank(&sm.k[row][0], b)[D]);
    for (int b = 0; b < C; ++b) {
      const float* ro = cluster.map_shared_rank(&sm.k[row][0], b);
      const float f = ro[D] == -INFINITY ? 0.0f : exp2f(ro[D] - top);  // -inf: no keys with weight
      const float4 v = *reinterpret_cast<const float4*>(ro + col);
      total += ro[D + 1] * f;
      o[0] += v.x * f;
      o[1] += v.y * f;
      o[2] += v.z * f;
      o[3] += v.w * f;
    }
    finish(t, col, top, total, o);
  }
  cluster.sync();  // the others have read this block's rows
}

template <int D, typename MaskT, bool kPaged, bool kQuant>
int launch(const ServeArgs& a, cudaStream_t st) {
  auto kern = serve_simt_kernel<D, MaskT, kPaged, kQuant>;
  const int smem = static_cast<int>(sizeof(SimtSmem<D, MaskT>));
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(serve_simt_kernel)");
  const long long slots = a.sq.T / kRows + static_cast<long long>(a.sq.start ? 2 : 1) * a.sq.S;
  // Blocks of a row tile: up to four while the launch has fewer than four an SM, and no more than the longest window can have key
  // tiles. With one, two and four: 82, 55 and 49 us in the case above, 94, 69 and 80 us for two prompts of 1,000 tokens with 8/8 heads,
  // 342, 400 and 543 us for four of 2,000 with 16/8.
  int C = 1;
  while (C < kCluster && slots * a.H * C < 4 * tiles::sm_count() && C * kKeys < a.sq.max_len) C *= 2;
  if (slots * C > 0x7fffffffLL) return fail(PLSH_ERR_RANGE, "too many row tiles");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(slots * C), a.H);
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
  e = cudaLaunchKernelEx(&cfg, kern, a, C);
  return e == cudaSuccess ? PLSH_OK : cuda_fail(e, "serve_simt_kernel launch");
}

template <int D, typename MaskT>
int launch_src(const ServeArgs& a, cudaStream_t st) {
  if (!a.paged) return launch<D, MaskT, false, false>(a, st);
  return a.pg.k_exp ? launch<D, MaskT, true, true>(a, st) : launch<D, MaskT, true, false>(a, st);
}

}  // namespace

int launch_serve_simt(const ServeArgs& a, cudaStream_t st) {
  if (a.d == 128) return a.s <= 32 ? launch_src<128, uint32_t>(a, st) : launch_src<128, unsigned long long>(a, st);
  return a.s <= 32 ? launch_src<64, uint32_t>(a, st) : launch_src<64, unsigned long long>(a, st);
}

}  // namespace plsh
