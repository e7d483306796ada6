// T~ for packed prompts and for chunks against the paged cache, in fp32 on the CUDA cores: the kernel
// for fp32 inputs (whose tolerance rules the tensor cores out).
//
//   O_i = sum_{j <= i} c_ij e^{S_ij} V_j / sum_{j <= i} c_ij e^{S_ij},  row_sum_i = ln sum_{j <= i} (c_ij / s) e^{S_ij},
// with c_ij = s - popcount(OR of the boundary masks over (j, i]) (blocks are contiguous).
//
// One block per (tile of 64 positions, query head): 64 rows against 64 keys at a time, from the
// diagonal down to the window's end, with a running maximum and sum. Tiles lie on the grid of
// absolute positions, so that the counts need one carry per row (the OR from the tile's end to the
// row) and one suffix OR per key; the diagonal tile's counts are scanned row by row.
#include "plsh_serve.cuh"

namespace plsh {
namespace {

using namespace serve;

constexpr int kRows = 64, kKeys = 64, kThreads = 256;

template <int D, typename MaskT>
struct SimtSmem {
  float q[kRows][D + 4];
  float k[kKeys][D + 4];
  float v[kKeys][D];
  float p[kRows][kKeys + 4];
  MaskT suf[kKeys];      // OR of the masks after key c, up to the tile's last key
  MaskT bm[kKeys];
  MaskT carry[kRows];    // OR of the masks from the tile's end (exclusive) to the row
  uint8_t c[kRows][kKeys];
  int sid;
};

template <typename T, int D, typename MaskT, bool kPaged, bool kQuant>
__global__ void __launch_bounds__(kThreads) serve_simt_kernel(ServeArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  auto& sm = *reinterpret_cast<SimtSmem<D, MaskT>*>(smem_raw);
  if (blockIdx.x == 0 && blockIdx.y == 0) check_seqs(a.sq, a.err);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int mult = a.sq.start ? 2 : 1;
  if (tid < 32) {
    const int s = warp_find(a.sq.cu, a.sq.S, 6, mult, blockIdx.x);
    if (tid == 0) sm.sid = s;
  }
  __syncthreads();
  const Seq sq = load_seq(a.sq, sm.sid);
  const int tile = (sq.pos0 >> 6) + static_cast<int>(blockIdx.x) - ((a.sq.cu[sm.sid] >> 6) + mult * sm.sid);
  const int end = sq.pos0 + sq.len;
  const int i0 = tile * kRows;
  if (tile < 0 || sq.len <= a.few || i0 >= end) return;
  const int h = blockIdx.y, kvh = h / (a.H / a.pg.H_kv);
  const MaskT* bm = static_cast<const MaskT*>(a.bmask) + static_cast<size_t>(h) * a.sq.max_len;
  const float sc = 1.4426950408889634f / sqrtf(static_cast<float>(D));

  // the row of the packed token at a position, or -1 where the position holds none of the new tokens
  auto token = [&](int p) { return (p >= sq.pos0 && p < end) ? sq.c0 + p - sq.pos0 : -1; };
  for (int e = tid; e < kRows * (D / 4); e += kThreads) {
    const int r = e / (D / 4), c = e % (D / 4) * 4;
    const int t = token(i0 + r);
    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (t >= 0) load4f(static_cast<const T*>(a.Q) + t * a.qs.token + h * a.qs.head + c, x);
#pragma unroll
    for (int u = 0; u < 4; ++u) sm.q[r][c + u] = x[u];
  }

  const int T128 = (a.sq.max_len + PLSH_TILE - 1) / PLSH_TILE;
  int lo = a.spans[(static_cast<size_t>(h) * T128 + (i0 >> 7)) * 2];
  if (lo < 0 || lo > i0) {
    if (lo < 0 && tid == 0) atomicOr(a.err, PLSH_DEVERR_WINDOW);
    lo = lo < 0 ? 0 : i0;
  }
  float m[4], l[4] = {0.0f, 0.0f, 0.0f, 0.0f}, acc[4][D / 16];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    m[r] = -INFINITY;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) acc[r][e] = 0.0f;
  }

  for (int j0 = i0; j0 > lo - kKeys && j0 >= 0; j0 -= kKeys) {
    __syncthreads();  // the previous tile has been read
    for (int e = tid; e < kKeys * (D / 4); e += kThreads) {
      const int r = e / (D / 4), c = e % (D / 4) * 4;
      const int p = j0 + r;
      float x[4] = {0.0f, 0.0f, 0.0f, 0.0f}, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (p < end) {
        if constexpr (kPaged) {
          const long long row = page_row(a.pg, sq.s, p, kvh, a.err);
          if (row >= 0) {
            if constexpr (kQuant) {
              e4m3_to_float4(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.pg.k) + row * D + c), x);
              e4m3_to_float4(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.pg.v) + row * D + c), y);
              const float sk = pow2(a.pg.k_exp[row]), sv = pow2(a.pg.v_exp[row]);
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                x[u] *= sk;
                y[u] *= sv;
              }
            } else {
              load4f(static_cast<const T*>(a.pg.k) + row * D + c, x);
              load4f(static_cast<const T*>(a.pg.v) + row * D + c, y);
            }
          }
        } else {
          const long long t = sq.c0 + p;
          load4f(static_cast<const T*>(a.K) + t * a.ks.token + kvh * a.ks.head + c, x);
          load4f(static_cast<const T*>(a.V) + t * a.vs.token + kvh * a.vs.head + c, y);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        sm.k[r][c + u] = x[u];
        sm.v[r][c + u] = y[u];
      }
    }
    if (tid < kKeys) sm.bm[tid] = j0 + tid < end ? bm[j0 + tid] : static_cast<MaskT>(0);
    __syncthreads();
    if (tid < kRows) {
      if (j0 == i0) {  // scan the row's keys from the row down
        MaskT R = 0;
        for (int c = kKeys - 1; c >= 0; --c) {
          if (c > tid) { sm.c[tid][c] = 0; continue; }
          sm.c[tid][c] = static_cast<uint8_t>(a.s - popc_mask<MaskT>(R));
          R |= sm.bm[c];
        }
        sm.carry[tid] = R;
      } else {  // suffix ORs of the tile's keys; thread c scans the keys after c
        MaskT R = 0;
        for (int c = tid + 1; c < kKeys; ++c) R |= sm.bm[c];
        sm.suf[tid] = R;
      }
    }
    __syncthreads();

    float x[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[r][e] = 0.0f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      float4 qa[4], ka[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) qa[r] = *reinterpret_cast<const float4*>(&sm.q[4 * ty + r][c]);
#pragma unroll
      for (int e = 0; e < 4; ++e) ka[e] = *reinterpret_cast<const float4*>(&sm.k[tx + 16 * e][c]);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[r][e] = fmaf(qa[r].x, ka[e].x, fmaf(qa[r].y, ka[e].y, fmaf(qa[r].z, ka[e].z, fmaf(qa[r].w, ka[e].w, x[r][e]))));
    }
    float alpha[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 4 * ty + r;
      int cn[4];
      float top = m[r];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = tx + 16 * e;
        cn[e] = j0 == i0 ? sm.c[row][key] : a.s - popc_mask<MaskT>(sm.carry[row] | sm.suf[key]);
        x[r][e] *= sc;
        if (cn[e] > 0) top = fmaxf(top, x[r][e]);
      }
#pragma unroll
      for (int o = 8; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      alpha[r] = top == -INFINITY ? 1.0f : exp2f(m[r] - top);
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = cn[e] > 0 ? static_cast<float>(cn[e]) * exp2f(x[r][e] - top) : 0.0f;
        sum += p;
        sm.p[row][tx + 16 * e] = p;
      }
      l[r] = l[r] * alpha[r] + sum;
      m[r] = top;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int e = 0; e < D / 16; ++e) acc[r][e] *= alpha[r];
    __syncthreads();
    if (tid < kRows && j0 != i0) sm.carry[tid] |= static_cast<MaskT>(sm.suf[0] | sm.bm[0]);
#pragma unroll 2
    for (int k = 0; k < kKeys; ++k) {
      float pr[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) pr[r] = sm.p[4 * ty + r][k];
#pragma unroll
      for (int e = 0; e < D / 64; ++e) {
        const float4 vv = *reinterpret_cast<const float4*>(&sm.v[k][64 * e + 4 * tx]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          acc[r][4 * e + 0] = fmaf(pr[r], vv.x, acc[r][4 * e + 0]);
          acc[r][4 * e + 1] = fmaf(pr[r], vv.y, acc[r][4 * e + 1]);
          acc[r][4 * e + 2] = fmaf(pr[r], vv.z, acc[r][4 * e + 2]);
          acc[r][4 * e + 3] = fmaf(pr[r], vv.w, acc[r][4 * e + 3]);
        }
      }
    }
  }

#pragma unroll
  for (int r = 0; r < 4; ++r) {
    float total = l[r];
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const int t = token(i0 + 4 * ty + r);
    if (t < 0) continue;
    const float inv = 1.0f / total;
#pragma unroll
    for (int e = 0; e < D / 64; ++e) {
      const float o[4] = {acc[r][4 * e] * inv, acc[r][4 * e + 1] * inv, acc[r][4 * e + 2] * inv, acc[r][4 * e + 3] * inv};
      store4f(static_cast<T*>(a.O) + (static_cast<size_t>(t) * a.H + h) * D + 64 * e + 4 * tx, o);
    }
    if (tx == 0)
      a.row_sum[static_cast<size_t>(t) * a.H + h] =
          (log2f(total) + m[r]) * 0.6931471805599453f - logf(static_cast<float>(a.s));
  }
}

template <typename T, int D, typename MaskT, bool kPaged, bool kQuant>
int launch(const ServeArgs& a, cudaStream_t st) {
  auto kern = serve_simt_kernel<T, D, MaskT, kPaged, kQuant>;
  const int smem = static_cast<int>(sizeof(SimtSmem<D, MaskT>));
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(serve_simt_kernel)");
  const dim3 grid(static_cast<unsigned>((a.sq.T >> 6) + (a.sq.start ? 2 : 1) * a.sq.S), a.H);
  kern<<<grid, kThreads, smem, st>>>(a);
  e = cudaGetLastError();
  return e == cudaSuccess ? PLSH_OK : cuda_fail(e, "serve_simt_kernel launch");
}

template <typename T, int D, typename MaskT>
int launch_src(const ServeArgs& a, cudaStream_t st) {
  if (!a.paged) return launch<T, D, MaskT, false, false>(a, st);
  return a.pg.k_exp ? launch<T, D, MaskT, true, true>(a, st) : launch<T, D, MaskT, true, false>(a, st);
}

template <typename T>
int launch_type(const ServeArgs& a, cudaStream_t st) {
  if (a.d == 128) return a.s <= 32 ? launch_src<T, 128, uint32_t>(a, st) : launch_src<T, 128, unsigned long long>(a, st);
  return a.s <= 32 ? launch_src<T, 64, uint32_t>(a, st) : launch_src<T, 64, unsigned long long>(a, st);
}

}  // namespace

int launch_serve_simt(const ServeArgs& a, cudaStream_t st) {
  return a.dtype == PLSH_BF16 ? launch_type<__nv_bfloat16>(a, st) : launch_type<float>(a, st);
}

}  // namespace plsh
