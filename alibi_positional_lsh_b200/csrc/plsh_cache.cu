// The paged cache: new rows of K and V written into it (quantised to e4m3, or copied), and a range
// of every sequence read back as packed tensors.
//
// A quantised row x of d numbers is held as RN_e4m3(x 2^-e) with one exponent e per (page, head, place):
// the least e >= -126 with max|x| <= 448 * 2^e (plsh_serve.cuh says why a power of two).
//
// Both directions are bound by memory: 2 (d es + d + 1) bytes a token and head. A block takes a few tokens with all their
// heads: it finds their sequences and pages once, then moves rows 16 bytes a lane on the packed side (16 lanes
// a row of 128 bf16), K and V of two rows in flight per lane; a row's largest magnitude is a butterfly over its lanes.
#include "plsh_serve.cuh"
#include "plsh_tile_common.cuh"

namespace plsh {
namespace {

using namespace serve;

constexpr int kThreads = 256;
constexpr int kTokens = 8;  // most tokens of a block

// The rows of head 0 of a block's tokens: -1 where the token is of no sequence, -2 where its page is not there.
__device__ __forceinline__ void find_rows(const SeqArgs& sq, const PageArgs& pg, int t0, int n, long long* base, uint32_t* err) {
  if (blockIdx.x == 0) check_seqs(sq, err);
  const int tid = threadIdx.x;
  if (tid < n) {
    const int t = t0 + tid;
    int lo = 0, hi = sq.S;  // the last sequence that begins at or before t
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (sq.cu[mid] <= t) lo = mid;
      else hi = mid;
    }
    const Seq q = load_seq(sq, lo);
    long long row = -1;
    if (t >= q.c0 && t < q.c0 + q.len) {
      row = page_row(pg, q.s, q.pos0 + t - q.c0, 0, err);
      if (row < 0) row = -2;
    }
    base[tid] = row;
  }
  __syncthreads();
}

template <typename T>
__device__ __forceinline__ void floats_of(const uint4& w, float (&x)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  } else {
    x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y); x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
  }
}

template <typename T, int D, bool kQuant>
__global__ void __launch_bounds__(kThreads)
append_kernel(const T* __restrict__ K, const T* __restrict__ V, RowStrides ks, RowStrides vs, SeqArgs sq, PageArgs pg, int tokens,
              uint32_t* __restrict__ err) {
  __shared__ long long base[kTokens];
  const int t0 = blockIdx.x * tokens, n = min(tokens, sq.T - t0);
  find_rows(sq, pg, t0, n, base, err);
  constexpr int E = 16 / sizeof(T), kLanes = D / E;  // elements a lane, lanes a row
  const int l = threadIdx.x % kLanes, rows = n * pg.H_kv;
  // (whole warps stay together: their butterflies need every lane)
#pragma unroll 2
  for (int i0 = 0; i0 < rows; i0 += kThreads / kLanes) {
    const int i = i0 + threadIdx.x / kLanes;
    const int k = i / pg.H_kv, h = i % pg.H_kv;
    const long long first = i < rows ? base[k] : -1, row = first + (static_cast<long long>(h) << pg.lg_page);
    const bool on = first >= 0;
    uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (on) {
      w[0] = __ldcs(reinterpret_cast<const uint4*>(K + (t0 + k) * ks.token + h * ks.head) + l);
      w[1] = __ldcs(reinterpret_cast<const uint4*>(V + (t0 + k) * vs.token + h * vs.head) + l);
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      void* pages = kv == 0 ? pg.k : pg.v;
      if constexpr (kQuant) {
        float x[E], m = 0.0f;
        floats_of<T>(w[kv], x);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const bool finite = fabsf(x[e]) <= 3.402823466e38f;
          if (!finite) x[e] = __int_as_float(0x7FC00000);
          m = fmaxf(m, finite ? fabsf(x[e]) : 0.0f);
        }
#pragma unroll
        for (int o = kLanes / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int ex = e4m3_exponent(m);
        const float inv = pow2(-ex);
        uint32_t q[E / 4];
#pragma unroll
        for (int e = 0; e < E; e += 4) q[e / 4] = e4m3x4(x[e] * inv, x[e + 1] * inv, x[e + 2] * inv, x[e + 3] * inv);
        if (on) {
          uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(pages) + row * D) + l * (E / 4);
          if constexpr (E == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(q[0], q[1]);
          else *dst = q[0];
          if (l == 0) (kv == 0 ? pg.k_exp : pg.v_exp)[row] = static_cast<int8_t>(ex);
        }
      } else {
        if (on) reinterpret_cast<uint4*>(static_cast<T*>(pages) + row * D)[l] = w[kv];
      }
    }
  }
}

template <typename T, int D, bool kQuant>
__global__ void __launch_bounds__(kThreads)
read_kernel(SeqArgs sq, PageArgs pg, int tokens, T* __restrict__ K, T* __restrict__ V, uint32_t* __restrict__ err) {
  __shared__ long long base[kTokens];
  const int t0 = blockIdx.x * tokens, n = min(tokens, sq.T - t0);
  find_rows(sq, pg, t0, n, base, err);
  constexpr int E = 16 / sizeof(T), kLanes = D / E;
  const int l = threadIdx.x % kLanes, rows = n * pg.H_kv;
#pragma unroll 2
  for (int i = threadIdx.x / kLanes; i < rows; i += kThreads / kLanes) {
    const int k = i / pg.H_kv, h = i % pg.H_kv;
    const long long out = (static_cast<long long>(t0 + k) * pg.H_kv + h) * D;
    if (base[k] < 0) {
      if (base[k] == -2) {
        __stcs(reinterpret_cast<uint4*>(K + out) + l, make_uint4(0, 0, 0, 0));
        __stcs(reinterpret_cast<uint4*>(V + out) + l, make_uint4(0, 0, 0, 0));
      }
      continue;
    }
    const long long row = base[k] + (static_cast<long long>(h) << pg.lg_page);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const void* pages = kv == 0 ? pg.k : pg.v;
      uint4 w;
      if constexpr (kQuant) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(pages) + row * D) + l * (E / 4);
        const float sc = pow2((kv == 0 ? pg.k_exp : pg.v_exp)[row]);
        if constexpr (E == 8) {
          const uint2 q = *reinterpret_cast<const uint2*>(src);
          float x[4], y[4];
          e4m3_to_float4(q.x, x);
          e4m3_to_float4(q.y, y);
          const __nv_bfloat162 b[4] = {__floats2bfloat162_rn(x[0] * sc, x[1] * sc), __floats2bfloat162_rn(x[2] * sc, x[3] * sc),
                                       __floats2bfloat162_rn(y[0] * sc, y[1] * sc), __floats2bfloat162_rn(y[2] * sc, y[3] * sc)};
          w = *reinterpret_cast<const uint4*>(b);
        } else {
          float x[4];
          e4m3_to_float4(*src, x);
          w = make_uint4(__float_as_uint(x[0] * sc), __float_as_uint(x[1] * sc), __float_as_uint(x[2] * sc), __float_as_uint(x[3] * sc));
        }
      } else {
        w = reinterpret_cast<const uint4*>(static_cast<const T*>(pages) + row * D)[l];
      }
      __stcs(reinterpret_cast<uint4*>((kv == 0 ? K : V) + out) + l, w);
    }
  }
}

// Tokens of a block: four blocks for every SM first, then up to 8 tokens, so that the rows' addresses are found once for many. With 1, 2, 4, 8
// and 16 tokens (bf16 into e4m3 and back, 8 heads, d 128): 10.6, 10.5, 14.3, 16.4 and 22.6 us for 100 tokens, 26.6, 22.5, 21.2, 22.5
// and 26.7 us for 4,000, 71.7, 51.2, 47.1, 45.1 and 48.3 us for 16,000.
int tokens_per_block(int T) {
  int n = 1;
  while (n < kTokens && T / (2 * n) >= 4 * tiles::sm_count()) n *= 2;
  return n;
}

}  // namespace

int launch_cache_append(const void* K, const void* V, int dtype, int d, RowStrides ks, RowStrides vs, const SeqArgs& sq,
                        const PageArgs& pg, uint32_t* err, cudaStream_t st) {
  const int tokens = tokens_per_block(sq.T);
  const unsigned grid = static_cast<unsigned>(ceil_div(sq.T, tokens));
  const bool q = pg.k_exp != nullptr;
#define PLSH_APPEND(T, D, Q) \
  append_kernel<T, D, Q><<<grid, kThreads, 0, st>>>(static_cast<const T*>(K), static_cast<const T*>(V), ks, vs, sq, pg, tokens, err)
  if (dtype == PLSH_BF16) {
    if (d == 128) { if (q) PLSH_APPEND(__nv_bfloat16, 128, true); else PLSH_APPEND(__nv_bfloat16, 128, false); }
    else { if (q) PLSH_APPEND(__nv_bfloat16, 64, true); else PLSH_APPEND(__nv_bfloat16, 64, false); }
  } else {
    if (d == 128) { if (q) PLSH_APPEND(float, 128, true); else PLSH_APPEND(float, 128, false); }
    else { if (q) PLSH_APPEND(float, 64, true); else PLSH_APPEND(float, 64, false); }
  }
#undef PLSH_APPEND
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PLSH_OK : cuda_fail(e, "append_kernel launch");
}

int launch_cache_read(void* K, void* V, int dtype, int d, const SeqArgs& sq, const PageArgs& pg, uint32_t* err,
                      cudaStream_t st) {
  const int tokens = tokens_per_block(sq.T);
  const unsigned grid = static_cast<unsigned>(ceil_div(sq.T, tokens));
  const bool q = pg.k_exp != nullptr;
#define PLSH_READ(T, D, Q) \
  read_kernel<T, D, Q><<<grid, kThreads, 0, st>>>(sq, pg, tokens, static_cast<T*>(K), static_cast<T*>(V), err)
  if (dtype == PLSH_BF16) {
    if (d == 128) { if (q) PLSH_READ(__nv_bfloat16, 128, true); else PLSH_READ(__nv_bfloat16, 128, false); }
    else { if (q) PLSH_READ(__nv_bfloat16, 64, true); else PLSH_READ(__nv_bfloat16, 64, false); }
  } else {
    if (d == 128) { if (q) PLSH_READ(float, 128, true); else PLSH_READ(float, 128, false); }
    else { if (q) PLSH_READ(float, 64, true); else PLSH_READ(float, 64, false); }
  }
#undef PLSH_READ
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PLSH_OK : cuda_fail(e, "read_kernel launch");
}

}  // namespace plsh
