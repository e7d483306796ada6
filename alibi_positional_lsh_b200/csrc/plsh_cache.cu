// The paged cache: new rows of K and V written into it (quantised to e4m3, or copied), and a range
// of every sequence read back as packed tensors.
//
// A quantised row x of d numbers is held as RN_e4m3(x 2^-e) with one exponent e per (page, head, place):
// the least e >= -126 with max|x| <= 448 * 2^e (plsh_serve.cuh says why a power of two).
#include "plsh_serve.cuh"

namespace plsh {
namespace {

using namespace serve;

constexpr int kWarps = 8;

// One warp per (token, head): its K row, then its V row. d / 4 lanes hold four elements each.
template <typename T, int D, bool kQuant>
__global__ void __launch_bounds__(kWarps * 32)
append_kernel(const T* __restrict__ K, const T* __restrict__ V, RowStrides ks, RowStrides vs, SeqArgs sq, PageArgs pg,
              uint32_t* __restrict__ err) {
  if (blockIdx.x == 0) check_seqs(sq, err);
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int t = static_cast<int>(w / pg.H_kv), h = static_cast<int>(w % pg.H_kv);
  if (t >= sq.T) return;
  const Seq q = load_seq(sq, warp_find_token(sq.cu, sq.S, t));
  if (t < q.c0 || t >= q.c0 + q.len) return;  // in no sequence
  const long long row = page_row(pg, q.s, q.pos0 + t - q.c0, h, err);
  if (row < 0) return;
  const bool on = 4 * lane < D;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const T* src = kv == 0 ? K + t * ks.token + h * ks.head : V + t * vs.token + h * vs.head;
    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (on) load4f(src + 4 * lane, x);
    void* pages = kv == 0 ? pg.k : pg.v;
    if constexpr (kQuant) {
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool finite = fabsf(x[i]) <= 3.402823466e38f;
        if (!finite) x[i] = __int_as_float(0x7FC00000);
        m = fmaxf(m, finite ? fabsf(x[i]) : 0.0f);
      }
      m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));  // non-negative floats order as their bits
      const int e = e4m3_exponent(m);
      const float inv = pow2(-e);
      if (on)
        reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(pages) + row * D)[lane] =
            e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
      if (lane == 0) (kv == 0 ? pg.k_exp : pg.v_exp)[row] = static_cast<int8_t>(e);
    } else {
      if (on) store4f(static_cast<T*>(pages) + row * D + 4 * lane, x);
    }
  }
}

template <typename T, int D, bool kQuant>
__global__ void __launch_bounds__(kWarps * 32)
read_kernel(SeqArgs sq, PageArgs pg, T* __restrict__ K, T* __restrict__ V, uint32_t* __restrict__ err) {
  if (blockIdx.x == 0) check_seqs(sq, err);
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int t = static_cast<int>(w / pg.H_kv), h = static_cast<int>(w % pg.H_kv);
  if (t >= sq.T) return;
  const Seq q = load_seq(sq, warp_find_token(sq.cu, sq.S, t));
  if (t < q.c0 || t >= q.c0 + q.len) return;
  const long long row = page_row(pg, q.s, q.pos0 + t - q.c0, h, err);
  if (row < 0 || 4 * lane >= D) return;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const void* pages = kv == 0 ? pg.k : pg.v;
    float x[4];
    if constexpr (kQuant) {
      e4m3_to_float4(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(pages) + row * D)[lane], x);
      const float sc = pow2((kv == 0 ? pg.k_exp : pg.v_exp)[row]);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] *= sc;
    } else {
      load4f(static_cast<const T*>(pages) + row * D + 4 * lane, x);
    }
    store4f((kv == 0 ? K : V) + w * D + 4 * lane, x);
  }
}

}  // namespace

int launch_cache_append(const void* K, const void* V, int dtype, int d, RowStrides ks, RowStrides vs, const SeqArgs& sq,
                        const PageArgs& pg, uint32_t* err, cudaStream_t st) {
  const long long rows = static_cast<long long>(sq.T) * pg.H_kv;
  const unsigned grid = static_cast<unsigned>((rows + kWarps - 1) / kWarps);
  const bool q = pg.k_exp != nullptr;
#define PLSH_APPEND(T, D, Q) \
  append_kernel<T, D, Q><<<grid, kWarps * 32, 0, st>>>(static_cast<const T*>(K), static_cast<const T*>(V), ks, vs, sq, pg, err)
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
  const long long rows = static_cast<long long>(sq.T) * pg.H_kv;
  const unsigned grid = static_cast<unsigned>((rows + kWarps - 1) / kWarps);
  const bool q = pg.k_exp != nullptr;
#define PLSH_READ(T, D, Q) \
  read_kernel<T, D, Q><<<grid, kWarps * 32, 0, st>>>(sq, pg, static_cast<T*>(K), static_cast<T*>(V), err)
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
