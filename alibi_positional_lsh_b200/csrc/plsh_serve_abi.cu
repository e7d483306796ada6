// Entry points of the serving operators (declared in include/plsh.h): argument checks, then the launch.
#include <type_traits>
#include <utility>

#include "plsh_internal.h"
#include "plsh_tile_common.cuh"

namespace plsh {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_seqs(const char* fn, int T, int S, const int32_t* cu, int max_len) {
  if (T < 1 || S < 1) return fail(PLSH_ERR_INVALID_ARG, "%s: need T >= 1 and S >= 1 (T=%d S=%d)", fn, T, S);
  if (T > (1 << 30) || S > (1 << 20)) return fail(PLSH_ERR_RANGE, "%s: T=%d exceeds 2^30 or S=%d exceeds 2^20", fn, T, S);
  if (max_len < 1 || max_len > (1 << 30))
    return fail(PLSH_ERR_INVALID_ARG, "%s: need 1 <= max_len <= 2^30 (max_len=%d)", fn, max_len);
  if (!cu) return fail(PLSH_ERR_INVALID_ARG, "%s: null pointer", fn);
  return PLSH_OK;
}

int check_heads(const char* fn, int T, int H, int H_kv, int dtype, int d) {
  if (H < 1 || H > 65535 || H_kv < 1 || H % H_kv != 0)
    return fail(PLSH_ERR_INVALID_ARG, "%s: need 1 <= H <= 65535 and H_kv dividing H (H=%d H_kv=%d)", fn, H, H_kv);
  if (dtype != PLSH_BF16 && dtype != PLSH_F32) return fail(PLSH_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
  if (d != 64 && d != 128) return fail(PLSH_ERR_UNSUPPORTED, "%s: head dim %d (64 or 128 supported)", fn, d);
  if (static_cast<long long>(T) * H > 0x7fffffffLL) return fail(PLSH_ERR_RANGE, "%s: T * H exceeds 2^31", fn);
  return PLSH_OK;
}

// Rows of d elements, 16-byte aligned, `token` elements from one token to the next and `head` between heads.
int check_rows(const char* fn, const char* what, const void* p, int dtype, int d, int heads, int T, long long token,
               long long head) {
  if (!p) return fail(PLSH_ERR_INVALID_ARG, "%s: null pointer (%s)", fn, what);
  const long long es = dtype == PLSH_BF16 ? 2 : 4;
  if (!aligned16(p) || token * es % 16 != 0 || head * es % 16 != 0)
    return fail(PLSH_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned, with strides of whole 16 bytes", fn, what);
  if ((T > 1 && token < d) || (heads > 1 && head < d))
    return fail(PLSH_ERR_INVALID_ARG, "%s: %s's rows overlap (strides %lld and %lld elements, rows of %d)", fn, what, token, head, d);
  return PLSH_OK;
}

int check_pages(const char* fn, const void* k, const void* v, const int8_t* ke, const int8_t* ve, const int32_t* table, int width,
                int num_pages, int page_size) {
  if (!k || !v || !table) return fail(PLSH_ERR_INVALID_ARG, "%s: null pointer", fn);
  if ((ke == nullptr) != (ve == nullptr))
    return fail(PLSH_ERR_INVALID_ARG, "%s: k_exp and v_exp must both be given (e4m3 pages) or both be NULL", fn);
  if (!aligned16(k) || !aligned16(v)) return fail(PLSH_ERR_INVALID_ARG, "%s: pages must be 16-byte aligned", fn);
  if (width < 1 || num_pages < 1)
    return fail(PLSH_ERR_INVALID_ARG, "%s: need num_pages >= 1 and a page table at least one page wide", fn);
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0)
    return fail(PLSH_ERR_UNSUPPORTED, "%s: page size %d (16, 32, 64, 128 or 256 supported)", fn, page_size);
  return PLSH_OK;
}

// Whether the longer sequences of a paged bf16 call are the tile kernel's, or all the rows kernel's, which is quicker for few tokens
// and rereads a window for every few of them. Rows and tiles, us, 16/8 heads, d 128, 4,000 tokens before the new ones, e4m3 (bf16)
// pages: 64 sequences of 8 tokens 72 and 138 (92 and 97), of 16 tokens 111 and 109 (156 and 71), of 24 tokens 181 and 117 (153
// and 78); 8 sequences of 16 tokens 40 and 47 (42 and 40); one of 16 tokens 23 and 42 (18 and 37).
bool tiles_wanted(int T, int max_new) { return max_new > kFewTokens || (max_new > 8 && T > 128); }

// Where the longer sequences are the tile kernel's, whether the others are worth a launch of the rows kernel, or a tile a head each. Rows and
// tiles, us, a chunk of 600 tokens and single ones, 4,000 tokens before each, d 128, e4m3 (bf16) pages: 12 of them, 16/8 heads, 64
// and 55 (57 and 43); 48, 16/8 heads, 91 and 101 (73 and 68); 24, 32/8 heads, 85 and 84 (79 and 69); 48, 32/8 heads, 81 and 121
// (72 and 101). The rule is one for both types of pages: at 768 sequence heads bf16 pages would have been 7 and 14% quicker as tiles. The
// lengths are on the device: few tokens besides the longest sequence's stand for short sequences.
bool rows_wanted(int T, int S, int max_new, int H) {
  return static_cast<long long>(S) * H > 5LL * tiles::sm_count() && T - max_new <= 8LL * S;
}

int lg2(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

PageArgs pages(const void* k, const void* v, const int8_t* ke, const int8_t* ve, const int32_t* table, int width, int num_pages,
               int page_size, int H_kv) {
  return PageArgs{const_cast<void*>(k), const_cast<void*>(v), const_cast<int8_t*>(ke), const_cast<int8_t*>(ve),
                  table, width, num_pages, lg2(page_size), H_kv};
}

int check_plan(const char* fn, int s, const int32_t* spans, const void* bmask, const void* O, const float* row_sum,
               const uint32_t* err) {
  if (s < 1 || s > PLSH_MAX_S) return fail(PLSH_ERR_INVALID_ARG, "%s: need 1 <= s <= %d (s=%d)", fn, PLSH_MAX_S, s);
  if (!spans || !bmask || !O || !row_sum || !err) return fail(PLSH_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned16(O)) return fail(PLSH_ERR_INVALID_ARG, "%s: O must be 16-byte aligned", fn);
  return PLSH_OK;
}

}  // namespace
}  // namespace plsh

using plsh::fail;

extern "C" int plsh_near_counts(const void* bmask_dev, int H, int s, int n, uint8_t* near_dev, void* stream) {
  const char* fn = "plsh_near_counts";
  if (H < 1 || H > 65535 || n < 1 || n > (1 << 30) || s < 1 || s > PLSH_MAX_S)
    return fail(PLSH_ERR_INVALID_ARG, "%s: need 1 <= H <= 65535, 1 <= n <= 2^30 and 1 <= s <= %d (H=%d n=%d s=%d)", fn, PLSH_MAX_S, H, n, s);
  if (!bmask_dev || !near_dev) return fail(PLSH_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!plsh::aligned16(near_dev)) return fail(PLSH_ERR_INVALID_ARG, "%s: near must be 16-byte aligned", fn);
  return plsh::launch_near(bmask_dev, H, s, n, near_dev, static_cast<cudaStream_t>(stream));
}

extern "C" int plsh_packed_fwd(const void* Q, int64_t q_token, int64_t q_head, const void* K, int64_t k_token, int64_t k_head,
                               const void* V, int64_t v_token, int64_t v_head, int dtype, int T, int S,
                               const int32_t* cu_dev, int H, int H_kv, int d, int s, int max_len,
                               const int32_t* tile_span_dev, const void* bmask_dev, const uint8_t* near_dev, void* O, float* row_sum,
                               uint32_t* err_dev, void* stream) {
  const char* fn = "plsh_packed_fwd";
  if (int rc = plsh::check_seqs(fn, T, S, cu_dev, max_len)) return rc;
  if (int rc = plsh::check_heads(fn, T, H, H_kv, dtype, d)) return rc;
  if (int rc = plsh::check_rows(fn, "Q", Q, dtype, d, H, T, q_token, q_head)) return rc;
  if (int rc = plsh::check_rows(fn, "K", K, dtype, d, H_kv, T, k_token, k_head)) return rc;
  if (int rc = plsh::check_rows(fn, "V", V, dtype, d, H_kv, T, v_token, v_head)) return rc;
  if (int rc = plsh::check_plan(fn, s, tile_span_dev, bmask_dev, O, row_sum, err_dev)) return rc;
  if (!near_dev || !plsh::aligned16(near_dev)) return fail(PLSH_ERR_INVALID_ARG, "%s: near_dev must be given, 16-byte aligned", fn);
  plsh::ServeArgs a{};
  a.near = near_dev;
  a.Q = Q; a.qs = {q_token, q_head};
  a.K = K; a.ks = {k_token, k_head};
  a.V = V; a.vs = {v_token, v_head};
  a.paged = false;
  a.pg.H_kv = H_kv;
  a.sq = {cu_dev, nullptr, S, T, max_len, T};
  a.dtype = dtype; a.H = H; a.H_kv = H_kv; a.d = d; a.s = s;
  a.spans = tile_span_dev; a.bmask = bmask_dev;
  a.O = O; a.row_sum = row_sum; a.err = err_dev;
  return dtype == PLSH_BF16 ? plsh::launch_serve_tc(a, static_cast<cudaStream_t>(stream))
                            : plsh::launch_serve_simt(a, static_cast<cudaStream_t>(stream));
}

extern "C" int plsh_cache_append(const void* K, int64_t k_token, int64_t k_head, const void* V, int64_t v_token, int64_t v_head,
                                 int dtype, int T, int S, const int32_t* cu_dev, const int32_t* start_dev, int H_kv, int d,
                                 void* k_pages, void* v_pages, int8_t* k_exp, int8_t* v_exp, const int32_t* page_table_dev,
                                 int table_width, int num_pages, int page_size, uint32_t* err_dev, void* stream) {
  const char* fn = "plsh_cache_append";
  if (int rc = plsh::check_seqs(fn, T, S, cu_dev, 1 << 30)) return rc;
  if (int rc = plsh::check_heads(fn, T, H_kv, H_kv, dtype, d)) return rc;
  if (int rc = plsh::check_rows(fn, "K", K, dtype, d, H_kv, T, k_token, k_head)) return rc;
  if (int rc = plsh::check_rows(fn, "V", V, dtype, d, H_kv, T, v_token, v_head)) return rc;
  if (int rc = plsh::check_pages(fn, k_pages, v_pages, k_exp, v_exp, page_table_dev, table_width, num_pages, page_size)) return rc;
  if (!start_dev || !err_dev) return fail(PLSH_ERR_INVALID_ARG, "%s: null pointer", fn);
  return plsh::launch_cache_append(K, V, dtype, d, {k_token, k_head}, {v_token, v_head}, {cu_dev, start_dev, S, T, 1 << 30, T},
                                   plsh::pages(k_pages, v_pages, k_exp, v_exp, page_table_dev, table_width, num_pages, page_size, H_kv),
                                   err_dev, static_cast<cudaStream_t>(stream));
}

extern "C" int plsh_cache_read(const void* k_pages, const void* v_pages, const int8_t* k_exp, const int8_t* v_exp,
                               const int32_t* page_table_dev, int table_width, int num_pages, int page_size, int T, int S,
                               const int32_t* cu_dev, const int32_t* start_dev, int H_kv, int d, int dtype, void* K, void* V,
                               uint32_t* err_dev, void* stream) {
  const char* fn = "plsh_cache_read";
  if (int rc = plsh::check_seqs(fn, T, S, cu_dev, 1 << 30)) return rc;
  if (int rc = plsh::check_heads(fn, T, H_kv, H_kv, dtype, d)) return rc;
  if (int rc = plsh::check_pages(fn, k_pages, v_pages, k_exp, v_exp, page_table_dev, table_width, num_pages, page_size)) return rc;
  if (!start_dev || !K || !V || !err_dev) return fail(PLSH_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!plsh::aligned16(K) || !plsh::aligned16(V)) return fail(PLSH_ERR_INVALID_ARG, "%s: K and V must be 16-byte aligned", fn);
  return plsh::launch_cache_read(K, V, dtype, d, {cu_dev, start_dev, S, T, 1 << 30, T},
                                 plsh::pages(k_pages, v_pages, k_exp, v_exp, page_table_dev, table_width, num_pages, page_size, H_kv),
                                 err_dev, static_cast<cudaStream_t>(stream));
}

extern "C" size_t plsh_paged_scratch_bytes(int T, int S, int max_new, int H_kv, int d, int max_window) {
  if (T < 1 || S < 1 || H_kv < 1 || d < 1 || max_window < 1 || !plsh::tiles_wanted(T, max_new)) return 0;
  return plsh::serve_scratch_bytes(T, S, H_kv, d, max_window);
}

extern "C" int plsh_paged_fwd(const void* Q, int64_t q_token, int64_t q_head, int dtype, int T, int S, const int32_t* cu_dev,
                              const int32_t* start_dev, int max_new, int H, int H_kv, int d, const void* k_pages,
                              const void* v_pages, const int8_t* k_exp, const int8_t* v_exp, const int32_t* page_table_dev,
                              int table_width, int num_pages, int page_size, int s, int max_len, const double* table_dev,
                              const int32_t* tile_span_dev, const void* bmask_dev, const uint8_t* near_dev,
                              const int32_t* windows_host,
                              void* scratch_dev, size_t scratch_bytes, void* O, float* row_sum, uint32_t* err_dev,
                              void* stream) {
  const char* fn = "plsh_paged_fwd";
  if (int rc = plsh::check_seqs(fn, T, S, cu_dev, max_len)) return rc;
  if (int rc = plsh::check_heads(fn, T, H, H_kv, dtype, d)) return rc;
  if (int rc = plsh::check_rows(fn, "Q", Q, dtype, d, H, T, q_token, q_head)) return rc;
  if (int rc = plsh::check_pages(fn, k_pages, v_pages, k_exp, v_exp, page_table_dev, table_width, num_pages, page_size)) return rc;
  if (int rc = plsh::check_plan(fn, s, tile_span_dev, bmask_dev, O, row_sum, err_dev)) return rc;
  if (!table_dev || !start_dev) return fail(PLSH_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!windows_host) return fail(PLSH_ERR_INVALID_ARG, "%s: null pointer", fn);
  int max_window = 0;
  for (int h = 0; h < H; ++h) {
    if (windows_host[h] < 1 || windows_host[h] > max_len)
      return fail(PLSH_ERR_INVALID_ARG, "%s: need 1 <= windows_host[h] <= max_len (%d for head %d)", fn, windows_host[h], h);
    if (windows_host[h] > max_window) max_window = windows_host[h];
  }
  const bool tiles = dtype == PLSH_BF16 && plsh::tiles_wanted(T, max_new);
  if (!near_dev || !plsh::aligned16(near_dev)) return fail(PLSH_ERR_INVALID_ARG, "%s: near_dev must be given, 16-byte aligned", fn);
  if (tiles && k_exp) {
    const size_t need = plsh_paged_scratch_bytes(T, S, max_new, H_kv, d, max_window);
    if (!scratch_dev || !plsh::aligned16(scratch_dev) || scratch_bytes < need)
      return fail(PLSH_ERR_INVALID_ARG, "%s: scratch (16-byte aligned) holds %zu bytes, %zu needed", fn, scratch_bytes, need);
  }
  if (max_new < 1) return fail(PLSH_ERR_INVALID_ARG, "%s: need max_new >= 1 (max_new=%d)", fn, max_new);
  plsh::ServeArgs a{};
  a.Q = Q; a.qs = {q_token, q_head};
  a.paged = true;
  a.near = near_dev;
  a.table = table_dev;
  a.scratch = scratch_dev;
  a.max_window = max_window;
  a.windows_host = windows_host;
  a.pg = plsh::pages(k_pages, v_pages, k_exp, v_exp, page_table_dev, table_width, num_pages, page_size, H_kv);
  a.sq = {cu_dev, start_dev, S, T, max_len, max_new};
  a.dtype = dtype; a.H = H; a.H_kv = H_kv; a.d = d; a.s = s;
  a.spans = tile_span_dev; a.bmask = bmask_dev;
  a.O = O; a.row_sum = row_sum; a.err = err_dev;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == PLSH_BF16) {
    a.few = !tiles ? plsh::kFewTokens : plsh::rows_wanted(T, S, max_new, H) ? plsh::rows_block_tokens(H / H_kv) : 0;
    if (a.few > 0)
      if (int rc = plsh::launch_serve_rows(a, st)) return rc;
    return tiles ? plsh::launch_serve_tc(a, st) : PLSH_OK;
  }
  return plsh::launch_serve_simt(a, st);
}

// The same calls with their arguments in an array.
namespace {
template <typename T>
T arg(int64_t x) {
  if constexpr (std::is_pointer_v<T>) return reinterpret_cast<T>(static_cast<uintptr_t>(x));
  else return static_cast<T>(x);
}
template <typename T>
bool fits(int64_t x) {
  if constexpr (std::is_same_v<T, int>) return x == static_cast<int>(x);
  else return true;
}
template <typename... P, size_t... I>
int spread(const char* fn, int (*f)(P...), const int64_t* args, std::index_sequence<I...>) {
  if (!(fits<P>(args[I]) && ...)) return fail(PLSH_ERR_RANGE, "%s: an argument does not fit its type", fn);
  return f(arg<P>(args[I])...);
}
template <typename... P>
int spread(const char* fn, int (*f)(P...), const int64_t* args, size_t bytes) {
  if (!args || bytes != sizeof...(P) * sizeof(int64_t))
    return fail(PLSH_ERR_INVALID_ARG, "%s: %zu bytes of arguments needed, %zu given", fn, sizeof...(P) * sizeof(int64_t), args ? bytes : 0);
  return spread(fn, f, args, std::make_index_sequence<sizeof...(P)>());
}
}  // namespace

extern "C" int plsh_packed_fwd_args(const int64_t* args, size_t bytes) { return spread("plsh_packed_fwd_args", plsh_packed_fwd, args, bytes); }
extern "C" int plsh_cache_append_args(const int64_t* args, size_t bytes) { return spread("plsh_cache_append_args", plsh_cache_append, args, bytes); }
extern "C" int plsh_cache_read_args(const int64_t* args, size_t bytes) { return spread("plsh_cache_read_args", plsh_cache_read, args, bytes); }
extern "C" int plsh_paged_fwd_args(const int64_t* args, size_t bytes) { return spread("plsh_paged_fwd_args", plsh_paged_fwd, args, bytes); }
