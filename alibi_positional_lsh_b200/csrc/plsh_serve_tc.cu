// T~ for packed prompts (and chunks against the paged cache) on the sm_100a tensor cores, bf16.
//
//   O_i = sum_{j <= i} c_ij e^{S_ij} V_j / sum_{j <= i} c_ij e^{S_ij},   S = Q K^T / sqrt(d),
// c_ij counting the hashes that put positions i and j into one bin (Positional LSH technical summary,
// Methodology 2; blocks are contiguous, Methodology 1).
//
// The counts are a matrix product. Take a key tile whose last key is e, and rows i > e. Hash k
// puts i and j together exactly if it has no block boundary in (j, e] and none in (e, i], so
//   c_ij = sum_k a_ik b_jk,   a_ik = [no boundary of k in (e, i]],   b_jk = [none in (j, e]],
// a product of two 0/1 matrices with one column per hash. They are written as e4m3 bytes and
// multiplied by the tensor cores beside S: one instruction per 32 hashes, instead of an OR, a
// population count and a conversion for every score. Both are exact (each byte is 2.0 or 0, so the product is
// 4 c; the 4 cancels in O and leaves row_sum as two in the logarithm). Only the counts of a row's own
// 64-key tile, where no key lies behind all rows, are read: they depend on the position and the head alone, and the plan
// holds them as bytes (near_kernel).
//
// Work. One item is a 128-row tile of one head, against 64-key tiles of K and V from the diagonal down. Two blocks share
// an SM, each with half of Tensor Memory, so that one's products run under the other's exponentials; persistent
// blocks walk the items, heads with the widest windows first. Eight warps: four of softmax threads (one row each), one that
// finds the items, one that loads Q, K and V by TMA, one that issues the MMAs and one that writes the counts' operands.
// Tensor Memory: S (64 columns), 4 c (64 columns, P over them as bf16), O (D columns).
//
// Per key tile g:
//   MMA      S(g) = Q K^T once S(g - 1) has been read,  O += P(g - 1) V,  C(g) = A B^T
//   softmax  P = 4c 2^(S log2e/sqrt(d) - m);  l += sum P
// The reference m starts at 0 and changes only where a row leaves the range it is good for: its sum above 2^62, or, in
// the tile of the row's own key (which has the largest count), below 2^-30 as soon as a key with weight is in it. fp32 and bf16
// hold P between these limits with full relative precision, and 2^62 leaves P V room in fp32 for any |V| up to 2^64, so no
// maximum is taken otherwise (a limit of 2^40, with room up to 2^80: scores around 15 +- 3, 24 prompts as below, 292 us instead of
// 154); these 32 keys are then done
// again with m = the maximum over those with c > 0, and what was summed before follows by the same power of two. Keys that
// come before the own one in its tile may hold all of the row's weight: below 2^-126 their P would be zero, and nothing
// could bring it back. No score of a key without weight can push a row's weights out of range.
//
// P is rounded to bf16 for the second product. O is divided by the sum of the rounded P over the row's own 32 keys (a block of the warp's) and of P
// before them, which takes back most of that rounding where few keys carry the weight (a row's only key then gives its V exactly) and
// costs nothing outside those tiles; row_sum is of P itself.
//
// Rows past a sequence's end hold another sequence's data: their K and V rows are cleared in shared memory before the
// products, so that nothing there, not even a NaN, meets a zero weight: a sequence's result has the same bits whatever it is packed with.
//
// What bounds it: the chain of one tile (S read, exponentials, P written, P V) with two blocks an SM to overlap it, and the size
// of its code; 24 prompts of 1 to 3,001 tokens, 32/8 heads, d 128: 158 us, the tensor pipe busy 26%, issue slots 32%, the special
// function unit 16%. Every fourth pair's exponentials as a polynomial on the FMA pipe: 184 us. Items fetched by cancelling
// unstarted blocks instead of the list dealt out in a snake: 170 us (every block reserves the widest items ahead of their use).
//
// Every barrier wait is bounded in time (PLSH_DEVERR_TIMEOUT), as in the fused kernel.
#include <cmath>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "plsh_serve.cuh"
#include "plsh_sm100.cuh"
#include "plsh_tile_common.cuh"

namespace plsh {
namespace {

using namespace sm100;
using namespace serve;
using tiles::regs_after_wait;

constexpr int kThreads = 256;
constexpr int kSoftmaxWarps = 4;
constexpr int kWarpItems = 4, kWarpLoad = 5, kWarpMma = 6;  // and 7, the counts' operands
constexpr int kRows = 128, kKeys = 64;
constexpr int kItems = 4;                     // item descriptors in flight
constexpr uint32_t kTmemCols = 256;           // half of Tensor Memory: two blocks share an SM
constexpr uint32_t kColS = 0, kColC = 64, kColO = 128;
constexpr float kSumMax = 4.6116860e18f, kSumMin = 9.3132257e-10f;  // 2^62, 2^-30
constexpr int kMaxSortedHeads = 256;
constexpr uint64_t kDrainNs = 100000000ull;
// Registers per thread: 256 x 128 at launch; the softmax warpgroup takes 216, the other one keeps 40 (192 and 64: 7% slower, by spills).
constexpr uint32_t kRegsSoftmax = 216, kRegsRest = 40;

// One row tile of one head: positions i0 .. i0 + 127 of sequence s, against key tiles top, top - 1, .., low.
struct Item {
  int valid, h, i0, c0, pos0, end, s, top, low;
  int kv0;  // row of K and V that holds position 0
  // K and V from pages: the first row reaches every key from `sure` on, and the lowest it reaches is `reach` (looked for on the way
  // down below `sure`; known already where that is 0)
  int reach, sure;
};

// The sum of 32 bf16, in fp32.
__device__ __forceinline__ float sum_bf16(const uint32_t (&w)[16]) {
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    asm("{.reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n add.rn.f32.bf16 %0, lo, %0;\n add.rn.f32.bf16 %1, hi, %1;}"
        : "+f"(s[2 * (i & 1)]), "+f"(s[2 * (i & 1) + 1]) : "r"(w[i]));
  return (s[0] + s[1]) + (s[2] + s[3]);
}

template <int D, typename MaskT>
struct __align__(1024) TcSmem {
  static constexpr int kQBytes = kRows * D * 2, kKBytes = kKeys * D * 2;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kVStages = D == 128 && sizeof(MaskT) == 8 ? 1 : kStages;  // 64 hashes' operands leave room for one
  static constexpr int kFeat = sizeof(MaskT) * 8;  // bytes of a row of a or b: one per hash
  uint8_t q[kQBytes];
  uint8_t k[kStages][kKBytes];
  uint8_t v[kVStages][kKBytes];
  // rows of a: 128 with the pivot before the row tile, then rows 64..127 with the pivot inside it (their operand
  // starts 64 rows earlier: the counts of its first 64 rows are not used)
  uint8_t a[(kRows + kRows / 2) * kFeat];
  uint8_t b[2][kKeys * kFeat];
  // [item parity]: OR of the boundary masks from the row tile's first row to the row, then for rows 64..127 from row 64 on
  MaskT rows[2][kRows + kRows / 2];
  MaskT gap[2], upper[2];   // [stage]: OR between the key tile and the row tile; OR of the key tile's keys 32..63
  Item item[kItems];
  int missing[2 * kItems], reach[2 * kItems];  // of an item, by its number (see the loads)
  int16_t order[kMaxSortedHeads];
  int32_t width[kMaxSortedHeads];
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t q_full, q_empty;
  uint64_t k_full[kStages], k_empty[kStages], v_full[kVStages], v_empty[kVStages];
  uint64_t feat_full[2], feat_empty[2];
  uint64_t s_free, c_full, p_full, o_full, drain;
  uint32_t tmem_base;
  int abort_flag;
};

struct TcParams {
  SeqArgs sq;
  int H, H_kv, s, slots, items;
  int few;       // sequences with at most this many tokens are the row kernel's
  int kv_pad;    // gathered K and V: rows before a sequence's new tokens (0: K and V are packed as Q)
  PageArgs pg;   // pages of bf16 (kPaged)
  int q_swap, k_swap, v_swap;  // tensor map's second coordinate is the token (head-major storage) instead of the head
  const int32_t* spans;
  const uint8_t* near;  // [H][max_len][64]: c of the keys of each position's own 64-key tile
  uint32_t wait_limit;  // of every barrier wait, in steps of 2^20 ns
  float log_s;
  int withhold_mma;
};

// ---- counts as a product

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 operands, fp32 accumulation, 32 columns of K
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

// K-major operand without swizzle: blocks of 8 rows x 16 bytes, 128 bytes apart along K, `group`
// bytes from one group of 8 rows to the next.
__device__ __forceinline__ uint64_t smem_desc_plain(uint32_t saddr, uint32_t group) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((128u >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((group >> 4) & 0x3FFFu) << 32;
  d |= 1ull << 46;
  return d;
}

__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

// A value that all lanes hold alike, known as such to the compiler.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// 32 bytes of a row, 16-byte aligned; in one store where `whole` says that the address is a multiple of 32 (two stores everywhere:
// 24 prompts of 1 to 3,001 tokens 176 us instead of 159).
__device__ __forceinline__ void store32(void* p, const uint32_t* w, bool whole) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    uint4* const dst = static_cast<uint4*>(p);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// Row r of a 0/1 operand: byte k is 0x40 (e4m3 2.0) where bit k is set. Four bits spread to four bytes by one multiply.
__device__ __forceinline__ uint32_t spread4(uint32_t bits) { return ((bits & 0xFu) * (0x00204081u << 6)) & 0x40404040u; }

template <typename MaskT>
__device__ __forceinline__ void put_bits(uint8_t* base, int r, MaskT bits) {
  constexpr int kChunks = sizeof(MaskT) / 2;  // 16 bytes (16 hashes) each
  uint8_t* row = base + (r >> 3) * (128 * kChunks) + (r & 7) * 16;
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const uint32_t w = static_cast<uint32_t>(bits >> (16 * c));
    *reinterpret_cast<uint4*>(row + 128 * c) = make_uint4(spread4(w), spread4(w >> 4), spread4(w >> 8), spread4(w >> 12));
  }
}

// mbar_wait (plsh_sm100.cuh) with the polling loop in place: a kernel that moves registers between its warpgroups cannot
// call a function, whose own registers would be those of the launch. It is kept short (the limit in steps of 2^20 ns, the error
// word written once at the kernel's end): at some twenty places, its code decides whether the kernel's loops stay in
// the instruction cache (with the longer form the kernel had 68 KB, and ran half as fast again).
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t limit) {
  uint32_t until = 0;
  while (!mbar_try_wait(bar, parity)) {
    const uint32_t now = static_cast<uint32_t>(global_timer_ns() >> 20);
    if (until == 0) until = now + limit;
    if (*abort_flag || static_cast<int32_t>(now - until) > 0) {
      *abort_flag = 1;
      return false;
    }
  }
  return true;
}

// near[h][p][k]: c of position p and key k of its own 64-key tile (0 past p). One thread per position scans from it down.
template <typename MaskT>
__global__ void __launch_bounds__(256) near_kernel(const MaskT* __restrict__ bmask, int s, int n, uint8_t* __restrict__ near) {
  const int p = blockIdx.x * 256 + threadIdx.x;
  if (p >= n) return;
  const MaskT* bm = bmask + static_cast<size_t>(blockIdx.y) * n;
  uint32_t* out = reinterpret_cast<uint32_t*>(near + (static_cast<size_t>(blockIdx.y) * n + p) * kKeys);
  const int j0 = p & ~(kKeys - 1);
  MaskT R = 0;
  for (int w = kKeys / 4 - 1; w >= 0; --w) {
    uint32_t four = 0;
    for (int e = 3; e >= 0; --e) {
      const int j = j0 + 4 * w + e;
      if (j > p) continue;
      four |= static_cast<uint32_t>(s - popc_mask<MaskT>(R)) << (8 * e);
      R = static_cast<MaskT>(R | bm[j]);
    }
    out[w] = four;
  }
}

// ---- the kernel

template <int D, typename MaskT, bool kPaged>
__global__ void __launch_bounds__(kThreads, 2)
serve_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ TcParams prm,
                const MaskT* __restrict__ bmask, __nv_bfloat16* __restrict__ O, float* __restrict__ row_sum,
                uint32_t* __restrict__ err) {
  using Smem = TcSmem<D, MaskT>;
  constexpr int kStages = Smem::kStages, kVStages = Smem::kVStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t smem_pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  auto& sm = *reinterpret_cast<Smem*>(smem_raw + smem_pad);
  volatile int* abort_flag = &sm.abort_flag;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int H = prm.H, s = prm.s, max_len = prm.sq.max_len;
  const int T128 = (max_len + PLSH_TILE - 1) / PLSH_TILE;
  const MaskT FULL = (s >= static_cast<int>(8 * sizeof(MaskT))) ? static_cast<MaskT>(~static_cast<MaskT>(0))
                                                                : static_cast<MaskT>((static_cast<MaskT>(1) << s) - 1);
  constexpr int kFeat = Smem::kFeat;
  constexpr uint32_t kFeatGroup = 128 * (kFeat / 16);

  if (blockIdx.x == 0) check_seqs(prm.sq, err);
  // heads by decreasing window width of the middle row tile
  if (H <= kMaxSortedHeads) {
#pragma unroll 1
    for (int h = threadIdx.x; h < H; h += kThreads) {
      const int t = T128 / 2;
      sm.width[h] = min(max_len, t * PLSH_TILE + PLSH_TILE) - prm.spans[(static_cast<size_t>(h) * T128 + t) * 2];
    }
    __syncthreads();
#pragma unroll 1
    for (int h = threadIdx.x; h < H; h += kThreads) {
      const int wh = sm.width[h];
      int rank = 0;
#pragma unroll 1
      for (int o = 0; o < H; ++o) {
        const int wo = sm.width[o];
        rank += (wo > wh) || (wo == wh && o < h);
      }
      sm.order[rank] = static_cast<int16_t>(h);
    }
  }
  if (threadIdx.x == 0) {
    sm.abort_flag = 0;
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&sm.item_full[i], 1);
      mbar_init(&sm.item_empty[i], kSoftmaxWarps + 3);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.feat_full[i], 1);
      mbar_init(&sm.feat_empty[i], kSoftmaxWarps + 1);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    mbar_init(&sm.s_free, kSoftmaxWarps);
    mbar_init(&sm.c_full, 1);
    mbar_init(&sm.p_full, kSoftmaxWarps);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.drain, 1);
    fence_mbarrier_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(&sm.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(sm.tmem_base);
  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_bounded(bar, parity & 1u, abort_flag, prm.wait_limit); };
  // the same by a whole warp: false in every lane if any gave up
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity & 1u))) return true;
    return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
  };

  if (warp < kSoftmaxWarps) {
    regs_raise<kRegsSoftmax>();
    // ------------------------------------------------------------ softmax: one row per thread
    const int rg = warp, r = threadIdx.x;
    const uint32_t base = tmem + (static_cast<uint32_t>(32 * rg) << 16);
    const float sc = 1.4426950408889634f / sqrtf(static_cast<float>(D));
    int g = 0, items = 0;
    int d_at = -1;  // the finished item's row of O (-1: none) and its sum and reference, until its epilogue
    float d_l = 1.0f, d_m = 0.0f, d_norm = 1.0f;
    bool pending = false;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!wait_all(&sm.item_full[k % kItems], k / kItems)) break;
      const Item& item = sm.item[k % kItems];
      const bool done = !item.valid;
      const int first = item.top, low = item.low, i0 = item.i0;
      // the row's place in O, [T][H] rows; -1 where it holds no token
      const int at = !done && i0 + r >= item.pos0 && i0 + r < item.end ? (item.c0 + i0 + r - item.pos0) * H + item.h : -1;
      // c of the 64 keys of the row's own key tile, one byte each
      const uint4* near = reinterpret_cast<const uint4*>(prm.near + (static_cast<size_t>(item.h) * max_len + (at >= 0 ? i0 + r : 0)) * kKeys);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_empty[k % kItems]);
      float m2 = 0.0f, l = 0.0f, dl = 0.0f;  // dl: what rounding P to bf16 adds to l, in the row's own 32 keys
      MaskT pre = 0, mid = 0;
      for (int u = first; done ? pending : u >= low; --u, ++g) {
        if (!done) {
          const int fs = g & 1, rel = u - (i0 >> 6);
          if (!wait_all(&sm.feat_full[fs], g >> 1)) { ok = false; break; }
          if (u == first) {
            pre = sm.rows[items & 1][r];
            if (rg >= 2) mid = sm.rows[items & 1][r + 64];
          }
          // which 32-key halves hold weight for some row of the warp, and where the counts come from
          const bool own = rel == (rg >> 1);
          uint32_t nc[16];  // its counts
          bool early = false;  // own tile of an odd block: keys with weight in the half before the row's own
          if (own) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              asm volatile("ld.global.ca.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(nc[4 * i]), "=r"(nc[4 * i + 1]), "=r"(nc[4 * i + 2]), "=r"(nc[4 * i + 3]) : "l"(near + i));
          }
          bool live0 = true, live1 = (rg & 1) != 0;  // own tile: the half of the warp's block, and for odd blocks the half before it
          if (rel > 0 && rg < 2) {
            live0 = live1 = false;
          } else if (!own) {
            const MaskT keep = static_cast<MaskT>(FULL & ~((rel == 0 ? mid : pre) | sm.gap[fs]));
            live1 = __any_sync(0xffffffffu, keep != 0);
            live0 = __any_sync(0xffffffffu, static_cast<MaskT>(keep & ~sm.upper[fs]) != 0);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.feat_empty[fs]);
          if (!wait_all(&sm.c_full, g)) { ok = false; break; }
          tc_fence_after();
          // P = 4c 2^(S sc - m) against the reference m, whatever S's maximum is: fp32 and bf16 hold P far beyond what the
          // softmax needs, so m has to be near the maximum only within some 2^60
          float lsum = 0.0f;
          // S and C of both halves into registers at once; S is then free for the next tile's
          uint32_t s0[32], s1[32], c0v[32], c1v[32];
          if (live0) tmem_ld32(base + kColS, s0);
          if (live1) tmem_ld32(base + kColS + 32u, s1);
          if (!own) {
            if (live0) tmem_ld32(base + kColC, c0v);
            if (live1) tmem_ld32(base + kColC + 32u, c1v);
          }
          tmem_wait_ld();
          regs_after_wait(s0);
          regs_after_wait(s1);
          regs_after_wait(c0v);
          regs_after_wait(c1v);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.s_free);
          if (own) {
            early = (rg & 1) && ((nc[0] | nc[1] | nc[2] | nc[3]) | (nc[4] | nc[5] | nc[6] | nc[7])) != 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {  // byte b as the float 2^23 + b, exactly; then 4 (f - 2^23)
              c0v[i] = __float_as_uint(fmaf(4.0f, __uint_as_float(__byte_perm(nc[i >> 2], 0x4B000000u, 0x7540u | (i & 3))), -33554432.0f));
              c1v[i] = __float_as_uint(fmaf(4.0f, __uint_as_float(__byte_perm(nc[8 + (i >> 2)], 0x4B000000u, 0x7540u | (i & 3))), -33554432.0f));
            }
          }
          // one half: P of 32 keys to their place over C, whose reading is done
          auto half = [&](int hf, bool live, const uint32_t (&sv)[32], const uint32_t (&cv)[32]) {
            uint32_t pk[16];
            if (!live) {
#pragma unroll
              for (int i = 0; i < 16; ++i) pk[i] = 0u;
            } else {
              float hsum;
              {
                const uint64_t sc2 = f2_pack(sc, sc), negm2 = f2_pack(-m2, -m2);
                uint64_t ls2[2] = {0ull, 0ull};
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  float x0, x1;
                  f2_unpack(f2_fma(f2_pack(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1])), sc2, negm2), x0, x1);
                  const uint64_t p2 = f2_mul(f2_pack(ex2_approx(x0), ex2_approx(x1)),
                                             f2_pack(__uint_as_float(cv[2 * i]), __uint_as_float(cv[2 * i + 1])));
                  ls2[i & 1] = f2_add(ls2[i & 1], p2);
                  float p0, p1;
                  f2_unpack(p2, p0, p1);
                  pk[i] = pack_bf16x2(p0, p1);
                }
                float a0, a1, b0, b1;
                f2_unpack(ls2[0], a0, a1);
                f2_unpack(ls2[1], b0, b1);
                hsum = (a0 + a1) + (b0 + b1);
              }
              // out of range: a sum too large (or NaN: an infinite exponential of a key without weight), or too small though keys
              // with weight are in it, the own tile's being the first of the row's
              const bool redo = at >= 0 && (!(l + lsum + hsum <= kSumMax) || (own && (hf == (rg & 1) || early) && l + lsum + hsum < kSumMin));
              if (__any_sync(0xffffffffu, redo)) {
                // these rows' reference becomes the maximum so far over keys with weight, rounded up to a whole number, so that
                // everything before follows by an exact power of two (PV(g - 1) has completed: C(g) came after it); the warp's other rows keep their bits
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (__uint_as_float(cv[i]) > 0.0f) top = fmaxf(top, __uint_as_float(sv[i]));
                float alpha = 1.0f;
                if (redo && top != -INFINITY) {
                  const float so_far = l + lsum;
                  const float m_new = ceilf(so_far > 0.0f ? fmaxf(top * sc, m2 + log2f(so_far)) : top * sc);
                  if (so_far > 0.0f) alpha = exp2f(fminf(fmaxf(m2 - m_new, -126.0f), 126.0f));
                  m2 = m_new;
                }
                l *= alpha;
                dl *= alpha;
                lsum *= alpha;
                tmem_wait_st();
                const uint32_t alpha2 = pack_bf16x2(alpha, alpha);
#pragma unroll 1
                for (int q4 = (u != first ? 0 : D / 16); q4 < D / 16 + hf; ++q4) {  // O unless the tile is the first, and P of the half before
                  const bool is_p = q4 == D / 16;
                  const uint32_t at = is_p ? base + kColC : base + kColO + 16u * q4;
                  uint32_t raw[16];
                  tmem_ld16(at, raw);
                  tmem_wait_ld();
                  regs_after_wait(raw);
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    const __nv_bfloat162 p2 = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&raw[e]),
                                                      *reinterpret_cast<const __nv_bfloat162*>(&alpha2));
                    raw[e] = is_p ? *reinterpret_cast<const uint32_t*>(&p2) : __float_as_uint(__uint_as_float(raw[e]) * alpha);
                  }
                  tmem_st16(at, raw);
                }
                float ls[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // summed in the order of the path above
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  float p[2];
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const float c = __uint_as_float(cv[2 * i + e]);
                    p[e] = c > 0.0f ? c * ex2_approx(fmaf(__uint_as_float(sv[2 * i + e]), sc, -m2)) : 0.0f;
                    ls[2 * (i & 1) + e] += p[e];
                  }
                  pk[i] = pack_bf16x2(p[0], p[1]);
                }
                hsum = (ls[0] + ls[1]) + (ls[2] + ls[3]);
              }
              lsum += hsum;
              if (own && hf == (rg & 1)) dl += sum_bf16(pk) - hsum;
            }
            tmem_st16(base + kColC + 16u * hf, pk);
          };
          half(0, live0, s0, c0v);
          half(1, live1, s1, c1v);
          l += lsum;
        }
        auto p_written = [&]() {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_full);
        };
        if (!pending) {
          p_written();
          continue;
        }
        // the finished item, whose last product has run under this tile's exponentials: O / l into registers before
        // this tile's product overwrites it, and from there to memory after P has been handed over
        pending = false;
        if (!wait_all(&sm.o_full, items - 1)) { ok = false; break; }
        tc_fence_after();
        {
          const float inv = 1.0f / d_norm;
          uint32_t o[D / 2];
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t raw[32];
            tmem_ld32(base + kColO + c, raw);
            tmem_wait_ld();
            regs_after_wait(raw);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[c / 2 + i] = pack_bf16x2(__uint_as_float(raw[2 * i]) * inv, __uint_as_float(raw[2 * i + 1]) * inv);
          }
          if (!done) p_written();
          if (d_at >= 0) {
            const bool whole = aligned32(O);
#pragma unroll
            for (int c = 0; c < D; c += 16) store32(O + static_cast<size_t>(d_at) * D + c, o + c / 2, whole);
            row_sum[d_at] = (__log2f(d_l) + d_m - 2.0f) * 0.6931471805599453f - prm.log_s;
          }
          if (kPaged && threadIdx.x == 0) {
            const int x = (items - 1) % (2 * kItems);
            if (sm.missing[x] >= sm.reach[x]) atomicOr(err, PLSH_DEVERR_PAGE);
          }
        }
        if (done) break;
      }
      if (done) break;
      d_at = at;
      d_l = l;
      d_norm = l + dl;
      d_m = m2;
      pending = true;
      ++items;
    }
  } else {
    regs_lower<kRegsRest>();
  if (warp == kWarpItems) {
    // ------------------------------------------------------------ items, a few ahead of their use
    int k = 0;
    bool ok = true;
    // every other round backwards: the items' costs fall along the list, so each block's early ones weigh against its late ones
    for (int round = 0; ok; ++round) {
      const long long x_ = static_cast<long long>(round) * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      if (static_cast<long long>(round) * gridDim.x >= prm.items) break;
      if (x_ >= prm.items) continue;
      const int x = static_cast<int>(x_);
      const int hr = x / prm.slots, slot = x % prm.slots;
      const int h = H <= kMaxSortedHeads ? static_cast<int>(sm.order[hr]) : hr;
      const int mult = prm.sq.start ? 2 : 1;
      const int si = warp_find(prm.sq.cu, prm.sq.S, 7, mult, slot);
      const Seq sq = load_seq(prm.sq, si);
      const int tile = (sq.pos0 >> 7) + slot - ((prm.sq.cu[si] >> 7) + mult * si);
      const int end = sq.pos0 + sq.len, i0 = kRows * tile;
      if (tile < 0 || sq.len <= prm.few || i0 >= end) continue;
      int lo = prm.spans[(static_cast<size_t>(h) * T128 + tile) * 2];
      if (lo < 0 || lo > i0) {
        if (lane == 0) atomicOr(err, PLSH_DEVERR_WINDOW);
        lo = i0;
      }
      // a tile that begins before the new tokens: its first row's window begins between this tile's own and the next one's
      int reach = lo, sure = 0;
      if (kPaged && i0 < sq.pos0) {
        sure = tile + 1 < T128 ? prm.spans[(static_cast<size_t>(h) * T128 + tile + 1) * 2] : end;
        reach = min(sure, sq.pos0);
      }
      const int at = k % kItems;
      if (k >= kItems && !wait_all(&sm.item_empty[at], k / kItems + 1)) { ok = false; break; }
      if (lane == 0) {
        sm.item[at] = Item{1, h, i0, sq.c0, sq.pos0, end, si, min((i0 + kRows - 1) >> 6, (end - 1) >> 6), lo >> 6,
                           sq.c0 - sq.pos0 + (prm.kv_pad ? (si + 1) * prm.kv_pad - kKeys : 0), reach, sure};
        mbar_arrive(&sm.item_full[at]);
      }
      ++k;
      __syncwarp();
    }
    if (ok) {  // the end marker
      const int at = k % kItems;
      if (k < kItems || wait_all(&sm.item_empty[at], k / kItems + 1)) {
        if (lane == 0) {
          sm.item[at].valid = 0;
          mbar_arrive(&sm.item_full[at]);
        }
      }
    }
  } else if (warp == kWarpLoad) {
    // ------------------------------------------------------------ Q and the K/V tiles
    if (lane == 0) {
      tma_prefetch_desc(&tmap_q);
      tma_prefetch_desc(&tmap_k);
      tma_prefetch_desc(&tmap_v);
      int n = 0, nv = 0, loads = 0;  // K, V and Q tiles so far
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!wait(&sm.item_full[k % kItems], k / kItems)) break;
        const Item it = sm.item[k % kItems];
        mbar_arrive(&sm.item_empty[k % kItems]);
        if (!it.valid) break;
        const int kvh = it.h / (H / prm.H_kv);
        // A tile of K or V: one box, or one for each page that it touches. Behind the sequence's end, and where the table names no page of
        // the pool, a box outside the tensor: zeros. The item's last position without a page is noted, and is an error if the item's rows
        // reach it, which the warp of the counts' operands finds out as it goes down the tiles (the epilogue compares).
        int missing = -1;
        auto load_tile = [&](uint8_t* dst, const CUtensorMap* map, int swap, int u, uint64_t* bar) {
          if constexpr (kPaged) {
            const int rows = min(kKeys, 1 << prm.pg.lg_page);
#pragma unroll 1
            for (int r = 0; r < kKeys; r += rows) {
              const int p = kKeys * u + r, page = p < it.end ? find_page(prm.pg, it.s, p) : -1;
              if (page < 0 && p < it.end) missing = max(missing, min(p + rows, it.end) - 1);
              const int plane = page < 0 ? -1 : page * prm.H_kv + kvh;
#pragma unroll 1
              for (int c = 0; c < D / 64; ++c)
                tma_load_3d(dst + c * (kKeys * 128) + r * 128, map, 64 * c, p & ((1 << prm.pg.lg_page) - 1), plane, bar);
            }
          } else {
            const int t = it.kv0 + kKeys * u;
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(dst + c * (kKeys * 128), map, 64 * c, swap ? t : kvh, swap ? kvh : t, bar);
          }
        };
        for (int u = it.top; u >= it.low; --u, ++n) {
          const int st = n % kStages;
          if (n >= kStages && !wait(&sm.k_empty[st], n / kStages + 1)) { ok = false; break; }
          mbar_arrive_expect_tx(&sm.k_full[st], Smem::kKBytes);
          load_tile(sm.k[st], &tmap_k, prm.k_swap, u, &sm.k_full[st]);
          if (kPaged) sm.missing[k % (2 * kItems)] = missing;  // read once the item's last V has been used
          if (u == it.top) {
            if (loads && !wait(&sm.q_empty, loads + 1)) { ok = false; ++n; break; }
            const int tq = it.c0 - it.pos0 + it.i0;
            mbar_arrive_expect_tx(&sm.q_full, Smem::kQBytes);
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(sm.q + c * (kRows * 128), &tmap_q, 64 * c, prm.q_swap ? tq : it.h, prm.q_swap ? it.h : tq, &sm.q_full);
            ++loads;
          }
          const int sv = n % kVStages;
          if (n >= kVStages && !wait(&sm.v_empty[sv], n / kVStages + 1)) { ok = false; ++n; break; }
          mbar_arrive_expect_tx(&sm.v_full[sv], Smem::kKBytes);
          load_tile(sm.v[sv], &tmap_v, prm.v_swap, u, &sm.v_full[sv]);
          nv = n + 1;
        }
      }
      if (*abort_flag) {
        // let every copy already issued land before the block can exit
        for (int i = max(0, n - kStages); i < n; ++i) mbar_wait_drain(&sm.k_full[i % kStages], (i / kStages) & 1, kDrainNs);
        for (int i = max(0, nv - kVStages); i < nv; ++i) mbar_wait_drain(&sm.v_full[i % kVStages], (i / kVStages) & 1, kDrainNs);
        if (loads) mbar_wait_drain(&sm.q_full, (loads + 1) & 1, kDrainNs);
      }
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMAs
    // The whole warp walks the tiles, one elected lane issues: descriptors and addresses then stay in uniform
    // registers, where the instructions take them from.
    const bool elected = elect_one();
    constexpr uint32_t idesc_qk = idesc_bf16_f32(kRows, kKeys, 0);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(kRows, D, 1);
    constexpr uint32_t idesc_c = idesc_e4m3_f32(kRows, kKeys);
    const uint64_t q_desc = smem_desc_sw128(smem_u32(sm.q), 16, 1024);
    const uint64_t k_desc = smem_desc_sw128(smem_u32(sm.k[0]), 16, 1024);
    const uint64_t v_desc = smem_desc_sw128(smem_u32(sm.v[0]), kKeys * 128, 1024);
    const uint64_t a_desc = smem_desc_plain(smem_u32(sm.a), kFeatGroup);
    const uint64_t b_desc = smem_desc_plain(smem_u32(sm.b[0]), kFeatGroup);
    constexpr bool kEarlyS = kVStages > 1;
    int n = 0, items = 0;   // tiles and items so far
    bool pend_first = false, pend_last = false;
    bool ok = !prm.withhold_mma;
    for (int k = 0; ok; ++k) {
      if (!wait_all(&sm.item_full[k % kItems], k / kItems)) { ok = false; break; }
      const Item& item = sm.item[k % kItems];
      const bool done = uniform(item.valid) == 0;
      const int top = uniform(item.top), low = uniform(item.low), row_tile = uniform(item.i0 >> 6);
      if (lane == 0) mbar_arrive(&sm.item_empty[k % kItems]);
      for (int u = top; done || u >= low; --u, ++n) {
        const int st = n % kStages, sv = (n - 1) % kVStages, fs = n & 1;
        // S(g), as soon as its operands are there and S(g - 1) has been read; then PV(g - 1), when P(g - 1) is there; then C(g), which goes
        // where P(g - 1) lies (the upper diagonal tile has none). Every wait but P's passes while the softmax works.
        auto issue_s = [&]() {
          tc_fence_after();
          const uint64_t kd = k_desc + static_cast<uint64_t>((st * Smem::kKBytes) >> 4);
          if (elected) {
#pragma unroll
            for (uint32_t kk = 0; kk < D / 16; ++kk)
              mma_ss(tmem + kColS, q_desc + (kk >> 2) * (kRows * 8) + (kk & 3) * 2, kd + (kk >> 2) * (kKeys * 8) + (kk & 3) * 2,
                     idesc_qk, kk > 0 ? 1u : 0u);
            mma_commit(&sm.k_empty[st]);
            if (u == low) mma_commit(&sm.q_empty);
          }
          __syncwarp();
        };
        // V(g - 1); Q (an item's first tile), K, the counts' operands, S(g - 1) read: one place for five waits. With one
        // place for V, V(g) comes after PV(g - 1), and the operands of a tile with cleared rows after V(g): S(g) then waits its turn.
        const int from = n > 0 ? 0 : 1, to = done ? 1 : kEarlyS ? (n > 0 ? 5 : 4) : 3;
#pragma unroll 1
        for (int i = from; ok && i < to; ++i) {
          if (i == 1 && u != top) continue;
          ok = wait_all(i == 0 ? &sm.v_full[sv] : i == 1 ? &sm.q_full : i == 2 ? &sm.k_full[st] : i == 3 ? &sm.feat_full[fs] : &sm.s_free,
                        i == 0 ? (n - 1) / kVStages : i == 1 ? items : i == 2 ? n / kStages : i == 3 ? n >> 1 : n - 1);
        }
        if (!ok) break;
        if (kEarlyS && !done) issue_s();
        if (n > 0) {
          ok = wait_all(&sm.p_full, n - 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = v_desc + static_cast<uint64_t>((sv * Smem::kKBytes) >> 4);
          if (elected) {
#pragma unroll
            for (uint32_t kk = 0; kk < kKeys / 16; ++kk)
              mma_ts(tmem + kColO, tmem + kColC + 8u * kk, vd + 128u * kk, idesc_pv, (!pend_first || kk > 0) ? 1u : 0u);
            mma_commit(&sm.v_empty[sv]);
            if (pend_last) mma_commit(&sm.o_full);
          }
          __syncwarp();
        }
        if (done) break;
        if (!kEarlyS) {
          ok = wait_all(&sm.feat_full[fs], n >> 1);
          if (!ok) break;
          issue_s();
        }
        const int rel = u - row_tile;  // 1: keys 64..127 of the row tile, 0: keys 0..63, < 0: before it
        const uint64_t ad = a_desc + static_cast<uint64_t>((rel == 0 ? kRows / 2 * kFeat : 0) >> 4);
        const uint64_t bd = b_desc + static_cast<uint64_t>((fs * (kKeys * kFeat)) >> 4);
        if (elected) {
          if (rel <= 0) {
#pragma unroll
            for (int c = 0; c < kFeat / 32; ++c) mma_f8(tmem + kColC, ad + 16u * c, bd + 16u * c, idesc_c, c > 0 ? 1u : 0u);
          }
          mma_commit(&sm.feat_empty[fs]);
          mma_commit(&sm.c_full);
        }
        __syncwarp();
        pend_first = u == top;
        pend_last = u == low;
      }
      if (done) break;
      ++items;
    }
    if (elected) {
      mma_commit(&sm.drain);  // every MMA issued so far completes before it arrives
      mbar_wait_drain(&sm.drain, 0, kDrainNs);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ the counts' operands
    int g = 0, items = 0, last_product = -1;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      if (!wait_all(&sm.item_full[k % kItems], k / kItems)) break;
      const Item& item = sm.item[k % kItems];
      const int valid = item.valid, first = item.top, low = item.low, end = item.end, i0 = item.i0, h = item.h;
      const int p0 = max(i0, item.pos0), sure = item.sure;  // p0: the first row
      int reach = item.reach;
      const MaskT* bm = bmask + static_cast<size_t>(h) * max_len;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_empty[k % kItems]);
      if (!valid) break;
      auto mask_at = [&](int p) { return p < max_len ? bm[p] : FULL; };
      // the rows' near counts into this SM's cache: the softmax comes for them with the diagonal tiles
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int p = i0 + 64 * q + 2 * lane;  // 128 bytes: two rows
        uint32_t x;
        if (p < end)
          asm volatile("ld.global.ca.u32 %0, [%1];" : "=r"(x) : "l"(prm.near + (static_cast<size_t>(h) * max_len + p) * kKeys));
      }
      MaskT rv[4], nx[2];  // masks of rows 32 q + lane, and of the first key tile
#pragma unroll
      for (int q = 0; q < 4; ++q) rv[q] = mask_at(i0 + 32 * q + lane);
#pragma unroll
      for (int q = 0; q < 2; ++q) nx[q] = mask_at(kKeys * first + 32 * q + lane);
      // published with the item's first tile; the item before last, which had this place, has been read once tile g - 2 has
      if (g >= 2 && !wait_all(&sm.feat_empty[g & 1], (g >> 1) + 1)) { ok = false; break; }
      const int rb = items & 1;
      MaskT* rows = sm.rows[rb];
#pragma unroll
      for (int q = 0; q < 4; ++q) rows[32 * q + lane] = rv[q];
      MaskT before = 0, before_mid = 0;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        const MaskT in = tiles::warp_prefix_or<MaskT>(rows[32 * q + lane], lane);
        const MaskT tot = __shfl_sync(0xffffffffu, in, 31);
        rows[32 * q + lane] = static_cast<MaskT>(before | in);
        before = static_cast<MaskT>(before | tot);
        if (q >= 2) {
          rows[64 + 32 * q + lane] = static_cast<MaskT>(before_mid | in);
          before_mid = tot;
        }
      }
      bool built = false;
      MaskT gap = 0;
      for (int u = first; ok && u >= low; --u, ++g) {
        const MaskT kv[2] = {nx[0], nx[1]};
        if (u > low) {
#pragma unroll
          for (int q = 0; q < 2; ++q) nx[q] = mask_at(kKeys * (u - 1) + 32 * q + lane);
        }
        const int rel = u - (i0 >> 6), fs = g & 1;
        if (g >= 2 && !wait_all(&sm.feat_empty[fs], (g >> 1) + 1)) { ok = false; break; }
        // keys: OR after the key, up to the tile's last
        const MaskT s1 = tiles::warp_suffix_or<MaskT>(kv[1], lane), s0 = tiles::warp_suffix_or<MaskT>(kv[0], lane);
        const MaskT t1 = __shfl_sync(0xffffffffu, s1, 0), t0 = __shfl_sync(0xffffffffu, s0, 0);
        MaskT a1 = __shfl_down_sync(0xffffffffu, s1, 1), a0 = __shfl_down_sync(0xffffffffu, s0, 1);
        if (lane == 31) a1 = a0 = 0;
        if (rel <= 0) {
          if (!built) {  // the rows' operands: the product before this one, the previous item's last, has read them
            built = true;
            if (last_product >= 0 && !wait_all(&sm.feat_empty[last_product & 1], last_product >> 1)) { ok = false; break; }
#pragma unroll 1
            for (int r = lane; r < kRows + kRows / 2; r += 32) put_bits<MaskT>(sm.a, r, static_cast<MaskT>(FULL & ~rows[r]));
          }
#pragma unroll 1
          for (int q = 0; q < 2; ++q)
            put_bits<MaskT>(sm.b[fs], 32 * q + lane, static_cast<MaskT>(FULL & ~((q ? a1 : static_cast<MaskT>(a0 | t1)) | gap)));
        }
        if (lane == 0) {
          sm.gap[fs] = gap;
          sm.upper[fs] = t1;
        }
        // rows past the end: another sequence's, or nothing at all. From pages, also rows of pages before the one of the lowest key
        // that the first row reaches (no later row reaches further): they are no longer the sequence's own.
        int own = 0;
        if constexpr (kPaged) {
          const int up = p0 - kKeys * u;  // the first row's place, if it lies in this tile
          if (kKeys * u < sure && up >= 0) {
            __syncwarp();
            // OR after the key up to the tile's end, and from there to the first row
            MaskT b0 = static_cast<MaskT>(a0 | t1), b1 = a1, between = 0;
            if (up >= kKeys) {
              between = rel < 0 ? static_cast<MaskT>(gap | rows[p0 - i0]) : rows[64 + p0 - i0];
            } else {  // only boundaries up to the first row
              b1 = tiles::warp_suffix_or<MaskT>(32 + lane <= up ? kv[1] : static_cast<MaskT>(0), lane);
              b0 = tiles::warp_suffix_or<MaskT>(lane <= up ? kv[0] : static_cast<MaskT>(0), lane);
              const MaskT u1 = __shfl_sync(0xffffffffu, b1, 0);
              b1 = __shfl_down_sync(0xffffffffu, b1, 1);
              b0 = __shfl_down_sync(0xffffffffu, b0, 1);
              if (lane == 31) b1 = b0 = 0;
              b0 = static_cast<MaskT>(b0 | u1);
            }
            const uint32_t n0 = __ballot_sync(0xffffffffu, static_cast<MaskT>(FULL & ~(b0 | between)) != 0);
            const uint32_t n1 = __ballot_sync(0xffffffffu, static_cast<MaskT>(FULL & ~(b1 | between)) != 0);
            if (n0 | n1) reach = min(reach, kKeys * u + (n0 ? __ffs(n0) - 1 : 31 + __ffs(n1)));
          }
          own = min(kKeys, max(0, (reach >> prm.pg.lg_page << prm.pg.lg_page) - kKeys * u));
          if (lane == 0) sm.reach[k % (2 * kItems)] = reach;
        }
        if (rel < 0) gap = static_cast<MaskT>(gap | t0 | t1);
        if (own > 0 || kKeys * (u + 1) > end) {
          const int st = g % kStages, sv = g % kVStages;
          if (!wait_all(&sm.k_full[st], g / kStages) || !wait_all(&sm.v_full[sv], g / kVStages)) { ok = false; break; }
          const int past = min(kKeys, end - kKeys * u);
#pragma unroll 1
          for (int e = lane; e < (own + kKeys - past) * (D / 8); e += 32) {
            const int r_ = e / (D / 8), r = r_ < own ? r_ : r_ - own + past, c = e % (D / 8);
            const int at = (c >> 3) * (kKeys * 128) + r * 128 + (c & 7) * 16;
            *reinterpret_cast<uint4*>(sm.k[st] + at) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(sm.v[sv] + at) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.feat_full[fs]);
      }
      last_product = g - 1;
      ++items;
    }
  }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) atomicOr(err, PLSH_DEVERR_TIMEOUT);
  if (warp == kWarpMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- host side

// Rows of D bf16 of a packed tensor [T][heads][D]: boxes of 64 columns x `rows` tokens of one head, 128-byte swizzle.
// Rows past T read as zero. `swap` says whether the token is the second coordinate (the smaller stride).
int make_rows_map(CUtensorMap* map, const void* p, RowStrides st, int T, int heads, int D, int rows, int* swap) {
  auto enc = tiles::get_encode_fn();
  if (!enc) return fail(PLSH_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  *swap = st.token < st.head ? 1 : 0;
  const cuuint64_t tok = static_cast<cuuint64_t>(st.token) * 2, hd = static_cast<cuuint64_t>(st.head) * 2;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(*swap ? T : heads),
                        static_cast<cuuint64_t>(*swap ? heads : T)};
  cuuint64_t strides[2] = {*swap ? tok : hd, *swap ? hd : tok};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(*swap ? rows : 1), static_cast<cuuint32_t>(*swap ? 1 : rows)};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PLSH_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return PLSH_OK;
}

// Pages [planes][rows][D] of bf16: boxes of 64 columns x up to 64 rows of one plane, 128-byte swizzle.
int make_pages_map(CUtensorMap* map, const void* p, int rows, long long planes, int D) {
  auto enc = tiles::get_encode_fn();
  if (!enc) return fail(PLSH_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(planes)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(rows) * D * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(rows < kKeys ? rows : kKeys), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PLSH_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return PLSH_OK;
}

// The e4m3 rows that the tile kernel's sequences need, as bf16 (exact), in front of their new tokens: row
// c0 + (s + 1) kv_pad - 64 + p - pos0 of [rows][H_kv][D] holds position p of sequence s. A block takes 64 positions of one
// KV head, from the window of its widest head on.
// What no head of the group reaches is none of the sequence's any more, whatever the table says: its pages' rows are zeros.
template <int D>
__global__ void __launch_bounds__(256) gather_kernel(SeqArgs sq, PageArgs pg, const int32_t* __restrict__ spans,
                                                     const double* __restrict__ table, int H, int s, int few, int kv_pad,
                                                     __nv_bfloat16* __restrict__ K, __nv_bfloat16* __restrict__ V,
                                                     uint32_t* __restrict__ err) {
  const int kvh = blockIdx.y, G = H / pg.H_kv, k = kv_pad / kKeys + 2;
  const int si = warp_find(sq.cu, sq.S, 6, k, blockIdx.x);
  const Seq q = load_seq(sq, si);
  if (q.len <= few) return;
  const int u = (q.pos0 >> 6) - kv_pad / kKeys + static_cast<int>(blockIdx.x) - ((sq.cu[si] >> 6) + k * si);
  const int end = q.pos0 + q.len;
  const int T128 = (sq.max_len + PLSH_TILE - 1) / PLSH_TILE, tile = q.pos0 >> 7, next = min(tile + 1, T128 - 1);
  int lo = q.pos0, sure = q.pos0;  // the group's window begins between these, and at lo where a row tile begins with pos0
  for (int h = 0; h < G; ++h) {
    const int32_t* span = spans + static_cast<size_t>(kvh * G + h) * T128 * 2;
    lo = min(lo, span[2 * tile]);
    sure = min(sure, span[2 * next]);
  }
  lo = max(lo, max(0, q.pos0 - (kv_pad - kKeys)));
  if (u < (lo >> 6) || kKeys * u >= end) return;
  // Rows from the page of the window's first key on are the sequence's. The last blocks of a window look for that key (1.4 us of
  // the launch's 14.6 for 8 chunks of 512 tokens after 0 to 15,000, 32/8 heads, d 128).
  int own = lo;
  if (q.pos0 % PLSH_TILE != 0 && (kKeys * u < sure || next == tile)) {
    __shared__ int first;
    if (threadIdx.x == 0) first = q.pos0;
    __syncthreads();
    for (int e = threadIdx.x; e < G * s; e += 256)
      atomicMin(&first, block_begin(Binning::from_table(table + (static_cast<size_t>(kvh) * G * s + e) * 2), q.pos0));
    __syncthreads();
    own = first;
  }
  own = own >> pg.lg_page << pg.lg_page;
  constexpr int kPer = D / 16;  // 16-byte pieces of a row
  const long long out0 = q.c0 + static_cast<long long>(si + 1) * kv_pad - kKeys - q.pos0;
  for (int e = threadIdx.x; e < kKeys * kPer; e += 256) {
    const int p = kKeys * u + e / kPer, c = e % kPer;
    if (p >= end) break;
    const long long row = p >= own ? page_row(pg, si, p, kvh, err) : -1;
    __nv_bfloat16* out[2] = {K + ((out0 + p) * pg.H_kv + kvh) * D + 16 * c, V + ((out0 + p) * pg.H_kv + kvh) * D + 16 * c};
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint4 w = make_uint4(0, 0, 0, 0);
      float sc = 0.0f;
      if (row >= 0) {
        w = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(kv ? pg.v : pg.k) + row * D) + c);
        sc = pow2((kv ? pg.v_exp : pg.k_exp)[row]);
      }
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f[4];
        e4m3_to_float4(ws[i], f);
        o[2 * i] = pack_bf16x2(f[0] * sc, f[1] * sc);
        o[2 * i + 1] = pack_bf16x2(f[2] * sc, f[3] * sc);
      }
      store32(out[kv], o, aligned32(out[kv]));
    }
  }
}

template <int D, typename MaskT, bool kPaged>
int launch(const ServeArgs& a, cudaStream_t st) {
  CUtensorMap mq, mk, mv;
  TcParams prm{};
  if (int rc = make_rows_map(&mq, a.Q, a.qs, a.sq.T, a.H, D, kRows, &prm.q_swap)) return rc;
  if (kPaged) {
    const long long planes = static_cast<long long>(a.pg.num_pages) * a.H_kv;
    if (int rc = make_pages_map(&mk, a.pg.k, 1 << a.pg.lg_page, planes, D)) return rc;
    if (int rc = make_pages_map(&mv, a.pg.v, 1 << a.pg.lg_page, planes, D)) return rc;
  } else {
    if (int rc = make_rows_map(&mk, a.K, a.ks, a.kv_rows, a.H_kv, D, kKeys, &prm.k_swap)) return rc;
    if (int rc = make_rows_map(&mv, a.V, a.vs, a.kv_rows, a.H_kv, D, kKeys, &prm.v_swap)) return rc;
  }
  prm.few = a.few;
  prm.kv_pad = a.kv_pad;
  prm.pg = a.pg;
  prm.sq = a.sq;
  prm.H = a.H;
  prm.H_kv = a.H_kv;
  prm.s = a.s;
  prm.slots = (a.sq.T >> 7) + (a.sq.start ? 2 : 1) * a.sq.S;
  if (static_cast<long long>(prm.slots) * a.H > 0x7fffffffLL) return fail(PLSH_ERR_RANGE, "too many row tiles");
  prm.items = prm.slots * a.H;
  prm.spans = a.spans;
  prm.near = a.near;
  prm.wait_limit = static_cast<uint32_t>(wait_limit_ns() >> 20) + 1;  // rounded up: a wait never ends before the limit
  prm.log_s = std::log(static_cast<float>(a.s));
  prm.withhold_mma = withhold_mma() ? 1 : 0;
  auto kern = serve_tc_kernel<D, MaskT, kPaged>;
  constexpr size_t smem = sizeof(TcSmem<D, MaskT>) + 1024;
  static_assert(smem <= 115712, "shared memory of two blocks on an SM");
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(serve_tc_kernel)");
  const int grid = prm.items < 2 * tiles::sm_count() ? prm.items : 2 * tiles::sm_count();
  kern<<<grid, kThreads, smem, st>>>(mq, mk, mv, prm, static_cast<const MaskT*>(a.bmask), static_cast<__nv_bfloat16*>(a.O),
                                     a.row_sum, a.err);
  e = cudaGetLastError();
  return e == cudaSuccess ? PLSH_OK : cuda_fail(e, "serve_tc_kernel launch");
}

}  // namespace

int launch_near(const void* bmask, int H, int s, int n, uint8_t* near, cudaStream_t st) {
  const dim3 grid(ceil_div(n, 256), H);
  if (s <= 32) near_kernel<uint32_t><<<grid, 256, 0, st>>>(static_cast<const uint32_t*>(bmask), s, n, near);
  else near_kernel<unsigned long long><<<grid, 256, 0, st>>>(static_cast<const unsigned long long*>(bmask), s, n, near);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PLSH_OK : cuda_fail(e, "near_kernel launch");
}

namespace {

template <bool kPaged>
int launch_types(const ServeArgs& a, cudaStream_t st) {
  if (a.d == 128) return a.s <= 32 ? launch<128, uint32_t, kPaged>(a, st) : launch<128, unsigned long long, kPaged>(a, st);
  return a.s <= 32 ? launch<64, uint32_t, kPaged>(a, st) : launch<64, unsigned long long, kPaged>(a, st);
}

}  // namespace

// Rows that a sequence's window may take before its new tokens, in whole key tiles (a row tile's window reaches up to 127 keys
// further down than a row's own), and a tile's slack at either end.
int serve_kv_pad(int max_window) { return ceil_div(max_window + 2 * PLSH_TILE, kKeys) * kKeys; }

// Sequences whose rows the scratch holds at a time. Their lengths are on the device, so each has room for the longest window; a call with
// more sequences than fit kScratchBytes runs in groups, one after another in the same scratch.
constexpr size_t kScratchBytes = size_t{2} << 30;
int serve_group(int S, int H_kv, int d, int kv_pad) {
  const size_t fit = kScratchBytes / (static_cast<size_t>(kv_pad) * H_kv * d * 4);
  return fit < 1 ? 1 : fit < static_cast<size_t>(S) ? static_cast<int>(fit) : S;
}

size_t serve_scratch_bytes(int T, int S, int H_kv, int d, int max_window) {
  const int kv_pad = serve_kv_pad(max_window);
  return 2 * (static_cast<size_t>(T) + static_cast<size_t>(serve_group(S, H_kv, d, kv_pad)) * kv_pad) * H_kv * d * 2;
}

int launch_serve_tc(const ServeArgs& a, cudaStream_t st) {
  if (!a.paged) {
    ServeArgs b = a;
    b.kv_rows = a.sq.T;
    return launch_types<false>(b, st);
  }
  if (!a.pg.k_exp) return launch_types<true>(a, st);
  // e4m3 pages: the rows in reach as bf16 in the caller's scratch, then as if they were packed
  ServeArgs b = a;
  b.kv_pad = serve_kv_pad(a.max_window);
  const int group = serve_group(a.sq.S, a.H_kv, a.d, b.kv_pad);
  const long long rows = static_cast<long long>(a.sq.T) + static_cast<long long>(group) * b.kv_pad;
  const long long slots = (a.sq.T >> 6) + static_cast<long long>(group) * (b.kv_pad / kKeys + 2);
  if (rows > 0x7fffffffLL || slots > 0x7fffffffLL) return fail(PLSH_ERR_RANGE, "plsh_paged_fwd: too many cached rows in reach");
  b.kv_rows = static_cast<int>(rows);
  __nv_bfloat16* k = static_cast<__nv_bfloat16*>(a.scratch);
  __nv_bfloat16* v = k + rows * a.H_kv * a.d;
  b.K = k;
  b.V = v;
  b.ks = b.vs = {static_cast<long long>(a.H_kv) * a.d, a.d};
  const dim3 grid(static_cast<unsigned>(slots), a.H_kv);
  for (int s = 0; s < a.sq.S; s += group) {
    b.sq.cu = a.sq.cu + s;
    b.sq.start = a.sq.start + s;
    b.sq.S = a.sq.S - s < group ? a.sq.S - s : group;
    b.pg.table = a.pg.table + static_cast<long long>(s) * a.pg.width;
    if (a.d == 128) gather_kernel<128><<<grid, 256, 0, st>>>(b.sq, b.pg, a.spans, a.table, a.H, a.s, a.few, b.kv_pad, k, v, a.err);
    else gather_kernel<64><<<grid, 256, 0, st>>>(b.sq, b.pg, a.spans, a.table, a.H, a.s, a.few, b.kv_pad, k, v, a.err);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "gather_kernel launch");
    if (int rc = launch_types<false>(b, st)) return rc;
  }
  return PLSH_OK;
}

}  // namespace plsh
