// Absorbed MLA decode over the 8-bit latent cache.
//
// The cache holds e4m3 codes c_j (512 latent values, then 64 rope values) and a
// scale s_j for each block of rows, so key row j is s_j c_j.  With u = w_uk[h] q
// (512 values, then q's 64 rope values) the scores are
//   t_j = scale * s_j * (u . c_j),      out = w_uv[h] sum_j p_j s_j c_j,
// p = softmax(t): the scale of a row is one factor on its score and one on its
// weight, so the tensor cores contract the codes as they are stored.
//
// Both contractions run as e4m3 x e4m3 MMAs with the keys as the M side:
//   S^T = C U^T   M = 128 keys,            N = query rows, K = 576
//   O^T = C^T P^T M = 128 latent columns,  N = query rows, K = 128 keys
// The second reads the same shared-memory tile as the first, MN-major.  A few
// heads then make a small N instead of an M padded to 128, and the fp32 result
// of up to 64 query rows (4 x 64 TMEM columns) fits beside two score buffers.
// u and p are not e4m3 values: each is split into two e4m3 terms,
//   x = e4m3(x) + e4m3(x - e4m3(x)),
// whose sum is within 2^-8 of x (a bf16 rounding's bound; 0.4 of its mean
// error), and each MMA is done once for either term.  That costs what one bf16
// MMA would and needs no widening of the cache in shared memory.
//
// Three launches:
//   1. q8_query_kernel   u = w_uk[h] q per head (tcgen05, bf16), a power-of-two
//      scale for each row, and the two terms: q8 [T*H][hi 576 | lo 576].
//   2. q8_attn_kernel    one CTA per (sequence, row tile, key partition).
//   3. q8_out_kernel     merges the partitions by LSE and multiplies by w_uv[h]
//      (tcgen05, the latent result as two bf16 terms).
#include <algorithm>
#include <mutex>

#include "kernels.cuh"

namespace mla {
namespace {

constexpr float kLn2q = 0.693147180559945309f;
constexpr float kInf = __builtin_huge_valf();

// x as two e4m3 terms, for a pair of values given as packed f16: the codes of
// the rounded values and of what that rounding left (the difference is exact).
__device__ __forceinline__ uint16_t e4m3x2_from_f16x2(uint32_t v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// ============================================================ 1. queries
// One cluster of four CTAs per (128 tokens, head): CTA r computes latent
// columns [128 r, 128 r + 128) of u for the head's 128 rows; CTA 3 also takes
// the rope part.  The largest value of a row (over all four CTAs, exchanged
// through distributed shared memory) sets its scale.  Reads w_uk once (16 MB
// at 128 heads): memory-bound.
constexpr int kQThreads = 192;
constexpr int Q_TILE = 128 * 128;                 // 128 rows of 64 bf16
constexpr int Q_SMEM_BAR = 4 * Q_TILE;            // two 64-column blocks of A and of B
constexpr int Q_SMEM_TOTAL = Q_SMEM_BAR + 1024 + 1024;

struct QuerySmem {
  uint64_t full[2], done;
  uint32_t tmem;
  int abort;
  float amax[128];
};

__global__ void __cluster_dims__(1, 4, 1) __launch_bounds__(kQThreads, 1)
    q8_query_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map,
                    const uint16_t* __restrict__ q, uint8_t* __restrict__ q8, float* __restrict__ q_scale, int T,
                    int H, int32_t* status) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  QuerySmem* sh = reinterpret_cast<QuerySmem*>(smem + Q_SMEM_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int h = blockIdx.y >> 2;
  const int m0 = blockIdx.x * 128;
  pdl_enter();
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&sh->full[0]), 1);
    mbar_init(smem_u32(&sh->full[1]), 1);
    mbar_init(smem_u32(&sh->done), 1);
    sh->abort = timed_out_before(status) ? 1 : 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh->tmem), 128);
    tmem_relinquish();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const bool work = !cluster_any(&sh->abort);
  const uint32_t tmem = sh->tmem;
  volatile int* abort_flag = &sh->abort;
  const int row = (warp & 3) * 32 + lane;          // epilogue warps 2..5
  const int t = m0 + row;
  const long long grow = static_cast<long long>(t) * H + h;
  uint32_t xb[128];                                // the row's 128 results, as bits
  float am = 0.f;
  bool ok = work;
  if (work && warp == 0) {
    if (elect_one()) {
      for (int kb = 0; kb < 2; ++kb) {
        const uint32_t full = smem_u32(&sh->full[kb]);
        const uint32_t a = smem_u32(smem + kb * 2 * Q_TILE);
        mbar_expect_tx(full, 2 * Q_TILE);
        tma_load_2d(a, &a_map, full, h * 192 + kb * 64, m0);
        tma_load_2d(a + Q_TILE, &b_map, full, kb * 64, h * 512 + rank * 128);
      }
      volatile int never = 0;
      mbar_wait(smem_u32(&sh->full[0]), 0, status, &never);
      mbar_wait(smem_u32(&sh->full[1]), 0, status, &never);
    }
    __syncwarp();
  } else if (work && warp == 1) {
    if (elect_one()) {
      bool good = true;
      for (int kb = 0; kb < 2 && good; ++kb) {
        if (!(good = mbar_wait(smem_u32(&sh->full[kb]), 0, status, abort_flag))) break;
        tc_fence_after();
        const uint32_t a = smem_u32(smem + kb * 2 * Q_TILE);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f16_ss(tmem, sdesc(a + k * 32, 16, 1024), sdesc(a + Q_TILE + k * 32, 16, 1024),
                     idesc_bf16(128, 128, false, false), (kb | k) != 0);
      }
      tc_commit(smem_u32(&sh->done));
      volatile int never = 0;
      mbar_wait(smem_u32(&sh->done), 0, status, &never);
    }
    __syncwarp();
  } else if (work) {
    ok = mbar_wait_warp(smem_u32(&sh->done), 0, status, abort_flag);
    if (ok) {
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 4; ++c)
        tmem_ld32(tmem + (uint32_t((warp & 3) * 32) << 16) + c * 32, *reinterpret_cast<uint32_t(*)[32]>(xb + 32 * c));
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 128; ++i) am = fmaxf(am, fabsf(__uint_as_float(xb[i])));
      if (rank == 3 && t < T) {
        const uint4* rp = reinterpret_cast<const uint4*>(q + grow * 192 + 128);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 v = __ldg(rp + i);
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) am = fmaxf(am, fmaxf(fabsf(bf16_lo(u[k])), fabsf(bf16_hi(u[k]))));
        }
      }
      sh->amax[row] = am;
    }
  }
  tc_fence_before();
  cluster_sync();
  if (warp >= 2 && ok && t < T) {
    for (uint32_t r = 0; r < 4; ++r) {
      if (static_cast<int>(r) == rank) continue;
      float o;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(o) : "r"(cluster_addr(smem_u32(&sh->amax[row]), r)) : "memory");
      am = fmaxf(am, o);
    }
    const float s = pow2_scale(am);
    const float inv = 1.0f / s;
    // An infinite query has no scale: its scores become NaN.
    if (rank == 0) q_scale[grow] = am < kInf ? s : __int_as_float(0x7fc00000);
    uint8_t* dst = q8 + grow * 1152 + rank * 128;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float v[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) v[y] = __uint_as_float(xb[16 * i + 4 * k + y]);
        // |v| inv <= 448; the remainder in fp32, so that f16 rounds only it.
        const uint16_t h0 = pack_e4m3(v[0] * inv, v[1] * inv), h1 = pack_e4m3(v[2] * inv, v[3] * inv);
        const float2 b0 = f16x2_to_float2(e4m3x2_to_f16x2(h0)), b1 = f16x2_to_float2(e4m3x2_to_f16x2(h1));
        hi[k] = static_cast<uint32_t>(h0) | (static_cast<uint32_t>(h1) << 16);
        lo[k] = static_cast<uint32_t>(pack_e4m3(v[0] * inv - b0.x, v[1] * inv - b0.y)) |
                (static_cast<uint32_t>(pack_e4m3(v[2] * inv - b1.x, v[3] * inv - b1.y)) << 16);
      }
      reinterpret_cast<uint4*>(dst)[i] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      reinterpret_cast<uint4*>(dst + 576)[i] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    if (rank == 3) {
      const uint4* rp = reinterpret_cast<const uint4*>(q + grow * 192 + 128);
      uint32_t* dr = reinterpret_cast<uint32_t*>(q8 + grow * 1152 + 512);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 v = __ldg(rp + i);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const float a0 = bf16_lo(u[k]) * inv, a1 = bf16_hi(u[k]) * inv;
          const float a2 = bf16_lo(u[k + 1]) * inv, a3 = bf16_hi(u[k + 1]) * inv;
          const uint16_t h0 = pack_e4m3(a0, a1), h1 = pack_e4m3(a2, a3);
          const float2 b0 = f16x2_to_float2(e4m3x2_to_f16x2(h0)), b1 = f16x2_to_float2(e4m3x2_to_f16x2(h1));
          dr[2 * i + k / 2] = static_cast<uint32_t>(h0) | (static_cast<uint32_t>(h1) << 16);
          dr[144 + 2 * i + k / 2] = static_cast<uint32_t>(pack_e4m3(a0 - b0.x, a1 - b0.y)) |
                                    (static_cast<uint32_t>(pack_e4m3(a2 - b1.x, a3 - b1.y)) << 16);
        }
      }
    }
  }
  cluster_sync();   // no CTA leaves while another may read its row maxima
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  }
}

// ============================================================ 2. attention
constexpr int BK = 128;                     // keys of a tile
constexpr int SLOT = BK * 128;              // one 128-column latent block of a tile, 16 KB
constexpr int ROPE = BK * 64;               // its rope part, 8 KB
constexpr float kShift = 5.0f;              // weights are kept around 2^5 of e4m3's 448
constexpr float kGrow = 8.0f;               // and may grow to 2^8 before the reference moves
constexpr uint32_t TM_S = 0, TM_O = 128;    // TMEM: scores 2 x 64 columns, O^T 4 x 64
constexpr uint32_t TM_COLS = 512;

// WIDE: 64 query rows, the two terms as two MMAs of N = 64.  Narrow: 32 query
// rows, both terms side by side in one MMA of N = 64 (an MMA this small is
// paced by its A operand, so the second term is free), the halves added when
// they are read; the smaller query buffer leaves room for two more key slots.
template <bool WIDE>
struct Shape {
  static constexpr int ROWS = WIDE ? 64 : 32;
  static constexpr int SLOTS = WIDE ? 8 : 10;
  static constexpr int ROPES = WIDE ? 1 : 2;
  static constexpr int QTERM = 4 * 8192 + 4096;           // 64 operand rows x 576
  static constexpr int QBYTES = WIDE ? 2 * QTERM : QTERM;
  static constexpr int PTERM = BK * 64;
  static constexpr int PBYTES = WIDE ? 2 * PTERM : PTERM;
  static constexpr int AT_ROPE = SLOTS * SLOT;
  static constexpr int AT_Q = AT_ROPE + ROPES * ROPE;
  static constexpr int AT_P = AT_Q + QBYTES;
  static constexpr int AT_BAR = AT_P + PBYTES;
  static constexpr int TOTAL = AT_BAR + 1920 + 1024;
  static_assert(TOTAL <= 227 * 1024, "shared memory");
};

struct AttnSmem {
  uint64_t k_full[10], k_empty[10];
  uint64_t r_full[2], r_empty[2];
  uint64_t q_full, s_full[2], s_free[2], p_full, pv_done, drain;
  uint32_t tmem;
  int abort;
  float2 rn[64];       // per query row: factor on the raw score, minus the reference (log2)
  float f[64], d[64];  // a moved reference: factor on what was summed, step of the exponent
  int lim[64];         // keys of the partition that the row sees
};
static_assert(sizeof(AttnSmem) <= 1920, "barrier block");

struct Q8Params {
  const float* q_scale;
  const float* kv_scales;
  const uint8_t* kv_cache;
  const uint32_t* iro;
  const uint32_t* cache_len;
  const int32_t* page_table;
  const int32_t* indices;
  const int32_t* topk;
  __half* o_part;          // [parts][R][512], O / (sum of weights * smax)
  float2* meta;            // [parts][R]: LSE in log2, smax (the partition's largest row scale)
  int indices_stride, num_pages, page_size, max_pages, scale_block;
  int B, H, R, parts, part_keys, m_tiles, max_seq, box;
  float scale_log2;
  int32_t* status;
};

// A sequence's new tokens and keys; false where it is left out (reported once).
struct SeqInfo {
  int qa, n;           // first token, new tokens
  int cb, L;           // cached tokens, keys
};
__device__ __forceinline__ bool q8_seq(const Q8Params& p, int b, SeqInfo& s) {
  const uint32_t qa = p.iro[b], qe = p.iro[b + 1];
  const uint32_t cb = p.cache_len[b];
  if (qe <= qa) return false;
  const uint64_t ctx = static_cast<uint64_t>(cb) + (qe - qa);
  if (static_cast<uint64_t>(qe) * static_cast<uint32_t>(p.H) > static_cast<uint64_t>(p.R) ||
      (p.indices == nullptr && ctx > static_cast<uint64_t>(p.max_seq))) {
    set_status(p.status, MLA_DEV_BAD_OFFSETS);
    return false;
  }
  s.qa = static_cast<int>(qa);
  s.n = static_cast<int>(qe - qa);
  s.cb = p.indices == nullptr ? static_cast<int>(cb) : 0;
  if (p.indices != nullptr) {
    const int k = p.topk != nullptr ? p.topk[b] : p.indices_stride;
    s.L = max(0, min(k, p.indices_stride));
  } else {
    s.L = static_cast<int>(ctx);
  }
  return true;
}
__device__ __forceinline__ int q8_part_count(const Q8Params& p, int L) {
  if (p.part_keys <= 0) return p.parts;
  return max(1, min(p.parts, (L + p.part_keys - 1) / p.part_keys));
}
__device__ __forceinline__ int q8_part_size(int L, int count) {
  const int per = L / count + (L % count != 0);
  return per <= 0x7FFFFF00 ? (per + BK - 1) / BK * BK : 0x7FFFFF00;
}

// Cache row of key `pos` of sequence b, or -1 (reported).
__device__ __forceinline__ int q8_row(const Q8Params& p, int b, int pos) {
  int row = -1;
  if (p.indices != nullptr) {
    row = p.indices[static_cast<long long>(b) * p.indices_stride + pos];
    if (row < 0 || row >= p.num_pages * p.page_size) row = -1;
  } else {
    const int pi = pos / p.page_size;
    const int page = pi < p.max_pages ? p.page_table[static_cast<long long>(b) * p.max_pages + pi] : -1;
    if (page >= 0 && page < p.num_pages) row = page * p.page_size + (pos - pi * p.page_size);
  }
  if (row < 0) set_status(p.status, MLA_DEV_BAD_PAGE);
  return row;
}

// Vote of the four softmax warps: whether any has a weight out of range, and
// whether any wait of theirs failed.  Both are uniform over the 128 threads, so
// that they leave their loop together.
__device__ __forceinline__ void softmax_vote(bool bad, bool fail, bool& any_bad, bool& any_fail) {
  const int lane = threadIdx.x & 31;
  const int mine = lane == 0 ? (bad ? 1 : 0) : (lane <= 5 ? (fail ? 1 : 0) : 0);
  int n;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %1, 0;\n\t"
      "barrier.cta.red.popc.aligned.u32 %0, 1, 128, p;\n\t}"
      : "=r"(n)
      : "r"(mine)
      : "memory");
  any_fail = n >= 5;
  any_bad = n % 5 != 0;
}
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync.aligned 1, 128;" ::: "memory"); }

// Order-preserving integer of a float (for the integer warp maximum) and back.
__device__ __forceinline__ int float_order(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float order_float(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7FFFFFFF)); }

constexpr int kSparseProducers = 2;   // eight warps in all, so that a thread may have 255 registers

// DENSE: a tile's rows come in runs of p.box consecutive rows of one page, each
// a rectangular TMA load.  Otherwise (listed rows, page sizes that are no
// multiple of 8) two warps copy the rows with cp.async.
template <bool DENSE, bool WIDE>
__global__ void __launch_bounds__(DENSE ? 192 : 192 + 32 * kSparseProducers, 1)
    q8_attn_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap qr_map,
                   const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap kr_map,
                   const Q8Params p) {
  using C = Shape<WIDE>;
  constexpr int ROWS = C::ROWS, SLOTS = C::SLOTS, ROPES = C::ROPES;
  constexpr uint32_t IDESC_QK = idesc_e4m3(128, 64, false, false);
  constexpr uint32_t IDESC_PV = idesc_e4m3(128, 64, true, true);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  AttnSmem* sh = reinterpret_cast<AttnSmem*>(smem + C::AT_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t* status = p.status;
  pdl_enter();

  // The item: row tile m of sequence b, key partition k.  Row tiles are
  // neighbours, so that they share their keys in L2.
  const int m = blockIdx.x % p.m_tiles;
  const int b = (blockIdx.x / p.m_tiles) % p.B;
  const int k = blockIdx.x / p.m_tiles / p.B;
  SeqInfo sq;
  if (!q8_seq(p, b, sq)) return;
  const long long rows_b = static_cast<long long>(sq.n) * p.H;
  const long long r0 = static_cast<long long>(m) * ROWS;
  if (r0 >= rows_b) return;
  const int nrows = static_cast<int>(min(static_cast<long long>(ROWS), rows_b - r0));
  const int row0 = static_cast<int>(static_cast<long long>(sq.qa) * p.H + r0);
  const int count = q8_part_count(p, sq.L);
  const int size = q8_part_size(sq.L, count);
  if (k >= count || static_cast<long long>(k) * size >= sq.L) return;
  const int key0 = k * size;
  int key1 = min(sq.L, key0 + size);
  if (p.indices == nullptr) {   // causal: the tile's last token sees keys up to cb + i
    key1 = min(key1, sq.cb + static_cast<int>((r0 + nrows - 1) / p.H) + 1);
    if (key1 <= key0) return;
  }
  const int n = (key1 - key0 + BK - 1) / BK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(smem_u32(&sh->k_full[s]), DENSE ? 1 : kSparseProducers);
      mbar_init(smem_u32(&sh->k_empty[s]), 1);
    }
    for (int s = 0; s < ROPES; ++s) {
      mbar_init(smem_u32(&sh->r_full[s]), DENSE ? 1 : kSparseProducers);
      mbar_init(smem_u32(&sh->r_empty[s]), 1);
    }
    mbar_init(smem_u32(&sh->q_full), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh->s_full[i]), 1);
      mbar_init(smem_u32(&sh->s_free[i]), 4);
    }
    mbar_init(smem_u32(&sh->p_full), 4);
    mbar_init(smem_u32(&sh->pv_done), 1);
    mbar_init(smem_u32(&sh->drain), 1);
    sh->abort = timed_out_before(status) ? 1 : 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh->tmem), TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem;
  volatile int* abort_flag = &sh->abort;

  if (warp == 0) {
    // ------------------------------------------------------------ queries, and the keys' TMA loads
    if (elect_one()) {
      const uint32_t qf = smem_u32(&sh->q_full);
      mbar_expect_tx(qf, C::QBYTES);
#pragma unroll
      for (int term = 0; term < 2; ++term) {
        // Wide: one buffer a term.  Narrow: the terms are rows 0..31 and 32..63 of one.
        const uint32_t base = smem_u32(smem + C::AT_Q + (WIDE ? term * C::QTERM : 0));
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tma_load_2d(base + c * 8192 + (WIDE ? 0 : term * 4096), &q_map, qf, term * 576 + c * 128, row0);
        tma_load_2d(base + 32768 + (WIDE ? 0 : term * 2048), &qr_map, qf, term * 576 + 512, row0);
      }
    }
    __syncwarp();
    uint32_t issued = 0, r_issued = 0;
    if constexpr (DENSE) {
      const int nbox = BK / p.box;
      bool ok = true;
      for (int j = 0; j < n && ok; ++j) {
        const int pos0 = key0 + j * BK;
        const int boxes = min(nbox, (key1 - pos0 + p.box - 1) / p.box);   // runs that hold a key
        int row = 0;
        if (lane < boxes) {
          row = q8_row(p, b, pos0 + lane * p.box);
          if (row < 0) row = p.num_pages * p.page_size;   // past the end: reads zeros
        }
        for (int c = 0; c < 5; ++c) {
          const bool rope = c == 4;
          const uint32_t u = rope ? r_issued : issued;
          const uint32_t cap = rope ? ROPES : SLOTS;
          const uint32_t s = u % cap;
          uint64_t* empty = rope ? &sh->r_empty[s] : &sh->k_empty[s];
          if (u >= cap && !(ok = mbar_wait_warp(smem_u32(empty), ((u / cap) & 1) ^ 1, status, abort_flag))) break;
          const uint32_t full = smem_u32(rope ? &sh->r_full[s] : &sh->k_full[s]);
          const int width = rope ? 64 : 128;
          if (lane == 0) mbar_expect_tx(full, boxes * p.box * width);
          __syncwarp();
          if (lane < boxes) {
            const uint32_t dst = smem_u32(smem + (rope ? C::AT_ROPE + s * ROPE : s * SLOT)) + lane * p.box * width;
            tma_load_2d(dst, rope ? &kr_map : &k_map, full, c * 128, row);
          }
          __syncwarp();
          if (rope) ++r_issued; else ++issued;
        }
      }
      // Every load lands before the CTA leaves.
      volatile int never = 0;
      for (uint32_t s = 0; s < SLOTS; ++s)
        if (issued > s) mbar_wait_warp(smem_u32(&sh->k_full[s]), ((issued - 1 - s) / SLOTS) & 1, status, &never);
      for (uint32_t s = 0; s < ROPES; ++s)
        if (r_issued > s) mbar_wait_warp(smem_u32(&sh->r_full[s]), ((r_issued - 1 - s) / ROPES) & 1, status, &never);
    }
    volatile int never_q = 0;
    mbar_wait_warp(smem_u32(&sh->q_full), 0, status, &never_q);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      const uint32_t q0 = smem_u32(smem + C::AT_Q);
      const uint32_t p0 = smem_u32(smem + C::AT_P);
      auto issue_qk = [&](int j) -> bool {
        const uint32_t sb = j & 1;
        if (j >= 2 && !mbar_wait(smem_u32(&sh->s_free[sb]), ((j >> 1) & 1) ^ 1, status, abort_flag)) return false;
        const uint32_t d = tmem + TM_S + sb * 64;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const uint32_t u = 4 * j + c, s = u % SLOTS;
          if (!mbar_wait(smem_u32(&sh->k_full[s]), (u / SLOTS) & 1, status, abort_flag)) return false;
          tc_fence_after();
          const uint32_t a = smem_u32(smem + s * SLOT);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t ad = sdesc(a + kk * 32, 16, 1024);
            mma_f8_ss(d, ad, sdesc(q0 + c * 8192 + kk * 32, 16, 1024), IDESC_QK, (c | kk) != 0);
            if (WIDE) mma_f8_ss(d, ad, sdesc(q0 + C::QTERM + c * 8192 + kk * 32, 16, 1024), IDESC_QK, 1);
          }
        }
        const uint32_t rs = j % ROPES;
        if (!mbar_wait(smem_u32(&sh->r_full[rs]), (j / ROPES) & 1, status, abort_flag)) return false;
        tc_fence_after();
        const uint32_t a = smem_u32(smem + C::AT_ROPE + rs * ROPE);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          const uint64_t ad = sdesc(a + kk * 32, 16, 512, kSwizzle64);
          mma_f8_ss(d, ad, sdesc(q0 + 32768 + kk * 32, 16, 512, kSwizzle64), IDESC_QK, 1);
          if (WIDE) mma_f8_ss(d, ad, sdesc(q0 + C::QTERM + 32768 + kk * 32, 16, 512, kSwizzle64), IDESC_QK, 1);
        }
        tc_commit(smem_u32(&sh->s_full[sb]));
        tc_commit(smem_u32(&sh->r_empty[rs]));
        return true;
      };
      auto issue_pv = [&](int j) -> bool {
        if (!mbar_wait(smem_u32(&sh->p_full), j & 1, status, abort_flag)) return false;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const uint32_t s = (4 * j + c) % SLOTS;
          const uint32_t a = smem_u32(smem + s * SLOT);
          const uint32_t d = tmem + TM_O + c * 64;
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk) {
            // 32 keys a step: both operands MN-major, groups of 8 keys 1024 (keys) and 512 (weights) bytes apart.
            const uint64_t ad = sdesc(a + kk * 4096, 16, 1024);
            mma_f8_ss(d, ad, sdesc(p0 + kk * 2048, 16, 512, kSwizzle64), IDESC_PV, (j | kk) != 0);
            if (WIDE) mma_f8_ss(d, ad, sdesc(p0 + C::PTERM + kk * 2048, 16, 512, kSwizzle64), IDESC_PV, 1);
          }
          tc_commit(smem_u32(&sh->k_empty[s]));
        }
        tc_commit(smem_u32(&sh->pv_done));
        return true;
      };
      bool ok = mbar_wait(smem_u32(&sh->q_full), 0, status, abort_flag);
      if (ok) ok = issue_qk(0);
      for (int j = 0; j < n && ok; ++j) {
        if (j + 1 < n) ok = issue_qk(j + 1);
        if (ok) ok = issue_pv(j);
      }
      tc_commit(smem_u32(&sh->drain));
      volatile int never = 0;
      mbar_wait(smem_u32(&sh->drain), 0, status, &never);
    }
    __syncwarp();
  } else if (warp < 6) {
    // ------------------------------------------------------------ softmax (thread = key), epilogue
    const int q4 = warp & 3;
    const int key = q4 * 32 + lane;
    const int tid = threadIdx.x - 64;                 // 0..127
    const uint32_t lane_off = uint32_t(q4 * 32) << 16;
    uint8_t* pbuf = smem + C::AT_P;
    if (tid < ROWS) {
      float rf = 0.f;
      int lim = 0;
      if (tid < nrows) {
        rf = p.q_scale[row0 + tid] * p.scale_log2;
        lim = key1 - key0;
        if (p.indices == nullptr) lim = min(lim, sq.cb + static_cast<int>((r0 + tid) / p.H) + 1 - key0);
      }
      sh->rn[tid] = make_float2(rf, 0.f);
      sh->lim[tid] = lim;
    }
    // Keys that every row of the tile sees.
    int all = key1 - key0;
    if (p.indices == nullptr) all = min(all, sq.cb + static_cast<int>(r0 / p.H) + 1 - key0);
    softmax_sync();
    bool seen = false;                                // this thread's row has a reference
    float l[ROWS];
#pragma unroll
    for (int c = 0; c < ROWS; ++c) l[c] = 0.f;
    float smax = 0.f;
    // The scale of this thread's key, one tile ahead.
    auto key_scale = [&](int j) -> float {
      const int pos = key0 + j * BK + key;
      if (j >= n || pos >= key1) return 1.f;
      const int row = q8_row(p, b, pos);
      return row < 0 ? 1.f : __ldg(p.kv_scales + row / p.scale_block);
    };
    float next = key_scale(0);
    bool fail = false;
    for (int j = 0; j < n; ++j) {
      const uint32_t sb = j & 1;
      float ksc = next;
      next = key_scale(j + 1);
      const bool valid = key0 + j * BK + key < key1;
      const bool broken = !(fabsf(ksc) < kInf);       // a scale that is no number: the key's scores are NaN
      if (broken) ksc = 1.f;
      if (valid) smax = fmaxf(smax, fabsf(ksc));
      const float lsc = __log2f(fabsf(ksc));
      float t[ROWS];
      const bool got = mbar_wait_warp(smem_u32(&sh->s_full[sb]), (j >> 1) & 1, status, abort_flag);
      fail |= !got;
      if (got) {
        tc_fence_after();
        uint32_t raw[64];
        tmem_ld32(tmem + lane_off + TM_S + sb * 64, *reinterpret_cast<uint32_t(*)[32]>(raw));
        tmem_ld32(tmem + lane_off + TM_S + sb * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(raw + 32));
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < ROWS; ++c)
          t[c] = WIDE ? __uint_as_float(raw[c]) : __uint_as_float(raw[c]) + __uint_as_float(raw[c + 32]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh->s_free[sb]));
      } else {
#pragma unroll
        for (int c = 0; c < ROWS; ++c) t[c] = 0.f;
      }
      const float xs = broken ? __int_as_float(0x7fc00000) : ksc;
      float mx = -kInf;
      const bool masked = (j + 1) * BK > all;         // some row does not see every key of the tile
#pragma unroll
      for (int c0 = 0; c0 < ROWS; c0 += 16) {
        if (c0 < nrows) {
#pragma unroll
          for (int c = c0; c < c0 + 16; ++c) {
            const float2 rn = sh->rn[c];
            t[c] = fmaf(t[c] * xs, rn.x, rn.y);
            if (masked) t[c] = j * BK + key < sh->lim[c] ? t[c] : -kInf;
            mx = fmaxf(mx, t[c]);
          }
        }
      }
      bool any_bad, any_fail;
      softmax_vote(__any_sync(0xffffffffu, mx + lsc > kGrow), fail, any_bad, any_fail);
      if (any_fail) { fail = true; break; }
      // The weights' buffer (and O, where the reference moves) is free once P V
      // of the tile before is done.
      const bool wait_pv = j > 0;
      if (j == 0 || any_bad) {
        // ---- move the reference of the rows that need it
        if (wait_pv && !mbar_wait_warp(smem_u32(&sh->pv_done), (j - 1) & 1, status, abort_flag)) fail = true;
        tc_fence_after();
        float* wmax = reinterpret_cast<float*>(pbuf);  // [4][ROWS], in the free weights' buffer
#pragma unroll
        for (int c0 = 0; c0 < ROWS; c0 += 32) {
          float mine = -kInf;
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float v = order_float(__reduce_max_sync(0xffffffffu, float_order(fmaxf(t[c0 + c] + lsc, -kInf))));
            if (lane == c) mine = v;
          }
          wmax[q4 * ROWS + c0 + lane] = mine;
        }
        softmax_sync();
        if (tid < ROWS) {
          const float mm = fmaxf(fmaxf(wmax[tid], wmax[ROWS + tid]), fmaxf(wmax[2 * ROWS + tid], wmax[3 * ROWS + tid]));
          float d = 0.f, f = 1.f;
          if (mm > -kInf) {
            if (!seen) {
              d = kShift - mm;
              seen = true;
            } else if (mm > kShift) {
              d = kShift - mm;
              f = ex2(d);
            }
          }
          sh->rn[tid].y += d;
          sh->d[tid] = d;
          sh->f[tid] = f;
        }
        softmax_sync();
#pragma unroll
        for (int c = 0; c < ROWS; ++c) {
          t[c] += sh->d[c];
          l[c] *= sh->f[c];
        }
        if (wait_pv && !fail) {
#pragma unroll 1
          for (int cb = 0; cb < 8; ++cb) {
            uint32_t r[32];
            const uint32_t ta = tmem + lane_off + TM_O + cb * 32;
            tmem_ld32(ta, r);
            tmem_ld_wait();
            const float* f = sh->f + (WIDE ? (cb & 1) * 32 : 0);
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f[i]);
            tmem_st32(ta, r);
          }
          tmem_st_wait();
        }
      } else if (wait_pv && !mbar_wait_warp(smem_u32(&sh->pv_done), (j - 1) & 1, status, abort_flag)) {
        fail = true;
      }
      // ---- weights: two e4m3 terms, key-major rows of 64 bytes (64-byte swizzle)
      uint32_t hi[ROWS / 4], lo[ROWS / 4];
#pragma unroll
      for (int i = 0; i < ROWS / 4; ++i) hi[i] = lo[i] = 0u;
#pragma unroll
      for (int c0 = 0; c0 < ROWS; c0 += 16) {
        if (c0 < nrows) {
#pragma unroll
          for (int c = c0; c < c0 + 16; c += 4) {
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              e[i] = ex2(t[c + i]);
              l[c + i] += e[i];
              e[i] *= ksc;
            }
            const uint32_t a = pack_f16(e[0], e[1]), bb = pack_f16(e[2], e[3]);
            const uint16_t ha = e4m3x2_from_f16x2(a), hb = e4m3x2_from_f16x2(bb);
            const uint16_t la = e4m3x2_from_f16x2(sub_f16x2(a, e4m3x2_to_f16x2(ha)));
            const uint16_t lb = e4m3x2_from_f16x2(sub_f16x2(bb, e4m3x2_to_f16x2(hb)));
            hi[c / 4] = static_cast<uint32_t>(ha) | (static_cast<uint32_t>(hb) << 16);
            lo[c / 4] = static_cast<uint32_t>(la) | (static_cast<uint32_t>(lb) << 16);
          }
        }
      }
      const int sw = (key >> 1) & 3;
      uint8_t* prow = pbuf + key * 64;
      if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          *reinterpret_cast<uint4*>(prow + ((i ^ sw) << 4)) = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
          *reinterpret_cast<uint4*>(prow + C::PTERM + ((i ^ sw) << 4)) = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          *reinterpret_cast<uint4*>(prow + ((i ^ sw) << 4)) = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
          *reinterpret_cast<uint4*>(prow + (((2 + i) ^ sw) << 4)) = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
        }
      }
      if (masked && j * BK + key >= all) {
        // A key that some row does not see: its weight is 0 there, but 0 times
        // a NaN code is NaN.  Rows past the partition become zeros (they may
        // hold anything); in the others every NaN code does (a row that sees
        // such a key has a NaN score, so its result is NaN all the same).
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint4* kr = reinterpret_cast<uint4*>(smem + ((4 * j + c) % SLOTS) * SLOT + key * 128);
          for (int i = 0; i < 8; ++i) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (valid) {
              v = kr[i];
              uint32_t* w = reinterpret_cast<uint32_t*>(&v);
              for (int x = 0; x < 4; ++x) {
                // Bytes equal to 0x7F after clearing the sign.
                const uint32_t nan = ((w[x] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                w[x] &= ~((nan >> 7) * 0xFFu);
              }
            }
            kr[i] = v;
          }
        }
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh->p_full));
    }
    // ------------------------------------------------------------ epilogue
    if (!fail && !mbar_wait_warp(smem_u32(&sh->pv_done), (n - 1) & 1, status, abort_flag)) fail = true;
    tc_fence_after();
    bool any_bad, any_fail;
    softmax_vote(false, fail, any_bad, any_fail);
    if (!any_fail) {
      // Sums over the keys: every thread's, through the key slots (all read by now).
      float* ls = reinterpret_cast<float*>(smem);
#pragma unroll
      for (int c = 0; c < ROWS; ++c) ls[key * ROWS + c] = l[c];
      float* sm = reinterpret_cast<float*>(pbuf);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, d));
      if (lane == 0) sm[q4] = smax;
      softmax_sync();
      if (tid < ROWS) {
        float sum = 0.f;
#pragma unroll 8
        for (int i = 0; i < BK; ++i) sum += ls[i * ROWS + tid];
        float s = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
        if (!(s > 0.f)) s = 1.f;
        sh->f[tid] = sum == 0.f ? 0.f : 1.0f / (sum * s);
        // Weights carry 2^-reference: log2 of the plain sum adds it back.
        if (tid < nrows)
          p.meta[static_cast<long long>(k) * p.R + row0 + tid] =
              make_float2(sum == 0.f ? -kInf : __log2f(sum) - sh->rn[tid].y, s);
      }
      softmax_sync();
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[64];
        tmem_ld32(tmem + lane_off + TM_O + c * 64, *reinterpret_cast<uint32_t(*)[32]>(o));
        tmem_ld32(tmem + lane_off + TM_O + c * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(o + 32));
        tmem_ld_wait();
        __half* dst = p.o_part + (static_cast<long long>(k) * p.R + row0) * 512 + c * 128 + key;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          float v = __uint_as_float(o[r]);
          if constexpr (!WIDE) v += __uint_as_float(o[32 + r]);
          if (r < nrows) dst[static_cast<long long>(r) * 512] = __float2half_rn(sh->f[r] == 0.f ? 0.f : v * sh->f[r]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ listed rows: cp.async
    if constexpr (!DENSE) {
      constexpr int RW = BK / kSparseProducers;       // this warp's keys [RW pw, RW pw + RW) of the tile
      const int pw = warp - 6;
      uint32_t issued = 0, r_issued = 0;
      uint32_t pend[4];                               // full barriers of the copies in flight
      int npend = 0;
      bool ok = true;
      auto landed = [&](uint32_t bar) {
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
      };
      for (int j = 0; j < n && ok; ++j) {
        int row[RW / 32];                             // key 32 x + lane
#pragma unroll
        for (int x = 0; x < RW / 32; ++x) {
          const int pos = key0 + j * BK + pw * RW + 32 * x + lane;
          row[x] = pos < key1 ? q8_row(p, b, pos) : 0;
          if (row[x] < 0) row[x] = 0;                 // reported; the result of its rows is not meaningful
        }
        for (int c = 0; c < 5; ++c) {
          const bool rope = c == 4;
          const uint32_t u = rope ? r_issued : issued;
          const uint32_t cap = rope ? ROPES : SLOTS;
          const uint32_t s = u % cap;
          if (u >= cap) {
            const uint32_t empty = smem_u32(rope ? &sh->r_empty[s] : &sh->k_empty[s]);
            const uint32_t parity = ((u / cap) & 1) ^ 1;
            if (!__all_sync(0xffffffffu, mbar_try_wait(empty, parity))) {
              // About to wait for the MMAs: they may be waiting for these copies.
              cp_async_wait<0>();
              for (int i = 0; i < npend; ++i) landed(pend[i]);
              npend = 0;
              if (!(ok = mbar_wait_warp(empty, parity, status, abort_flag))) break;
            }
          }
          const uint32_t full = smem_u32(rope ? &sh->r_full[s] : &sh->k_full[s]);
          if (!rope) {
            const uint32_t dst = smem_u32(smem + s * SLOT) + pw * RW * 128;
#pragma unroll
            for (int i = 0; i < RW / 4; ++i) {        // four rows of 8 chunks an instruction
              const int r = 4 * i + (lane >> 3), ch = lane & 7;
              const int src = __shfl_sync(0xffffffffu, row[i / 8], r & 31);
              cp_async16(dst + r * 128 + ((ch ^ (r & 7)) << 4), p.kv_cache + static_cast<size_t>(src) * 576 + c * 128 + ch * 16);
            }
          } else {
            const uint32_t dst = smem_u32(smem + C::AT_ROPE + s * ROPE) + pw * RW * 64;
#pragma unroll
            for (int i = 0; i < RW / 8; ++i) {        // eight rows of 4 chunks
              const int r = 8 * i + (lane >> 2), ch = lane & 3;
              const int src = __shfl_sync(0xffffffffu, row[i / 4], r & 31);
              cp_async16(dst + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4), p.kv_cache + static_cast<size_t>(src) * 576 + 512 + ch * 16);
            }
          }
          cp_async_commit();
          if (npend == 3) {
            cp_async_wait<3>();
            landed(pend[0]);
            pend[0] = pend[1];
            pend[1] = pend[2];
            pend[2] = full;
          } else {
            pend[npend++] = full;
          }
          if (rope) ++r_issued; else ++issued;
        }
      }
      cp_async_wait<0>();
      for (int i = 0; i < npend; ++i) landed(pend[i]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
}

// ============================================================ 3. merge and w_uv
// One CTA per (head, NT tokens): the partitions' latent results are merged by
// LSE in fp32 (with the attention sink in the denominator), split into two
// bf16 terms (their sum within 2^-16) and multiplied by w_uv[h]: D^T [128
// values, NT tokens] = w_uv[h] [128, 512] . o^T, so that few tokens make a
// small N.  Reads w_uv[h] once per token tile.
constexpr int kOutThreads = 256;

template <int NT>
struct OutShape {
  static constexpr int W = 8 * 16384;                // w_uv[h], eight 64-column blocks
  static constexpr int TERM = 8 * NT * 128;
  static constexpr int AT_O = W;
  static constexpr int AT_BAR = AT_O + 2 * TERM;
  static constexpr int TOTAL = AT_BAR + 1024 + 1024;
};
struct OutSmem {
  uint64_t full, done;
  uint32_t tmem;
  int abort;
  int used[32];      // partitions that hold keys of the token; -1: its rows are not written
  float sink[32];    // log2 units
};

template <int NT>
__global__ void __launch_bounds__(kOutThreads, 1)
    q8_out_kernel(const __grid_constant__ CUtensorMap w_map, const Q8Params p, const float* __restrict__ sink,
                  __nv_bfloat16* __restrict__ out, float* __restrict__ lse, int T) {
  using C = OutShape<NT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  OutSmem* sh = reinterpret_cast<OutSmem*>(smem + C::AT_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * NT, h = blockIdx.y;
  pdl_enter();
  if (timed_out_before(p.status)) return;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&sh->full), 1);
    mbar_init(smem_u32(&sh->done), 1);
    sh->abort = 0;
    fence_mbar_init();
    const uint32_t full = smem_u32(&sh->full);
    mbar_expect_tx(full, C::W);
    for (int kb = 0; kb < 8; ++kb) tma_load_2d(smem_u32(smem + kb * 16384), &w_map, full, kb * 64, h * 128);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh->tmem), 32);
    tmem_relinquish();
  }
  if (threadIdx.x >= 64 && threadIdx.x < 64 + NT) {
    const int i = threadIdx.x - 64, t = t0 + i;
    int used = -1;
    float sk = -kInf;
    if (t < T) {
      int lo = 0, hi = p.B;   // largest b with iro[b] <= t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.iro + mid) <= static_cast<uint32_t>(t)) lo = mid; else hi = mid;
      }
      SeqInfo s;
      if (q8_seq(p, lo, s) && s.qa <= t && t < s.qa + s.n) {
        const int count = q8_part_count(p, s.L);
        const int size = q8_part_size(s.L, count);
        const int keys = p.indices != nullptr ? s.L : min(s.L, s.cb + (t - s.qa) + 1);
        used = size > 0 ? min(count, keys / size + (keys % size != 0)) : 0;
        if (sink != nullptr) sk = __ldg(sink + lo) * 1.4426950408889634f;
      }
    }
    sh->used[i] = used;
    sh->sink[i] = sk;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem;

  for (int i = warp; i < NT; i += kOutThreads / 32) {
    const int used = sh->used[i];
    const long long grow = static_cast<long long>(t0 + i) * p.H + h;
    float o[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = 0.f;
    float mx = -kInf, tot = 0.f;
    constexpr int KU = 4;                           // partitions loaded together
    for (int k0 = 0; k0 < used; k0 += KU) {
      uint4 a[KU], c[KU];
      float2 mt[KU];
#pragma unroll
      for (int x = 0; x < KU; ++x) {
        const long long at = static_cast<long long>(k0 + x) * p.R + grow;
        const bool in = k0 + x < used;
        mt[x] = in ? __ldg(p.meta + at) : make_float2(-kInf, 0.f);
        const uint4* src = reinterpret_cast<const uint4*>(p.o_part + at * 512);
        a[x] = in ? __ldg(src + lane) : make_uint4(0u, 0u, 0u, 0u);
        c[x] = in ? __ldg(src + 32 + lane) : make_uint4(0u, 0u, 0u, 0u);
      }
      float nm = mx;
#pragma unroll
      for (int x = 0; x < KU; ++x) nm = fmaxf(nm, mt[x].x);
      const float keep = mx == -kInf ? 0.f : ex2(mx - nm);
      tot *= keep;
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] *= keep;
#pragma unroll
      for (int x = 0; x < KU; ++x) {
        const float w = mt[x].x == -kInf ? 0.f : ex2(mt[x].x - nm);
        tot += w;
        const float ws = w * mt[x].y;
        const uint32_t u[8] = {a[x].x, a[x].y, a[x].z, a[x].w, c[x].x, c[x].y, c[x].z, c[x].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 v = f16x2_to_float2(u[e]);
          o[2 * e] = fmaf(ws, v.x, o[2 * e]);
          o[2 * e + 1] = fmaf(ws, v.y, o[2 * e + 1]);
        }
      }
      mx = nm;
    }
    float l2 = tot == 0.f ? -kInf : mx + __log2f(tot);
    float w = tot == 0.f ? 0.f : 1.0f / tot;
    const float sk = sh->sink[i];
    if (sink != nullptr && used >= 0) {
      // The sink is one more logit without a value: LSE' = log(e^LSE + e^sink).
      const float top = fmaxf(l2, sk);
      if (top > -kInf) {
        const float both = ex2(l2 - top) + ex2(sk - top);
        const float l3 = top + __log2f(both);
        w *= l2 == -kInf ? 0.f : ex2(l2 - top) / both;
        l2 = l3;
      }
    }
    if (lse != nullptr && used >= 0 && lane == 0) lse[grow] = l2 * kLn2q;
    // Latents 8 lane .. +7 and 256 + 8 lane .. +7: block 64 columns, 16-byte chunk lane & 7.
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = o[8 * half + 2 * e] * w, y = o[8 * half + 2 * e + 1] * w;
        hi[e] = pack_bf16(x, y);
        lo[e] = pack_bf16(x - bf16_lo(hi[e]), y - bf16_hi(hi[e]));
      }
      const int kb = half * 4 + (lane >> 3);
      uint8_t* dst = smem + C::AT_O + kb * NT * 128 + i * 128 + (((lane & 7) ^ (i & 7)) << 4);
      *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(dst + C::TERM) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
  fence_async_smem();
  __syncthreads();
  volatile int never = 0;
  if (warp == 0) {
    if (elect_one()) {
      if (mbar_wait(smem_u32(&sh->full), 0, p.status, &never)) {
        tc_fence_after();
        for (int kb = 0; kb < 8; ++kb) {
          const uint32_t a = smem_u32(smem + kb * 16384);
          const uint32_t o = smem_u32(smem + C::AT_O + kb * NT * 128);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t ad = sdesc(a + kk * 32, 16, 1024);
            mma_f16_ss(tmem, ad, sdesc(o + kk * 32, 16, 1024), idesc_bf16(128, NT, false, false), (kb | kk) != 0);
            mma_f16_ss(tmem, ad, sdesc(o + C::TERM + kk * 32, 16, 1024), idesc_bf16(128, NT, false, false), 1);
          }
        }
      } else {
        sh->abort = 1;
      }
      tc_commit(smem_u32(&sh->done));
    }
    __syncwarp();
  }
  const bool ok = mbar_wait_warp(smem_u32(&sh->done), 0, p.status, &never);
  tc_fence_after();
  if (warp < 4 && ok && *reinterpret_cast<volatile int*>(&sh->abort) == 0) {
    uint32_t r[32];
    tmem_ld32(tmem + (uint32_t(warp * 32) << 16), r);   // 32 columns are allocated; NT of them used
    tmem_ld_wait();
    __nv_bfloat16* dst = out + (static_cast<long long>(t0) * p.H + h) * 128 + warp * 32 + lane;
#pragma unroll
    for (int i = 0; i < NT; ++i)
      if (sh->used[i] >= 0) dst[static_cast<long long>(i) * p.H * 128] = __float2bfloat16_rn(__uint_as_float(r[i]));
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 32);
  }
}

template <typename K>
cudaError_t opt_in_smem(K kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// Largest power of two, at most 128, that divides the page size.
int run_rows(int page_size) {
  int g = 1;
  while (g < BK && page_size % (2 * g) == 0) g *= 2;
  return g;
}

template <bool DENSE, bool WIDE>
cudaError_t launch_attn(const CUtensorMap& q_map, const CUtensorMap& qr_map, const CUtensorMap& k_map,
                        const CUtensorMap& kr_map, const Q8Params& p, long long items, cudaStream_t stream) {
  cudaError_t e = opt_in_smem(q8_attn_kernel<DENSE, WIDE>, Shape<WIDE>::TOTAL);
  if (e != cudaSuccess) return e;
  const int threads = DENSE ? 192 : 192 + 32 * kSparseProducers;
  return launch_pdl(q8_attn_kernel<DENSE, WIDE>, dim3(static_cast<unsigned>(items)), dim3(threads),
                    Shape<WIDE>::TOTAL, stream, q_map, qr_map, k_map, kr_map, p);
}

template <int NT>
cudaError_t launch_out(const CUtensorMap& w_map, const Q8Params& p, const DecodeQ8Args& a, cudaStream_t stream) {
  cudaError_t e = opt_in_smem(q8_out_kernel<NT>, OutShape<NT>::TOTAL);
  if (e != cudaSuccess) return e;
  return launch_pdl(q8_out_kernel<NT>, dim3((a.T + NT - 1) / NT, a.H), dim3(kOutThreads), OutShape<NT>::TOTAL, stream,
                    w_map, p, a.sink, static_cast<__nv_bfloat16*>(a.out), a.lse, a.T);
}

// 64 query rows a tile where a sequence can fill more than 32.
bool wide_rows(int H, int max_new) { return static_cast<long long>(H) * max_new > 32; }

}  // namespace

DecodeQ8Layout decode_q8_layout(int T, int H, int parts) {
  const size_t R = static_cast<size_t>(T) * H;
  DecodeQ8Layout L;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  L.q8 = take(R * 1152);
  L.q_scale = take(R * 4);
  L.o_part = take(static_cast<size_t>(parts) * R * 512 * 2);
  L.meta = take(static_cast<size_t>(parts) * R * 8);
  L.total = off;
  return L;
}

DecodePartitioning decode_q8_partitioning(int B, int H, int max_new, int max_keys) {
  const long long sms = sm_count();
  const int rows = wide_rows(H, max_new) ? 64 : 32;
  const long long m_tiles = (static_cast<long long>(std::max(1, max_new)) * H + rows - 1) / rows;
  const long long keys = std::max(1, max_keys);
  long long pk = static_cast<long long>(B) * m_tiles * keys / sms;
  pk = std::min<long long>(4096, std::max<long long>(256, (pk + BK - 1) / BK * BK));
  DecodePartitioning d;
  d.part_keys = static_cast<int>(pk);
  d.parts = static_cast<int>(std::min<long long>(256, std::max(1ll, (keys + pk - 1) / pk)));
  return d;
}

cudaError_t launch_decode_q8(const DecodeQ8Args& a, cudaStream_t stream) {
  const int H = a.H, T = a.T;
  const long long R = static_cast<long long>(T) * H;
  if (T == 0) return cudaSuccess;
  const DecodeQ8Layout L = decode_q8_layout(T, H, a.parts);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  uint8_t* q8 = ws + L.q8;
  float* q_scale = reinterpret_cast<float*>(ws + L.q_scale);
  const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const bool wide = wide_rows(H, a.max_new);
  const int rows = wide ? 64 : 32;

  CUtensorMap qa_map, wuk_map;
  if (!encode_2d(&qa_map, a.q, bf, static_cast<uint64_t>(H) * 192, T, static_cast<uint64_t>(H) * 384, 64, 128,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&wuk_map, a.w_uk, bf, 128, static_cast<uint64_t>(H) * 512, 256, 64, 128,
                 CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  cudaError_t e = opt_in_smem(q8_query_kernel, Q_SMEM_TOTAL);
  if (e != cudaSuccess) return e;
  e = launch_pdl(q8_query_kernel, dim3((T + 127) / 128, 4 * H), dim3(kQThreads), Q_SMEM_TOTAL, stream, qa_map, wuk_map,
                 static_cast<const uint16_t*>(a.q), q8, q_scale, T, H, a.status);
  if (e != cudaSuccess) return e;

  Q8Params p;
  p.q_scale = q_scale;
  p.kv_scales = a.kv_scales;
  p.kv_cache = static_cast<const uint8_t*>(a.kv_cache);
  p.iro = a.iro;
  p.cache_len = a.cache_len;
  p.page_table = a.page_table;
  p.indices = a.indices;
  p.topk = a.topk;
  p.o_part = reinterpret_cast<__half*>(ws + L.o_part);
  p.meta = reinterpret_cast<float2*>(ws + L.meta);
  p.indices_stride = a.indices_stride;
  p.num_pages = a.num_pages;
  p.page_size = a.page_size;
  p.max_pages = a.max_pages;
  p.scale_block = a.scale_block;
  p.B = a.B;
  p.H = H;
  p.R = static_cast<int>(R);
  p.parts = a.parts;
  p.part_keys = a.part_keys;
  p.m_tiles = static_cast<int>((static_cast<long long>(a.max_new) * H + rows - 1) / rows);
  p.max_seq = a.max_seq;
  p.box = run_rows(a.page_size);
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.status = a.status;
  const bool dense = a.indices == nullptr && p.box >= 8;
  const uint64_t cache_rows = static_cast<uint64_t>(a.num_pages) * a.page_size;
  const uint32_t box = dense ? p.box : 8;
  CUtensorMap q_map, qr_map, k_map, kr_map;
  if (!encode_2d(&q_map, q8, u8, 1152, R, 1152, 128, rows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&qr_map, q8, u8, 1152, R, 1152, 64, rows, CU_TENSOR_MAP_SWIZZLE_64B) ||
      !encode_2d(&k_map, a.kv_cache, u8, 576, cache_rows, 576, 128, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&kr_map, a.kv_cache, u8, 576, cache_rows, 576, 64, box, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  const long long items = static_cast<long long>(a.B) * a.parts * p.m_tiles;
  if (dense)
    e = wide ? launch_attn<true, true>(q_map, qr_map, k_map, kr_map, p, items, stream)
             : launch_attn<true, false>(q_map, qr_map, k_map, kr_map, p, items, stream);
  else
    e = wide ? launch_attn<false, true>(q_map, qr_map, k_map, kr_map, p, items, stream)
             : launch_attn<false, false>(q_map, qr_map, k_map, kr_map, p, items, stream);
  if (e != cudaSuccess) return e;

  CUtensorMap wuv_map;
  if (!encode_2d(&wuv_map, a.w_uv, bf, 512, static_cast<uint64_t>(H) * 128, 1024, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  return T > 16 ? launch_out<32>(wuv_map, p, a, stream) : launch_out<16>(wuv_map, p, a, stream);
}

}  // namespace mla
