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
// u and p are not e4m3 values: each is split into two 8-bit terms,
//   x = e4m3(x) + (x - e4m3(x)),
// and each MMA is done once for either term.  That costs what one bf16 MMA
// would and needs no widening of the cache in shared memory.  The second term of
// p is e4m3 times 2^5 where the terms have accumulators of their own (0.4 of a
// bf16 rounding's mean error), and e5m2 where they share one (0.75 of it); the
// sum is within 2^-8 of x, a bf16 rounding's bound, as long as x is not far below
// the window's top: 2^8 to 2^8.75 for p, whose error is at least 2^-15 (2^-14, or
// 1/8 of x) there.  A row's reference therefore follows its keys both ways: it
// moves when a tile's largest weight leaves 2^-3 .. 2^8 (2^-2 .. 2^8.75), so that
// an error is at most 2^-12 of the largest weight among the tile's 128 keys or
// 2^-8 of the weight.  A key far above all others costs only its own tile's keys
// bits, and is put at the window's top, which leaves them most: with 500 keys 14
// nats below one without value the result is 0.6 % off.  (64 sequences of 128 heads: 287 us, against 278 with
// references that only rise; 330 and 308 where scores spread by 2 nats, not 1.)  The
// denominator sums the weights before they are split: the terms' errors have
// either sign, so that their sum's is relatively no larger, and the LSE has none.
//
// Three launches:
//   1. q8_query_kernel   u = w_uk[h] q per head (tcgen05, bf16), a power-of-two
//      scale for each row, and the two terms: q8 [T*H][hi 576 | lo 576].  A CTA
//      of its own writes the plan: the batch's work as one line of units.
//   2. q8_attn_kernel    one CTA per piece of that line (and row tile).
//   3. q8_out_kernel     merges the pieces' results by LSE and multiplies by
//      w_uv[h] (tcgen05, the latent result as two bf16 terms).
//
// The line: a sequence with n new tokens and L keys has ceil(n H / rows) row
// tiles; `members` of them (a token's heads) make an item, and each item is
// ceil(L / 128) units, one 128-key tile each.  The line of all items' units is
// cut into `pieces` equal parts whatever the sequences' lengths, so every SM
// gets the same number of tiles; the members of a piece walk it at the same
// time on neighbouring CTAs and share its keys in L2.  A piece that ends inside
// an item leaves a partial result in the slot (piece + item), which no other
// (piece, item) pair has.
#include <algorithm>
#include <type_traits>

#include "kernels.cuh"

namespace mla {
namespace {

constexpr float kLn2q = 0.693147180559945309f;
constexpr float kInf = __builtin_huge_valf();

struct PlanEntry {     // a sequence with work, in batch order
  int b, qa, n, cb;    // sequence, first token, new tokens, cached tokens (0 in the sparse form)
  int L, tiles;        // keys, ceil(L / 128)
  int units, items;    // units and items before it
};
struct PlanHead {
  int entries, units;
};
struct PlanArgs {
  PlanHead* head;
  PlanEntry* entries;
  const uint32_t* iro;
  const uint32_t* cache_len;
  const int32_t* topk;
  int B, H, T, max_seq, indices_stride, sparse, item_rows;   // rows of an item: members * rows of a tile
  int32_t* status;
};
constexpr int BK = 128;                     // keys of a tile

// Position of the last of n ascending numbers, `step` ints apart, that is not
// above x (0 if none): 32 probes of a warp at a time.
__device__ __forceinline__ int last_not_above(const int* at, int step, int n, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
#pragma unroll 1
  for (int hi = n; hi - lo > 1;) {
    const int d = (hi - lo + 31) / 32;
    const long long i = lo + static_cast<long long>(lane) * d;
    const int below = __popc(__ballot_sync(0xffffffffu, i < hi && __ldg(at + i * step) <= x));
    lo += max(below - 1, 0) * d;
    hi = min(hi, lo + d);
  }
  return lo;
}
constexpr int kEntryInts = sizeof(PlanEntry) / 4;

// The plan, by 128 threads (tid) of one CTA: scans over the sequences, 128 at
// a time.  A sequence is left out if it is empty, ends past the call's tokens,
// begins before an earlier one ends, or (dense) is longer than max_seq; all but
// the first are reported.  What is kept is disjoint and ascending, so there are
// at most T entries.  `scr`: 4 x 4 ints.
__device__ void q8_plan(const PlanArgs& a, int tid, int (*scr)[4]) {
  const int warp = tid >> 5, lane = tid & 31;
  int entries = 0, units = 0, items = 0;
  uint32_t reach = 0;                       // end of the last sequence so far
  for (int b0 = 0; b0 < a.B; b0 += 128) {
    const int b = b0 + tid;
    PlanEntry e;
    e.b = b;
    e.n = 0;
    uint32_t qa = 0, qe = 0;
    bool ok = false, some = false;
    int u = 0, it = 0;
    if (b < a.B) {
      qa = __ldg(a.iro + b);
      qe = __ldg(a.iro + b + 1);
      const uint32_t cb = __ldg(a.cache_len + b);
      some = qe != qa;
      if (qe > qa && qe <= static_cast<uint32_t>(a.T)) {
        const uint64_t ctx = static_cast<uint64_t>(cb) + (qe - qa);
        e.qa = static_cast<int>(qa);
        e.n = static_cast<int>(qe - qa);
        e.cb = a.sparse ? 0 : static_cast<int>(cb);
        if (a.sparse) {
          const int k = a.topk != nullptr ? __ldg(a.topk + b) : a.indices_stride;
          e.L = max(0, min(k, a.indices_stride));
          ok = true;
        } else {
          e.L = static_cast<int>(ctx);
          ok = ctx <= static_cast<uint64_t>(a.max_seq);
        }
        e.tiles = (e.L + BK - 1) / BK;
      }
    }
    // Ends of the sequences before this one (of those that may be kept).
    uint32_t end = ok ? qe : 0u;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, end, d);
      if (lane >= d) end = max(end, o);
    }
    uint32_t before = __shfl_up_sync(0xffffffffu, end, 1);
    if (lane == 0) before = 0u;
    if (lane == 31) scr[0][warp] = static_cast<int>(end);
    asm volatile("barrier.cta.sync.aligned 1, 128;" ::: "memory");
    before = max(before, reach);
    for (int w = 0; w < warp; ++w) before = max(before, static_cast<uint32_t>(scr[0][w]));
    if (some && (!ok || qa < before)) set_status(a.status, MLA_DEV_BAD_OFFSETS);
    ok = ok && qa >= before;
    if (ok) {
      it = static_cast<int>((static_cast<long long>(e.n) * a.H + a.item_rows - 1) / a.item_rows);
      u = it * e.tiles;
    }
    int sc = ok ? 1 : 0, su = u, si = it;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sc, d), y = __shfl_up_sync(0xffffffffu, su, d);
      const int z = __shfl_up_sync(0xffffffffu, si, d);
      if (lane >= d) {
        sc += x;
        su += y;
        si += z;
      }
    }
    if (lane == 31) {
      scr[1][warp] = sc;
      scr[2][warp] = su;
      scr[3][warp] = si;
    }
    asm volatile("barrier.cta.sync.aligned 1, 128;" ::: "memory");
    int at = entries + sc - (ok ? 1 : 0);
    e.units = units + su - u;
    e.items = items + si - it;
    for (int w = 0; w < 4; ++w) {
      if (w < warp) {
        at += scr[1][w];
        e.units += scr[2][w];
        e.items += scr[3][w];
      }
      entries += scr[1][w];
      units += scr[2][w];
      items += scr[3][w];
      reach = max(reach, static_cast<uint32_t>(scr[0][w]));
    }
    if (ok) {
      reinterpret_cast<int4*>(a.entries + at)[0] = make_int4(e.b, e.qa, e.n, e.cb);
      reinterpret_cast<int4*>(a.entries + at)[1] = make_int4(e.L, e.tiles, e.units, e.items);
    }
    asm volatile("barrier.cta.sync.aligned 1, 128;" ::: "memory");   // scr is rewritten
  }
  if (tid == 0) {
    a.head->entries = entries;
    a.head->units = units;
    a.entries[entries].units = units;       // where the last entry's units end
  }
}

// ============================================================ 1. queries
// One cluster of two CTAs per (128 tokens, head): CTA r computes latent columns
// [256 r, 256 r + 256) of u for the head's 128 rows; CTA 1 also takes the rope
// part.  The largest value of a row (over both CTAs, exchanged through
// distributed shared memory) sets its scale.  Reads w_uk once (16 MB at 128
// heads).  Two CTAs a head, two on an SM: 128 heads run in one wave (four CTAs a
// head, in two waves, took half as long again); 15 us for 96 tokens, of which
// the operands' loads are a third and the conversion to two terms a quarter.
constexpr int kQThreads = 320;                    // TMA, MMA, 8 epilogue warps
constexpr int Q_A = 128 * 128;                    // 128 rows of 64 bf16
constexpr int Q_B = 256 * 128;
constexpr int Q_SMEM_BAR = 2 * (Q_A + Q_B);       // two 64-column blocks of A and of B; then the results
constexpr int Q_OUT = 128 * 128;                  // 128 rows of 128 bytes: [term][half] of codes, the rope part
constexpr int Q_SMEM_TOTAL = Q_SMEM_BAR + 2048 + 1024;

struct QuerySmem {
  uint64_t full[2], done;
  uint32_t tmem;
  int abort;
  float amax[2][128];        // [half of the CTA's columns][row]
  int scr[4][4];
};

// x in two e4m3 terms, four values.  Rows reach up to 448, where the first term
// is at most 16 off, so the second is kept 16 times as large: what both leave is
// 2^-14 at most where x is small, 2^-21 of the row's largest.
constexpr float kQueryLow = 16.f;
__device__ __forceinline__ void two_terms(const float (&v)[4], uint32_t& hi, uint32_t& lo) {
  const uint16_t h0 = pack_e4m3(v[0], v[1]), h1 = pack_e4m3(v[2], v[3]);
  const float2 b0 = f16x2_to_float2(e4m3x2_to_f16x2(h0)), b1 = f16x2_to_float2(e4m3x2_to_f16x2(h1));
  hi = static_cast<uint32_t>(h0) | (static_cast<uint32_t>(h1) << 16);
  lo = static_cast<uint32_t>(pack_e4m3((v[0] - b0.x) * kQueryLow, (v[1] - b0.y) * kQueryLow)) |
       (static_cast<uint32_t>(pack_e4m3((v[2] - b1.x) * kQueryLow, (v[3] - b1.y) * kQueryLow)) << 16);
}

__global__ void __cluster_dims__(1, 2, 1) __launch_bounds__(kQThreads, 2)
    q8_query_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map,
                    const __grid_constant__ CUtensorMap o_map,
                    const uint16_t* __restrict__ q, uint8_t* __restrict__ q8, float* __restrict__ q_scale, int T,
                    int H, int32_t* status, const PlanArgs plan) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  QuerySmem* sh = reinterpret_cast<QuerySmem*>(smem + Q_SMEM_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int h = static_cast<int>(blockIdx.y >> 1) - 1;
  const int m0 = blockIdx.x * 128;
  if (threadIdx.x == 0 && h >= 0) {                // w_uk on its way while the kernel before ends
    tma_prefetch_2d(&b_map, 0, h * 512 + rank * 256);
    tma_prefetch_2d(&b_map, 64, h * 512 + rank * 256);
  }
  pdl_enter();
  if (h < 0) {                                     // the first clusters: one CTA of them writes the plan
    if (blockIdx.x == 0 && rank == 0 && threadIdx.x < 128 && !timed_out_before(status))
      q8_plan(plan, threadIdx.x, sh->scr);
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&sh->full[0]), 1);
    mbar_init(smem_u32(&sh->full[1]), 1);
    mbar_init(smem_u32(&sh->done), 1);
    sh->abort = timed_out_before(status) ? 1 : 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh->tmem), 256);
    tmem_relinquish();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const bool work = !cluster_any(&sh->abort);
  const uint32_t tmem = sh->tmem;
  volatile int* abort_flag = &sh->abort;
  const int half = (warp - 2) >> 2;                // epilogue warps 2..9: columns [128 half, 128 half + 128)
  const int row = (warp & 3) * 32 + lane;
  const int t = m0 + row;
  const long long grow = static_cast<long long>(t) * H + h;
  const uint32_t tm = tmem + (uint32_t((warp & 3) * 32) << 16) + half * 128;
  float am = 0.f;
  bool ok = work;
  if (work && warp == 0) {
    if (elect_one()) {
#pragma unroll 1
      for (int kb = 0; kb < 2; ++kb) {
        const uint32_t full = smem_u32(&sh->full[kb]);
        const uint32_t a = smem_u32(smem + kb * (Q_A + Q_B));
        mbar_expect_tx(full, Q_A + Q_B);
        tma_load_2d(a, &a_map, full, h * 192 + kb * 64, m0);
        tma_load_2d(a + Q_A, &b_map, full, kb * 64, h * 512 + rank * 256);
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
        const uint32_t a = smem_u32(smem + kb * (Q_A + Q_B));
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f16_ss(tmem, sdesc(a + k * 32, 16, 1024), sdesc(a + Q_A + k * 32, 16, 1024),
                     idesc_bf16(128, 256, false, false), (kb | k) != 0);
      }
      tc_commit(smem_u32(&sh->done));
      volatile int never = 0;
      mbar_wait(smem_u32(&sh->done), 0, status, &never);
    }
    __syncwarp();
  } else if (work) {
    // The rope part is read while the operands load, and kept in shared memory
    // as soon as the MMAs do not need that any more.
    uint4 rv[8];
    if (rank == 1 && half == 1) {
      const uint4* rp = reinterpret_cast<const uint4*>(q + grow * 192 + 128);
#pragma unroll
      for (int i = 0; i < 8; ++i) rv[i] = t < T ? __ldg(rp + i) : make_uint4(0u, 0u, 0u, 0u);
    }
    ok = mbar_wait_warp(smem_u32(&sh->done), 0, status, abort_flag);
    if (ok) {
      tc_fence_after();
      if (rank == 1 && half == 1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t u[4] = {rv[i].x, rv[i].y, rv[i].z, rv[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) am = fmaxf(am, fmaxf(fabsf(bf16_lo(u[k])), fabsf(bf16_hi(u[k]))));
          *reinterpret_cast<uint4*>(smem + 4 * Q_OUT + row * 128 + ((i ^ (row & 7)) << 4)) = rv[i];
        }
      }
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t x[32];
        tmem_ld32(tm + c * 32, x);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) am = fmaxf(am, fabsf(__uint_as_float(x[i])));
      }
      sh->amax[half][row] = am;
    }
  }
  tc_fence_before();
  cluster_sync();
  if (warp >= 2 && ok) {
    am = fmaxf(sh->amax[0][row], sh->amax[1][row]);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float o;
      asm volatile("ld.shared::cluster.f32 %0, [%1];"
                   : "=f"(o)
                   : "r"(cluster_addr(smem_u32(&sh->amax[x][row]), rank ^ 1))
                   : "memory");
      am = fmaxf(am, o);
    }
    const float s = pow2_scale<-120>(am);   // (queries may be as small as keys are large)
    const float inv = 1.0f / s;
    // An infinite query has no scale: its scores become NaN.
    if (rank == 0 && half == 0 && t < T) q_scale[grow] = am < kInf ? s : __int_as_float(0x7fc00000);
    // The results once more from TMEM, 32 columns at a time (few registers, so
    // that two of these CTAs share an SM), and through shared memory (the
    // operands are not needed any more) to a bulk store: a row of the result
    // is H * 1152 bytes on, and 16 bytes of 32 rows at a time took 32 passes.
    uint8_t* dst = smem + half * Q_OUT + row * 128;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t x[32];
      tmem_ld32(tm + c * 32, x);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float v[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) v[y] = __uint_as_float(x[16 * i + 4 * k + y]) * inv;
          two_terms(v, hi[k], lo[k]);
        }
        uint8_t* at = dst + (((2 * c + i) ^ (row & 7)) << 4);
        *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(at + 2 * Q_OUT) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
    fence_async_smem();
    asm volatile("barrier.cta.sync.aligned %0, 128;" ::"r"(1 + half) : "memory");   // the half's four warps
    if (threadIdx.x == 64 + 128 * half) {
#pragma unroll
      for (int term = 0; term < 2; ++term)         // (rows past the last token are clipped)
        tma_store_2d(&o_map, smem_u32(smem + (2 * term + half) * Q_OUT), h * 1152 + term * 576 + rank * 256 + half * 128, m0);
      bulk_commit();
    }
    if (rank == 1 && half == 1 && t < T) {
      uint4* dr = reinterpret_cast<uint4*>(q8 + grow * 1152 + 512);
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint4 v = *reinterpret_cast<const uint4*>(smem + 4 * Q_OUT + row * 128 + (((2 * i + k) ^ (row & 7)) << 4));
          const float a[4] = {bf16_lo(v.x) * inv, bf16_hi(v.x) * inv, bf16_lo(v.y) * inv, bf16_hi(v.y) * inv};
          const float b[4] = {bf16_lo(v.z) * inv, bf16_hi(v.z) * inv, bf16_lo(v.w) * inv, bf16_hi(v.w) * inv};
          two_terms(a, hi[2 * k], lo[2 * k]);
          two_terms(b, hi[2 * k + 1], lo[2 * k + 1]);
        }
        dr[i] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        dr[36 + i] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
    }
    if (threadIdx.x == 64 + 128 * half) bulk_wait<0>();
  }
  cluster_sync();   // no CTA leaves while another may read its row maxima
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ============================================================ 2. attention
// The bounded waits of this kernel: one try (which itself waits for some 2700
// clk) where they stand, the rest out of line.  Inline, the code of a wait that
// runs out lies between the instructions of the loops, which then do not fit
// the instruction cache.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, int32_t* status, volatile int* abort_flag) {
  return mbar_wait(bar, parity, status, abort_flag);
}
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, int32_t* status, volatile int* abort_flag) {
  return mbar_try_wait(bar, parity) || wait_long(bar, parity, status, abort_flag);
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, int32_t* status, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, wait_one(bar, parity, status, abort_flag));
}

// A ring slot holds half of a tile's latent columns (two 128-column blocks) in
// groups of eight keys: [key / 8][block][key % 8][128 bytes], swizzled within
// the 1 KB of each group and block.  One TMA instruction then loads both blocks
// of a whole run of keys (a lone lane needs about 130 clk for an instruction,
// so their number counts), and runs follow each other at the stride of a group.
constexpr int SLOT = BK * 256;              // 32 KB
constexpr int GROUP = 2048;                 // eight keys of a slot
constexpr int ROPE = BK * 64;               // its rope part, 8 KB
constexpr float kAlone = 8.0f;              // how far (log2) a weight that stands alone is above the others
constexpr float kReach = 32.0f;             // how far (log2) a row's reference falls behind its highest

// A tile has 64, 32 or 16 query rows.  The query operand holds both terms,
// the first terms' rows above the second's, so one MMA of N = 128, 64 or 32
// gives both products and the softmax adds them.  The weights' terms: up to 32
// rows lie side by side in one operand and O has two halves, added when it is
// read; for 64 rows that would fill the whole TMEM with O, so there the terms are
// two MMAs of N = 64 on the same accumulator.  (An MMA of M = 128 from shared
// memory takes 40, 48, 64 clk at N = 32, 64, 128, measured: half of it at
// N = 64 is its A operand's 128 bytes a clk.)  The smaller the query buffer, the
// more key slots.
template <int R>
struct Shape {
  static constexpr int ROWS = R;
  static constexpr bool WIDE = R == 64;
  static constexpr int GROUPS = ROWS / 16;                // softmax warpgroups, 16 rows each
  static constexpr int THREADS = 96 + 128 * GROUPS;       // producer, MMA, softmax and scale warps
  static constexpr int NQ = 2 * ROWS;                     // score columns of a tile
  static constexpr int SLOTS = R == 64 ? 4 : (R == 32 ? 5 : 6);
  static constexpr int ROPES = R == 32 ? 2 : 1;
  static constexpr int QBLOCK = NQ * 128;                 // query operand, 128 columns
  static constexpr int QBYTES = NQ * 576;
  static constexpr int NP = WIDE ? 64 : 2 * ROWS;         // columns of a value MMA, bytes of a key's weights
  static constexpr int PTERM = BK * NP;
  // Where a tile's largest weight (log2) may lie before the row's reference
  // moves, and where it is put then: in the first tile, from above and from
  // below (a larger one leaves room for the next, a smaller one is most often
  // the lowest of many).  One that stands alone is put a quarter below HIGH.
  static constexpr float HIGH = WIDE ? 8.75f : 8.0f, LOW = WIDE ? -2.0f : -3.0f;
  static constexpr float FIRST = 5.0f, UP = WIDE ? 7.5f : 7.0f, DOWN = 3.0f;
  // What a second term is multiplied by where it has its own columns of O; in
  // the others it is e5m2, whose steps go down to 2^-16.
  static constexpr float LO = WIDE ? 1.0f : 32.0f;
  static constexpr int PBYTES = WIDE ? 2 * PTERM : PTERM;
  static constexpr int AT_ROPE = SLOTS * SLOT;
  static constexpr int AT_Q = AT_ROPE + ROPES * ROPE;
  static constexpr int AT_P = AT_Q + QBYTES;
  static constexpr int AT_BAR = AT_P + PBYTES;
  static constexpr int TOTAL = AT_BAR + 3 * 1024 + (WIDE ? 0 : 256);
  static constexpr uint32_t TM_S = 0, TM_O = 2 * NQ;      // TMEM: two score buffers, O^T 4 x NP columns
  static constexpr uint32_t TM_COLS = R == 16 ? 256 : 512;
  static_assert(TOTAL <= 227 * 1024 && TM_O + 4 * NP <= TM_COLS, "shared memory, TMEM");
};

template <int SLOTS, int ROPES>
struct AttnSmem {
  uint64_t k_full[SLOTS], k_empty[SLOTS];
  uint64_t r_full[ROPES], r_empty[ROPES];     // rope parts
  uint64_t fixed;                     // a masked tile's values have been cleaned
  uint64_t q_full, q_free, s_full[2], s_free[2], p_full, pv_done, o_free, drain, group[4];
  uint32_t tmem;
  int abort;
  alignas(16) float rf[64];   // per query row: factor on the raw score,
  alignas(16) float ry[64];   // minus the reference (log2 units),
  alignas(16) float f[64];    // when that moves: factor on what was summed,
  alignas(16) float d[64];    // and step of the exponent;
  int top[64];                // largest result of a row (order-preserving integers)
  int lim[64];                // keys of the segment that the row sees
  // [tile & 1][group][warp]: rows without a weight of LOW or more (row r: bit
  // 15 - r), and bit 16 unless there is one above HIGH.
  alignas(16) uint32_t range[2][4][4];
  uint32_t care[4];           // [group]: rows whose reference may fall
  float ksc[2][128];          // [tile & 1]: the keys' scales (1 past the segment)
  int run[32], last[4];      // cache rows of the runs that are loaded next, and of the tile before them
};

struct Q8Params {
  const PlanHead* head;
  const PlanEntry* entries;
  const float* q_scale;
  const float* kv_scales;
  const uint8_t* kv_cache;
  const int32_t* page_table;
  const int32_t* indices;
  __half* o_part;          // [slot][members][rows][512], O times a power of two, largest in [2^14, 2^15)
  float2* meta;            // [slot][members][rows]: LSE in log2, 1 / (that power times the sum of weights)
  int indices_stride, num_pages, max_pages, cache_rows;
  FastDiv page, block;     // page size and scale_block
  int H, R, T, pieces, members, box;
  float scale_log2;
  int32_t* status;
};

__device__ __forceinline__ PlanEntry load_entry(const PlanEntry* e) {
  const int4 x = __ldg(reinterpret_cast<const int4*>(e)), y = __ldg(reinterpret_cast<const int4*>(e) + 1);
  PlanEntry r;
  r.b = x.x; r.qa = x.y; r.n = x.z; r.cb = x.w;
  r.L = y.x; r.tiles = y.y; r.units = y.z; r.items = y.w;
  return r;
}
// First unit of piece g, floor(g units / pieces) (pieces <= 2^15, so that the
// remainders' product has 32 bits), and the piece of unit u.
__device__ __forceinline__ int piece_begin(int g, int pieces, int units) {
  const uint32_t q = static_cast<uint32_t>(units) / pieces, r = static_cast<uint32_t>(units) - q * pieces;
  return static_cast<int>(g * q + g * r / static_cast<uint32_t>(pieces));
}
__device__ __forceinline__ int piece_of(int u, int pieces, int units) {
  return static_cast<int>((static_cast<long long>(u + 1) * pieces - 1) / units);
}

// One item's share of a piece.
struct Segment {
  int b, n;              // sequence, tiles to visit
  int row0, nrows;       // first global query row of this CTA's tile, valid rows
  int r0;                // first row of the tile within the sequence's rows
  int cb;                // cached tokens
  int key0, key1;        // keys (key1 before the tile's causal limit)
  int slot;
};

// The segments of a piece in order.  Every role of the CTA walks them by itself.
struct Walk {
  int u, u1, e, end;      // next unit, the piece's end, entry, where its units end
  PlanEntry pe;
};
__device__ __forceinline__ Walk walk_begin(const Q8Params& p, int piece) {
  Walk w;
  const int entries = __ldg(&p.head->entries), units = __ldg(&p.head->units);
  w.e = 0;
  // No more pieces than units, so that none between two others is empty.
  const int pieces = min(p.pieces, units);
  w.u = w.u1 = 0;
  if (piece >= pieces) return w;
  w.u = piece_begin(piece, pieces, units);
  w.u1 = piece_begin(piece + 1, pieces, units);
  // Last entry with units <= u that has any (a search over ascending numbers;
  // entries without units share the next one's number and come before it).
  const int lo = last_not_above(&p.entries[0].units, kEntryInts, entries, w.u);
  w.e = lo;
  w.pe = load_entry(p.entries + lo);
  w.end = __ldg(&p.entries[lo + 1].units);
  return w;
}
template <int ROWS, bool DENSE>
__device__ __forceinline__ bool walk_next(const Q8Params& p, Walk& w, int member, int piece, Segment& s) {
  while (w.u < w.u1) {
    if (w.u >= w.end) {
      w.pe = load_entry(p.entries + ++w.e);          // units remain, so there is one
      w.end = __ldg(&p.entries[w.e + 1].units);
      continue;
    }
    const int off = w.u - w.pe.units;
    const int item = off / w.pe.tiles, tile = off - item * w.pe.tiles;
    const int len = min(w.pe.tiles - tile, w.u1 - w.u);
    w.u += len;
    const long long rows = static_cast<long long>(w.pe.n) * p.H;
    const long long r0 = (static_cast<long long>(item) * p.members + member) * ROWS;
    if (r0 >= rows) continue;
    s.b = w.pe.b;
    s.r0 = static_cast<int>(r0);
    s.nrows = static_cast<int>(min(static_cast<long long>(ROWS), rows - r0));
    s.row0 = static_cast<int>(static_cast<long long>(w.pe.qa) * p.H + r0);
    s.cb = w.pe.cb;
    s.key0 = tile * BK;
    s.key1 = min(w.pe.L, (tile + len) * BK);
    if (DENSE || p.indices == nullptr)   // causal: the tile's last token sees keys up to cb + i
      s.key1 = min(s.key1, s.cb + (s.r0 + s.nrows - 1) / p.H + 1);
    if (s.key1 <= s.key0) continue;
    s.n = (s.key1 - s.key0 + BK - 1) / BK;
    s.slot = (piece + w.pe.items + item) * p.members + member;
    return true;
  }
  return false;
}

// Cache row of key `pos` of sequence b, in two steps, so that the table read can
// be issued a tile or more before its value is looked at: the page id (or the
// listed row), then the row or -1 (reported).
template <bool DENSE>
__device__ __forceinline__ int q8_entry(const Q8Params& p, int b, int pos) {
  if (!DENSE && p.indices != nullptr) return __ldg(p.indices + static_cast<long long>(b) * p.indices_stride + pos);
  const int pi = fast_div(pos, p.page);
  return pi < p.max_pages ? __ldg(p.page_table + static_cast<long long>(b) * p.max_pages + pi) : -1;
}
template <bool DENSE>
__device__ __forceinline__ int q8_row(const Q8Params& p, int pos, int entry) {
  int row = -1;
  if (!DENSE && p.indices != nullptr) {
    if (entry >= 0 && entry < p.cache_rows) row = entry;
  } else if (entry >= 0 && entry < p.num_pages) {
    row = entry * p.page.d + pos - fast_div(pos, p.page) * p.page.d;
  }
  if (row < 0) set_status(p.status, MLA_DEV_BAD_PAGE);
  return row;
}

// A softmax warpgroup's barrier, arrived at and waited on apart: its warps
// go on between the two, and the wait is bounded (a warp that gave up ends the
// others' waits through the abort flag).
struct GroupBar {
  uint32_t bar, phase;
};
__device__ __forceinline__ void group_arrive(const GroupBar& g) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(g.bar);
}
__device__ __forceinline__ bool group_wait(GroupBar& g, int32_t* status, volatile int* abort_flag) {
  const bool ok = wait_warp(g.bar, g.phase & 1, status, abort_flag);
  ++g.phase;
  return ok;
}
__device__ __forceinline__ bool group_sync(GroupBar& g, int32_t* status, volatile int* abort_flag) {
  group_arrive(g);
  return group_wait(g, status, abort_flag);
}

__device__ __forceinline__ uint4 ld_shared_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// Order-preserving integer of a float (for the integer warp maximum) and back.
__device__ __forceinline__ int float_order(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float order_float(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7FFFFFFF)); }

// op over the 32 lanes of each of a lane's 16 values; lane l returns value
// l / 2's.  Lanes exchange halves of their values: 16 shuffles, not 80.
template <typename Op>
__device__ __forceinline__ float reduce16(float (&v)[16], Op op) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 8; n >= 1; n >>= 1) {
    const bool up = (lane & (2 * n)) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = up ? v[i + n] : v[i], give = up ? v[i] : v[i + n];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, 2 * n));
    }
  }
  return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

constexpr int kSparseProducers = 2;   // warp 0 and another one

// TWICE: a tile's latent blocks are loaded for its scores and again (from L2)
// for its values, in the order in which the MMAs take them: scores 0, scores 1,
// values 0, scores 2, values 1, ...  The ring then holds nothing but loads in
// flight.  Otherwise a tile stays in its slots from its scores to its values:
// half the reads of L2, but a slot is held through the softmax.  64 rows leave
// room for two tiles: 64 sequences of 4096 to 16384 keys, 128 heads, take 284 us
// twice and 312 once.  16 rows leave room for three: 32 sequences of 16384 to
// 32768 keys, 16 heads, take 96 us once and 105 twice.  (32 rows, which stay in
// place too, would be faster twice by now: 96 us against 104, 64 sequences of 32
// heads, and 108 against 112, 32 long ones; in an earlier state of the loops it was
// the other way round.)  Listed rows, whose copies cost more, are loaded once.
//
// DENSE: a tile's rows come in runs of p.box consecutive rows of one page, each
// a rectangular TMA load.  Otherwise (listed rows, page sizes that are no
// multiple of 32) warps copy the rows with cp.async.
template <bool DENSE, int R>
__global__ void __launch_bounds__(Shape<R>::THREADS + (DENSE ? 0 : 32 * (kSparseProducers - 1)), 1)
    q8_attn_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap qr_map,
                   const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap kr_map,
                   const Q8Params p) {
  using C = Shape<R>;
  constexpr int ROWS = C::ROWS, GROUPS = C::GROUPS, SLOTS = C::SLOTS, ROPES = C::ROPES, NQ = C::NQ;
  constexpr bool WIDE = C::WIDE, TWICE = WIDE && DENSE;
  constexpr uint32_t TM_S = C::TM_S, TM_O = C::TM_O, TM_COLS = C::TM_COLS;
  constexpr uint32_t IDESC_QK = idesc_e4m3(128, NQ, false, false);
  constexpr uint32_t IDESC_PV = idesc_e4m3(128, C::NP, true, true);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;   // every byte is used: the base itself is a multiple of 1024 (checked below)
  using Smem = AttnSmem<C::SLOTS, C::ROPES>;
  static_assert(sizeof(Smem) <= C::TOTAL - C::AT_BAR, "barrier block");
  Smem* sh = reinterpret_cast<Smem*>(smem + C::AT_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int member = blockIdx.x % p.members, piece = blockIdx.x / p.members;
  int32_t* status = p.status;
  pdl_enter();
  if ((smem_u32(smem_raw) & 1023u) != 0) {           // a launch without that alignment would compute nonsense
    set_status(status, MLA_DEV_TIMEOUT);
    return;
  }

  if (threadIdx.x == 0) {
    // A block's load is counted in bytes (DENSE), or by the copying threads' arrivals.
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(smem_u32(&sh->k_full[s]), DENSE ? 1 : 32 * kSparseProducers);
      mbar_init(smem_u32(&sh->k_empty[s]), 1);
    }
    for (int s = 0; s < ROPES; ++s) {
      mbar_init(smem_u32(&sh->r_full[s]), DENSE ? 1 : 32 * kSparseProducers);
      mbar_init(smem_u32(&sh->r_empty[s]), 1);
    }
    mbar_init(smem_u32(&sh->fixed), 4 * GROUPS);
    mbar_init(smem_u32(&sh->q_full), 1);
    mbar_init(smem_u32(&sh->q_free), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&sh->s_full[i]), 2);         // the scores, and the keys' scales
      mbar_init(smem_u32(&sh->s_free[i]), 4 * GROUPS);
    }
    mbar_init(smem_u32(&sh->p_full), 4 * GROUPS);
    mbar_init(smem_u32(&sh->pv_done), 1);
    mbar_init(smem_u32(&sh->o_free), 4 * GROUPS);
    mbar_init(smem_u32(&sh->drain), 1);
    for (int i = 0; i < GROUPS; ++i) {
      mbar_init(smem_u32(&sh->group[i]), 4);
    }
    // An earlier kernel timed out: no work (and no plan to read).
    sh->abort = timed_out_before(status) ? 1 : 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh->tmem), TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  cluster_sync();            // (a wait that runs out raises the flag of the cluster's other CTA too)
  tc_fence_after();
  const uint32_t tmem = sh->tmem;
  volatile int* abort_flag = &sh->abort;
  const bool dead = sh->abort != 0;
  __syncthreads();                                   // the flag may be raised from here on
  Segment sg;
  Walk wk;
  if (!dead) wk = walk_begin(p, piece); else wk.u = wk.u1 = 0;

  // A segment's queries: warp 0, or, where that copies rows, the scales' warp.
  auto load_q = [&](const Segment& of, uint32_t seg) -> bool {
    if (seg > 0 && !wait_warp(smem_u32(&sh->q_free), (seg - 1) & 1, status, abort_flag)) return false;
    if (elect_one()) {
      const uint32_t qf = smem_u32(&sh->q_full);
      mbar_expect_tx(qf, C::QBYTES);
#pragma unroll
      for (int term = 0; term < 2; ++term) {
        // The second term's rows follow the first's.
        const uint32_t base = smem_u32(smem + C::AT_Q);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tma_load_2d(base + c * C::QBLOCK + term * ROWS * 128, &q_map, qf, term * 576 + c * 128, of.row0);
        tma_load_2d(base + 4 * C::QBLOCK + term * ROWS * 64, &qr_map, qf, term * 576 + 512, of.row0);
      }
    }
    __syncwarp();
    return true;
  };
  // The last queries land before the CTA leaves.
  auto drain_q = [&](uint32_t seg) {
    volatile int never = 0;
    if (seg > 0) wait_warp(smem_u32(&sh->q_full), (seg - 1) & 1, status, &never);
  };

  if (DENSE && warp == 0) {
    // ------------------------------------------------------------ queries, and the keys' TMA loads
    // One elected lane waits, counts and issues for a whole tile, in straight
    // code; the warp only looks up the rows (a warp-wide step for every block
    // took 700 clk, three times the load itself).
    uint32_t seg = 0;
    uint32_t sk = 0, tk = 0, sr = 0, tr = 0;          // slot and turn of the next latent block and rope part
    bool ok = true;
    const int nbox = BK / p.box;                      // runs of a tile, 4 at most
    const int span = 32 / nbox;                       // tiles whose runs the warp looks up together
    while (ok && walk_next<ROWS, DENSE>(p, wk, member, piece, sg)) {
      if constexpr (DENSE) {
        // Lane l has run l % nbox of tile j0 + l / nbox; the next tiles' table
        // entries are read while these are loaded.
        const int n = sg.n;
        auto entry_of = [&](int j0) -> int {
          const int pos = sg.key0 + j0 * BK + lane * p.box;
          return pos < sg.key1 ? q8_entry<DENSE>(p, sg.b, pos) : 0;
        };
        int entry = entry_of(0);
        const bool late = seg > 0;
        int base = 0, row = 0;                            // first tile of the batch, this lane's run in it
        auto runs = [&](int j) { return j + 1 < n ? nbox : (sg.key1 - (sg.key0 + j * BK) + p.box - 1) / p.box; };
        // One elected lane: a tile's two slots, and its rope part.
        auto blocks = [&](int j, bool rope) -> bool {
          const int boxes = runs(j);
          const int* rows = j >= base ? sh->run + (j - base) * nbox : sh->last;
#pragma unroll(TWICE ? 2 : 1)   // (64 sequences of 128 heads: 284 us, against 298 rolled; 16 heads: 96 either way)
          for (int c = 0; c < 2; ++c) {
            if (tk > 0 && !wait_one(smem_u32(&sh->k_empty[sk]), (tk & 1) ^ 1, status, abort_flag)) return false;
            const uint32_t full = smem_u32(&sh->k_full[sk]);
            mbar_expect_tx(full, boxes * p.box * 256);
            const uint32_t dst = smem_u32(smem) + sk * SLOT;
#pragma unroll 2                                       // (pages of 64, 128 heads: 307 us, 320 by four, 301 rolled)
            for (int x = 0; x < boxes; ++x) tma_load_4d(dst + x * p.box * 256, &k_map, full, 0, 0, 2 * c, rows[x] >> 3);
            if (++sk == SLOTS) {
              sk = 0;
              ++tk;
            }
          }
          if (rope) {
            if (tr > 0 && !wait_one(smem_u32(&sh->r_empty[sr]), (tr & 1) ^ 1, status, abort_flag)) return false;
            const uint32_t full = smem_u32(&sh->r_full[sr]);
            mbar_expect_tx(full, boxes * p.box * 64);
            const uint32_t dst = smem_u32(smem + C::AT_ROPE) + sr * ROPE;
            for (int x = 0; x < boxes; ++x) tma_load_2d(dst + x * p.box * 64, &kr_map, full, 512, rows[x]);
            if (++sr == ROPES) {
              sr = 0;
              ++tr;
            }
          }
          return true;
        };
        for (int j0 = 0; j0 < n && ok; j0 += span) {
          const int pos = sg.key0 + j0 * BK + lane * p.box;
          // The batch before was full: its last tile's values are still to come.
          if (lane >= 32 - nbox) sh->last[lane - (32 - nbox)] = row;
          row = pos < sg.key1 ? q8_row<DENSE>(p, pos, entry) : 0;
          if (row < 0) row = p.cache_rows;                   // past the end: reads zeros
          sh->run[lane] = row;
          base = j0;
          entry = entry_of(j0 + span);
          __syncwarp();
          // One place that loads keys, and one for the queries: what is
          // inlined twice is fetched twice (the instruction cache misses all
          // the time; this and the MMAs' small loops made both 16 and 128 heads
          // 7 % faster).  Values a tile behind, the last one's at the end.
          const int j1 = min(n, j0 + span), end = j1 + (TWICE && j1 == n ? 1 : 0);
#pragma unroll 1
          for (int step = j0 == 0 ? 0 : 2; step < 3 && ok; ++step) {
            // A later segment's queries wait for the scores before them; its
            // first keys need not.
            if (step == 1) {
              ok = load_q(sg, seg++);
              continue;
            }
            const int first = step == 0 ? 0 : (late && j0 == 0 ? 1 : j0), stop = step == 0 ? (late ? 1 : 0) : end;
            bool good = true;
            if (elect_one()) {
#pragma unroll 1
              for (int j = first; j < stop && good; ++j)
#pragma unroll 1
                for (int v = j < n ? 0 : 1; v < (TWICE && j > 0 ? 2 : 1) && good; ++v) good = blocks(j - v, v == 0);
            }
            ok = __all_sync(0xffffffffu, good);
          }
        }
      }
    }
    // Every load lands before the CTA leaves: the last use of each slot.  (The
    // elected lane is the same one throughout: it has the counters.)
    if constexpr (DENSE) {
      if (elect_one()) {
        volatile int never = 0;
        for (uint32_t s = 0; s < SLOTS; ++s) {
          const uint32_t uses = tk + (s < sk ? 1 : 0);
          if (uses > 0) wait_one(smem_u32(&sh->k_full[s]), (uses - 1) & 1, status, &never);
        }
        for (uint32_t s = 0; s < ROPES; ++s) {
          const uint32_t uses = tr + (s < sr ? 1 : 0);
          if (uses > 0) wait_one(smem_u32(&sh->r_full[s]), (uses - 1) & 1, status, &never);
        }
      }
      __syncwarp();
    }
    drain_q(seg);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // One elected lane, from descriptors that only need an addition (computed
    // for each MMA they took longer than the MMAs).
    if (elect_one()) {
      const uint64_t a0 = sdesc(smem_u32(smem), 16, GROUP);                    // slot 0, as keys and as values
      const uint64_t ar0 = sdesc(smem_u32(smem + C::AT_ROPE), 16, 512, kSwizzle64);
      const uint64_t b0 = sdesc(smem_u32(smem + C::AT_Q), 16, 1024);
      const uint64_t br0 = sdesc(smem_u32(smem + C::AT_Q + 4 * C::QBLOCK), 16, 512, kSwizzle64);
      const uint64_t w0 = sdesc(smem_u32(smem + C::AT_P), 16, 8 * C::NP, C::NP == 64 ? kSwizzle64 : kSwizzle32);
      uint32_t seg = 0, g0 = 0, masked_tiles = 0;      // segments done, tiles before this one's, cleaned tiles
      uint32_t sk = 0, tk = 0;                         // slot and turn of the next latent block
      uint32_t vk = 0;                                 // loaded once: slot of the next values
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_one(smem_u32(bar), parity, status, abort_flag); };
      auto landed = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (!wait(bar, parity)) return false;
        tc_fence_after();
        if (!DENSE) fence_async_smem();                // the rows came by cp.async
        return true;
      };
      auto scores = [&](uint32_t g, bool last) -> bool {
        const uint32_t sb = g & 1, d = tmem + TM_S + sb * NQ;
        if (g >= 2 && !wait(&sh->s_free[sb], ((g >> 1) & 1) ^ 1)) return false;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          if (!landed(&sh->k_full[sk], tk & 1)) return false;
          const uint64_t ad = a0 + sk * (SLOT >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)                 // blocks 2 c and 2 c + 1, 32 columns a step
            mma_f8_ss(d, ad + (kk >> 2) * 64 + (kk & 3) * 2, b0 + (2 * c + (kk >> 2)) * (C::QBLOCK >> 4) + (kk & 3) * 2,
                      IDESC_QK, (c | kk) != 0);
          if (TWICE) tc_commit(smem_u32(&sh->k_empty[sk]));
          if (++sk == SLOTS) {
            sk = 0;
            ++tk;
          }
        }
        const uint32_t rs = g % ROPES;
        if (!landed(&sh->r_full[rs], (g / ROPES) & 1)) return false;
        const uint64_t ad = ar0 + rs * (ROPE >> 4);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) mma_f8_ss(d, ad + kk * 2, br0 + kk * 2, IDESC_QK, 1);
        tc_commit(smem_u32(&sh->s_full[sb]));
        tc_commit(smem_u32(&sh->r_empty[rs]));
        if (last) tc_commit(smem_u32(&sh->q_free));
        return true;
      };
      auto values = [&](uint32_t g, bool first, bool masked) -> bool {
        if (!wait(&sh->p_full, g & 1)) return false;
        // O is free once the segment before has been read.
        if (first && seg > 0 && !wait(&sh->o_free, (seg - 1) & 1)) return false;
        if (masked && !wait(&sh->fixed, masked_tiles++ & 1)) return false;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          if (TWICE && !landed(&sh->k_full[sk], tk & 1)) return false;
          const uint32_t slot = TWICE ? sk : vk;
          const uint64_t ad = a0 + slot * (SLOT >> 4);
#pragma unroll(TWICE ? 4 : 8)
          for (int kk = 0; kk < 8; ++kk) {
            // Block 2 c + kk / 4, 32 keys a step: both operands MN-major, groups of 8 keys
            // 2048 (keys) and 8 NP (weights) bytes apart.
            const uint64_t av = ad + (kk >> 2) * 64 + (kk & 3) * (4 * GROUP >> 4), wv = w0 + (kk & 3) * (4 * 8 * C::NP >> 4);
            const uint32_t d = tmem + TM_O + (2 * c + (kk >> 2)) * C::NP;
            mma_f8_ss(d, av, wv, IDESC_PV, !first || (kk & 3) != 0);
            if (WIDE) mma_f8_ss(d, av, wv + (C::PTERM >> 4), IDESC_PV | kIdescB_e5m2, 1);
          }
          tc_commit(smem_u32(&sh->k_empty[slot]));
          if (!TWICE) {
            if (++vk == SLOTS) vk = 0;
          } else if (++sk == SLOTS) {
            sk = 0;
            ++tk;
          }
        }
        tc_commit(smem_u32(&sh->pv_done));
        return true;
      };
      while (ok && walk_next<ROWS, DENSE>(p, wk, member, piece, sg)) {
        // Tiles that hold a key which some row does not see.
        int all = sg.key1 - sg.key0;
        if (DENSE || p.indices == nullptr) all = min(all, sg.cb + sg.r0 / p.H + 1 - sg.key0);
        ok = wait(&sh->q_full, seg & 1);
#pragma unroll 1
        for (int j = 0; j <= sg.n && ok; ++j) {          // scores a tile ahead of values
          if (j < sg.n) ok = scores(g0 + j, j + 1 == sg.n);
          if (j > 0) ok = ok && values(g0 + j - 1, j == 1, j * BK > all);
        }
        g0 += sg.n;
        ++seg;
      }
      tc_commit(smem_u32(&sh->drain));
      volatile int never = 0;
      wait_one(smem_u32(&sh->drain), 0, status, &never);
    }
    __syncwarp();
  } else if (warp >= 2 && warp < 2 + 4 * GROUPS) {
    // ------------------------------------------------------------ softmax (thread = key), epilogue
    // Warpgroups with all 128 keys and 16 of the tile's query rows each.  The
    // code of a tile is kept small and there once: with 32 rows a thread and a
    // second copy for a moving reference it did not fit the instruction cache,
    // and every warp of the kernel ran at a fifth of its speed.
    const int wg = (warp - 2) >> 2;
    GroupBar gb{smem_u32(&sh->group[wg]), 0u};
    const int c0 = wg * 16;                           // first query row of the group
    const int q4 = warp & 3;
    const int key = q4 * 32 + lane;
    const int tid = (warp - 2 - 4 * wg) * 32 + lane;  // 0..127 in the group
    const uint32_t lane_off = uint32_t(q4 * 32) << 16;
    uint8_t* pbuf = smem + C::AT_P;
    // 16-byte chunk c of a key's weights.
    auto p_chunk = [&](int k, int c) -> uint8_t* {
      return pbuf + k * C::NP + ((c ^ (C::NP == 64 ? (k >> 1) & 3 : (k >> 2) & 1)) << 4);
    };
    uint32_t seg = 0, g0 = 0;                         // segments done, tiles before this one's
    bool fail = false;
    while (!fail && walk_next<ROWS, DENSE>(p, wk, member, piece, sg)) {
      const int mine = min(16, sg.nrows - c0);        // rows of this group (none: it only keeps the pace)
      const int span = sg.key1 - sg.key0;
      float lowest = kInf;                            // least ry of this thread's row, once it has a reference
      if (tid < 16) {
        const int r = c0 + tid;
        float rf = 0.f;
        int lim = 0;
        if (tid < mine) {
          rf = p.q_scale[sg.row0 + r] * p.scale_log2;
          lim = span;
          if (DENSE || p.indices == nullptr) lim = min(lim, sg.cb + (sg.r0 + r) / p.H + 1 - sg.key0);
        }
        sh->rf[r] = rf;
        sh->ry[r] = tid < mine ? 0.f : -kInf;         // rows past the last: no weight
        sh->lim[r] = lim;
        sh->top[r] = float_order(-kInf);
      }
      // Keys that every row of the tile sees.
      int all = span;
      if (DENSE || p.indices == nullptr) all = min(all, sg.cb + sg.r0 / p.H + 1 - sg.key0);
      if (!group_sync(gb, status, abort_flag)) {
        fail = true;
        break;
      }
      float2 l[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) l[c] = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int j = 0; j < sg.n; ++j) {
        const uint32_t g = g0 + j, sb = g & 1;
        const bool masked = (j + 1) * BK > all;       // some row does not see every key of the tile
        if (!wait_warp(smem_u32(&sh->s_full[sb]), (g >> 1) & 1, status, abort_flag)) {
          fail = true;
          break;
        }
        tc_fence_after();
        float ksc = sh->ksc[sb][key];
        const bool broken = !(fabsf(ksc) < kInf);     // a scale that is no number: the key's scores are NaN
        if (broken) ksc = 1.f;
        const float lsc = __log2f(fabsf(ksc));
        const float xv = broken ? __int_as_float(0x7fc00000) : ksc;
        // The first tile sets the rows' references; in a later one the weights
        // are computed against them, and once more if one has to move.
        bool move = j == 0;
        if (move && g > 0 && !wait_warp(smem_u32(&sh->pv_done), (g - 1) & 1, status, abort_flag)) {
          fail = true;
          break;
        }
        float2 t[8];
        uint32_t hi[4], lo[4];
        while (true) {
          // Exponents (log2 units) of the key's weights.
          {
            uint32_t a[16], b[16];
            tmem_ld16(tmem + lane_off + TM_S + sb * NQ + c0, a);
            tmem_ld16(tmem + lane_off + TM_S + sb * NQ + ROWS + c0, b);
            tmem_ld_wait();
            const float2 xs = make_float2(xv, xv), low = make_float2(1.f / kQueryLow, 1.f / kQueryLow);
#pragma unroll
            for (int c = 0; c < 8; c += 2) {
              const float4 rf = *reinterpret_cast<const float4*>(sh->rf + c0 + 2 * c);
              const float4 ry = *reinterpret_cast<const float4*>(sh->ry + c0 + 2 * c);
              const float2 u = __ffma2_rn(make_float2(__uint_as_float(b[2 * c]), __uint_as_float(b[2 * c + 1])), low,
                                          make_float2(__uint_as_float(a[2 * c]), __uint_as_float(a[2 * c + 1])));
              const float2 v = __ffma2_rn(make_float2(__uint_as_float(b[2 * c + 2]), __uint_as_float(b[2 * c + 3])), low,
                                          make_float2(__uint_as_float(a[2 * c + 2]), __uint_as_float(a[2 * c + 3])));
              t[c] = __ffma2_rn(__fmul2_rn(u, xs), make_float2(rf.x, rf.y), make_float2(ry.x, ry.y));
              t[c + 1] = __ffma2_rn(__fmul2_rn(v, xs), make_float2(rf.z, rf.w), make_float2(ry.z, ry.w));
            }
          }
          uint32_t rows = 0xFFFFu;                    // that see any key of the tile
          if (__builtin_expect(masked, 0)) {
            uint32_t some = 0u;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const int x = sh->lim[c0 + 2 * c] - j * BK, y = sh->lim[c0 + 2 * c + 1] - j * BK;
              t[c].x = key < x ? t[c].x : -kInf;
              t[c].y = key < y ? t[c].y : -kInf;
              some = some << 2 | (x > 0 ? 2u : 0u) | (y > 0 ? 1u : 0u);
            }
            rows = some;
          }
          if (__builtin_expect(!move, 1)) {
            // Whether a key has a weight above the range, and which rows have
            // none within it: told to the group's other warps here, looked at
            // when the weights are ready.
            float mx = -kInf;
#pragma unroll
            for (int c = 0; c < 8; ++c) mx = fmax3(mx, t[c].x, t[c].y);
            const float2 off = make_float2(lsc - C::LOW, lsc - C::LOW);
            uint32_t range = mx + lsc > C::HIGH ? 0u : 1u;
#pragma unroll
            for (int c = 0; c < 8; ++c) {                // the signs, the first row's on top
              const float2 v = __fadd2_rn(t[c], off);
              range = __funnelshift_l(__float_as_uint(v.x), range, 1);
              range = __funnelshift_l(__float_as_uint(v.y), range, 1);
            }
            range = __reduce_and_sync(0xffffffffu, range);
            if (lane == 0) sh->range[g & 1][wg][q4] = range;
            group_arrive(gb);
          } else {
            // ---- move the reference of the rows that need it
            float v[16];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              v[2 * c] = t[c].x + lsc;
              v[2 * c + 1] = t[c].y + lsc;
            }
            const float m = reduce16(v, [](float x, float y) { return fmaxf(x, y); });
            // Each warp's largest of a row, in the group's share of the weights'
            // buffer (the weights that come next are not there yet).
            auto warp_top = [&](int w, int r) {
              return reinterpret_cast<float*>(p_chunk(4 * w + (r >> 2), wg)) + (r & 3);
            };
            if ((lane & 1) == 0) *warp_top(q4, lane >> 1) = m;
            if (!group_sync(gb, status, abort_flag)) {
              fail = true;
              break;
            }
            if (tid < 16) {
              const float x0 = *warp_top(0, tid), x1 = *warp_top(1, tid), x2 = *warp_top(2, tid), x3 = *warp_top(3, tid);
              const float a = fmaxf(x0, x1), b = fmaxf(x2, x3), mm = fmaxf(a, b), ry = sh->ry[c0 + tid];
              // No other warp's keys come near the largest: it is put at the top,
              // which leaves the others most bits.  (So it is where one tile is
              // all, which needs no room above.)
              const float next = fmaxf(fminf(a, b), a > b ? fminf(x0, x1) : fminf(x2, x3));
              const bool alone = mm - next > kAlone || sg.n == 1;
              float d = 0.f, f = 1.f;
              if (mm > -kInf) {
                if (lowest == kInf) {
                  d = (alone ? C::HIGH - 0.25f : C::FIRST) - mm;
                } else if (mm > C::HIGH) {
                  d = (alone ? C::HIGH - 0.25f : C::UP) - mm;
                  f = ex2(d);
                } else if (mm < C::LOW) {
                  // At most so far that the sums' exponents have room; what
                  // lies that far below the row's largest weights counts for nothing.
                  d = fmaxf(fminf(C::DOWN - mm, lowest + kReach - ry), 0.f);
                  f = ex2(d);
                }
                lowest = fminf(lowest, ry + d);
              }
              sh->ry[c0 + tid] = ry + d;
              sh->d[c0 + tid] = d;
              sh->f[c0 + tid] = f;
              const uint32_t may = __ballot_sync(0xffffu, tid < mine && ry + d < lowest + kReach - 1.f);
              if (tid == 0) sh->care[wg] = __brev(may) >> 16;
            }
            if (!group_sync(gb, status, abort_flag)) {
              fail = true;
              break;
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              t[c] = __fadd2_rn(t[c], *reinterpret_cast<const float2*>(sh->d + c0 + 2 * c));
              l[c] = __fmul2_rn(l[c], *reinterpret_cast<const float2*>(sh->f + c0 + 2 * c));
            }
            if (j > 0) {
#pragma unroll 1
              for (int cb = 0; cb < (WIDE ? 4 : 8); ++cb) {
                uint32_t r[16];
                const uint32_t ta = tmem + lane_off + TM_O + cb * ROWS + c0;
                tmem_ld16(ta, r);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * sh->f[c0 + i]);
                tmem_st16(ta, r);
              }
              tmem_st_wait();
            }
          }
          // ---- weights, and their two terms
          {
            const float2 ks = make_float2(ksc * C::LO, ksc * C::LO);
            // Rounds to four bits (Veltkamp's split): y = x (2^20 + 1) has 24
            // bits, 20 of which y - (y - x) cancels.  What is added to y keeps
            // its last bit at 2^-9 of a weight or above, the first term's step
            // below e4m3's normal range, so that the second term is what is
            // missing there too.
            const float2 split = make_float2(1048577.f, 1048577.f);
            const float2 least = make_float2(16384.f * C::LO, 16384.f * C::LO);
#pragma unroll
            for (int c = 0; c < 8; c += 2) {
              uint16_t h[2], w[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float2 e = make_float2(ex2(t[c + i].x), ex2(t[c + i].y));
                t[c + i] = e;
                const float2 x = __fmul2_rn(e, ks);
                const float2 y = __ffma2_rn(x, split, least);
                const float2 z = __fadd2_rn(y, make_float2(-x.x, -x.y));
                float2 a = __fadd2_rn(y, make_float2(-z.x, -z.y));
                const float2 b = __fadd2_rn(x, make_float2(-a.x, -a.y));
                if constexpr (!WIDE) a = __fmul2_rn(a, make_float2(1.f / C::LO, 1.f / C::LO));
                h[i] = pack_e4m3(a.x, a.y);
                w[i] = WIDE ? pack_e5m2(b.x, b.y) : pack_e4m3(b.x, b.y);
              }
              hi[c / 2] = static_cast<uint32_t>(h[0]) | (static_cast<uint32_t>(h[1]) << 16);
              lo[c / 2] = static_cast<uint32_t>(w[0]) | (static_cast<uint32_t>(w[1]) << 16);
            }
          }
          if (move) break;
          // The weights' buffer (and O, where the reference moves) is free once
          // P V of the tile before is done.
          if (!group_wait(gb, status, abort_flag) ||
              !wait_warp(smem_u32(&sh->pv_done), (g - 1) & 1, status, abort_flag)) {
            fail = true;
            break;
          }
          // (The words are written again two tiles on, by warps that know
          // all of the group to have arrived at the next tile.)
          const uint4 word = ld_shared_u4(smem_u32(sh->range[g & 1][wg]));
          const uint32_t range = (word.x & word.y) & (word.z & word.w);
          move = range < 0x10000u || (range & rows & *const_cast<const volatile uint32_t*>(&sh->care[wg])) != 0u;
          if (!move) break;
          tc_fence_after();
        }
        if (fail) break;
#pragma unroll
        for (int c = 0; c < 8; ++c) l[c] = __fadd2_rn(l[c], t[c]);
        // Key-major rows of NP bytes (64- or 32-byte swizzle): chunk wg, and the
        // second term in a buffer of its own (wide) or ROWS bytes on.
        if (mine > 0) {
          *reinterpret_cast<uint4*>(p_chunk(key, wg)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(WIDE ? p_chunk(key, wg) + C::PTERM : p_chunk(key, ROWS / 16 + wg)) =
              make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&sh->p_full));
          mbar_arrive(smem_u32(&sh->s_free[sb]));
        }
        if (__builtin_expect(masked, 0)) {
          // A key that some row does not see: its weight is 0 there, but 0 times
          // a NaN code is NaN.  Rows past the segment become zeros (they may
          // hold anything); in the others every NaN code does (a row that sees
          // such a key has a NaN score, so its result is NaN all the same).
          // The first two warpgroups have one of the tile's two value slots
          // each, when it lands (a single one has both).
#pragma unroll 1
          for (int half = wg; half < 2; half += GROUPS) {
            const uint32_t u = half + (TWICE ? 4 * g0 + (j + 1 < sg.n ? 4 * j + 4 : 4 * j + 2) : 2 * g);
            const uint32_t slot = u % SLOTS;
            if (!wait_warp(smem_u32(&sh->k_full[slot]), (u / SLOTS) & 1, status, abort_flag)) {
              fail = true;
              break;
            }
            if (j * BK + key >= all) {
              uint8_t* kr = smem + slot * SLOT + (key >> 3) * GROUP + (key & 7) * 128;
#pragma unroll 1
              for (int i = 0; i < 16; ++i) {
                uint4* at = reinterpret_cast<uint4*>(kr + (i >> 3) * 1024) + (i & 7);
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (j * BK + key < span) {
                  v = *at;
                  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                  for (int x = 0; x < 4; ++x) {
                    // Bytes equal to 0x7F after clearing the sign.
                    const uint32_t nan = ((w[x] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                    w[x] &= ~((nan >> 7) * 0xFFu);
                  }
                }
                *at = v;
              }
            }
            fence_async_smem();
          }
          if (fail) break;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh->fixed));
        }
      }
      if (fail) break;
      g0 += sg.n;
      // ---------------------------------------------------------- epilogue
      if (!wait_warp(smem_u32(&sh->pv_done), (g0 - 1) & 1, status, abort_flag) ||
          !group_sync(gb, status, abort_flag)) {      // every warp is past the row arrays' last use
        fail = true;
        break;
      }
      tc_fence_after();
      // 128 latent columns of the result, one a thread: the group's rows.
      auto result = [&](int c, uint32_t (&o)[16]) {
        const uint32_t ta = tmem + lane_off + TM_O + c * C::NP + c0;
        tmem_ld16(ta, o);
        if constexpr (!WIDE) {
          uint32_t o2[16];
          tmem_ld16(ta + ROWS, o2);
          tmem_ld_wait();
#pragma unroll
          for (int r = 0; r < 16; ++r)
            o[r] = __float_as_uint(fmaf(__uint_as_float(o2[r]), 1.f / C::LO, __uint_as_float(o[r])));
        } else {
          tmem_ld_wait();
        }
      };
      // Sums over the keys: within each warp, then over the four warps through
      // the row arrays that the segment no longer needs.  And each row's largest
      // result, whose exponent the row is stored relative to, in fp16: what a row
      // is made of then does not depend on any key that has no weight in it.
      if (mine > 0) {
        float m[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) m[r] = 0.f;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[16];
          result(c, o);
#pragma unroll
          for (int r = 0; r < 16; ++r) m[r] = fmaxf(m[r], fabsf(__uint_as_float(o[r])));
        }
        const float mx = reduce16(m, [](float x, float y) { return fmaxf(x, y); });
        if ((lane & 1) == 0) atomicMax(&sh->top[c0 + (lane >> 1)], float_order(mx));   // a maximum: in any order
      }
      {
        float v[16];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          v[2 * c] = l[c].x;
          v[2 * c + 1] = l[c].y;
        }
        const float sum = reduce16(v, [](float x, float y) { return x + y; });
        float* part = q4 == 0 ? sh->rf : (q4 == 1 ? sh->d : (q4 == 2 ? sh->f : reinterpret_cast<float*>(sh->lim)));
        if ((lane & 1) == 0) part[c0 + (lane >> 1)] = sum;
      }
      if (!group_sync(gb, status, abort_flag)) {
        fail = true;
        break;
      }
      if (tid < 16) {
        const int r = c0 + tid;
        const float sum = (sh->rf[r] + sh->d[r]) + (sh->f[r] + __int_as_float(sh->lim[r]));
        // 2^e, which puts the largest in [2^14, 2^15) (an infinite one stays that).
        const int e = min(14 + 127 - (__float_as_int(order_float(sh->top[r])) >> 23 & 255), 126);
        sh->f[r] = sum == 0.f ? 0.f : __int_as_float((e + 127) << 23);
        // Weights carry 2^-reference: log2 of the plain sum adds it back.
        if (tid < mine)
          p.meta[static_cast<long long>(sg.slot) * ROWS + r] =
              make_float2(sum == 0.f ? -kInf : __log2f(sum) - sh->ry[r],
                          sum == 0.f ? 0.f : __int_as_float((127 - e) << 23) * (1.0f / sum));
      }
      if (!group_sync(gb, status, abort_flag)) {
        fail = true;
        break;
      }
      if (mine > 0) {
        __half* dst = p.o_part + (static_cast<long long>(sg.slot) * ROWS + c0) * 512 + key;
#pragma unroll 1
        for (int c = 0; c < 4; ++c, dst += 128) {
          uint32_t o[16];
          result(c, o);
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const float f = sh->f[c0 + r];
            if (r < mine) dst[r * 512] = __float2half_rn(f == 0.f ? 0.f : __uint_as_float(o[r]) * f);
          }
        }
        tc_fence_before();
      }
      if (!group_sync(gb, status, abort_flag)) {      // the row arrays are rewritten by the next segment
        fail = true;
        break;
      }
      if (lane == 0) mbar_arrive(smem_u32(&sh->o_free));
      ++seg;
    }
  } else if (warp == 2 + 4 * GROUPS) {
    // ------------------------------------------------------------ the keys' scales, a tile ahead
    uint32_t g = 0, seg = 0;
    bool ok = true;
    while (ok && walk_next<ROWS, DENSE>(p, wk, member, piece, sg)) {
      if (!DENSE && !(ok = load_q(sg, seg++))) break;
      const int n = sg.key1 - sg.key0;
      int entry[4];
      auto entries = [&](int k0) {
#pragma unroll
        for (int x = 0; x < 4; ++x) entry[x] = k0 + 32 * x + lane < n ? q8_entry<DENSE>(p, sg.b, sg.key0 + k0 + 32 * x + lane) : 0;
      };
      entries(0);
#pragma unroll 1
      for (int k0 = 0; k0 < n && ok; k0 += BK, ++g) {
        float v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int k = k0 + 32 * x + lane;
          v[x] = 1.f;
          if (k < n) {
            const int row = q8_row<DENSE>(p, sg.key0 + k, entry[x]);
            if (row >= 0) v[x] = __ldg(p.kv_scales + fast_div(row, p.block));
          }
        }
        entries(k0 + BK);
        const uint32_t sb = g & 1;
        if (g >= 2 && !(ok = wait_warp(smem_u32(&sh->s_free[sb]), ((g >> 1) & 1) ^ 1, status, abort_flag))) break;
#pragma unroll
        for (int x = 0; x < 4; ++x) sh->ksc[sb][32 * x + lane] = v[x];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh->s_full[sb]));
      }
    }
    if (!DENSE) drain_q(seg);
  } else {
    // ------------------------------------------------------------ listed rows: cp.async
    if constexpr (!DENSE) {
      constexpr int RW = BK / kSparseProducers;       // this warp's keys [RW pw, RW pw + RW) of the tile
      const int pw = warp == 0 ? 0 : 1;
      uint32_t issued = 0, ropes = 0;
      bool ok = true;
      while (ok && walk_next<ROWS, DENSE>(p, wk, member, piece, sg)) {
        int row[RW / 32], next[RW / 32];              // key 32 x + lane: this tile's row, the next one's table entry
        auto entries = [&](int j, int (&r)[RW / 32]) {
#pragma unroll
          for (int x = 0; x < RW / 32; ++x) {
            const int pos = sg.key0 + j * BK + pw * RW + 32 * x + lane;
            r[x] = j < sg.n && pos < sg.key1 ? q8_entry<DENSE>(p, sg.b, pos) : 0;
          }
        };
        // A tile's two slots (a chunk of 16 bytes a lane, two rows an
        // instruction), counted as they land.
        auto latent = [&](const int (&r)[RW / 32]) -> bool {
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            const uint32_t s = issued % SLOTS, turn = issued / SLOTS;
            if (turn > 0 && !wait_warp(smem_u32(&sh->k_empty[s]), (turn & 1) ^ 1, status, abort_flag)) return false;
            const uint32_t dst = smem_u32(smem + s * SLOT) + pw * (RW / 8) * GROUP + ((lane >> 3) & 1) * 1024;
            const uint8_t* src = p.kv_cache + c * 256 + (lane & 15) * 16;
#pragma unroll
            for (int i = 0; i < RW / 2; ++i) {
              const int k = 2 * i + (lane >> 4);
              const int at = __shfl_sync(0xffffffffu, r[i / 16], k & 31);
              cp_async16(dst + (k >> 3) * GROUP + (k & 7) * 128 + (((lane & 7) ^ (k & 7)) << 4), src + static_cast<size_t>(at) * 576);
            }
            cp_async_arrive(smem_u32(&sh->k_full[s]));
            ++issued;
          }
          return true;
        };
        entries(0, next);
        for (int j = 0; j < sg.n && ok; ++j) {
#pragma unroll
          for (int x = 0; x < RW / 32; ++x) {
            const int pos = sg.key0 + j * BK + pw * RW + 32 * x + lane;
            row[x] = pos < sg.key1 ? q8_row<DENSE>(p, pos, next[x]) : 0;
            if (row[x] < 0) row[x] = 0;               // reported; the result of its rows is not meaningful
          }
          entries(j + 1, next);                       // in flight while the tile is copied
          if (!(ok = latent(row))) break;
          const uint32_t s = ropes % ROPES, turn = ropes / ROPES;
          if (turn > 0 && !(ok = wait_warp(smem_u32(&sh->r_empty[s]), (turn & 1) ^ 1, status, abort_flag))) break;
          const uint32_t dst = smem_u32(smem + C::AT_ROPE + s * ROPE) + pw * RW * 64;
#pragma unroll
          for (int i = 0; i < RW / 8; ++i) {          // eight rows of 4 chunks
            const int k = 8 * i + (lane >> 2), ch = lane & 3;
            const int at = __shfl_sync(0xffffffffu, row[i / 4], k & 31);
            cp_async16(dst + k * 64 + ((ch ^ ((k >> 1) & 3)) << 4), p.kv_cache + static_cast<size_t>(at) * 576 + 512 + ch * 16);
          }
          cp_async_arrive(smem_u32(&sh->r_full[s]));
          ++ropes;
        }
      }
      // Every copy lands, and its arrival with it, before the CTA leaves.
      cp_async_commit();
      cp_async_wait<0>();
      volatile int never = 0;
      if (ok) {
        for (uint32_t s = 0; s < SLOTS; ++s)
          if (issued > s) wait_warp(smem_u32(&sh->k_full[s]), ((issued - 1 - s) / SLOTS) & 1, status, &never);
        for (uint32_t s = 0; s < ROPES; ++s)
          if (ropes > s) wait_warp(smem_u32(&sh->r_full[s]), ((ropes - 1 - s) / ROPES) & 1, status, &never);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();            // neither CTA leaves while the other may still raise its flag
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
}

// ============================================================ 3. merge and w_uv
// One CTA per (head, up to 16 tokens): the segments' latent results are merged
// by LSE in fp32 (with the attention sink in the denominator), split into two
// bf16 terms (their sum within 2^-16) and multiplied by w_uv[h]: D^T [128
// values, 32] = w_uv[h] [128, 512] . o^T, both terms of 16 tokens side by side,
// so that few tokens make a small N.  w_uv[h] is loaded from before the
// attention has ended.  16 warps: with few tokens several of them share one
// token's segments (a single long sequence has one for every SM) and join
// through shared memory.
//
// RING: blocks of w_uv[h] (of eight) in shared memory.  All of them where one
// wave of CTAs holds every token; else four, so that two CTAs share an SM, one's
// chains of reads under the other's: 64 tokens of 128 heads 17.7 us, against 20.9
// with one CTA an SM, 32 tokens and all blocks.  (In one wave the ring of four
// makes a decode of 16 heads 2 to 3 % longer.)
constexpr int kOutWarps = 16;
constexpr int NT = 16;
constexpr int W_BLOCK = 128 * 128;                   // 128 rows of 64 bf16
constexpr int O_BLOCK = 2 * NT * 128;                // 64 columns of both terms

template <int R>
struct OutShape {
  static constexpr int RING = R;
  static constexpr int CTAS = RING == 8 ? 1 : 2;     // on an SM
  static constexpr int KU = RING == 8 ? 4 : 2;       // segments loaded together (registers)
  static constexpr int AT_O = RING * W_BLOCK;
  static constexpr int AT_JOIN = AT_O + 8 * O_BLOCK; // [warp][512] partial sums, where warps share a token
  static constexpr int AT_BAR = AT_JOIN + (RING == 8 ? kOutWarps * 2048 : 0);
  static constexpr int TOTAL = AT_BAR + 1024 + 1024;
  static_assert(CTAS * (TOTAL + 1024) <= 228 * 1024, "shared memory");
};
struct OutSmem {
  uint64_t full[8], empty[8], done;
  uint32_t tmem;
  int abort;
  int used[NT];      // segments that hold keys of the token; -1: its rows are not written
  long long first[NT];   // row of the first one's results (in slots), the others `step` apart
  float sink[NT];    // log2 units
  float2 join[kOutWarps];   // a warp's maximum and sum
};
static_assert(sizeof(OutSmem) <= 1024, "barrier block");

// Running merge of segments: maximum, sum of weights, weighted sums of 16 latents.
struct Merge {
  float mx, tot, o[16];
};
__device__ __forceinline__ void merge_scale(Merge& m, float nm) {
  const float keep = m.mx == -kInf ? 0.f : ex2(m.mx - nm);
  m.tot *= keep;
#pragma unroll
  for (int e = 0; e < 16; ++e) m.o[e] *= keep;
  m.mx = nm;
}

template <int RING>
__global__ void __launch_bounds__(32 * kOutWarps, OutShape<RING>::CTAS)
    q8_out_kernel(const __grid_constant__ CUtensorMap w_map, const Q8Params p, const FastDiv item_rows,
                  const float* __restrict__ sink, __nv_bfloat16* __restrict__ out, float* __restrict__ lse, int T,
                  int tokens) {
  using C = OutShape<RING>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  OutSmem* sh = reinterpret_cast<OutSmem*>(smem + C::AT_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * tokens, h = blockIdx.y;
  const int n = min(tokens, T - t0);                 // tokens of this CTA, NT at most
  auto load_w = [&](int kb) {
    const uint32_t full = smem_u32(&sh->full[kb % RING]);
    mbar_expect_tx(full, W_BLOCK);
    tma_load_2d(smem_u32(smem + (kb % RING) * W_BLOCK), &w_map, full, kb * 64, h * 128);
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < RING; ++i) {
      mbar_init(smem_u32(&sh->full[i]), 1);
      mbar_init(smem_u32(&sh->empty[i]), 1);
    }
    mbar_init(smem_u32(&sh->done), 1);
    sh->abort = 0;
    fence_mbar_init();
    // The weights do not come from the kernel before, and whatever wrote them
    // had completed when that kernel let this one start (it waits for its own
    // predecessor first).
#pragma unroll 1
    for (int kb = 0; kb < RING; ++kb) load_w(kb);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh->tmem), 2 * NT);
    tmem_relinquish();
  }
  pdl_enter();
  const bool dead = __any_sync(0xffffffffu, timed_out_before(p.status));   // no work, and no plan to read
  const int entries = dead ? 0 : __ldg(&p.head->entries), units = dead ? 0 : __ldg(&p.head->units);
  const long long step = item_rows.d;                // slots between a token's segments
  // A token, looked up by a warp.
  auto look_up = [&](int i) {
    const int t = t0 + i;
    int used = -1;
    long long first = 0;
    float sk = -kInf;
    if (entries > 0) {
      const int e_at = last_not_above(&p.entries[0].qa, kEntryInts, entries, t);
      const PlanEntry e = load_entry(p.entries + e_at);
      if (e.qa <= t && t < e.qa + e.n) {
        const int keys = p.indices != nullptr ? e.L : min(e.L, e.cb + (t - e.qa) + 1);
        const int r = (t - e.qa) * p.H + h;
        const int item = fast_div(r, item_rows);
        used = 0;
        if (keys > 0) {
          const int u = e.units + item * e.tiles;
          const int pieces = min(p.pieces, units), g0 = piece_of(u, pieces, units);
          used = piece_of(u + (keys + BK - 1) / BK - 1, pieces, units) - g0 + 1;
          first = static_cast<long long>(g0 + e.items + item) * item_rows.d + (r - item * item_rows.d);
        }
        if (sink != nullptr) sk = __ldg(sink + e.b) * 1.4426950408889634f;
      }
    }
    if (lane == 0) {
      sh->used[i] = used;
      sh->first[i] = first;
      sh->sink[i] = sk;
    }
  };
  // Warps of a token: a power of two, so that they divide the 16.
  int share = 1;
  while (RING == 8 && 2 * share * n <= kOutWarps) share *= 2;
  const int part = warp % share;
  Merge m;
  // One token's segments part, part + share, ...
  auto gather = [&](int i) {
    const int used = sh->used[i];
    const long long first = sh->first[i];
    m.mx = -kInf;
    m.tot = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) m.o[e] = 0.f;
    constexpr int KU = C::KU;
#pragma unroll 1
    for (int k0 = part; k0 < used; k0 += KU * share) {
      uint4 a[KU], c[KU];
      float2 mt[KU];
#pragma unroll
      for (int x = 0; x < KU; ++x) {
        const int k = k0 + x * share;
        const long long at = first + k * step;
        const bool in = k < used;
        mt[x] = in ? __ldg(p.meta + at) : make_float2(-kInf, 0.f);
        const uint4* src = reinterpret_cast<const uint4*>(p.o_part + at * 512);
        a[x] = in ? __ldg(src + lane) : make_uint4(0u, 0u, 0u, 0u);
        c[x] = in ? __ldg(src + 32 + lane) : make_uint4(0u, 0u, 0u, 0u);
      }
      float nm = m.mx;
#pragma unroll
      for (int x = 0; x < KU; ++x) nm = fmaxf(nm, mt[x].x);
      merge_scale(m, nm);
#pragma unroll
      for (int x = 0; x < KU; ++x) {
        const float w = mt[x].x == -kInf ? 0.f : ex2(mt[x].x - nm);
        m.tot += w;
        const float ws = w * mt[x].y;
        const uint32_t u[8] = {a[x].x, a[x].y, a[x].z, a[x].w, c[x].x, c[x].y, c[x].z, c[x].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 v = f16x2_to_float2(u[e]);
          m.o[2 * e] = fmaf(ws, v.x, m.o[2 * e]);
          m.o[2 * e + 1] = fmaf(ws, v.y, m.o[2 * e + 1]);
        }
      }
    }
  };
  // The merged token i into the operand: latents 8 lane .. +7 and 256 + 8 lane ..
  // +7, that is block of 64 columns lane / 8 (+ 4), 16-byte chunk lane & 7.
  auto finish = [&](int i) {
    const int used = sh->used[i];
    const float sk = sh->sink[i];
    float l2 = m.tot == 0.f ? -kInf : m.mx + __log2f(m.tot);
    float w = m.tot == 0.f ? 0.f : 1.0f / m.tot;
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
    if (lse != nullptr && used >= 0 && lane == 0) lse[static_cast<long long>(t0 + i) * p.H + h] = l2 * kLn2q;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = m.o[8 * half + 2 * e] * w, y = m.o[8 * half + 2 * e + 1] * w;
        hi[e] = pack_bf16(x, y);
        lo[e] = pack_bf16(x - bf16_lo(hi[e]), y - bf16_hi(hi[e]));
      }
      uint8_t* dst = smem + C::AT_O + (half * 4 + (lane >> 3)) * O_BLOCK + i * 128 + (((lane & 7) ^ (i & 7)) << 4);
      *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(dst + NT * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  };
  // (Operand rows past the last token hold anything: their results are not stored.)
  // (The code of a step is there once, in loops: fetching unrolled copies takes
  // longer than the chains of reads that they would overlap.)
#pragma unroll 1
  for (int i = warp / share; i < n; i += kOutWarps / share) look_up(i);
  __syncwarp();
#pragma unroll 1
  for (int i = warp / share;; i += kOutWarps) {
    if (i < n) gather(i);
    if (share > 1) {                                   // one turn: share * n <= 16
      float* join = reinterpret_cast<float*>(smem + C::AT_JOIN) + warp * 512;
      if (i < n && part > 0) {
#pragma unroll
        for (int e = 0; e < 16; ++e) join[e * 32 + lane] = m.o[e];
        if (lane == 0) sh->join[warp] = make_float2(m.mx, m.tot);
      }
      __syncthreads();
      if (i < n && part == 0) {
#pragma unroll 1
        for (int x = 1; x < share; ++x) {              // in order: the result does not depend on timing
          const float2 mt = sh->join[warp + x];
          if (mt.y == 0.f) continue;                   // no key with a weight
          merge_scale(m, fmaxf(m.mx, mt.x));
          const float w = mt.x == -kInf ? 0.f : ex2(mt.x - m.mx);
          m.tot = fmaf(w, mt.y, m.tot);
#pragma unroll
          for (int e = 0; e < 16; ++e) m.o[e] = fmaf(w, join[x * 512 + e * 32 + lane], m.o[e]);
        }
      }
    }
    if (i < n && part == 0) finish(i);
    if (share > 1 || i + kOutWarps >= n) break;
  }
  fence_async_smem();
  tc_fence_before();
  const bool stop = __syncthreads_or(dead ? 1 : 0) != 0;   // an earlier kernel timed out
  tc_fence_after();
  const uint32_t tmem = sh->tmem;
  volatile int never = 0;
  if (warp == 0) {
    if (elect_one()) {
      // (What was loaded lands before the CTA leaves, whether there is work or not.)
      const uint64_t a0 = sdesc(smem_u32(smem), 16, 1024), o0 = sdesc(smem_u32(smem + C::AT_O), 16, 1024);
      int loaded = RING;
      bool good = true;
#pragma unroll 1
      for (int kb = 0; kb < loaded; ++kb) {
        const int s = kb % RING;
        good = mbar_wait(smem_u32(&sh->full[s]), (kb / RING) & 1, p.status, &never) && good;
        if (stop || !good) continue;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f16_ss(tmem, a0 + s * (W_BLOCK >> 4) + kk * 2, o0 + kb * (O_BLOCK >> 4) + kk * 2,
                     idesc_bf16(128, 2 * NT, false, false), (kb | kk) != 0);
        if (RING < 8) {
          tc_commit(smem_u32(&sh->empty[s]));
          // The block before has been multiplied: its place takes the next one.
          if (kb >= 1 && loaded < 8) {
            good = mbar_wait(smem_u32(&sh->empty[(kb - 1) % RING]), ((kb - 1) / RING) & 1, p.status, &never);
            if (good) load_w(loaded++);
          }
        }
      }
      if (!good) sh->abort = 1;
      tc_commit(smem_u32(&sh->done));
    }
    __syncwarp();
  }
  const bool ok = mbar_wait_warp(smem_u32(&sh->done), 0, p.status, &never);
  tc_fence_after();
  if (warp < 4 && !stop && ok && *reinterpret_cast<volatile int*>(&sh->abort) == 0) {
    const int v = warp * 32;
    __nv_bfloat16* dst = out + (static_cast<long long>(t0) * p.H + h) * 128 + v + lane;
    uint32_t r[16], r2[16];
    tmem_ld16(tmem + (uint32_t(v) << 16), r);
    tmem_ld16(tmem + (uint32_t(v) << 16) + NT, r2);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < NT; ++i)
      if (i < n && sh->used[i] >= 0)
        dst[static_cast<long long>(i) * p.H * 128] = __float2bfloat16_rn(__uint_as_float(r[i]) + __uint_as_float(r2[i]));
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 2 * NT);
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

template <bool DENSE, int ROWS>
cudaError_t launch_attn(const CUtensorMap& q_map, const CUtensorMap& qr_map, const CUtensorMap& k_map,
                        const CUtensorMap& kr_map, const Q8Params& p, long long ctas, cudaStream_t stream) {
  cudaError_t e = opt_in_smem(q8_attn_kernel<DENSE, ROWS>, Shape<ROWS>::TOTAL);
  if (e != cudaSuccess) return e;
  const int threads = Shape<ROWS>::THREADS + (DENSE ? 0 : 32 * (kSparseProducers - 1));
  // Members of a piece read the same keys at the same time: as a cluster they
  // sit on neighbouring SMs, on one die, and share its half of L2.  (Left to the
  // order in which SMs became free, 64 x 128 heads took 376 us, not 320, when the
  // kernels before kept some SMs longer than others; now 284 either way.)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = Shape<ROWS>::TOTAL;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.members % 2 == 0 ? 2 : 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, q8_attn_kernel<DENSE, ROWS>, q_map, qr_map, k_map, kr_map, p);
}

template <int RING>
cudaError_t launch_out(const CUtensorMap& w_map, const Q8Params& p, const DecodeQ8Args& a, int rows, int tokens,
                       cudaStream_t stream) {
  cudaError_t e = opt_in_smem(q8_out_kernel<RING>, OutShape<RING>::TOTAL);
  if (e != cudaSuccess) return e;
  return launch_pdl(q8_out_kernel<RING>, dim3((a.T + tokens - 1) / tokens, a.H), dim3(32 * kOutWarps),
                    OutShape<RING>::TOTAL, stream, w_map, p, fast_divisor(p.members * rows), a.sink,
                    static_cast<__nv_bfloat16*>(a.out), a.lse, a.T, tokens);
}

// Query rows of a tile: as many as a sequence can fill, 16, 32 or 64.  (64
// sequences of 4096 to 16384 keys in tiles of 16, 32 and 64 rows: 87, 101, 109
// us with 16 heads and one token; 140, 104, 112 with two tokens; 255, 175, 122
// with four.  128 heads, 1 or 2 tokens: 516, 401, 284.)
int tile_rows(int H, int max_new) {
  const long long rows = static_cast<long long>(H) * max_new;
  return rows > 32 ? 64 : (rows > 16 ? 32 : 16);
}
// Row tiles that walk a piece together: those of one token's heads, eight at most.
int item_members(int H, int rows) { return std::min(8, (H + rows - 1) / rows); }

}  // namespace

DecodeQ8Layout decode_q8_layout(int T, int H, int pieces) {
  const size_t R = static_cast<size_t>(T) * H;
  DecodeQ8Layout L;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  L.head = take(sizeof(PlanHead));
  L.entries = take(sizeof(PlanEntry) * (static_cast<size_t>(T) + 1));
  L.q8 = take(R * 1152);
  L.q_scale = take(R * 4);
  // Slots: one for each piece and item.  Items: R / (rows of an item), and one
  // more for every sequence whose rows do not fill their last one (T sequences
  // at most).  For either number of rows, as max_new is not known here.
  size_t slot_rows = 0;
  for (int rows : {16, 32, 64}) {
    const size_t item = static_cast<size_t>(rows) * item_members(H, rows);
    const size_t items = (R + item - 1) / item + (H % static_cast<int>(item) == 0 ? 0 : T);
    slot_rows = std::max(slot_rows, (items + pieces) * item);
  }
  L.o_part = take(slot_rows * 512 * 2);
  L.meta = take(slot_rows * 8);
  L.total = off;
  return L;
}

int decode_q8_pieces(int B, int H, int max_new, int max_keys) {
  // One piece (of `members` CTAs) for the SMs at a time, as long as there is a tile for each.
  const int rows = tile_rows(H, std::max(1, max_new)), members = item_members(H, rows);
  const long long item = static_cast<long long>(rows) * members;
  const long long items = B * ((static_cast<long long>(std::max(1, max_new)) * H + item - 1) / item);
  const long long tiles = (static_cast<long long>(std::max(1, max_keys)) + BK - 1) / BK;
  return static_cast<int>(std::min<long long>(std::max(1, sm_count() / members), items * tiles));
}

cudaError_t launch_decode_q8(const DecodeQ8Args& a, cudaStream_t stream) {
  const int H = a.H, T = a.T;
  const long long R = static_cast<long long>(T) * H;
  if (T == 0) return cudaSuccess;
  const DecodeQ8Layout L = decode_q8_layout(T, H, a.pieces);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  uint8_t* q8 = ws + L.q8;
  float* q_scale = reinterpret_cast<float*>(ws + L.q_scale);
  const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const int rows = tile_rows(H, a.max_new), members = item_members(H, rows);

  CUtensorMap qa_map, wuk_map, u_map;
  if (!encode_2d(&qa_map, a.q, bf, static_cast<uint64_t>(H) * 192, T, static_cast<uint64_t>(H) * 384, 64, 128,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&wuk_map, a.w_uk, bf, 128, static_cast<uint64_t>(H) * 512, 256, 64, 256,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&u_map, q8, u8, static_cast<uint64_t>(H) * 1152, T, static_cast<uint64_t>(H) * 1152, 128, 128,
                 CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  PlanArgs plan;
  plan.head = reinterpret_cast<PlanHead*>(ws + L.head);
  plan.entries = reinterpret_cast<PlanEntry*>(ws + L.entries);
  plan.iro = a.iro;
  plan.cache_len = a.cache_len;
  plan.topk = a.topk;
  plan.B = a.B;
  plan.H = H;
  plan.T = T;
  plan.max_seq = std::min(a.max_seq, kMaxContext);
  plan.indices_stride = a.indices_stride;
  plan.sparse = a.indices != nullptr ? 1 : 0;
  plan.item_rows = rows * members;
  plan.status = a.status;
  cudaError_t e = opt_in_smem(q8_query_kernel, Q_SMEM_TOTAL);
  if (e != cudaSuccess) return e;
  e = launch_pdl(q8_query_kernel, dim3((T + 127) / 128, 2 * H + 2), dim3(kQThreads), Q_SMEM_TOTAL, stream, qa_map, wuk_map, u_map,
                 static_cast<const uint16_t*>(a.q), q8, q_scale, T, H, a.status, plan);
  if (e != cudaSuccess) return e;

  Q8Params p;
  p.head = plan.head;
  p.entries = plan.entries;
  p.q_scale = q_scale;
  p.kv_scales = a.kv_scales;
  p.kv_cache = static_cast<const uint8_t*>(a.kv_cache);
  p.page_table = a.page_table;
  p.indices = a.indices;
  p.o_part = reinterpret_cast<__half*>(ws + L.o_part);
  p.meta = reinterpret_cast<float2*>(ws + L.meta);
  p.indices_stride = a.indices_stride;
  p.num_pages = a.num_pages;
  p.max_pages = a.max_pages;
  p.cache_rows = a.num_pages * a.page_size;
  p.page = fast_divisor(a.page_size);
  p.block = fast_divisor(a.scale_block);
  p.H = H;
  p.R = static_cast<int>(R);
  p.T = T;
  p.pieces = a.pieces;
  p.members = members;
  p.box = run_rows(a.page_size);
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.status = a.status;
  // Runs of 32 rows or more by TMA, shorter ones row by row: pages of 32 take 345
  // us by TMA and 340 by rows with 64 sequences and 128 heads, 98 and 102 with 32
  // and 16; pages of 16 342 and 108 by rows (by TMA, in an earlier state in which
  // they took 346 and 106 by rows, 407 and 108).
  const bool dense = a.indices == nullptr && p.box >= 32;
  const uint64_t cache_rows = static_cast<uint64_t>(a.num_pages) * a.page_size;
  const uint32_t box = dense ? p.box : 8;
  CUtensorMap q_map, qr_map, k_map, kr_map;
  if (!encode_2d(&q_map, q8, u8, 1152, R, 1152, 128, rows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&qr_map, q8, u8, 1152, R, 1152, 64, rows, CU_TENSOR_MAP_SWIZZLE_64B) ||
      !encode_4d(&k_map, a.kv_cache, u8, {128, 8, 4, cache_rows / 8 > 0 ? cache_rows / 8 : 1}, {576, 128, 8 * 576},
                 {128, 8, 2, box / 8}, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&kr_map, a.kv_cache, u8, 576, cache_rows, 576, 64, box, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  const long long ctas = static_cast<long long>(a.pieces) * members;
  auto attend = [&](auto rows_of_tile) {
    constexpr int R = decltype(rows_of_tile)::value;
    return dense ? launch_attn<true, R>(q_map, qr_map, k_map, kr_map, p, ctas, stream)
                 : launch_attn<false, R>(q_map, qr_map, k_map, kr_map, p, ctas, stream);
  };
  if (rows == 64) e = attend(std::integral_constant<int, 64>());
  else if (rows == 32) e = attend(std::integral_constant<int, 32>());
  else e = attend(std::integral_constant<int, 16>());
  if (e != cudaSuccess) return e;

  CUtensorMap wuv_map;
  if (!encode_2d(&wuv_map, a.w_uv, bf, 512, static_cast<uint64_t>(H) * 128, 1024, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  // Tokens a CTA: as few as one wave of CTAs allows, 16 where it takes more.
  int tokens = 1;
  while (tokens < NT && static_cast<long long>(H) * ((T + tokens - 1) / tokens) > sm_count()) tokens *= 2;
  if (static_cast<long long>(H) * ((T + tokens - 1) / tokens) <= sm_count())
    return launch_out<8>(wuv_map, p, a, rows, tokens, stream);
  return launch_out<4>(wuv_map, p, a, rows, NT, stream);
}

}  // namespace mla
