// Key selection for sparse decode: a cheap score for every block of keys and
// new token, and the best blocks of every token as the list of physical cache
// rows that the sparse decode calls take.
//
// Scores: with index queries q[t][h] and one index key k_j per cached token
// (128 values each, kept in a paged cache of their own under the same page
// table),
//   score(t, i) = max over visible j in block i of s_j sum_h w[t][h] relu(q[t][h] . k_j).
#include <algorithm>

#include "kernels.cuh"

namespace mla {
namespace {

constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float max_nan(float a, float b) {   // a NaN wins
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

// acc += sum over 16 heads of relu(product) * weight.
__device__ __forceinline__ void weigh(const uint32_t (&d)[16], uint32_t weights, float2& acc) {
  float2 a1 = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < 16; k += 4) {
    const float4 wv = ld_shared_f4(weights + 4 * k);
    acc = __ffma2_rn(make_float2(max_nan(__uint_as_float(d[k]), 0.f), max_nan(__uint_as_float(d[k + 1]), 0.f)),
                     make_float2(wv.x, wv.y), acc);
    a1 = __ffma2_rn(make_float2(max_nan(__uint_as_float(d[k + 2]), 0.f), max_nan(__uint_as_float(d[k + 3]), 0.f)),
                    make_float2(wv.z, wv.w), a1);
  }
  acc = __fadd2_rn(acc, a1);
}

__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// ============================================================ scores
// Keys are the M side of the MMA (128 keys a tile) and the heads of a batch of
// tokens the N side (K = 128), so a thread of the epilogue holds one key's
// products with all of them in its own TMEM lane and the weighted sums need no
// other thread.  One CTA per (sequence, group of its new tokens, range of
// positions): the group's queries stay in shared memory, key tiles stream
// through a ring, and the two epilogue warpgroups take the (tile, batch) units
// in turn, each with its own TMEM buffer of up to 128 columns.  Two CTAs share
// an SM, one's start under the other's work.
//
// With one new token a sequence the call is bound by reading the keys: 64
// sequences of 4096 to 16384 keys, 64 heads, bf16, 35 us (4.9 TB/s).  With
// more it is bound by the epilogue, which takes a maximum and half a packed FMA
// for every product on the CUDA cores: about 1000 tokens, 32 heads, 8000 8-bit
// keys, blocks of 64, 77 us (3.2 T products/s; 37 us with the epilogue's inner
// loop taken out).  A batch of tokens therefore fills a buffer, so that an
// MMA's latency (some 600 clk to its barrier) is paid once for all of them
// (batches half as large, with two buffers a warpgroup, took 24 % longer), and
// the loop stays small: four chunks in flight in a warp took 18 % longer than two.
constexpr int IT = 128;                             // keys of a tile
constexpr int I_QMAX = 32 * 1024;                   // query bytes of a group with several tokens, at most
constexpr int GROUPS = 2;                           // epilogue warpgroups and TMEM buffers
constexpr int kScoreThreads = 64 + 128 * GROUPS;    // producer, MMA and epilogue warps
constexpr int I_MAXG = 16;                          // tokens of a group at most
constexpr int I_MAXSTAGES = 8;

struct ScoreSmem {
  uint64_t k_full[I_MAXSTAGES], k_empty[I_MAXSTAGES], q_full, d_full[2], d_free[2], drain;
  uint32_t tmem;
  int abort;
  unsigned long long sum[kScoreThreads / 32];   // the split of the work among the CTAs
  int scan[kScoreThreads / 32], seq, nth, runs;
  float part[2][2][8][4];         // [warpgroup][unit & 1][token][warp]: maxima, for blocks of more than 32 keys
};
constexpr int I_BAR = 1024;
static_assert(sizeof(ScoreSmem) <= I_BAR, "barrier block");

struct ScoreParams {
  float* scores;
  const float* w;
  const uint8_t* keys;
  const float* key_scales;
  const uint32_t* iro;
  const uint32_t* cache_len;
  const int32_t* page_table;
  FastDiv page;
  int num_pages, max_pages, block, B, Hi, NP, T, max_new, groups, places, shares, max_seq, stride, box;
  int G, batch;              // tokens of a group and of an MMA
  int stages, cols;          // ring stages, TMEM columns allocated
  int at_w, at_ring, at_bar; // shared memory: queries, weights [G][NP], ring, barriers
  int32_t* status;
};

__device__ __forceinline__ int score_row(const ScoreParams& p, int b, int pos) {
  const int pi = fast_div(pos, p.page);
  const int page = pi < p.max_pages ? __ldg(p.page_table + static_cast<long long>(b) * p.max_pages + pi) : -1;
  if (page >= 0 && page < p.num_pages) return page * p.page.d + (pos - pi * p.page.d);
  set_status(p.status, MLA_DEV_BAD_PAGE);
  return -1;
}

// A sequence's groups of new tokens and tiles of keys; none if it is left out.
struct Scored {
  int groups, tiles;
};
__device__ __forceinline__ Scored scored(const ScoreParams& p, int b, bool report) {
  const uint32_t qa = __ldg(p.iro + b), qe = __ldg(p.iro + b + 1), cached = __ldg(p.cache_len + b);
  if (qe <= qa) {
    if (report && qe < qa) set_status(p.status, MLA_DEV_BAD_OFFSETS);
    return {0, 0};
  }
  const uint64_t ctx = static_cast<uint64_t>(cached) + (qe - qa);
  if (qe > static_cast<uint32_t>(p.T) || ctx > static_cast<uint64_t>(p.max_seq)) {
    if (report) set_status(p.status, MLA_DEV_BAD_OFFSETS);
    return {0, 0};
  }
  const int n = static_cast<int>(min(qe - qa, static_cast<uint32_t>(p.max_new)));
  return {(n + p.G - 1) / p.G, static_cast<int>((ctx + IT - 1) / IT)};
}

template <bool E8, bool DENSE>
__global__ void __launch_bounds__(kScoreThreads, 2)
    index_scores_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                        const ScoreParams p) {
  constexpr int KB = E8 ? 1 : 2;                    // 128-byte blocks of a row
  constexpr int ELT = E8 ? 1 : 2;
  constexpr int STAGE = KB * IT * 128;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  ScoreSmem* sh = reinterpret_cast<ScoreSmem*>(smem + p.at_bar);
  float* sw = reinterpret_cast<float*>(smem + p.at_w);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_enter();

  // ---- this CTA's sequence, group and run of tiles
  int b, nth = blockIdx.x, runs = 1, span = 0x7FFFFFFF;
  if (p.places == 0) {                               // many pairs of sequence and group: a CTA each
    b = nth / p.groups;
    nth -= b * p.groups;
    if (nth == 0 && threadIdx.x == 0) scored(p, b, true);
  } else {
    unsigned long long total = 0;
    for (int i = threadIdx.x; i < p.B; i += kScoreThreads) {
      const Scored w = scored(p, i, blockIdx.x == 0);
      total += static_cast<unsigned long long>(w.groups) * w.tiles;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    if (lane == 0) sh->sum[warp] = total;
    if (threadIdx.x == 0) sh->seq = -1;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kScoreThreads / 32; ++w) total += sh->sum[w];
    // Tiles of a run: an equal share, eight at least (a start costs about three).
    // In fp32, rounded up by one: every CTA gets the same number.
    span = max(8, static_cast<int>(fminf(__fdividef(static_cast<float>(total), static_cast<float>(p.shares)), 1e9f)) + 1);
    int base = 0;
    for (int i0 = 0; i0 < p.B && base <= nth; i0 += kScoreThreads) {
      Scored w = {0, 0};
      if (i0 + static_cast<int>(threadIdx.x) < p.B) w = scored(p, i0 + threadIdx.x, false);
      const int each = (w.tiles + span - 1) / span, mine = w.groups * each;
      int incl = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
      }
      if (lane == 31) sh->scan[warp] = incl;
      __syncthreads();
      int before = base;
      for (int w2 = 0; w2 < kScoreThreads / 32; ++w2) {
        if (w2 < warp) before += sh->scan[w2];
        base += sh->scan[w2];
      }
      before += incl - mine;
      if (before <= nth && nth < before + mine) {
        sh->seq = i0 + threadIdx.x;
        sh->nth = nth - before;
        sh->runs = each;
      }
      __syncthreads();
    }
    b = sh->seq;
    nth = sh->nth;
    runs = sh->runs;
    if (b < 0) return;                               // fewer runs than CTAs
  }
  const Scored work = scored(p, b, false);
  const int g = nth / runs, sp = nth - g * runs;
  if (g >= work.groups) return;
  const int n_new = static_cast<int>(min(p.iro[b + 1] - p.iro[b], static_cast<uint32_t>(p.max_new)));
  const int i0 = g * p.G;
  const int ng = min(p.G, n_new - i0);
  const int t0 = static_cast<int>(p.iro[b]) + i0;
  const int pos_first = static_cast<int>(p.cache_len[b]) + i0;   // position of the group's first token
  const int pos_last = pos_first + ng - 1;
  // Runs of a pair differ by one tile at most.
  const int each = work.tiles / runs, more = work.tiles - each * runs;
  const int tile0 = each * sp + min(sp, more), tiles = each + (sp < more ? 1 : 0);
  const long long base0 = static_cast<long long>(tile0) * IT;
  const int n = base0 > pos_last ? 0 : static_cast<int>(min(static_cast<long long>(tiles), (pos_last - base0) / IT + 1));
  const int batches = (ng + p.batch - 1) / p.batch;

  if (n > 0) {
    if (threadIdx.x == 0) {
      for (int s = 0; s < p.stages; ++s) {
        mbar_init(smem_u32(&sh->k_full[s]), 1);
        mbar_init(smem_u32(&sh->k_empty[s]), 1);
      }
      mbar_init(smem_u32(&sh->q_full), 1);
      for (int i = 0; i < GROUPS; ++i) {
        mbar_init(smem_u32(&sh->d_full[i]), 1);
        mbar_init(smem_u32(&sh->d_free[i]), 4);
      }
      mbar_init(smem_u32(&sh->drain), 1);
      sh->abort = timed_out_before(p.status) ? 1 : 0;
      fence_mbar_init();
    }
    if (warp == 1) {
      tmem_alloc(smem_u32(&sh->tmem), p.cols);
      tmem_relinquish();
    }
    // The group's weights, heads past the last one zero.
    for (int i = warp; i < ng; i += kScoreThreads / 32)
      for (int h = lane; h < p.NP; h += 32)
        sw[i * p.NP + h] = h < p.Hi ? __ldg(p.w + static_cast<long long>(t0 + i) * p.Hi + h) : 0.f;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    volatile int* abort_flag = &sh->abort;
    const bool dead = sh->abort != 0;                  // an earlier kernel timed out: no work
    __syncthreads();                                   // the flag may be raised from here on

    if (dead) {
    } else if (warp == 0) {
      // ---------------------------------------------------------- producer
      if (elect_one()) {
        const uint32_t qf = smem_u32(&sh->q_full);
        mbar_expect_tx(qf, ng * KB * p.NP * 128);
#pragma unroll 1
        for (int i = 0; i < ng; ++i)
#pragma unroll
          for (int c = 0; c < KB; ++c)
            tma_load_2d(smem_u32(smem) + (c * p.G + i) * p.NP * 128, &q_map, qf, c * (128 / ELT), (t0 + i) * p.Hi);
      }
      __syncwarp();
      bool ok = true;
      uint32_t issued = 0;
      int pend = -1;
      int s = 0, turn = 0;
#pragma unroll 1
      for (int j = 0; j < n && ok; ++j) {
        const int pos0 = static_cast<int>(base0) + j * IT;
        const uint32_t full = smem_u32(&sh->k_full[s]);
        const uint32_t dst = smem_u32(smem) + p.at_ring + s * STAGE;
        const int have = min(IT, pos_last + 1 - pos0);   // keys that some token sees
        if constexpr (DENSE) {
          const int boxes = (have + p.box - 1) / p.box;
          int row = 0;
          if (lane < boxes) {
            row = score_row(p, b, pos0 + lane * p.box);
            if (row < 0) row = p.num_pages * p.page.d;   // past the end: reads zeros
          }
          if (turn > 0 && !(ok = mbar_wait_warp(smem_u32(&sh->k_empty[s]), (turn & 1) ^ 1, p.status, abort_flag))) break;
          if (lane == 0) mbar_expect_tx(full, boxes * p.box * 128 * KB);
          __syncwarp();
          if (lane < boxes)
            for (int c = 0; c < KB; ++c)
              tma_load_2d(dst + c * IT * 128 + lane * p.box * 128, &k_map, full, c * (128 / ELT), row);
          __syncwarp();
        } else {
          int row[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            row[x] = 32 * x + lane < have ? score_row(p, b, pos0 + 32 * x + lane) : 0;
            if (row[x] < 0) row[x] = 0;                    // reported
          }
          if (turn > 0) {
            // The ring is full: what was copied has to be counted before waiting.
            if (pend >= 0) {
              cp_async_wait<0>();
              fence_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&sh->k_full[pend]));
              pend = -1;
            }
            if (!(ok = mbar_wait_warp(smem_u32(&sh->k_empty[s]), (turn & 1) ^ 1, p.status, abort_flag))) break;
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int r = 4 * i + (lane >> 3), ch = lane & 7;
            const int src = __shfl_sync(0xffffffffu, row[i / 8], r & 31);
#pragma unroll
            for (int c = 0; c < KB; ++c)
              cp_async16(dst + c * IT * 128 + r * 128 + ((ch ^ (r & 7)) << 4),
                         p.keys + static_cast<size_t>(src) * (128 * KB) + c * 128 + ch * 16);
          }
          cp_async_commit();
          if (pend >= 0) {
            cp_async_wait<1>();
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh->k_full[pend]));
          }
          pend = s;
        }
        ++issued;
        if (++s == p.stages) {
          s = 0;
          ++turn;
        }
      }
      if constexpr (!DENSE) {
        cp_async_wait<0>();
        fence_async_smem();
        __syncwarp();
        if (pend >= 0 && lane == 0) mbar_arrive(smem_u32(&sh->k_full[pend]));
      }
      volatile int never = 0;
      mbar_wait_warp(smem_u32(&sh->q_full), 0, p.status, &never);
      for (int x = 0; x < p.stages; ++x) {
        const int uses = turn + (x < s ? 1 : 0);
        if (uses > 0) mbar_wait_warp(smem_u32(&sh->k_full[x]), (uses - 1) & 1, p.status, &never);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      if (elect_one()) {
        bool ok = mbar_wait(smem_u32(&sh->q_full), 0, p.status, abort_flag);
        const uint64_t q0 = sdesc(smem_u32(smem), 16, 1024), k0 = sdesc(smem_u32(smem) + p.at_ring, 16, 1024);
        const uint32_t qblock = static_cast<uint32_t>(p.G * p.NP * 128) >> 4;
        uint32_t u = 0;
        int s = 0, turn = 0;
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j) {
          if (!(ok = mbar_wait(smem_u32(&sh->k_full[s]), turn & 1, p.status, abort_flag))) break;
          tc_fence_after();
          const uint64_t ad = k0 + s * (STAGE >> 4);
#pragma unroll 1
          for (int i = 0; i < batches; ++i, ++u) {
            const uint32_t buf = u % GROUPS;
            if (u >= GROUPS && !(ok = mbar_wait(smem_u32(&sh->d_free[buf]), ((u / GROUPS) & 1) ^ 1, p.status, abort_flag))) break;
            tc_fence_after();
            const int cols = min(p.batch, ng - i * p.batch) * p.NP;
            const uint32_t idesc = E8 ? idesc_e4m3(128, cols, false, false) : idesc_bf16(128, cols, false, false);
            const uint32_t d = tmem + buf * (p.cols / GROUPS);
            const uint64_t bd = q0 + static_cast<uint32_t>(i * p.batch * p.NP * 128 >> 4);
#pragma unroll
            for (int c = 0; c < KB; ++c)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                if (E8) mma_f8_ss(d, ad + kk * 2, bd + kk * 2, idesc, kk != 0);
                else mma_f16_ss(d, ad + c * (IT * 128 >> 4) + kk * 2, bd + c * qblock + kk * 2, idesc, (c | kk) != 0);
              }
            tc_commit(smem_u32(&sh->d_full[buf]));
          }
          tc_commit(smem_u32(&sh->k_empty[s]));
          if (++s == p.stages) {
            s = 0;
            ++turn;
          }
        }
        tc_commit(smem_u32(&sh->drain));
        volatile int never = 0;
        mbar_wait(smem_u32(&sh->drain), 0, p.status, &never);
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------- weighted sums
      const int e = (warp - 2) >> 2;                   // warpgroup: units u with u % GROUPS == e
      const int q4 = warp & 3;
      const int key = q4 * 32 + lane;
      const int tid = threadIdx.x - 64 - 128 * e;
      const uint32_t ta = tmem + (uint32_t(q4 * 32) << 16) + e * (p.cols / GROUPS);
      const int shift = __ffs(p.block) - 1;
      const bool pair = p.batch > 1;                   // two tokens a turn
      uint32_t mine = 0;
      int j = e / batches, i = e - j * batches;        // tile and batch of the unit
      // This key's scale in the unit's tile is read a unit ahead, its page id two.
      const int32_t* table = p.page_table + static_cast<long long>(b) * p.max_pages;
      struct Where {
        int page, slot;       // slot -1: no key of the call, or no scales
      };
      auto where = [&](int tile) -> Where {
        const int pos = static_cast<int>(base0) + tile * IT + key;
        if (p.key_scales == nullptr || tile >= n || pos > pos_last) return {0, -1};
        const int pi = fast_div(pos, p.page);
        return {pi < p.max_pages ? __ldg(table + pi) : -1, pos - pi * p.page.d};
      };
      auto scale_of = [&](const Where& w) -> float {
        if (w.slot < 0) return 1.f;
        if (w.page >= 0 && w.page < p.num_pages) return __ldg(p.key_scales + w.page * p.page.d + w.slot);
        set_status(p.status, MLA_DEV_BAD_PAGE);
        return 1.f;
      };
      // The tile (and batch) of the warpgroup's next unit.
      auto step = [&](int& tile, int& batch) {
        for (batch += GROUPS; batch >= batches; batch -= batches) ++tile;
      };
      float next = scale_of(where(j));
      int j1 = j, i1 = i;
      step(j1, i1);
      Where at = where(j1);
#pragma unroll 1
      while (j < n) {
        const int pos = static_cast<int>(base0) + j * IT + key;
        const float ks = next;
        next = scale_of(at);
        int j2 = j1, i2 = i1;
        step(j2, i2);
        at = where(j2);
        const bool ok = mbar_wait_warp(smem_u32(&sh->d_full[e]), mine & 1, p.status, abort_flag);
        ++mine;
        tc_fence_after();
        const int tok0 = i * p.batch, toks = ok ? min(p.batch, ng - tok0) : 0;
        // Two chunks of 16 columns at a time, of two tokens or, in batches of one,
        // of the same: two chains in flight in each of the warps.
#pragma unroll 1
        for (int y0 = 0; y0 < toks; y0 += pair ? 2 : 1) {
          const int other = pair ? (y0 + 1 < toks ? p.NP : 0) : 16;   // columns to the second chunk
          const uint32_t col = ta + y0 * p.NP, w = smem_u32(sw) + (tok0 + y0) * p.NP * 4;
          float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
          for (int c = 0; c < p.Hi; c += pair ? 16 : 32) {
            const bool both = pair || c + 16 < p.Hi;
            uint32_t d[2][16];
            tmem_ld16(col + c, d[0]);
            tmem_ld16(col + c + (both ? other : 0), d[1]);
            tmem_ld_wait();
            if (__builtin_expect(p.Hi - c < (pair ? 16 : 32), 0)) {
              // Columns past the last head hold the next token's products.
              const int h0 = p.Hi - c, h1 = pair ? h0 : h0 - 16;
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                if (k >= h0) d[0][k] = 0u;
                if (k >= h1) d[1][k] = 0u;
              }
            }
            weigh(d[0], w + 4 * c, acc[0]);
            if (both) weigh(d[1], w + 4 * (c + other), acc[1]);
          }
          float v0 = acc[0].x + acc[0].y, v1 = acc[1].x + acc[1].y;
          if (!pair) v0 += v1;
          v0 *= ks;
          v1 *= ks;
          const int ahead = pos - (pos_first + tok0 + y0);   // not visible to the token
          if (ahead > 0) v0 = -kInf;
          if (ahead > 1) v1 = -kInf;
          if (p.block >= 32) {
            v0 = warp_max_nan(v0);
            if (pair) v1 = warp_max_nan(v1);
          } else {
#pragma unroll 1
            for (int r = 1; r < p.block; r <<= 1) {
              v0 = max_nan(v0, __shfl_xor_sync(0xffffffffu, v0, r));
              v1 = max_nan(v1, __shfl_xor_sync(0xffffffffu, v1, r));
            }
          }
          const bool second = pair && y0 + 1 < toks;
          if (p.block > 32) {
            if (lane == 0) {
              sh->part[e][mine & 1][y0][q4] = v0;
              if (second) sh->part[e][mine & 1][y0 + 1][q4] = v1;
            }
          } else if ((lane & (p.block - 1)) == 0 && (pos >> shift) < p.stride) {
            float* dst = p.scores + static_cast<long long>(t0 + tok0 + y0) * p.stride + (pos >> shift);
            dst[0] = v0;
            if (second) dst[p.stride] = v1;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(smem_u32(&sh->d_free[e]));
        if (p.block > 32) {
          // Blocks of 64 or 128 keys: two or four warps' maxima, a thread for
          // each token and block.  (Its warps leave this loop together: a wait
          // that ran out in one of them is known to the others by the barrier.)
          const int blocks = IT >> shift, warps = p.block >> 5;
          int bad;
          asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\t"
                       "barrier.cta.red.or.pred.aligned q, %2, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
                       : "=r"(bad) : "r"(ok ? 0 : 1), "r"(e + 1) : "memory");
          const int y = tid >> (7 - shift), x = tid & (blocks - 1);
          if (y < toks) {
            float m = sh->part[e][mine & 1][y][x * warps];
#pragma unroll 1
            for (int k = 1; k < warps; ++k) m = max_nan(m, sh->part[e][mine & 1][y][x * warps + k]);
            const int at = ((static_cast<int>(base0) + j * IT) >> shift) + x;
            if (at < p.stride) p.scores[static_cast<long long>(t0 + tok0 + y) * p.stride + at] = m;
          }
          if (bad) break;
        } else if (!ok) {
          break;
        }
        j = j1;
        i = i1;
        j1 = j2;
        i1 = i2;
      }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
      tc_fence_after();
      tmem_dealloc(tmem, p.cols);
    }
    if (dead) return;
  } else if (timed_out_before(p.status)) {
    return;
  }
  // Blocks past the run's last key, and a share of those past the sequence's
  // last tile: -infinity.
  const int shift = __ffs(p.block) - 1;
  auto fill = [&](long long from, long long to) {
    to = min(to, static_cast<long long>(p.stride));
    for (int i = warp; i < ng; i += kScoreThreads / 32)
      for (long long x = from + lane; x < to; x += 32) p.scores[static_cast<long long>(t0 + i) * p.stride + x] = -kInf;
  };
  fill((base0 + static_cast<long long>(n) * IT) >> shift, (base0 + static_cast<long long>(tiles) * IT) >> shift);
  const long long end = static_cast<long long>(work.tiles) * IT >> shift;
  if (end < p.stride) {
    const int rest = p.stride - static_cast<int>(end), part = rest / runs + 1;   // (the last shares may be empty)
    fill(end + static_cast<long long>(part) * sp, end + static_cast<long long>(part) * (sp + 1));
  }
}

// ============================================================ selection
// A cluster of CTAs per token, each with a contiguous slice of the token's
// block scores (kept in shared memory where it fits).  The k-th largest score
// is found digit by digit (four of 8 bits of an order-preserving integer,
// histograms summed over the cluster through distributed shared memory), then
// the chosen blocks are written in position order: those above it, and as many
// equal to it as are missing, lowest first.
//
// Bound by latency: a chain of barriers, and reads of other CTAs' counters.
// Digits of 8 bits keep those few: with 2048 counters (three passes) a cluster
// of eight spent 9000 clk of each pass on reading them.
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelMaxCluster = 16;
constexpr int kSelCacheFloats = 40 * 1024;           // slice kept in shared memory, 160 KB

struct SelectSmem {
  uint32_t hist[4][256];
  uint32_t scan[8];
  uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
  uint32_t total[2];           // chosen-for-sure and equal blocks of this CTA
  uint32_t bin, need, whole;   // whole: all keys of the digit are chosen
  int seq, pos;
};

__device__ __forceinline__ uint32_t select_key(float s) {
  if (s != s) s = -kInf;                             // NaN counts as -infinity
  const uint32_t u = __float_as_uint(s + 0.0f);      // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t ld_cluster_u32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(smem_u32(p), rank)) : "memory");
  return v;
}

__global__ void __launch_bounds__(kSelThreads)
    index_select_kernel(const IndexSelectArgs a, const FastDiv page, int cached) {
  extern __shared__ __align__(16) uint32_t cache[];
  __shared__ SelectSmem sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t C = cluster_size(), rank = cluster_rank();
  const int t = blockIdx.x / C;
  (&sh.hist[0][0])[tid] = 0u;
  pdl_enter();
  // Decreasing offsets are reported once (the search below reads the same words).
  if (blockIdx.x == 0)
    for (int x = tid; x < a.B; x += kSelThreads)
      if (__ldg(a.iro + x + 1) < __ldg(a.iro + x)) set_status(a.status, MLA_DEV_BAD_OFFSETS);
  // The token's sequence: the last b with iro[b] <= t, 1024 probes at a time.
  int b = 0;
  for (int end = a.B; end - b > 1;) {
    const int step = (end - b + kSelThreads - 1) / kSelThreads;
    const int x = static_cast<int>(min(static_cast<long long>(b) + static_cast<long long>(tid) * step, 0x7FFFFFFFll));
    const int below = __syncthreads_count(x < end && __ldg(a.iro + x) <= static_cast<uint32_t>(t));
    b += max(below - 1, 0) * step;
    end = min(end, b + step);
  }
  if (tid == 0) {
    int seq = -1, pos = 0;
    if (!timed_out_before(a.status)) {
      const uint32_t qa = __ldg(a.iro + b), qe = __ldg(a.iro + b + 1), cached_tokens = __ldg(a.cache_len + b);
      if (qa <= static_cast<uint32_t>(t) && static_cast<uint32_t>(t) < qe) {
        // (The whole sequence's context: the scores leave it out as one.)
        const uint64_t ctx = static_cast<uint64_t>(cached_tokens) + (qe - qa);
        if (ctx <= static_cast<uint64_t>(a.max_seq) && qe <= static_cast<uint32_t>(a.T)) {
          seq = b;
          pos = static_cast<int>(cached_tokens + (static_cast<uint32_t>(t) - qa));
        } else {
          set_status(a.status, MLA_DEV_BAD_OFFSETS);
        }
      }
    }
    sh.seq = seq;
    sh.pos = pos;
  }
  cluster_sync();
  // The token's sequence is read from CTA 0, so that all CTAs agree.
  const int seq = static_cast<int>(ld_cluster_u32(&sh.seq, 0)), pos = static_cast<int>(ld_cluster_u32(&sh.pos, 0));
  if (seq < 0) {                                     // outside every sequence: left as it was
    cluster_sync();
    return;
  }
  const int nb = pos / a.block + 1;                  // visible blocks
  const int k = min(a.top, nb);
  const int slice = ((nb + static_cast<int>(C) - 1) / static_cast<int>(C) + 31) / 32 * 32;
  const int lo = min(nb, static_cast<int>(rank) * slice), cnt = min(nb, lo + slice) - lo;
  const float* src = a.scores + static_cast<long long>(t) * a.stride + lo;
  const int local_from = nb - a.local - lo;          // slice index of the first always-chosen block
  auto load = [&](int i) -> uint32_t { return i >= local_from ? 0xFFFFFFFFu : select_key(__ldg(src + i)); };
  // Keys i .. i + 3 (i is a multiple of 4); 0, below every key, past the slice.
  auto quad = [&](int i, uint32_t (&u)[4]) {
    if (cached) {
      const uint4 v = *reinterpret_cast<const uint4*>(cache + i);
      u[0] = v.x; u[1] = v.y; u[2] = v.z; u[3] = v.w;
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (i + x >= cnt) u[x] = 0u;
      else if (!cached) u[x] = load(i + x);
    }
  };

  if (cached || k < nb) {
    // The first digit's counts, and the slice into shared memory.
    constexpr int U = 4;                             // loads in flight
    for (int i0 = tid; i0 < cnt; i0 += U * kSelThreads) {
      uint32_t u[U];
#pragma unroll
      for (int x = 0; x < U; ++x) u[x] = i0 + x * kSelThreads < cnt ? load(i0 + x * kSelThreads) : 0u;
#pragma unroll
      for (int x = 0; x < U; ++x) {
        if (i0 + x * kSelThreads < cnt) {
          if (cached) cache[i0 + x * kSelThreads] = u[x];
          if (k < nb) atomicAdd(&sh.hist[0][u[x] >> 24], 1u);
        }
      }
    }
  }
  uint32_t thr = 0u, need = 0u;
  if (k < nb) {
    need = k;
    uint32_t mask = 0u;
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      uint32_t* hist = sh.hist[pass];
      if (pass > 0)
        for (int i = 4 * tid; i < cnt; i += 4 * kSelThreads) {
          uint32_t u[4];
          quad(i, u);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (i + x < cnt && (u[x] & mask) == thr) atomicAdd(&hist[(u[x] >> shift) & 255u], 1u);
        }
      cluster_sync();
      // A digit a thread, from the largest down: the cluster's count of it and
      // how many keys have a larger one.
      uint32_t c = 0, before = 0;
      if (tid < 256) {
        uint32_t v[kSelMaxCluster];
#pragma unroll
        for (uint32_t r = 0; r < kSelMaxCluster; ++r) {
          v[r] = 0;
          if (r < C) v[r] = ld_cluster_u32(hist + 255 - tid, r);
        }
#pragma unroll
        for (uint32_t r = 0; r < kSelMaxCluster; ++r) c += v[r];
        uint32_t incl = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += o;
        }
        if (lane == 31) sh.scan[warp] = incl;
        before = incl - c;
        asm volatile("barrier.cta.sync.aligned 1, 256;" ::: "memory");
#pragma unroll
        for (int w = 0; w < 8; ++w) before += w < warp ? sh.scan[w] : 0u;
        if (before < need && need <= before + c) {
          sh.bin = 255 - tid;
          sh.need = need - before;
          sh.whole = need - before == c ? 1u : 0u;
        }
      }
      __syncthreads();
      thr |= sh.bin << shift;
      need = sh.need;
      mask |= 255u << shift;
      if (sh.whole != 0u && thr != 0u) {               // nothing to tell apart: the last pass is mostly spared
        thr -= 1u;
        need = 0u;
        break;
      }
    }
  } else {
    __syncthreads();                                 // the slice is in shared memory
  }

  // Chosen and equal blocks before each warp's part of the slice.
  const int seg = ((cnt + kSelWarps - 1) / kSelWarps + 127) / 128 * 128;
  const int s0 = min(cnt, warp * seg), s1 = min(cnt, s0 + seg);
  uint32_t gt = 0, eq = 0;
  for (int i = s0 + 4 * lane; i < s1; i += 128) {
    uint32_t u[4];
    quad(i, u);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      gt += i + x < cnt && u[x] > thr ? 1u : 0u;
      eq += i + x < cnt && u[x] == thr ? 1u : 0u;
    }
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    sh.warp_gt[warp] = gt;
    sh.warp_eq[warp] = eq;
  }
  __syncthreads();
  gt = sh.warp_gt[lane];
  eq = sh.warp_eq[lane];
  if (warp == 0) {
    const uint32_t x = __reduce_add_sync(0xffffffffu, gt), y = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
      sh.total[0] = x;
      sh.total[1] = y;
    }
  }
  gt = __reduce_add_sync(0xffffffffu, lane < warp ? gt : 0u);
  eq = __reduce_add_sync(0xffffffffu, lane < warp ? eq : 0u);
  cluster_sync();
  {
    const bool other = lane < static_cast<int>(rank);
    const uint32_t x = other ? ld_cluster_u32(&sh.total[0], lane) : 0u, y = other ? ld_cluster_u32(&sh.total[1], lane) : 0u;
    gt += __reduce_add_sync(0xffffffffu, x);
    eq += __reduce_add_sync(0xffffffffu, y);
  }

  int32_t* out = a.rows + static_cast<long long>(t) * a.rows_stride;
  const int32_t* table = a.page_table + static_cast<long long>(seq) * a.max_pages;
  auto entry_of = [&](int pi) -> int { return pi < a.max_pages ? __ldg(table + pi) : -1; };
  auto row_of = [&](int x, int pi, int entry) -> int32_t {
    if (entry >= 0 && entry < a.num_pages) return entry * page.d + (x - pi * page.d);
    set_status(a.status, MLA_DEV_BAD_PAGE);
    return -1;
  };
  // Single keys: the page id of a lane's first key is read an iteration ahead.
  int pi_next = 0, entry_next = -1;
  auto ahead = [&](int i) {
    if (a.block == 1 && i < s1) {
      pi_next = fast_div(lo + i, page);
      entry_next = entry_of(pi_next);
    }
  };
  ahead(s0 + 4 * lane);
#pragma unroll 1
  for (int i0 = s0; i0 < s1; i0 += 128) {
    const int i = i0 + 4 * lane;
    const int pi0 = pi_next, entry0 = entry_next;
    ahead(i + 128);
    uint32_t u[4];
    quad(i, u);
    uint32_t mine = 0;                               // above, and equal << 16
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (i + x < cnt) mine += u[x] > thr ? 1u : (u[x] == thr ? 0x10000u : 0u);
    uint32_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    uint32_t g = gt + ((incl - mine) & 0xFFFFu), e = eq + ((incl - mine) >> 16);
    const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const bool in = i + x < cnt, above = in && u[x] > thr, equal = in && u[x] == thr;
      const bool chosen = above || (equal && e < need);
      const uint32_t at = g + min(e, need);          // chosen blocks before
      g += above ? 1 : 0;
      e += equal ? 1 : 0;
      if (a.block == 1) {
        if (chosen) {
          const int key = lo + i + x, pi = x == 0 ? pi0 : fast_div(key, page);
          out[at] = row_of(key, pi, pi == pi0 ? entry0 : entry_of(pi));
        }
      } else {
        uint32_t todo = __ballot_sync(0xffffffffu, chosen);
        while (todo) {
          const int from = __ffs(todo) - 1;
          todo &= todo - 1;
          const long long o = static_cast<long long>(__shfl_sync(0xffffffffu, at, from)) * a.block;
          const int first = (lo + i0 + 4 * from + x) * a.block;
          for (int r = lane; r < a.block; r += 32) {
            const int key = first + r, pi = fast_div(key, page);
            out[o + r] = key <= pos ? row_of(key, pi, entry_of(pi)) : -1;
          }
        }
      }
      // The last visible block may be cut by the token's position.
      if (in && lo + i + x == nb - 1) a.count[t] = chosen ? (k - 1) * a.block + pos % a.block + 1 : k * a.block;
    }
    gt += all & 0xFFFFu;
    eq += all >> 16;
  }
  for (long long x = static_cast<long long>(k) * a.block + rank * kSelThreads + tid; x < a.rows_stride; x += C * kSelThreads)
    out[x] = -1;
  cluster_sync();   // no CTA leaves while another may read its counts
}

}  // namespace

cudaError_t launch_index_scores(const IndexScoresArgs& a, cudaStream_t stream) {
  if (a.T == 0 || a.max_new == 0) return cudaSuccess;
  const bool e8 = a.dtype == MLA_E4M3;
  const int kb = e8 ? 1 : 2;
  ScoreParams p;
  p.scores = a.scores;
  p.w = a.w;
  p.keys = static_cast<const uint8_t*>(a.keys);
  p.key_scales = a.key_scales;
  p.iro = a.iro;
  p.cache_len = a.cache_len;
  p.page_table = a.page_table;
  p.num_pages = a.num_pages;
  p.page = fast_divisor(a.page_size);
  p.max_pages = a.max_pages;
  p.block = a.block;
  p.B = a.B;
  p.max_new = a.max_new;
  p.Hi = a.Hi;
  p.NP = (a.Hi + 15) / 16 * 16;
  p.T = a.T;
  p.max_seq = std::min(a.max_seq, kMaxContext);
  p.stride = a.stride;
  p.status = a.status;
  const int stage = kb * IT * 128;
  // Tokens of a group: as many queries as 32 KB hold; of an MMA: 128 columns, eight at most.
  p.G = std::max(1, std::min({I_MAXG, a.max_new, I_QMAX / (p.NP * 128 * kb)}));
  p.batch = std::min({p.G, 8, 128 / p.NP});
  p.groups = (a.max_new + p.G - 1) / p.G;
  int box = 1;
  while (box < IT && a.page_size % (2 * box) == 0) box *= 2;
  p.box = box;
  p.cols = 32;
  while (p.cols < GROUPS * p.batch * p.NP) p.cols *= 2;
  const int q_bytes = p.G * p.NP * 128 * kb, w_bytes = (p.G * p.NP * 4 + 1023) / 1024 * 1024;
  const int room = 112 * 1024 - q_bytes - w_bytes - I_BAR - 1024;
  p.stages = std::max(2, std::min(I_MAXSTAGES, room / stage));
  p.at_ring = q_bytes;
  p.at_w = p.at_ring + p.stages * stage;
  p.at_bar = p.at_w + w_bytes;
  const int smem = p.at_bar + I_BAR + 1024;
  // The pairs' tiles in runs of equal length, for the places of one round of
  // CTAs (two rounds with several tokens): the lengths are only known on the
  // device, where each CTA finds its run.  Half a run a pair is lost to
  // rounding, so the share leaves that many places: 304 shares for 64 sequences
  // made more CTAs than places, and a second round (46 us, not 36).  Ranges cut
  // on the host by max_seq_len took 41 to 43 us, more where that is far above
  // the contexts.  Many pairs need no cutting, and finding a run among as many
  // sequences would take longer than it saves.
  const long long pairs = static_cast<long long>(a.B) * p.groups;
  const long long places = (p.G == 1 ? 2ll : 4ll) * sm_count();
  p.places = pairs >= 4 * places ? 0 : static_cast<int>(places);
  p.shares = std::max(p.places / 2, p.places - static_cast<int>(std::min(pairs / 2, places)));
  const long long items = pairs + p.places;
  if (items >= (1ll << 31)) return cudaErrorInvalidValue;
  const CUtensorMapDataType dt = e8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int cols = e8 ? 128 : 64;
  // Runs of 8 keys or more by TMA, shorter ones key by key (a decode step on pages
  // of 8: 43 us, against 49).
  const bool dense = box >= 8;
  CUtensorMap q_map, k_map;
  if (!encode_2d(&q_map, a.iq, dt, 128, static_cast<uint64_t>(a.T) * a.Hi, 128 * kb, cols, p.NP,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&k_map, a.keys, dt, 128, static_cast<uint64_t>(a.num_pages) * a.page_size, 128 * kb, cols,
                 dense ? box : 8, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  auto go = [&](auto kernel) -> cudaError_t {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(items)), dim3(kScoreThreads), static_cast<size_t>(smem), stream,
                      q_map, k_map, p);
  };
  if (e8) return dense ? go(index_scores_kernel<true, true>) : go(index_scores_kernel<true, false>);
  return dense ? go(index_scores_kernel<false, true>) : go(index_scores_kernel<false, false>);
}

cudaError_t launch_index_select(const IndexSelectArgs& a, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  IndexSelectArgs b = a;
  b.max_seq = std::min(a.max_seq, kMaxContext);
  // One CTA a token, or, where the tokens leave SMs idle and the rows are
  // long, up to 16 (at least 4096 scores each): two tokens of 131000 scores
  // took 22 us with eight and 19 with 16.
  int C = 1;
  while (C < kSelMaxCluster && static_cast<long long>(a.T) * 2 * C <= sm_count() && a.stride / (2 * C) >= 4096) C *= 2;
  cudaError_t e = cudaFuncSetAttribute(index_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSelCacheFloats * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  auto shape = [&] {
    const long long slice = ((static_cast<long long>(a.stride) + C - 1) / C + 31) / 32 * 32;
    cfg.dynamicSmemBytes = slice <= kSelCacheFloats ? static_cast<size_t>(slice) * 4 : 16;
    cfg.gridDim = dim3(static_cast<unsigned>(C) * static_cast<unsigned>(a.T));
    attr[0].val.clusterDim.x = C;
    return slice <= kSelCacheFloats ? 1 : 0;
  };
  int cached = shape();
  if (C == 16) {
    // Above the portable size; a device (or the part of one) that cannot place
    // such a cluster gets eight CTAs.
    e = cudaFuncSetAttribute(index_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    cfg.numAttrs = 1;
    int fit = 0;
    if (e != cudaSuccess || cudaOccupancyMaxActiveClusters(&fit, index_select_kernel, &cfg) != cudaSuccess || fit < 1) {
      cudaGetLastError();
      C = 8;
      cached = shape();
    }
  }
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, index_select_kernel, b, fast_divisor(a.page_size), cached);
}

}  // namespace mla
