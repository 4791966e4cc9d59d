// Absorbed MLA attention of a chunk of new tokens of every sequence over the
// paged cache: a draft tree that is verified, or the next tokens of a prompt
// ("mla_prefill_decode_graph_bf16", Args w_uk, w_uv; the mask of its Parameters
// replaced by one among the new tokens).
//
//   q_lat = w_uk[h] q_nope;  s_j = scale (q_lat . c_j + q_rope . r_j)
//   out = w_uv[h] sum_j softmax(s)_j c_j
//
// over the cached positions, all of them visible, and the new tokens of the
// sequence that the mask row names.  For chunks of up to about 170 tokens this
// is less work than up-projecting the context: 2176 operations for each (row,
// key) against 262144 for each (head, key) and 640 for each pair.
//
// Launches: the query projection with the plan in a CTA of its own; the
// attention; a merge; the output projection.
//
// The attention runs on pairs of SMs.  A pair holds 128 query rows (token,
// head) of one sequence, 64 in each CTA, and walks 256-key tiles: S = Q K^T and
// O += P V are two-SM MMAs with M = 128 and N = 256, whose accumulators lie two
// columns of a row over each other: lanes 0..63 hold the rows' first N / 2
// columns, lanes 64..127 the rest.  So the fp32 O of 64 rows x 512 columns takes
// 256 TMEM columns, two score tiles the other 256, and two threads share a row:
// a thread's softmax has 128 of the 256 keys, against 4352 clk of MMAs a tile.
// Scores run a tile ahead, so the softmax is hidden entirely.
//
// What bounds it: both operands of both products come from shared memory, and K
// and V are the same bytes needed in different halves (CTA r takes keys 128r..
// of a tile for S, latent columns 128r.. of each 256 for O), so each CTA writes
// and reads 147 KB and 131 KB a tile, and reads 74 KB of Q and twice 32 KB of P:
// 5600 clk at 128 bytes a clk.  Measured: 64 tokens over 65536 keys, 128 heads, 750
// us, 1560 TFLOP/s, 6900 clk a tile (with a ring of 5 and 6 stages 11 and 3 % more);
// 805 to 835 us in thousands of such calls, which run at the card's power limit and
// 1700 to 1870 MHz.
// Where a row tile is alone with its context, HBM's latency and the second read of
// a tile from L2 come on top: 32 sequences of 8 tokens over 20000 keys, 16 heads,
// 203 us for 740 MB, 4.6 us a tile; on pages of 16, whose tiles are 16 boxes, the
// loads' issue (10 tokens: 277 us on pages of 64, 368 on pages of 16).  A short
// context is chains of dependent loads: 32 us for one tree over 1000 keys.
//
// Who does what, found on the device from the lengths: the row tiles of a
// sequence, two by two, are items that two pairs work at side by side (class
// 0), a last odd one is an item of a single pair (class 1).  Of each class,
// workers first take whole items in turn, so that the 76 pairs are at the same
// few sequences at any time and HBM is read once or twice, not once a row tile;
// what is left is a line of key tiles that is cut so that all workers end
// with the same load.  A row tile that a cut splits leaves (O, max, sum) in
// fp32, which the merge joins; all others are finished by their pair.
#include <algorithm>

#include "chunk_plan.cuh"
#include "kernels.cuh"

namespace mla {
namespace {
using namespace chunk;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kRescale = 8.0f;             // a row's reference moves when its maximum grows by 2^8

constexpr int kStage = 16 * 1024;
// Small calls (launch_chunk_attn has the rule) hold the softmax weights in two bf16
// terms.  Results over 300 to 2500 keys are 0.0025 off in the 2-norm with one term
// and 0.0022 with two, of which the output's own rounding is 0.0017 and the
// projected query's 0.0014.  A small call waits for chains of loads, not for MMAs,
// and is as fast on a ring of 5 stages, which leaves room for the second term: one
// tree of 6 over 1000 keys, 16 heads, 30.0 us with one and 31.7 with two.  Of larger
// calls the products are what bounds them: 8 chunks of 64 over 2000 keys, 128 heads,
// took 340 us with one and 499 with two (on seven stages, a tile in two steps).
__host__ __device__ constexpr int ring_stages(bool two) { return two ? 5 : 7; }
constexpr int kQBytes = 9 * 64 * 128;        // 64 rows x 576 columns in blocks of 64
constexpr int kPBytes = 4 * 64 * 128;        // 64 rows x 256 keys in blocks of 64
constexpr int kSmemQ = 0;
constexpr int kSmemP = kSmemQ + kQBytes;
__host__ __device__ constexpr int smem_ring(bool two) { return kSmemP + (two ? 2 : 1) * kPBytes; }
constexpr int kFound = 4;                    // tiles whose rows have been looked up
constexpr int kSmemBoxes = smem_ring(false) + ring_stages(false) * kStage;      // their boxes: 4 groups of 64 rows each
constexpr int kSmemRed = kSmemBoxes + kFound * 4 * 64 * 8;    // a row's maxima and sums of both threads
constexpr int kSmemBar = kSmemRed + 2 * 128 * 4;
constexpr int kSmemTotal = kSmemBar + 1024 + 1024;
static_assert(kSmemTotal <= 227 * 1024, "shared memory");
static_assert(smem_ring(true) + ring_stages(true) * kStage <= kSmemBoxes, "shared memory");
constexpr int kProducers = 4;                // warps 0, 7, 8, 9
constexpr int kThreads = 192 + 32 * kProducers;   // with MMA (1), softmax (2 .. 5), row lookup (6)
static_assert((kProducers & (kProducers - 1)) == 0, "whose stage it is: a difference modulo 2^32");
constexpr uint32_t kTmO = 256;               // TMEM: S 2 x 128, O 2 x 128 columns
constexpr uint32_t kIdescS = idesc_bf16(kRows, kTile, false, false);
constexpr uint32_t kIdescO = idesc_bf16(kRows, 256, false, true);

// Boxes of 1, 2, .. 128 rows x 64 columns of the cache: a run of rows that ends
// anywhere is a few of them.  wide: 64 rows x 2 blocks of 64 columns.
struct CacheMaps {
  CUtensorMap box[8], wide;
};

struct ChunkParams {
  const uint32_t* iro;
  const uint32_t* cache_len;
  const int32_t* page_table;
  const uint32_t* mask;
  const float* sink;
  const Base* base;          // [B + 1]
  const Schedule* schedule;
  __nv_bfloat16* o_lat;      // [R][2][512]
  float* lse;                // [R] or null
  float4* o_part;            // [4 pairs][2][64][128]: a pair's first and last segment of each line
  float2* ml_part;           // [4 pairs][128] (max, sum)
  SplitTile* split;          // [2 pairs]
  bool by_tile;              // a row tile's place there is its number
  const uint32_t* odd_rows;  // [(T + 31) / 32]: tokens whose rows hold an infinity or NaN
  int num_pages, page_size, max_pages, cache_rows;
  FastDiv by_page;
  int B, H, T, words;
  float scale_log2;
  int32_t* status;
};

// ------------------------------------------------------------------ segments
struct Segment {
  int b, row0, r0, rows;      // sequence, first global row, first row within the sequence, valid rows
  int k0, k1, kt;             // key tiles [k0, k1) of the row tile's kt
  int tiles;                  // of them, those that a row sees any key of (-1: no more segments)
  int cached, n, L;
  int c, x;                   // class; the position of k0 on the class's line (-1: a whole item taken in turn)
};
struct Walk {
  int c, pair, b;
  int item, left, stride;     // whole items: the next one, how many more
  int x, x1;                  // this worker's part of the line
  int left1, stride1, tail1, end1;   // the same for class 1, while at class 0
  bool begun;
};

// (All that the schedule says of a pair is loaded at once: one latency.)
__device__ __forceinline__ Walk walk_start(const ChunkParams& p, int pair) {
  const Schedule& sc = *p.schedule;
  const int g = pair >> 1;
  Walk w;
  w.c = 0;
  w.pair = pair;
  w.b = 0;
  w.begun = false;
  w.item = g;
  w.stride = sc.workers[0];
  w.left = sc.whole[0];
  w.x = sc.tail[0][g];
  w.x1 = sc.tail[0][g + 1];
  w.stride1 = sc.workers[1];
  w.left1 = sc.whole[1];
  w.tail1 = sc.tail[1][pair];
  w.end1 = sc.tail[1][pair + 1];
  if (g >= w.stride) w.left = w.x = w.x1 = 0;
  if (pair >= w.stride1) w.left1 = w.tail1 = w.end1 = 0;
  return w;
}

// By a warp.
__device__ __forceinline__ bool walk_next(const ChunkParams& p, Walk& w, Segment& s) {
  if (w.left == 0 && w.x >= w.x1) {
    if (w.c == 1) return false;
    w.c = 1;
    w.item = w.pair;
    w.left = w.left1;
    w.stride = w.stride1;
    w.x = w.tail1;
    w.x1 = w.end1;
    w.begun = false;
    if (w.left == 0 && w.x >= w.x1) return false;
  }
  const int c = w.c;
  int i;                       // item within the sequence
  if (w.left > 0) {
    w.b = last_of(p.B, [&](int b) { return p.base[b].items[c] <= w.item; });
    i = w.item - p.base[w.b].items[c];
    w.item += w.stride;
    --w.left;
  } else {
    if (!w.begun) w.b = last_of(p.B, [&](int b) { return p.base[b].units[c] <= w.x; });
    w.begun = true;
    while (p.base[w.b + 1].units[c] <= w.x) ++w.b;
    i = -1;
  }
  s.c = c;
  s.b = w.b;
  const int q0 = static_cast<int>(p.iro[w.b]);
  s.n = static_cast<int>(p.iro[w.b + 1]) - q0;
  s.cached = static_cast<int>(p.cache_len[w.b]);
  s.L = s.cached + s.n;
  s.kt = (s.L + kTile - 1) / kTile;
  if (i >= 0) {
    s.k0 = 0;
    s.k1 = s.kt;
    s.x = -1;
  } else {
    const int off = w.x - p.base[w.b].units[c];
    i = off / s.kt;
    s.k0 = off - i * s.kt;
    s.k1 = static_cast<int>(min(static_cast<long long>(s.kt), static_cast<long long>(s.k0) + (w.x1 - w.x)));
    s.x = w.x;
    w.x += s.k1 - s.k0;
  }
  const long long rows = static_cast<long long>(s.n) * p.H;
  const int m = c == 0 ? 2 * i + (w.pair & 1) : static_cast<int>((rows - 1) / kRows);
  s.r0 = m * kRows;
  s.rows = static_cast<int>(min(static_cast<long long>(kRows), rows - s.r0));
  s.row0 = static_cast<int>(static_cast<long long>(q0) * p.H + s.r0);
  int last = s.L;             // causal: the tile's last token sees cached + i + 1 keys
  if (p.mask == nullptr) last = s.cached + (s.r0 + s.rows - 1) / p.H + 1;
  s.tiles = max(0, min(s.k1, (last + kTile - 1) / kTile) - s.k0);
  return true;
}

constexpr int kSegments = 4;     // segments that the lookup warp is ahead by

struct ChunkSmem {
  uint64_t full[ring_stages(false)], empty[ring_stages(false)];
  uint64_t q_full, q_free;
  uint64_t s_full[2], p_full, pv_done, drain;
  uint64_t swapped[2];       // the two warps that share rows have both written their words
  uint32_t tmem;
  int abort;
  uint64_t found[kFound], taken[kFound];
  alignas(16) int row[kFound][4];   // first cache row of a group of 64 consecutive ones, or -1:
  int boxes[kFound][4];      // it is this many boxes
  uint64_t seg_full[kSegments], seg_free[kSegments];
  Segment segment[kSegments];
};
static_assert(sizeof(ChunkSmem) <= 1024, "barrier block");

// The bits of 32 new tokens from token t on (of T).
__device__ __forceinline__ uint32_t odd_bits(const ChunkParams& p, int t) {
  const int words = (p.T + 31) / 32, w = t >> 5, by = t & 31;
  const uint32_t lo = w < words ? p.odd_rows[w] : 0u, hi = w + 1 < words ? p.odd_rows[w + 1] : 0u;
  return __funnelshift_r(lo, hi, by);
}

// ------------------------------------------------------------------ attention
template <bool TWO>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CacheMaps maps,
                      const __grid_constant__ ChunkParams p) {
  constexpr int kStages = ring_stages(TWO);
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  ChunkSmem* sh = reinterpret_cast<ChunkSmem*>(smem + kSmemBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  int32_t* const status = p.status;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&sh->full[s]), 1);    // (CTA 0's counts both CTAs' bytes)
      mbar_init(smem_u32(&sh->empty[s]), 1);
    }
    mbar_init(smem_u32(&sh->q_full), 1);
    mbar_init(smem_u32(&sh->q_free), 1);
    mbar_init(smem_u32(&sh->s_full[0]), 1);
    mbar_init(smem_u32(&sh->s_full[1]), 1);
    mbar_init(smem_u32(&sh->p_full), 8);
    mbar_init(smem_u32(&sh->pv_done), 1);
    mbar_init(smem_u32(&sh->drain), 1);
    for (int s = 0; s < kFound; ++s) {
      mbar_init(smem_u32(&sh->found[s]), 1);
      mbar_init(smem_u32(&sh->taken[s]), kProducers);
    }
    for (int s = 0; s < kSegments; ++s) {
      mbar_init(smem_u32(&sh->seg_full[s]), 1);
      mbar_init(smem_u32(&sh->seg_free[s]), kProducers + 4 + (rank == 0));
    }
    mbar_init(smem_u32(&sh->swapped[0]), 2);
    mbar_init(smem_u32(&sh->swapped[1]), 2);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&sh->tmem), 512);
    tmem_relinquish_pair();
  }
  pdl_enter();               // (what comes before reads nothing of earlier kernels)
  if (threadIdx.x == 0) sh->abort = timed_out_before(status) ? 1 : 0;
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sh->tmem;
  volatile int* const abort_flag = &sh->abort;
  const bool stop = cluster_any(abort_flag);     // an earlier kernel timed out: no work
  const uint32_t ring = smem_u32(smem + smem_ring(TWO));
  volatile int never = 0;
  // The next segment that the lookup warp has found (by a warp; by one lane of the
  // MMA warp).
  uint32_t seg = 0;
  auto next_segment = [&](Segment& s, bool alone) {
    const uint32_t i = seg % kSegments, full = smem_u32(&sh->seg_full[i]), parity = (seg / kSegments) & 1;
    if (alone) {
      if (!mbar_wait(full, parity, status, abort_flag)) return false;
    } else if (!mbar_wait_warp(full, parity, status, abort_flag)) {
      return false;
    }
    s = sh->segment[i];
    if (!alone) __syncwarp();
    if (alone || lane == 0) mbar_arrive(smem_u32(&sh->seg_free[i]));
    ++seg;
    return s.tiles >= 0;
  };

  if (stop) {
    // (the barriers below are passed by all)
  } else if (warp == 0 || (warp >= 7 && warp < 6 + kProducers)) {
    // ---------------------------------------------------------------- producers
    // Warps that take stages in turn: one lane's loop takes about 60 clk an
    // operation and 200 a stage, too slow for the 256 clk of a stage's MMAs.
    const uint32_t turn = warp == 0 ? 0 : warp - 6;
    const int2* const boxes = reinterpret_cast<const int2*>(smem + kSmemBoxes);
    Segment s;
    uint32_t stage = 0, phase = 0, segments = 0, used = 0, tile = 0;
    bool ok = true;
    // Both CTAs' loads count at CTA 0's barriers, whose MMAs wait for them.
    const uint32_t full0 = cluster_addr(smem_u32(&sh->full[0]), 0);
    // Stage `used`, when its last reader is through with it.
    auto ready = [&](uint32_t st, uint32_t ph, uint32_t n) {
      return n < kStages || mbar_wait(smem_u32(&sh->empty[st]), ph ^ 1, status, abort_flag);
    };
    // n stages, issued by one lane (what the loop costs for each stage bounds the
    // loads: with a warp's votes and the rows read for each stage, 495 clk).
    auto load = [&](uint32_t n, auto boxes_of) {
      if (elect_one()) {
        // The first stage from `used` on that is this warp's.
        uint32_t i = (turn - used) % kProducers;
        uint32_t st = stage + i, ph = phase;
        if (st >= kStages) st -= kStages, ph ^= 1;
        for (; i < n; i += kProducers) {
          if (!(ok = ready(st, ph, used + i))) break;
          if (rank == 0) mbar_expect_tx(smem_u32(&sh->full[st]), 2 * kStage);
          boxes_of(i, ring + st * kStage, full0 + st * 8);
          if ((st += kProducers) >= kStages) st -= kStages, ph ^= 1;
        }
      }
      __syncwarp();
      ok = __all_sync(0xffffffffu, ok);
      used += n;
      stage += n;
      while (stage >= kStages) stage -= kStages, phase ^= 1;
    };
    // The boxes of group g.
    auto group = [&](int slot, int g, uint32_t dst, uint32_t bar, int col) {
      const int y = sh->row[slot][g];
      if (y >= 0) {
        tma_load_2d_pair(dst, &maps.box[6], bar, col, y);
        return;
      }
      const int n = sh->boxes[slot][g];
      const int2* const list = boxes + (slot * 4 + g) * 64;
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const int2 b = list[i];
        tma_load_2d_pair(dst + (b.y >> 8) * 128, &maps.box[b.y & 255], bar, col, b.x);
      }
    };
    // K of tile j, V of the tile before, in the order of use.
    const int vcol = 128 * static_cast<int>(rank);
    while (ok && next_segment(s, false)) {
      if (s.tiles == 0) continue;
      if (segments > 0 && !(ok = mbar_wait_warp(smem_u32(&sh->q_free), (segments - 1) & 1, status, abort_flag))) break;
      if (turn == 0 && elect_one()) {
        if (rank == 0) mbar_expect_tx(smem_u32(&sh->q_full), 2 * kQBytes);
        const uint32_t bar = cluster_addr(smem_u32(&sh->q_full), 0);
        for (int c = 0; c < 9; ++c)
          tma_load_2d_pair(smem_u32(smem + kSmemQ) + c * 8192, &q_map, bar, c * 64, s.row0 + 64 * static_cast<int>(rank));
      }
      __syncwarp();
      ++segments;
#pragma unroll 1
      for (int j = 0; j <= s.tiles && ok; ++j) {
        if (j < s.tiles) {
          const int slot = (tile + j) % kFound;
          if (!(ok = mbar_wait_warp(smem_u32(&sh->found[slot]), ((tile + j) / kFound) & 1, status, abort_flag))) break;
          const int y0 = sh->row[slot][2 * rank], y1 = sh->row[slot][2 * rank + 1];
          if (y0 >= 0 && y1 == y0 + 64) {
            load(9, [&](int c, uint32_t dst, uint32_t bar) {
              tma_load_2d_pair(dst, &maps.box[7], bar, c * 64, y0);
            });
          } else if ((y0 | y1) >= 0) {
            load(9, [&](int c, uint32_t dst, uint32_t bar) {
              tma_load_2d_pair(dst, &maps.box[6], bar, c * 64, y0);
              tma_load_2d_pair(dst + 8192, &maps.box[6], bar, c * 64, y1);
            });
          } else {
            load(9, [&](int c, uint32_t dst, uint32_t bar) {
              group(slot, 2 * rank, dst, bar, c * 64);
              group(slot, 2 * rank + 1, dst + 8192, bar, c * 64);
            });
          }
        }
        if (j > 0 && ok) {
          const int slot = (tile + j - 1) % kFound;
          const int4 y = *reinterpret_cast<const int4*>(sh->row[slot]);
          if ((y.x | y.y | y.z | y.w) >= 0) {
            load(8, [&](int i, uint32_t dst, uint32_t bar) {
              const int g = i >> 1;
              const int row = g == 0 ? y.x : g == 1 ? y.y : g == 2 ? y.z : y.w;
              tma_load_3d_pair(dst, &maps.wide, bar, 0, row, 4 * (i & 1) + 2 * static_cast<int>(rank));
            });
          } else {
            load(8, [&](int i, uint32_t dst, uint32_t bar) {
              const int col = 256 * (i & 1) + vcol;
              group(slot, i >> 1, dst, bar, col);
              group(slot, i >> 1, dst + 8192, bar, col + 64);
            });
          }
          if (lane == 0) mbar_arrive(smem_u32(&sh->taken[slot]));
        }
      }
      tile += s.tiles;
    }
    // Nothing may be on its way into this CTA when it leaves: the loads (if the
    // MMAs did not get to wait for them) and the releases of the stages.
    if (elect_one()) {
      const uint32_t n = min(used, static_cast<uint32_t>(kStages));
      for (uint32_t i = 0; i < n && ok; ++i) {
        const uint32_t u = used - 1 - i;
        ok = mbar_wait(smem_u32(&sh->empty[u % kStages]), (u / kStages) & 1, status, abort_flag);
      }
      if (segments > 0) ok = ok && mbar_wait(smem_u32(&sh->q_free), (segments - 1) & 1, status, abort_flag);
      if (rank == 1 && turn == 0) mbar_wait(smem_u32(&sh->drain), 0, status, &never);
      if (!ok) {      // loads that nobody waits for land long before this ends
        const uint64_t t0 = globaltimer();
        while (globaltimer() - t0 < 1000000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMAs
    if (elect_one()) {
      if (rank == 0) {
        Segment s;
        uint32_t stage = 0, phase = 0, segments = 0, tile = 0, p_phase = 0;
        bool ok = true;
        const uint32_t sq = smem_u32(smem + kSmemQ), sp = smem_u32(smem + kSmemP);
        auto take = [&]() {
          ok = ok && mbar_wait(smem_u32(&sh->full[stage]), phase, status, abort_flag);
          tc_fence_after();
          return ok;
        };
        auto give = [&]() {
          tc_commit_pair(smem_u32(&sh->empty[stage]), 3);
          if (++stage == kStages) stage = 0, phase ^= 1;
        };
        auto scores = [&](uint32_t buf) {
          for (int c = 0; c < 9; ++c) {
            if (!take()) return;
            const uint32_t k = ring + stage * kStage;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mma_f16_ss_pair(tmem + buf * 128, sdesc(sq + c * 8192 + e * 32, 16, 1024), sdesc(k + e * 32, 16, 1024),
                              kIdescS, (c | e) != 0);
            give();
          }
          tc_commit_pair(smem_u32(&sh->s_full[buf]), 3);
        };
        while (ok && next_segment(s, true)) {
          if (s.tiles == 0) continue;
          if (!(ok = mbar_wait(smem_u32(&sh->q_full), segments & 1, status, abort_flag))) break;
          ++segments;
          tc_fence_after();
          scores(tile & 1);
          if (s.tiles == 1 && ok) tc_commit_pair(smem_u32(&sh->q_free), 3);
          for (int j = 0; j < s.tiles && ok; ++j) {
            if (j + 1 < s.tiles) {
              scores((tile + 1) & 1);
              if (j + 2 == s.tiles && ok) tc_commit_pair(smem_u32(&sh->q_free), 3);
            }
            if (!ok || !(ok = mbar_wait(smem_u32(&sh->p_full), p_phase, status, abort_flag))) break;
            p_phase ^= 1;
            tc_fence_after();
            for (int g = 0; g < 4; ++g) {
              for (int m = 0; m < 2; ++m) {
                if (!take()) break;
                const uint32_t v = ring + stage * kStage;
#pragma unroll
                for (int e = 0; e < (TWO ? 8 : 4); ++e)              // (term, 16 keys)
                  mma_f16_ss_pair(tmem + kTmO + m * 128,
                                  sdesc(sp + (e >> 2) * kPBytes + g * 8192 + (e & 3) * 32, 16, 1024),
                                  sdesc(v + (e & 3) * 2048, 8192, 1024), kIdescO, (j | g | e) != 0);
                give();
              }
            }
            if (ok) tc_commit_pair(smem_u32(&sh->pv_done), 3);
            ++tile;
          }
        }
        // The last arrival of this CTA's commits in either CTA.  (A producer of the
        // other CTA waits for it when it is through: a wait is for one step of the
        // pipeline, never for as long as the call takes.)
        tc_commit_pair(smem_u32(&sh->drain), 3);
        mbar_wait(smem_u32(&sh->drain), 0, status, &never);
      }
    }
    __syncwarp();
  } else if (warp == 6) {
    // ---------------------------------------------------------------- row lookup
    // The segments in order, for all roles (a walk is a chain of loads), and:
    // Where a tile's rows are in the cache.  Four groups of 64 that each are
    // consecutive rows need a row each; any other group is a list of boxes
    // (cache row, first row << 8 | log2 rows): every run of consecutive rows is
    // cut into powers of two, largest first.  Rows past the context, or without
    // a page, are boxes behind the cache's end, which read as zeros: no row that
    // nobody has written reaches a product.
    int2* const boxes = reinterpret_cast<int2*>(smem + kSmemBoxes);
    Walk w = walk_start(p, pair);
    Segment s;
    uint32_t tile = 0;
    bool ok = true;
    const bool aligned = p.page_size % 64 == 0;
    for (bool more = true; ok && more;) {
      more = walk_next(p, w, s);
      if (!more) s.tiles = -1;
      const uint32_t i = seg % kSegments;
      if (seg >= kSegments &&
          !(ok = mbar_wait_warp(smem_u32(&sh->seg_free[i]), ((seg / kSegments) & 1) ^ 1, status, abort_flag)))
        break;
      if (lane == 0) {
        sh->segment[i] = s;
        mbar_arrive(smem_u32(&sh->seg_full[i]));
      }
      ++seg;
      const int32_t* const pages = p.page_table + static_cast<size_t>(s.b) * p.max_pages;
#pragma unroll 1
      for (int j = 0; j < s.tiles; ++j, ++tile) {
        const int slot = tile % kFound;
        const int first = (s.k0 + j) * kTile;
        const int token0 = static_cast<int>(p.iro[s.b]) - s.cached;     // a new token's number less its position
        // The page of a position (-1: none there), and its row.
        auto page_of = [&](int pos) {
          const int i = fast_div(pos, p.by_page);
          return pos < s.L && i < p.max_pages ? pages[i] : -1;
        };
        auto row_of = [&](int pos, int page) {
          if (pos >= s.L) return -1;
          if (page >= 0 && page < p.num_pages) return page * p.page_size + (pos - fast_div(pos, p.by_page) * p.page_size);
          set_status(status, MLA_DEV_BAD_PAGE);
          return -1;
        };
        int whole = -1;                                   // lane g < 4: group g
        const int at = first + 64 * lane, to = at + 64;
        if (aligned && lane < 4 && to <= s.L) {
          const int page = page_of(at);
          // (Rows of new tokens before bit 0 of a word are others': a group that is
          // taken for odd by them is only taken apart.)
          const bool odd = to > s.cached && (odd_bits(p, token0 + max(at, s.cached)) | odd_bits(p, token0 + max(to - 32, s.cached)));
          if (!odd) whole = row_of(at, page);
        }
        const unsigned parts = __ballot_sync(0xffffffffu, whole < 0) & 15u;
        if (tile >= kFound &&
            !(ok = mbar_wait_warp(smem_u32(&sh->taken[slot]), ((tile / kFound) & 1) ^ 1, status, abort_flag)))
          break;
        if (lane < 4) sh->row[slot][lane] = whole;
        if (parts != 0) {                                 // all lookups in flight together
          int* const rows = reinterpret_cast<int*>(boxes + slot * 256);
          int page[8];
          bool odd[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) page[e] = page_of(first + 32 * e + lane);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int pos = first + 32 * e + lane;
            odd[e] = pos >= s.cached && pos < s.L && (odd_bits(p, token0 + pos) & 1u);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int row = row_of(first + 32 * e + lane, page[e]);
            rows[(e >> 1) * 128 + (e & 1) * 32 + lane] = odd[e] ? -1 : row;
          }
        }
#pragma unroll 1
        for (int g = 0; g < 4; ++g) {
          if (!(parts >> g & 1)) continue;
          const int* const rows = reinterpret_cast<const int*>(boxes + (slot * 4 + g) * 64);
          const int row0 = rows[lane], row1 = rows[32 + lane];
          __syncwarp();                                   // the list takes their place
          // Bit i: row i of the group does not continue row i - 1.
          const int last0 = __shfl_sync(0xffffffffu, row0, 31);
          int before0 = __shfl_up_sync(0xffffffffu, row0, 1), before1 = __shfl_up_sync(0xffffffffu, row1, 1);
          if (lane == 0) before1 = last0;
          auto cut = [](int row, int before) { return row < 0 ? before >= 0 : before < 0 || row != before + 1; };
          const unsigned lo = __ballot_sync(0xffffffffu, lane == 0 || cut(row0, before0));
          const unsigned hi = __ballot_sync(0xffffffffu, cut(row1, before1));
          const unsigned long long cuts = static_cast<unsigned long long>(hi) << 32 | lo;
          int count = 0;
#pragma unroll 1
          for (int u = 0; u < 2; ++u) {
            const int i = 32 * u + lane, row = u ? row1 : row0;
            const unsigned long long upto = cuts & (~0ull >> (63 - i)), past = i == 63 ? 0 : cuts >> (i + 1);
            const int at = i - (63 - __clzll(upto));                       // within its run
            const int left = past ? __ffsll(past) : 64 - i;                // rows of the run from here on
            const bool starts = at == 0 || left < (at & -at);
            const unsigned m = __ballot_sync(0xffffffffu, starts);
            if (starts)
              boxes[(slot * 4 + g) * 64 + count + __popc(m & ((1u << lane) - 1))] =
                  make_int2(row < 0 ? p.cache_rows : row, i << 8 | (31 - __clz(left)));
            count += __popc(m);
          }
          if (lane == 0) sh->boxes[slot][g] = count;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh->found[slot]));
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    // Two threads share a row: half of a tile's keys and of O's columns each, as
    // its two TMEM lanes hold them.  (Two warps for each quarter of the lanes take
    // as long: the softmax is not what a tile waits for.)
    constexpr int kChunks = 4;                   // of 32 keys
    const int quarter = warp & 3;
    const int tl = quarter * 32 + lane;          // TMEM lane
    const int row = tl & 63, half = tl >> 6;     // row of this CTA; which columns of it
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t o_at = tmem + lane_off + kTmO;
    float* const red = reinterpret_cast<float*>(smem + kSmemRed);     // [2][2][64]
    // The warp's part of P: 32 rows of two blocks of 64 keys.
    const uint32_t mine = smem_u32(smem + kSmemP) + half * 2 * 8192 + (tl & 32) * 128;
    const uint32_t p_bar = cluster_addr(smem_u32(&sh->p_full), 0);
    Segment s;
    uint32_t tile = 0, swaps = 0;
    bool ok = true;
    // The words of the row's two threads (two sets: a set is written again only
    // after the other has been swapped).
    auto swap = [&](float v, float (&all)[2]) {
      float* const words = red + (swaps & 1) * 128;
      words[(half) * 64 + row] = v;
      __syncwarp();
      const uint32_t bar = smem_u32(&sh->swapped[quarter & 1]);
      if (lane == 0) mbar_arrive(bar);
      if (!mbar_wait_warp(bar, swaps & 1, status, abort_flag)) return false;
      ++swaps;
      all[0] = words[row], all[1] = words[64 + row];
      return true;
    };
    while (ok && next_segment(s, false)) {
      const int local = static_cast<int>(rank) * 64 + row;            // row of the pair's tile
      const bool live = local < s.rows;
      const int token = live ? (s.r0 + local) / p.H : 0;              // within the sequence
      const int token0 = static_cast<int>(p.iro[s.b]);
      const uint32_t* mask_row = p.mask != nullptr ? p.mask + static_cast<size_t>(token0 + token) * p.words : nullptr;
      float ref = kNegInf, sum = 0.0f;
      for (int j = 0; j < s.tiles; ++j, ++tile) {
        const uint32_t buf = tile & 1;
        const int k0 = (s.k0 + j) * kTile + half * 128;
        const bool partly = k0 + 32 * kChunks > s.cached;
        uint32_t see[kChunks];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) see[c] = 0xffffffffu;
        if (partly) {
          // Which of the thread's keys the row sees, a bit each (loaded while the
          // scores are computed).
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const int i = k0 + c * 32 - s.cached;                     // new token of the first key
            if (i + 32 <= 0) continue;
            if (mask_row != nullptr) {
              const int wi = i >> 5, by = i & 31;                     // floor for i < 0, too
              const uint32_t lo = wi >= 0 && wi < p.words ? mask_row[wi] : 0u;
              const uint32_t hi = wi + 1 >= 0 && wi + 1 < p.words ? mask_row[wi + 1] : 0u;
              see[c] = by ? (lo >> by) | (hi << (32 - by)) : lo;
              if (i < 0) see[c] |= (1u << -i) - 1u;                   // cached keys (i > -32)
            } else {
              const int n = token + 1 - i;                            // keys from the first on
              see[c] = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
            }
            const int n = s.n - i;                                    // keys that there are
            see[c] &= n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
            // New tokens among them that are no finite numbers.
            if (n > 0 && (see[c] >> max(-i, 0) & odd_bits(p, token0 + max(i, 0))) != 0)
              sum = __int_as_float(0x7FC00000);
          }
        }
        if (!(ok = mbar_wait_warp(smem_u32(&sh->s_full[buf]), (tile >> 1) & 1, status, abort_flag))) break;
        tc_fence_after();
        // Two passes over the scores, 32 at a time (unrolled further they are code
        // that a short context fetches from L2 for one use): the maximum, then the
        // weights.  In a tile that the row does not see all of, the first pass
        // stores the scores back with -infinity in them.
        const uint32_t sc = tmem + lane_off + buf * 128;
        float top = kNegInf;
#pragma unroll 1
        for (int c = 0; c < kChunks; ++c) {
          uint32_t x[32];
          tmem_ld32(sc + c * 32, x);
          tmem_ld_wait();
          if (partly) {
            const uint32_t m = c & 2 ? (c & 1 ? see[3] : see[2]) : c & 1 ? see[1] : see[0];
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(m >> e & 1)) x[e] = __float_as_uint(kNegInf);
            tmem_st32(sc + c * 32, x);
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2) top = fmax3(top, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
        }
        if (partly) tmem_st_wait();
        float all[2];
        if (!(ok = swap(top, all))) break;
        top = fmaxf(all[0], all[1]) * p.scale_log2;
        float factor = 1.0f;
        if (top > ref + kRescale || (ref == kNegInf && top > kNegInf)) {
          factor = ref == kNegInf ? 0.0f : ex2(ref - top);
          ref = top;
          sum *= factor;
        }
        // P of the tile before is read, O holds its product.
        if (tile > 0 && !(ok = mbar_wait_warp(smem_u32(&sh->pv_done), (tile - 1) & 1, status, abort_flag))) break;
        tc_fence_after();
        if (j > 0 && __any_sync(0xffffffffu, factor != 1.0f)) {
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[32];
            tmem_ld32(o_at + c * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              // (No part of the sum is left at a factor of 0, but a NaN that a key of
              // weight 0 with an infinite value has brought.)
              const float v = __uint_as_float(o[e]);
              o[e] = __float_as_uint(factor != 0.0f ? v * factor : v == v ? 0.0f : v);
            }
            tmem_st32(o_at + c * 32, o);
          }
          tmem_st_wait();
        }
        const float shift = ref == kNegInf ? 0.0f : ref;
#pragma unroll 1
        for (int c = 0; c < kChunks; ++c) {
          uint32_t x[32];
          tmem_ld32(sc + c * 32, x);
          tmem_ld_wait();
          // Chunks of 8 keys (16 bytes) of the row, in the 128-byte swizzle.
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t pk[4], rest[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = ex2(fmaf(__uint_as_float(x[u * 8 + 2 * e]), p.scale_log2, -shift));
              const float b = ex2(fmaf(__uint_as_float(x[u * 8 + 2 * e + 1]), p.scale_log2, -shift));
              sum += a + b;
              pk[e] = pack_bf16(a, b);
              if (TWO) rest[e] = pack_bf16(a - bf16_lo(pk[e]), b - bf16_hi(pk[e]));
            }
            const uint32_t at = mine + (c >> 1) * 8192 + lane * 128 + ((((c & 1) * 4 + u) ^ (lane & 7)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(pk[0]), "r"(pk[1]), "r"(pk[2]), "r"(pk[3])
                         : "memory");
            if (TWO)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + kPBytes), "r"(rest[0]), "r"(rest[1]),
                           "r"(rest[2]), "r"(rest[3])
                           : "memory");
          }
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(p_bar);
      }
      if (!ok) break;
      if (s.tiles > 0) {
        if (!(ok = mbar_wait_warp(smem_u32(&sh->pv_done), (tile - 1) & 1, status, abort_flag))) break;
        tc_fence_after();
      }
      float all[2];
      if (!(ok = swap(sum, all))) break;
      sum = all[0] + all[1];
      const bool none = sum == 0.0f;                 // the row saw nothing
      const bool starts = s.k0 == 0, ends = s.k1 == s.kt, first = half == 0;
      if (starts && ends) {
        if (p.sink != nullptr) {
          const float sk = p.sink[s.b] * kLog2e;
          const float m = fmaxf(ref, sk), f = ref == kNegInf ? 0.0f : ex2(ref - m);
          const float add = sk == kNegInf ? 0.0f : ex2(sk - m);
          if (p.lse != nullptr && live && first)
            p.lse[s.row0 + local] = m == kNegInf && none ? kNegInf : (m + log2f(fmaf(sum, f, add))) * kLn2;
          sum = fmaf(sum, f, add);
          sum = f == 0.0f && none ? __builtin_huge_valf() : sum / f;
        } else if (p.lse != nullptr && live && first) {
          p.lse[s.row0 + local] = none ? kNegInf : (ref + log2f(sum)) * kLn2;
        }
        // (A row that saw nothing has zeros in O: what it does not see is finite.
        // Logits of -infinity alone, of keys with infinite values, leave NaN there.)
        const float unit = none ? 0.0f : 1.0f / sum;
        // 32 columns at a time through the warp's part of P (32 rows x 128 bytes):
        // the first term, the upper halves of the floats, then the second, what is
        // left of them, so that rows leave in whole sectors.
#pragma unroll 1
        for (int u = 0; u < 8; ++u) {
          uint32_t o[32];
          tmem_ld32(o_at + u * 32, o);
          tmem_ld_wait();
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t h[4], l[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = __uint_as_float(o[e * 8 + 2 * i]) * unit, b = __uint_as_float(o[e * 8 + 2 * i + 1]) * unit;
              h[i] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
              l[i] = pack_bf16(a - __uint_as_float(__float_as_uint(a) & 0xFFFF0000u),
                               b - __uint_as_float(__float_as_uint(b) & 0xFFFF0000u));
            }
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mine + lane * 128 + ((e ^ (lane & 7)) << 4)),
                         "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                         : "memory");
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mine + lane * 128 + (((4 + e) ^ (lane & 7)) << 4)),
                         "r"(l[0]), "r"(l[1]), "r"(l[2]), "r"(l[3])
                         : "memory");
          }
          __syncwarp();
          const int chunk = lane & 7;
          __nv_bfloat16* const dst =
              p.o_lat + (chunk >> 2) * 512 + (u >> 2) * 256 + half * 128 + (u & 3) * 32 + (chunk & 3) * 8;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = i * 4 + (lane >> 3);
            uint4 v;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(mine + r * 128 + ((chunk ^ (r & 7)) << 4))
                         : "memory");
            const int to = static_cast<int>(rank) * 64 + (tl & 32) + r;
            if (to < s.rows) *reinterpret_cast<uint4*>(dst + static_cast<size_t>(s.row0 + to) * 1024) = v;
          }
        }
        __syncwarp();
      } else {
        const int worker = s.c == 0 ? pair >> 1 : pair;
        const int* const tail = p.schedule->tail[s.c];
        const int slot = 4 * pair + 2 * s.c + (s.x == tail[worker] ? 0 : 1);
        // (A sum below 0 says that there is no O.)
        if (first && live) p.ml_part[slot * kRows + local] = make_float2(ref, s.tiles > 0 ? sum : -1.0f);
        if (s.tiles > 0) {
          // Laid out as the threads hold it: [CTA][column / 4 of the 256][TMEM lane].
          float4* dst = p.o_part + ((static_cast<size_t>(slot) * 2 + rank) * 64) * 128 + tl;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[32];
            tmem_ld32(o_at + c * 32, o);
            tmem_ld_wait();
            if (!live) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[(c * 8 + e) * 128] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                   __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
          }
        }
        if (ends && tl == 0 && rank == 0) {
          // The worker in whose part of the line the row tile begins.
          const int x0 = s.x - s.k0;
          int from = worker;
          while (tail[from] > x0) --from;
          SplitTile t;
          t.row0 = s.row0;
          t.rows = s.rows;
          t.seq = s.b;
          t.c = s.c;
          t.odd = pair & 1;
          t.first = from;
          t.slot = tail[from] == x0 ? 0 : 1;
          t.parts[0] = t.parts[1] = t.parts[2] = 0;
          for (int q = from; q <= worker; ++q)           // (parts of the line may be empty)
            if (tail[q] != tail[q + 1]) t.parts[(q - from) >> 5] |= 1u << ((q - from) & 31);
          const Base before = p.base[s.b];
          p.split[p.by_tile ? 2 * before.items[0] + before.items[1] + s.r0 / kRows : s.c * pairs + pair] = t;
        }
      }
      tc_fence_before();
      // (The next segment's first product is ordered behind these reads by the
      // arrival on p_full.)
    }
  }

  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ------------------------------------------------------------------ merge
// Split row tiles, blockIdx.x.  A warp takes 32 of the attention's threads' rows and
// COLS of their 256 columns.  What is waited for here are chains of loads, so the
// sums and the rows of PARTS parts are asked for at once, as soon as the tile's
// record is there.  The fewer row tiles there are, the more parts they have and the
// more warps it takes to keep the SMs busy; with many of them warps cost more than
// they bring.  (Whole calls with 4, 16, 32 columns: 4 tokens over 40000 keys, 16
// heads, one row tile of 76 parts, 50, 67, 92 us; 12 tokens over 20000, 128 heads, 12
// row tiles, 80, 78, 82; 76 sequences of 8 tokens over 2000, 16 heads, 76 row tiles
// that nothing splits, 100, 85, 83.)
constexpr int kMergeWarps = 8;
constexpr int merge_slices(int cols) { return 8 * 256 / cols / kMergeWarps; }

template <int COLS, int PARTS>
__global__ void __launch_bounds__(kMergeWarps * 32) chunk_merge_kernel(const ChunkParams p) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const SplitTile t = p.split[blockIdx.x];
  constexpr int kBlocks = 256 / COLS, kVecs = COLS / 4;
  const int unit = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  const int part = unit % kBlocks, quarter = unit / kBlocks & 3, rank = unit / kBlocks >> 2;   // columns; rows, CTA
  const int tl = quarter * 32 + lane, half = tl >> 6;
  const int r = rank * 64 + (tl & 63);
  if (timed_out_before(p.status) || t.rows <= 0) return;
  // The slots of the parts, in order (found one after the other they took as long as
  // the loads).
  __shared__ int slots[kMergeWarps][96];
  int* const slot_of = slots[threadIdx.x >> 5];
  int n = 0;
#pragma unroll
  for (int w = 0; w < 3; ++w) {
    const int q = t.first + 32 * w + lane;
    if (t.parts[w] >> lane & 1)
      slot_of[n + __popc(t.parts[w] & ((1u << lane) - 1))] =
          4 * (t.c == 0 ? 2 * q + t.odd : q) + 2 * t.c + (q == t.first ? t.slot : 0);
    n += __popc(t.parts[w]);
  }
  __syncwarp();
  if (r >= t.rows) return;
  const float sink = p.sink != nullptr ? p.sink[t.seq] * kLog2e : kNegInf;
  float top = sink, sum = sink == kNegInf ? 0.0f : 1.0f;
  float4 o[kVecs] = {};
  for (int k = 0; k < n; k += PARTS) {
    float4 v[PARTS][kVecs];
    float2 ml[PARTS];
    float most = top;
#pragma unroll
    for (int u = 0; u < PARTS; ++u) {
      ml[u] = make_float2(kNegInf, -1.0f);
      if (k + u >= n) continue;
      const int slot = slot_of[k + u];
      ml[u] = p.ml_part[slot * kRows + r];
      const float4* src = p.o_part + ((static_cast<size_t>(slot) * 2 + rank) * 64 + part * kVecs) * 128 + tl;
#pragma unroll
      for (int e = 0; e < kVecs; ++e) v[u][e] = __ldcs(src + e * 128);
    }
#pragma unroll
    for (int u = 0; u < PARTS; ++u) most = fmaxf(most, ml[u].x);
    const float keep = top == kNegInf ? 0.0f : ex2(top - most);
    top = most;
    sum *= keep;
#pragma unroll
    for (int e = 0; e < kVecs; ++e) o[e].x *= keep, o[e].y *= keep, o[e].z *= keep, o[e].w *= keep;
#pragma unroll
    for (int u = 0; u < PARTS; ++u) {
      if (ml[u].y < 0.0f) continue;            // it had no tiles and stored no rows
      const float f = ml[u].x == kNegInf ? ml[u].y * 0.0f : ex2(ml[u].x - top);
      sum = fmaf(ml[u].y, f, sum);
#pragma unroll
      for (int e = 0; e < kVecs; ++e) {
        o[e].x = fmaf(v[u][e].x, f, o[e].x);
        o[e].y = fmaf(v[u][e].y, f, o[e].y);
        o[e].z = fmaf(v[u][e].z, f, o[e].z);
        o[e].w = fmaf(v[u][e].w, f, o[e].w);
      }
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int col = part * COLS;           // of the 256: 128 of each half of the 512
  __nv_bfloat16* hi = p.o_lat + static_cast<size_t>(t.row0 + r) * 1024 + (col >> 7) * 256 + half * 128 + (col & 127);
  uint2 h[kVecs], l[kVecs];
#pragma unroll
  for (int e = 0; e < kVecs; ++e) {
    const float x[4] = {o[e].x * inv, o[e].y * inv, o[e].z * inv, o[e].w * inv};
    h[e] = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
    l[e] = make_uint2(pack_bf16(x[0] - bf16_lo(h[e].x), x[1] - bf16_hi(h[e].x)),
                      pack_bf16(x[2] - bf16_lo(h[e].y), x[3] - bf16_hi(h[e].y)));
  }
  if constexpr (kVecs == 1) {
    *reinterpret_cast<uint2*>(hi) = h[0];
    *reinterpret_cast<uint2*>(hi + 512) = l[0];
  } else {
#pragma unroll
    for (int e = 0; e < kVecs; e += 2) {
      *reinterpret_cast<uint4*>(hi + 4 * e) = make_uint4(h[e].x, h[e].y, h[e + 1].x, h[e + 1].y);
      *reinterpret_cast<uint4*>(hi + 512 + 4 * e) = make_uint4(l[e].x, l[e].y, l[e + 1].x, l[e + 1].y);
    }
  }
  if (p.lse != nullptr && part == 0 && half == 0)
    p.lse[t.row0 + r] = sum == 0.0f ? kNegInf : (top + log2f(sum)) * kLn2;
}

struct Layout {
  size_t q_full, o_lat, base, schedule, token_seq, odd_rows, o_part, ml_part, split, total;
};
Layout layout(int B, int H, int T) {
  const size_t R = static_cast<size_t>(T) * H;
  Layout L;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  L.q_full = take(R * 1152);
  L.o_lat = take(R * 2048);
  L.base = take(sizeof(Base) * (static_cast<size_t>(B) + 1));
  L.schedule = take(sizeof(Schedule));
  L.token_seq = take(sizeof(int32_t) * static_cast<size_t>(T));
  L.odd_rows = take(sizeof(uint32_t) * ((static_cast<size_t>(T) + 31) / 32));
  L.o_part = take(static_cast<size_t>(4 * kMaxPairs) * kRows * 512 * sizeof(float));
  L.ml_part = take(static_cast<size_t>(4 * kMaxPairs) * kRows * sizeof(float2));
  L.split = take(2 * kMaxPairs * sizeof(SplitTile));
  L.total = off;
  return L;
}

}  // namespace

size_t chunk_attn_workspace(int B, int H, int T) { return layout(B, H, T).total; }

cudaError_t launch_chunk_attn(const ChunkAttnArgs& a, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  const size_t R = static_cast<size_t>(a.T) * a.H;
  const Layout L = layout(a.B, a.H, a.T);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  __nv_bfloat16* q_full = reinterpret_cast<__nv_bfloat16*>(ws + L.q_full);
  const int pairs = std::max(2, std::min(kMaxPairs, sm_count() / 2));
  const long long row_tiles = static_cast<long long>(R) / kRows + a.B;      // at most

  ChunkParams p;
  p.iro = a.iro;
  p.cache_len = a.cache_len;
  p.page_table = a.page_table;
  p.mask = a.mask;
  p.sink = a.sink;
  p.base = reinterpret_cast<const Base*>(ws + L.base);
  p.schedule = reinterpret_cast<const Schedule*>(ws + L.schedule);
  p.o_lat = reinterpret_cast<__nv_bfloat16*>(ws + L.o_lat);
  p.lse = a.lse;
  p.o_part = reinterpret_cast<float4*>(ws + L.o_part);
  p.ml_part = reinterpret_cast<float2*>(ws + L.ml_part);
  p.split = reinterpret_cast<SplitTile*>(ws + L.split);
  p.by_tile = row_tiles <= 2 * pairs;
  p.odd_rows = reinterpret_cast<const uint32_t*>(ws + L.odd_rows);
  p.num_pages = a.num_pages;
  p.page_size = a.page_size;
  p.max_pages = a.max_pages;
  p.by_page = fast_divisor(a.page_size);
  p.cache_rows = a.num_pages * a.page_size;
  p.B = a.B;
  p.H = a.H;
  p.T = a.T;
  p.words = a.mask_words;
  p.scale_log2 = a.scale * kLog2e;
  p.status = a.status;
  const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap q_map;
  CacheMaps maps;
  if (!encode_2d(&q_map, q_full, bf, 576, R, 1152, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B)) return cudaErrorInvalidValue;
  const uint64_t rows = static_cast<uint64_t>(p.cache_rows);
  if (!encode_3d(&maps.wide, a.kv_cache, bf, {64, rows, 9}, {1152, 128}, {64, 64, 2}, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  for (int e = 0; e < 8; ++e)
    if (!encode_2d(&maps.box[e], a.kv_cache, bf, 576, rows, 1152, 64, 1u << e,
                   CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;

  ChunkPlanArgs pa;
  pa.iro = a.iro;
  pa.cache_len = a.cache_len;
  pa.base = reinterpret_cast<Base*>(ws + L.base);
  pa.schedule = reinterpret_cast<Schedule*>(ws + L.schedule);
  pa.token_seq = reinterpret_cast<int32_t*>(ws + L.token_seq);
  pa.split = p.split;
  pa.B = a.B;
  pa.H = a.H;
  pa.T = a.T;
  pa.words = a.mask_words;
  pa.pairs = pairs;
  pa.masked = a.mask != nullptr;
  pa.status = a.status;
  pa.kv_cache = a.kv_cache;
  pa.page_table = a.page_table;
  pa.num_pages = a.num_pages;
  pa.page_size = a.page_size;
  pa.max_pages = a.max_pages;
  pa.odd_rows = ws + L.odd_rows;
  cudaError_t e = launch_project_queries(a.q, a.w_uk, q_full, a.T, a.H, &pa, a.status, stream);
  if (e != cudaSuccess) return e;
  // Two terms where a pair has one tile or two at most, by what the host knows: the
  // row tiles that there can be, and the tiles of the longest context that the page
  // table holds.
  const long long key_tiles = std::min((static_cast<long long>(a.max_pages) * a.page_size + kTile - 1) / kTile,
                                       static_cast<long long>(kMaxContext));
  const auto kernel = row_tiles * key_tiles <= 2 * pairs ? chunk_attn_kernel<true> : chunk_attn_kernel<false>;
  if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemTotal)) != cudaSuccess)
    return e;
  if ((e = launch_pdl(kernel, dim3(2 * pairs), dim3(kThreads), kSmemTotal, stream, q_map, maps, p)) !=
      cudaSuccess)
    return e;
  const int cols = row_tiles <= 8 ? 4 : row_tiles <= pairs / 2 ? 16 : 32;
  const auto merge = cols == 4 ? chunk_merge_kernel<4, 16> : cols == 16 ? chunk_merge_kernel<16, 4> : chunk_merge_kernel<32, 2>;
  const dim3 merge_grid(p.by_tile ? static_cast<int>(row_tiles) : 2 * pairs, merge_slices(cols));
  if ((e = launch_pdl(merge, merge_grid, dim3(kMergeWarps * 32), 0, stream, p)) != cudaSuccess) return e;
  return launch_project_outputs(p.o_lat, true, a.w_uv, a.out, a.T, a.H, pa.token_seq, a.status, stream);
}

}  // namespace mla
