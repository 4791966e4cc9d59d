// Who does what in chunk attention (chunk_attn.cu), found on the device from the
// sequences' lengths.
#pragma once

#include "kernels.cuh"

namespace mla {

namespace chunk {
constexpr int kTile = 256;                   // keys of a tile
constexpr int kRows = 128;                   // query rows of a pair of SMs
constexpr int kMaxPairs = 76;
static_assert(kMaxPairs <= 96, "bits of SplitTile::parts");

// A split row tile, noted by the worker in whose part of the line it ends: in the
// place of the row tile, where there are no more of them than 2 pairs, else in the
// worker's.
struct SplitTile {
  int row0, rows, seq;
  int c, odd;           // class; which pair of a group
  int first, slot;      // the worker in whose part it begins, and its slot there
  uint32_t parts[3];    // bit q: worker first + q holds a part of it
};

// Items of class c have workers(c) workers: groups of two pairs, or pairs.
__host__ __device__ constexpr int workers_of(int pairs, int c) { return c == 0 ? pairs / 2 : pairs; }
struct Schedule {
  int workers[2];                        // that have any work
  int whole[2];                          // items that each worker takes whole, in turn
  int tail[2][kMaxPairs + 1];            // then [tail[w], tail[w + 1]) of the class's line of key tiles
};
// Before sequence b: items and key tiles of them, of class 0 and 1.
struct Base {
  int items[2], units[2];
};

// Items of every sequence, their prefix sums, the workers' shares, and each
// token's sequence.  A sequence is left out (no items, no tokens) if its rows
// are not there, or if its context is longer than its row of the page table: a
// wrong length costs the other sequences nothing.
struct ChunkPlanArgs {
  const uint32_t* iro;
  const uint32_t* cache_len;
  Base* base;
  Schedule* schedule;
  int32_t* token_seq;
  SplitTile* split;
  int B, H, T, words, pairs;
  bool masked;
  int32_t* status;
  // The new tokens' cache rows, and where those with a value that is no finite
  // number among their 512 latent ones are noted, a bit a token.
  const void* kv_cache;      // bf16 [num_pages * page_size][576]
  const int32_t* page_table;
  int num_pages, page_size, max_pages;
  uint8_t* odd_rows;         // [(T + 7) / 8]
};

// The sequence of item i of class c: the last one with base <= i.
__device__ __forceinline__ int sequence_of(const Base* base, int B, int c, int i) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (base[mid].items[c] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The last b of [0, B) that is 0 or has before(b), which holds up to some b, by a
// warp: 32 of them are looked at in one step of what is a chain of loads.
template <typename F>
__device__ __forceinline__ int last_of(int B, F before) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
    lo += step * __popc(__ballot_sync(0xffffffffu, at < hi && before(at)));
    hi = min(hi, lo + step);
  }
  return lo;
}

// By one CTA of kPlanThreads, with kKeepBases Base of shared memory: the bases are
// searched there if they fit.  (500 sequences of 3 tokens over 600 keys, 16 heads: a
// call takes 182 us with that and the pairs' searches by warps, 203 without.)
template <int kPlanThreads, int kKeepBases>
__device__ __forceinline__ void chunk_plan(const ChunkPlanArgs& a, Base* kept) {
  constexpr int kWarps = kPlanThreads / 32;
  static_assert(kPlanThreads >= 64 + kMaxPairs, "a thread for each worker");
  __shared__ int4 warp_sum[kWarps];
  __shared__ int whole[2], rest[2][kMaxPairs];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  struct Lengths {
    uint32_t q0, q1, cached;
  };
  auto lengths = [&](int b) { return b < a.B ? Lengths{a.iro[b], a.iro[b + 1], a.cache_len[b]} : Lengths{}; };
  Lengths next = lengths(t);
  bool bad = t == 0 && a.iro[0] != 0;
  for (int b = t; b < a.B; b += kPlanThreads) bad |= a.iro[b + 1] < a.iro[b];
  if (t < 2) whole[t] = 0x7FFFFFFF;
  for (int i = t; i < a.T; i += kPlanThreads) a.token_seq[i] = -1;
  for (int i = t; i < 2 * a.pairs; i += kPlanThreads) a.split[i].rows = 0;
  const bool all_bad = __syncthreads_or(bad);
  const bool keep = a.B < kKeepBases;
  const Base* const base = keep ? kept : a.base;
  if (all_bad && t == 0) set_status(a.status, MLA_DEV_BAD_OFFSETS);
  int4 before = make_int4(0, 0, 0, 0);          // items of class 0 and 1, units of class 0 and 1
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + t;
    int4 own = make_int4(0, 0, 0, 0);
    int token0 = 0, tokens = 0;
    const Lengths at = next;
    next = lengths(b + kPlanThreads);
    if (b < a.B && !all_bad) {
      const long long n = at.q1 - at.q0, L = static_cast<long long>(at.cached) + n;
      if (at.q1 > static_cast<uint32_t>(a.T) || (a.masked && n > 32ll * a.words) || L > kMaxContext) {
        set_status(a.status, MLA_DEV_BAD_OFFSETS);
      } else if (n > 0 && L > static_cast<long long>(a.max_pages) * a.page_size) {
        set_status(a.status, MLA_DEV_BAD_PAGE);
      } else if (n > 0) {
        const long long tiles = (n * a.H + kRows - 1) / kRows, kt = (L + kTile - 1) / kTile;
        own.x = static_cast<int>(tiles / 2);
        own.y = static_cast<int>(tiles & 1);
        // (2^31 units are some 100 to 200 s of work, at 3.6 us a tile; sums saturate and
        // the call is refused, see below.)
        own.z = static_cast<int>(min(tiles / 2 * kt, 0x7FFFFFFFll));
        own.w = own.y ? static_cast<int>(kt) : 0;
        token0 = static_cast<int>(at.q0);
        tokens = static_cast<int>(n);
      }
    }
    // A sequence's first tokens by its thread, more of them by the warp.  (All by the
    // warp: 5 us for 32 sequences, one after the other.)
    constexpr int kFew = 32;
#pragma unroll 1
    for (int i = 0; i < min(tokens, kFew); ++i) a.token_seq[token0 + i] = b;
    for (unsigned m = __ballot_sync(0xffffffffu, tokens > kFew); m != 0; m &= m - 1) {
      const int from = __ffs(m) - 1;
      const int first = __shfl_sync(0xffffffffu, token0, from), n = __shfl_sync(0xffffffffu, tokens, from);
#pragma unroll 1
      for (int i = kFew + lane; i < n; i += 32) a.token_seq[first + i] = b - lane + from;
    }
    // Sums that would not fit stay at the largest number.
    auto add = [](int x, int y) { return static_cast<int>(min(static_cast<unsigned>(x) + static_cast<unsigned>(y), 0x7FFFFFFFu)); };
    int4 s = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, s.x, d), y = __shfl_up_sync(0xffffffffu, s.y, d);
      const int z = __shfl_up_sync(0xffffffffu, s.z, d), w = __shfl_up_sync(0xffffffffu, s.w, d);
      if (lane >= d) s.x += x, s.y += y, s.z = add(s.z, z), s.w = add(s.w, w);
    }
    if (lane == 31) warp_sum[warp] = s;
    __syncthreads();
    int4 off = before;
    for (int w = 0; w < kWarps; ++w) {
      const int4 v = warp_sum[w];
      if (w < warp) off.x += v.x, off.y += v.y, off.z = add(off.z, v.z), off.w = add(off.w, v.w);
      before.x += v.x, before.y += v.y, before.z = add(before.z, v.z), before.w = add(before.w, v.w);
    }
    if (b < a.B) {
      const int4 upto = make_int4(off.x + s.x, off.y + s.y, add(off.z, s.z), add(off.w, s.w));
      Base v;
      v.items[0] = upto.x, v.items[1] = upto.y, v.units[0] = upto.z, v.units[1] = upto.w;
      a.base[b + 1] = v;
      if (keep) kept[b + 1] = v;
    }
    __syncthreads();
  }
  if (t == 0) {
    a.base[0] = Base{};
    if (keep) kept[0] = Base{};
  }
  const bool over = before.z == 0x7FFFFFFF || before.w == 0x7FFFFFFF;
  if (over && t == 0) set_status(a.status, MLA_DEV_BAD_OFFSETS);
  __syncthreads();
  // Threads 0 .. and 64 .. are the workers of class 0 and 1 (no more of them than
  // there are units, so that no part of a short line is empty).
  const int c = t >= 64, w = c ? t - 64 : t;
  const int items = c == 0 ? before.x : before.y, units = over ? 0 : c == 0 ? before.z : before.w;
  const int n = max(1, min(workers_of(a.pairs, c), units));
  const bool worker = w < n;
  auto length = [&](int item) {
    const int b = sequence_of(base, a.B, c, item);
    return (base[b + 1].units[c] - base[b].units[c]) / (base[b + 1].items[c] - base[b].items[c]);
  };
  int mine = 0;
  if (worker) {
    // Whole items, as many as no worker is overloaded by.
    int load = 0, k = 0;
    for (; !over && w + static_cast<long long>(k) * n < items; ++k) {
      load += length(w + k * n);
      if (load > units / n) break;
    }
    atomicMin(&whole[c], k);
  }
  __syncthreads();
  if (worker) {
    for (int k = 0; k < whole[c]; ++k) mine += length(w + k * n);
    // units (w + 1) / n - units w / n, rounded down both
    const int each = units / n, more = units - each * n;
    mine = each + more * (w + 1) / n - more * w / n - mine;
    rest[c][w] = mine;
    if (w == 0) a.schedule->whole[c] = whole[c], a.schedule->workers[c] = n;
  }
  __syncthreads();
  if (worker) {
    const int first = whole[c] * n;                 // the first item on the line
    int at = units;
    if (first < items && !over) {
      const int b = sequence_of(base, a.B, c, first);
      at = base[b].units[c] + (first - base[b].items[c]) * length(first);
    }
    for (int v = 0; v < w; ++v) at += rest[c][v];
    a.schedule->tail[c][w] = at;
    if (w == n - 1) a.schedule->tail[c][n] = at + mine;
  }
  if (over)                                         // nobody has work: no token has a result
    for (int i = t; i < a.T; i += kPlanThreads) a.token_seq[i] = -1;
}

// Bits of the tokens [8 group, 8 group + 8), by one CTA.  A key that a row does
// not see has weight 0, and 0 times infinity or NaN is NaN: rows with such values
// are left out of the products (a row of zeros is loaded instead), and who sees
// one gets NaN.  Only new tokens can be hidden from a row of their sequence.
template <int kThreads>
__device__ __forceinline__ void find_odd_rows(const ChunkPlanArgs& a, int group) {
  __shared__ unsigned bits;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) bits = 0;
  __syncthreads();
  // Every warp finds the rows of all eight tokens, token i in lane i: the sequence
  // of the first by a search, those of the others among the next 32.
  const int t0 = 8 * group, t = t0 + lane;
  const int first = last_of(a.B, [&](int b) { return a.iro[b] <= static_cast<uint32_t>(t0); });
  const int begins = first + 1 + lane;
  const uint32_t begin = begins < a.B ? a.iro[begins] : 0xFFFFFFFFu;
  int lo = first;
  for (int i = 0; i < 8; ++i) {
    const int more = __popc(__ballot_sync(0xffffffffu, begin <= static_cast<uint32_t>(t0 + i)));
    const int b = more < 32 ? first + more : last_of(a.B, [&](int b) { return a.iro[b] <= static_cast<uint32_t>(t0 + i); });
    if (lane == i) lo = b;
  }
  long long row = -1;
  if (lane < 8 && t < a.T) {
    const uint32_t q0 = a.iro[lo], q1 = a.iro[lo + 1], cached = a.cache_len[lo];
    if (q0 <= static_cast<uint32_t>(t) && static_cast<uint32_t>(t) < q1) {
      const long long pos = static_cast<long long>(cached) + (t - static_cast<long long>(q0)), j = pos / a.page_size;
      const int page = j < a.max_pages ? a.page_table[static_cast<size_t>(lo) * a.max_pages + j] : -1;
      if (page >= 0 && page < a.num_pages) row = static_cast<long long>(page) * a.page_size + (pos - j * a.page_size);
    }
  }
  constexpr int kWarps = kThreads / 32, kEach = (8 + kWarps - 1) / kWarps;
  uint4 v[kEach][2] = {};
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    const int i = warp + u * kWarps;
    const long long r = __shfl_sync(0xffffffffu, row, i & 7);
    if (i >= 8 || r < 0) continue;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.kv_cache) + r * 1152);
    v[u][0] = src[lane], v[u][1] = src[32 + lane];
  }
#pragma unroll
  for (int u = 0; u < kEach; ++u) {
    bool odd = false;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t x[4] = {v[u][e].x, v[u][e].y, v[u][e].z, v[u][e].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) odd |= (x[k] & 0x7F80u) == 0x7F80u || (x[k] & 0x7F800000u) == 0x7F800000u;
    }
    if (__any_sync(0xffffffffu, odd) && lane == 0) atomicOr(&bits, 1u << (warp + u * kWarps));
  }
  __syncthreads();
  if (threadIdx.x == 0 && t0 < a.T) a.odd_rows[group] = static_cast<uint8_t>(bits);
}

}  // namespace chunk
}  // namespace mla
