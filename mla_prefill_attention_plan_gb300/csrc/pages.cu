// The bookkeeping of the paged cache: page tables and reference counts (fork,
// reserve, free, compact), and the data that they move (page copies in every
// layer, accepted rows moved together).  The pages have no counterpart: they
// take a cache whose pages somebody else hands out ("mla_prefill_decode_graph_bf16",
// Args: kv_collection).
//
// The state of a pool is its reference counts alone: page p is free iff
// ref[p] == 0, and pages are handed out lowest first.  A result is therefore a
// function of the inputs, whatever order atomics take: sums commute, and every
// rank is a prefix sum over page ids or (sequence, page) order.
//
// The reserving and compacting kernels are one cluster each: what they compute
// is a chain of scans (who writes shared pages, how many pages each sequence
// wants, which pages are free) that other kernels could only share by more
// launches, and one SM alone reads a pool of 10^5 counts too slowly.  A warp
// owns a contiguous range of page ids, so a scan costs one barrier, not one a
// round.
#include <algorithm>
#include <atomic>

#include "kernels.cuh"

namespace mla {
namespace {

constexpr int kPoolCtas = 16;       // CTAs of a bookkeeping cluster (the most there can be), or one
constexpr int kPoolThreads = 1024;
constexpr int kPoolWarps = kPoolThreads / 32;

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }
__device__ __forceinline__ long long warp_sum64(int v) {     // of values >= 0
  return static_cast<long long>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(v) >> 16)) * 65536 +
         __reduce_add_sync(0xffffffffu, static_cast<unsigned>(v) & 0xFFFFu);
}
__device__ __forceinline__ int warp_scan(int v, int lane) {   // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}
// All threads of the CTAs that share the work.
template <int CTAS>
__device__ __forceinline__ void pool_sync() {
  if (CTAS > 1) cluster_sync();
  else __syncthreads();
}
__device__ __forceinline__ int ld_remote(const int* local, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(smem_u32(local), rank)) : "memory");
  return v;
}

// ============================================================ fork
// CTAs 0 .. dst_batch - 1 write a row of the new table; CTA dst_batch + a adds
// (children of row a) - 1 to the counts of the pages that row a holds.
__global__ void __launch_bounds__(256) fork_kernel(PagesForkArgs a) {
  pdl_enter();
  if (timed_out_before(a.status)) return;
  const int t = threadIdx.x;
  if (blockIdx.x < static_cast<unsigned>(a.dst_batch)) {
    const int b = blockIdx.x;
    const int p = a.parents[b];
    const bool ok = p >= 0 && p < a.src_batch;
    if (t == 0) {
      if (!ok && p != -1) set_status(a.status, MLA_DEV_BAD_OFFSETS);
      a.dst_lengths[b] = ok ? a.src_lengths[p] : 0u;
    }
    const int32_t* src = a.src_table + static_cast<size_t>(ok ? p : 0) * a.max_pages;
    int32_t* dst = a.dst_table + static_cast<size_t>(b) * a.max_pages;
    for (int j = t; j < a.max_pages; j += 256) {
      int v = ok ? src[j] : -1;
      if (v >= a.num_pages) {
        set_status(a.status, MLA_DEV_BAD_PAGE);
        v = -1;
      }
      dst[j] = v < 0 ? -1 : v;
    }
    return;
  }
  const int row = blockIdx.x - a.dst_batch;
  int n = 0;
  for (int b = t; b < a.dst_batch; b += 256) n += a.parents[b] == row;
  __shared__ int sums[8];
  n = warp_sum(n);
  if ((t & 31) == 0) sums[t >> 5] = n;
  __syncthreads();
  int more = -1;
#pragma unroll
  for (int w = 0; w < 8; ++w) more += sums[w];
  if (more == 0) return;
  const int32_t* src = a.src_table + static_cast<size_t>(row) * a.max_pages;
  for (int j = t; j < a.max_pages; j += 256) {
    const int v = src[j];
    if (v >= 0 && v < a.num_pages) atomicAdd(a.refs + v, more);
  }
}

// ============================================================ free
__global__ void __launch_bounds__(256) free_kernel(PagesFreeArgs a) {
  pdl_enter();
  if (timed_out_before(a.status)) return;
  const int b = blockIdx.x;
  const uint32_t len = a.lengths[b];
  const uint32_t keep = a.keep != nullptr ? min(len, a.keep[b]) : 0u;
  const uint32_t first = keep / a.page_size + (keep % a.page_size != 0);
  __syncthreads();                     // every thread has read the length (keep may be the same array)
  if (threadIdx.x == 0) a.lengths[b] = keep;
  int32_t* row = a.table + static_cast<size_t>(b) * a.max_pages;
  for (long long j = static_cast<long long>(first) + threadIdx.x; j < a.max_pages; j += 256) {
    const int v = row[j];
    if (v < 0) continue;
    row[j] = -1;
    // A count that is already zero stays so.
    if (v >= a.num_pages || atomicSub(a.refs + v, 1) <= 0) {
      if (v < a.num_pages) atomicAdd(a.refs + v, 1);
      set_status(a.status, MLA_DEV_BAD_PAGE);
    }
  }
}

// ============================================================ reserve
struct PoolSmem {
  int warp_count[kPoolWarps];     // free (live) pages in the warp's range
  int tally[4];                   // of this CTA: pages wanted (live), movers, free pages, flags
  int shared_tally[2];            // pages wanted and copies once the sharers are known
  int scan[kPoolWarps], scan2[kPoolWarps];
  int n_long, long_ones[kPoolThreads];
};

// The warp's contiguous range of page ids, a multiple of 128 long (an int4 a
// lane) so that 16-byte loads of an aligned array stay aligned.
template <int CTAS>
__device__ __forceinline__ void warp_range(int n, int rank, int warp, int& lo, int& hi) {
  const int parts = CTAS * kPoolWarps;
  const long long per = ((static_cast<long long>(n) + parts - 1) / parts + 127) / 128 * 128;
  const long long at = per * (rank * kPoolWarps + warp);
  lo = static_cast<int>(min(at, static_cast<long long>(n)));
  hi = static_cast<int>(min(at + per, static_cast<long long>(n)));
}

// Four counts from index i on; past the end of the range they read as `past`.
__device__ __forceinline__ int4 load4(const int32_t* p, int i, int hi, bool wide, int past) {
  if (wide && i + 4 <= hi) return __ldcg(reinterpret_cast<const int4*>(p + i));
  int4 v;
  v.x = i < hi ? __ldcg(p + i) : past;
  v.y = i + 1 < hi ? __ldcg(p + i + 1) : past;
  v.z = i + 2 < hi ? __ldcg(p + i + 2) : past;
  v.w = i + 3 < hi ? __ldcg(p + i + 3) : past;
  return v;
}

constexpr int kRowUnroll = 8;         // table entries that a lane has in flight
constexpr int kNoEntry = -0x7FFFFFFF - 1;   // (past the range; an entry below 0 is a missing page)
enum { kBadPage = 1, kShared = 2, kStop = 4 };

// The pages that sequence b writes to: [first, end) of its row, or none.
struct Touched {
  int first, end, len;
  bool part;      // the first of them holds rows that are to be kept
};
__device__ __forceinline__ bool touched(const PagesReserveArgs& a, int b, Touched& t) {
  const uint32_t len = a.lengths[b], n = a.fresh[b];
  t.first = t.end = 0;
  if (n == 0) return true;
  const unsigned long long end = (static_cast<unsigned long long>(len) + n + a.page_size - 1) / a.page_size;
  if (end > static_cast<unsigned long long>(a.max_pages)) return false;
  t.first = static_cast<int>(len / a.page_size);
  t.end = static_cast<int>(end);
  t.part = len % a.page_size != 0;
  return true;
}

// Sequences [b0, b1) of a CTA, 1024 at a time: those that write to few pages by
// a thread each (one_thread(b, pages)), the others by a warp each (one_warp).
constexpr int kFewPages = 4;
template <typename Thread, typename Warp>
__device__ __forceinline__ void for_sequences(const PagesReserveArgs& a, int b0, int b1, PoolSmem& sh, Thread one_thread,
                                              Warp one_warp) {
  for (int base = b0; base < b1; base += kPoolThreads) {
    __syncthreads();
    if (threadIdx.x == 0) sh.n_long = 0;
    __syncthreads();
    const int b = base + threadIdx.x;
    if (b < b1) {
      Touched s;
      const bool fits = touched(a, b, s);
      if (s.end - s.first <= kFewPages) one_thread(b, s, fits);
      else sh.long_ones[atomicAdd(&sh.n_long, 1)] = b;
    }
    __syncthreads();
    for (int i = threadIdx.x >> 5; i < sh.n_long; i += kPoolWarps) {
      Touched s;
      touched(a, sh.long_ones[i], s);
      one_warp(sh.long_ones[i], s);
    }
  }
}

template <int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kPoolThreads, 1) reserve_kernel(PagesReserveArgs a) {
  __shared__ PoolSmem sh;
  pdl_enter();
  const bool stop = timed_out_before(a.status);   // the CTAs agree on it below
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int rank = CTAS > 1 ? static_cast<int>(cluster_rank()) : 0;
  const bool wide = (reinterpret_cast<uintptr_t>(a.refs) & 15u) == 0;
  const int per = (a.batch + CTAS - 1) / CTAS;
  const int b0 = min(a.batch, rank * per), b1 = min(a.batch, b0 + per);
  if (t < 4) sh.tally[t] = 0;
  if (t < 2) sh.shared_tally[t] = 0;
  __syncthreads();

  // First look: missing pages are counted.  The scratch words of pages that are
  // there: their count now (the counts themselves change while others still
  // decide), writers, last writer.
  int flags = stop ? kStop : 0, wants = 0;
  auto look = [&](int v) {
    if (v < 0) return 1;
    if (v >= a.num_pages) {
      flags |= kBadPage;
    } else {
      const int r = a.refs[v];
      a.before[v] = r;
      a.writers[v] = 0;
      a.last[v] = -1;
      if (r > 1) flags |= kShared;
    }
    return 0;
  };
  for_sequences(a, b0, b1, sh,
                [&](int b, const Touched& s, bool fits) {
                  if (!fits) flags |= kBadPage;
                  const int32_t* row = a.table + static_cast<size_t>(b) * a.max_pages;
                  int missing = 0;
                  for (int j = s.first; j < s.end; ++j) missing += look(row[j]);
                  a.want[b] = make_int2(missing, 0);
                  wants += missing;
                },
                [&](int b, const Touched& s) {
                  const int32_t* row = a.table + static_cast<size_t>(b) * a.max_pages;
                  int missing = 0;
                  for (int j0 = s.first; j0 < s.end; j0 += 32 * kRowUnroll) {
                    int v[kRowUnroll];
#pragma unroll
                    for (int e = 0; e < kRowUnroll; ++e) {
                      const int j = j0 + e * 32 + lane;
                      v[e] = j < s.end ? row[j] : kNoEntry;
                    }
#pragma unroll
                    for (int e = 0; e < kRowUnroll; ++e)
                      if (v[e] != kNoEntry) missing += look(v[e]);
                  }
                  missing = warp_sum(missing);
                  if (lane == 0) {
                    a.want[b] = make_int2(missing, 0);
                    wants += missing;
                  }
                });
  int lo, hi, n_free = 0;
  warp_range<CTAS>(a.num_pages, rank, warp, lo, hi);
  for (int i = lo + 4 * lane; i < hi; i += 128 * 4) {
    int4 v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = load4(a.refs, i + 128 * e, hi, wide, 1);
#pragma unroll
    for (int e = 0; e < 4; ++e) n_free += (v[e].x == 0) + (v[e].y == 0) + (v[e].z == 0) + (v[e].w == 0);
  }
  n_free = warp_sum(n_free);
  wants = warp_sum(wants);
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (lane == 0) {
    sh.warp_count[warp] = n_free;
    atomicAdd(&sh.tally[2], n_free);
    if (wants) atomicAdd(&sh.tally[0], wants);
    if (flags) atomicOr(&sh.tally[3], flags);
  }
  pool_sync<CTAS>();
  // What the CTAs found: sums of all of them and of those before this one.
  int all = 0, free_before = 0, want_before = 0, copy_before = 0, copies = 0;
  long long want_total = 0, free_total = 0;
  {
    const bool on = lane < CTAS;
    const int w = on ? ld_remote(&sh.tally[0], lane) : 0, f = on ? ld_remote(&sh.tally[2], lane) : 0;
    all = __reduce_or_sync(0xffffffffu, on ? ld_remote(&sh.tally[3], lane) : 0);
    free_total = warp_sum(f);
    free_before = warp_sum(lane < rank ? f : 0);
    want_total = warp_sum64(w);
    want_before = warp_sum(lane < rank ? w : 0);
  }
  if (all & kStop) {
    pool_sync<CTAS>();    // no CTA leaves while another reads its shared memory
    return;
  }
  // A writer of a shared page takes a copy, but for the last one if nobody
  // else holds the page.
  auto takes = [&](int v, int b) {
    const int r = __ldcg(a.before + v), w = __ldcg(a.writers + v), l = __ldcg(a.last + v);
    return r > 1 && !(w >= r && l == b);
  };
  if (all & kShared) {
    auto count = [&](int v, int b) {
      if (v >= 0 && v < a.num_pages && __ldcg(a.before + v) > 1) {
        atomicAdd(a.writers + v, 1);
        atomicMax(a.last + v, b);
      }
    };
    for_sequences(a, b0, b1, sh,
                  [&](int b, const Touched& s, bool) {
                    for (int j = s.first; j < s.end; ++j) count(a.table[static_cast<size_t>(b) * a.max_pages + j], b);
                  },
                  [&](int b, const Touched& s) {
                    for (int j = s.first + lane; j < s.end; j += 32)
                      count(a.table[static_cast<size_t>(b) * a.max_pages + j], b);
                  });
    pool_sync<CTAS>();
    int want_sum = 0, copy_sum = 0;
    for_sequences(a, b0, b1, sh,
                  [&](int b, const Touched& s, bool) {
                    int want = 0, copy = 0;
                    for (int j = s.first; j < s.end; ++j) {
                      const int v = a.table[static_cast<size_t>(b) * a.max_pages + j];
                      if (v >= a.num_pages) continue;
                      const bool shared = v >= 0 && takes(v, b);
                      want += v < 0 || shared;
                      copy += shared && s.part && j == s.first;
                    }
                    a.want[b] = make_int2(want, copy);
                    want_sum += want;
                    copy_sum += copy;
                  },
                  [&](int b, const Touched& s) {
                    int want = 0, copy = 0;
                    for (int j = s.first + lane; j < s.end; j += 32) {
                      const int v = a.table[static_cast<size_t>(b) * a.max_pages + j];
                      if (v >= a.num_pages) continue;
                      const bool shared = v >= 0 && takes(v, b);
                      want += v < 0 || shared;
                      copy += shared && s.part && j == s.first;
                    }
                    want = warp_sum(want);
                    copy = warp_sum(copy);
                    if (lane == 0) {
                      a.want[b] = make_int2(want, copy);
                      want_sum += want;
                      copy_sum += copy;
                    }
                  });
    want_sum = warp_sum(want_sum);
    copy_sum = warp_sum(copy_sum);
    if (lane == 0) {
      if (want_sum) atomicAdd(&sh.shared_tally[0], want_sum);
      if (copy_sum) atomicAdd(&sh.shared_tally[1], copy_sum);
    }
    pool_sync<CTAS>();
    const bool on = lane < CTAS;
    const int w = on ? ld_remote(&sh.shared_tally[0], lane) : 0, c = on ? ld_remote(&sh.shared_tally[1], lane) : 0;
    want_total = warp_sum64(w);
    want_before = warp_sum(lane < rank ? w : 0);
    copies = warp_sum(c);
    copy_before = warp_sum(lane < rank ? c : 0);
  }
  const bool ok = !(all & kBadPage) && want_total <= free_total;
  if (!ok) copies = 0;
  if (rank == 0 && t == 0) {
    *a.copy_count = copies;
    if (!ok) set_status(a.status, (all & kBadPage) ? MLA_DEV_BAD_PAGE : MLA_DEV_NO_PAGES);
  }
  for (int i = copies + rank * kPoolThreads + t; i < a.batch; i += CTAS * kPoolThreads)
    a.copy_src[i] = a.copy_dst[i] = -1;
  if (ok) {
    // The free pages in order, as many as are wanted.
    int at = free_before;
    at += warp_sum(lane < warp ? sh.warp_count[lane] : 0);
    for (int i = lo; i < hi && at < want_total; i += 128 * 2) {
      int4 v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) v[e] = load4(a.refs, i + 128 * e + 4 * lane, hi, wide, 1);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int f[4] = {v[e].x == 0, v[e].y == 0, v[e].z == 0, v[e].w == 0};
        const int mine = f[0] + f[1] + f[2] + f[3];
        const int upto = warp_scan(mine, lane);
        int k = at + upto - mine;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (f[u] && k < want_total) a.free_list[k] = i + 128 * e + 4 * lane + u;
          k += f[u];
        }
        at += __shfl_sync(0xffffffffu, upto, 31);
      }
    }
    // Where each sequence's pages and copies begin.
    for (int base = b0; base < b1; base += kPoolThreads) {
      const int b = base + t;
      const int2 w = b < b1 ? __ldcg(a.want + b) : make_int2(0, 0);
      const int sw = warp_scan(w.x, lane), sc = warp_scan(w.y, lane);
      __syncthreads();
      if (lane == 31) sh.scan[warp] = sw, sh.scan2[warp] = sc;
      __syncthreads();
      const int ow = sh.scan[lane], oc = sh.scan2[lane];      // (as many warps as lanes)
      const int bw = warp_sum(lane < warp ? ow : 0), bc = warp_sum(lane < warp ? oc : 0);
      if (b < b1) a.want[b] = make_int2(want_before + bw + sw - w.x, copy_before + bc + sc - w.y);
      want_before += warp_sum(ow);
      copy_before += warp_sum(oc);
    }
  }
  pool_sync<CTAS>();      // the last one: no CTA reads another's shared memory behind it
  if (!ok) return;
  auto put = [&](int32_t* row, int j, int v, bool shared, int page, const Touched& s, int copy) {
    row[j] = page;
    a.refs[page] = 1;
    if (shared) {
      atomicSub(a.refs + v, 1);
      if (s.part && j == s.first) {
        a.copy_src[copy] = v;
        a.copy_dst[copy] = page;
      }
    }
  };
  for_sequences(a, b0, b1, sh,
                [&](int b, const Touched& s, bool) {
                  if (s.first == s.end) return;
                  const int2 base = __ldcg(a.want + b);
                  int32_t* row = a.table + static_cast<size_t>(b) * a.max_pages;
                  int at = base.x;
                  for (int j = s.first; j < s.end; ++j) {
                    const int v = row[j];
                    const bool shared = (all & kShared) && v >= 0 && takes(v, b);
                    if (v < 0 || shared) put(row, j, v, shared, __ldcg(a.free_list + at++), s, base.y);
                  }
                },
                [&](int b, const Touched& s) {
                  const int2 base = __ldcg(a.want + b);
                  int32_t* row = a.table + static_cast<size_t>(b) * a.max_pages;
                  int at = base.x;
                  for (int j0 = s.first; j0 < s.end; j0 += 32 * kRowUnroll) {
                    int v[kRowUnroll], rank_of[kRowUnroll], page[kRowUnroll];
                    bool shared[kRowUnroll];
#pragma unroll
                    for (int e = 0; e < kRowUnroll; ++e) {
                      const int j = j0 + e * 32 + lane;
                      v[e] = j < s.end ? row[j] : kNoEntry;
                    }
#pragma unroll
                    for (int e = 0; e < kRowUnroll; ++e) {
                      shared[e] = (all & kShared) && v[e] >= 0 && takes(v[e], b);
                      const bool want = (v[e] < 0 && v[e] != kNoEntry) || shared[e];
                      const unsigned m = __ballot_sync(0xffffffffu, want);
                      rank_of[e] = want ? at + __popc(m & ((1u << lane) - 1)) : -1;
                      at += __popc(m);
                    }
#pragma unroll
                    for (int e = 0; e < kRowUnroll; ++e)
                      page[e] = rank_of[e] >= 0 ? __ldcg(a.free_list + rank_of[e]) : -1;
#pragma unroll
                    for (int e = 0; e < kRowUnroll; ++e)
                      if (rank_of[e] >= 0) put(row, j0 + e * 32 + lane, v[e], shared[e], page[e], s, base.y);
                  }
                });
}

// ============================================================ compact
// With L live pages, the k-th highest live page moves to the k-th lowest free
// one for as long as that is lower, which is for exactly the live pages >= L:
// as many free pages lie below L.  So each page finds from its own rank
// whether it takes part.
template <int CTAS>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(kPoolThreads, 1) compact_kernel(PagesCompactArgs a) {
  __shared__ PoolSmem sh;
  pdl_enter();
  const bool stop = timed_out_before(a.status);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int rank = CTAS > 1 ? static_cast<int>(cluster_rank()) : 0;
  const bool wide = (reinterpret_cast<uintptr_t>(a.refs) & 15u) == 0;
  if (t < 4) sh.tally[t] = 0;
  __syncthreads();
  int lo, hi, n_live = 0;
  warp_range<CTAS>(a.num_pages, rank, warp, lo, hi);
  for (int i = lo + 4 * lane; i < hi; i += 128 * 4) {
    int4 v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = load4(a.refs, i + 128 * e, hi, wide, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) n_live += (v[e].x > 0) + (v[e].y > 0) + (v[e].z > 0) + (v[e].w > 0);
  }
  n_live = warp_sum(n_live);
  if (lane == 0) {
    sh.warp_count[warp] = n_live;
    atomicAdd(&sh.tally[0], n_live);
  }
  if (stop) sh.tally[3] = kStop;
  pool_sync<CTAS>();
  const bool on = lane < CTAS;
  const int found = on ? ld_remote(&sh.tally[0], lane) : 0;
  const int all = __reduce_or_sync(0xffffffffu, on ? ld_remote(&sh.tally[3], lane) : 0);
  const int live = warp_sum(found);
  int at = warp_sum(lane < rank ? found : 0);
  if (all & kStop) {
    pool_sync<CTAS>();
    return;
  }
  at += warp_sum(lane < warp ? sh.warp_count[lane] : 0);
  int movers = 0;
  for (int i = lo; i < hi; i += 128) {
    const int4 v = load4(a.refs, i + 4 * lane, hi, wide, 0);
    const int is[4] = {v.x > 0, v.y > 0, v.z > 0, v.w > 0};
    const int mine = is[0] + is[1] + is[2] + is[3];
    const int upto = warp_scan(mine, lane);
    int k = at + upto - mine;                       // live pages below p
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int p = i + 4 * lane + e;
      if (p < hi) {
        if (is[e] && p >= live) {
          ++movers;
          if (live - 1 - k < a.max_copies) a.copy_src[live - 1 - k] = p;
        } else if (!is[e] && p < live && p - k < a.max_copies) {
          a.copy_dst[p - k] = p;
        }
      }
      k += is[e];
    }
    at += __shfl_sync(0xffffffffu, upto, 31);
  }
  movers = warp_sum(movers);
  if (lane == 0 && movers) atomicAdd(&sh.tally[1], movers);
  pool_sync<CTAS>();
  const int n = min(warp_sum(on ? ld_remote(&sh.tally[1], lane) : 0), a.max_copies);
  if (rank == 0 && t == 0) *a.copy_count = n;
  for (int k = rank * kPoolThreads + t; k < a.max_copies; k += CTAS * kPoolThreads) {
    if (k < n) {
      const int p = __ldcg(a.copy_src + k), q = __ldcg(a.copy_dst + k);
      a.refs[q] = a.refs[p];
      a.refs[p] = 0;
      a.moved[p] = k;
    } else {
      a.copy_src[k] = a.copy_dst[k] = -1;
    }
  }
  pool_sync<CTAS>();      // no CTA leaves while another reads its shared memory
}

// Table entries of moved pages; bad entries are reported whether any page moves or
// not.  A page's word of the scratch is only good if the move that it names is that
// page's.
__global__ void __launch_bounds__(256) remap_kernel(PagesCompactArgs a) {
  pdl_enter();
  if (timed_out_before(a.status)) return;
  const int n = *a.copy_count;
  const int lowest = n > 0 ? a.copy_src[n - 1] : a.num_pages;     // sources come highest first
  const long long entries = static_cast<long long>(a.batch) * a.max_pages;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < entries; i += gridDim.x * 256ll) {
    const int v = a.table[i];
    if (v < lowest) continue;
    if (v >= a.num_pages) {
      set_status(a.status, MLA_DEV_BAD_PAGE);
      continue;
    }
    const int k = a.moved[v];
    if (k >= 0 && k < n && a.copy_src[k] == v) a.table[i] = a.copy_dst[k];
  }
}

// ============================================================ copies
// Page copies in every layer: pieces of kCopyPiece bytes, four vectors a
// thread in flight before the first is stored.  Bound by HBM: each byte is
// read and written once.
constexpr int kCopyThreads = 256, kCopyUnroll = 4;

template <typename V>
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(PagesCopyArgs a) {
  pdl_enter();
  if (timed_out_before(a.status)) return;
  const int n = min(*a.count, a.max_copies);
  const unsigned per_piece = kCopyThreads * kCopyUnroll;
  const unsigned vecs = static_cast<unsigned>(a.page_bytes / sizeof(V));
  const unsigned pieces = (vecs + per_piece - 1) / per_piece;
  const long long units = static_cast<long long>(max(n, 0)) * a.layers * pieces;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const unsigned piece = static_cast<unsigned>(u % pieces);
    const long long v = u / pieces;
    const int k = static_cast<int>(v % n), layer = static_cast<int>(v / n);
    const int src = a.src[k], dst = a.dst[k];
    if (static_cast<unsigned>(src) >= static_cast<unsigned>(a.num_pages) ||
        static_cast<unsigned>(dst) >= static_cast<unsigned>(a.num_pages)) {
      if (threadIdx.x == 0) set_status(a.status, MLA_DEV_BAD_PAGE);
      continue;
    }
    char* base = a.cache + static_cast<size_t>(layer) * a.layer_stride;
    const V* from = reinterpret_cast<const V*>(base + static_cast<size_t>(src) * a.page_bytes);
    V* to = reinterpret_cast<V*>(base + static_cast<size_t>(dst) * a.page_bytes);
    const unsigned i0 = piece * per_piece + threadIdx.x;
    V x[kCopyUnroll];
#pragma unroll
    for (int e = 0; e < kCopyUnroll; ++e)
      if (i0 + e * kCopyThreads < vecs) x[e] = __ldcs(from + i0 + e * kCopyThreads);
#pragma unroll
    for (int e = 0; e < kCopyUnroll; ++e)
      if (i0 + e * kCopyThreads < vecs) __stcs(to + i0 + e * kCopyThreads, x[e]);
  }
}

// Accepted rows of a sequence (blockIdx.x) in layers blockIdx.y, + gridDim.y, ..
// The list ascends strictly, so keep[k] >= k: a round reads rows of the list
// before any of it is stored, and what it stores lies below all that later
// rounds read.  Where the rows are is found once for all layers.  A thread holds
// one vector of kKeepUnroll rows.
constexpr int kKeepThreads = 288, kKeepUnroll = 4, kKeepRound = 1024;

template <typename V>
__global__ void __launch_bounds__(kKeepThreads) keep_rows_kernel(KeepRowsArgs a) {
  __shared__ int from[kKeepRound], to[kKeepRound];
  pdl_enter();
  if (timed_out_before(a.status)) return;
  const int b = blockIdx.x, t = threadIdx.x;
  const int n = a.counts[b];
  if (n <= 0) return;
  const int32_t* keep = a.keep + static_cast<size_t>(b) * a.keep_stride;
  const int32_t* pages = a.table + static_cast<size_t>(b) * a.max_pages;
  const uint32_t len = a.lengths[b];
  // The row of position len + i, or -1.
  auto row_of = [&](int i) {
    const unsigned long long p = static_cast<unsigned long long>(len) + static_cast<unsigned>(i);
    const unsigned long long j = p / static_cast<unsigned>(a.page_size);
    if (j >= static_cast<unsigned long long>(a.max_pages)) return -1;
    const int page = pages[j];
    if (page < 0 || page >= a.num_pages) return -1;
    return page * a.page_size + static_cast<int>(p - j * a.page_size);
  };
  // The whole list is looked over first: a sequence is moved whole or not at all.
  int bad = n > a.keep_stride ? 1 : 0;
  if (!bad)
    for (int k = t; k < n; k += kKeepThreads) {
      const int i = keep[k], before = k > 0 ? keep[k - 1] : -1;
      int src = -1, dst = -1;
      if (i < 0 || before >= i) bad |= 1;
      else if ((src = row_of(i)) < 0 || (dst = row_of(k)) < 0) bad |= 2;
      if (k < kKeepRound) from[k] = src, to[k] = dst;
    }
  const bool bad_list = __syncthreads_or(bad & 1), bad_page = __syncthreads_or(bad & 2);
  if (bad_list || bad_page) {
    if (t == 0) set_status(a.status, bad_list ? MLA_DEV_BAD_OFFSETS : MLA_DEV_BAD_PAGE);
    return;
  }
  const int cols = static_cast<int>(a.row_bytes / sizeof(V));
  const int wide = min(cols, kKeepThreads);             // threads on a row
  const int lines = kKeepThreads / wide;                // rows side by side
  const int line = t / wide, col0 = t - line * wide;
  for (int first = 0; first < n; first += kKeepRound) {
    const int m = min(n - first, kKeepRound);
    if (first > 0) {                                    // (the first of them are there already)
      __syncthreads();
      for (int k = t; k < m; k += kKeepThreads) from[k] = row_of(keep[first + k]), to[k] = row_of(first + k);
      __syncthreads();
    }
    for (int layer = blockIdx.y; layer < a.layers; layer += gridDim.y) {
      char* base = a.cache + static_cast<size_t>(layer) * a.layer_stride;
      for (int c0 = 0; c0 < cols; c0 += wide) {
        const int c = c0 + col0;
        const bool on = line < lines && c < cols;
        for (int k0 = 0; k0 < m; k0 += lines * kKeepUnroll) {
          V x[kKeepUnroll];
#pragma unroll
          for (int e = 0; e < kKeepUnroll; ++e) {
            const int k = k0 + e * lines + line;
            if (on && k < m && from[k] != to[k])
              x[e] = reinterpret_cast<const V*>(base + static_cast<size_t>(from[k]) * a.row_bytes)[c];
          }
          __syncthreads();
#pragma unroll
          for (int e = 0; e < kKeepUnroll; ++e) {
            const int k = k0 + e * lines + line;
            if (on && k < m && from[k] != to[k])
              reinterpret_cast<V*>(base + static_cast<size_t>(to[k]) * a.row_bytes)[c] = x[e];
          }
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_pages_fork(const PagesForkArgs& a, cudaStream_t stream) {
  const int grid = a.dst_batch + a.src_batch;
  if (grid == 0) return cudaSuccess;
  return launch_pdl(fork_kernel, dim3(grid), dim3(256), 0, stream, a);
}

cudaError_t launch_pages_free(const PagesFreeArgs& a, cudaStream_t stream) {
  if (a.batch == 0) return cudaSuccess;
  return launch_pdl(free_kernel, dim3(a.batch), dim3(256), 0, stream, a);
}

// One CTA where there is little to look at (a pool's counts, the tables'
// entries): it has no cluster barriers to wait at, nor atomics on words that
// other SMs hold.  (256 samples of 16 prompts, their copies included: 68 us with
// one CTA, 79 with 16.  512 prompts in 171386 pages have 16: 28 us; the counts
// alone are 670 KB.)
static bool one_cta(int num_pages, int batch, int max_pages) {
  return num_pages <= 32768 && batch <= kPoolThreads && static_cast<long long>(batch) * max_pages <= 65536;
}

// Clusters of more than 8 CTAs have to be allowed, once a device and kernel.
// (Two threads may both do it: it is the same call.)
using DeviceFlags = std::atomic<bool>[64];
static cudaError_t allow_big_clusters(const void* kernel, DeviceFlags& allowed) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && allowed[dev].load(std::memory_order_acquire))) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && dev < 64) allowed[dev].store(true, std::memory_order_release);
  return e;
}

cudaError_t launch_pages_reserve(const PagesReserveArgs& a, cudaStream_t stream) {
  if (one_cta(a.num_pages, a.batch, a.max_pages))
    return launch_pdl(reserve_kernel<1>, dim3(1), dim3(kPoolThreads), 0, stream, a);
  static DeviceFlags allowed;
  cudaError_t e = allow_big_clusters(reinterpret_cast<const void*>(reserve_kernel<kPoolCtas>), allowed);
  if (e != cudaSuccess) return e;
  return launch_pdl(reserve_kernel<kPoolCtas>, dim3(kPoolCtas), dim3(kPoolThreads), 0, stream, a);
}

cudaError_t launch_pages_compact(const PagesCompactArgs& a, cudaStream_t stream) {
  cudaError_t e;
  if (one_cta(a.num_pages, 0, 0)) {
    e = launch_pdl(compact_kernel<1>, dim3(1), dim3(kPoolThreads), 0, stream, a);
  } else {
    static DeviceFlags allowed;
    if ((e = allow_big_clusters(reinterpret_cast<const void*>(compact_kernel<kPoolCtas>), allowed)) != cudaSuccess)
      return e;
    e = launch_pdl(compact_kernel<kPoolCtas>, dim3(kPoolCtas), dim3(kPoolThreads), 0, stream, a);
  }
  if (e != cudaSuccess) return e;
  const long long entries = static_cast<long long>(a.batch) * a.max_pages;
  if (entries == 0) return cudaSuccess;
  const int grid = static_cast<int>(std::min<long long>((entries + 255) / 256, 4ll * sm_count()));
  return launch_pdl(remap_kernel, dim3(grid), dim3(256), 0, stream, a);
}

cudaError_t launch_pages_copy(const PagesCopyArgs& a, cudaStream_t stream) {
  const bool wide = ((reinterpret_cast<uintptr_t>(a.cache) | a.page_bytes | a.layer_stride) & 15u) == 0;
  const long long vecs = a.page_bytes / (wide ? 16 : 4);
  const long long pieces = (vecs + kCopyThreads * kCopyUnroll - 1) / (kCopyThreads * kCopyUnroll);
  const long long units = std::min<long long>(static_cast<long long>(a.max_copies) * a.layers, 1ll << 40) * pieces;
  if (units == 0) return cudaSuccess;
  const int grid = static_cast<int>(std::min<long long>(units, 8ll * sm_count()));
  return wide ? launch_pdl(pages_copy_kernel<uint4>, dim3(grid), dim3(kCopyThreads), 0, stream, a)
              : launch_pdl(pages_copy_kernel<unsigned>, dim3(grid), dim3(kCopyThreads), 0, stream, a);
}

cudaError_t launch_keep_rows(const KeepRowsArgs& a, cudaStream_t stream) {
  if (a.batch == 0 || a.layers == 0) return cudaSuccess;
  const bool wide = ((reinterpret_cast<uintptr_t>(a.cache) | a.row_bytes | a.layer_stride) & 15u) == 0;
  // One wave of CTAs (7 fit an SM), each for several layers where there are many.
  const int most = std::max(1, 7 * sm_count() / a.batch);
  const dim3 grid(a.batch, std::min(a.layers, most));
  return wide ? launch_pdl(keep_rows_kernel<uint4>, grid, dim3(kKeepThreads), 0, stream, a)
              : launch_pdl(keep_rows_kernel<unsigned>, grid, dim3(kKeepThreads), 0, stream, a);
}

}  // namespace mla
