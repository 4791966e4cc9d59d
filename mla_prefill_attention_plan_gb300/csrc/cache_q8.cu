// The 8-bit latent cache: e4m3 rows of 576 values with one float32 scale, a
// power of two, for each block of scale_block consecutive slots of a page.
// Writing (RMSNorm, RoPE, quantisation) and the gather of one plan chunk as
// bf16 rows.
//
// A block's scale is the smallest power of two s with |value| <= 448 s for
// every value of its rows.  Rows arrive over many calls, so the scale may have
// to grow: the rows before are then requantised by the ratio of the scales.
// The ratio is a power of two, so that changes their codes' exponents only and
// is exact but for codes that leave e4m3's normal range.
#include "kernels.cuh"

namespace mla {

namespace {

constexpr int kWriteThreads = 256;
constexpr int kWriteWarps = kWriteThreads / 32;
constexpr float kInf = __builtin_huge_valf();

// hi + lo += x, keeping the rounding error of the sum in lo (Knuth's two-sum; a
// hi that overflows leaves lo as NaN).
__device__ __forceinline__ void add_two(float& hi, float& lo, float x) {
  const float s = hi + x;
  const float b = s - hi;
  lo += (hi - (s - b)) + (x - b);
  hi = s;
}

// a c - b d with one rounding of each product's error taken back (Kahan's; the
// plain form loses up to three roundings, which moves codes next to a border).
// An infinite product has no error.
__device__ __forceinline__ float diff_of_products(float a, float c, float b, float d) {
  const float w = b * d;
  const float e = fmaf(-b, d, w), r = fmaf(a, c, -w);
  return fabsf(w) < kInf ? r + e : r;
}
__device__ __forceinline__ float2 rotate2(float re, float im, float c, float s) {
  return make_float2(diff_of_products(re, c, im, s), diff_of_products(re, s, -im, c));
}

// One row's 576 values before quantisation, held by a warp: lane l has latent
// values 8l..8l+7 and 256+8l..256+8l+7 and rope values 2l, 2l+1.
struct RowValues {
  float y[16];
  float2 rope;
};

__device__ __forceinline__ RowValues row_values(const uint16_t* __restrict__ row, const float* __restrict__ gamma,
                                                const float* __restrict__ freq, float eps) {
  const int lane = threadIdx.x & 31;
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(row) + lane);
  const uint4 b = __ldg(reinterpret_cast<const uint4*>(row) + 32 + lane);
  const uint32_t r = __ldg(reinterpret_cast<const uint32_t*>(row + 512) + lane);
  const float2 f = __ldg(reinterpret_cast<const float2*>(freq) + lane);
  const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  RowValues v;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v.y[2 * i] = bf16_lo(u[i]);
    v.y[2 * i + 1] = bf16_hi(u[i]);
  }
  float hi, lo;
  // Once, but for rows whose squares leave fp32's range: those are scaled by a
  // power of two first, which the norm takes back.
#pragma unroll 1
  for (bool once = true;; once = false) {
    // Sum of squares in two floats (a bf16 square is exact in fp32).
    hi = 0.f;
    lo = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) add_two(hi, lo, v.y[i] * v.y[i]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const float oh = __shfl_xor_sync(0xffffffffu, hi, d), ol = __shfl_xor_sync(0xffffffffu, lo, d);
      // Both lanes of a pair add the same two numbers in the same order.
      const bool up = (lane & d) != 0;
      float h = up ? oh : hi, l = up ? ol : lo;
      add_two(h, l, up ? hi : oh);
      hi = h;
      lo = l + (up ? lo : ol);
    }
    if (__builtin_expect(!once || (hi >= 0x1p-100f && hi <= 0x1p126f), 1)) break;   // (the same in every lane)
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v.y[i]));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (m == kInf) lo = 0.f;                           // an infinite value: the others become 0, it NaN
    if (m == kInf || (m < 1.f && eps >= 0x1p-80f)) break;
    const float k = m < 1.f ? 0x1p100f : 0x1p-80f;
    eps = eps * k * k;
#pragma unroll
    for (int i = 0; i < 16; ++i) v.y[i] *= k;
  }
  // 1 / sqrt(mean + eps) as rh + rl: the hardware's approximation and one
  // Newton step whose residual 1 - s rh^2 is formed in two floats.
  float sh = hi * (1.0f / 512.0f), sl = lo * (1.0f / 512.0f);
  add_two(sh, sl, eps);
  const float rh = rsqrtf(sh);
  const float th = rh * rh, tl = fmaf(rh, rh, -th);
  const float res = fmaf(-sh, th, 1.0f) - fmaf(sh, tl, sl * th);
  const float rl = sh < kInf ? 0.5f * rh * res : 0.f;
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const float4 g = __ldg(reinterpret_cast<const float4*>(gamma + (i < 8 ? 0 : 256) + 8 * lane) + ((i & 4) >> 2));
    const float gv[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float p = v.y[i + k] * gv[k];
      const float e = fmaf(v.y[i + k], gv[k], -p);
      // rh + rl is finite unless the row is all zero with eps 0 (then NaN, as x / 0).
      v.y[i + k] = fmaf(p, rh, fmaf(p, rl, e * rh));
    }
  }
  v.rope = rotate2(bf16_lo(r), bf16_hi(r), f.x, f.y);
  return v;
}

__device__ __forceinline__ float row_amax(const RowValues& v) {
  float m = fmaxf(fabsf(v.rope.x), fabsf(v.rope.y));
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v.y[i]));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  return m;
}

__device__ __forceinline__ void store_row(uint8_t* __restrict__ dst, const RowValues& v, float inv) {
  const int lane = threadIdx.x & 31;
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = static_cast<uint32_t>(pack_e4m3(v.y[4 * i] * inv, v.y[4 * i + 1] * inv)) |
           (static_cast<uint32_t>(pack_e4m3(v.y[4 * i + 2] * inv, v.y[4 * i + 3] * inv)) << 16);
  reinterpret_cast<uint2*>(dst)[lane] = make_uint2(c[0], c[1]);
  reinterpret_cast<uint2*>(dst + 256)[lane] = make_uint2(c[2], c[3]);
  reinterpret_cast<uint16_t*>(dst + 512)[lane] = pack_e4m3(v.rope.x * inv, v.rope.y * inv);
}

// Four e4m3 codes times a power of two, back to e4m3.
__device__ __forceinline__ uint32_t requantise4(uint32_t c, float ratio) {
  const float2 a = f16x2_to_float2(e4m3x2_to_f16x2(static_cast<uint16_t>(c & 0xFFFFu)));
  const float2 b = f16x2_to_float2(e4m3x2_to_f16x2(static_cast<uint16_t>(c >> 16)));
  return static_cast<uint32_t>(pack_e4m3(a.x * ratio, a.y * ratio)) |
         (static_cast<uint32_t>(pack_e4m3(b.x * ratio, b.y * ratio)) << 16);
}

// Position of the last of n ascending offsets that is not above x (0 if none):
// 32 probes of a warp at a time.
__device__ __forceinline__ int last_offset(const uint32_t* __restrict__ at, int n, uint32_t x) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
#pragma unroll 1
  for (int hi = n; hi - lo > 1;) {
    const int step = (hi - lo + 31) / 32;
    const long long i = lo + static_cast<long long>(lane) * step;
    const int below = __popc(__ballot_sync(0xffffffffu, i < hi && __ldg(at + i) <= x));
    lo += max(below - 1, 0) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// Position of token t in its sequence b's context, or -1 (reported).
__device__ __forceinline__ int token_position(const CacheWriteQ8Args& a, int t, int b) {
  const uint32_t first = __ldg(a.iro + b), end = __ldg(a.iro + b + 1), cached = __ldg(a.cache_len + b);
  if (first <= static_cast<uint32_t>(t) && static_cast<uint32_t>(t) < end) {
    const uint64_t p = static_cast<uint64_t>(cached) + (static_cast<uint32_t>(t) - first);
    if (p < static_cast<uint64_t>(a.max_seq_len)) return static_cast<int>(p);
  }
  set_status(a.status, MLA_DEV_BAD_OFFSETS);
  return -1;
}

// The first a.row_ctas CTAs write the cache, each the rows of all blocks that
// begin (or are entered) at one of its a.chunk tokens; the others rotate the
// query heads, a token at a time.  HBM-bound: per token 1152 bytes of latent
// read, 576 written, 256 of frequencies, and 4 * 64 * H of queries read and
// written.
//
// Rows: a block's rows are taken by a group of warps (eight, or as many as the
// block has slots), a row a warp: first their largest value, then, with the
// scale known, the codes (the rows are read again, from L1).  64 rows take some
// 25 us that way, bound by latency, so these CTAs come first and run under the
// others: with the two kinds of work in one CTA per token, 8 prompts of 256 to
// 2048 tokens, 128 heads, took 75 us, now 55 (5.6 TB/s).
//
// Queries: a thread's first four pieces (all of them with 128 heads) are read
// before anything is known of the token, over the chain of reads that finds its
// position.
constexpr int kMaxChunk = 128;   // tokens of a row CTA

struct RowJob {
  long long row;                 // cache row of the first token
  int t, pos, slot, rows;        // first token, its position and slot in the block, rows to write
};
struct WriteSmem {
  float amax[kWriteWarps];
  int jobs, pos;
  RowJob job[kMaxChunk];
};

__device__ __forceinline__ void write_rows(const CacheWriteQ8Args& a, WriteSmem& sh, int t0) {
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint16_t* latent = static_cast<const uint16_t*>(a.kv_latent);
  uint8_t* cache = static_cast<uint8_t*>(a.kv_cache);
  if (tid == 0) sh.jobs = 0;
  __syncthreads();
  if (32 * warp < a.chunk) {
    const int t = t0 + tid;
    int b = last_offset(a.iro, a.B, static_cast<uint32_t>(t0));
    if (tid < a.chunk && t < a.T) {
      while (b + 1 < a.B && __ldg(a.iro + b + 1) <= static_cast<uint32_t>(t)) ++b;
      const int pos = token_position(a, t, b);
      const int slot = pos < 0 ? 1 : pos % a.scale_block;
      const uint32_t first = __ldg(a.iro + b), end = __ldg(a.iro + b + 1);
      if (pos >= 0 && (slot == 0 || static_cast<uint32_t>(t) == first)) {
        // This block's new rows: up to its end, the sequence's last new
        // token, the last row of the call and the last position.
        int rows = a.scale_block - slot;
        rows = static_cast<int>(min(static_cast<uint32_t>(rows), min(end, static_cast<uint32_t>(a.T)) - t));
        rows = min(rows, a.max_seq_len - pos);
        const int pidx = pos / a.page_size;
        const int page = pidx < a.max_pages ? __ldg(a.page_table + static_cast<size_t>(b) * a.max_pages + pidx) : -1;
        if (page >= 0 && page < a.num_pages) {
          RowJob& j = sh.job[atomicAdd(&sh.jobs, 1)];   // (in any order: jobs do not meet)
          j.row = static_cast<long long>(page) * a.page_size + pos % a.page_size;
          j.t = t;
          j.pos = pos;
          j.slot = slot;
          j.rows = rows;
        } else {
          set_status(a.status, MLA_DEV_BAD_PAGE);
        }
      }
    }
  }
  __syncthreads();
  const int width = a.group_warps, group = warp / width, part = warp - group * width;
  const int threads = 32 * width, me = tid - group * threads;
  auto sync = [&] { asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(group + 1), "r"(threads) : "memory"); };
#pragma unroll 1
  for (int i = group; i < sh.jobs; i += kWriteWarps / width) {
    const RowJob j = sh.job[i];
    const uint16_t* src = latent + static_cast<size_t>(j.t) * 576;
    RowValues v;
    float m = 0.f;
#pragma unroll 1
    for (int r = part; r < j.rows; r += width) {
      v = row_values(src + static_cast<size_t>(r) * 576, a.gamma, a.freqs + static_cast<size_t>(j.pos + r) * 64, a.eps);
      m = fmaxf(m, row_amax(v));
    }
    if ((tid & 31) == 0) sh.amax[warp] = m;
    sync();
    for (int w = 0; w < width; ++w) m = fmaxf(m, sh.amax[group * width + w]);
    float scale = pow2_scale(m);
    float* sp = a.kv_scales + j.row / a.scale_block;
    if (j.slot > 0) {
      // Rows before, written by earlier calls under the block's scale.
      const float was = *sp;
      if (was > 0.f && was < __int_as_float(0x7f800000)) {
        if (was >= scale) {
          scale = was;
        } else {
          uint4* old = reinterpret_cast<uint4*>(cache + static_cast<size_t>(j.row - j.slot) * 576);
          const float ratio = was / scale;
          for (int x = me; x < j.slot * 36; x += threads) {
            const uint4 c = old[x];
            old[x] = make_uint4(requantise4(c.x, ratio), requantise4(c.y, ratio), requantise4(c.z, ratio),
                                requantise4(c.w, ratio));
          }
        }
      }
    }
    sync();                      // every thread has read the old scale (and the maxima)
    if (me == 0) *sp = scale;
    const float inv = 1.0f / scale;   // exact for a power of two
#pragma unroll 1
    for (int r = part; r < j.rows; r += width) {
      if (j.rows > width)
        v = row_values(src + static_cast<size_t>(r) * 576, a.gamma, a.freqs + static_cast<size_t>(j.pos + r) * 64, a.eps);
      store_row(cache + static_cast<size_t>(j.row + r) * 576, v, inv);
    }
  }
}

__device__ __forceinline__ void rotate_queries(const CacheWriteQ8Args& a, WriteSmem& sh, int t) {
  constexpr int QU = 4;          // query pieces of a thread in flight
  const int tid = threadIdx.x;
  // Piece m of head h holds rope values 8m .. 8m+7 (pairs 4m .. 4m+3).
  uint16_t* qt = static_cast<uint16_t*>(a.q) + static_cast<size_t>(t) * a.H * 192 + 128 + 8 * (tid & 7);
  const int pieces = 8 * a.H;
  auto piece = [&](int i) { return reinterpret_cast<uint4*>(qt + static_cast<size_t>(i >> 3) * 192); };
  uint4 x[QU];
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < QU; ++k)
      if (i0 + k * kWriteThreads < pieces) x[k] = *piece(i0 + k * kWriteThreads);
  };
  load(tid);
  if (tid < 32) {
    const int b = last_offset(a.iro, a.B, static_cast<uint32_t>(t));
    if (tid == 0) sh.pos = token_position(a, t, b);
  }
  __syncthreads();
  const int pos = sh.pos;
  if (pos >= 0) {
    const float4* fr = reinterpret_cast<const float4*>(a.freqs + static_cast<size_t>(pos) * 64) + 2 * (tid & 7);
    const float4 fa = __ldg(fr), fb = __ldg(fr + 1);
    for (int i0 = tid;;) {
#pragma unroll
      for (int k = 0; k < QU; ++k) {
        if (i0 + k * kWriteThreads < pieces) {
          const float2 a0 = rotate2(bf16_lo(x[k].x), bf16_hi(x[k].x), fa.x, fa.y);
          const float2 a1 = rotate2(bf16_lo(x[k].y), bf16_hi(x[k].y), fa.z, fa.w);
          const float2 a2 = rotate2(bf16_lo(x[k].z), bf16_hi(x[k].z), fb.x, fb.y);
          const float2 a3 = rotate2(bf16_lo(x[k].w), bf16_hi(x[k].w), fb.z, fb.w);
          *piece(i0 + k * kWriteThreads) =
              make_uint4(pack_bf16(a0.x, a0.y), pack_bf16(a1.x, a1.y), pack_bf16(a2.x, a2.y), pack_bf16(a3.x, a3.y));
        }
      }
      i0 += QU * kWriteThreads;
      if (i0 >= pieces) break;
      load(i0);
    }
  }
  __syncthreads();               // the position is rewritten for the next token
}

__global__ void __launch_bounds__(kWriteThreads, 4) cache_write_q8_kernel(const CacheWriteQ8Args a) {
  __shared__ WriteSmem sh;
  pdl_enter();
  if (timed_out_before(a.status)) return;
  const int c = blockIdx.x;
  if (c < a.row_ctas) {
    write_rows(a, sh, c * a.chunk);
  } else {
    for (int t = c - a.row_ctas; t < a.T; t += gridDim.x - a.row_ctas) rotate_queries(a, sh, t);
  }
}

// ------------------------------------------------------------------ gather
// As the bf16 gather: each CTA owns 32 consecutive buffer rows, resolves their
// addresses, then moves them in pieces of 8 codes, which become 16 bytes of
// bf16 (code times scale in fp32, rounded once; exact for the powers of two that
// the write stores).  HBM-bound: 576 bytes read and 1152 written a row.  Pieces
// of 16 codes made a store instruction cover every other 16 bytes, half a
// sector at a time: 164 us for 524288 rows, against 137 (6.6 TB/s).
constexpr int kGatherRows = 32;
constexpr int kGatherThreads = 256;
constexpr int kPieces = 72;   // 8-byte pieces of a row

__device__ __forceinline__ uint2 dequant4(uint32_t c, float s) {
  const float2 a = f16x2_to_float2(e4m3x2_to_f16x2(static_cast<uint16_t>(c & 0xFFFFu)));
  const float2 b = f16x2_to_float2(e4m3x2_to_f16x2(static_cast<uint16_t>(c >> 16)));
  return make_uint2(pack_bf16(a.x * s, a.y * s), pack_bf16(b.x * s, b.y * s));
}

__global__ void __launch_bounds__(kGatherThreads) gather_q8_kernel(const GatherQ8Args a) {
  constexpr int kVecs = kGatherRows * kPieces;
  constexpr int kPer = kVecs / kGatherThreads;
  static_assert(kVecs % kGatherThreads == 0, "every thread has as many pieces");
  __shared__ long long s_src[kGatherRows];   // cache row, or -1
  __shared__ float s_scale[kGatherRows];
  pdl_enter();
  if (timed_out_before(a.status)) return;
  const int n = min(a.bl[a.chunk], static_cast<int>(a.S));
  const int r0 = blockIdx.x * kGatherRows;
  if (r0 >= n) return;
  const uint32_t* bro = a.bro + static_cast<size_t>(a.chunk) * (a.B + 1);
  const uint32_t* co = a.co + static_cast<size_t>(a.chunk) * a.B;
  if (threadIdx.x < kGatherRows) {
    const int r = r0 + threadIdx.x;
    long long src = -1;
    if (r < n) {
      int lo = 0, hi = a.B;   // bro[lo] <= r < bro[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (bro[mid] <= static_cast<uint32_t>(r)) lo = mid; else hi = mid;
      }
      const uint32_t pos = co[lo] + (static_cast<uint32_t>(r) - bro[lo]);
      const uint32_t pidx = pos / static_cast<uint32_t>(a.page_size);
      const int page = pidx < static_cast<uint32_t>(a.max_pages)
                           ? a.page_table[static_cast<size_t>(lo) * a.max_pages + pidx] : -1;
      if (page >= 0 && page < a.num_pages) {
        src = static_cast<long long>(page) * a.page_size + pos % a.page_size;
        s_scale[threadIdx.x] = __ldg(a.kv_scales + src / a.scale_block);
      } else {
        set_status(a.status, MLA_DEV_BAD_PAGE);
      }
    }
    s_src[threadIdx.x] = src;
  }
  __syncthreads();
  uint2 v[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int idx = threadIdx.x + k * kGatherThreads;
    const int row = idx / kPieces, col = idx - row * kPieces;
    const long long src = s_src[row];
    if (src >= 0)
      v[k] = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.kv_cache) + src * 576) + col);
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int idx = threadIdx.x + k * kGatherThreads;
    const int row = idx / kPieces, col = idx - row * kPieces;
    if (s_src[row] < 0) continue;
    const float s = s_scale[row];
    const uint2 p0 = dequant4(v[k].x, s), p1 = dequant4(v[k].y, s);
    const size_t r = static_cast<size_t>(r0 + row);
    uint4* dst = col < 64 ? reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.c_kv_buf) + r * 512) + col
                          : reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.k_rope_buf) + r * 64) + (col - 64);
    *dst = make_uint4(p0.x, p0.y, p1.x, p1.y);
  }
}

}  // namespace

cudaError_t launch_cache_write_q8(const CacheWriteQ8Args& args, cudaStream_t stream) {
  if (args.T <= 0) return cudaSuccess;
  CacheWriteQ8Args a = args;
  // Tokens of a row CTA: a block's, in whole warps, or eight small blocks.
  a.chunk = a.scale_block > 8 ? (a.scale_block + 31) / 32 * 32 : 8;
  a.group_warps = 1;
  while (a.group_warps < kWriteWarps && 2 * a.group_warps <= a.scale_block) a.group_warps *= 2;
  a.row_ctas = (a.T + a.chunk - 1) / a.chunk;
  const int rotating = a.q == nullptr ? 0 : (a.T < 16 * sm_count() ? a.T : 16 * sm_count());
  return launch_pdl(cache_write_q8_kernel, dim3(a.row_ctas + rotating), dim3(kWriteThreads), 0, stream, a);
}

cudaError_t launch_gather_q8(const GatherQ8Args& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((static_cast<uint64_t>(a.S) + kGatherRows - 1) / kGatherRows);
  return launch_pdl(gather_q8_kernel, dim3(grid), dim3(kGatherThreads), 0, stream, a);
}

}  // namespace mla
