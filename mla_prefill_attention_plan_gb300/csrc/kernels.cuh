// Internal launchers of the sm_103a kernels (host side).  The public C ABI in
// mla_prefill.h validates arguments and calls these.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sm100.cuh"

namespace mla {

// Launch with programmatic stream serialization: the kernel may begin while
// the previous kernel of the stream finishes; it calls pdl_enter() before it
// touches global memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

// n / d for 0 <= n < 2^31 by a multiplication: with l = ceil(log2 d) and
// m = ceil(2^(31 + l) / d), m d exceeds 2^(31 + l) by less than 2^l, so the
// product's error stays below 2^(31 + l) / d.
struct FastDiv {
  uint32_t m;
  int shift, d;
};
__device__ __forceinline__ int fast_div(int n, const FastDiv& f) {
  return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * f.m) >> f.shift);
}
inline FastDiv fast_divisor(int d) {
  int l = 0;
  while ((1ll << l) < d) ++l;
  FastDiv f;
  f.m = static_cast<uint32_t>(((1ull << (31 + l)) + d - 1) / d);
  f.shift = 31 + l;
  f.d = d;
  return f;
}

// Longest context of the 8-bit decode, the key scores and the selection: room
// for a few tiles past it in a 32-bit position.
constexpr int kMaxContext = 0x7FFFFFFF - 8191;

cudaError_t launch_plan(uint32_t* bro, uint32_t* co, int32_t* bl, const uint32_t* iro,
                        const uint32_t* cache_len, int B, int max_chunks, uint32_t S,
                        int32_t* status, cudaStream_t stream);

struct CacheWriteArgs {
  void* kv_cache;
  void* q;                  // bf16 [T][H][192] or null
  const void* kv_latent;    // bf16 [T][576]
  const float* gamma;       // [512]
  const float* freqs;       // [max_seq_len][64]
  const uint32_t* iro;
  const uint32_t* cache_len;
  const int32_t* page_table;
  int num_pages, page_size, max_pages, B, H, T, max_seq_len;
  float eps, inv_scale;
  int elt_bytes;            // cache storage: 2 (bf16) or 1 (e4m3)
  const uint32_t* rope_positions = nullptr;   // [T], or null: the context position
  int32_t* status;
};
cudaError_t launch_cache_write(const CacheWriteArgs& a, cudaStream_t stream);

cudaError_t launch_gather(void* c_kv_buf, void* k_rope_buf, const void* kv_cache,
                          const int32_t* page_table, int num_pages, int page_size, int max_pages,
                          const uint32_t* bro, const uint32_t* co, const int32_t* bl, int chunk,
                          int B, uint32_t S, int elt_bytes, int32_t* status, cudaStream_t stream);

// Per chunk, the cache row of every buffer row (gather.cu).
cudaError_t launch_cache_rows(int32_t* cache_rows, const int32_t* page_table, int num_pages,
                              int page_size, int max_pages, const uint32_t* bro, const uint32_t* co,
                              const int32_t* bl, int max_chunks, int B, uint32_t S, int32_t* status,
                              cudaStream_t stream);

struct UpprojArgs {
  void* k_nope;
  void* v;
  const void* c_kv;
  const void* w_k;
  const void* w_uv;
  const int32_t* buffer_lengths;
  int chunk;
  uint32_t S;
  int H;
  int dtype;
  float out_scale;
  int32_t* status;
  // A rows straight from the paged cache (kv_cache given): buffer row r of
  // the chunk is cache row cache_rows[r] (< num_cache_rows).
  const void* kv_cache = nullptr;
  const int32_t* cache_rows = nullptr;
  int num_cache_rows = 0;
};
// The GEMM on two-SM pairs (cta_group::2 clusters, 256 x 256 tiles); an
// error where the device cannot keep such a cluster resident.
cudaError_t launch_upproject(const UpprojArgs& a, cudaStream_t stream);

struct AttnArgs {
  void* out;
  float* lse;
  float* o_acc;
  float* lse_acc;
  const void* q;
  const void* k_nope;
  const void* v;
  const void* k_rope;           // [S][64] buffer, or null when k_rope comes from the paged cache
  const void* kv_cache = nullptr;      // paged cache rows [num_cache_rows][576] (k_rope = columns 512..575)
  const int32_t* cache_rows = nullptr;  // the chunk's cache row of each buffer row
  int num_cache_rows = 0;
  const uint32_t* iro;
  const uint32_t* cache_len;
  const uint32_t* bro;
  const uint32_t* co;
  const int32_t* bl;
  int chunk;
  int max_chunks;
  int B;
  int H;
  int max_prompt_len;
  int T_q;
  uint32_t S;
  float scale;  // softmax scale times the q and k descales
  float v_scale;
  int dtype;
  int32_t* status;
};
// bf16 attention on two-SM pairs (cta_group::2 clusters); e4m3 Q / K with V
// as f16 holding e4m3-rounded values (as mla_upproject writes it), on the
// same pairs.  An error where the device cannot keep such a cluster resident.
cudaError_t launch_attention(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attention_pair(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_attention_pair_e4m3(const AttnArgs& a, cudaStream_t stream);

// Absorbed MLA decode (decode.cu).
struct DecodeArgs {
  void* out;                  // [T][H][128] bf16
  float* lse;                 // [T][H] or null
  const void* q;              // [T][H][192] bf16
  const void* kv_cache;       // [num_pages][page_size][576] bf16
  const int32_t* page_table;  // [B][max_pages]
  int num_pages = 0, page_size = 0, max_pages = 0;
  const void* w_uk;           // [H][512][128] bf16
  const void* w_uv;           // [H][128][512] bf16
  const uint32_t* iro;
  const uint32_t* cache_len;
  int B, H, T, max_new, parts;
  int part_keys;              // > 0: about this many keys a partition, at most `parts` of them
  float scale;
  const int32_t* indices;     // sparse: [B][indices_stride] physical cache rows, or null
  int indices_stride;
  const int32_t* topk;        // sparse: [B] or null
  const float* sink;          // [B] or null
  void* workspace;
  int32_t* status;
};
struct DecodeLayout {
  size_t q_full, o_part, lse_part, o_lat, total;
};
DecodeLayout decode_layout(int T, int H, int parts);
// The library's partitioning: about part_keys keys a partition (at most
// `parts` of them), from the batch's sizes and its longest key list.
constexpr int kDecodeMaxParts = 64;
struct DecodePartitioning {
  int parts, part_keys;
};
DecodePartitioning decode_partitioning(int B, int H, int max_new, int max_keys);
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t stream);

// The decode's per-head projections (decode.cu), for other absorbed attentions:
// q_full [T*H][576] = (w_uk[h] q_nope, q_rope); out[t][h] = w_uv[h] o_lat[t][h]
// with o_lat [T*H][512], or (two_terms) the sum of [T*H][2][512].  Rows t with
// row_seq[t] < 0 are not written (row_seq may be null).  With plan given, the
// same launch finds chunk attention's schedule (chunk_plan.cuh).
namespace chunk {
struct ChunkPlanArgs;
}
cudaError_t launch_project_queries(const void* q, const void* w_uk, __nv_bfloat16* q_full, int T, int H,
                                   const chunk::ChunkPlanArgs* plan, int32_t* status, cudaStream_t stream);
cudaError_t launch_project_outputs(const __nv_bfloat16* o_lat, bool two_terms, const void* w_uv, void* out, int T,
                                   int H, const int32_t* row_seq, int32_t* status, cudaStream_t stream);

// Absorbed attention of chunks of new tokens over the paged cache (chunk_attn.cu).
struct ChunkAttnArgs {
  void* out;                  // [T][H][128] bf16
  float* lse;                 // [T][H] or null
  const void* q;              // [T][H][192] bf16
  const void* kv_cache;       // [num_pages][page_size][576] bf16
  const int32_t* page_table;  // [B][max_pages]
  int num_pages, page_size, max_pages;
  const void* w_uk;           // [H][512][128] bf16
  const void* w_uv;           // [H][128][512] bf16
  const uint32_t* iro;
  const uint32_t* cache_len;
  const uint32_t* mask;       // [T][mask_words] or null (causal)
  int mask_words;
  const float* sink;          // [B] or null
  int B, H, T;
  float scale;
  void* workspace;
  int32_t* status;
};
size_t chunk_attn_workspace(int B, int H, int T);
cudaError_t launch_chunk_attn(const ChunkAttnArgs& a, cudaStream_t stream);

// The 8-bit latent cache (cache_q8.cu): e4m3 rows, one power-of-two scale for
// each block of scale_block slots of a page (scale_block divides page_size,
// so cache row r has scale r / scale_block).
struct CacheWriteQ8Args {
  void* kv_cache;           // e4m3 [num_pages][page_size][576]
  float* kv_scales;         // [num_pages * page_size / scale_block]
  void* q;                  // bf16 [T][H][192] or null
  const void* kv_latent;    // bf16 [T][576]
  const float* gamma;       // [512]
  const float* freqs;       // [max_seq_len][64]
  const uint32_t* iro;
  const uint32_t* cache_len;
  const int32_t* page_table;
  int num_pages, page_size, max_pages, scale_block, B, H, T, max_seq_len;
  float eps;
  int32_t* status;
  // Set by the launch: CTAs that write rows, the tokens of one, warps that share a block.
  int row_ctas, chunk, group_warps;
};
cudaError_t launch_cache_write_q8(const CacheWriteQ8Args& a, cudaStream_t stream);

struct GatherQ8Args {
  void* c_kv_buf;           // bf16 [S][512]
  void* k_rope_buf;         // bf16 [S][64]
  const void* kv_cache;
  const float* kv_scales;
  const int32_t* page_table;
  int num_pages, page_size, max_pages, scale_block;
  const uint32_t* bro;
  const uint32_t* co;
  const int32_t* bl;
  int chunk, B;
  uint32_t S;
  int32_t* status;
};
cudaError_t launch_gather_q8(const GatherQ8Args& a, cudaStream_t stream);

// Absorbed MLA decode over the 8-bit cache (decode_q8.cu).
struct DecodeQ8Args {
  void* out;                  // [T][H][128] bf16
  float* lse;                 // [T][H] or null
  const void* q;              // [T][H][192] bf16
  const void* kv_cache;       // e4m3 [num_pages][page_size][576]
  const float* kv_scales;
  const int32_t* page_table;  // [B][max_pages], or null with indices
  int num_pages, page_size, max_pages, scale_block;
  const void* w_uk;           // [H][512][128] bf16
  const void* w_uv;           // [H][128][512] bf16
  const uint32_t* iro;
  const uint32_t* cache_len;
  int B, H, T, max_new, max_seq;
  int pieces;                 // equal parts that the batch's key tiles are cut into
  float scale;
  const int32_t* indices;     // sparse: [B][indices_stride] physical cache rows, or null
  int indices_stride;
  const int32_t* topk;        // sparse: [B] or null
  const float* sink;          // [B] or null
  void* workspace;
  int32_t* status;
};
struct DecodeQ8Layout {
  size_t head, entries, q8, q_scale, o_part, meta, total;
};
DecodeQ8Layout decode_q8_layout(int T, int H, int pieces);
int decode_q8_pieces(int B, int H, int max_new, int max_keys);
cudaError_t launch_decode_q8(const DecodeQ8Args& a, cudaStream_t stream);

// Key scores and block selection for sparse decode (index.cu).
struct IndexScoresArgs {
  float* scores;              // [T][stride]
  const void* iq;             // [T][Hi][128]
  const float* w;             // [T][Hi]
  const void* keys;           // [num_pages][page_size][128]
  const float* key_scales;    // [num_pages * page_size] or null
  const uint32_t* iro;
  const uint32_t* cache_len;
  const int32_t* page_table;
  int num_pages, page_size, max_pages, block, B, Hi, T, max_new, max_seq, stride;
  int dtype;
  int32_t* status;
};
cudaError_t launch_index_scores(const IndexScoresArgs& a, cudaStream_t stream);

struct IndexSelectArgs {
  int32_t* rows;              // [T][rows_stride]
  int32_t* count;             // [T]
  const float* scores;        // [T][stride]
  const uint32_t* iro;
  const uint32_t* cache_len;
  const int32_t* page_table;
  int num_pages, page_size, max_pages, block, top, local, B, T, max_seq, stride, rows_stride;
  int32_t* status;
};
cudaError_t launch_index_select(const IndexSelectArgs& a, cudaStream_t stream);

// Bookkeeping of the paged cache (pages.cu).
struct PagesForkArgs {
  int32_t* dst_table;         // [dst_batch][max_pages]
  uint32_t* dst_lengths;
  const int32_t* src_table;   // [src_batch][max_pages]
  const uint32_t* src_lengths;
  int32_t* refs;              // [num_pages]
  const int32_t* parents;     // [dst_batch], -1 for none
  int num_pages, max_pages, dst_batch, src_batch;
  int32_t* status;
};
cudaError_t launch_pages_fork(const PagesForkArgs& a, cudaStream_t stream);

struct PagesFreeArgs {
  int32_t* table;
  int32_t* refs;
  uint32_t* lengths;
  const uint32_t* keep;       // [batch] or null (nothing is kept)
  int num_pages, page_size, max_pages, batch;
  int32_t* status;
};
cudaError_t launch_pages_free(const PagesFreeArgs& a, cudaStream_t stream);

struct PagesReserveArgs {
  int32_t* table;
  int32_t* refs;
  const uint32_t* lengths;
  const uint32_t* fresh;      // [batch] tokens to come
  int32_t* copy_src;          // [batch]
  int32_t* copy_dst;
  int32_t* copy_count;
  int num_pages, page_size, max_pages, batch;
  // Scratch: of each page its count before the call, its writers and the last
  // of them; the free pages in order; of each sequence (pages, copies).
  int32_t *before, *writers, *last, *free_list;
  int2* want;
  int32_t* status;
};
cudaError_t launch_pages_reserve(const PagesReserveArgs& a, cudaStream_t stream);

struct PagesCompactArgs {
  int32_t* table;
  int32_t* refs;
  int32_t* copy_src;          // [max_copies]
  int32_t* copy_dst;
  int32_t* copy_count;
  int max_copies, num_pages, max_pages, batch;
  int32_t* moved;             // scratch [num_pages]: the page's move
  int32_t* status;
};
cudaError_t launch_pages_compact(const PagesCompactArgs& a, cudaStream_t stream);

struct PagesCopyArgs {
  char* cache;                // [layers] of [num_pages][page_bytes], layer_stride bytes apart
  size_t page_bytes, layer_stride;
  int layers;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* count;
  int max_copies, num_pages;
  int32_t* status;
};
cudaError_t launch_pages_copy(const PagesCopyArgs& a, cudaStream_t stream);

struct KeepRowsArgs {
  char* cache;                // [layers] of [num_pages * page_size][row_bytes]
  size_t row_bytes, layer_stride;
  int layers;
  const uint32_t* lengths;
  const int32_t* keep;        // [batch][keep_stride]
  int keep_stride;
  const int32_t* counts;
  const int32_t* table;
  int num_pages, page_size, max_pages, batch;
  int32_t* status;
};
cudaError_t launch_keep_rows(const KeepRowsArgs& a, cudaStream_t stream);

// Self-test of the bounded waits (selftest.cu): one cluster of `cluster`
// CTAs waiting on barriers nothing arrives at.
cudaError_t launch_bounded_wait_selftest(int32_t* status, long long* elapsed_ns, uint64_t limit_ns,
                                         int cluster, cudaStream_t stream);

// Tensor-map encoder and device properties (abi.cu).
bool encode_2d(CUtensorMap* map, const void* base, CUtensorMapDataType dt, uint64_t inner,
               uint64_t outer, uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer,
               CUtensorMapSwizzle swizzle);
// Three and four dimensions, strides (bytes) of all but the innermost.
bool encode_3d(CUtensorMap* map, const void* base, CUtensorMapDataType dt, const uint64_t (&dims)[3],
               const uint64_t (&strides)[2], const uint32_t (&box)[3], CUtensorMapSwizzle swizzle);
bool encode_4d(CUtensorMap* map, const void* base, CUtensorMapDataType dt, const uint64_t (&dims)[4],
               const uint64_t (&strides)[3], const uint32_t (&box)[4], CUtensorMapSwizzle swizzle);
int sm_count();

}  // namespace mla
