// The paged-cache entry points: argument checks, the choice of kernel, launch.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "paged_internal.h"

namespace gqa {
namespace {

bool misaligned(const void* p, uintptr_t a = 16) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

constexpr int kMaxLength = 1 << 30;  // of a sequence: slot numbers rounded up to tiles stay within 32 bits

int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

// The dims alone.  `evict`: only the fields that describe the cache.
gqa_status_t check_paged_dims(const gqa_paged_dims_t* d, bool evict) {
  if (!d) return GQA_ERR_INVALID_ARGUMENT;
  if (d->batch < 1 || d->kv_num_heads < 1 || d->num_pages < 1 || d->max_pages < 1) return GQA_ERR_INVALID_ARGUMENT;
  if (d->head_size < 8 || d->head_size > 256 || d->head_size % 8 != 0) return GQA_ERR_INVALID_ARGUMENT;
  if (d->page_size < 8 || d->page_size > 1024 || (d->page_size & (d->page_size - 1))) return GQA_ERR_INVALID_ARGUMENT;
  if (d->dtype != GQA_DTYPE_FP16 && d->dtype != GQA_DTYPE_BF16) return GQA_ERR_INVALID_ARGUMENT;
  if (!evict) {
    if (d->total_tokens < 1 || d->max_new_tokens < 1 || d->num_heads < 1) return GQA_ERR_INVALID_ARGUMENT;
    if (d->num_heads % d->kv_num_heads != 0) return GQA_ERR_INVALID_ARGUMENT;
    if (d->rotary_interleaved != 0 && d->rotary_interleaved != 1) return GQA_ERR_INVALID_ARGUMENT;
    if ((long long)d->total_tokens * d->num_heads >= (1ll << 31)) return GQA_ERR_UNSUPPORTED;
    // a packed row's length in elements
    if (((long long)d->num_heads + 2ll * d->kv_num_heads) * d->head_size >= (1ll << 31)) return GQA_ERR_UNSUPPORTED;
  }
  // row indices of the pool (tensor-map coordinates) and grid dimensions
  if ((long long)d->num_pages * d->kv_num_heads * d->page_size >= (1ll << 31)) return GQA_ERR_UNSUPPORTED;
  if (d->batch > 65535 || d->kv_num_heads > 65535) return GQA_ERR_UNSUPPORTED;
  return GQA_OK;
}

PagedView view_of(const gqa_paged_dims_t* d, const int32_t* table, const int32_t* cu, const int32_t* seqlens,
                  int total, int* err) {
  return PagedView{table, cu, seqlens, err, d->batch, d->total_tokens, d->max_new_tokens, total,
                   log2_of(d->page_size), d->num_pages, d->max_pages};
}

// The checks that gqa_paged_attention and gqa_paged_key_weights share, and
// the resolved call.
gqa_status_t resolve(const gqa_paged_dims_t* d, const void* query, const void* k_pages, const int32_t* table,
                     const int32_t* cu, const int32_t* seqlens, int total, float scale, int window, void* stream,
                     PagedArgs& a) {
  const gqa_status_t st = check_paged_dims(d, false);
  if (st != GQA_OK) return st;
  if (!query || !k_pages || !table || !cu || !seqlens) return GQA_ERR_INVALID_ARGUMENT;
  if (misaligned(query) || misaligned(k_pages) || misaligned(table, 4) || misaligned(cu, 4) || misaligned(seqlens, 4))
    return GQA_ERR_INVALID_ARGUMENT;
  if (total < 1 || !std::isfinite(scale)) return GQA_ERR_INVALID_ARGUMENT;
  if (total > kMaxLength) return GQA_ERR_UNSUPPORTED;
  if (total > (long long)d->max_pages * d->page_size) return GQA_ERR_KV_OVERFLOW;
  a.v = view_of(d, table, cu, seqlens, total, nullptr);
  a.H = d->num_heads;
  a.Hkv = d->kv_num_heads;
  a.D = d->head_size;
  a.page = d->page_size;
  a.dtype = d->dtype;
  a.window = window > 0 ? window : 0;
  a.scale = scale > 0.f ? scale : 1.0f / std::sqrt((float)a.D);
  a.q = query;
  a.k_pages = k_pages;
  a.stream = static_cast<cudaStream_t>(stream);
  return GQA_OK;
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

PagedPlan chunk_plan(const gqa_paged_dims_t& d, int num_sms) {
  // at most two cut items a CTA, each with two tiles of 128 rows
  PagedPlan pl;
  pl.path = PagedPath::kPrefill;
  pl.ctas = num_sms;
  pl.slots = 2 * num_sms;
  pl.part_o_off = align_up(((size_t)num_sms * 2 + 1) * sizeof(unsigned long long), 256);
  pl.part_ml_off = align_up(pl.part_o_off + (size_t)pl.slots * 256 * d.head_size * sizeof(float), 256);
  pl.total_bytes = align_up(pl.part_ml_off + (size_t)pl.slots * 256 * 2 * sizeof(float), 256);
  return pl;
}

}  // namespace

PagedPlan make_paged_plan(const gqa_paged_dims_t& d, int total, int num_sms) {
  PagedPlan pl;
  const int G = d.num_heads / d.kv_num_heads;
  if ((d.head_size != 64 && d.head_size != 128) || G > 128) return pl;
  const long long rows = (long long)d.max_new_tokens * G;
  if (rows <= kPagedDecodeColumns) {
    pl.path = PagedPath::kDecode;
    pl.columns = (int)rows;
    pl.ctas = num_sms * paged_decode_ctas_per_sm(pl.columns, d.head_size, device_smem_per_sm());
    // (items cut into several chunks hold fewer partials than this: see make_plan)
    pl.slots = 2 * kDecodeChunksPerCta * pl.ctas;
    pl.sched_off = 0;
    pl.part_o_off = align_up((size_t)(1 + pl.slots) * sizeof(unsigned long long), 256);
    pl.part_ml_off = align_up(pl.part_o_off + (size_t)pl.slots * pl.columns * d.head_size * sizeof(float), 256);
    pl.total_bytes = align_up(pl.part_ml_off + (size_t)pl.slots * pl.columns * 2 * sizeof(float), 256);
    // With many columns of head size 128 the few-row kernel's mma.sync takes
    // longer than its stream, and the chunk kernel, whose start and merges cost
    // more but whose products do not depend on the columns, is faster where the
    // call is long enough to make up for them.  Key tiles a CTA (16-bit,
    // 32 on 8 heads, us few-row / chunk): 32 columns 3.4 tiles 42 / 46, 6.7 tiles
    // 52 / 44, 27 tiles 101 / 74; 24 columns 6.7 tiles 38 / 44, 13 tiles 56 / 54,
    // 27 tiles 87 / 74; 16 columns 27 tiles 72 / 74.  With head size 64 the few-row
    // kernel stays ahead (79 tiles, 32 columns 117 / 128).
    if (d.head_size != 128 || rows <= 16) return pl;
    const long long tiles = (long long)d.batch * d.kv_num_heads * (((long long)total + 127) / 128);
    const size_t few_rows_bytes = pl.total_bytes;
    const bool chunk = tiles >= (rows > 24 ? 5ll : 16ll) * num_sms;
    PagedPlan pc = chunk_plan(d, num_sms);
    if (chunk) pl = pc;
    pl.total_bytes = std::max(few_rows_bytes, pc.total_bytes);  // the same for every length
    return pl;
  }
  return chunk_plan(d, num_sms);
}

}  // namespace gqa

using namespace gqa;

extern "C" {

size_t gqa_paged_workspace_size(const gqa_paged_dims_t* dims, int32_t total_sequence_length,
                                int32_t local_window_size) {
  if (check_paged_dims(dims, false) != GQA_OK || total_sequence_length < 1) return 0;
  (void)local_window_size;
  return make_paged_plan(*dims, total_sequence_length, device_sm_count()).total_bytes;
}

gqa_status_t gqa_paged_append(const gqa_paged_dims_t* dims, const void* query, const void* key, const void* value,
                              const void* q_norm_weight, const void* k_norm_weight, float norm_eps,
                              const void* cos_cache, const void* sin_cache, const int32_t* positions, void* k_pages,
                              void* v_pages, const int32_t* block_table, const int32_t* cu_seqlens,
                              const int32_t* seqlens_k, int32_t total_sequence_length, void* query_out,
                              void* stream) {
  gqa_paged_dims_t d0;
  if (dims) {
    d0 = *dims;
    d0.max_new_tokens = INT32_MAX;  // not a limit here
  }
  const gqa_status_t st = check_paged_dims(dims ? &d0 : nullptr, false);
  if (st != GQA_OK) return st;
  const gqa_paged_dims_t* d = &d0;
  const bool packed = !key && !value;
  if (packed && query_out == query) return GQA_ERR_INVALID_ARGUMENT;
  if (packed && query) {
    key = static_cast<const uint8_t*>(query) + (size_t)d->num_heads * d->head_size * 2;
    value = static_cast<const uint8_t*>(key) + (size_t)d->kv_num_heads * d->head_size * 2;
  }
  if (!query || !key || !value || !k_pages || !v_pages || !block_table || !cu_seqlens || !seqlens_k || !query_out)
    return GQA_ERR_INVALID_ARGUMENT;
  if (k_pages == v_pages) return GQA_ERR_INVALID_ARGUMENT;
  if (misaligned(query) || misaligned(key) || misaligned(value) || misaligned(k_pages) || misaligned(v_pages) ||
      misaligned(query_out) || misaligned(q_norm_weight) || misaligned(k_norm_weight) || misaligned(cos_cache) ||
      misaligned(sin_cache) || misaligned(positions, 4) || misaligned(block_table, 4) || misaligned(cu_seqlens, 4) ||
      misaligned(seqlens_k, 4))
    return GQA_ERR_INVALID_ARGUMENT;
  if ((cos_cache == nullptr) != (sin_cache == nullptr)) return GQA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(norm_eps) || norm_eps < 0.f) return GQA_ERR_INVALID_ARGUMENT;
  if (total_sequence_length < 1) return GQA_ERR_INVALID_ARGUMENT;
  if (total_sequence_length > kMaxLength) return GQA_ERR_UNSUPPORTED;
  if (total_sequence_length > (long long)d->max_pages * d->page_size) return GQA_ERR_KV_OVERFLOW;
  if (cos_cache && (d->cos_cache_rows < 1 || (!positions && d->cos_cache_rows < total_sequence_length)))
    return GQA_ERR_INVALID_ARGUMENT;
  int* err = device_error_word();
  if (!err) return GQA_ERR_CUDA;
  const int row = (packed ? d->num_heads + 2 * d->kv_num_heads : d->num_heads) * d->head_size;
  AppendArgs a{};
  a.v = view_of(d, block_table, cu_seqlens, seqlens_k, total_sequence_length, err);
  a.H = d->num_heads;
  a.Hkv = d->kv_num_heads;
  a.D = d->head_size;
  a.page = d->page_size;
  a.dtype = d->dtype;
  a.q = query;
  a.k = key;
  a.value = value;
  a.q_stride = row;
  a.kv_stride = packed ? row : d->kv_num_heads * d->head_size;
  a.qw = q_norm_weight;
  a.kw = k_norm_weight;
  a.eps = norm_eps;
  a.cos = cos_cache;
  a.sin = sin_cache;
  a.positions = positions;
  a.cos_rows = d->cos_cache_rows;
  a.interleaved = d->rotary_interleaved;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.q_out = query_out;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_paged_append(a) == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

gqa_status_t gqa_paged_attention(const gqa_paged_dims_t* dims, const void* query, const void* k_pages,
                                 const void* v_pages, const int32_t* block_table, const int32_t* cu_seqlens,
                                 const int32_t* seqlens_k, int32_t total_sequence_length, float scale,
                                 int32_t local_window_size, void* output, float* lse, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  PagedArgs a{};
  const gqa_status_t st = resolve(dims, query, k_pages, block_table, cu_seqlens, seqlens_k, total_sequence_length,
                                  scale, local_window_size, stream, a);
  if (st != GQA_OK) return st;
  if (!v_pages || !output || misaligned(v_pages) || misaligned(output) || misaligned(lse, 4) || v_pages == k_pages)
    return GQA_ERR_INVALID_ARGUMENT;
  if (output == query) return GQA_ERR_INVALID_ARGUMENT;  // other rows' queries are still to be read
  a.num_sms = device_sm_count();
  const PagedPlan pl = make_paged_plan(*dims, total_sequence_length, a.num_sms);
  if (workspace_bytes < pl.total_bytes || (pl.total_bytes > 0 && (!workspace || misaligned(workspace))))
    return GQA_ERR_INVALID_ARGUMENT;
  a.v.err = device_error_word();
  if (!a.v.err) return GQA_ERR_CUDA;
  a.v_pages = v_pages;
  a.out = output;
  a.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const cudaError_t e = pl.path == PagedPath::kDecode    ? launch_paged_decode(a, pl, ws, next_epoch())
                        : pl.path == PagedPath::kPrefill ? launch_paged_prefill(a, pl, ws, next_epoch())
                                                         : launch_paged_generic(a);
  return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

gqa_status_t gqa_paged_key_weights(const gqa_paged_dims_t* dims, const void* query, const float* lse,
                                   const void* k_pages, const int32_t* block_table, const int32_t* cu_seqlens,
                                   const int32_t* seqlens_k, int32_t total_sequence_length, float scale,
                                   int32_t local_window_size, const float* weights_in, float* weights,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  PagedArgs a{};
  const gqa_status_t st = resolve(dims, query, k_pages, block_table, cu_seqlens, seqlens_k, total_sequence_length,
                                  scale, local_window_size, stream, a);
  if (st != GQA_OK) return st;
  if (!lse || !weights_in || !weights || misaligned(lse, 4) || misaligned(weights_in) || misaligned(weights))
    return GQA_ERR_INVALID_ARGUMENT;
  (void)workspace;
  (void)workspace_bytes;
  a.v.err = device_error_word();
  if (!a.v.err) return GQA_ERR_CUDA;
  a.lse = const_cast<float*>(lse);
  a.num_sms = device_sm_count();
  const cudaError_t e = paged_weights_tensor(a) ? launch_paged_weights(a, weights_in, weights)
                                                : launch_paged_weights_generic(a, weights_in, weights);
  return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

gqa_status_t gqa_paged_evict(const gqa_paged_dims_t* dims, void* k_pages, void* v_pages, float* weights,
                             const int32_t* block_table, const int32_t* dst_block_table, int32_t dst_max_pages,
                             const int32_t* seqlens_k, int32_t total_sequence_length, int32_t budget,
                             int32_t recent, int32_t* kept, int32_t* new_seqlens, void* workspace,
                             size_t workspace_bytes, void* stream) {
  (void)workspace;
  (void)workspace_bytes;
  const gqa_status_t st = check_paged_dims(dims, true);
  if (st != GQA_OK) return st;
  if (!k_pages || !v_pages || !weights || !block_table || !seqlens_k || !kept) return GQA_ERR_INVALID_ARGUMENT;
  if (misaligned(k_pages) || misaligned(v_pages) || misaligned(weights) || misaligned(block_table, 4) ||
      misaligned(dst_block_table, 4) || misaligned(seqlens_k, 4) || misaligned(kept, 4) || misaligned(new_seqlens, 4))
    return GQA_ERR_INVALID_ARGUMENT;
  if (k_pages == v_pages || new_seqlens == seqlens_k) return GQA_ERR_INVALID_ARGUMENT;
  if (budget < 1 || recent < 0 || recent > budget || total_sequence_length < 1) return GQA_ERR_INVALID_ARGUMENT;
  if (dst_block_table && dst_max_pages < 1) return GQA_ERR_INVALID_ARGUMENT;
  if (total_sequence_length > kMaxLength) return GQA_ERR_UNSUPPORTED;
  if (total_sequence_length > (long long)dims->max_pages * dims->page_size) return GQA_ERR_KV_OVERFLOW;
  EvictArgs a{};
  a.v = view_of(dims, block_table, nullptr, seqlens_k, total_sequence_length, device_error_word());
  if (!a.v.err) return GQA_ERR_CUDA;
  a.v.T = 0;
  a.v.max_new = 0;
  a.Hkv = dims->kv_num_heads;
  a.D = dims->head_size;
  a.page = dims->page_size;
  a.dtype = dims->dtype;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.weights = weights;
  // the source's own table as the destination is the in-place form too
  a.in_place = !dst_block_table || dst_block_table == block_table;
  a.dst = a.in_place ? block_table : dst_block_table;
  a.dst_max_pages = a.in_place ? dims->max_pages : dst_max_pages;
  a.budget = budget;
  a.recent = recent;
  a.kept = kept;
  a.new_seqlens = new_seqlens;
  a.stream = static_cast<cudaStream_t>(stream);
  a.num_sms = device_sm_count();
  return launch_paged_evict(a) == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // extern "C"
