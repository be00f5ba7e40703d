// Host-side interfaces of the paged-cache entry points (gqa_paged.h).
#pragma once

#include "gqa_paged.h"
#include "internal.h"

namespace gqa {

// What every kernel over the paged cache needs to find its rows.
struct PagedView {
  const int32_t* table;    // [B, max_pages]
  const int32_t* cu;       // [B + 1], nullptr: no new tokens (eviction)
  const int32_t* seqlens;  // [B]
  int* err;                // device error word
  int B, T, max_new, total;
  int page_log2, num_pages, max_pages;
};

// One validated call.
struct PagedArgs {
  PagedView v;
  int H, Hkv, D, page, dtype;
  int window;   // 0: none
  float scale;  // resolved (> 0)
  const void* q;
  const void* k_pages;
  const void* v_pages;
  void* out;
  float* lse;
  cudaStream_t stream;
  int num_sms;
};

struct AppendArgs {
  PagedView v;
  int H, Hkv, D, page, dtype;
  const void* q;
  const void* k;
  const void* value;
  int q_stride, kv_stride;  // elements between consecutive tokens' rows
  const void* qw;           // norm weights, nullptr: no norm
  const void* kw;
  float eps;
  const void* cos;  // nullptr: no rotation
  const void* sin;
  const int32_t* positions;  // nullptr: slots
  int cos_rows, interleaved;
  void* k_pages;
  void* v_pages;
  void* q_out;
  cudaStream_t stream;
};

struct EvictArgs {
  PagedView v;
  int Hkv, D, page, dtype;
  void* k_pages;
  void* v_pages;
  float* weights;
  const int32_t* dst;  // == v.table in place
  int dst_max_pages;
  int in_place;
  int budget, recent;
  int32_t* kept;
  int32_t* new_seqlens;
  cudaStream_t stream;
  int num_sms;
};

// Which attention kernel runs and how the workspace is carved up: a function
// of the dims and total_sequence_length, total_bytes of the dims alone.
enum class PagedPath { kDecode, kPrefill, kGeneric };
struct PagedPlan {
  PagedPath path = PagedPath::kGeneric;
  int ctas = 0;      // persistent grid
  int columns = 0;   // decode: (token, head) columns of a partial
  int slots = 0;     // partial slots
  size_t sched_off = 0, part_o_off = 0, part_ml_off = 0;
  size_t total_bytes = 0;
};
PagedPlan make_paged_plan(const gqa_paged_dims_t& d, int total, int num_sms);

// Split-KV attention of few new rows (max_new * G <= kPagedDecodeColumns)
// with head size 64 or 128.
constexpr int kPagedDecodeColumns = 32;
int paged_decode_ctas_per_sm(int columns, int head_size, int smem_per_sm);
cudaError_t launch_paged_decode(const PagedArgs& a, const PagedPlan& plan, uint8_t* workspace, uint32_t epoch);

// tcgen05 attention of chunks (more rows than that, or many of them over much
// work, see make_paged_plan) with head size 64 or 128, G <= 128.
cudaError_t launch_paged_prefill(const PagedArgs& a, const PagedPlan& plan, uint8_t* workspace, uint32_t epoch);

cudaError_t launch_paged_append(const AppendArgs& a);
// Any head size, on CUDA cores.
cudaError_t launch_paged_generic(const PagedArgs& a);
cudaError_t launch_paged_weights_generic(const PagedArgs& a, const float* w_in, float* w_out);
// Tensor-core key weights (head size 64 or 128, G <= 128).
bool paged_weights_tensor(const PagedArgs& a);
cudaError_t launch_paged_weights(const PagedArgs& a, const float* w_in, float* w_out);
cudaError_t launch_paged_evict(const EvictArgs& a);

}  // namespace gqa
