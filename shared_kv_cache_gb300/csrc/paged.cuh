// Device helpers shared by the kernels over the paged cache.
#pragma once

#include "common.cuh"
#include "paged_internal.h"

namespace gqa {
namespace paged {

// Sequence b of a call: its rows q0 .. q0 + n - 1 of the token arrays, its
// `past` cached tokens and its length L with the new ones.
struct Seq {
  int q0, n, past, L;
};

// Checks a sequence from its list entries.  False: it is skipped (it has no
// new tokens, or `code` is the error it raises).
__device__ __forceinline__ bool check_seq(const PagedView& v, int past, int q0, int q1, Seq& s, int& code) {
  s.past = past;
  s.q0 = q0;
  code = 0;
  // (compared before subtracting: q1 - q0 may not fit 32 bits)
  if (past < 0 || q0 < 0 || q1 < q0 || q1 > v.T || q1 - q0 > v.max_new) {
    code = GQA_ERR_INVALID_ARGUMENT;
    s.n = s.L = 0;
    return false;
  }
  s.n = q1 - q0;
  const long long L = (long long)past + s.n;
  if (L > ((long long)v.max_pages << v.page_log2)) code = GQA_ERR_KV_OVERFLOW;
  else if (L > v.total) code = GQA_ERR_INVALID_ARGUMENT;
  s.L = code ? 0 : (int)L;
  return !code && (s.n > 0 || !v.cu);
}
// Reads and checks sequence b.
__device__ __forceinline__ bool load_seq(const PagedView& v, int b, Seq& s, int& code) {
  return check_seq(v, v.seqlens[b], v.cu ? v.cu[b] : 0, v.cu ? v.cu[b + 1] : 0, s, code);
}

// First slot that new token `slot` (its own slot) sees.
__host__ __device__ __forceinline__ int first_visible(int slot, int window) {
  return window > 0 && slot >= window ? slot - window + 1 : 0;
}

// Page of slot `s`: -1 for an entry outside the pool (recorded).
__device__ __forceinline__ int page_of(const PagedView& v, const int32_t* row, int s) {
  const int pg = row[s >> v.page_log2];
  if ((unsigned)pg >= (unsigned)v.num_pages) {
    record_error(v.err, GQA_ERR_INVALID_ARGUMENT);
    return -1;
  }
  return pg;
}

// Row index of slot s on page pg for KV head kh, in a pool [pages, Hkv, page].
__device__ __forceinline__ size_t pool_row(const PagedView& v, int Hkv, int pg, int kh, int s) {
  return (((size_t)pg * Hkv + kh) << v.page_log2) + (s & ((1 << v.page_log2) - 1));
}

}  // namespace paged
}  // namespace gqa
