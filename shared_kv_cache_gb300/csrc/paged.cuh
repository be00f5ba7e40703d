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

// Bit 15 (31) of the result: the low (high) 16-bit value of w is infinite or
// NaN (its exponent's ones carry into the sign's place).
template <typename T>
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) {
  constexpr uint32_t kExp = Elem<T>::is_bf16 ? 0x7F80u : 0x7C00u, kOne = Elem<T>::is_bf16 ? 0x0080u : 0x0400u;
  return ((w & (kExp * 0x10001u)) + kOne * 0x10001u) & 0x80008000u;
}
template <typename T>
__device__ __forceinline__ bool nonfinite(const uint4& v) {
  return (nonfinite2<T>(v.x) | nonfinite2<T>(v.y) | nonfinite2<T>(v.z) | nonfinite2<T>(v.w)) != 0;
}
// w with its infinite and NaN values replaced by zeros.
template <typename T>
__device__ __forceinline__ uint32_t finite_only2(uint32_t w) {
  const uint32_t b = nonfinite2<T>(w);
  return w & ~((b & 0x8000u ? 0xFFFFu : 0u) | (b & 0x80000000u ? 0xFFFF0000u : 0u));
}
template <typename T>
__device__ __forceinline__ uint4 finite_only(const uint4& v) {
  return make_uint4(finite_only2<T>(v.x), finite_only2<T>(v.y), finite_only2<T>(v.z), finite_only2<T>(v.w));
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this CTA's shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t at_rank(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void store_at(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ long long warp_sum_ll(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---------------------------------------------------------------------------
// Loads of 128-key tiles of the tensor-core kernels.  A tile is held as its
// 64-dimension halves, kBox bytes apart, 128 rows of 128 bytes each with the
// 128-byte swizzle.  A tile of a paged cache takes one bulk-tensor box per
// page and half (or per 128 rows of a larger page); the block-table entries of
// coming tiles are kept in registers, 32 at a time, one batch ahead.  Boxes
// without a slot in [lo, L) are aimed beyond the pool, which reads as zeros.
// ---------------------------------------------------------------------------
constexpr int kBN = 128;         // keys per tile
constexpr int kBox = kBN * 128;  // one half of a tile: 16 KB

struct TileLoader {
  const PagedView* v;
  const int32_t* tab;
  int Hkv, pool_rows, kh, lo, L;
  int plog, rows, nsub, e0, e_end, cur, nxt;

  __device__ __forceinline__ int entry(int e) const { return e <= e_end ? __ldg(tab + e) : -1; }
  // (whole warp) tiles [t0, t0 + n) of sequence b and KV head kh, in order
  __device__ __forceinline__ void begin(const PagedView& view, int Hkv_, int pool_rows_, int b, int kh_, int lo_, int L_,
                                        int t0, int n, int lane) {
    v = &view;
    Hkv = Hkv_;
    pool_rows = pool_rows_;
    kh = kh_;
    lo = lo_;
    L = L_;
    plog = view.page_log2;
    rows = min(1 << plog, kBN);
    nsub = kBN / rows;
    tab = view.table + (size_t)b * view.max_pages;
    e0 = (t0 * kBN) >> plog;
    e_end = (min((t0 + n) * kBN, L) - 1) >> plog;
    cur = entry(e0 + lane);
    nxt = entry(e0 + 32 + lane);
  }
  // (whole warp) tile t's halves [h0, h1) to `dst`, completing on `bar`
  __device__ __forceinline__ void issue(const CUtensorMap* map, int t, uint32_t dst, int h0, int h1, uint32_t bar,
                                        int lane) {
    const int s = t * kBN + min(lane, nsub - 1) * rows;  // first slot of the lane's box
    const int e = s >> plog;
    if (__shfl_sync(0xffffffffu, e, 0) >= e0 + 32) {
      cur = nxt;
      e0 += 32;
      nxt = entry(e0 + 32 + lane);
    }
    const int pg = __shfl_sync(0xffffffffu, cur, e - e0);
    int y = pool_rows;
    if (lane < nsub && s < L && s + rows > lo) {
      if ((unsigned)pg < (unsigned)v->num_pages)
        y = ((pg * Hkv + kh) << plog) + (s & ((1 << plog) - 1));
      else
        record_error(v->err, GQA_ERR_INVALID_ARGUMENT);
    }
    if (lane < nsub)
      for (int h = h0; h < h1; ++h) tma_load_2d(dst + h * kBox + lane * rows * 128, map, h * 64, y, bar);
  }
};

}  // namespace paged
}  // namespace gqa
