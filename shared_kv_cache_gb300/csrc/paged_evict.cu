// Eviction from a paged cache by accumulated attention weight.
//
// Of the n > budget tokens of a (sequence, KV head), the `recent` last stay
// and, of the n - recent others, the budget - recent of the largest weights
// (equal weights: the lower slot).
//
// evict_select_kernel finds them by radix selection: the weights map to
// unsigned integers of the same order (NaN below all), and from the top digit
// down a histogram tells which digit the last one kept has; the digits found
// are the threshold, and one more walk in slot order writes the slots above
// it, and the first of those equal to it, to `kept`.  evict_copy_kernel moves
// the rows to other pages; in place, evict_shift_kernel moves them down,
// chunk after chunk.
#include <algorithm>

#include "paged.cuh"

namespace gqa {
namespace {

using paged::Seq;

constexpr int kSelThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyRows = 64;   // kept tokens per CTA of the copy
constexpr int kShiftThreads = 512;
constexpr int kShiftVecs = 8;   // 16-byte units per thread and chunk of the in-place move

struct EvictParams {
  PagedView v;
  void* k_pages;
  void* v_pages;
  float* weights;
  const int32_t* dst;
  int dst_max_pages;
  int Hkv, D, budget, recent, in_place;
  int32_t* kept;
  int32_t* new_seqlens;
};

// Tokens that sequence b keeps: -1 when it fails the checks (`code`).
__device__ __forceinline__ int kept_tokens(const EvictParams& p, int b, int& n, int& code) {
  Seq s;
  paged::load_seq(p.v, b, s, code);
  n = s.past;
  if (code) return -1;
  const int m = min(n, p.budget);
  if (!p.in_place && m > ((long long)p.dst_max_pages << p.v.page_log2)) {
    code = GQA_ERR_KV_OVERFLOW;
    return -1;
  }
  return m;
}

// A weight as an unsigned integer of the same order; NaN is 0, below all.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);  // (-0 equals +0)
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

// Inclusive sum over the block of a packed pair of 16-bit counts, and the
// block's total (the running sum of a pair stays below 2^16: at most one item
// a thread).
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* s_warp, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  __syncthreads();  // s_warp of the previous round has been read
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  uint32_t base = 0;
  total = 0;
  for (int i = 0; i < kSelThreads / 32; ++i) {
    if (i == warp) base = total;
    total += s_warp[i];
  }
  return v + base;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  __shared__ uint32_t s_hist[256];
  __shared__ uint32_t s_warp[kSelThreads / 32];
  __shared__ uint32_t s_digit, s_left;
  const int b = blockIdx.y, kh = blockIdx.x, tid = threadIdx.x;
  int n, code;
  const int m = kept_tokens(p, b, n, code);
  int32_t* kept = p.kept + ((size_t)b * p.Hkv + kh) * p.budget;
  if (code && kh == 0 && tid == 0) record_error(p.v.err, code);
  if (p.new_seqlens && kh == 0 && tid == 0) p.new_seqlens[b] = m < 0 ? n : m;
  for (int i = max(m, 0) + tid; i < p.budget; i += kSelThreads) kept[i] = -1;
  if (m <= 0) return;
  if (m == n) {
    for (int i = tid; i < n; i += kSelThreads) kept[i] = i;
    return;
  }
  const int32_t* tab = p.v.table + (size_t)b * p.v.max_pages;
  const int cand = n - p.recent, need = p.budget - p.recent;
  auto key = [&](int i) {
    const int pg = paged::page_of(p.v, tab, i);
    return pg < 0 ? 0u : order_key(p.weights[paged::pool_row(p.v, p.Hkv, pg, kh, i)]);
  };
  uint32_t thr = 0;      // the digits found
  uint32_t left = need;  // of those with these digits, so many are kept
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelThreads) s_hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < cand; i += kSelThreads) {
        const uint32_t u = key(i);
        if (shift == 24 || (u >> (shift + 8)) == (thr >> (shift + 8))) atomicAdd(&s_hist[(u >> shift) & 255], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        uint32_t l = left;
        int d = 255;
        while (d > 0 && s_hist[d] < l) l -= s_hist[d--];
        s_digit = d;
        s_left = l;
      }
      __syncthreads();
      thr |= s_digit << shift;
      left = s_left;
    }
  } else {
    thr = 0xFFFFFFFFu;  // above every key
  }
  // kept slots in order: above the threshold, and the first `left` equal to it
  uint32_t out = 0, ties = 0;
  for (int i0 = 0; i0 < cand; i0 += kSelThreads) {
    const int i = i0 + tid;
    const uint32_t u = i < cand && need > 0 ? key(i) : 0u;
    const bool gt = i < cand && need > 0 && u > thr, eq = i < cand && need > 0 && u == thr;
    uint32_t total;
    const uint32_t inc = block_scan((gt ? 1u : 0u) | (eq ? 0x10000u : 0u), s_warp, total);
    const uint32_t tie = ties + (inc >> 16) - (eq ? 1u : 0u);  // ties before this slot
    const uint32_t pos = out + (inc & 0xFFFFu) - (gt ? 1u : 0u) + min(tie, left);
    if (gt || (eq && tie < left)) kept[pos] = i;
    out += total & 0xFFFFu;
    ties += total >> 16;
  }
  for (int i = tid; i < p.recent; i += kSelThreads) kept[need + i] = cand + i;
}

// Kept token i of (b, kh): the pool rows it moves from and to; false when one
// of its pages is outside the pool.
__device__ __forceinline__ bool move_rows(const EvictParams& p, int b, int kh, int i, const int32_t* kept,
                                          size_t& from, size_t& to) {
  const int s = kept[i];
  const int pf = paged::page_of(p.v, p.v.table + (size_t)b * p.v.max_pages, s);
  const int32_t* drow = p.dst + (size_t)b * (p.in_place ? p.v.max_pages : p.dst_max_pages);
  const int pt = paged::page_of(p.v, drow, i);
  if (pf < 0 || pt < 0) return false;
  from = paged::pool_row(p.v, p.Hkv, pf, kh, s);
  to = paged::pool_row(p.v, p.Hkv, pt, kh, i);
  return true;
}

// To other pages: kCopyRows kept tokens of one (sequence, KV head) a CTA.
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const EvictParams p) {
  __shared__ size_t s_from[kCopyRows], s_to[kCopyRows];
  __shared__ int s_ok[kCopyRows];
  const int b = blockIdx.z, kh = blockIdx.y, tid = threadIdx.x;
  int n, code;
  const int m = kept_tokens(p, b, n, code);
  const int r0 = blockIdx.x * kCopyRows;
  if (r0 >= m) return;
  const int rows = min(kCopyRows, m - r0);
  const int32_t* kept = p.kept + ((size_t)b * p.Hkv + kh) * p.budget;
  if (tid < rows) {
    size_t f = 0, t = 0;
    const bool ok = move_rows(p, b, kh, r0 + tid, kept, f, t);
    s_from[tid] = f;
    s_to[tid] = t;
    s_ok[tid] = ok;
    if (ok) p.weights[t] = p.weights[f];
  }
  __syncthreads();
  const int nvec = p.D / 8;  // 16-byte units per row
  for (int u = tid; u < rows * nvec; u += kCopyThreads) {
    const int r = u / nvec, c = u - r * nvec;
    if (!s_ok[r]) continue;
    const uint4 k = *(reinterpret_cast<const uint4*>(p.k_pages) + s_from[r] * nvec + c);
    const uint4 v = *(reinterpret_cast<const uint4*>(p.v_pages) + s_from[r] * nvec + c);
    *(reinterpret_cast<uint4*>(p.k_pages) + s_to[r] * nvec + c) = k;
    *(reinterpret_cast<uint4*>(p.v_pages) + s_to[r] * nvec + c) = v;
  }
}

// In place: one CTA moves the K rows, the V rows or the weights of a
// (sequence, KV head) down.  Token i comes from slot kept[i] >= i, so the
// stores of a chunk cover only slots below every source of later chunks; a
// barrier between a chunk's loads and its stores keeps its own sources safe.
__global__ void __launch_bounds__(kShiftThreads) evict_shift_kernel(const EvictParams p) {
  const int b = blockIdx.z, kh = blockIdx.y, kind = blockIdx.x, tid = threadIdx.x;
  int n, code;
  const int m = kept_tokens(p, b, n, code);
  if (m <= 0 || m == n) return;
  const int32_t* kept = p.kept + ((size_t)b * p.Hkv + kh) * p.budget;
  if (kind == 2) {
    for (int i0 = 0; i0 < m; i0 += kShiftThreads) {
      const int i = i0 + tid;
      size_t f, t;
      const bool ok = i < m && move_rows(p, b, kh, i, kept, f, t);
      const float w = ok ? p.weights[f] : 0.f;
      __syncthreads();
      if (ok) p.weights[t] = w;
    }
    return;
  }
  uint4* pool = static_cast<uint4*>(kind ? p.v_pages : p.k_pages);
  const int nvec = p.D / 8;
  const long long units = (long long)m * nvec;
  for (long long u0 = 0; u0 < units; u0 += kShiftThreads * kShiftVecs) {
    uint4 x[kShiftVecs];
    size_t to[kShiftVecs];
    bool ok[kShiftVecs];
#pragma unroll
    for (int k = 0; k < kShiftVecs; ++k) {
      const long long u = u0 + k * kShiftThreads + tid;
      ok[k] = false;
      if (u < units) {
        const int i = (int)(u / nvec), c = (int)(u - (long long)i * nvec);
        size_t f, t;
        ok[k] = move_rows(p, b, kh, i, kept, f, t);
        if (ok[k]) {
          x[k] = pool[f * nvec + c];
          to[k] = t * nvec + c;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kShiftVecs; ++k)
      if (ok[k]) pool[to[k]] = x[k];
  }
}

}  // namespace

cudaError_t launch_paged_evict(const EvictArgs& a) {
  const EvictParams p{a.v, a.k_pages, a.v_pages, a.weights, a.dst, a.dst_max_pages, a.Hkv, a.D, a.budget, a.recent,
                      a.in_place, a.kept, a.new_seqlens};
  evict_select_kernel<<<dim3(a.Hkv, a.v.B), kSelThreads, 0, a.stream>>>(p);
  const int most = std::min(a.budget, a.v.total);  // tokens a sequence can keep
  if (a.in_place)
    evict_shift_kernel<<<dim3(3, a.Hkv, a.v.B), kShiftThreads, 0, a.stream>>>(p);
  else
    evict_copy_kernel<<<dim3((most + kCopyRows - 1) / kCopyRows, a.Hkv, a.v.B), kCopyThreads, 0, a.stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gqa
