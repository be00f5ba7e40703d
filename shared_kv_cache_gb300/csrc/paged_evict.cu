// Eviction from a paged cache by accumulated attention weight.
//
// Of the n > budget tokens of a (sequence, KV head), the `recent` last stay
// and, of the n - recent others, the budget - recent of the largest weights
// (equal weights: the lower slot).
//
// evict_select_kernel finds them by radix selection: the weights map to
// unsigned integers of the same order (NaN below all), and from the top digit
// down a histogram tells which digit the last one kept has; the digits found
// are the threshold.  A cluster of kCluster CTAs shares a (sequence, KV head):
// each holds a range of slots in shared memory, so the weights are read once,
// and leaves its histogram with every CTA through distributed shared memory
// (plain stores: atomic additions there took 5 times as long), one cluster
// barrier a digit.  A scan of each CTA's counts of
// keys above and at the threshold, exchanged the same way, then places the
// kept slots in order.  (One CTA a (sequence, KV head) that reads the weights
// in each of five passes: 95 us for 64 of them with 16-32K tokens, 24 us for
// 8 with 2047.)
//
// evict_copy_kernel moves the rows to other pages, bound by memory; in place,
// evict_shift_kernel moves them down, chunk after chunk.
#include <algorithm>

#include "paged.cuh"

namespace gqa {
namespace {

using paged::Seq;

constexpr int kSelThreads = 512;
constexpr int kCluster = 8;             // CTAs per (sequence, KV head)
constexpr int kMaxHeld = 40 * 1024;     // keys a CTA holds in shared memory at most
constexpr int kHistCopies = 4;          // local histograms, by lane (equal digits are common)
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

// Where key i of a CTA's range sits: a spare word every 8, so that threads
// walking 8 keys each meet different banks.
__device__ __forceinline__ int key_at(int i) { return i + (i >> 3); }
constexpr int key_words(int n) { return n + n / 8 + 1; }

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSelThreads)
    evict_select_kernel(const __grid_constant__ EvictParams p, int held) {
  extern __shared__ uint32_t s_keys[];  // the first `held` keys of the range
  __shared__ uint32_t s_local[kHistCopies][256];
  __shared__ uint32_t s_hist[2][kCluster][256];  // the cluster's histograms, digits in turn
  __shared__ uint32_t s_total[256];              // their sum
  __shared__ uint32_t s_above[kCluster], s_equal[kCluster];
  __shared__ unsigned long long s_warp[kSelThreads / 32];
  const int b = blockIdx.z, kh = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = (int)cluster_rank();
  pdl_launch_dependents();
  pdl_wait_primary();
  int n, code;
  const int m = kept_tokens(p, b, n, code);  // (uniform over the cluster)
  int32_t* kept = p.kept + ((size_t)b * p.Hkv + kh) * p.budget;
  const int all = kCluster * kSelThreads, mine = rank * kSelThreads + tid;
  if (code && kh == 0 && mine == 0) record_error(p.v.err, code);
  if (p.new_seqlens && kh == 0 && mine == 0) p.new_seqlens[b] = m < 0 ? n : m;
  for (int i = max(m, 0) + mine; i < p.budget; i += all) kept[i] = -1;
  if (m <= 0) return;
  if (m == n) {
    for (int i = mine; i < n; i += all) kept[i] = i;
    return;
  }
  const int cand = n - p.recent, need = p.budget - p.recent;
  for (int i = mine; i < p.recent; i += all) kept[need + i] = cand + i;
  if (need == 0) return;

  const int32_t* tab = p.v.table + (size_t)b * p.v.max_pages;
  const int seg = (cand + kCluster - 1) / kCluster;
  const int s0 = rank * seg, len = max(0, min(seg, cand - s0));  // this CTA's slots: s0 .. s0 + len - 1
  auto read_key = [&](int i) {
    const int pg = paged::page_of(p.v, tab, s0 + i);
    return pg < 0 ? 0u : order_key(p.weights[paged::pool_row(p.v, p.Hkv, pg, kh, s0 + i)]);
  };
#pragma unroll 4
  for (int i = tid; i < min(len, held); i += kSelThreads) s_keys[key_at(i)] = read_key(i);
  auto key = [&](int i) { return i < held ? s_keys[key_at(i)] : read_key(i); };
  cluster_sync();  // every CTA of the cluster has started

  uint32_t thr = 0, left = need;  // the digits found; of the keys with them, so many are kept
#pragma unroll 1
  for (int d = 0; d < 4; ++d) {
    const int shift = 24 - 8 * d;
    for (int i = tid; i < kHistCopies * 256; i += kSelThreads) s_local[i >> 8][i & 255] = 0;
    __syncthreads();
    for (int i = tid; i < len; i += kSelThreads) {
      const uint32_t u = key(i);
      if (d == 0 || (u >> (shift + 8)) == (thr >> (shift + 8)))
        atomicAdd(&s_local[lane & (kHistCopies - 1)][(u >> shift) & 255], 1u);
    }
    __syncthreads();
    for (int i = tid; i < 256 * kCluster; i += kSelThreads) {
      const int bin = i & 255;
      uint32_t v = 0;
#pragma unroll
      for (int k = 0; k < kHistCopies; ++k) v += s_local[k][bin];
      store_at(at_rank(&s_hist[d & 1][rank][bin], i >> 8), v);
    }
    cluster_sync();  // (a buffer is written again two digits on, a barrier after its last reader)
    if (tid < 256) {
      uint32_t v = 0;
#pragma unroll
      for (int k = 0; k < kCluster; ++k) v += s_hist[d & 1][k][tid];
      s_total[tid] = v;
    }
    __syncthreads();
    // every warp finds the digit for itself: lane l holds the bins 255 - 8 l
    // down to 248 - 8 l
    uint32_t bin[8], sum = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += bin[k] = s_total[255 - 8 * lane - k];
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const int l = __ffs(__ballot_sync(0xffffffffu, incl >= left)) - 1;  // (the last lane's sum is >= left)
    uint32_t before = incl - sum, digit = 255 - 8 * lane;
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (before + bin[k] < left) {
        before += bin[k];
        --digit;
      } else {
        break;
      }
    digit = __shfl_sync(0xffffffffu, digit, l);
    left -= __shfl_sync(0xffffffffu, before, l);
    thr |= digit << shift;
  }
  // the keys above the threshold and those equal to it, a run of keys a thread
  const int per = (len + kSelThreads - 1) / kSelThreads;
  const int r0 = min(len, tid * per), r1 = min(len, r0 + per);
  uint32_t above = 0, equal = 0;
  for (int i = r0; i < r1; ++i) {
    const uint32_t u = key(i);
    above += u > thr;
    equal += u == thr;
  }
  unsigned long long v = ((unsigned long long)equal << 32) | above;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  unsigned long long base = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kSelThreads / 32; ++i) {
    if (i == warp) base = total;
    total += s_warp[i];
  }
  v += base;
  if (tid < kCluster) {
    store_at(at_rank(&s_above[rank], tid), (uint32_t)total);
    store_at(at_rank(&s_equal[rank], tid), (uint32_t)(total >> 32));
  }
  cluster_sync();
  uint32_t out = (uint32_t)v - above, ties = (uint32_t)(v >> 32) - equal;  // before this thread's run
  for (int i = 0; i < rank; ++i) {
    out += s_above[i];
    ties += s_equal[i];
  }
  for (int i = r0; i < r1; ++i) {
    const uint32_t u = key(i);
    if (u > thr) {
      kept[out++ + min(ties, left)] = s0 + i;
    } else if (u == thr) {
      if (ties < left) kept[out + ties] = s0 + i;
      ++ties;
    }
  }
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
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const __grid_constant__ EvictParams p) {
  __shared__ size_t s_from[kCopyRows], s_to[kCopyRows];
  __shared__ int s_ok[kCopyRows];
  const int b = blockIdx.z, kh = blockIdx.y, tid = threadIdx.x;
  pdl_wait_primary();
  pdl_launch_dependents();
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
  constexpr int kUnits = 4;  // of K and of V in flight per thread
  for (int u0 = tid; u0 < rows * nvec; u0 += kUnits * kCopyThreads) {
    uint4 k[kUnits], v[kUnits];
    size_t to[kUnits];
    bool ok[kUnits];
#pragma unroll
    for (int x = 0; x < kUnits; ++x) {
      const int u = u0 + x * kCopyThreads, r = u / nvec, c = u - r * nvec;
      ok[x] = u < rows * nvec && s_ok[r];
      if (ok[x]) {
        const size_t from = s_from[r] * nvec + c;
        to[x] = s_to[r] * nvec + c;
        k[x] = __ldg(reinterpret_cast<const uint4*>(p.k_pages) + from);
        v[x] = __ldg(reinterpret_cast<const uint4*>(p.v_pages) + from);
      }
    }
#pragma unroll
    for (int x = 0; x < kUnits; ++x)
      if (ok[x]) {
        *(reinterpret_cast<uint4*>(p.k_pages) + to[x]) = k[x];
        *(reinterpret_cast<uint4*>(p.v_pages) + to[x]) = v[x];
      }
  }
}

// In place: one CTA moves the K rows, the V rows or the weights of a
// (sequence, KV head) down.  Token i comes from slot kept[i] >= i, so the
// stores of a chunk cover only slots below every source of later chunks; a
// barrier between a chunk's loads and its stores keeps its own sources safe.
__global__ void __launch_bounds__(kShiftThreads) evict_shift_kernel(const __grid_constant__ EvictParams p) {
  const int b = blockIdx.z, kh = blockIdx.y, kind = blockIdx.x, tid = threadIdx.x;
  pdl_wait_primary();
  pdl_launch_dependents();
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
  // (keys beyond the shared memory are read again in each pass)
  const int held = std::min((a.v.total + kCluster - 1) / kCluster, kMaxHeld);
  const int smem = key_words(held) * 4;
  static std::atomic<int> smem_set[kMaxDevices];
  cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(evict_select_kernel), smem, smem_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster, a.Hkv, a.v.B);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, held);
  if (e != cudaSuccess) return e;
  cfg.dynamicSmemBytes = 0;
  const int most = std::min(a.budget, a.v.total);  // tokens a sequence can keep
  if (a.in_place) {
    cfg.gridDim = dim3(3, a.Hkv, a.v.B);
    cfg.blockDim = dim3(kShiftThreads);
    return cudaLaunchKernelEx(&cfg, evict_shift_kernel, p);
  }
  cfg.gridDim = dim3((most + kCopyRows - 1) / kCopyRows, a.Hkv, a.v.B);
  cfg.blockDim = dim3(kCopyThreads);
  return cudaLaunchKernelEx(&cfg, evict_copy_kernel, p);
}

}  // namespace gqa
