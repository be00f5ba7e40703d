// Eviction from a paged cache by accumulated attention weight.
//
// Of the n > budget tokens of a (sequence, KV head), the `recent` last stay
// and, of the n - recent others, the budget - recent of the largest weights
// (equal weights: the lower slot).
//
// Selection is by radix: the weights map to unsigned integers of the same order
// (NaN below all), and from the top digit down a histogram tells which digit
// the last one kept has; the digits found are the threshold.  A cluster of up
// to 8 CTAs (as many as run at once, two an SM) shares a (sequence, KV head):
// each holds a range of slots in shared memory, so the weights are read once,
// and leaves its histogram with every CTA through distributed shared memory
// (plain stores: atomic additions there took 5 times as long), one cluster
// barrier a digit.  The digits stop early when the bin found is kept whole.  A
// scan of each CTA's counts of keys above and at the threshold, exchanged the
// same way, then places the kept slots in order.  (One CTA a (sequence, KV
// head) that reads the weights in each of five passes took 95 us for 64 of them
// with 16-32K tokens, 24 us for 8 with 2047.)  Few candidates are selected by one
// CTA of the cluster, whose own barriers cost less.
//
// A thread sums one bin's copies and the bins are scanned once a CTA: when each
// warp read all bins for itself, from copies that lay 256 words apart (one
// bank for all counts of a digit), a digit took 1.4 us of shared-memory
// traffic instead of 1.0 with 2047 keys, 3.3 instead of 1.9 with 6000.
//
// Measured with 8 KV heads of 128, bf16: 8 sequences of 16 to 32 thousand tokens
// cut to 4096 63 us, of which the moved rows (277 MB) take 41 at the rate of a
// copy and the selection most of the rest (moving the recent tokens before it
// was slower, 69: the two copies of the moving loop spill); one of 2047 cut to
// 1024 11.8 us, a chain of dependent steps (lists, weights, three digits, two
// barriers, pages, rows).
//
// The same cluster then moves the kept rows, K, V and weight, bound by memory:
// in rounds, each CTA a run of rows whose units of 16 bytes are all loaded
// before one is stored.  Token i comes from slot kept[i] >= i, so in place a
// round's stores cover only slots below every source of later rounds; a
// cluster barrier between a round's loads and its stores keeps its own.
#include <algorithm>

#include "paged.cuh"

namespace gqa {
namespace {

using paged::at_rank;
using paged::cluster_rank;
using paged::cluster_sync;
using paged::Seq;
using paged::store_at;

constexpr int kSelThreads = 512;
constexpr int kMaxHeld = 40 * 1024;     // keys a CTA holds in shared memory at most
constexpr int kSolo = 8192;             // up to so many candidates one CTA selects: no cluster barriers
constexpr int kHistCopies = 8;          // local histograms, by lane, a bin's side by side: equal digits are common
constexpr int kHistStride = 12;         // words of a bin: vector reads of 8 neighbouring bins meet all 32 banks
constexpr int kUnits = 8;               // 16-byte units in flight per thread of a move

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

// Where key i of a CTA's range sits: a spare word every 8, so that threads
// walking 8 keys each meet different banks.
__device__ __forceinline__ int key_at(int i) { return i + (i >> 3); }
constexpr int key_words(int n) { return n + n / 8 + 9; }

// Writes the kept slots of (b, kh), m of n (0 < m < n), in order: the whole
// cluster.  s_keys holds the first `held` keys of this CTA's range.
template <int kCluster>
__device__ __forceinline__ void select_slots(const EvictParams& p, int b, int kh, int rank, int n, int32_t* kept,
                                             uint32_t* s_keys, int held) {
  __shared__ __align__(16) uint32_t s_local[256][kHistStride];  // this CTA's histogram
  __shared__ uint32_t s_hist[2][kCluster][256];                 // the cluster's, digits in turn
  __shared__ uint32_t s_sum[8], s_found[3];
  __shared__ uint32_t s_above[kCluster], s_equal[kCluster];
  __shared__ unsigned long long s_warp[kSelThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int all = kCluster * kSelThreads, mine = rank * kSelThreads + tid;
  const int cand = n - p.recent, need = p.budget - p.recent;
  for (int i = mine; i < p.recent; i += all) kept[need + i] = cand + i;
  const int peers = cand <= kSolo ? 1 : kCluster;  // CTAs that select
  if (need == 0 || rank >= peers) return;

  const int32_t* tab = p.v.table + (size_t)b * p.v.max_pages;
  const int seg = ((cand + peers - 1) / peers + 7) / 8 * 8;
  const int s0 = rank * seg, len = max(0, min(seg, cand - s0));  // this CTA's slots: s0 .. s0 + len - 1
  auto sync = [&]() {
    if (peers > 1) cluster_sync();
    else __syncthreads();
  };
  auto read_key = [&](int i) {
    const int pg = paged::page_of(p.v, tab, s0 + i);
    return pg < 0 ? 0u : order_key(p.weights[paged::pool_row(p.v, p.Hkv, pg, kh, s0 + i)]);
  };
  for (int i = tid; i < kHistStride * 256; i += kSelThreads) (&s_local[0][0])[i] = 0;
  // eight slots, of one page (s0 and the page size are multiples of 8), a step
  for (int i = 8 * tid; i < min(len, held); i += 8 * kSelThreads) {
    const int pg = paged::page_of(p.v, tab, s0 + i);
    float4 a = make_float4(NAN, NAN, NAN, NAN), c = a;
    if (pg >= 0) {
      const float4* src = reinterpret_cast<const float4*>(p.weights + paged::pool_row(p.v, p.Hkv, pg, kh, s0 + i));
      a = src[0];
      c = src[1];
    }
    uint32_t* dst = s_keys + key_at(i);  // (the spare word comes after these eight)
    dst[0] = order_key(a.x), dst[1] = order_key(a.y), dst[2] = order_key(a.z), dst[3] = order_key(a.w);
    dst[4] = order_key(c.x), dst[5] = order_key(c.y), dst[6] = order_key(c.z), dst[7] = order_key(c.w);
  }
  auto key = [&](int i) { return i < held ? s_keys[key_at(i)] : read_key(i); };
  sync();  // the keys are there, and every CTA has started

  uint32_t thr = 0, left = need;  // the digits found; of the keys with them, so many are kept
#pragma unroll 1
  for (int d = 0; d < 4; ++d) {
    const int shift = 24 - 8 * d;
    for (int i = tid; i < len; i += kSelThreads) {
      const uint32_t u = key(i);
      if (d == 0 || (u >> (shift + 8)) == (thr >> (shift + 8)))
        atomicAdd(&s_local[(u >> shift) & 255][lane & (kHistCopies - 1)], 1u);
    }
    __syncthreads();
    // thread t < 256 takes the bin 255 - t: counts it, and how many are in the bins down to it
    const int bin = 255 - tid;
    uint32_t count = 0, incl = 0;
    if (tid < 256) {
      uint4* h = reinterpret_cast<uint4*>(s_local[bin]);
#pragma unroll
      for (int k = 0; k < kHistCopies / 4; ++k) {
        const uint4 v = h[k];
        count += v.x + v.y + v.z + v.w;
        h[k] = make_uint4(0, 0, 0, 0);  // (for the next digit)
      }
    }
    if (peers > 1) {
      if (tid < 256)
#pragma unroll
        for (int r = 0; r < kCluster; ++r) store_at(at_rank(&s_hist[d & 1][rank][bin], r), count);
      cluster_sync();  // (a buffer is written again two digits on, a barrier after its last reader)
      if (tid < 256) {
        count = 0;
#pragma unroll
        for (int r = 0; r < kCluster; ++r) count += s_hist[d & 1][r][bin];
      }
    }
    if (tid < 256) {
      incl = count;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) s_sum[warp] = incl;
    }
    __syncthreads();
    if (tid < 256) {
#pragma unroll
      for (int i = 0; i < 8; ++i) incl += i < warp ? s_sum[i] : 0;
      if (incl >= left && incl - count < left) {  // (one bin: there are at least `left` keys)
        s_found[0] = bin;
        s_found[1] = left - (incl - count);
        s_found[2] = count;
      }
    }
    __syncthreads();
    thr |= s_found[0] << shift;
    left = s_found[1];
    if (left == s_found[2] && thr > 0) {
      // all keys with these digits are kept: those above the key before them
      // (with distinct weights mostly so after three digits)
      --thr;
      left = 0;
      break;
    }
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
  if (tid < peers) {
    store_at(at_rank(&s_above[rank], tid), (uint32_t)total);
    store_at(at_rank(&s_equal[rank], tid), (uint32_t)(total >> 32));
  }
  sync();
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

// Kept token i of (b, kh), from slot s: the pool rows it moves from and to;
// false when one of its pages is outside the pool.
__device__ __forceinline__ bool move_rows(const EvictParams& p, int b, int kh, int i, int s, size_t& from, size_t& to) {
  const int pf = paged::page_of(p.v, p.v.table + (size_t)b * p.v.max_pages, s);
  const int32_t* drow = p.dst + (size_t)b * (p.in_place ? p.v.max_pages : p.dst_max_pages);
  const int pt = paged::page_of(p.v, drow, i);
  if (pf < 0 || pt < 0) return false;
  from = paged::pool_row(p.v, p.Hkv, pf, kh, s);
  to = paged::pool_row(p.v, p.Hkv, pt, kh, i);
  return true;
}

template <int kCluster>
__global__ void __launch_bounds__(kSelThreads, 2) evict_kernel(const __grid_constant__ EvictParams p, int held) {
  extern __shared__ uint32_t s_keys[];
  __shared__ size_t s_from[2][kSelThreads], s_to[2][kSelThreads];  // rows of a round, rounds in turn
  const int b = blockIdx.z, kh = blockIdx.y, tid = threadIdx.x;
  const int rank = (int)cluster_rank();
  pdl_wait_primary();
  pdl_launch_dependents();
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
    if (p.in_place) return;
  } else {
    select_slots<kCluster>(p, b, kh, rank, n, kept, s_keys, held);
  }
  cluster_sync();  // kept is written

  constexpr size_t kNone = ~size_t(0);
  const int nvec = p.D / 8;  // 16-byte units of a row
  const int rows = min(kSelThreads, kUnits * kSelThreads / (2 * nvec));  // of a CTA and round
  const int step = kCluster * rows;
  uint4* kp = static_cast<uint4*>(p.k_pages);
  uint4* vp = static_cast<uint4*>(p.v_pages);
  auto places = [&](int r0, int buf) {  // of the round from kept token r0 on
    if (tid >= rows) return;
    const int i = r0 + rank * rows + tid;
    size_t from = kNone, to = kNone;
    if (i < m && !move_rows(p, b, kh, i, __ldcg(kept + i), from, to)) from = to = kNone;
    s_from[buf][tid] = from;
    s_to[buf][tid] = to;
  };
  places(0, 0);
  __syncthreads();
  for (int r0 = 0, buf = 0; r0 < m; r0 += step, buf ^= 1) {
    const size_t from = tid < rows ? s_from[buf][tid] : kNone;
    const float w = from != kNone ? p.weights[from] : 0.f;
    uint4 x[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int at = u * kSelThreads + tid, r = at / (2 * nvec), c = at - r * 2 * nvec;
      if (r < rows && s_from[buf][r] != kNone)
        x[u] = c < nvec ? kp[s_from[buf][r] * nvec + c] : vp[s_from[buf][r] * nvec + c - nvec];
    }
    if (r0 + step < m) places(r0 + step, buf ^ 1);  // (while the rows are on their way)
    if (p.in_place) cluster_sync();
    if (from != kNone) p.weights[s_to[buf][tid]] = w;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int at = u * kSelThreads + tid, r = at / (2 * nvec), c = at - r * 2 * nvec;
      if (r < rows && s_from[buf][r] != kNone)
        (c < nvec ? kp[s_to[buf][r] * nvec + c] : vp[s_to[buf][r] * nvec + c - nvec]) = x[u];
    }
    __syncthreads();  // the next round's places are written, this one's read
  }
}

template <int kCluster>
cudaError_t launch_cluster(const EvictArgs& a, const EvictParams& p) {
  // (keys beyond the shared memory are read again in each pass)
  const int range = ((a.v.total + kCluster - 1) / kCluster + 7) / 8 * 8;
  const int held = std::min(std::max(range, (std::min(a.v.total, kSolo) + 7) / 8 * 8), kMaxHeld);
  const int smem = key_words(held) * 4;
  static std::atomic<int> smem_set[kMaxDevices];
  const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(evict_kernel<kCluster>), smem, smem_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster, a.Hkv, a.v.B);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_kernel<kCluster>, p, held);
}

}  // namespace

cudaError_t launch_paged_evict(const EvictArgs& a) {
  const EvictParams p{a.v, a.k_pages, a.v_pages, a.weights, a.dst, a.dst_max_pages, a.Hkv, a.D, a.budget, a.recent,
                      a.in_place, a.kept, a.new_seqlens};
  // the largest cluster with which all run at once: 64 items of 16-32K tokens
  // take 72 us in clusters of 8 (two waves), 63 in clusters of 4, 94 of 2
  const long long items = (long long)a.v.B * a.Hkv, slots = 2ll * a.num_sms;
  if (items * 8 <= slots) return launch_cluster<8>(a, p);
  if (items * 4 <= slots) return launch_cluster<4>(a, p);
  return launch_cluster<2>(a, p);
}

}  // namespace gqa
