// Attention over the paged cache, and the weight each key receives, on CUDA
// cores for any head size D (a multiple of 8, at most 256): the shapes that
// the tensor-core kernels do not take.
//
// Attention: a CTA of eight warps (a cluster of CTAs where there are few rows)
// per (token, query head); each warp takes four slots in turn with an online
// softmax in fp32, and the warps' (and CTAs') states are merged in shared memory.  Key
// weights: one warp per (sequence, KV head, slot), which walks the new tokens
// that see the slot in order, so that the sum's order is fixed.  Bound by the
// latency of the loads, and with many rows by reading each key row once a
// row: one token of each of 16 sequences of 4000, 32 on 8 heads of 96, takes 328 us
// (a warp a row took 6390), 2 sequences of 8000 with 16 heads of 256 130 (12048), a
// prompt of 512 tokens with 32 heads of 96 505 (734).
#include <algorithm>

#include "paged.cuh"

namespace gqa {
namespace {

using paged::Seq;

constexpr int kWarps = 4;
constexpr int kAttnWarps = 8;  // of a (token, query head): they take its slots in turn ...
constexpr int kKeys = 4;       // ... so many at a time, whose loads go out together
constexpr int kClusterCtas = 8;
static_assert(kAttnWarps * 32 >= 256, "a thread an output dimension");

struct GenParams {
  PagedView v;
  const void* q;
  const void* k_pages;
  const void* v_pages;
  void* out;
  float* lse;
  const float* w_in;
  float* w_out;
  int H, Hkv, D, window;
  float scale_log2;
};

__device__ __forceinline__ float warp_sum_f(float s) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  return s;
}

// The sequence of row t of the token arrays (-1: none), by bisection over
// cu_seqlens.
__device__ __forceinline__ int seq_of_row(const PagedView& v, int t) {
  int lo = 0, hi = v.B;  // the first b with cu[b + 1] > t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (v.cu[mid + 1] > t) hi = mid;
    else lo = mid + 1;
  }
  return lo < v.B && v.cu[lo] <= t ? lo : -1;
}

// Lane l owns the dimension pairs l, l + 32, ... of a row: NP of them, as far as
// the head has so many.
template <typename T>
__device__ __forceinline__ float2 pair_of(const T* row, int i, bool there) {
  return there ? Elem<T>::unpack2(reinterpret_cast<const uint32_t*>(row)[i]) : make_float2(0.f, 0.f);
}

template <typename T, int NP, int kCluster>
__global__ void __launch_bounds__(kAttnWarps * 32) paged_attn_generic_kernel(GenParams p) {
  using E = Elem<T>;
  __shared__ float s_o[kAttnWarps][64 * NP];
  __shared__ float s_m[kAttnWarps], s_l[kAttnWarps];
  __shared__ float c_o[kCluster][64 * NP], c_m[kCluster], c_l[kCluster];  // (of rank 0: the CTAs' states)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x / kCluster;  // (T * H * kCluster < 2^31)
  const int rank = kCluster > 1 ? (int)paged::cluster_rank() : 0;
  if (blockIdx.x == 0)  // sequences that fail the checks are reported once
    for (int b = threadIdx.x; b < p.v.B; b += blockDim.x) {
      Seq s;
      int code;
      paged::load_seq(p.v, b, s, code);
      if (code) record_error(p.v.err, code);
    }
  const int t = row / p.H, h = row - t * p.H;
  const int b = seq_of_row(p.v, t);
  if (b < 0) return;  // (so do all CTAs of the cluster)
  Seq s;
  int code;
  if (!paged::load_seq(p.v, b, s, code) || t >= s.q0 + s.n) return;
  const int kh = h / (p.H / p.Hkv), pairs = p.D / 2;
  const int pos = s.past + t - s.q0;
  const int32_t* tab = p.v.table + (size_t)b * p.v.max_pages;
  const T* qrow = static_cast<const T*>(p.q) + (size_t)row * p.D;
  float2 q[NP], o[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    q[i] = pair_of(qrow, lane + 32 * i, lane + 32 * i < pairs);
    o[i] = make_float2(0.f, 0.f);
  }
  float m = -INFINITY, l = 0.f;
  // (64 bits: the last step may pass 2^31)
  for (long long j0 = paged::first_visible(pos, p.window) + kKeys * (rank * kAttnWarps + warp); j0 <= pos;
       j0 += kKeys * kAttnWarps * kCluster) {
    float x[kKeys];
    float2 v[kKeys][NP];
    bool there[kKeys];
#pragma unroll
    for (int u = 0; u < kKeys; ++u) {
      const int j = (int)j0 + u;
      const int pg = j <= pos ? paged::page_of(p.v, tab, j) : -1;
      there[u] = pg >= 0;
      const size_t r = there[u] ? paged::pool_row(p.v, p.Hkv, pg, kh, j) * p.D : 0;
      x[u] = 0.f;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const bool in = there[u] && lane + 32 * i < pairs;
        const float2 k = pair_of(static_cast<const T*>(p.k_pages) + r, lane + 32 * i, in);
        v[u][i] = pair_of(static_cast<const T*>(p.v_pages) + r, lane + 32 * i, in);
        x[u] = fmaf(q[i].x, k.x, fmaf(q[i].y, k.y, x[u]));
      }
    }
    float mn = m;
#pragma unroll
    for (int u = 0; u < kKeys; ++u) {
      x[u] = there[u] ? warp_sum_f(x[u]) * p.scale_log2 : -INFINITY;
      mn = fmaxf(mn, x[u]);
    }
    const float mu = mn == -INFINITY ? 0.f : mn;
    const float corr = fast_exp2(m - mu);
    l *= corr;
#pragma unroll
    for (int i = 0; i < NP; ++i) o[i] = make_float2(o[i].x * corr, o[i].y * corr);
#pragma unroll
    for (int u = 0; u < kKeys; ++u) {
      const float pj = fast_exp2(x[u] - mu);
      l += pj;
#pragma unroll
      for (int i = 0; i < NP; ++i) o[i] = make_float2(fmaf(pj, v[u][i].x, o[i].x), fmaf(pj, v[u][i].y, o[i].y));
    }
    m = mn;
  }
  // the warps' states, merged in their order, and then the CTAs'
#pragma unroll
  for (int i = 0; i < NP; ++i) *reinterpret_cast<float2*>(&s_o[warp][2 * (lane + 32 * i)]) = o[i];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  const int d = threadIdx.x;
  // state `n` of ms, ls and os into (M, L, a), a the thread's dimension
  auto merge = [&](const float* ms, const float* ls, const float* os, int n, float& M, float& L, float& a) {
    M = -INFINITY;
    for (int w = 0; w < n; ++w) M = fmaxf(M, ms[w]);
    const float base = M == -INFINITY ? 0.f : M;
    L = a = 0.f;
    for (int w = 0; w < n; ++w) {
      const float f = fast_exp2(ms[w] - base);
      L += ls[w] * f;
      if (d < p.D) a = fmaf(os[w * 64 * NP + d], f, a);
    }
  };
  float M, L, a;
  if (kCluster > 1) paged::cluster_sync();  // (every CTA has started: its shared memory may be written)
  else __syncthreads();
  merge(s_m, s_l, s_o[0], kAttnWarps, M, L, a);
  if (kCluster > 1) {
    if (d < p.D) paged::store_at(paged::at_rank(&c_o[rank][d], 0), __float_as_uint(a));
    if (d == 0) {
      paged::store_at(paged::at_rank(&c_m[rank], 0), __float_as_uint(M));
      paged::store_at(paged::at_rank(&c_l[rank], 0), __float_as_uint(L));
    }
    paged::cluster_sync();
    if (rank != 0) return;
    merge(c_m, c_l, c_o[0], kCluster, M, L, a);
  }
  if (d < p.D) static_cast<T*>(p.out)[(size_t)row * p.D + d] = E::from_f(a / L);
  if (p.lse && d == 0) p.lse[row] = M * kLn2 + logf(L);
}

template <typename T, int NP>
__global__ void __launch_bounds__(kWarps * 32) paged_weights_generic_kernel(GenParams p) {
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.z, kh = blockIdx.y;
  Seq s;
  int code;
  const bool any = paged::load_seq(p.v, b, s, code);
  if (code && blockIdx.x == 0 && kh == 0 && threadIdx.x == 0) record_error(p.v.err, code);
  if (!any) return;
  const int G = p.H / p.Hkv, pairs = p.D / 2;
  const int32_t* tab = p.v.table + (size_t)b * p.v.max_pages;
  for (int j = paged::first_visible(s.past, p.window) + blockIdx.x * kWarps + (threadIdx.x >> 5); j < s.L;
       j += gridDim.x * kWarps) {
    const int pg = paged::page_of(p.v, tab, j);
    if (pg < 0) continue;
    const size_t r = paged::pool_row(p.v, p.Hkv, pg, kh, j);
    const T* kr = static_cast<const T*>(p.k_pages) + r * p.D;
    float2 k[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) k[i] = pair_of(kr, lane + 32 * i, lane + 32 * i < pairs);
    // tokens i0 .. i1 - 1 see slot j
    const int i0 = max(0, j - s.past);
    const int i1 = p.window > 0 ? (int)min((long long)s.n, (long long)j + p.window - s.past) : s.n;
    float w = 0.f;
    for (int i = i0; i < i1; ++i)
      for (int g = 0; g < G; ++g) {
        const size_t row = (size_t)(s.q0 + i) * p.H + kh * G + g;
        const T* qrow = static_cast<const T*>(p.q) + row * p.D;
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          const float2 q = pair_of(qrow, lane + 32 * e, lane + 32 * e < pairs);
          x = fmaf(k[e].x, q.x, fmaf(k[e].y, q.y, x));
        }
        x = warp_sum_f(x);
        w += fast_exp2(fmaf(x, p.scale_log2, -p.lse[row] * kLog2e));
      }
    if (lane == 0) p.w_out[r] = (j < s.past ? p.w_in[r] : 0.f) + w;
  }
}

GenParams params_of(const PagedArgs& a) {
  return GenParams{a.v, a.q, a.k_pages, a.v_pages, a.out, a.lse, nullptr, nullptr, a.H, a.Hkv, a.D, a.window,
                   a.scale * kLog2e};
}

template <typename T, int NP, int kCluster>
cudaError_t launch_attention(const PagedArgs& a, const GenParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.v.T * a.H * kCluster));
  cfg.blockDim = dim3(kAttnWarps * 32);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_attn_generic_kernel<T, NP, kCluster>, p);
}

template <typename T, int NP>
cudaError_t launch_np(const PagedArgs& a, const GenParams& p) {
  if (p.w_out) {
    // a few CTAs per (sequence, KV head), each walking slots
    const int per = (int)std::min<long long>(((long long)a.v.total + kWarps - 1) / kWarps, 512);
    paged_weights_generic_kernel<T, NP><<<dim3(per, a.Hkv, a.v.B), kWarps * 32, 0, a.stream>>>(p);
    return cudaGetLastError();
  }
  // few rows over many slots: a cluster of CTAs a row.  us, one CTA / a cluster,
  // with head size 96: 128 rows of 256 slots 29 / 17, of 4096 355 / 99; 512 rows of 256
  // 33 / 52, of 1024 105 / 111, of 4096 394 / 337
  const long long rows = (long long)a.v.T * a.H;
  const int reach = a.window > 0 ? std::min(a.window, a.v.total) : a.v.total;
  if ((rows <= a.num_sms && reach >= 256) || (rows <= 4ll * a.num_sms && reach >= 2048))
    return launch_attention<T, NP, kClusterCtas>(a, p);
  return launch_attention<T, NP, 1>(a, p);
}

template <typename T>
cudaError_t launch_t(const PagedArgs& a, const GenParams& p) {
  switch ((a.D + 63) / 64) {
    case 1: return launch_np<T, 1>(a, p);
    case 2: return launch_np<T, 2>(a, p);
    case 3: return launch_np<T, 3>(a, p);
    default: return launch_np<T, 4>(a, p);
  }
}

}  // namespace

cudaError_t launch_paged_generic(const PagedArgs& a) {
  const GenParams p = params_of(a);
  return a.dtype == GQA_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, p) : launch_t<__half>(a, p);
}

cudaError_t launch_paged_weights_generic(const PagedArgs& a, const float* w_in, float* w_out) {
  GenParams p = params_of(a);
  p.w_in = w_in;
  p.w_out = w_out;
  return a.dtype == GQA_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, p) : launch_t<__half>(a, p);
}

}  // namespace gqa
