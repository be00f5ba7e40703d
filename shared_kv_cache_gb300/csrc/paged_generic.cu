// Attention over the paged cache, and the weight each key receives, on CUDA
// cores for any head size D (a multiple of 8, at most 256): the shapes that
// the tensor-core kernels do not take.
//
// Attention: one warp per (token, query head), lane l owning dimensions l,
// l + 32, ...; online softmax in fp32 over the visible slots.  Key weights:
// one warp per (sequence, KV head, slot), which walks the new tokens that see
// the slot in order, so that the sum's order is fixed.  Both are bound by the
// latency of their dependent loads; they are the plain statement of the two
// operators on the GPU.
#include <algorithm>

#include "paged.cuh"

namespace gqa {
namespace {

using paged::Seq;

constexpr int kWarps = 4;

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

template <typename T, int NT>
__global__ void __launch_bounds__(kWarps * 32) paged_attn_generic_kernel(GenParams p) {
  using E = Elem<T>;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (blockIdx.x == 0)  // sequences that fail the checks are reported once
    for (int b = threadIdx.x; b < p.v.B; b += blockDim.x) {
      Seq s;
      int code;
      paged::load_seq(p.v, b, s, code);
      if (code) record_error(p.v.err, code);
    }
  if (row >= (long long)p.v.T * p.H) return;
  const int t = (int)(row / p.H), h = (int)(row - (long long)t * p.H);
  const int b = seq_of_row(p.v, t);
  if (b < 0) return;
  Seq s;
  int code;
  if (!paged::load_seq(p.v, b, s, code) || t >= s.q0 + s.n) return;
  const int kh = h / (p.H / p.Hkv);
  const int pos = s.past + t - s.q0;
  const int32_t* tab = p.v.table + (size_t)b * p.v.max_pages;
  const T* qrow = static_cast<const T*>(p.q) + (size_t)row * p.D;
  float q[NT], o[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int d = lane + 32 * i;
    q[i] = d < p.D ? E::to_f(qrow[d]) : 0.f;
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = paged::first_visible(pos, p.window); j <= pos; ++j) {
    const int pg = paged::page_of(p.v, tab, j);
    if (pg < 0) continue;
    const size_t r = paged::pool_row(p.v, p.Hkv, pg, kh, j) * p.D;
    const T* kr = static_cast<const T*>(p.k_pages) + r;
    const T* vr = static_cast<const T*>(p.v_pages) + r;
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int d = lane + 32 * i;
      if (d < p.D) x = fmaf(q[i], E::to_f(kr[d]), x);
    }
    x = warp_sum_f(x) * p.scale_log2;
    const float mn = fmaxf(m, x);
    const float mu = mn == -INFINITY ? 0.f : mn;
    const float corr = fast_exp2(m - mu), pj = fast_exp2(x - mu);
    l = l * corr + pj;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int d = lane + 32 * i;
      o[i] = o[i] * corr + (d < p.D ? pj * E::to_f(vr[d]) : 0.f);
    }
    m = mn;
  }
  T* orow = static_cast<T*>(p.out) + (size_t)row * p.D;
  const float inv = 1.f / l;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int d = lane + 32 * i;
    if (d < p.D) orow[d] = E::from_f(o[i] * inv);
  }
  if (p.lse && lane == 0) p.lse[row] = m * kLn2 + logf(l);
}

template <typename T, int NT>
__global__ void __launch_bounds__(kWarps * 32) paged_weights_generic_kernel(GenParams p) {
  using E = Elem<T>;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.z, kh = blockIdx.y;
  Seq s;
  int code;
  const bool any = paged::load_seq(p.v, b, s, code);
  if (code && blockIdx.x == 0 && kh == 0 && threadIdx.x == 0) record_error(p.v.err, code);
  if (!any) return;
  const int G = p.H / p.Hkv;
  const int32_t* tab = p.v.table + (size_t)b * p.v.max_pages;
  for (int j = paged::first_visible(s.past, p.window) + blockIdx.x * kWarps + (threadIdx.x >> 5); j < s.L;
       j += gridDim.x * kWarps) {
    const int pg = paged::page_of(p.v, tab, j);
    if (pg < 0) continue;
    const size_t r = paged::pool_row(p.v, p.Hkv, pg, kh, j);
    const T* kr = static_cast<const T*>(p.k_pages) + r * p.D;
    float k[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int d = lane + 32 * i;
      k[i] = d < p.D ? E::to_f(kr[d]) : 0.f;
    }
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
        for (int e = 0; e < NT; ++e) {
          const int d = lane + 32 * e;
          if (d < p.D) x = fmaf(k[e], E::to_f(qrow[d]), x);
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

template <typename T, int NT>
cudaError_t launch_nt(const PagedArgs& a, const GenParams& p) {
  if (p.w_out) {
    // a few CTAs per (sequence, KV head), each walking slots
    const int per = (int)std::min<long long>(((long long)a.v.total + kWarps - 1) / kWarps, 512);
    paged_weights_generic_kernel<T, NT><<<dim3(per, a.Hkv, a.v.B), kWarps * 32, 0, a.stream>>>(p);
  } else {
    const long long rows = (long long)a.v.T * a.H;
    paged_attn_generic_kernel<T, NT><<<(unsigned)((rows + kWarps - 1) / kWarps), kWarps * 32, 0, a.stream>>>(p);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const PagedArgs& a, const GenParams& p) {
  switch ((a.D + 31) / 32) {
    case 1: return launch_nt<T, 1>(a, p);
    case 2: return launch_nt<T, 2>(a, p);
    case 3: return launch_nt<T, 3>(a, p);
    case 4: return launch_nt<T, 4>(a, p);
    case 5: return launch_nt<T, 5>(a, p);
    case 6: return launch_nt<T, 6>(a, p);
    case 7: return launch_nt<T, 7>(a, p);
    default: return launch_nt<T, 8>(a, p);
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
