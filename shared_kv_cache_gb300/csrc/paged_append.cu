// The new rows of a paged cache in one pass: per-head RMS norm of queries and
// keys, rotary embedding, and the scatter of keys and values into the pages.
//
//   x' = x * rsqrt(mean(x^2) + eps) * w         (per head, where w is given)
//   y1 = x1' c - x2' s,  y2 = x2' c + x1' s     (pairs (j, j + D/2) or (2j, 2j + 1))
//
// all in fp32, rounded to T once, so norm and rotation cost no extra rounding
// and no extra trip through memory.
//
// Bound by memory: each row is read and written once.  A warp takes one token
// (or, when there are few tokens, every parts-th slice of one), and its lanes
// a slice of 32 / LP heads at a time: a lane holds VEC dimensions of the lower
// half of a head and the VEC they pair with (interleaved: 2 VEC neighbours),
// so the rotation is thread-local and the norm takes log2(LP) shuffles.  The
// slices of a batch are loaded together before any is computed.
#include <algorithm>

#include "paged.cuh"

namespace gqa {
namespace {

using paged::Seq;

constexpr int kWarps = 4;
constexpr int kBatch = 3;  // slices in flight per warp

struct AppendParams {
  AppendArgs a;
  int parts;  // warps per token
};

// First sequence b with cu[b + 1] > t (v.B: none), 32 candidates a round.
__device__ __forceinline__ int find_sequence(const PagedView& v, int t, int lane) {
  int lo = 0, hi = v.B;  // the answer is in [lo, hi], hi when none of [lo, hi) is it
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5;
    const int probe = min(lo + (lane + 1) * step, hi);  // is cu[probe] > t?
    const unsigned above = __ballot_sync(0xffffffffu, v.cu[probe] > t);
    if (!above) return hi;
    const int first = __ffs(above) - 1;
    const int nlo = lo + first * step;
    hi = min(nlo + step, hi) - 1;
    lo = nlo;
  }
  return lo;
}

template <typename T, int VEC, int LP>
__global__ void __launch_bounds__(kWarps * 32) paged_append_kernel(const __grid_constant__ AppendParams pp) {
  using E = Elem<T>;
  using V = VecT<T, VEC>;
  using V8 = VecT<T, 8>;
  constexpr int kHeads = 32 / LP;  // heads per slice
  const AppendArgs& p = pp.a;
  const int lane = threadIdx.x & 31;
  // the previous kernel may still be writing this one's inputs; the next one
  // may start once they are complete (it waits for this grid before it reads
  // what is written here)
  pdl_wait_primary();
  pdl_launch_dependents();
  if (blockIdx.x == 0)  // sequences that fail the checks are reported once
    for (int b = threadIdx.x; b < p.v.B; b += blockDim.x) {
      Seq s;
      int code;
      paged::load_seq(p.v, b, s, code);
      if (code) record_error(p.v.err, code);
    }
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = (int)(w / pp.parts), part = (int)(w - (long long)t * pp.parts);
  if (t >= p.v.T) return;
  const int b = find_sequence(p.v, t, lane);
  if (b >= p.v.B) return;  // rows behind the last sequence stay as they are
  Seq s;
  int code;
  if (!paged::load_seq(p.v, b, s, code) || t < s.q0 || t >= s.q0 + s.n) return;
  const int slot = s.past + t - s.q0;
  const int pos = p.positions ? p.positions[t] : slot;
  if (p.cos && (unsigned)pos >= (unsigned)p.cos_rows) {
    if (lane == 0) record_error(p.v.err, GQA_ERR_INVALID_ARGUMENT);
    return;
  }
  const int pg = paged::page_of(p.v, p.v.table + (size_t)b * p.v.max_pages, slot);
  const int D = p.D, half = D / 2;
  const int li = lane % LP, gi = lane / LP;
  const bool act = li * VEC < half;
  const bool inter = p.interleaved != 0;
  // the lane's two vectors of a head: pair members (x1, x2), or neighbours
  const int off1 = inter ? 2 * li * VEC : li * VEC;
  const int off2 = inter ? off1 + VEC : half + off1;
  V cv, sv, qw1, qw2, kw1, kw2;
  if (act) {
    if (p.cos) {
      const size_t r = (size_t)pos * half + li * VEC;
      cv = *reinterpret_cast<const V*>(static_cast<const T*>(p.cos) + r);
      sv = *reinterpret_cast<const V*>(static_cast<const T*>(p.sin) + r);
    }
    if (p.qw) {
      qw1 = *reinterpret_cast<const V*>(static_cast<const T*>(p.qw) + off1);
      qw2 = *reinterpret_cast<const V*>(static_cast<const T*>(p.qw) + off2);
    }
    if (p.kw) {
      kw1 = *reinterpret_cast<const V*>(static_cast<const T*>(p.kw) + off1);
      kw2 = *reinterpret_cast<const V*>(static_cast<const T*>(p.kw) + off2);
    }
  }
  const T* qrow = static_cast<const T*>(p.q) + (size_t)t * p.q_stride;
  const T* krow = static_cast<const T*>(p.k) + (size_t)t * p.kv_stride;
  const T* vrow = static_cast<const T*>(p.value) + (size_t)t * p.kv_stride;
  T* qout = static_cast<T*>(p.q_out) + (size_t)t * p.H * D;
  T* kp = static_cast<T*>(p.k_pages);
  T* vp = static_cast<T*>(p.v_pages);
  const int nq = (p.H + kHeads - 1) / kHeads, nk = (p.Hkv + kHeads - 1) / kHeads;

  for (int s0 = part; s0 < nq + nk; s0 += kBatch * pp.parts) {
    V x1[kBatch], x2[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int sl = s0 + u * pp.parts;
      const bool isq = sl < nq;
      const int head = (isq ? sl : sl - nq) * kHeads + gi;
      if (act && sl < nq + nk && head < (isq ? p.H : p.Hkv)) {
        const T* src = (isq ? qrow : krow) + (size_t)head * D;
        x1[u] = *reinterpret_cast<const V*>(src + off1);
        x2[u] = *reinterpret_cast<const V*>(src + off2);
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) x1[u].v[e] = x2[u].v[e] = E::from_f(0.f);
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int sl = s0 + u * pp.parts;
      if (sl >= nq + nk) break;  // (uniform over the warp)
      const bool isq = sl < nq;
      const int head = (isq ? sl : sl - nq) * kHeads + gi;
      float f1[VEC], f2[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) f1[e] = E::to_f(x1[u].v[e]), f2[e] = E::to_f(x2[u].v[e]);
      if (isq ? p.qw != nullptr : p.kw != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss = fmaf(f1[e], f1[e], fmaf(f2[e], f2[e], ss));
#pragma unroll
        for (int o = LP / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = rsqrtf(ss / (float)D + p.eps);
        const V& a1 = isq ? qw1 : kw1;
        const V& a2 = isq ? qw2 : kw2;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          f1[e] = f1[e] * inv * E::to_f(a1.v[e]);
          f2[e] = f2[e] * inv * E::to_f(a2.v[e]);
        }
      }
      V y1, y2;
      if (p.cos && !inter) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float a, c;
          rotate_pair(f1[e], f2[e], E::to_f(cv.v[e]), E::to_f(sv.v[e]), a, c);
          y1.v[e] = E::from_f(a);
          y2.v[e] = E::from_f(c);
        }
      } else if (p.cos) {
        // pairs (2e, 2e + 1) of the 2 VEC neighbours
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float* f = e < VEC / 2 ? f1 : f2;
          V& y = e < VEC / 2 ? y1 : y2;
          const int o = 2 * (e % (VEC / 2));
          float a, c;
          rotate_pair(f[o], f[o + 1], E::to_f(cv.v[e]), E::to_f(sv.v[e]), a, c);
          y.v[o] = E::from_f(a);
          y.v[o + 1] = E::from_f(c);
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) y1.v[e] = E::from_f(f1[e]), y2.v[e] = E::from_f(f2[e]);
      }
      if (act && head < (isq ? p.H : p.Hkv) && (isq || pg >= 0)) {
        T* dst = isq ? qout + (size_t)head * D : kp + paged::pool_row(p.v, p.Hkv, pg, head, slot) * D;
        *reinterpret_cast<V*>(dst + off1) = y1;
        *reinterpret_cast<V*>(dst + off2) = y2;
      }
    }
  }
  if (pg < 0) return;
  // the value rows, 16 bytes a lane
  const int nvec = p.Hkv * D / 8;
  for (int i0 = part * 32 + lane; i0 < nvec; i0 += 2 * 32 * pp.parts) {
    const int i1 = i0 + 32 * pp.parts;
    V8 a, c;
    a = *reinterpret_cast<const V8*>(vrow + (size_t)i0 * 8);
    if (i1 < nvec) c = *reinterpret_cast<const V8*>(vrow + (size_t)i1 * 8);
    {
      const int head = i0 * 8 / D;
      *reinterpret_cast<V8*>(vp + paged::pool_row(p.v, p.Hkv, pg, head, slot) * D + (i0 * 8 - head * D)) = a;
    }
    if (i1 < nvec) {
      const int head = i1 * 8 / D;
      *reinterpret_cast<V8*>(vp + paged::pool_row(p.v, p.Hkv, pg, head, slot) * D + (i1 * 8 - head * D)) = c;
    }
  }
}

template <typename T, int VEC, int LP>
cudaError_t launch_lp(const AppendArgs& a, int num_sms) {
  constexpr int kHeads = 32 / LP;
  const int slices = (a.H + kHeads - 1) / kHeads + (a.Hkv + kHeads - 1) / kHeads;
  // enough warps to keep every SM loading (16 each), at least one batch of
  // slices a warp
  const long long want = 16ll * num_sms;
  long long parts = (want + a.v.T - 1) / a.v.T;
  parts = std::max(1ll, std::min<long long>(parts, (slices + kBatch - 1) / kBatch));
  AppendParams p{a, (int)parts};
  const long long warps = (long long)a.v.T * parts;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((warps + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_append_kernel<T, VEC, LP>, p);
}

template <typename T>
cudaError_t launch_t(const AppendArgs& a) {
  const int sms = device_sm_count(), half = a.D / 2;
  if (half % 8 == 0) {
    const int n = half / 8;
    if (n <= 4) return launch_lp<T, 8, 4>(a, sms);
    if (n <= 8) return launch_lp<T, 8, 8>(a, sms);
    return launch_lp<T, 8, 16>(a, sms);
  }
  const int n = half / 4;
  if (n <= 8) return launch_lp<T, 4, 8>(a, sms);
  return launch_lp<T, 4, 32>(a, sms);
}

}  // namespace

cudaError_t launch_paged_append(const AppendArgs& a) {
  return a.dtype == GQA_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a) : launch_t<__half>(a);
}

}  // namespace gqa
