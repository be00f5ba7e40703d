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
// slices of a batch are loaded together before any is computed.  The products
// of norm weights with cos and sin are taken once per token, not per head, and
// the arithmetic runs two fp32 lanes an instruction: 23 instructions an
// element (from element-wise code) had cost more time than the memory.
//
// Measured with norms, rotation and 32 + 2 x 8 heads of 128: 4 x 2048 tokens
// 37.7 us, 5.4 TB/s (a copy reaches 6.8); one token of each of 16 sequences
// 4.3 us, which is the launch and the chain of dependent loads (lists, then page
// and rotation, then nothing but stores).
#include <algorithm>

#include "paged.cuh"

namespace gqa {
namespace {

using paged::Seq;

constexpr int kWarps = 4;
constexpr int kBatch = 4;         // slices in flight per warp
constexpr int kBlocks = 5;        // resident CTAs an SM: at most 96 registers a thread
constexpr int kWarpsPerSm = 16;   // warps aimed at when there are few tokens

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

// The two members of the pairs that a lane holds, two pairs a float2: from
// the vectors of the halves, or of neighbouring elements (interleaved).
template <typename T, int VEC, bool kInter>
__device__ __forceinline__ void split(const VecT<T, VEC>& a, const VecT<T, VEC>& b, float2 (&x1)[VEC / 2],
                                      float2 (&x2)[VEC / 2]) {
  using E = Elem<T>;
  const uint32_t* wa = reinterpret_cast<const uint32_t*>(&a);
  const uint32_t* wb = reinterpret_cast<const uint32_t*>(&b);
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) {
    if constexpr (kInter) {
      const float2 u = E::unpack2(2 * j < VEC / 2 ? wa[2 * j] : wb[2 * j - VEC / 2]);
      const float2 v = E::unpack2(2 * j + 1 < VEC / 2 ? wa[2 * j + 1] : wb[2 * j + 1 - VEC / 2]);
      x1[j] = make_float2(u.x, v.x);
      x2[j] = make_float2(u.y, v.y);
    } else {
      x1[j] = E::unpack2(wa[j]);
      x2[j] = E::unpack2(wb[j]);
    }
  }
}
template <typename T, int VEC, bool kInter>
__device__ __forceinline__ void join(const float2 (&y1)[VEC / 2], const float2 (&y2)[VEC / 2], VecT<T, VEC>& a,
                                     VecT<T, VEC>& b) {
  using E = Elem<T>;
  uint32_t* wa = reinterpret_cast<uint32_t*>(&a);
  uint32_t* wb = reinterpret_cast<uint32_t*>(&b);
#pragma unroll
  for (int j = 0; j < VEC / 2; ++j) {
    if constexpr (kInter) {
      (2 * j < VEC / 2 ? wa[2 * j] : wb[2 * j - VEC / 2]) = E::pack2(y1[j].x, y2[j].x);
      (2 * j + 1 < VEC / 2 ? wa[2 * j + 1] : wb[2 * j + 1 - VEC / 2]) = E::pack2(y1[j].y, y2[j].y);
    } else {
      wa[j] = E::pack2(y1[j].x, y1[j].y);
      wb[j] = E::pack2(y2[j].x, y2[j].y);
    }
  }
}

template <typename T, int VEC, int LP, bool kInter>
__global__ void __launch_bounds__(kWarps * 32, kBlocks)
    paged_append_kernel(const __grid_constant__ AppendParams pp) {
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
  // the lane's two vectors of a head: pair members (x1, x2), or neighbours
  const int off1 = kInter ? 2 * li * VEC : li * VEC;
  const int off2 = kInter ? off1 + VEC : half + off1;
  V cv, sv;
#pragma unroll
  for (int e = 0; e < VEC; ++e) cv.v[e] = E::from_f(1.f), sv.v[e] = E::from_f(0.f);
  if (act && p.cos) {
    const size_t r = (size_t)pos * half + li * VEC;
    cv = *reinterpret_cast<const V*>(static_cast<const T*>(p.cos) + r);
    sv = *reinterpret_cast<const V*>(static_cast<const T*>(p.sin) + r);
  }

  // the slices part, part + parts, ... of one row of `heads` heads: src to
  // dst, whose heads lie dst_stride elements apart
  auto heads_of = [&](const T* src, int heads, const void* weight, T* dst, size_t dst_stride) {
    const int slices = (heads + kHeads - 1) / kHeads;
    const bool norm = weight != nullptr, rot = p.cos != nullptr;
    // with a norm: y1 = r (a x1 - b x2), y2 = r (c x2 + d x1), r = 1 / rms and
    // a = w1 cos, b = w2 sin, c = w2 cos, d = w1 sin; without: a = cos, b = sin
    float2 ca[VEC / 2], cb[VEC / 2], cc[VEC / 2], cd[VEC / 2];
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
      ca[j] = E::unpack2(reinterpret_cast<const uint32_t*>(&cv)[j]);
      cb[j] = E::unpack2(reinterpret_cast<const uint32_t*>(&sv)[j]);
    }
    if (norm) {
      V w1{}, w2{};
      if (act) {
        w1 = *reinterpret_cast<const V*>(static_cast<const T*>(weight) + off1);
        w2 = *reinterpret_cast<const V*>(static_cast<const T*>(weight) + off2);
      }
      float2 f1[VEC / 2], f2[VEC / 2];
      split<T, VEC, kInter>(w1, w2, f1, f2);
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) {
        const float2 c = ca[j], sn = cb[j];
        ca[j] = mul2(f1[j], c);
        cb[j] = mul2(f2[j], make_float2(-sn.x, -sn.y));
        cc[j] = mul2(f2[j], c);
        cd[j] = mul2(f1[j], sn);
      }
    }
    for (int s0 = part; s0 < slices; s0 += kBatch * pp.parts) {
      V x1[kBatch], x2[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int head = (s0 + u * pp.parts) * kHeads + gi;
        x1[u] = V{};
        x2[u] = V{};
        if (act && head < heads) {
          x1[u] = *reinterpret_cast<const V*>(src + (size_t)head * D + off1);
          x2[u] = *reinterpret_cast<const V*>(src + (size_t)head * D + off2);
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (s0 + u * pp.parts >= slices) break;  // (uniform over the warp)
        const int head = (s0 + u * pp.parts) * kHeads + gi;
        if (norm || rot) {
          float2 f1[VEC / 2], f2[VEC / 2];
          split<T, VEC, kInter>(x1[u], x2[u], f1, f2);
          if (norm) {
            float2 q = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) q = fma2(f1[j], f1[j], fma2(f2[j], f2[j], q));
            float ss = q.x + q.y;
#pragma unroll
            for (int o = LP / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float r = rsqrtf(ss / (float)D + p.eps);
            const float2 r2 = make_float2(r, r);
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
              const float2 y1 = mul2(fma2(f2[j], cb[j], mul2(f1[j], ca[j])), r2);
              f2[j] = mul2(fma2(f1[j], cd[j], mul2(f2[j], cc[j])), r2);
              f1[j] = y1;
            }
          } else {
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
              float2 y1, y2;
              rotate_pair2(f1[j], f2[j], ca[j], cb[j], y1, y2);
              f1[j] = y1;
              f2[j] = y2;
            }
          }
          join<T, VEC, kInter>(f1, f2, x1[u], x2[u]);
        }
        if (act && head < heads) {
          *reinterpret_cast<V*>(dst + head * dst_stride + off1) = x1[u];
          *reinterpret_cast<V*>(dst + head * dst_stride + off2) = x2[u];
        }
      }
    }
  };
  if (pg >= 0) {
    const size_t row0 = paged::pool_row(p.v, p.Hkv, pg, 0, slot) * D, stride = (size_t)D << p.v.page_log2;
    heads_of(static_cast<const T*>(p.k) + (size_t)t * p.kv_stride, p.Hkv, p.kw, static_cast<T*>(p.k_pages) + row0,
             stride);
    // the value rows, 16 bytes a lane
    const T* vrow = static_cast<const T*>(p.value) + (size_t)t * p.kv_stride;
    T* vp = static_cast<T*>(p.v_pages) + row0;
    const int nvec = p.Hkv * D / 8;
    for (int i0 = part * 32 + lane; i0 < nvec; i0 += kBatch * 32 * pp.parts) {
      V8 x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * 32 * pp.parts;
        if (i < nvec) x[u] = *reinterpret_cast<const V8*>(vrow + (size_t)i * 8);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * 32 * pp.parts;
        if (i < nvec) {
          const int head = i * 8 / D;
          *reinterpret_cast<V8*>(vp + head * stride + (i * 8 - head * D)) = x[u];
        }
      }
    }
  }
  heads_of(static_cast<const T*>(p.q) + (size_t)t * p.q_stride, p.H, p.qw, static_cast<T*>(p.q_out) + (size_t)t * p.H * D,
           D);
}

template <typename T, int VEC, int LP>
cudaError_t launch_lp(const AppendArgs& a, int num_sms) {
  constexpr int kHeads = 32 / LP;
  const int slices = (a.H + kHeads - 1) / kHeads + (a.Hkv + kHeads - 1) / kHeads;
  // enough warps to keep every SM loading, at least one slice a warp (16 single
  // tokens 4.3 us; at least a batch of slices a warp: 5.1)
  const long long want = (long long)kWarpsPerSm * num_sms;
  long long parts = (want + a.v.T - 1) / a.v.T;
  parts = std::max(1ll, std::min<long long>(parts, slices));
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
  return a.interleaved ? cudaLaunchKernelEx(&cfg, paged_append_kernel<T, VEC, LP, true>, p)
                       : cudaLaunchKernelEx(&cfg, paged_append_kernel<T, VEC, LP, false>, p);
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
