// Attention of a few new tokens per sequence over a paged cache (one token
// of a decode step, or a few drafted ones): split-KV with dynamic chunks and
// the split combine inside the kernel, head size D of 64 or 128.
//
//   s_j = scale q.k_j,  p_j = 2^(s_j log2 e - m),  o = sum p_j v_j / sum p_j
//
// Bound by memory: each visible K and V row is read once for all the rows of
// its KV head (G query heads times the sequence's new tokens, at most
// kPagedDecodeColumns), so the kernel is built around the stream of tiles.
// The keys of every (sequence, KV head) item are cut into tiles (64 keys, or
// 128 with D = 64: 16 KB of K and of V) and those into chunks that a persistent grid takes by ticket (decode_sched.cuh:
// about one chunk a CTA for short calls, two for long ones, so that CTAs that
// the memory system serves faster take more).
//
// Inside a CTA warp 4, the producer, takes chunks, hands the consumers a
// descriptor with the chunk's query rows, and streams K and V tiles into a
// ring of stages by bulk-tensor copies with 128-byte swizzle: one box per page
// (or per tile's rows of a larger page), addressed through the block table, whose
// entries the warp keeps 32 at a time in registers, one batch ahead.  Boxes of
// pages that hold no visible slot are aimed beyond the pool, where the copy
// fills zeros.  Warps 0..3 each own a quarter of every tile's keys and run
// S^T = K Q^T and O^T += V^T P^T with mma.sync m16n8k16: the keys are the 16
// rows, the (token, head) pairs the 8-wide columns (NT tiles of them), so
// that one loaded tile serves all columns and no row is padding.  Warp 5
// merges the partials of items that were cut (epoch-tagged arrival counters),
// off the consumers' path.
//
// Measured (a copy reaches 6.8 TB/s): 8 sequences of 16 to 32 thousand tokens, 64
// heads on 8 of 128, 121 us, 6.4 TB/s; 16 sequences of up to 4096, 32 on 8
// heads, 25.0 us, 5.2 TB/s (5.5 us are start, first tiles and the last merges);
// 32 sequences of up to 6000 with 2 to 6 tokens each, 32 on 8 heads of 64, 48.5
// us, 3.9 TB/s: four warps a CTA work on 24 columns there and wait on their own
// chains (23% of the issue slots and 16% of the tensor pipe are taken).
//
// Rounding: scores, softmax statistics and O are fp32; P is rounded to T for
// its product with V, and for items of at most 256 keys its rounding residue
// is added as a second product (there a few keys can carry all the weight).
#include <algorithm>
#include <type_traits>

#include "decode_sched.cuh"
#include "paged.cuh"

namespace gqa {
namespace {

using namespace dsched;
using paged::Seq;

constexpr int kCW = 4;                    // consumer warps
constexpr int kThreads = (kCW + 2) * 32;  // consumers, producer, merger
constexpr int kProducer = kCW, kMerger = kCW + 1;
constexpr int kSlots = 2;                 // descriptor slots
constexpr int kMail = 4;
constexpr int kSeqCache = 128;            // sequences whose lengths are kept in shared memory
constexpr int kPrefetchTiles = 4;         // tiles asked of L2 before the previous kernel has ended
constexpr int kMergeBatch = 5;            // partials loaded per round of a merge
constexpr float kRescaleThresh = 8.0f;    // log2 units

template <int D, int NT>
struct Cfg {
  static constexpr int kTile = 8192 / D;              // keys per stage: 16 KB of K and of V
  static constexpr int kWB = kTile / kCW / 16;        // blocks of 16 keys per consumer warp and stage
  static constexpr int kHalves = D / 64;
  static constexpr int kBoxBytes = kTile * 128;       // a stage's keys x 64 dimensions
  static constexpr int kTileBytes = kHalves * kBoxBytes;
  static constexpr int kStageBytes = 2 * kTileBytes;
  // two CTAs an SM unless the accumulators (NT * D / 4 registers a thread) forbid it
  static constexpr int kCtas = NT * D <= 256 ? 2 : 1;
  static constexpr int kStages = kCtas == 2 ? 3 : 5;
  static constexpr int kQRow = D * 2;
  static constexpr int kSlotBytes = 64 + 8 * NT * kQRow;
  static constexpr int kHandFloats = NT * ((D / 16) * 128 + 128);  // one warp's O^T fragments and (m, l) pairs
  // the warps' states merge through an area of their own where there is room
  // for it, else through the stage of the chunk's last tile
  static constexpr bool kMergeInStage = kCtas == 2 && NT * D > 128;
  static constexpr bool kMergePairs = !kMergeInStage || 2 * kHandFloats * 4 <= kStageBytes;  // two states at a time
  static_assert(!kMergeInStage || kHandFloats * 4 <= kStageBytes, "merge area in a stage");
  static constexpr int kMergeOff = kStages * kStageBytes;
  static constexpr int kSlotOff = kMergeOff + (kMergeInStage ? 0 : 2 * kHandFloats * 4);
  static constexpr int kSeqOff = kSlotOff + kSlots * kSlotBytes;
  static constexpr int kBadOff = kSeqOff + (2 * kSeqCache + 1) * 4;  // [2] chunks in turn: values were taken out
  static constexpr int kMailOff = (kBadOff + 8 + 15) / 16 * 16;
  static constexpr int kBarOff = kMailOff + kMail * 16;
  static constexpr int kSmem = kBarOff + (2 * kStages + 2 * kSlots + 2 * kMail) * 8 + 1024;
  static_assert(kCtas * (kSmem + 1024) <= 233472, "shared memory of one SM");
};

struct DecParams {
  PagedView v;
  const void* q;
  const void* k_pages;
  const void* v_pages;
  void* out;
  float* lse;      // nullptr: not wanted
  float* part_o;   // [slots][columns][D]
  float* part_ml;  // [slots][columns][2]
  unsigned long long* ticket;
  unsigned long long* arrivals;
  int H, Hkv, G, window, P, chunks_per_cta, columns, pool_rows;
  uint32_t epoch;
  float scale_log2;
};

// Byte offset of 16-byte chunk c of key row r in a tile of D dimensions.
template <int D>
__device__ __forceinline__ uint32_t sw_off(int r, int c) {
  return (uint32_t)((c >> 3) * Cfg<D, 1>::kBoxBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// The tiles of a checked sequence: its visible keys are [lo, L), its tiles
// start at multiples of kTile.
template <int kTile>
__device__ __forceinline__ int tiles_of(const Seq& s, bool any, int window, int& lo, int& L) {
  lo = L = 0;
  if (!any) return 0;
  lo = paged::first_visible(s.past, window);
  L = s.L;
  return (L + kTile - 1) / kTile - lo / kTile;
}

// The batch as the partition sees it; past / cu in shared memory for small
// batches, else the arrays themselves.
template <int kTile>
struct PagedSrc {
  const PagedView& v;
  const int* past;
  const int* cu;
  int window, B, Hkv, P, chunks_per_cta;
  __device__ PagedSrc(const DecParams& p, const int* past_, const int* cu_)
      : v(p.v), past(past_), cu(cu_), window(p.window), B(p.v.B), Hkv(p.Hkv), P(p.P),
        chunks_per_cta(p.chunks_per_cta) {}
  __device__ __forceinline__ int tiles(int b, int& lo, int& L) const {
    Seq s;
    int code;
    const bool any = paged::check_seq(v, past[b], cu[b], cu[b + 1], s, code);
    return tiles_of<kTile>(s, any, window, lo, L);
  }
};

// The state of one consumer warp over a chunk.
template <typename T, int D, int NT>
struct Acc {
  using E = Elem<T>;
  static constexpr bool kBF16 = E::is_bf16;
  static constexpr int kD16 = D / 16;
  static constexpr int kWB = Cfg<D, NT>::kWB;  // blocks of 16 keys per tile
  static constexpr int kWK = 16 * kWB;         // keys per tile

  float o[NT][kD16][4];      // O^T fragments: dimensions x columns
  float mh[NT][2], lh[NT][2];
  uint32_t qb[NT][kD16][2];  // query fragments
  int lim[NT][2];            // the thread's columns see keys < lim ...
  int low[NT][2];            // ... and >= low

  __device__ __forceinline__ void begin(uint32_t q_smem, int lane, int G, int past, int n, int window) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint32_t qrow = q_smem + (8 * nt + (lane & 7)) * (D * 2);
#pragma unroll
      for (int j = 0; j < kD16 / 2; ++j)
        ldsm_x4(qrow + (4 * j + (lane >> 3)) * 16, qb[nt][2 * j][0], qb[nt][2 * j][1], qb[nt][2 * j + 1][0],
                qb[nt][2 * j + 1][1]);
#pragma unroll
      for (int i = 0; i < kD16; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mh[nt][e] = -INFINITY;
        lh[nt][e] = 0.f;
        const int pos = past + min((8 * nt + 2 * (lane & 3) + e) / G, n - 1);
        lim[nt][e] = pos + 1;
        low[nt][e] = paged::first_visible(pos, window);
      }
    }
  }

  // Value rows of keys outside [lo, L) are zeroed, so that P = 0 meets finite
  // values.  Returns whether this warp wrote the tile.
  __device__ __forceinline__ bool clear(uint8_t* vt, int warp, int lane, int tk0, int lo, int L) const {
    const int w0 = tk0 + warp * kWK;
    if (w0 >= lo && w0 + kWK <= L) return false;
    for (int idx = lane; idx < kWK * (D / 8); idx += 32) {
      const int r = idx / (D / 8), c = idx % (D / 8);
      if (w0 + r < lo || w0 + r >= L)
        *reinterpret_cast<uint4*>(vt + sw_off<D>(warp * kWK + r, c)) = make_uint4(0, 0, 0, 0);
    }
    __syncwarp();
    return true;
  }

  // Keys that some new tokens see and others do not (past `past` or before
  // `all_lo`): a value row among them that is not finite must not meet the
  // others' P = 0 as NaN.  Its infinities and NaN leave the tile here; the
  // outputs that see them are corrected when they are written.
  __device__ __forceinline__ bool sanitize(uint8_t* vt, int warp, int lane, int tk0, int past, int all_lo) const {
    bool found = false;
#pragma unroll 1
    for (int idx = lane; idx < kWK * (D / 8); idx += 32) {
      const int r = idx / (D / 8), c = idx % (D / 8), key = tk0 + warp * kWK + r;
      if (key <= past && key >= all_lo) continue;
      uint4* at = reinterpret_cast<uint4*>(vt + sw_off<D>(warp * kWK + r, c));
      if (paged::nonfinite<T>(*at)) {
        *at = paged::finite_only<T>(*at);
        found = true;
      }
    }
    return __any_sync(0xffffffffu, found);
  }

  // kMask: some column does not see some key of the tile.
  template <bool kMask, bool kSplit>
  __device__ __forceinline__ void tile(uint32_t kst, uint32_t vst, int warp, int lane, int tk0, float scale_log2) {
    const int gq = lane >> 2, wr0 = warp * kWK, mi = lane >> 3;
    float sc[kWB][NT][4];
#pragma unroll
    for (int w = 0; w < kWB; ++w) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) sc[w][nt][0] = sc[w][nt][1] = sc[w][nt][2] = sc[w][nt][3] = 0.f;
      const int kr = wr0 + 16 * w + ((mi & 1) << 3) + (lane & 7);
#pragma unroll
      for (int ks = 0; ks < kD16; ++ks) {
        uint32_t a[4];
        ldsm_x4(kst + sw_off<D>(kr, 2 * ks + (mi >> 1)), a[0], a[1], a[2], a[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_16816<kBF16>(sc[w][nt], a, qb[nt][ks][0], qb[nt][ks][1]);
      }
    }
    const int key0 = tk0 + wr0 + gq;  // the thread's keys of block w: key0 + 16 w, and 8 on
    float mx[NT][2];                  // the thread's largest score of each column
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      mx[nt][0] = mx[nt][1] = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWB; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = sc[w][nt][e] * scale_log2;
          const int key = key0 + 16 * w + (e >> 1) * 8;
          sc[w][nt][e] = !kMask || (key < lim[nt][e & 1] && key >= low[nt][e & 1]) ? v : -INFINITY;
          mx[nt][e & 1] = fmaxf(mx[nt][e & 1], sc[w][nt][e]);
        }
    }
    // the reference of each column's exponents moves only when a score passes
    // it by more than 2^8 (P then stays below 2^8): mostly one vote per tile
    bool grows = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) grows |= mx[nt][e] > mh[nt][e] + kRescaleThresh;
    if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float m = mx[nt][e];
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
          const float mn = fmaxf(mh[nt][e], m);
          const float corr = fast_exp2(mh[nt][e] - (mn == -INFINITY ? 0.f : mn));
          mh[nt][e] = mn;
          lh[nt][e] *= corr;
#pragma unroll
          for (int md = 0; md < kD16; ++md) {
            o[nt][md][e] *= corr;
            o[nt][md][e + 2] *= corr;
          }
        }
    }
    uint32_t bh[kWB][NT][2], bl[kWB][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float m[2] = {mh[nt][0] == -INFINITY ? 0.f : mh[nt][0], mh[nt][1] == -INFINITY ? 0.f : mh[nt][1]};
#pragma unroll
      for (int w = 0; w < kWB; ++w) {
        float* x = sc[w][nt];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = fast_exp2(x[e] - m[e & 1]);
        lh[nt][0] += x[0] + x[2];
        lh[nt][1] += x[1] + x[3];
        const uint32_t h0 = E::pack2(x[0], x[1]);
        const uint32_t h1 = E::pack2(x[2], x[3]);
        bh[w][nt][0] = movmatrix_trans(h0);
        bh[w][nt][1] = movmatrix_trans(h1);
        if (kSplit) {
          const float2 f0 = E::unpack2(h0), f1 = E::unpack2(h1);
          bl[w][nt][0] = movmatrix_trans(E::pack2(x[0] - f0.x, x[1] - f0.y));
          bl[w][nt][1] = movmatrix_trans(E::pack2(x[2] - f1.x, x[3] - f1.y));
        }
      }
    }
#pragma unroll
    for (int w = 0; w < kWB; ++w) {
      const int vr = wr0 + 16 * w + ((mi >> 1) << 3) + (lane & 7);
#pragma unroll
      for (int md = 0; md < kD16; ++md) {
        uint32_t a[4];
        ldsm_x4_t(vst + sw_off<D>(vr, 2 * md + (mi & 1)), a[0], a[1], a[2], a[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_16816<kBF16>(o[nt][md], a, bh[w][nt][0], bh[w][nt][1]);
          if (kSplit) mma_16816<kBF16>(o[nt][md], a, bl[w][nt][0], bl[w][nt][1]);
        }
      }
    }
  }

  __device__ __forceinline__ void reduce_sums() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = lh[nt][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        lh[nt][e] = l;
      }
  }

  __device__ __forceinline__ void hand_off(float* dst, int lane) const {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int md = 0; md < kD16; ++md)
        *reinterpret_cast<float4*>(dst + ((nt * kD16 + md) * 32 + lane) * 4) =
            make_float4(o[nt][md][0], o[nt][md][1], o[nt][md][2], o[nt][md][3]);
      *reinterpret_cast<float4*>(dst + NT * kD16 * 128 + (nt * 32 + lane) * 4) =
          make_float4(mh[nt][0], lh[nt][0], mh[nt][1], lh[nt][1]);
    }
  }

  // (o, m, l) merged with another warp's: m* = max(m, m2), the rest scaled to it
  __device__ __forceinline__ void absorb(const float* src, int lane) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float4 ml = *reinterpret_cast<const float4*>(src + NT * kD16 * 128 + (nt * 32 + lane) * 4);
      float f1[2], f2[2];
      const float m2[2] = {ml.x, ml.z}, l2[2] = {ml.y, ml.w};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ms = fmaxf(mh[nt][e], m2[e]);
        const float su = ms == -INFINITY ? 0.f : ms;
        f1[e] = fast_exp2(mh[nt][e] - su);
        f2[e] = fast_exp2(m2[e] - su);
        lh[nt][e] = lh[nt][e] * f1[e] + l2[e] * f2[e];
        mh[nt][e] = ms;
      }
#pragma unroll
      for (int md = 0; md < kD16; ++md) {
        const float4 a = *reinterpret_cast<const float4*>(src + ((nt * kD16 + md) * 32 + lane) * 4);
        o[nt][md][0] = o[nt][md][0] * f1[0] + a.x * f2[0];
        o[nt][md][1] = o[nt][md][1] * f1[1] + a.y * f2[1];
        o[nt][md][2] = o[nt][md][2] * f1[0] + a.z * f2[0];
        o[nt][md][3] = o[nt][md][3] * f1[1] + a.w * f2[1];
      }
    }
  }

  // The four consumer warps' states into warp 0's, through one or two hand-off areas.
  template <bool kPairs>
  __device__ __forceinline__ void merge_warps(float* mw, int floats, int warp, int lane) {
    if (!kPairs) {
#pragma unroll
      for (int w = 1; w < kCW; ++w) {
        if (warp == w) hand_off(mw, lane);
        named_bar_sync(1, kCW * 32);
        if (warp == 0) absorb(mw, lane);
        if (w + 1 < kCW) named_bar_sync(1, kCW * 32);
      }
      return;
    }
    if (warp >= 2) hand_off(mw + (warp - 2) * floats, lane);
    named_bar_sync(1, kCW * 32);
    if (warp < 2) absorb(mw + warp * floats, lane);
    named_bar_sync(1, kCW * 32);
    if (warp == 1) hand_off(mw, lane);
    named_bar_sync(1, kCW * 32);
    if (warp == 0) absorb(mw, lane);
  }

  // Warp 0: the output rows (and lse) of the item's R columns; column r is
  // token r / G, head r % G; out and lse at the item's first row and head.
  __device__ __forceinline__ void store_output(T* out, float* lse, int R, int G, int H, int lane) const {
    const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nt + 2 * tq + e;
        if (r >= R) continue;
        const size_t row = (size_t)(r / G) * H + r % G;
        const float inv = 1.f / lh[nt][e];
        T* dst = out + row * D;
#pragma unroll
        for (int md = 0; md < kD16; ++md) {
          dst[16 * md + gq] = E::from_f(o[nt][md][e] * inv);
          dst[16 * md + gq + 8] = E::from_f(o[nt][md][e + 2] * inv);
        }
        if (lse && gq == 0) lse[row] = mh[nt][e] * kLn2 + logf(lh[nt][e]);
      }
  }

  // Warp 0: the fp32 partial, o into po [columns][D], (m, l) into pm [columns][2].
  // (a negative sum: values were taken out)
  __device__ __forceinline__ void store_partial(float* po, float* pm, int R, int lane, bool corrected) const {
    const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * nt + 2 * tq + e;
        if (r >= R) continue;
#pragma unroll
        for (int md = 0; md < kD16; ++md) {
          po[(size_t)r * D + 16 * md + gq] = o[nt][md][e];
          po[(size_t)r * D + 16 * md + gq + 8] = o[nt][md][e + 2];
        }
        if (gq == 0) *reinterpret_cast<float2*>(pm + 2 * r) = make_float2(mh[nt][e], corrected ? -lh[nt][e] : lh[nt][e]);
      }
  }
};

// (whole warp) adds to the item's outputs, which are stored, the infinities and
// NaN of the value rows that a new token of sequence b sees and others of its n
// do not.
template <typename T, int D>
__device__ __noinline__ void correct_rows(const DecParams& p, int b, int kh, int q0, int past, int n, int lane) {
  using E = Elem<T>;
  const int32_t* tab = p.v.table + (size_t)b * p.v.max_pages;
  const int all_lo = paged::first_visible(past + n - 1, p.window);
  __syncwarp();  // (the rows were stored by other lanes)
  for (int i = 0; i < n; ++i) {
    const int pos = past + i;
    for (int key = paged::first_visible(pos, p.window); key <= pos; ++key) {
      if (key >= all_lo && key <= past) {
        key = past;  // (seen by all: never taken out)
        continue;
      }
      const int pg = tab[key >> p.v.page_log2];
      if ((unsigned)pg >= (unsigned)p.v.num_pages) continue;
      const T* v = static_cast<const T*>(p.v_pages) + paged::pool_row(p.v, p.Hkv, pg, kh, key) * D;
      for (int d = lane; d < D; d += 32) {
        const float x = E::to_f(v[d]);
        if (isfinite(x)) continue;
        for (int g = 0; g < p.G; ++g) {
          T* o = static_cast<T*>(p.out) + ((size_t)(q0 + i) * p.H + kh * p.G + g) * D + d;
          *o = E::from_f(E::to_f(*o) + x);
        }
      }
    }
  }
}

// The chunk descriptor's spare words
enum { kPadRow = 0, kPadNew = 1 };  // the sequence's first row, its new tokens

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::kCtas)
    paged_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const __grid_constant__ DecParams p) {
  using E = Elem<T>;
  using C = Cfg<D, NT>;
  constexpr int kTile = C::kTile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar_full = sbase + C::kBarOff;
  const uint32_t bar_empty = bar_full + C::kStages * 8;
  const uint32_t bar_dfull = bar_empty + C::kStages * 8;
  const uint32_t bar_dempty = bar_dfull + kSlots * 8;
  const uint32_t bar_mfull = bar_dempty + kSlots * 8;
  const uint32_t bar_mempty = bar_mfull + kMail * 8;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x, G = p.G;

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(bar_full + 8 * i, 1);
      mbar_init(bar_empty + 8 * i, kCW);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(bar_dfull + 8 * i, 1);
      mbar_init(bar_dempty + 8 * i, kCW);
    }
    for (int i = 0; i < kMail; ++i) {
      mbar_init(bar_mfull + 8 * i, 1);
      mbar_init(bar_mempty + 8 * i, 1);
    }
    fence_mbar_init();
    reinterpret_cast<int*>(smem + C::kBadOff)[0] = reinterpret_cast<int*>(smem + C::kBadOff)[1] = 0;
  }
  if (warp == kProducer && lane == 0) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  __syncthreads();
  pdl_launch_dependents();

  if (warp == kProducer) {
    // ---------------- producer ----------------
    const int plog = p.v.page_log2, page = 1 << plog;
    const int rows = min(page, kTile);   // rows of one box
    const int nsub = kTile / rows;       // boxes per tile and 64-dimension half
    // While the previous kernel may still run: a speculative look at the
    // lists of a small batch (through L2) gives the partition and this CTA's
    // first chunk, whose query rows and first tiles are asked of L2 (a
    // prefetch reads nothing into registers that is used later).  It is kept
    // if the lists are the same after the wait.
    int s_past = 0, s_q0 = 0, s_q1 = 0;
    Partition pt{};
    ChunkDesc first{};
    first.u = -1;
    const bool small = p.v.B <= 32;
    auto locate_small = [&]() {
      Seq s;
      int code = 0, lo = 0, L = 0;
      const bool any = lane < p.v.B && paged::check_seq(p.v, s_past, s_q0, s_q1, s, code);
      const int tb = tiles_of<kTile>(s, any, p.window, lo, L);
      first = partition_and_locate_small(PagedSrc<kTile>(p, nullptr, nullptr), tb, lo, L, c, lane, pt);
    };
    auto read_small = [&](int& past, int& q0, int& q1) {
      past = lane < p.v.B ? __ldcg(p.v.seqlens + lane) : 0;
      q0 = lane < p.v.B ? __ldcg(p.v.cu + lane) : 0;
      q1 = lane < p.v.B ? __ldcg(p.v.cu + lane + 1) : 0;
    };
    if (small) {
      read_small(s_past, s_q0, s_q1);
      locate_small();
      if (first.u >= 0) {
        const ChunkDesc& d = first;
        const int tile0 = d.klo / kTile + d.t0;
        const int nt = min(d.t1 - d.t0, kPrefetchTiles);
        if (lane < nt * nsub) {
          const int s = tile0 * kTile + lane * rows;
          if (s < d.L && s + rows > d.klo) {
            const int pg = __ldcg(p.v.table + (size_t)d.b * p.v.max_pages + (s >> plog));
            if ((unsigned)pg < (unsigned)p.v.num_pages) {
              const size_t off = paged::pool_row(p.v, p.Hkv, pg, d.kh, s) * D;
              bulk_prefetch_l2(static_cast<const T*>(p.k_pages) + off, rows * D * 2);
              bulk_prefetch_l2(static_cast<const T*>(p.v_pages) + off, rows * D * 2);
            }
          }
        }
        const int q0 = __shfl_sync(0xffffffffu, s_q0, d.b), q1 = __shfl_sync(0xffffffffu, s_q1, d.b);
        if (lane < q1 - q0)
          bulk_prefetch_l2(static_cast<const T*>(p.q) + ((size_t)(q0 + lane) * p.H + d.kh * G) * D, G * D * 2);
      }
    }
    pdl_wait_primary();  // inputs may be written by the previous kernel in the stream

    int* sm_past = reinterpret_cast<int*>(smem + C::kSeqOff);
    int* sm_cu = sm_past + kSeqCache;
    const bool cached = p.v.B <= kSeqCache;
    if (cached) {
      for (int i = lane; i < p.v.B; i += 32) sm_past[i] = __ldcg(p.v.seqlens + i);
      for (int i = lane; i <= p.v.B; i += 32) sm_cu[i] = __ldcg(p.v.cu + i);
    }
    __syncwarp();
    const PagedSrc<kTile> src(p, cached ? sm_past : p.v.seqlens, cached ? sm_cu : p.v.cu);
    if (c == 0)  // sequences that fail the checks are skipped and reported once
      for (int i = lane; i < p.v.B; i += 32) {
        Seq s;
        int code;
        paged::check_seq(p.v, src.past[i], src.cu[i], src.cu[i + 1], s, code);
        if (code) record_error(p.v.err, code);
      }
    if (small) {
      const int past = lane < p.v.B ? sm_past[lane] : 0, q0 = lane < p.v.B ? sm_cu[lane] : 0,
                q1 = lane < p.v.B ? sm_cu[lane + 1] : 0;
      if (!__all_sync(0xffffffffu, past == s_past && q0 == s_q0 && q1 == s_q1)) {
        s_past = past;
        s_q0 = q0;
        s_q1 = q1;
        locate_small();
      }
    } else {
      pt = make_partition(src, lane);
      if (c < pt.U) first = locate_chunk(src, pt, c, lane);
    }

    int u = first.u;
    int gt = 0;  // tiles issued by this CTA
    bool ok = true;
    // (whole warp) the tiles [d.t0, d.t1) of chunk d into the ring
    auto issue_tiles = [&](const ChunkDesc& d) {
      const int32_t* tab = p.v.table + (size_t)d.b * p.v.max_pages;
      const int k0 = (d.klo / kTile + d.t0) * kTile;     // first key of the first tile
      const int k1 = min((d.klo / kTile + d.t1) * kTile, d.L);
      int e0 = k0 >> plog;                                // the register batch holds entries e0 .. e0 + 31
      const int e_end = (k1 - 1) >> plog;
      auto entry = [&](int e) { return e <= e_end ? __ldg(tab + e) : -1; };
      int cur = entry(e0 + lane), nxt = entry(e0 + 32 + lane);
      for (int t = d.t0; t < d.t1; ++t, ++gt) {
        const int st = gt % C::kStages, round = gt / C::kStages;
        if (round > 0) {
          const bool w = mbar_wait(bar_empty + 8 * st, (round - 1) & 1, p.v.err);
          if (!__all_sync(0xffffffffu, w)) {
            ok = false;
            return;
          }
        }
        const uint32_t fb = bar_full + 8 * st;
        if (lane == 0) mbar_arrive_expect_tx(fb, C::kStageBytes);
        const int s = (d.klo / kTile + t) * kTile + min(lane, nsub - 1) * rows;  // first slot of the lane's box
        int e = s >> plog;
        if (__shfl_sync(0xffffffffu, e, 0) >= e0 + 32) {
          cur = nxt;
          e0 += 32;
          nxt = entry(e0 + 32 + lane);
        }
        // (a tile's entries lie in one batch: e0 starts at a tile and 32 is a multiple of nsub)
        int pg = __shfl_sync(0xffffffffu, cur, e - e0);
        int y = p.pool_rows;  // beyond the pool: zeros
        if (lane < nsub && s < d.L && s + rows > d.klo) {
          if ((unsigned)pg < (unsigned)p.v.num_pages)
            y = ((pg * p.Hkv + d.kh) << plog) + (s & (page - 1));
          else
            record_error(p.v.err, GQA_ERR_INVALID_ARGUMENT);
        }
        __syncwarp();
        if (lane < nsub) {
          const uint32_t kd = sbase + st * C::kStageBytes + lane * rows * 128;
          const uint32_t vd = kd + C::kTileBytes;
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h) {
            tma_load_2d(kd + h * C::kBoxBytes, &kmap, h * 64, y, fb);
            tma_load_2d(vd + h * C::kBoxBytes, &vmap, h * 64, y, fb);
          }
        }
      }
    };
    int dk = 0;  // descriptors issued
    bool first_take = true;
    while (true) {
      ChunkDesc d;
      if (dk == 0) {
        d = first;
      } else if (u >= 0) {
        d = locate_chunk(src, pt, u, lane);
      } else {
        d = ChunkDesc{};
        d.u = -1;
      }
      const int ds = dk % kSlots;
      if (dk >= kSlots && !mbar_wait(bar_dempty + 8 * ds, ((dk / kSlots) - 1) & 1, p.v.err)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) d.u = -1;  // a wait ran out: stop the consumers
      uint8_t* slot = smem + C::kSlotOff + ds * C::kSlotBytes;
      const uint32_t fb = bar_dfull + 8 * ds;
      int q0 = 0, n = 0;
      if (d.u >= 0) {
        q0 = src.cu[d.b];
        n = src.cu[d.b + 1] - q0;
      }
      if (lane == 0) {
        d.pad[kPadRow] = q0;
        d.pad[kPadNew] = n;
        *reinterpret_cast<ChunkDesc*>(slot) = d;
        if (d.u >= 0)
          mbar_arrive_expect_tx(fb, (uint32_t)(n * G * D * 2));
        else
          mbar_arrive(fb);  // the terminating descriptor
      }
      __syncwarp();
      if (d.u >= 0 && lane < n)  // (n <= kPagedDecodeColumns)
        bulk_g2s(smem_u32(slot) + 64 + lane * G * D * 2,
                 static_cast<const T*>(p.q) + ((size_t)(q0 + lane) * p.H + d.kh * G) * D, G * D * 2, fb);
      ++dk;
      if (d.u < 0) break;
      issue_tiles(d);
      // the next chunk's ticket (its latency hides behind the tiles queued in
      // the ring); the call's last ticket resets the counter
      int nu = -1;
      if (lane == 0 && ok) {
        if (first_take) epoch_install(p.ticket, p.epoch);
        const uint32_t t = epoch_take(p.ticket, p.epoch, p.v.err);
        if (t != 0xFFFFFFFFu) {
          if ((int)t == pt.U - 1) atomicExch(p.ticket, 0ull);
          nu = p.P + (int)t < pt.U ? p.P + (int)t : -1;
        }
      }
      first_take = false;
      u = __shfl_sync(0xffffffffu, nu, 0);
    }
    // leave no copy in flight into this CTA's shared memory
    if (lane == 0) {
      for (int t = max(0, gt - C::kStages); t < gt; ++t)
        mbar_wait(bar_full + 8 * (t % C::kStages), (t / C::kStages) & 1, p.v.err);
      for (int k = max(0, dk - kSlots); k < dk; ++k)
        mbar_wait(bar_dfull + 8 * (k % kSlots), (k / kSlots) & 1, p.v.err);
    }
    return;
  }

  // (not for data, which the producer's own wait covers: the limits of the waits
  // below leave out what the previous kernel still takes)
  pdl_wait_primary();
  if (warp == kMerger) {
    // ---------------- merger ----------------
    int mk = 0;
    while (true) {
      const int ms = mk % kMail;
      if (!__all_sync(0xffffffffu, mbar_wait(bar_mfull + 8 * ms, (mk / kMail) & 1, p.v.err))) break;
      const int4 mail = *reinterpret_cast<const int4*>(smem + C::kMailOff + ms * 16);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_mempty + 8 * ms);
      ++mk;
      const int first = mail.x, n = mail.y, b = mail.z, kh = mail.w;
      if (first < 0) break;  // the consumers are done
      unsigned long long* arr = p.arrivals + first;
      if (b < 0) {
        // a chunk of the item has started here: its counter holds this call's
        // epoch before this CTA counts itself in
        if (lane == 0) epoch_install(arr, p.epoch);
        continue;
      }
      uint32_t cnt = 0;
      if (lane == 0) {
        // release: the partial is visible before the count; acquire: the last
        // chunk sees the others' partials
        unsigned long long old;
        asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], 1;" : "=l"(old) : "l"(arr) : "memory");
        if ((uint32_t)(old >> 32) != p.epoch) {
          record_error(p.v.err, GQA_ERR_INVALID_ARGUMENT);  // the workspace changed under the call
          cnt = 0xFFFFFFFFu;
        } else {
          cnt = (uint32_t)old;
        }
      }
      cnt = __shfl_sync(0xffffffffu, cnt, 0);
      if (cnt != (uint32_t)(n - 1)) continue;
      // the item's last chunk: merge its n partials.  Heads in rounds of four,
      // partials kMergeBatch at a time with a running max: the loads of a
      // round are independent.  Lane l takes D / 32 dimensions.
      __syncwarp();
      constexpr int kV = D / 32;
      using F = VecT<float, kV>;
      const int q0 = p.v.cu[b], R = (p.v.cu[b + 1] - q0) * G;
      const float* ml0 = p.part_ml + (size_t)first * p.columns * 2;
      const float* po0 = p.part_o + (size_t)first * p.columns * D;
      bool corrected = false;
      for (int r0 = 0; r0 < R; r0 += 4) {
        float mrun[4], l[4], acc[4][kV];
#pragma unroll
        for (int gi = 0; gi < 4; ++gi) {
          mrun[gi] = -INFINITY;
          l[gi] = 0.f;
#pragma unroll
          for (int x = 0; x < kV; ++x) acc[gi][x] = 0.f;
        }
        for (int k0 = 0; k0 < n; k0 += kMergeBatch) {
          F ov[kMergeBatch][4];
          float2 mlv[kMergeBatch][4];
#pragma unroll
          for (int q = 0; q < kMergeBatch; ++q)
#pragma unroll
            for (int gi = 0; gi < 4; ++gi) {
              const int k = k0 + q, r = r0 + gi;
              const bool v = k < n && r < R;
              const size_t at = (size_t)k * p.columns + r;
              if (v) {
                if constexpr (kV == 4) {
                  const float4 x = __ldcg(reinterpret_cast<const float4*>(po0 + at * D) + lane);
                  ov[q][gi].v[0] = x.x, ov[q][gi].v[1] = x.y, ov[q][gi].v[2] = x.z, ov[q][gi].v[3] = x.w;
                } else {
                  const float2 x = __ldcg(reinterpret_cast<const float2*>(po0 + at * D) + lane);
                  ov[q][gi].v[0] = x.x, ov[q][gi].v[1] = x.y;
                }
                mlv[q][gi] = __ldcg(reinterpret_cast<const float2*>(ml0 + at * 2));
              } else {
#pragma unroll
                for (int x = 0; x < kV; ++x) ov[q][gi].v[x] = 0.f;
                mlv[q][gi] = make_float2(-INFINITY, 0.f);
              }
            }
#pragma unroll
          for (int gi = 0; gi < 4; ++gi) {
            float mb = mrun[gi];
#pragma unroll
            for (int q = 0; q < kMergeBatch; ++q) mb = fmaxf(mb, mlv[q][gi].x);
            const float base = mb == -INFINITY ? 0.f : mb;
            const float sc = fast_exp2(mrun[gi] - base);
            mrun[gi] = mb;
            l[gi] *= sc;
#pragma unroll
            for (int x = 0; x < kV; ++x) acc[gi][x] *= sc;
#pragma unroll
            for (int q = 0; q < kMergeBatch; ++q) {
              const float w = fast_exp2(mlv[q][gi].x - base);
              l[gi] += w * fabsf(mlv[q][gi].y);
              corrected |= __float_as_int(mlv[q][gi].y) < 0;
#pragma unroll
              for (int x = 0; x < kV; ++x) acc[gi][x] += w * ov[q][gi].v[x];
            }
          }
        }
#pragma unroll
        for (int gi = 0; gi < 4; ++gi) {
          const int r = r0 + gi;
          if (r >= R) continue;
          const size_t row = (size_t)(q0 + r / G) * p.H + kh * G + r % G;
          const float inv = 1.f / l[gi];
          VecT<uint32_t, kV / 2> packed;
#pragma unroll
          for (int x = 0; x < kV / 2; ++x) packed.v[x] = E::pack2(acc[gi][2 * x] * inv, acc[gi][2 * x + 1] * inv);
          *reinterpret_cast<VecT<uint32_t, kV / 2>*>(static_cast<T*>(p.out) + row * D + lane * kV) = packed;
          if (p.lse && lane == 0) p.lse[row] = mrun[gi] * kLn2 + logf(l[gi]);
        }
      }
      if (__any_sync(0xffffffffu, corrected)) correct_rows<T, D>(p, b, kh, q0, p.v.seqlens[b], R / G, lane);
      if (lane == 0) atomicExch(arr, 0ull);  // ready for the next call
    }
    return;
  }

  // ---------------- consumers (warps 0..3) ----------------
  int gt = 0;  // tiles consumed by this CTA
  int dk = 0;  // descriptors consumed
  int mk = 0;  // mails to the merger (warp 0)
  volatile int* bad = reinterpret_cast<int*>(smem + C::kBadOff);
  auto mail = [&](int x, int y, int z, int w) {
    if (lane == 0) {
      const int ms = mk % kMail;
      if (mk >= kMail) mbar_wait(bar_mempty + 8 * ms, ((mk / kMail) - 1) & 1, p.v.err);
      *reinterpret_cast<int4*>(smem + C::kMailOff + ms * 16) = make_int4(x, y, z, w);
      mbar_arrive(bar_mfull + 8 * ms);
    }
    ++mk;
  };
  while (true) {
    const int ds = dk % kSlots;
    if (!__all_sync(0xffffffffu, mbar_wait(bar_dfull + 8 * ds, (dk / kSlots) & 1, p.v.err))) break;
    const uint8_t* slot = smem + C::kSlotOff + ds * C::kSlotBytes;
    const ChunkDesc d = *reinterpret_cast<const ChunkDesc*>(slot);
    if (d.u < 0) break;
    ++dk;
    if (warp == 0 && d.slot >= 0) mail(d.first_slot, d.n, -1, 0);  // a chunk of this item starts here
    const int n = d.pad[kPadNew], past = d.L - n, R = n * G;
    const bool splitp = d.L - d.klo <= 256;
    Acc<T, D, NT> acc;
    acc.begin(smem_u32(slot) + 64, lane, G, past, n, p.window);
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_dempty + 8 * ds);
    // keys that every column sees: [all_lo, past]
    const int all_lo = paged::first_visible(d.L - 1, p.window);
    bool ok = true;
    for (int t = d.t0; t < d.t1; ++t, ++gt) {
      const int st = gt % C::kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(bar_full + 8 * st, (gt / C::kStages) & 1, p.v.err))) {
        ok = false;
        break;
      }
      const uint32_t kst = sbase + st * C::kStageBytes, vst = kst + C::kTileBytes;
      const int tk0 = (d.klo / kTile + t) * kTile;
      bool touched = acc.clear(smem + (vst - sbase), warp, lane, tk0, d.klo, d.L);
      const bool mask = tk0 < all_lo || tk0 + kTile > past + 1;
      if (mask && n > 1 && acc.sanitize(smem + (vst - sbase), warp, lane, tk0, past, all_lo)) {
        touched = true;
        bad[dk & 1] = 1;
      }
      if (splitp)
        acc.template tile<true, true>(kst, vst, warp, lane, tk0, p.scale_log2);
      else if (mask)
        acc.template tile<true, false>(kst, vst, warp, lane, tk0, p.scale_log2);
      else
        acc.template tile<false, false>(kst, vst, warp, lane, tk0, p.scale_log2);
      __syncwarp();
      if (C::kMergeInStage && t + 1 == d.t1) continue;  // released after the merge
      if (lane == 0) {
        if (touched) fence_proxy_async_smem();  // the next copy into this stage comes after these writes
        mbar_arrive(bar_empty + 8 * st);
      }
    }
    acc.reduce_sums();
    // every warp has left its tiles (and warp 0 the previous chunk's merge);
    // all leave together if a wait ran out
    if (!named_bar_and(1, kCW * 32, ok)) break;
    const int last = (gt - 1) % C::kStages;
    acc.template merge_warps<C::kMergePairs>(reinterpret_cast<float*>(smem + (C::kMergeInStage ? last * C::kStageBytes : C::kMergeOff)),
                    C::kHandFloats, warp, lane);
    if (C::kMergeInStage) {
      __syncwarp();
      if (lane == 0) {
        fence_proxy_async_smem();
        mbar_arrive(bar_empty + 8 * last);
      }
    }
    if (warp == 0) {
      // (the other warps are at most one chunk ahead, in the other flag)
      const bool corrected = n > 1 && bad[dk & 1] != 0;
      __syncwarp();
      if (corrected && lane == 0) bad[dk & 1] = 0;
      __syncwarp();
      if (d.slot < 0) {
        const size_t row = (size_t)d.pad[kPadRow] * p.H + d.kh * G;
        acc.store_output(static_cast<T*>(p.out) + row * D, p.lse ? p.lse + row : nullptr, R, G, p.H, lane);
        if (corrected) correct_rows<T, D>(p, d.b, d.kh, d.pad[kPadRow], past, n, lane);
      } else {
        acc.store_partial(p.part_o + (size_t)d.slot * p.columns * D, p.part_ml + (size_t)d.slot * p.columns * 2, R,
                          lane, corrected);
        __syncwarp();
        mail(d.first_slot, d.n, d.b, d.kh);
      }
    }
  }
  if (warp == 0) mail(-1, 0, 0, 0);  // no more partials
}

template <typename T, int D, int NT>
cudaError_t launch_nt(const PagedArgs& a, const PagedPlan& plan, uint8_t* ws, uint32_t epoch) {
  using C = Cfg<D, NT>;
  const CUtensorMapDataType dt =
      a.dtype == GQA_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const long long pool_rows = (long long)a.v.num_pages * a.Hkv * a.page;
  CUtensorMap kmap, vmap;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)pool_rows};
  const cuuint64_t strides[1] = {(cuuint64_t)D * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)std::min(a.page, C::kTile)};
  if (!encode_tensor_map(&kmap, dt, 2, const_cast<void*>(a.k_pages), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tensor_map(&vmap, dt, 2, const_cast<void*>(a.v_pages), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  DecParams p{};
  p.v = a.v;
  p.q = a.q;
  p.k_pages = a.k_pages;
  p.v_pages = a.v_pages;
  p.out = a.out;
  p.lse = a.lse;
  p.part_o = reinterpret_cast<float*>(ws + plan.part_o_off);
  p.part_ml = reinterpret_cast<float*>(ws + plan.part_ml_off);
  p.ticket = reinterpret_cast<unsigned long long*>(ws + plan.sched_off);
  p.arrivals = p.ticket + 1;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.G = a.H / a.Hkv;
  p.window = a.window;
  p.P = plan.ctas;
  p.chunks_per_cta = kDecodeChunksPerCta;
  p.columns = plan.columns;
  p.pool_rows = (int)pool_rows;
  p.epoch = epoch;
  p.scale_log2 = a.scale * kLog2e;
  auto kern = paged_decode_kernel<T, D, NT>;
  static std::atomic<int> smem_set[kMaxDevices];
  const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(kern), C::kSmem, smem_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, kmap, vmap, p);
}

template <typename T, int D>
cudaError_t launch_d(const PagedArgs& a, const PagedPlan& plan, uint8_t* ws, uint32_t epoch) {
  return plan.columns <= 8    ? launch_nt<T, D, 1>(a, plan, ws, epoch)
         : plan.columns <= 16 ? launch_nt<T, D, 2>(a, plan, ws, epoch)
         : plan.columns <= 24 ? launch_nt<T, D, 3>(a, plan, ws, epoch)
                              : launch_nt<T, D, 4>(a, plan, ws, epoch);
}

template <typename T>
cudaError_t launch_t(const PagedArgs& a, const PagedPlan& plan, uint8_t* ws, uint32_t epoch) {
  return a.D == 64 ? launch_d<T, 64>(a, plan, ws, epoch) : launch_d<T, 128>(a, plan, ws, epoch);
}

}  // namespace

int paged_decode_ctas_per_sm(int columns, int head_size, int smem_per_sm) {
  const int nt = (columns + 7) / 8;
  const int smem = head_size == 64 ? (nt == 1   ? Cfg<64, 1>::kSmem
                                      : nt == 2 ? Cfg<64, 2>::kSmem
                                      : nt == 3 ? Cfg<64, 3>::kSmem
                                                : Cfg<64, 4>::kSmem)
                                   : (nt == 1   ? Cfg<128, 1>::kSmem
                                      : nt == 2 ? Cfg<128, 2>::kSmem
                                      : nt == 3 ? Cfg<128, 3>::kSmem
                                                : Cfg<128, 4>::kSmem);
  const int n = smem_per_sm / (smem + 1024);
  return n < 1 ? 1 : (n > 2 ? 2 : n);
}

cudaError_t launch_paged_decode(const PagedArgs& a, const PagedPlan& plan, uint8_t* workspace, uint32_t epoch) {
  return a.dtype == GQA_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, plan, workspace, epoch)
                                   : launch_t<__half>(a, plan, workspace, epoch);
}

}  // namespace gqa
