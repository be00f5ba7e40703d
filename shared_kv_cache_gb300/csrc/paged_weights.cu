// The attention weight every cached key receives from the new tokens, on the
// 5th-generation tensor cores (head size D of 64 or 128):
//
//   w_j = (j < P_b ? w_in_j : 0) + sum over the rows r that see j of 2^(scale log2 e k_j.q_r - lse_r log2 e)
//
// with the rows r = (new token, query head of the KV head).
//
// The product is taken as S^T = K Q^T: a key is a row (a TMEM lane, a
// thread), the query rows are the columns.  Each thread then sums its own
// key's weights over the columns, with no reduction across threads, no atomics
// and a fixed order; the causal mask and the window are a range of columns.
//
// A CTA takes two key tiles of 128 keys (one or two softmax warpgroups each),
// keeps them in shared memory and passes the query rows over them in blocks of up to
// 128 columns (128 / G tokens with their G heads; one block of 16 or 32 columns
// when a decode step has no more).  Items (two tiles of a sequence and KV head) are
// dealt out by their number of blocks, contiguous ranges per CTA of a
// persistent grid.
//
// Bound: with few rows by the stream of K (each key row read once): one token of
// each of 16 sequences of up to 4096, 32 on 8 heads of 128, 15.9 us, 4.2 TB/s, of
// which some 6 us are start and end.  With many rows by the hand-over between
// product and 2^x: 8 chunks of 128 tokens after up to 3968, 29.3 us.  There an
// item of two tiles and four blocks takes 5 us, its products 1.4 of them and
// its 2^x 2.2 (four warpgroups at once); a block's product waits for its
// warpgroup's previous block to be read, since TMEM holds one block for each.
// (Query blocks from two producer warps or in three stages instead of two: no
// faster.  Blocks of 64 columns, two a warpgroup, would cost the products half
// as much again.)
#include <algorithm>

#include "paged.cuh"
#include "prefill_common.cuh"
#include "tc.cuh"

namespace gqa {
namespace {

using paged::kBN;
using paged::kBox;
using paged::Seq;
using paged::TileLoader;

constexpr int kItemCost = 1;  // an item's fixed cost in column blocks
constexpr int kDescs = 4;

// N: columns of a block (16 and 32 for decode steps, or 128).  The small
// blocks run two CTAs an SM: their K stream needs the overlap of one's start
// and end with the other's.
template <int D, int N>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * kBox;
  static constexpr bool kSmall = N < 128;
  static constexpr int kCtas = kSmall ? 2 : 1;
  // warpgroups per key tile: with many blocks two take them in turn, since one
  // a tile (two warps a scheduler) waits more than it computes (8 chunks of 128
  // tokens: 38 us with one, 32 with two)
  static constexpr int kTurns = kSmall ? 1 : 2;
  static constexpr int kThreads = 128 + 256 * kTurns;
  static constexpr int kKSt = (D == 128 ? 1 : 2) * (kSmall ? 3 : 4);  // K tiles in the ring
  static constexpr int kQBox = N * 128;                        // one half of a query block
  static constexpr int kQBytes = kHalves * kQBox;
  static constexpr int kQSt = kSmall ? (kQBytes <= 4096 ? 3 : 1) : 2 * 128 / D;  // query blocks in the ring
  static constexpr int kBufCols = kSmall ? 32 : 128;             // TMEM columns of a score block
  static constexpr uint32_t kTmemCols = 4 * kBufCols;            // two tiles, two blocks each
  static constexpr int kQOff = kKSt * kTileBytes;
  static constexpr int kLseOff = kQOff + kQSt * kQBytes;       // [softmax warps][N] floats
  static constexpr int kSumOff = kLseOff + 8 * kTurns * N * 4;  // [kDescs][2 tiles][128] floats: the other turn's sums
  static constexpr int kMetaOff = kSumOff + (kTurns == 2 ? kDescs * 2 * 128 * 4 : 0);
  // k_full/empty, q_full/empty, s_full[2][2], s_empty[2][2], d_full/empty, drain, sums[kDescs][2]
  static constexpr int kNumBars = 2 * kKSt + 2 * kQSt + 8 + 4 * kDescs + 1;
  static constexpr int kDescOff = (kMetaOff + kNumBars * 8 + 8 + 15) / 16 * 16;
  static constexpr int kSmem = kDescOff + kDescs * 64 + 1024;
  static_assert(kCtas * (kSmem + 1024) <= 233472, "the shared memory of one SM");
};

// One item: key tiles t0 .. t0 + nt - 1 (nt 1 or 2) of a sequence and KV
// head, and the column blocks [cb0, cb0 + ncb) that see them.
struct __align__(16) Item {
  int b, kh;  // b < 0: no more items
  int q0, n, past, L, lo;
  int t0, nt, cb0, ncb;
  int pad[5];
};
static_assert(sizeof(Item) == 64, "descriptor size");

struct WParams {
  PagedView v;
  const float* lse;   // [T, H]
  const float* w_in;  // [pages, Hkv, page]
  float* w_out;
  int H, Hkv, G, window, tpt, pool_rows;
  float scale_log2;
};

__device__ __forceinline__ int num_pairs(const WParams& p, const Seq& s, int& lo) {
  lo = paged::first_visible(s.past, p.window);
  return ((s.L + kBN - 1) / kBN - lo / kBN + 1) / 2;
}
// Key tiles and column blocks of pair x.
__device__ __forceinline__ void pair_range(const WParams& p, const Seq& s, int lo, int x, int& t0, int& nt, int& cb0,
                                           int& ncb) {
  const int t_end = (s.L + kBN - 1) / kBN;
  t0 = lo / kBN + 2 * x;
  nt = min(2, t_end - t0);
  const int kf = max(lo, t0 * kBN), kl = min(s.L, (t0 + nt) * kBN) - 1;
  const int i0 = max(0, kf - s.past);  // first token that sees one of the keys, and the last
  const int i1 = p.window > 0 ? (int)min((long long)s.n - 1, (long long)kl + p.window - 1 - s.past) : s.n - 1;
  cb0 = i0 / p.tpt;
  ncb = i1 / p.tpt + 1 - cb0;
}
__device__ __forceinline__ int pair_units(const WParams& p, const Seq& s, int lo, int x) {
  int t0, nt, cb0, ncb;
  pair_range(p, s, lo, x, t0, nt, cb0, ncb);
  return ncb + kItemCost;
}
// Units of one KV head of sequence b (0: skipped).
__device__ __forceinline__ long long seq_units(const WParams& p, int b, Seq& s) {
  int code, lo;
  if (!paged::load_seq(p.v, b, s, code)) return 0;
  const int np = num_pairs(p, s, lo);
  if (s.n <= p.tpt) return (long long)np * (1 + kItemCost);  // one block sees everything
  long long u = 0;
  for (int x = 0; x < np; ++x) u += pair_units(p, s, lo, x);
  return u;
}

// Items in the order (sequence, KV head, pair); an item belongs to the CTA in
// whose range of units it starts.
struct Pos {
  int b, kh, pair;
  long long start;  // the item's first unit
};
// (whole warp) the first item that starts at unit x or later; `first`: the
// units of sequence `lane`
__device__ Pos locate(const WParams& p, long long x, int lane, long long first) {
  long long base = 0;
  for (int b0 = 0; b0 < p.v.B; b0 += 32) {
    Seq s;
    const long long mine = b0 == 0 ? first : b0 + lane < p.v.B ? seq_units(p, b0 + lane, s) : 0;
    long long incl = mine * p.Hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const long long total = __shfl_sync(0xffffffffu, incl, 31);
    if (x < base + total) {
      const int l = __ffs(__ballot_sync(0xffffffffu, base + incl > x)) - 1;
      const long long u = __shfl_sync(0xffffffffu, mine, l);
      long long start = base + __shfl_sync(0xffffffffu, incl, l) - u * p.Hkv;
      Pos r{b0 + l, 0, 0, 0};
      r.kh = (int)((x - start) / u);
      start += u * r.kh;
      int code, lo;
      paged::load_seq(p.v, r.b, s, code);
      const int np = num_pairs(p, s, lo);
      if (s.n <= p.tpt) {
        r.pair = (int)((x - start + kItemCost) / (1 + kItemCost));
        start += (long long)r.pair * (1 + kItemCost);
      } else {
        while (start < x && r.pair < np) start += pair_units(p, s, lo, r.pair++);
      }
      r.start = start;  // (pair == np: the walk steps on to the next KV head)
      return r;
    }
    base += total;
  }
  return Pos{p.v.B, 0, 0, base};
}

// Adds to acc the weights of kW columns from `col` on (scores sv, -lse log2 e
// at ls); kMask: only columns [c_lo, c_hi) count.
template <int kW, bool kMask>
__device__ __forceinline__ void add_columns(const uint32_t (&sv)[kW], const float* ls, float scale_log2, int col,
                                            int c_lo, int c_hi, float2 (&acc)[4]) {
  const float2 sc2 = make_float2(scale_log2, scale_log2);
#pragma unroll
  for (int e = 0; e < kW; e += 4) {
    const float4 l4 = *reinterpret_cast<const float4*>(ls + col + e);
    float2 z0 = fma2(make_float2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), sc2, make_float2(l4.x, l4.y));
    float2 z1 = fma2(make_float2(__uint_as_float(sv[e + 2]), __uint_as_float(sv[e + 3])), sc2,
                     make_float2(l4.z, l4.w));
    if (kMask) {
      const int k = col + e;
      if (k < c_lo || k >= c_hi) z0.x = -INFINITY;
      if (k + 1 < c_lo || k + 1 >= c_hi) z0.y = -INFINITY;
      if (k + 2 < c_lo || k + 2 >= c_hi) z1.x = -INFINITY;
      if (k + 3 < c_lo || k + 3 >= c_hi) z1.y = -INFINITY;
    }
    const int a = (e >> 1) & 2;
    acc[a] = add2(acc[a], make_float2(fast_exp2(z0.x), fast_exp2(z0.y)));
    acc[a + 1] = add2(acc[a + 1], make_float2(fast_exp2(z1.x), fast_exp2(z1.y)));
  }
}

// One block of N columns, scores at TMEM address tb; `freed` is arrived at
// once they are in registers.
template <int N, bool kMask>
__device__ __forceinline__ void weigh_block(uint32_t tb, const float* ls, float scale_log2, int c_lo, int c_hi,
                                            float2 (&acc)[4], uint32_t freed) {
  if constexpr (N <= 32) {
    uint32_t sv[N];
    if constexpr (N == 16)
      tc::ld16(tb, sv);
    else
      tc::ld32(tb, sv);
    tc::wait_ld();
    tc::fence_before();
    mbar_arrive(freed);
    add_columns<N, kMask>(sv, ls, scale_log2, 0, c_lo, c_hi, acc);
  } else {
    // 16 columns at a time, the next 16 on their way meanwhile
    uint32_t even[16], odd[16];
    tc::ld16(tb, even);
    tc::wait_ld16(even);
#pragma unroll
    for (int y = 0; y < N; y += 32) {
      tc::ld16(tb + y + 16, odd);
      add_columns<16, kMask>(even, ls, scale_log2, y, c_lo, c_hi, acc);
      tc::wait_ld16(odd);
      if (y + 32 < N) {
        tc::ld16(tb + y + 32, even);
      } else {
        tc::fence_before();
        mbar_arrive(freed);
      }
      add_columns<16, kMask>(odd, ls, scale_log2, y + 16, c_lo, c_hi, acc);
      if (y + 32 < N) tc::wait_ld16(even);
    }
  }
}

template <typename T, int D, int N>
__global__ void __launch_bounds__(Cfg<D, N>::kThreads, Cfg<D, N>::kCtas)
    paged_weights_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ WParams p) {
  using E = Elem<T>;
  using C = Cfg<D, N>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const uint32_t k_full = sb + C::kMetaOff, k_empty = k_full + 8 * C::kKSt;
  const uint32_t q_full = k_empty + 8 * C::kKSt, q_empty = q_full + 8 * C::kQSt;
  const uint32_t s_full = q_empty + 8 * C::kQSt, s_empty = s_full + 32;  // [tile][buffer]
  const uint32_t d_full = s_empty + 32, d_empty = d_full + 8 * kDescs, drain = d_empty + 8 * kDescs, sums = drain + 8;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::kMetaOff + C::kNumBars * 8);
  Item* descs = reinterpret_cast<Item*>(smem + C::kDescOff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x, P = gridDim.x;

  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < C::kKSt; ++i) {
      mbar_init(k_full + 8 * i, 1);
      mbar_init(k_empty + 8 * i, 1);
    }
    for (int i = 0; i < C::kQSt; ++i) {
      mbar_init(q_full + 8 * i, 1);
      mbar_init(q_empty + 8 * i, 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(s_empty + 8 * i, 128);
    }
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(d_full + 8 * i, 1);
      mbar_init(d_empty + 8 * i, 2 + 8 * C::kTurns);  // warps 1, 2 and the softmax warps
    }
    mbar_init(drain, 1);
    for (int i = 0; i < 2 * kDescs; ++i) mbar_init(sums + 8 * i, 128);
    fence_mbar_init();
  }
  if (warp == 1) tc::alloc(smem_u32(tslot), C::kTmemCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tbase = *tslot;

  // (whole warp) the k-th item of this CTA, and the release of its slot
  auto next_item = [&](int k, Item& w) {
    if (!__all_sync(0xffffffffu, mbar_wait(d_full + 8 * (k % kDescs), (k / kDescs) & 1, p.v.err))) {
      w.b = -1;
      return false;
    }
    w = descs[k % kDescs];
    __syncwarp();
    if (lane == 0) mbar_arrive(d_empty + 8 * (k % kDescs));
    return w.b >= 0;
  };

  if (warp < 4) {
    if (warp == 0) {
      // ---------------- the items, and the K tiles ----------------
      if (lane == 0) prefetch_tensormap(&kmap);
      pdl_wait_primary();
      long long W = 0, first = 0;
      for (int b0 = 0; b0 < p.v.B; b0 += 32) {
        Seq s;
        const long long u = b0 + lane < p.v.B ? seq_units(p, b0 + lane, s) : 0;
        if (b0 == 0) first = u;
        W += paged::warp_sum_ll(u);
      }
      W *= p.Hkv;
      if (c == 0)  // sequences that fail the checks are reported once
        for (int b = lane; b < p.v.B; b += 32) {
          Seq s;
          int code;
          paged::load_seq(p.v, b, s, code);
          if (code) record_error(p.v.err, code);
        }
      const long long end = (c + 1) * W / P;
      Pos cur = locate(p, c * W / P, lane, first);
      int gk = 0, k = 0, sb_ = -1, lo = 0, np = 0;
      bool ok = true, any = false;
      Seq s{};
      TileLoader ld;
      int ld_b = -1, ld_kh = -1;
      while (ok) {
        Item w{};
        w.b = -1;
        while (cur.b < p.v.B && cur.start < end) {
          if (sb_ != cur.b) {
            int code;
            any = paged::load_seq(p.v, cur.b, s, code);
            np = any ? num_pairs(p, s, lo) : 0;
            sb_ = cur.b;
          }
          if (cur.pair >= np) {
            cur.pair = 0;
            if (++cur.kh >= p.Hkv || !any) {
              cur.kh = 0;
              ++cur.b;
            }
            continue;
          }
          w.b = cur.b;
          w.kh = cur.kh;
          w.q0 = s.q0;
          w.n = s.n;
          w.past = s.past;
          w.L = s.L;
          w.lo = lo;
          pair_range(p, s, lo, cur.pair, w.t0, w.nt, w.cb0, w.ncb);
          cur.start += w.ncb + kItemCost;
          ++cur.pair;
          break;
        }
        const int ds = k % kDescs;
        if (k >= kDescs) ok = mbar_wait(d_empty + 8 * ds, ((k / kDescs) - 1) & 1, p.v.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) w.b = -1;
        if (lane == 0) {
          descs[ds] = w;
          mbar_arrive(d_full + 8 * ds);
        }
        ++k;
        if (w.b < 0) break;
        if (w.b != ld_b || w.kh != ld_kh) {
          // the tiles of this KV head from here on, as far as the walk may go
          ld.begin(p.v, p.Hkv, p.pool_rows, w.b, w.kh, w.lo, w.L, w.t0, (w.L + kBN - 1) / kBN - w.t0, lane);
          ld_b = w.b;
          ld_kh = w.kh;
        }
        for (int x = 0; x < w.nt; ++x, ++gk) {
          const int st = gk % C::kKSt;
          if (gk >= C::kKSt) {
            ok = __all_sync(0xffffffffu, mbar_wait(k_empty + 8 * st, ((gk / C::kKSt) - 1) & 1, p.v.err));
            if (!ok) break;
          }
          if (lane == 0) mbar_arrive_expect_tx(k_full + 8 * st, C::kTileBytes);
          __syncwarp();
          ld.issue(&kmap, w.t0 + x, sb + st * C::kTileBytes, 0, C::kHalves, k_full + 8 * st, lane);
        }
      }
      // no copy may still be in flight into shared memory when the CTA exits
      for (int t = max(0, gk - C::kKSt); t < gk; ++t) mbar_wait(k_full + 8 * (t % C::kKSt), (t / C::kKSt) & 1, p.v.err);
    } else if (warp == 1) {
      // ---------------- MMA issuer ----------------
      const uint32_t id = tc::idesc_f16(E::is_bf16, kBN, N, false, false);
      constexpr uint32_t kHi = tc::desc_hi(1024, tc::kSwizzle128B);
      int gk = 0, gq = 0;     // K tiles and query blocks consumed
      int gs[2][2] = {};      // score blocks of each tile and buffer
      bool ok = true;
      Item w;
      int k = 0;
      pdl_wait_primary();  // (so that no wait's limit counts what the previous kernel still takes)
      for (; next_item(k, w); ++k) {
        if (lane == 0 && ok) {
          for (int cb = 0; cb < w.ncb && ok; ++cb, ++gq) {
            const int qs = gq % C::kQSt;
            if (!mbar_wait(q_full + 8 * qs, (gq / C::kQSt) & 1, p.v.err)) { ok = false; break; }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (x >= w.nt) break;
              const int st = (gk + x) % C::kKSt;
              // the buffers take turns: with two warpgroups a tile by the
              // block's number, with one over all blocks
              const int buf = C::kTurns == 2 ? cb & 1 : (gs[x][0] + gs[x][1]) & 1;
              const int n = buf ? gs[x][1] : gs[x][0];
              if (cb == 0 && !mbar_wait(k_full + 8 * st, ((gk + x) / C::kKSt) & 1, p.v.err)) { ok = false; break; }
              if (n > 0 && !mbar_wait(s_empty + 16 * x + 8 * buf, (n - 1) & 1, p.v.err)) { ok = false; break; }
              tc::fence_after();
              const uint32_t kl = tc::desc_lo(sb + st * C::kTileBytes, 16);
              const uint32_t ql = tc::desc_lo(sb + C::kQOff + qs * C::kQBytes, 16);
#pragma unroll
              for (int y = 0; y < D / 16; ++y) {
                const uint32_t ko = ((y >> 2) * kBox + (y & 3) * 32) >> 4;
                const uint32_t qo = ((y >> 2) * C::kQBox + (y & 3) * 32) >> 4;
                tc::mma_ss(tbase + (2 * x + buf) * C::kBufCols, kl + ko, ql + qo, kHi, id, y > 0 ? 1u : 0u);
              }
              tc::commit(s_full + 16 * x + 8 * buf);
              if (buf) ++gs[x][1];
              else ++gs[x][0];
              if (cb + 1 == w.ncb) tc::commit(k_empty + 8 * st);
            }
            if (ok) tc::commit(q_empty + 8 * qs);
          }
          gk += w.nt;
        }
        __syncwarp();
      }
      // every MMA issued has completed before TMEM is released
      if (lane == 0) {
        tc::commit(drain);
        mbar_wait(drain, 0, p.v.err);
      }
      __syncwarp();
    } else if (warp == 2) {
      // ---------------- query blocks ----------------
      if (lane == 0) prefetch_tensormap(&qmap);
      pdl_wait_primary();
      int gq = 0;
      bool ok = true;
      Item w;
      for (int k = 0; next_item(k, w); ++k) {
        if (lane == 0)
          for (int cb = 0; cb < w.ncb && ok; ++cb, ++gq) {
            const int qs = gq % C::kQSt;
            if (gq >= C::kQSt && !mbar_wait(q_empty + 8 * qs, ((gq / C::kQSt) - 1) & 1, p.v.err)) { ok = false; break; }
            mbar_arrive_expect_tx(q_full + 8 * qs, C::kHalves * p.G * p.tpt * 128);
            for (int h = 0; h < C::kHalves; ++h)
              pf::tma_load_4d(sb + C::kQOff + qs * C::kQBytes + h * C::kQBox, &qmap, 0, w.kh * p.G,
                              w.q0 + (w.cb0 + cb) * p.tpt, h, q_full + 8 * qs);
          }
        __syncwarp();
      }
      for (int t = max(0, gq - C::kQSt); t < gq; ++t) mbar_wait(q_full + 8 * (t % C::kQSt), (t / C::kQSt) & 1, p.v.err);
    }
  } else {
    // ---------------- softmax warpgroups: key tile x, blocks in turn q ----------------
    const int wg = (warp - 4) >> 2, x = wg & 1, q = wg >> 1;
    const int row = 32 * (warp & 3) + lane;  // TMEM lane = key of the tile
    const uint32_t tS = tbase + 2 * x * C::kBufCols + ((uint32_t)(32 * (warp & 3)) << 16);
    float* ls = reinterpret_cast<float*>(smem + C::kLseOff) + (warp - 4) * N;
    // the warp's own copy of a block's lse, kPer columns a lane (one copy a
    // warpgroup took a barrier of its four warps a block)
    constexpr int kPer = (N + 31) / 32;
    int off[kPer];  // of the lane's columns, from the block's first in lse
#pragma unroll
    for (int e = 0; e < kPer; ++e) off[e] = (lane + 32 * e) / p.G * p.H + (lane + 32 * e) % p.G;
    int gs = 0;
    pdl_wait_primary();  // lse and weights_in may be the previous kernel's
    // lse of the lane's columns of block cb (used first a block later, so that
    // nobody waits for the load)
    auto load_lse = [&](const Item& w, int cb, float (&v)[kPer]) {
      const int i0 = (w.cb0 + cb) * p.tpt, nv = min(p.tpt, w.n - i0) * p.G;
      const float* src = p.lse + (size_t)(w.q0 + i0) * p.H + w.kh * p.G;
#pragma unroll
      for (int e = 0; e < kPer; ++e) v[e] = lane + 32 * e < nv ? src[off[e]] : 0.f;
    };
    // The k-th item: its descriptor stays in its slot until the item is done,
    // and what the item needs first (its lse, its key's page) is loaded an item
    // ahead.
    float nl[kPer] = {};
    int pg = -1;
    auto begin = [&](int k) {
      if (!__all_sync(0xffffffffu, mbar_wait(d_full + 8 * (k % kDescs), (k / kDescs) & 1, p.v.err))) return false;
      const Item& w = descs[k % kDescs];
      if (w.b < 0) return false;
      if (x < w.nt) {
        if (q < w.ncb) load_lse(w, q, nl);
        const int key = (w.t0 + x) * kBN + row;
        if (key >= w.lo && key < w.L) pg = p.v.table[(size_t)w.b * p.v.max_pages + (key >> p.v.page_log2)];
      }
      return true;
    };
    bool have = begin(0);
    for (int k = 0; have; ++k) {
      const Item& w = descs[k % kDescs];
      // where the key's weight goes
      const int key = (w.t0 + x) * kBN + row;
      const int ncb = x < w.nt ? w.ncb : 0;
      // with two turns, the one with the last block writes
      const bool writer = C::kTurns == 1 || q == ((ncb - 1) & 1);
      const bool stored = writer && x < w.nt && key >= w.lo && key < w.L;
      size_t at = 0;
      float base = 0.f;
      bool good = false;
      if (stored) {
        good = (unsigned)pg < (unsigned)p.v.num_pages;
        if (good) {
          at = paged::pool_row(p.v, p.Hkv, pg, w.kh, key);
          if (key < w.past) base = p.w_in[at];
        } else {
          record_error(p.v.err, GQA_ERR_INVALID_ARGUMENT);
        }
      }
      float nl0[kPer];
#pragma unroll
      for (int e = 0; e < kPer; ++e) nl0[e] = nl[e];
      have = begin(k + 1);
      float2 acc[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = make_float2(0.f, 0.f);
      bool ok = true;
      for (int cb = q; cb < ncb; cb += C::kTurns, ++gs) {
        __syncwarp();
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (N % 32 == 0 || lane < N) ls[lane + 32 * e] = -nl0[e] * kLog2e;
        __syncwarp();
        if (cb + C::kTurns < ncb) load_lse(w, cb + C::kTurns, nl0);
        const int buf = C::kTurns == 2 ? q : gs & 1, n = C::kTurns == 2 ? gs : gs >> 1;
        if (!__all_sync(0xffffffffu, mbar_wait(s_full + 16 * x + 8 * buf, n & 1, p.v.err))) { ok = false; break; }
        tc::fence_after();
        // the columns (rows of the block) that see this key: [c_lo, c_hi)
        const int i0 = (w.cb0 + cb) * p.tpt;
        const int nv = min(p.tpt, w.n - i0) * p.G;
        const int c_lo = max(0, key - w.past - i0) * p.G;
        const int c_hi = p.window > 0 ? (int)min((long long)nv, ((long long)key + p.window - w.past - i0) * p.G) : nv;
        const bool all = __all_sync(0xffffffffu, c_lo <= 0 && c_hi >= N);
        const uint32_t tb = tS + C::kBufCols * buf, freed = s_empty + 16 * x + 8 * buf;
        if (all)
          weigh_block<N, false>(tb, ls, p.scale_log2, c_lo, c_hi, acc, freed);
        else
          weigh_block<N, true>(tb, ls, p.scale_log2, c_lo, c_hi, acc, freed);
      }
      if (!ok) break;
      const float2 t0 = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
      float sum = t0.x + t0.y;
      if (C::kTurns == 2) {
        // the other turn's sum joins the writer's.  The place and its barrier
        // belong to the descriptor's slot: the other turn cannot come back to
        // them before the writer has given this item's descriptor back, so it
        // is never a phase ahead of the wait.
        const uint32_t bar = sums + 16 * (k % kDescs) + 8 * x;
        float* other = reinterpret_cast<float*>(smem + C::kSumOff) + (k % kDescs) * 256 + x * 128 + row;
        if (!writer) {
          *other = sum;
          mbar_arrive(bar);
        } else {
          if (!__all_sync(0xffffffffu, mbar_wait(bar, (k / kDescs) & 1, p.v.err))) break;
          sum += *other;
        }
      }
      if (good) p.w_out[at] = base + sum;
      __syncwarp();
      if (lane == 0) mbar_arrive(d_empty + 8 * (k % kDescs));
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc(tbase, C::kTmemCols);
  }
}

template <typename T, int D, int N>
cudaError_t launch_n(const PagedArgs& a, const float* w_in, float* w_out, int tpt) {
  using C = Cfg<D, N>;
  const CUtensorMapDataType dt =
      a.dtype == GQA_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int G = a.H / a.Hkv;
  const long long pool_rows = (long long)a.v.num_pages * a.Hkv * a.page;
  CUtensorMap qmap, kmap;
  {
    // (dimension within a half, head, token, half), as in the chunk attention
    const cuuint64_t dims[4] = {64, (cuuint64_t)a.H, (cuuint64_t)a.v.T, (cuuint64_t)C::kHalves};
    const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)a.H * D * 2, 128};
    const cuuint32_t box[4] = {64, (cuuint32_t)G, (cuuint32_t)tpt, 1};
    if (!encode_tensor_map(&qmap, dt, 4, const_cast<void*>(a.q), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  {
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)pool_rows};
    const cuuint64_t strides[1] = {(cuuint64_t)D * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)std::min(a.page, kBN)};
    if (!encode_tensor_map(&kmap, dt, 2, const_cast<void*>(a.k_pages), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  const WParams p{a.v, a.lse, w_in, w_out, a.H, a.Hkv, G, a.window, tpt, (int)pool_rows, a.scale * kLog2e};
  auto kern = paged_weights_kernel<T, D, N>;
  static std::atomic<int> smem_set[kMaxDevices];
  const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(kern), C::kSmem, smem_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.num_sms * C::kCtas);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, qmap, kmap, p);
}

template <typename T, int D>
cudaError_t launch_d(const PagedArgs& a, const float* w_in, float* w_out) {
  const int G = a.H / a.Hkv;
  // a small block that holds all rows of a decode step has less to read and
  // exponentiate than one of 128
  const long long rows = (long long)a.v.max_new * G;
  if (rows <= 16) return launch_n<T, D, 16>(a, w_in, w_out, 16 / G);
  if (rows <= 32) return launch_n<T, D, 32>(a, w_in, w_out, 32 / G);
  return launch_n<T, D, 128>(a, w_in, w_out, 128 / G);
}

}  // namespace

bool paged_weights_tensor(const PagedArgs& a) { return (a.D == 64 || a.D == 128) && a.H / a.Hkv <= 128; }

cudaError_t launch_paged_weights(const PagedArgs& a, const float* w_in, float* w_out) {
  if (a.dtype == GQA_DTYPE_BF16)
    return a.D == 64 ? launch_d<__nv_bfloat16, 64>(a, w_in, w_out) : launch_d<__nv_bfloat16, 128>(a, w_in, w_out);
  return a.D == 64 ? launch_d<__half, 64>(a, w_in, w_out) : launch_d<__half, 128>(a, w_in, w_out);
}

}  // namespace gqa
