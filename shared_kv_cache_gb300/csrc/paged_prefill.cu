// Attention of chunks of new tokens over a paged cache on the 5th-generation
// tensor cores (tcgen05, accumulators in TMEM), head size D of 64 or 128.
//
//   S = Q K^T,  P = 2^(scale log2 e S - m),  O += P V,  out = O / l
//
// Rows.  The G query heads of a KV head share its keys, so a 128-row tile
// holds TPT = 128 / G new tokens with all their G heads (row r: token r / G,
// head r % G), and a CTA works on two such tiles (a block of 2 TPT tokens)
// over the same K and V tiles: each loaded tile serves 256 rows, a chunk of a
// few tokens fills a tile as far as it can, and the two tiles' softmaxes
// alternate with each other's matrix products.  A block of one tile only
// leaves the second idle.
//
// Work.  A batch mixes long prompts, chunks on long pasts and single tokens,
// so the work is cut by key tiles (128 keys), not by items: an item (block,
// KV head) of n tiles counts n + kItemCost units, and CTA c of the persistent
// grid takes the units [c W / P, (c + 1) W / P) of the W in all (a boundary
// closer than kSnap tiles to an item's end moves there).  Every CTA finds its
// range itself, from seqlens_k and cu_seqlens.  An item that a boundary cuts
// leaves fp32 partials (O, m, l), at most two a CTA, which a small second
// kernel merges; the others write their output directly.
//
// Inside a CTA (384 threads): warp 0 walks the CTA's pieces, publishes their
// descriptors and loads K tiles, warps 2 and 3 load V (one 64-dimension half
// each) and the query tiles, warp 1 issues the matrix products, warps 4..7 and
// 8..11 are the softmax of the two tiles, a thread a row.  K and V tiles come
// through rings of bulk-tensor copies, one box per page and half (or per 128
// rows of a larger page), aimed through the block table; boxes without a
// visible slot are aimed beyond the pool and read as zeros.
//
// TMEM columns: tile i's O at [256 i, 256 i + D), its S (and P over it, as
// 16-bit pairs) at [256 i + 128, 256 i + 256).
//
// Rounding: scores, statistics and O are fp32; P is rounded to T for its
// product with V.  With bf16 and rows of at most 256 visible keys, where a few
// keys can carry all the weight, P's rounding residue is added as a second
// product.  O is rescaled only when a row's maximum grew by more than 2^8
// (P then stays below 2^8, exact in either type's range).
#include <algorithm>
#include <type_traits>

#include "paged.cuh"
#include "prefill_common.cuh"
#include "tc.cuh"

namespace gqa {
namespace {

using paged::kBN;
using paged::kBox;
using paged::Seq;
using paged::TileLoader;
using paged::warp_sum_ll;

constexpr int kBM = 128;       // rows per tile
constexpr int kThreads = 384;  // three warpgroups
constexpr int kRegsLow = 80;
constexpr int kRegsHigh = (384 * 168 - 128 * kRegsLow) / 256 / 8 * 8;
static_assert(128 * kRegsLow + 256 * kRegsHigh <= 384 * 168, "the register split of the launch's registers");
constexpr int kItemCost = 1;     // an item's fixed cost in key tiles (query load, output)
constexpr int kSnap = 2;         // no piece shorter than this many tiles, unless its item is
constexpr int kMinUnits = 3;     // units per CTA at least: a small call takes fewer CTAs
constexpr int kDescs = 3;        // piece descriptors in flight
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleThresh = 8.0f;  // log2 units

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * kBox;  // a K, V or query tile
  static constexpr int kSt = D == 128 ? 2 : 4;       // ring stages of K and of V
  static constexpr int kQOff = 0;
  static constexpr int kKOff = 2 * kTileBytes;
  static constexpr int kVOff = kKOff + kSt * kTileBytes;
  static constexpr int kStageOff = kVOff + kSt * kTileBytes;  // output staging, 4 KB a softmax warp
  static constexpr int kMetaOff = kStageOff + 8 * 4096;
  // barriers: q_full, q_free, drain, k_full/empty, v_full/empty, s_full[2], p_full[2], o_done[2], o_free[2],
  // d_full/d_empty
  static constexpr int kNumBars = 3 + 4 * kSt + 8 + 2 * kDescs;
  static constexpr int kDescOff = kMetaOff + kNumBars * 8 + 8;
  static constexpr int kSmem = (kDescOff + 15) / 16 * 16 + kDescs * 64 + 16 + 1024;
  static_assert(kSmem <= 232448, "the shared memory of one CTA");
};

// One CTA's part of an item: key tiles [t0, t0 + n_kv) of a block's rows.
struct __align__(16) Piece {
  int b, kh;       // b < 0: no more pieces
  int q0, n;       // the sequence's first row, its new tokens
  int past, L;
  int i0;          // first token of the block
  int nact;        // row tiles with tokens: 1 or 2
  int lo;          // first key the block's rows see
  int t0, n_kv;
  int slot;        // partial slot, -1: the piece is the whole item
  int pad[4];
};
static_assert(sizeof(Piece) == 64, "descriptor size");

// Where CTA c's range starts, for the merge: item (b, blk, kh), and whether
// the item began before.
struct Bound {
  int b, blk, kh, inside;
};

struct PreParams {
  PagedView v;
  void* out;
  float* lse;     // nullptr: not wanted
  float* part_o;  // [2 P][2][D / 4][128] float4
  float* part_ml; // [2 P][2][128] float2 (max in log2 units, sum)
  Bound* bounds;  // [P + 1]
  int H, Hkv, G, window, tpt, pool_rows;
  float scale_log2;
};

// ---------------------------------------------------------------------------
// the partition
// ---------------------------------------------------------------------------
// Key tiles of block blk of a sequence, and its first visible key.
__device__ __forceinline__ int block_tiles(const PreParams& p, const Seq& s, int blk, int& lo) {
  const int i0 = blk * 2 * p.tpt, i1 = min(i0 + 2 * p.tpt, s.n);
  lo = paged::first_visible(s.past + i0, p.window);
  return (s.past + i1 + kBN - 1) / kBN - lo / kBN;
}
// Units of one KV head's items of sequence b (0: skipped).
__device__ __forceinline__ long long seq_units(const PreParams& p, int b, Seq& s) {
  int code;
  if (!paged::load_seq(p.v, b, s, code)) return 0;
  long long u = 0;
  int lo;
  for (int blk = 0; blk * 2 * p.tpt < s.n; ++blk) u += block_tiles(p, s, blk, lo) + kItemCost;
  return u;
}

// A position in the sequence of all items' tiles: tile `off` of item (b,
// blk, kh); b == v.B is the end.
struct Pos {
  int b, blk, kh, off;
};

// The whole warp: the position of unit x (of the batch's W), snapped.
__device__ Pos locate(const PreParams& p, long long x, int lane) {
  long long base = 0;
  for (int b0 = 0; b0 < p.v.B; b0 += 32) {
    Seq s;
    const long long mine = b0 + lane < p.v.B ? seq_units(p, b0 + lane, s) * p.Hkv : 0;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const long long total = __shfl_sync(0xffffffffu, incl, 31);
    if (x < base + total) {
      const int l = __ffs(__ballot_sync(0xffffffffu, base + incl > x)) - 1;
      Pos r{b0 + l, 0, 0, 0};
      long long left = x - base - __shfl_sync(0xffffffffu, incl - mine, l);
      int code, lo;
      paged::load_seq(p.v, r.b, s, code);
      while (true) {
        const int n = block_tiles(p, s, r.blk, lo), u = n + kItemCost;
        if (left < (long long)u * p.Hkv) {
          r.kh = (int)(left / u);
          const int off = max(0, (int)(left - (long long)r.kh * u) - kItemCost);
          r.off = off < kSnap ? 0 : n - off < kSnap ? n : off;
          return r;
        }
        left -= (long long)u * p.Hkv;
        ++r.blk;
      }
    }
    base += total;
  }
  return Pos{p.v.B, 0, 0, 0};
}

// ---------------------------------------------------------------------------
// the attention kernel
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, const __grid_constant__ PreParams p) {
  using E = Elem<T>;
  using C = Cfg<D>;
  constexpr bool kBF16 = E::is_bf16;
  constexpr int kSt = C::kSt;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const uint32_t q_full = sb + C::kMetaOff, q_free = q_full + 8, drain = q_full + 16;
  const uint32_t k_full = q_full + 24, k_empty = k_full + 8 * kSt;
  const uint32_t v_full = k_empty + 8 * kSt, v_empty = v_full + 8 * kSt;
  const uint32_t s_full = v_empty + 8 * kSt, p_full = s_full + 16, o_done = p_full + 16, o_free = o_done + 16;
  const uint32_t d_full = o_free + 16, d_empty = d_full + 8 * kDescs;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::kMetaOff + C::kNumBars * 8);
  Piece* descs = reinterpret_cast<Piece*>(smem + (C::kDescOff + 15) / 16 * 16);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x, P = gridDim.x;

  pdl_launch_dependents();
  if (tid == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    mbar_init(drain, 1);
    for (int s = 0; s < kSt; ++s) {
      mbar_init(k_full + 8 * s, 1);
      mbar_init(k_empty + 8 * s, 1);
      mbar_init(v_full + 8 * s, C::kHalves);  // a producer warp per half
      mbar_init(v_empty + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, 128);
      mbar_init(o_done + 8 * i, 1);
      mbar_init(o_free + 8 * i, 128);
    }
    for (int s = 0; s < kDescs; ++s) {
      mbar_init(d_full + 8 * s, 1);
      mbar_init(d_empty + 8 * s, 11);  // every warp but the publisher
    }
    fence_mbar_init();
  }
  if (warp == 1) tc::alloc(smem_u32(tslot), kTmemCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tbase = *tslot;

  // (whole warp) the k-th piece of this CTA, and the release of its slot
  auto next_piece = [&](int k, Piece& w) {
    if (!__all_sync(0xffffffffu, mbar_wait(d_full + 8 * (k % kDescs), (k / kDescs) & 1, p.v.err))) return false;
    w = descs[k % kDescs];
    __syncwarp();
    if (lane == 0) mbar_arrive(d_empty + 8 * (k % kDescs));
    return w.b >= 0;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
    if (warp == 0) {
      // ---------------- the pieces, and the K tiles ----------------
      if (lane == 0) prefetch_tensormap(&kmap);
      pdl_wait_primary();  // lists, queries and rows may be the previous kernel's
      long long W = 0;
      for (int b0 = 0; b0 < p.v.B; b0 += 32) {
        Seq s;
        W += warp_sum_ll(b0 + lane < p.v.B ? seq_units(p, b0 + lane, s) : 0);
      }
      W *= p.Hkv;
      if (c == 0)  // sequences that fail the checks are reported once
        for (int b = lane; b < p.v.B; b += 32) {
          Seq s;
          int code;
          paged::load_seq(p.v, b, s, code);
          if (code) record_error(p.v.err, code);
        }
      const long long Pe = max(1ll, min((long long)P, W / kMinUnits));  // CTAs with work
      Pos cur = c < Pe ? locate(p, c * W / Pe, lane) : Pos{p.v.B, 0, 0, 0};
      const Pos end = c + 1 < Pe ? locate(p, (c + 1) * W / Pe, lane) : Pos{p.v.B, 0, 0, 0};
      if (lane == 0) {
        // an offset at the item's end is the next item's start: not inside
        Seq s;
        int code, lo, n = 0;
        if (cur.off > 0) {
          paged::load_seq(p.v, cur.b, s, code);
          n = block_tiles(p, s, cur.blk, lo);
        }
        p.bounds[c] = Bound{cur.b, cur.blk, cur.kh, cur.off > 0 && cur.off < n};
        if (c == P - 1) p.bounds[P] = Bound{p.v.B, 0, 0, 0};
      }
      int gk = 0, k = 0;
      bool ok = true;
      Seq s{};
      int sb_ = -1;       // the sequence held in s
      bool any = false;
      while (ok) {
        // the next piece: tiles [cur.off, e) of item (cur.b, cur.blk, cur.kh)
        Piece w{};
        w.b = -1;
        while (cur.b < p.v.B) {
          if (sb_ != cur.b) {
            int code;
            any = paged::load_seq(p.v, cur.b, s, code);
            sb_ = cur.b;
          }
          if (!any || cur.blk * 2 * p.tpt >= s.n) {
            cur = Pos{cur.b + 1, 0, 0, 0};
            continue;
          }
          // past the range's end?
          if (cur.b > end.b || (cur.b == end.b && (cur.blk > end.blk || (cur.blk == end.blk && cur.kh > end.kh)))) break;
          const bool last = cur.b == end.b && cur.blk == end.blk && cur.kh == end.kh;
          int lo;
          const int n = block_tiles(p, s, cur.blk, lo);
          const int e = last ? min(end.off, n) : n;
          if (cur.off < e) {
            w.b = cur.b;
            w.kh = cur.kh;
            w.q0 = s.q0;
            w.n = s.n;
            w.past = s.past;
            w.L = s.L;
            w.i0 = cur.blk * 2 * p.tpt;
            w.nact = w.i0 + p.tpt < s.n ? 2 : 1;
            w.lo = lo;
            w.t0 = lo / kBN + cur.off;
            w.n_kv = e - cur.off;
            w.slot = cur.off > 0 ? 2 * c : e < n ? 2 * c + 1 : -1;
          }
          if (last) cur = Pos{p.v.B, 0, 0, 0};
          else if (cur.kh + 1 < p.Hkv) cur = Pos{cur.b, cur.blk, cur.kh + 1, 0};
          else cur = Pos{cur.b, cur.blk + 1, 0, 0};
          if (w.b >= 0) break;
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
        TileLoader ld;
        ld.begin(p.v, p.Hkv, p.pool_rows, w.b, w.kh, w.lo, w.L, w.t0, w.n_kv, lane);
        for (int j = 0; j < w.n_kv; ++j, ++gk) {
          const int st = gk % kSt;
          if (gk >= kSt) {
            ok = __all_sync(0xffffffffu, mbar_wait(k_empty + 8 * st, ((gk / kSt) - 1) & 1, p.v.err));
            if (!ok) break;
          }
          if (lane == 0) mbar_arrive_expect_tx(k_full + 8 * st, C::kTileBytes);
          __syncwarp();
          ld.issue(&kmap, w.t0 + j, sb + C::kKOff + st * C::kTileBytes, 0, C::kHalves, k_full + 8 * st, lane);
        }
      }
      // no copy may still be in flight into shared memory when the CTA exits
      for (int t = max(0, gk - kSt); t < gk; ++t) mbar_wait(k_full + 8 * (t % kSt), (t / kSt) & 1, p.v.err);
    } else if (warp >= 2) {
      // ---------------- V tiles (a half each) and, warp 3, the query tiles ----------------
      const bool is_q = warp == 3, is_v = warp - 2 < C::kHalves;
      if (lane == 0) {
        if (is_q) prefetch_tensormap(&qmap);
        prefetch_tensormap(&vmap);
      }
      pdl_wait_primary();
      int gv = 0;
      bool ok = true;
      int k = 0;
      Piece w;
      for (; ok && next_piece(k, w); ++k) {
        if (is_q) {
          // the query buffers are free once the previous piece's score MMAs are done
          if (k > 0) ok = __all_sync(0xffffffffu, mbar_wait(q_free, (k - 1) & 1, p.v.err));
          if (!ok) break;
          if (lane == 0) {
            // tokens past the sequence's end are other rows of the batch (or
            // zeros past the arrays'): their results are never stored
            mbar_arrive_expect_tx(q_full, w.nact * C::kHalves * p.G * p.tpt * 128);
            for (int i = 0; i < w.nact; ++i)
              for (int h = 0; h < C::kHalves; ++h)
                pf::tma_load_4d(sb + C::kQOff + i * C::kTileBytes + h * kBox, &qmap, 0, w.kh * p.G,
                                w.q0 + w.i0 + i * p.tpt, h, q_full);
          }
          __syncwarp();
        }
        if (!is_v) continue;
        TileLoader ld;
        ld.begin(p.v, p.Hkv, p.pool_rows, w.b, w.kh, w.lo, w.L, w.t0, w.n_kv, lane);
        for (int j = 0; j < w.n_kv; ++j, ++gv) {
          const int st = gv % kSt;
          if (gv >= kSt) {
            ok = __all_sync(0xffffffffu, mbar_wait(v_empty + 8 * st, ((gv / kSt) - 1) & 1, p.v.err));
            if (!ok) break;
          }
          if (lane == 0) mbar_arrive_expect_tx(v_full + 8 * st, kBox);
          __syncwarp();
          ld.issue(&vmap, w.t0 + j, sb + C::kVOff + st * C::kTileBytes, warp - 2, warp - 1, v_full + 8 * st, lane);
        }
      }
      if (is_q && k > 0) mbar_wait(q_full, (k - 1) & 1, p.v.err);
      if (is_v)
        for (int t = max(0, gv - kSt); t < gv; ++t) mbar_wait(v_full + 8 * (t % kSt), (t / kSt) & 1, p.v.err);
    } else {
      // ---------------- MMA issuer ----------------
      const uint32_t id_s = tc::idesc_f16(kBF16, kBM, kBN, false, false);
      const uint32_t id_o = tc::idesc_f16(kBF16, kBM, D, false, true);
      constexpr uint32_t kHi = tc::desc_hi(1024, tc::kSwizzle128B);
      int g = 0;                     // key tiles, over the CTA's pieces
      int gt1 = 0, kq1 = 0;          // tile 1's score tiles and pieces (tile 0's are g and k)
      int k = 0;
      Piece w;
      bool ok = true;
      for (; next_piece(k, w); ++k) {
        if (lane == 0 && ok) {
          const bool splitp = kBF16 && w.past + w.i0 + 1 <= 256;
          const bool two = w.nact == 2;
          auto issue_s = [&](int i, int stage) {  // S_i = Q_i K^T
            const uint32_t d = tbase + 256 * i + 128;
            const uint32_t ql = tc::desc_lo(sb + C::kQOff + i * C::kTileBytes, 16);
            const uint32_t kl = tc::desc_lo(sb + C::kKOff + stage * C::kTileBytes, 16);
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
              const uint32_t off = ((x >> 2) * kBox + (x & 3) * 32) >> 4;
              tc::mma_ss(d, ql + off, kl + off, kHi, id_s, x > 0 ? 1u : 0u);
            }
            tc::commit(s_full + 8 * i);
          };
          auto issue_pv = [&](int i, int stage, bool first) {  // O_i += P_i V, P from TMEM
            const uint32_t tO = tbase + 256 * i, pa = tO + 128;
            const uint32_t vb = tc::desc_lo(sb + C::kVOff + stage * C::kTileBytes, kBox);
#pragma unroll
            for (int x = 0; x < kBN / 16; ++x)
              tc::mma_ts(tO, pa + x * 8, vb + x * (2048 >> 4), kHi, id_o, (x > 0 || !first) ? 1u : 0u);
            if (splitp)
#pragma unroll
              for (int x = 0; x < kBN / 16; ++x) tc::mma_ts(tO, pa + 64 + x * 8, vb + x * (2048 >> 4), kHi, id_o, 1u);
            tc::commit(o_done + 8 * i);
          };
          ok = mbar_wait(q_full, k & 1, p.v.err) && mbar_wait(k_full + 8 * (g % kSt), (g / kSt) & 1, p.v.err);
          if (ok) {
            tc::fence_after();
            issue_s(0, g % kSt);
            if (two) issue_s(1, g % kSt);
            tc::commit(k_empty + 8 * (g % kSt));
            if (w.n_kv == 1) tc::commit(q_free);
          }
          for (int j = 0; j < w.n_kv && ok; ++j, ++g) {
            const int vs = g % kSt, ks = (g + 1) % kSt;
            if (!mbar_wait(v_full + 8 * vs, (g / kSt) & 1, p.v.err)) { ok = false; break; }
            const bool more = j + 1 < w.n_kv;
            for (int i = 0; i < w.nact && ok; ++i) {
              // P_i(j) V_j, then S_i(j + 1) over the same TMEM columns; the
              // first product of a piece overwrites O_i, which must have been read
              const int gt = i ? gt1 : g, kq = i ? kq1 : k;
              if (!mbar_wait(p_full + 8 * i, gt & 1, p.v.err)) { ok = false; break; }
              if (j == 0 && kq > 0 && !mbar_wait(o_free + 8 * i, (kq - 1) & 1, p.v.err)) { ok = false; break; }
              tc::fence_after();
              issue_pv(i, vs, j == 0);
              const bool lasti = i + 1 == w.nact;
              if (lasti) tc::commit(v_empty + 8 * vs);
              if (more) {
                if (i == 0 && !mbar_wait(k_full + 8 * ks, ((g + 1) / kSt) & 1, p.v.err)) { ok = false; break; }
                tc::fence_after();
                issue_s(i, ks);
                if (lasti) {
                  tc::commit(k_empty + 8 * ks);
                  if (j + 2 == w.n_kv) tc::commit(q_free);  // the piece's last score MMAs
                }
              }
            }
            if (two) ++gt1;
          }
          if (two) ++kq1;
          tc::commit(drain);  // the piece's MMAs
        }
        __syncwarp();
      }
      // every MMA issued has completed before TMEM is released
      if (lane == 0 && k > 0) mbar_wait(drain, (k - 1) & 1, p.v.err);
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
    // ---------------- softmax: tile 0 (warps 4..7), tile 1 (warps 8..11) ----------------
    const int ti = (warp - 4) >> 2;
    const int row = 32 * (warp & 3) + lane;  // TMEM lane of this thread = row of the tile
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tO = tbase + 256 * ti + lane_off;
    const uint32_t tS = tO + 128;
    const uint32_t sf = s_full + 8 * ti, pfb = p_full + 8 * ti, od = o_done + 8 * ti;
    const float sc = p.scale_log2;
    const int rt = row / p.G, rg = row - rt * p.G;  // the row's token in the tile, its head
    int gt = 0;  // score tiles of this row tile
    Piece w;
    for (int k = 0; next_piece(k, w); ++k) {
      if (ti >= w.nact) continue;
      const int i = w.i0 + ti * p.tpt + rt;            // the row's token
      const bool valid = rt < p.tpt && i < w.n;
      const bool live = __any_sync(0xffffffffu, valid);  // the warp has a row to compute
      const int pos = w.past + min(i, w.n - 1);
      const int first_pos = w.past + w.i0 + ti * p.tpt;
      const int last_pos = w.past + min(w.i0 + (ti + 1) * p.tpt, w.n) - 1;
      const int all_lo = paged::first_visible(last_pos, p.window), my_lo = paged::first_visible(pos, p.window);
      const bool splitp = kBF16 && w.past + w.i0 + 1 <= 256;
      float m_ref = -INFINITY, l_run = 0.f;
      bool ok = true;
      for (int j = 0; j < w.n_kv; ++j, ++gt) {
        const int k0 = (w.t0 + j) * kBN;
        if (!__all_sync(0xffffffffu, mbar_wait(sf, gt & 1, p.v.err))) { ok = false; break; }
        tc::fence_after();
        if (live) {
          uint32_t sv[4][32];
#pragma unroll
          for (int x = 0; x < 4; ++x) tc::ld32(tS + 32 * x, sv[x]);
          tc::wait_ld();
          if (k0 + kBN - 1 > first_pos || k0 < all_lo) {
            // column e is visible when my_lo - k0 <= e <= pos - k0
            const int hi = pos - k0, lo = my_lo - k0;
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (x * 32 + e > hi || x * 32 + e < lo) sv[x][e] = __float_as_uint(-INFINITY);
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              mx[(e >> 1) & 3] = max3(mx[(e >> 1) & 3], __uint_as_float(sv[x][e]), __uint_as_float(sv[x][e + 1]));
          const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;  // (scale > 0)
          const float m_new = fmaxf(m_ref, mt);
          const bool need = m_new > m_ref + kRescaleThresh;
          const bool any_need = __any_sync(0xffffffffu, need);
          const float f_resc = need ? fast_exp2(m_ref - m_new) : 1.f;
          if (need) {
            m_ref = m_new;
            l_run *= f_resc;
          }
          const float mu = m_ref == -INFINITY ? 0.f : m_ref;
          const float2 sc2 = make_float2(sc, sc), nmu2 = make_float2(-mu, -mu);
          float2 rs2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          auto make_p = [&](auto split_c) {
            constexpr bool kSplit = decltype(split_c)::value;
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // score columns 64 h .. -> P columns 32 h ..
              uint32_t pk[32];
#pragma unroll
              for (int c2 = 0; c2 < 2; ++c2)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const int x = 2 * h + c2;
                  const float2 z = fma2(make_float2(__uint_as_float(sv[x][2 * e]), __uint_as_float(sv[x][2 * e + 1])),
                                        sc2, nmu2);
                  const float a = fast_exp2(z.x), bb = fast_exp2(z.y);
                  rs2[e & 1] = add2(rs2[e & 1], make_float2(a, bb));
                  pk[c2 * 16 + e] = E::pack2(a, bb);
                  if (kSplit) {
                    sv[x][2 * e] = __float_as_uint(a);
                    sv[x][2 * e + 1] = __float_as_uint(bb);
                  }
                }
              tc::st32(tS + 32 * h, pk);
            }
            if (kSplit) {
              // P's rounding residue in columns [64, 128)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t res[32];
#pragma unroll
                for (int c2 = 0; c2 < 2; ++c2)
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    const int x = 2 * h + c2;
                    const float a = __uint_as_float(sv[x][2 * e]), bb = __uint_as_float(sv[x][2 * e + 1]);
                    const float2 hv = E::unpack2(E::pack2(a, bb));
                    res[c2 * 16 + e] = E::pack2(a - hv.x, bb - hv.y);
                  }
                tc::st32(tS + 64 + 32 * h, res);
              }
            }
          };
          if (splitp)
            make_p(std::true_type{});
          else
            make_p(std::false_type{});
          l_run += (rs2[0].x + rs2[1].x) + (rs2[0].y + rs2[1].y);
          if (any_need && j > 0) {
            // O holds the earlier tiles' sum once P(j-1) V_(j-1) has completed
            // (it has: S(j), issued after it, has)
            if (!__all_sync(0xffffffffu, mbar_wait(od, (gt - 1) & 1, p.v.err))) { ok = false; break; }
            tc::fence_after();
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
              uint32_t r[32];
              tc::ld32(tO + x * 32, r);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f_resc);
              tc::st32(tO + x * 32, r);
            }
          }
          tc::wait_st();
        }
        // value rows of slots outside [lo, L) must not meet P = 0 as NaN:
        // tile 0's warps clear them before its P is ready, and tile 1's
        // product is issued after tile 0's
        if (ti == 0 && (k0 + kBN > w.L || k0 < w.lo)) {
          const int vs = gt % kSt;  // (tile 0 counts every key tile)
          if (!__all_sync(0xffffffffu, mbar_wait(v_full + 8 * vs, (gt / kSt) & 1, p.v.err))) { ok = false; break; }
          if (k0 + row >= w.L || k0 + row < w.lo) {
            uint8_t* vt = smem + C::kVOff + vs * C::kTileBytes + row * 128;
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
              for (int x = 0; x < 8; ++x) *reinterpret_cast<uint4*>(vt + h * kBox + x * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tc::fence_before();
        mbar_arrive(pfb);
      }
      if (!ok) break;
      // the piece's MMAs have completed
      if (!__all_sync(0xffffffffu, mbar_wait(drain, k & 1, p.v.err))) break;
      tc::fence_after();
      if (w.slot >= 0) {
        // fp32 partial: 16-byte units of a row apart by the tile's 128 rows,
        // so that a warp's stores are contiguous
        float4* po = reinterpret_cast<float4*>(p.part_o) + ((size_t)w.slot * 2 + ti) * (D / 4) * kBM + row;
        if (live) {
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            uint32_t r[32];
            tc::ld32(tO + 32 * x, r);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e)
              po[(size_t)(x * 8 + e) * kBM] = make_float4(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1]),
                                                          __uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3]));
          }
          reinterpret_cast<float2*>(p.part_ml)[((size_t)w.slot * 2 + ti) * kBM + row] = make_float2(m_ref, l_run);
        }
      } else if (live) {
        // O / l, 64 dimensions at a time through the warp's stage (32 rows of
        // 128 bytes, 16-byte units swizzled), so that the stores to the output
        // rows are 128 contiguous bytes
        const float inv = 1.f / l_run;
        const size_t orow = (size_t)(w.q0 + i) * p.H + w.kh * p.G + rg;
        const long long mine = valid ? (long long)orow : -1;
        uint8_t* stg = smem + C::kStageOff + (warp - 4) * 4096;
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t r[32];
            tc::ld32(tO + 64 * h + 32 * x, r);
            tc::wait_ld();
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint32_t* rr = r + 8 * u;
              uint4 v;
              v.x = E::pack2(__uint_as_float(rr[0]) * inv, __uint_as_float(rr[1]) * inv);
              v.y = E::pack2(__uint_as_float(rr[2]) * inv, __uint_as_float(rr[3]) * inv);
              v.z = E::pack2(__uint_as_float(rr[4]) * inv, __uint_as_float(rr[5]) * inv);
              v.w = E::pack2(__uint_as_float(rr[6]) * inv, __uint_as_float(rr[7]) * inv);
              *reinterpret_cast<uint4*>(stg + lane * 128 + (((4 * x + u) ^ (lane & 7)) << 4)) = v;
            }
          }
          __syncwarp();
#pragma unroll
          for (int g8 = 0; g8 < 8; ++g8) {
            const int r = g8 * 4 + (lane >> 3), u = lane & 7;
            const long long at = __shfl_sync(0xffffffffu, mine, r);
            const uint4 v = *reinterpret_cast<const uint4*>(stg + r * 128 + ((u ^ (r & 7)) << 4));
            if (at >= 0) *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + at * D + h * 64 + u * 8) = v;
          }
          __syncwarp();
        }
        if (p.lse && valid) p.lse[orow] = m_ref * kLn2 + logf(l_run);
      }
      // O is read: the next piece's first P V may overwrite it
      tc::fence_before();
      mbar_arrive(o_free + 8 * ti);
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc(tbase, kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// the merge of the items that a boundary cut
// ---------------------------------------------------------------------------
// CTA (c, row tile, 32 dimensions): if boundary c is the first inside its
// item, the item's partials: CTA c - 1's last piece, then the first pieces of
// CTAs c, c + 1, ... as long as their boundaries lie inside the same item.
template <typename T, int D>
__global__ void __launch_bounds__(kBM) paged_merge_kernel(const __grid_constant__ PreParams p) {
  using E = Elem<T>;
  pdl_wait_primary();
  pdl_launch_dependents();
  const int c = blockIdx.x, ti = blockIdx.y, d0 = blockIdx.z * 32, row = threadIdx.x;
  const Bound b = p.bounds[c];
  auto same = [&](const Bound& x) { return x.inside && x.b == b.b && x.blk == b.blk && x.kh == b.kh; };
  if (!b.inside || (c > 0 && same(p.bounds[c - 1]))) return;
  Seq s;
  int code;
  paged::load_seq(p.v, b.b, s, code);
  const int rt = row / p.G, i = b.blk * 2 * p.tpt + ti * p.tpt + rt;
  if (rt >= p.tpt || i >= s.n) return;
  const float4* po = reinterpret_cast<const float4*>(p.part_o);
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  float m = -INFINITY, l = 0.f;
  float acc[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) acc[e] = 0.f;
  int slot = 2 * (c - 1) + 1;
  for (int x = c;;) {
    const size_t at = (size_t)slot * 2 + ti;
    const float2 v = ml[at * kBM + row];
    float4 o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = po[(at * (D / 4) + d0 / 4 + e) * kBM + row];
    const float mn = fmaxf(m, v.x), mu = mn == -INFINITY ? 0.f : mn;
    const float f = fast_exp2(m - mu), g = fast_exp2(v.x - mu);
    l = l * f + v.y * g;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      acc[4 * e] = acc[4 * e] * f + o[e].x * g;
      acc[4 * e + 1] = acc[4 * e + 1] * f + o[e].y * g;
      acc[4 * e + 2] = acc[4 * e + 2] * f + o[e].z * g;
      acc[4 * e + 3] = acc[4 * e + 3] * f + o[e].w * g;
    }
    m = mn;
    if (x > (int)gridDim.x - 1 || !same(p.bounds[x])) break;
    slot = 2 * x++;
  }
  const size_t orow = (size_t)(s.q0 + i) * p.H + b.kh * p.G + (row - rt * p.G);
  const float inv = 1.f / l;
  T* dst = static_cast<T*>(p.out) + orow * D + d0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint4 v;
    v.x = E::pack2(acc[8 * e] * inv, acc[8 * e + 1] * inv);
    v.y = E::pack2(acc[8 * e + 2] * inv, acc[8 * e + 3] * inv);
    v.z = E::pack2(acc[8 * e + 4] * inv, acc[8 * e + 5] * inv);
    v.w = E::pack2(acc[8 * e + 6] * inv, acc[8 * e + 7] * inv);
    *reinterpret_cast<uint4*>(dst + 8 * e) = v;
  }
  if (p.lse && d0 == 0) p.lse[orow] = m * kLn2 + logf(l);
}

template <typename T, int D>
cudaError_t launch_d(const PagedArgs& a, const PagedPlan& plan, uint8_t* ws) {
  using C = Cfg<D>;
  const CUtensorMapDataType dt =
      a.dtype == GQA_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int G = a.H / a.Hkv, tpt = kBM / G;
  const long long pool_rows = (long long)a.v.num_pages * a.Hkv * a.page;
  CUtensorMap qmap, kmap, vmap;
  {
    // (dimension within a half, head, token, half): a box of G heads and tpt
    // tokens lands as the tile's rows, 128 bytes each
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
    if (!encode_tensor_map(&kmap, dt, 2, const_cast<void*>(a.k_pages), dims, strides, box,
                           CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_tensor_map(&vmap, dt, 2, const_cast<void*>(a.v_pages), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  PreParams p{};
  p.v = a.v;
  p.out = a.out;
  p.lse = a.lse;
  p.part_o = reinterpret_cast<float*>(ws + plan.part_o_off);
  p.part_ml = reinterpret_cast<float*>(ws + plan.part_ml_off);
  p.bounds = reinterpret_cast<Bound*>(ws + plan.sched_off);
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.G = G;
  p.window = a.window;
  p.tpt = tpt;
  p.pool_rows = (int)pool_rows;
  p.scale_log2 = a.scale * kLog2e;
  auto kern = paged_prefill_kernel<T, D>;
  static std::atomic<int> smem_set[kMaxDevices];
  cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(kern), C::kSmem, smem_set);
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
  e = cudaLaunchKernelEx(&cfg, kern, qmap, kmap, vmap, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(plan.ctas, 2, D / 32);
  cfg.blockDim = dim3(kBM);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel<T, D>, p);
}

template <typename T>
cudaError_t launch_t(const PagedArgs& a, const PagedPlan& plan, uint8_t* ws) {
  return a.D == 64 ? launch_d<T, 64>(a, plan, ws) : launch_d<T, 128>(a, plan, ws);
}

}  // namespace

size_t paged_prefill_bounds_bytes(int ctas) { return (size_t)(ctas + 1) * sizeof(Bound); }

cudaError_t launch_paged_prefill(const PagedArgs& a, const PagedPlan& plan, uint8_t* workspace) {
  return a.dtype == GQA_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, plan, workspace) : launch_t<__half>(a, plan, workspace);
}

}  // namespace gqa
