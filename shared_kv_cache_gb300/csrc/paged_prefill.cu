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
// range itself, from seqlens_k and cu_seqlens.  The pieces of an item that
// boundaries cut (at most two a CTA) are merged by the one that finishes last:
// the others leave fp32 partials (O, m, l) and count themselves in on a counter
// of the item's (epoch-tagged, as in the decode kernels; nobody waits).
//
// With many items a CTA, none of them large, items are not cut but handed out
// whole by a ticket counter, each sequence's last (longest) blocks first: the
// CTAs then end together although some run faster than others.
//
// Inside a CTA (384 threads): warp 0 walks the CTA's pieces, publishes their
// descriptors and loads K tiles, warps 2 and 3 load V (one 64-dimension half
// each) and the query tiles, warp 1 issues the matrix products, warps 4..7 and
// 8..11 are the softmax of the two tiles, a thread a row.  A piece's output is
// written after the next piece's first softmax, so that neither its last
// product nor the next one's first is waited for.  K and V tiles come
// through rings of bulk-tensor copies, one box per page and half (or per 128
// rows of a larger page), aimed through the block table; boxes without a
// visible slot are aimed beyond the pool and read as zeros.
//
// Measured: 2048 tokens after 30,000, 32 on 8 heads of 128, fp16, 780 us, 1.33
// PFLOP/s (of 1.87 that a plain matrix product reaches); 4 prompts of 2048 tokens
// 138 us, 1.00 PFLOP/s; 8 chunks of 128 tokens after up to 3968 52 us.  Bound by
// the chain from a tile's scores through its softmax to its product (the two
// tiles cover each other's chains for the most part; two score buffers a tile
// do not fit TMEM's 512 columns beside O), and with short items by the 3.5 us that each takes to
// start and to write.
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

#include "decode_sched.cuh"
#include "paged.cuh"
#include "prefill_common.cuh"
#include "tc.cuh"

namespace gqa {
namespace {

using dsched::epoch_install;
using dsched::epoch_take;
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
constexpr int kItemCost = 2;     // an item's fixed cost in key tiles: 3.5 us of output and restart, a tile takes 1.9
constexpr int kSnap = 3;         // no piece shorter than this many tiles, unless its item is (8 chunks of
                                 // 128 tokens: 54.5 us with 2, 52.5 with 3 or 4)
constexpr int kMinUnits = 3;     // units per CTA at least: a small call takes fewer CTAs
constexpr int kDescs = 3;        // piece descriptors in flight
constexpr int kTicketItems = 4;  // whole items by ticket from so many items a CTA on ...
constexpr int kTicketPart = 3;   // ... none of which takes more than this part of a CTA's share
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
  // barriers: q_full[2], q_free[2], drain, k_full/empty, v_full/empty, s_full[2], p_full[2], o_done[2], o_free[2],
  // d_full/d_empty
  static constexpr int kNumBars = 5 + 4 * kSt + 8 + 2 * kDescs;
  static constexpr int kFlagOff = kMetaOff + kNumBars * 8 + 8;  // one int a softmax warpgroup
  static constexpr int kDescOff = (kFlagOff + 8 + 15) / 16 * 16;
  static constexpr int kSmem = kDescOff + kDescs * 64 + 1024;
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
  int cf, np;      // cut items: the first boundary inside the item, its pieces
  int pad[2];
};
static_assert(sizeof(Piece) == 64, "descriptor size");

struct PreParams {
  PagedView v;
  const void* q;
  const void* k_pages;
  const void* v_pages;
  void* out;
  float* lse;     // nullptr: not wanted
  float* part_o;  // [2 P][2][D / 4][128] float4
  float* part_ml; // [2 P][2][128] float2 (max in log2 units, sum)
  unsigned long long* arrivals;  // [P][2] finished pieces (epoch, count) of the item whose first boundary is c
  unsigned long long* ticket;    // (epoch, count) of items handed out
  int H, Hkv, G, window, tpt, pool_rows;
  uint32_t epoch;
  float scale_log2;
};

// The merge of a cut item's parts by one thread a row: part q at slot(q) (a row's
// stat in ml, its 16-byte units in po, 128 rows apart), added in their order,
// each scaled and rounded by itself, so that which piece came last changes
// nothing.  Returns (m, l) and whether the row is not finite.  Loads
// two parts ahead.
template <typename T, int D>
__device__ __forceinline__ bool merge_parts(const float4* po, const float2* ml, int first, int np, int ti, T* out,
                                            float2& stat) {
  using E = Elem<T>;
  auto slot = [&](int q) { return 2 * (q == 0 ? 2 * first - 1 : 2 * (first + q - 1)) + ti; };
  auto stats = [&](int q0, float2 (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = q0 + e < np ? __ldcg(ml + (size_t)slot(q0 + e) * kBM) : make_float2(-INFINITY, 0.f);
  };
  float2 v[8];
  float m = -INFINITY, l = 0.f;
  for (int q0 = 0; q0 < np; q0 += 8) {
    stats(q0, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, v[e].x);
  }
  const float base = m == -INFINITY ? 0.f : m;
  for (int q0 = 0; q0 < np; q0 += 8) {
    if (np > 8) stats(q0, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) l = __fadd_rn(l, __fmul_rn(v[e].y, fast_exp2(v[e].x - base)));
  }
  stat = make_float2(m, l);
  const float inv = 1.f / l;
  struct Part {
    float4 y[8];
    float m;
  } pa{}, pb{};
  auto fetch = [&](int x, int q, Part& t) {
    if (q >= np || x >= D / 32) return;
    const float4* src = po + ((size_t)slot(q) * (D / 4) + x * 8) * kBM;
#pragma unroll
    for (int e = 0; e < 8; ++e) t.y[e] = __ldcg(src + e * kBM);
    t.m = __ldcg(ml + (size_t)slot(q) * kBM).x;
  };
  fetch(0, 0, pa);
  fetch(0, 1, pb);
  float odd = 0.f;  // 0 times the outputs: not 0 where one is not finite
#pragma unroll 1
  for (int x = 0; x < D / 32; ++x) {
    float acc[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) acc[e] = 0.f;
    auto add = [&](int q, Part& t) {  // then the next but one, of these dimensions or the next ones
      const float g = fast_exp2(t.m - base);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        acc[4 * e] = __fadd_rn(acc[4 * e], __fmul_rn(t.y[e].x, g));
        acc[4 * e + 1] = __fadd_rn(acc[4 * e + 1], __fmul_rn(t.y[e].y, g));
        acc[4 * e + 2] = __fadd_rn(acc[4 * e + 2], __fmul_rn(t.y[e].z, g));
        acc[4 * e + 3] = __fadd_rn(acc[4 * e + 3], __fmul_rn(t.y[e].w, g));
      }
      if (q + 2 < np) fetch(x, q + 2, t);
      else fetch(x + 1, q & 1, t);
    };
#pragma unroll 1
    for (int q = 0; q < np; q += 2) {
      add(q, pa);
      if (q + 1 < np) add(q + 1, pb);
    }
#pragma unroll
    for (int e = 0; e < 32; ++e) odd = fmaf(acc[e], 0.f, odd);
    if (out)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint4 w;
        w.x = E::pack2(acc[8 * u] * inv, acc[8 * u + 1] * inv);
        w.y = E::pack2(acc[8 * u + 2] * inv, acc[8 * u + 3] * inv);
        w.z = E::pack2(acc[8 * u + 4] * inv, acc[8 * u + 5] * inv);
        w.w = E::pack2(acc[8 * u + 6] * inv, acc[8 * u + 7] * inv);
        *reinterpret_cast<uint4*>(out + 32 * x + 8 * u) = w;
      }
  }
  return odd != 0.f;
}

// ---------------------------------------------------------------------------
// Rows whose output is not finite.  The product adds P = 0 times the value rows
// of slots that a token does not see but others of its block do: exact zeros,
// unless such a value is infinite or NaN.  A row that came out so is looked at
// again: if a value that its token does not see can be to blame, the row is
// computed anew from the slots it sees, by itself.  (To look for such values
// before every masked tile's product cost 5 to 8 of 139 us with 4 x 2048 tokens,
// as it stands in the chain from scores to product; to look at the outputs, 2.
// Eight rows at a time halved what such a row costs, 561 to 319 ms for a chunk of
// 128 tokens after 100,000 whose last value row holds a NaN, but the larger
// kernel took 6 us more for every call with 4 x 2048 tokens.)
// ---------------------------------------------------------------------------
struct RowCheck {
  int Hkv, b, kh;
  int lo, hi;  // slots [lo, hi) took part in the row's tiles
  int window;
  float scale_log2;
  // where the row's output goes (-1: not a row), its token's slot, and its
  // softmax state; odd: the output is not finite
  int row, pos;
  float m, l;
  bool odd;
  // parts to merge first (0: the output is there): the first boundary of the
  // item, the tile, the thread's place in a part
  int np, first, ti, at;
};
// (whole warp) the row of the token at slot pos with query row q, softmax state
// (m in log2 units, l) and output row out; a lane takes a slot.
template <typename T, int D>
__device__ __forceinline__ void recheck_row(const PreParams& p, const RowCheck& c, int pos, const T* q, float m, float l,
                                         T* out, int lane) {
  using E = Elem<T>;
  constexpr int kN = D / 32, kU = D / 8;
  const int32_t* tab = p.v.table + (size_t)c.b * p.v.max_pages;
  const int first = paged::first_visible(pos, c.window);
  // element offset of slot s's row (-1: none)
  auto row_of = [&](int s) -> long long {
    const int pg = tab[s >> p.v.page_log2];
    return (unsigned)pg < (unsigned)p.v.num_pages ? (long long)paged::pool_row(p.v, c.Hkv, pg, c.kh, s) * D : -1;
  };
  bool unseen = false;
  for (int s0 = c.lo; s0 < c.hi && !unseen; s0 += 32) {
    if (s0 >= first && s0 + 31 <= pos) {
      s0 += (pos + 1 - s0) / 32 * 32 - 32;  // (to the last of the seen 32s)
      continue;
    }
    const int s = s0 + lane;
    const long long at = s < c.hi && (s < first || s > pos) ? row_of(s) : -1;
    bool odd = false;
    if (at >= 0)
#pragma unroll
      for (int u = 0; u < kU; ++u)
        odd |= paged::nonfinite<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(p.v_pages) + at + 8 * u));
    unseen = __any_sync(0xffffffffu, odd);
  }
  if (!unseen) return;
  float acc[kN];
#pragma unroll
  for (int e = 0; e < kN; ++e) acc[e] = 0.f;
  for (int s0 = first; s0 <= pos; s0 += 32) {
    const int s = s0 + lane;
    const long long at = s <= pos ? row_of(s) : -1;
    float w = 0.f;
    if (at >= 0) {
      float z = 0.f;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint4 a = *reinterpret_cast<const uint4*>(q + 8 * u);
        const uint4 b = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.k_pages) + at + 8 * u);
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = E::unpack2(aw[e]), y = E::unpack2(bw[e]);
          z = fmaf(x.x, y.x, fmaf(x.y, y.y, z));
        }
      }
      w = fast_exp2(fmaf(z, c.scale_log2, -m));
    }
#pragma unroll 8
    for (int j = 0; j < 32; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const long long aj = __shfl_sync(0xffffffffu, at, j);
      const T* v = static_cast<const T*>(p.v_pages) + aj;
#pragma unroll
      for (int e = 0; e < kN; ++e) acc[e] = fmaf(wj, aj >= 0 ? E::to_f(v[lane + 32 * e]) : 0.f, acc[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < kN; ++e) out[lane + 32 * e] = E::from_f(acc[e] / l);
}

// What only some pieces need after their output, in one out-of-line call: with
// its code in line, or in two calls, the kernel spilled registers and 4 x 2048
// tokens took 5 to 10 us more.
template <typename T, int D>
__device__ __noinline__ void merge_and_recheck(const PreParams& p, RowCheck& c, int lane) {
  T* out = static_cast<T*>(p.out);
  if (c.np > 0) {
    float2 stat;
    c.odd = merge_parts<T, D>(reinterpret_cast<const float4*>(p.part_o) + c.at,
                              reinterpret_cast<const float2*>(p.part_ml) + c.at, c.first, c.np, c.ti,
                              c.row >= 0 ? out + (size_t)c.row * D : nullptr, stat);
    c.m = stat.x;
    c.l = stat.y;
    if (p.lse && c.row >= 0) p.lse[c.row] = c.m * kLn2 + logf(c.l);
  }
  // (a sum that is not finite: so is every output, by the scores that it sees)
  unsigned again = __ballot_sync(0xffffffffu, c.odd && c.row >= 0 && isfinite(c.l));
  for (__syncwarp(); again; again &= again - 1) {
    const int r = __ffs(again) - 1;
    const int at = __shfl_sync(0xffffffffu, c.row, r), pos = __shfl_sync(0xffffffffu, c.pos, r);
    const float m = __shfl_sync(0xffffffffu, c.m, r), l = __shfl_sync(0xffffffffu, c.l, r);
    recheck_row<T, D>(p, c, pos, static_cast<const T*>(p.q) + (size_t)at * D, m, l, out + (size_t)at * D, lane);
  }
}

// ---------------------------------------------------------------------------
// the partition
// ---------------------------------------------------------------------------
// Key tiles of block blk of a sequence, and its first visible key.
__device__ __forceinline__ int block_tiles(const PreParams& p, const Seq& s, int blk, int& lo) {
  const int i0 = blk * 2 * p.tpt, i1 = min(i0 + 2 * p.tpt, s.n);
  lo = paged::first_visible(s.past + i0, p.window);
  return (s.past + i1 + kBN - 1) / kBN - lo / kBN;
}
// The batch as classes of Hkv items each, in the order of the walk: the
// blocks of a sequence one by one where there are few in all (a lane then
// looks at one block), else a sequence's blocks together (a lane adds them
// up).
struct Classes {
  int nb;  // blocks of a sequence as classes of their own, 0: together
  int n;   // classes
};
__device__ __forceinline__ Classes classes_of(const PreParams& p) {
  const int r = 2 * p.tpt, nb = (min(p.v.max_new, p.v.T) + r - 1) / r;
  if ((long long)nb * p.v.B <= 1024) return Classes{nb, nb * p.v.B};
  return Classes{0, p.v.B};
}
// Units of one KV head's items of class f (0: none).
__device__ __forceinline__ long long class_units(const PreParams& p, const Classes& cl, int f, Seq& s) {
  int code, lo;
  if (cl.nb > 0) {
    const int b = f / cl.nb, blk = f - b * cl.nb;
    return paged::load_seq(p.v, b, s, code) && blk * 2 * p.tpt < s.n ? block_tiles(p, s, blk, lo) + kItemCost : 0;
  }
  if (!paged::load_seq(p.v, f, s, code)) return 0;
  long long u = 0;
  for (int blk = 0; blk * 2 * p.tpt < s.n; ++blk) u += block_tiles(p, s, blk, lo) + kItemCost;
  return u;
}

// A position in the sequence of all items' tiles: tile `off` of item (b,
// blk, kh); b == v.B is the end.
struct Pos {
  int b, blk, kh, off;
  long long start;  // the item's first unit
};

// The whole warp: the position of unit x (of the batch's W), snapped; `first`:
// the units of class `lane`.
__device__ Pos locate(const PreParams& p, const Classes& cl, long long x, int lane, long long first) {
  long long base = 0;
  for (int f0 = 0; f0 < cl.n; f0 += 32) {
    Seq s;
    const long long mine = p.Hkv * (f0 == 0 ? first : f0 + lane < cl.n ? class_units(p, cl, f0 + lane, s) : 0);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const long long total = __shfl_sync(0xffffffffu, incl, 31);
    if (x < base + total) {
      const int l = __ffs(__ballot_sync(0xffffffffu, base + incl > x)) - 1;
      Pos r{f0 + l, 0, 0, 0, 0};
      if (cl.nb > 0) {
        r.b = (f0 + l) / cl.nb;
        r.blk = f0 + l - r.b * cl.nb;
      }
      long long left = x - base - __shfl_sync(0xffffffffu, incl - mine, l);
      int code, lo;
      paged::load_seq(p.v, r.b, s, code);
      while (true) {
        const int n = block_tiles(p, s, r.blk, lo), u = n + kItemCost;
        if (left < (long long)u * p.Hkv) {
          r.kh = (int)(left / u);
          left -= (long long)r.kh * u;
          r.start = x - left;
          const int off = max(0, (int)left - kItemCost);
          r.off = off < kSnap ? 0 : n - off < kSnap ? n : off;
          return r;
        }
        left -= (long long)u * p.Hkv;
        ++r.blk;
      }
    }
    base += total;
  }
  return Pos{p.v.B, 0, 0, 0, 0};
}

// Tickets: the classes block by block from each sequence's last one back.
// (whole warp) the class of the x-th one with rows; x < all of them.
__device__ Pos nth_block(const PreParams& p, const Classes& cl, int x, int lane) {
  for (int f0 = 0; f0 < cl.n; f0 += 32) {
    const int f = f0 + lane, level = f / p.v.B, b = f - level * p.v.B;
    Seq s;
    int code, blk = -1;
    if (f < cl.n && paged::load_seq(p.v, b, s, code)) blk = (s.n + 2 * p.tpt - 1) / (2 * p.tpt) - 1 - level;
    unsigned have = __ballot_sync(0xffffffffu, blk >= 0);
    if (x < __popc(have)) {
      for (; x > 0; --x) have &= have - 1;  // the x-th set bit
      const int l = __ffs(have) - 1;
      return Pos{__shfl_sync(0xffffffffu, b, l), __shfl_sync(0xffffffffu, blk, l), 0, 0, 0};
    }
    x -= __popc(have);
  }
  return Pos{p.v.B, 0, 0, 0, 0};
}

// ---------------------------------------------------------------------------
// the attention kernel
// ---------------------------------------------------------------------------
// L2 prefetch of a query tile's box.
__device__ __forceinline__ void prefetch_4d(const CUtensorMap* map, int y, int z, int w) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(0), "r"(y), "r"(z), "r"(w)
               : "memory");
}

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
  const uint32_t q_full = sb + C::kMetaOff, q_free = q_full + 16, drain = q_full + 32;
  const uint32_t k_full = q_full + 40, k_empty = k_full + 8 * kSt;
  const uint32_t v_full = k_empty + 8 * kSt, v_empty = v_full + 8 * kSt;
  const uint32_t s_full = v_empty + 8 * kSt, p_full = s_full + 16, o_done = p_full + 16, o_free = o_done + 16;
  const uint32_t d_full = o_free + 16, d_empty = d_full + 8 * kDescs;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + C::kMetaOff + C::kNumBars * 8);
  Piece* descs = reinterpret_cast<Piece*>(smem + C::kDescOff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x, P = gridDim.x;

  pdl_launch_dependents();
  if (tid == 0) {
    mbar_init(drain, 1);
    for (int s = 0; s < kSt; ++s) {
      mbar_init(k_full + 8 * s, 1);
      mbar_init(k_empty + 8 * s, 1);
      mbar_init(v_full + 8 * s, C::kHalves);  // a producer warp per half
      mbar_init(v_empty + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + 8 * i, 1);
      mbar_init(q_free + 8 * i, 1);
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
      const Classes cl = classes_of(p);
      long long longest = 0, items = 0, first = 0;
      for (int f0 = 0; f0 < cl.n; f0 += 32) {
        Seq s;
        const long long u = f0 + lane < cl.n ? class_units(p, cl, f0 + lane, s) : 0;
        if (f0 == 0) first = u;
        W += u;
        longest = max(longest, u);
        items += u > 0;
      }
      W = warp_sum_ll(W);
      items = warp_sum_ll(items) * p.Hkv;
      // whole items by ticket: at least kTicketItems a CTA, none above a
      // kTicketPart-th of a CTA's share
      const bool tickets = cl.nb > 0 && items >= (long long)kTicketItems * P &&
                           !__any_sync(0xffffffffu, longest * kTicketPart * P > W * p.Hkv);
      W *= p.Hkv;
      if (c == 0)  // sequences that fail the checks are reported once
        for (int b = lane; b < p.v.B; b += 32) {
          Seq s;
          int code;
          paged::load_seq(p.v, b, s, code);
          if (code) record_error(p.v.err, code);
        }
      const long long Pe = max(1ll, min((long long)P, W / kMinUnits));  // CTAs with work
      Pos cur{p.v.B, 0, 0, 0, 0}, end{p.v.B, 0, 0, 0, 0};
      if (!tickets) {
        if (c < Pe) cur = locate(p, cl, c * W / Pe, lane, first);
        if (c + 1 < Pe) end = locate(p, cl, (c + 1) * W / Pe, lane, first);
      }
      int item = c;  // (tickets) the CTA's next item: the first is its own number
      int gk = 0, k = 0;
      bool ok = true;
      Seq s{};
      int sb_ = -1;       // the sequence held in s
      bool any = false;
      while (ok) {
        // the next piece: tiles [cur.off, e) of item (cur.b, cur.blk, cur.kh)
        Piece w{};
        w.b = -1;
        if (tickets) {
          if (k > 0) {
            uint32_t t = 0;
            if (lane == 0) {
              if (k == 1) epoch_install(p.ticket, p.epoch);
              t = epoch_take(p.ticket, p.epoch, p.v.err);
              if (t == (uint32_t)(items - 1)) atomicExch(p.ticket, 0ull);  // each item takes one: this is the last
            }
            t = __shfl_sync(0xffffffffu, t, 0);
            item = t == 0xFFFFFFFFu || t >= (uint32_t)items ? (int)items : P + (int)t;
          }
          cur = Pos{p.v.B, 0, 0, 0, 0};
          if (item < items) {
            cur = nth_block(p, cl, item / p.Hkv, lane);
            cur.kh = item % p.Hkv;
          }
        }
        while (cur.b < p.v.B) {
          if (sb_ != cur.b) {
            int code;
            any = paged::load_seq(p.v, cur.b, s, code);
            sb_ = cur.b;
          }
          if (!any || cur.blk * 2 * p.tpt >= s.n) {
            cur = Pos{cur.b + 1, 0, 0, 0, cur.start};
            continue;
          }
          // past the range's end?
          if (!tickets && (cur.b > end.b || (cur.b == end.b && (cur.blk > end.blk || (cur.blk == end.blk && cur.kh > end.kh))))) break;
          const bool last = !tickets && cur.b == end.b && cur.blk == end.blk && cur.kh == end.kh;
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
            if (w.slot >= 0) {
              // boundaries x (at unit floor(x W / Pe)) with kSnap tiles or
              // more of the item on either side: the first and the last
              const long long u = cur.start + kItemCost + kSnap;
              w.cf = (int)((u * Pe + W - 1) / W);
              const int cx = (int)(((u + n - 2 * kSnap + 1) * Pe + W - 1) / W) - 1;
              w.np = cx - w.cf + 2;
              if (lane < 2) epoch_install(p.arrivals + 2 * w.cf + lane, p.epoch);
            }
          }
          const long long next = cur.start + n + kItemCost;
          if (last) cur = Pos{p.v.B, 0, 0, 0, 0};
          else if (cur.kh + 1 < p.Hkv) cur = Pos{cur.b, cur.blk, cur.kh + 1, 0, next};
          else cur = Pos{cur.b, cur.blk + 1, 0, 0, next};
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
      int q1 = 0;  // loads of tile 1's queries
      bool ok = true;
      int k = 0;
      Piece w;
      for (; ok && next_piece(k, w); ++k) {
        if (is_q) {
          // tokens past the sequence's end are other rows of the batch (or
          // zeros past the arrays'): their results are never stored
          if (lane < C::kHalves * w.nact)
            prefetch_4d(&qmap, w.kh * p.G, w.q0 + w.i0 + (lane / C::kHalves) * p.tpt, lane % C::kHalves);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (i >= w.nact || !ok) break;
            // a tile's buffer is free once the score MMAs of its previous piece
            // are done (tile 0 has rows in every piece)
            const int n = i ? q1 : k;
            if (n > 0) ok = __all_sync(0xffffffffu, mbar_wait(q_free + 8 * i, (n - 1) & 1, p.v.err));
            if (lane == 0 && ok) {
              mbar_arrive_expect_tx(q_full + 8 * i, C::kHalves * p.G * p.tpt * 128);
              for (int h = 0; h < C::kHalves; ++h)
                pf::tma_load_4d(sb + C::kQOff + i * C::kTileBytes + h * kBox, &qmap, 0, w.kh * p.G,
                                w.q0 + w.i0 + i * p.tpt, h, q_full + 8 * i);
            }
          }
          if (ok && w.nact == 2) ++q1;
          __syncwarp();
          if (!ok) break;
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
      if (is_q) {
        if (k > 0) mbar_wait(q_full, (k - 1) & 1, p.v.err);
        if (q1 > 0) mbar_wait(q_full + 8, (q1 - 1) & 1, p.v.err);
      }
      if (is_v)
        for (int t = max(0, gv - kSt); t < gv; ++t) mbar_wait(v_full + 8 * (t % kSt), (t / kSt) & 1, p.v.err);
    } else {
      // ---------------- MMA issuer ----------------
      const uint32_t id_s = tc::idesc_f16(kBF16, kBM, kBN, false, false);
      const uint32_t id_o = tc::idesc_f16(kBF16, kBM, D, false, true);
      constexpr uint32_t kHi = tc::desc_hi(1024, tc::kSwizzle128B);
      // Tile i's products run P_i(j) V(j), S_i(j + 1), P_i(j + 1) V(j + 1), ...
      // across pieces: the next piece's first scores are issued with this
      // piece's last products, so no piece boundary drains the pipe.
      pdl_wait_primary();  // (so that no wait's limit counts what the previous kernel still takes)
      if (lane == 0) {
        struct Next {
          int nact, n_kv;
          bool splitp;
        };
        auto take = [&](int k, Next& w) {
          const uint32_t slot = 8 * (k % kDescs);
          if (!mbar_wait(d_full + slot, (k / kDescs) & 1, p.v.err)) return false;
          const Piece& d = descs[k % kDescs];
          const bool more = d.b >= 0;
          w = Next{d.nact, d.n_kv, kBF16 && d.past + d.i0 + 1 <= 256};
          mbar_arrive(d_empty + slot);
          return more;
        };
        auto issue_s = [&](int i, int stage, bool last) {  // S_i = Q_i K^T; the piece's last scores free its queries
          const uint32_t d = tbase + 256 * i + 128;
          const uint32_t ql = tc::desc_lo(sb + C::kQOff + i * C::kTileBytes, 16);
          const uint32_t kl = tc::desc_lo(sb + C::kKOff + stage * C::kTileBytes, 16);
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            const uint32_t off = ((x >> 2) * kBox + (x & 3) * 32) >> 4;
            tc::mma_ss(d, ql + off, kl + off, kHi, id_s, x > 0 ? 1u : 0u);
          }
          tc::commit(s_full + 8 * i);
          if (last) tc::commit(q_free + 8 * i);
        };
        auto issue_pv = [&](int i, int stage, bool first, bool splitp) {  // O_i += P_i V, P from TMEM
          const uint32_t tO = tbase + 256 * i, pa = tO + 128;
          const uint32_t vb = tc::desc_lo(sb + C::kVOff + stage * C::kTileBytes, kBox);
#pragma unroll
          for (int x = 0; x < kBN / 16; ++x)
            tc::mma_ts(tO, pa + x * 8, vb + x * (2048 >> 4), kHi, id_o, (x > 0 || !first) ? 1u : 0u);
          if (splitp)
#pragma unroll 1
            for (int x = 0; x < kBN / 16; ++x) tc::mma_ts(tO, pa + 64 + x * 8, vb + x * (2048 >> 4), kHi, id_o, 1u);
          tc::commit(o_done + 8 * i);
        };
        auto wait = [&](uint32_t bar, int n) { return mbar_wait(bar, n & 1, p.v.err); };
        int g = 0;             // key tiles, over the CTA's pieces
        int gt1 = 0, kq1 = 0;  // tile 1's score tiles and pieces (tile 0's are g and k)
        int k = 0;
        Next w{}, w2{};
        bool have = take(0, w), have2 = false, ok = true;
        if (have) {
          ok = wait(q_full, 0) && wait(k_full, 0) && (w.nact == 1 || wait(q_full + 8, 0));
          if (ok) {
            tc::fence_after();
            issue_s(0, 0, w.n_kv == 1);
            if (w.nact == 2) issue_s(1, 0, w.n_kv == 1);
            tc::commit(k_empty);
          }
        }
        while (have && ok) {
          const int two = w.nact - 1;
          for (int j = 0; j < w.n_kv && ok; ++j, ++g) {
            const int vs = g % kSt, ks = (g + 1) % kSt;
            const bool last = j + 1 == w.n_kv;
            if (last) have2 = take(k + 1, w2);
            // the scores that follow: of the next tile, or of the next piece's first
            const int next = !last ? w.nact : have2 ? w2.nact : 0;
            const bool frees = last ? w2.n_kv == 1 : j + 2 == w.n_kv;
            ok = wait(v_full + 8 * vs, g / kSt);
            for (int i = 0; i < 2 && ok; ++i) {
              if (i <= two) {
                // the first product of a piece overwrites O_i, which must have been read
                const int kq = i ? kq1 : k;
                if (!wait(p_full + 8 * i, i ? gt1 : g) || (j == 0 && kq > 0 && !wait(o_free + 8 * i, kq - 1))) { ok = false; break; }
                tc::fence_after();
                issue_pv(i, vs, j == 0, w.splitp);
                if (i == two) tc::commit(v_empty + 8 * vs);
              }
              if (i < next) {
                if ((i == 0 && !wait(k_full + 8 * ks, (g + 1) / kSt)) ||
                    (last && !wait(q_full + 8 * i, i ? kq1 + two : k + 1))) { ok = false; break; }
                tc::fence_after();
                issue_s(i, ks, frees);
                if (i + 1 == next) tc::commit(k_empty + 8 * ks);
              }
            }
            gt1 += two;
          }
          kq1 += two;
          ++k;
          w = w2;
          have = have2;
        }
        // every MMA issued has completed before TMEM is released
        tc::commit(drain);
        mbar_wait(drain, 0, p.v.err);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
    // ---------------- softmax: tile 0 (warps 4..7), tile 1 (warps 8..11) ----------------
    pdl_wait_primary();
    const int ti = (warp - 4) >> 2;
    const int row = 32 * (warp & 3) + lane;  // TMEM lane of this thread = row of the tile
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t tO = tbase + 256 * ti + lane_off;
    const uint32_t tS = tO + 128;
    const uint32_t sf = s_full + 8 * ti, pfb = p_full + 8 * ti, od = o_done + 8 * ti;
    const float sc = p.scale_log2;
    const int rt = row / p.G, rg = row - rt * p.G;  // the row's token in the tile, its head
    int gt = 0;  // score tiles of this row tile
    // The previous piece, whose output is still to be written: its rows'
    // place in the output (-1: not a row), softmax state, and partial.
    bool pending = false, pend_live = false;
    int pend_row = -1, pend_slot = -1, pend_cf = 0, pend_np = 0;
    float pend_m = 0.f, pend_l = 0.f;
    int pend_b = 0, pend_kh = 0, pend_pos = 0, pend_lo = 0, pend_hi = 0;  // (for rows that are looked at again)
    int* flag = reinterpret_cast<int*>(smem + C::kFlagOff) + ti;
    // Writes it, its products having completed; once O has been read the next
    // piece's first product may overwrite it.
    auto finish = [&]() {
      pending = false;
      const bool cut = pend_slot >= 0;
      bool in_tmem = true;  // this piece's O: in TMEM, or among the partials
      const int self = 2 * pend_slot + ti;
      // (of two parts the other: the item's first is the end of CTA cf - 1's range, the second the start of cf's)
      const int other = 2 * (pend_slot & 1 ? 2 * pend_cf : 2 * pend_cf - 1) + ti;
      float4* po = reinterpret_cast<float4*>(p.part_o) + row;  // 16-byte units of a row lie apart by the tile's 128 rows
      float2* ml = reinterpret_cast<float2*>(p.part_ml) + row;
      unsigned long long* cnt = p.arrivals + 2 * pend_cf + ti;
      float m = pend_m, l = pend_l, f = 1.f, fo = 0.f;
      if (cut) {
        // a piece of a cut item: the last one to finish merges them all
        const unsigned long long full = ((unsigned long long)p.epoch << 32) | (uint32_t)(pend_np - 1);
        if (row == 0) {
          unsigned long long v;
          asm volatile("ld.acquire.gpu.global.b64 %0, [%1];" : "=l"(v) : "l"(cnt) : "memory");
          *flag = v == full;
        }
        named_bar_sync(1 + ti, kBM);
        bool last = *flag != 0;
        named_bar_sync(1 + ti, kBM);  // (the flag is read before it is set again)
        // (the second of two that finds the first's part keeps its own in TMEM)
        if (!last || pend_np > 2) {
          in_tmem = false;
          if (pend_live) {
#pragma unroll 1
            for (int x = 0; x < D / 32; ++x) {
              uint32_t r[32];
              tc::ld32(tO + 32 * x, r);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e)
                po[((size_t)self * (D / 4) + x * 8 + e) * kBM] =
                    make_float4(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1]), __uint_as_float(r[4 * e + 2]),
                                __uint_as_float(r[4 * e + 3]));
            }
            ml[(size_t)self * kBM] = make_float2(m, l);
          }
          tc::fence_before();
          mbar_arrive(o_free + 8 * ti);  // O is read: the next piece's first product may overwrite it
          if (!last) {
            named_bar_sync(1 + ti, kBM);
            if (row == 0) {
              // release: the partial is visible before the count; acquire: the
              // last one sees the others'
              unsigned long long v;
              asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], 1;" : "=l"(v) : "l"(cnt) : "memory");
              if ((uint32_t)(v >> 32) != p.epoch) record_error(p.v.err, GQA_ERR_INVALID_ARGUMENT);  // the workspace changed under the call
              *flag = v == full;
            }
            named_bar_sync(1 + ti, kBM);
            last = *flag != 0;
            named_bar_sync(1 + ti, kBM);
            if (!last) return;
          }
        }
        if (row == 0) atomicExch(cnt, 0ull);  // ready for the next call
        if (in_tmem) {
          const float2 v = __ldcg(ml + (size_t)other * kBM);
          m = fmaxf(m, v.x);
          const float base = m == -INFINITY ? 0.f : m;
          f = fast_exp2(pend_m - base);
          fo = fast_exp2(v.x - base);
          l = __fadd_rn(__fmul_rn(pend_l, f), __fmul_rn(v.y, fo));
        }
      }
      bool odd = false;  // the row's output is not finite
      if (in_tmem) {
        const float inv = 1.f / l;
        uint8_t* stg = smem + C::kStageOff + (warp - 4) * 4096;
        // O / l goes out through the warp's stage, 32 dimensions at a time (32
        // rows of 64 bytes, 16-byte units swizzled, two buffers), so that the
        // stores to the output rows are 64 contiguous bytes.  A rolled loop: this
        // code runs once an item, so its time is that of fetching it.
        // Of a cut item in two parts the other's is loaded a step ahead, into y.
        const float4* src = po + (size_t)other * (D / 4) * kBM;
        float4 y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = cut && in_tmem ? __ldcg(src + e * kBM) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int x = 0; x < D / 32; ++x) {
          uint32_t o[32];
          tc::ld32(tO + 32 * x, o);
          tc::wait_ld();
          if (x + 1 == D / 32) {
            tc::fence_before();
            mbar_arrive(o_free + 8 * ti);
          }
          if (cut) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float z[4] = {y[e].x, y[e].y, y[e].z, y[e].w};
#pragma unroll
              for (int k = 0; k < 4; ++k)
                o[4 * e + k] = __float_as_uint(
                    __fadd_rn(__fmul_rn(__uint_as_float(o[4 * e + k]), f), __fmul_rn(z[k], fo)));
            }
            if (x + 1 < D / 32) {
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = __ldcg(src + ((x + 1) * 8 + e) * kBM);
            }
          }
          uint8_t* buf = stg + (x & 1) * 2048;
          float sum = 0.f;  // 0 * o: not 0 where some o is not finite
#pragma unroll
          for (int e = 0; e < 32; ++e) sum = fmaf(__uint_as_float(o[e]), 0.f, sum);
          odd |= sum != 0.f;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t* rr = o + 8 * u;
            uint4 v;
            v.x = E::pack2(__uint_as_float(rr[0]) * inv, __uint_as_float(rr[1]) * inv);
            v.y = E::pack2(__uint_as_float(rr[2]) * inv, __uint_as_float(rr[3]) * inv);
            v.z = E::pack2(__uint_as_float(rr[4]) * inv, __uint_as_float(rr[5]) * inv);
            v.w = E::pack2(__uint_as_float(rr[6]) * inv, __uint_as_float(rr[7]) * inv);
            *reinterpret_cast<uint4*>(buf + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4)) = v;
          }
          __syncwarp();
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int r = y * 8 + (lane >> 2), u = lane & 3;
            const int at = __shfl_sync(0xffffffffu, pend_row, r);
            const uint4 v = *reinterpret_cast<const uint4*>(buf + r * 64 + ((u ^ ((r >> 1) & 3)) << 4));
            if (at >= 0) *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (size_t)at * D + x * 32 + u * 8) = v;
          }
        }
        if (p.lse && pend_row >= 0) p.lse[pend_row] = m * kLn2 + logf(l);
      }
      if (!in_tmem || __any_sync(0xffffffffu, odd)) {
        RowCheck chk{p.Hkv, pend_b, pend_kh, pend_lo, pend_hi, p.window, sc, pend_row, pend_pos, m, l, odd,
                     in_tmem ? 0 : pend_np, pend_cf, ti, row};
        merge_and_recheck<T, D>(p, chk, lane);
      }
    };
    Piece w{};
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const bool have = next_piece(k, w);
      const bool active = have && ti < w.nact;
      if (!have && !pending) break;
      const int i = w.i0 + ti * p.tpt + rt;            // the row's token
      const bool valid = rt < p.tpt && i < w.n;
      const bool live = __any_sync(0xffffffffu, valid);  // the warp has a row to compute
      const int pos = w.past + min(i, w.n - 1);
      const int first_pos = w.past + w.i0 + ti * p.tpt;
      const int last_pos = w.past + min(w.i0 + (ti + 1) * p.tpt, w.n) - 1;
      const int all_lo = paged::first_visible(last_pos, p.window), my_lo = paged::first_visible(pos, p.window);
      const bool splitp = kBF16 && w.past + w.i0 + 1 <= 256;
      float m_ref = -INFINITY, l_run = 0.f;
      // (a tile without rows in this piece, or without a piece, only writes
      // what is pending)
      for (int j = 0; j < (active ? w.n_kv : 1); ++j) {
        const int k0 = (w.t0 + j) * kBN;
        // this tile's scores; pending without a piece: the last products
        if (!__all_sync(0xffffffffu, active ? mbar_wait(sf, gt & 1, p.v.err) : !pending || mbar_wait(od, (gt - 1) & 1, p.v.err))) {
          ok = false;
          break;
        }
        tc::fence_after();
        if (active && live) {
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
            for (int h = 0; h < 4; ++h) {  // score columns 32 h .. -> P columns 16 h ..
              uint32_t pk[16], res[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 z = fma2(make_float2(__uint_as_float(sv[h][2 * e]), __uint_as_float(sv[h][2 * e + 1])),
                                      sc2, nmu2);
                const float a = fast_exp2(z.x), bb = fast_exp2(z.y);
                rs2[e & 1] = add2(rs2[e & 1], make_float2(a, bb));
                pk[e] = E::pack2(a, bb);
                if (kSplit) {
                  const float2 hv = E::unpack2(pk[e]);
                  res[e] = E::pack2(a - hv.x, bb - hv.y);
                }
              }
              tc::st16(tS + 16 * h, pk);
              if (kSplit) tc::st16(tS + 64 + 16 * h, res);  // P's rounding residue in columns [64, 128)
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
        if (active && ti == 0 && (k0 + kBN > w.L || k0 < w.lo)) {
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
        if (active) {
          tc::fence_before();
          mbar_arrive(pfb);
          ++gt;
        }
        if (pending) finish();  // (S of this tile, or the wait above: its products have completed)
      }
      if (!ok || !have) break;
      if (active) {
        pending = true;
        pend_live = live;
        pend_row = valid ? (w.q0 + i) * p.H + w.kh * p.G + rg : -1;
        pend_b = w.b;
        pend_kh = w.kh;
        pend_pos = pos;
        pend_lo = w.lo;
        pend_hi = min(w.L, (w.past + min(w.i0 + 2 * p.tpt, w.n) + kBN - 1) / kBN * kBN);
        pend_slot = w.slot;
        pend_cf = w.cf;
        pend_np = w.np;
        pend_m = m_ref;
        pend_l = l_run;
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    tc::dealloc(tbase, kTmemCols);
  }
}

template <typename T, int D>
cudaError_t launch_d(const PagedArgs& a, const PagedPlan& plan, uint8_t* ws, uint32_t epoch) {
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
  p.q = a.q;
  p.k_pages = a.k_pages;
  p.v_pages = a.v_pages;
  p.out = a.out;
  p.lse = a.lse;
  p.part_o = reinterpret_cast<float*>(ws + plan.part_o_off);
  p.part_ml = reinterpret_cast<float*>(ws + plan.part_ml_off);
  p.arrivals = reinterpret_cast<unsigned long long*>(ws + plan.sched_off);
  p.ticket = p.arrivals + 2 * plan.ctas;
  p.epoch = epoch;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.G = G;
  p.window = a.window;
  p.tpt = tpt;
  p.pool_rows = (int)pool_rows;
  p.scale_log2 = a.scale * kLog2e;
  auto kern = paged_prefill_kernel<T, D>;
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
  return cudaLaunchKernelEx(&cfg, kern, qmap, kmap, vmap, p);
}

template <typename T>
cudaError_t launch_t(const PagedArgs& a, const PagedPlan& plan, uint8_t* ws, uint32_t epoch) {
  return a.D == 64 ? launch_d<T, 64>(a, plan, ws, epoch) : launch_d<T, 128>(a, plan, ws, epoch);
}

}  // namespace

cudaError_t launch_paged_prefill(const PagedArgs& a, const PagedPlan& plan, uint8_t* workspace, uint32_t epoch) {
  return a.dtype == GQA_DTYPE_BF16 ? launch_t<__nv_bfloat16>(a, plan, workspace, epoch)
                                   : launch_t<__half>(a, plan, workspace, epoch);
}

}  // namespace gqa
