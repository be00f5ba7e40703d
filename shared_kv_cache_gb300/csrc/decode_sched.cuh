// Work distribution of the split-KV decode kernels with dynamic chunks: the
// partition of every (sequence, KV head) item's key tiles into chunks, the
// counters that hand chunks out and count finished ones in, and the bulk
// copies their producers use.
//
// The functions take the batch as a `Src`: its B, Hkv, P (CTAs) and
// chunks_per_cta, and tiles(b, lo, L), the key tiles of sequence b (0: skipped)
// with its keys [lo, L).
#pragma once
#include "common.cuh"

namespace gqa {
namespace dsched {

#ifndef GQA_DECODE_SHORT_TILES
#define GQA_DECODE_SHORT_TILES 24
#endif
constexpr int kShortTilesPerCta = GQA_DECODE_SHORT_TILES;  // see chunk_target

// Descriptor of one chunk, written by the producer into a staging slot.
struct ChunkDesc {
  int u;           // chunk index, -1: no more chunks
  int b, kh;       // item
  int t0, t1, tb;  // tile range [t0, t1) of the item's tb tiles
  int klo, L;      // keys [klo, L) of the item
  int slot;        // partial slot of this chunk, -1: the item is one chunk
  int first_slot;  // the item's first partial slot (its arrival counter)
  int n;           // chunks of the item
  int pad[5];
};
static_assert(sizeof(ChunkDesc) == 64, "descriptor size");

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ int warp_incl_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  return v;
}

// (epoch, count) counters.  Before its first count in a call, a user makes
// sure the word holds this call's epoch: it reads the word and, if the word
// holds another epoch (left by an earlier call, or never initialised),
// replaces exactly that value by (epoch, 0) -- one compare-and-swap, which
// fails harmlessly when another user has installed the epoch first.  Counts
// are then plain atomic additions.  The last user of the call resets the
// word to 0, before which every user has made its installation attempt.
__device__ __forceinline__ void epoch_install(unsigned long long* c, uint32_t epoch) {
  unsigned long long v;
  asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(v) : "l"(c) : "memory");
  if ((uint32_t)(v >> 32) != epoch) atomicCAS(c, v, (unsigned long long)epoch << 32);
}
// Returns the count before this one, or 0xFFFFFFFF (recorded as a device
// error) if the word does not hold this call's epoch.
__device__ __forceinline__ uint32_t epoch_take(unsigned long long* c, uint32_t epoch, int* err) {
  const unsigned long long old = atomicAdd(c, 1ull);
  if ((uint32_t)(old >> 32) != epoch) {
    record_error(err, GQA_ERR_INVALID_ARGUMENT);  // the workspace changed under the call
    return 0xFFFFFFFFu;
  }
  return (uint32_t)old;
}

__device__ __forceinline__ void bulk_prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// Chunks the partition aims at for T tiles in all.  A short call (at most
// kShortTilesPerCta tiles per CTA on average) takes one chunk per CTA: each
// chunk boundary and each split item's merge costs more than the balance that
// more chunks buy there.  Longer calls take p.chunks_per_cta chunks per CTA, so
// that the chunk tickets can even out the CTAs' end times.
template <class Src>
__device__ __forceinline__ int chunk_target(const Src& p, int T) {
  return T <= kShortTilesPerCta * p.P ? p.P : p.chunks_per_cta * p.P;
}

// The partition, computed identically by every producer warp: the chunk
// size C, and each item's chunks in two groups -- its whole chunks of C
// tiles, then (when C does not divide its tiles) one shorter remainder chunk.
// Chunks are numbered all whole chunks first, then all remainders, so the
// chunks handed out last by the ticket are the short ones and the CTAs'
// end times stay close.  In a batch of at most 32 sequences the remainders
// go longest first (ties: lower sequence first), so that the very last ones
// are the shortest.  An item of n >= 2 chunks keeps n partial slots, whole
// chunks first.
struct Partition {
  int C;
  int UA, U;  // whole chunks; all chunks
};
__device__ __forceinline__ void item_chunks(int C, int tb, int& nA, int& nB) {
  nA = tb / C;
  nB = tb - nA * C > 0 ? 1 : 0;
}
template <class Src>
__device__ Partition make_partition(const Src& p, int lane) {
  int T = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    int lo, L;
    const int b = b0 + lane;
    T += warp_sum(b < p.B ? p.tiles(b, lo, L) : 0);
  }
  T *= p.Hkv;
  const int target = chunk_target(p, T);
  Partition pt{max(2, (T + target - 1) / target), 0, 0};
  int UA = 0, UB = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    int lo, L, nA, nB;
    const int b = b0 + lane;
    item_chunks(pt.C, b < p.B ? p.tiles(b, lo, L) : 0, nA, nB);
    UA += warp_sum(nA);
    UB += warp_sum(nB);
  }
  pt.UA = UA * p.Hkv;
  pt.U = (UA + UB) * p.Hkv;
  return pt;
}

// The first remainder chunk of lane's sequence when a batch of at most 32
// sequences takes its remainders longest first: the remainders (`ch` chunks
// of `rlen` tiles per lane) of every lane that sorts before this one.
__device__ __forceinline__ int rem_sorted_start(int rlen, int ch, int lane) {
  int start = 0;
#pragma unroll 8
  for (int i = 0; i < 32; ++i) {
    const int ri = __shfl_sync(0xffffffffu, rlen, i);
    const int ci = __shfl_sync(0xffffffffu, ch, i);
    if (ri > rlen || (ri == rlen && i < lane)) start += ci;
  }
  return start;
}

// Chunk u within one block of 32 sequences b0 + lane.  Each lane brings its
// sequence's tile count, key range and chunk counts; incl / sincl are the
// block's inclusive scans of this group's chunks and of partial slots, cbase
// / sbase those of earlier blocks; v counts chunks within the group.  With
// `sorted` (remainders of a batch of at most 32 sequences) the group is in
// the longest-first order instead of the sequence order.
__device__ __forceinline__ ChunkDesc chunk_in_block(const Partition& pt, int u, int v, bool rem,
                                                    int b0, int tb, int lo, int L, int nA, int nB, int ch, int sl_n,
                                                    int incl, int sincl, int cbase, int sbase, bool sorted) {
  int l, c0;
  if (rem && sorted) {
    const int st = rem_sorted_start(nB ? tb - nA * pt.C : 0, ch, threadIdx.x & 31);
    l = __ffs(__ballot_sync(0xffffffffu, ch > 0 && st <= v && v < st + ch)) - 1;
    c0 = __shfl_sync(0xffffffffu, st, l);
  } else {
    l = __ffs(__ballot_sync(0xffffffffu, cbase + incl > v)) - 1;
    c0 = cbase + __shfl_sync(0xffffffffu, incl - ch, l);
  }
  ChunkDesc d;
  d.b = b0 + l;
  const int s0 = sbase + __shfl_sync(0xffffffffu, sincl - sl_n, l);
  d.tb = __shfl_sync(0xffffffffu, tb, l);
  d.klo = __shfl_sync(0xffffffffu, lo, l);
  d.L = __shfl_sync(0xffffffffu, L, l);
  const int na = __shfl_sync(0xffffffffu, nA, l), nb = __shfl_sync(0xffffffffu, nB, l);
  d.n = na + nb;
  const int np = rem ? nb : na;  // this group's chunks of each of the sequence's items
  const int r = v - c0;
  d.kh = r / np;
  const int k = r - d.kh * np;
  d.t0 = rem ? na * pt.C : k * pt.C;
  d.t1 = rem ? d.tb : d.t0 + pt.C;
  d.u = u;
  d.first_slot = d.n > 1 ? s0 + d.kh * d.n : -1;
  d.slot = d.n > 1 ? d.first_slot + (rem ? na : k) : -1;
  return d;
}

// Batches of at most 32 sequences: the partition and chunk u (u < 0: none)
// in one warp pass; sequence lane has tb tiles (0 past the batch) over the
// keys [lo, L).
template <class Src>
__device__ ChunkDesc partition_and_locate_small(const Src& p, int tb, int lo, int L, int u, int lane, Partition& pt) {
  const int T = warp_sum(tb) * p.Hkv;
  const int target = chunk_target(p, T);
  pt.C = max(2, (T + target - 1) / target);
  int nA, nB;
  item_chunks(pt.C, tb, nA, nB);
  pt.UA = warp_sum(nA) * p.Hkv;
  pt.U = pt.UA + warp_sum(nB) * p.Hkv;
  if (u < 0 || u >= pt.U) {
    ChunkDesc d{};
    d.u = -1;
    return d;
  }
  const bool rem = u >= pt.UA;
  const int v = rem ? u - pt.UA : u;
  const int ch = (rem ? nB : nA) * p.Hkv;
  const int sl_n = nA + nB > 1 ? (nA + nB) * p.Hkv : 0;
  const int incl = warp_incl_scan(ch, lane);
  const int sincl = warp_incl_scan(sl_n, lane);
  return chunk_in_block(pt, u, v, rem, 0, tb, lo, L, nA, nB, ch, sl_n, incl, sincl, 0, 0, true);
}

// Warp-cooperative: the item and tile range of chunk u (< U).
template <class Src>
__device__ ChunkDesc locate_chunk(const Src& p, const Partition& pt, int u, int lane) {
  const bool rem = u >= pt.UA;
  const int v = rem ? u - pt.UA : u;
  int cbase = 0, sbase = 0;  // this group's chunks and partial slots of the sequences before b0
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    int lo, L, nA, nB;
    const int b = b0 + lane;
    const int tb = b < p.B ? p.tiles(b, lo, L) : 0;
    item_chunks(pt.C, tb, nA, nB);
    const int ch = (rem ? nB : nA) * p.Hkv;
    const int sl_n = nA + nB > 1 ? (nA + nB) * p.Hkv : 0;
    const int incl = warp_incl_scan(ch, lane);
    const int sincl = warp_incl_scan(sl_n, lane);
    const int chunk_total = __shfl_sync(0xffffffffu, incl, 31);
    if (v < cbase + chunk_total)
      return chunk_in_block(pt, u, v, rem, b0, tb, lo, L, nA, nB, ch, sl_n, incl, sincl, cbase, sbase, p.B <= 32);
    cbase += chunk_total;
    sbase += __shfl_sync(0xffffffffu, sincl, 31);
  }
  ChunkDesc d{};
  d.u = -1;
  return d;
}

}  // namespace dsched
}  // namespace gqa
