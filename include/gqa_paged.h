/*
 * gqa_paged.h -- C ABI of libgqa for a PAGED key/value cache: the rows of a
 * sequence live in pages of a shared pool instead of one BNSH buffer per
 * sequence, so a server can batch sequences of different lengths without
 * reserving max_seq_len slots for each.
 *
 *   gqa_paged_append       per-head RMS norm of the new queries and keys, rotary
 *                          embedding and scatter into the pages, in one pass
 *   gqa_paged_attention    attention of the new tokens (a chunk of each sequence,
 *                          or one token each) over the pages
 *   gqa_paged_key_weights  the attention weight every cached key receives from
 *                          the new tokens, accumulated
 *   gqa_paged_evict        keeps the heaviest and the most recent tokens of every
 *                          (sequence, KV head)
 *
 * The cache.  k_pages, v_pages: T [num_pages, Hkv, page_size, D].  Slot s of
 * sequence b is row s % page_size of page block_table[b, s / page_size].  The
 * entries of block_table that hold no slot the call needs are not read (they
 * may be -1).  A needed entry outside [0, num_pages) is recorded on the device
 * as GQA_ERR_INVALID_ARGUMENT; nothing is read or written through it, and what
 * the call computes for that sequence is undefined.  Pages may be shared by
 * sequences as long as no call writes to them.
 *
 * The new tokens.  Token arrays hold total_tokens rows; sequence b owns rows
 * cu_seqlens[b] .. cu_seqlens[b + 1] - 1 (n_b of them, 0 allowed).  Rows at or
 * behind cu_seqlens[B] belong to nobody and are left as they are.  With
 * P_b = seqlens_k[b] tokens already cached, new token i of the sequence has
 * slot P_b + i.
 *
 * Masked places.  Rows of the pool that a token does not see (pages' ends, other
 * pages, slots before its window, later tokens of its own sequence) may hold
 * anything, infinities and NaN included: they do not reach its output.  (Value
 * rows that are not finite and are seen by some of a prompt's tokens only cost
 * time: the other tokens' rows are computed a second time, at a thousandth of
 * the usual rate.  With more than 100,000 slots before them the kernel's waits
 * may run out, which is GQA_ERR_TIMEOUT.)
 *
 * Checks.  What the host can see is reported before any launch.
 * total_sequence_length above 2^30 is GQA_ERR_UNSUPPORTED.  A sequence
 * with P_b < 0, n_b < 0, n_b > max_new_tokens, rows outside the token arrays
 * or P_b + n_b > total_sequence_length records GQA_ERR_INVALID_ARGUMENT on the
 * device, one with P_b + n_b > max_pages * page_size GQA_ERR_KV_OVERFLOW; such
 * a sequence is skipped entirely.
 *
 * The conventions of gqa.h hold: 16-byte aligned device pointers on the
 * current device (int32 arrays: 4 bytes), caller-owned buffers, no allocation,
 * asynchronous on `stream`, no exceptions, gqa_check_device_status() for what
 * only the device can see.  The calls can be captured into CUDA graphs.
 */
#ifndef GQA_PAGED_H_
#define GQA_PAGED_H_

#include "gqa.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int32_t batch;              /* B >= 1 sequences */
  int32_t total_tokens;       /* rows of the token arrays; >= 1, >= cu_seqlens[B] */
  int32_t max_new_tokens;     /* an upper bound on every n_b; >= 1 (gqa_paged_append ignores it) */
  int32_t num_heads;          /* H: query heads */
  int32_t kv_num_heads;       /* Hkv; H % Hkv == 0 */
  int32_t head_size;          /* D: multiple of 8, at most 256 */
  int32_t page_size;          /* slots per page: a power of two from 8 to 1024 */
  int32_t num_pages;          /* pages in the pool */
  int32_t max_pages;          /* columns of block_table */
  int32_t dtype;              /* gqa_dtype_t: element type T */
  int32_t rotary_interleaved; /* 0: dimension j pairs with j + D/2; 1: 2j with 2j + 1 */
  int32_t cos_cache_rows;     /* rows of cos/sin caches; ignored when cos_cache is NULL */
} gqa_paged_dims_t;

/*
 * gqa_paged_append -- the new rows enter the cache.
 *
 *   query            T [total_tokens, H*D], or packed QKV (key and value NULL):
 *                    T [total_tokens, (H + 2 Hkv)*D] as in gqa_forward
 *   key, value       T [total_tokens, Hkv*D], or both NULL (packed)
 *   q_norm_weight,   T [D] each, or NULL: each query (key) head x becomes
 *   k_norm_weight    x * w / sqrt(mean(x^2) + norm_eps) before the rotation
 *                    (NULL: no norm).  norm_eps >= 0, finite.
 *   cos_cache,       T [cos_cache_rows, D/2], both NULL: no rotation.
 *   sin_cache
 *   positions        int32 [total_tokens]: the rotary position of every token;
 *                    NULL: its slot P_b + i (then cos_cache_rows must be at least
 *                    total_sequence_length).  After an eviction a sequence's
 *                    slots and positions differ.  A position outside
 *                    [0, cos_cache_rows) records GQA_ERR_INVALID_ARGUMENT and that
 *                    token is skipped.
 *   query_out        T [total_tokens, H*D]: the normed, rotated queries.  May be
 *                    `query` itself when key and value are given.
 *
 * Norm and rotation are computed in fp32 and rounded to T once.  Without norm
 * weights the rows are bit for bit those of gqa_forward's append.
 */
gqa_status_t gqa_paged_append(const gqa_paged_dims_t* dims,
                              const void* query, const void* key, const void* value,
                              const void* q_norm_weight, const void* k_norm_weight, float norm_eps,
                              const void* cos_cache, const void* sin_cache, const int32_t* positions,
                              void* k_pages, void* v_pages, const int32_t* block_table,
                              const int32_t* cu_seqlens, const int32_t* seqlens_k,
                              int32_t total_sequence_length, void* query_out, void* stream);

/*
 * gqa_paged_attention -- new token i of sequence b attends over the slots
 * j <= P_b + i (its own row included: append first) and, when
 * local_window_size W > 0, j > P_b + i - W, of KV head h / (H / Hkv).
 *
 *   query            T [total_tokens, H*D], as gqa_paged_append leaves it
 *   output           T [total_tokens, H*D]
 *   lse              float [total_tokens, H], or NULL: the natural logarithm of
 *                    the sum of exp(scale * q.k) over the visible keys
 *   scale            <= 0 means 1/sqrt(D)
 *   workspace        device scratch of gqa_paged_workspace_size() bytes; calls
 *                    that can run at the same time need one each
 */
gqa_status_t gqa_paged_attention(const gqa_paged_dims_t* dims, const void* query,
                                 const void* k_pages, const void* v_pages, const int32_t* block_table,
                                 const int32_t* cu_seqlens, const int32_t* seqlens_k,
                                 int32_t total_sequence_length, float scale, int32_t local_window_size,
                                 void* output, float* lse, void* workspace, size_t workspace_bytes,
                                 void* stream);

/*
 * gqa_paged_key_weights -- for every slot j of sequence b in reach of its new
 * tokens (one of them sees it) and every KV head,
 *   weights[j] = (j < P_b ? weights_in[j] : 0)
 *                + sum over the new tokens i that see j and the H / Hkv query
 *                  heads of the KV head of exp(scale * q_i.k_j - lse_i).
 * Slots out of reach keep their weights[j].  The order of the sums is fixed:
 * equal inputs give equal bits.
 *
 *   query, lse, scale, local_window_size   as in (and from) gqa_paged_attention
 *   weights_in,      float [num_pages, Hkv, page_size], paged by block_table like
 *   weights          the keys; may be the same array
 */
gqa_status_t gqa_paged_key_weights(const gqa_paged_dims_t* dims, const void* query, const float* lse,
                                   const void* k_pages, const int32_t* block_table,
                                   const int32_t* cu_seqlens, const int32_t* seqlens_k,
                                   int32_t total_sequence_length, float scale, int32_t local_window_size,
                                   const float* weights_in, float* weights, void* workspace,
                                   size_t workspace_bytes, void* stream);

/*
 * gqa_paged_evict -- cuts every sequence to at most `budget` tokens.  Of the
 * n = seqlens_k[b] tokens of each (sequence, KV head), n > budget, the `recent`
 * last ones stay and, of the others, the budget - recent of the largest
 * weights (equal weights: the lower slot; NaN counts as the smallest).  The
 * kept tokens keep their order: their key and value rows and weights move to
 * slots 0, 1, ... of the sequence's pages in dst_block_table.  A sequence with
 * n <= budget keeps all its tokens.  Each KV head keeps its own tokens.
 *
 *   dst_block_table  int32 [B, dst_max_pages], its pages disjoint from those of
 *                    block_table that hold a slot of the call; or NULL: in place
 *                    (dst_max_pages is ignored).  In place, no page may belong to
 *                    two sequences.
 *   kept             int32 [B, Hkv, budget]: the old slots of the kept tokens,
 *                    ascending, -1 behind the last
 *   new_seqlens      int32 [B]: min(n, budget), or NULL
 *   dims             total_tokens, max_new_tokens, num_heads and the rotary
 *                    fields are ignored
 *   0 <= recent <= budget, budget >= 1.  total_sequence_length: an upper bound
 *   on every n.  A sequence that fails the checks is skipped: its kept row is
 *   -1 and its new_seqlens entry is its old length.
 */
gqa_status_t gqa_paged_evict(const gqa_paged_dims_t* dims, void* k_pages, void* v_pages, float* weights,
                             const int32_t* block_table, const int32_t* dst_block_table,
                             int32_t dst_max_pages, const int32_t* seqlens_k,
                             int32_t total_sequence_length, int32_t budget, int32_t recent,
                             int32_t* kept, int32_t* new_seqlens, void* workspace, size_t workspace_bytes,
                             void* stream);

/*
 * gqa_paged_workspace_size -- bytes of device scratch that any of the calls
 * above needs at most for these dims, total_sequence_length and
 * local_window_size on the current device; never more than for a larger
 * total_sequence_length or without a window.  0 for invalid dims (and when no
 * scratch is needed).  Only gqa_paged_attention uses scratch at present; the
 * others also take a null workspace.
 */
size_t gqa_paged_workspace_size(const gqa_paged_dims_t* dims, int32_t total_sequence_length,
                                int32_t local_window_size);

#ifdef __cplusplus
}
#endif

#endif /* GQA_PAGED_H_ */
