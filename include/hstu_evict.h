/*
 * hstu_evict.h — C ABI of eviction from a paged KV cache (GB300, sm_103a): the attention weight
 * that every cached key has received, the choice of the rows to keep by it, and moving those
 * together. hstu_kv.h has the cache, its page table and the attention over it.
 *
 * A step of a serving loop: hstu_kv_append (with the weights, whose entries of the new rows become
 * 0), hstu_softmax_fwd (with lse), hstu_kv_weights with that lse; and where a cache has to become
 * shorter, hstu_kv_select and hstu_kv_compact, after which the tables that hstu_kv_select has written
 * describe it. Pages that they no longer name are free.
 *
 * Ownership, streams, errors and what only the device can see are as in hstu_kv.h: nothing is
 * allocated, synchronised or kept between calls, status codes are returned, and an invalid sequence
 * is left out. For these calls no page may belong to two sequences or twice to one.
 */
#ifndef HSTU_EVICT_H_
#define HSTU_EVICT_H_

#include "hstu_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Attention weights of the cached keys. For key j of a sequence with n queries and Lk keys, and kv
 * head hk, the sum over the queries i that see j (all, or j <= Lk - n + i if causal) and the heads h
 * of hk (h / (Nq / Nk) = hk) of
 *   exp(alpha * sum_d q[i, h, d] * k[j, hk, d] - lse[i, h])
 * is added to weights[page, hk, row of j], or stored there. (Rows behind those that hstu_kv_compact has
 * moved together, and rows of pages that are used again, have entries of earlier rows until
 * hstu_kv_append, with the weights, sets them to 0.) Every cached row of a valid sequence
 * takes part: where no query sees it, 0 is added or stored. Elements of weights that belong to no
 * cached row are left alone; a key that holds an infinity or a NaN may be given a NaN. Scores and
 * sums are fp32, products exact (bf16 queries over an E4M3 or E2M1 cache: as hstu_softmax_fwd has
 * them, or exact). The result does not depend on the order in which anything runs.
 */
typedef struct {
  const void* q;          /* as in hstu_softmax_args */
  long long q_stride;
  const void* seq_offsets;
  long long total_tokens; /* T; without tokens q and lse may be NULL */
  int dtype;
  int num_heads_q;
  int max_seqlen;
  int max_seqlen_k;
  int causal;
  float alpha;
  const float* lse;       /* [T, Nq], 4-byte aligned: hstu_softmax_fwd's */
  float* weights;         /* [num_pages, Nk, page_size], 16-byte aligned */
  int accumulate;         /* 1: add, 0: store */
  int reserved;           /* must be 0 */
} hstu_weights_args;

HSTU_API hstu_status hstu_kv_weights(const hstu_kv_cache* cache, const hstu_weights_args* args,
                                     void* stream);

/*
 * Which rows to keep. Of every sequence (length Lk) and kv head, keep = min(Lk, budget) positions:
 * the last min(recent, keep), and those of the largest weights among the others; of equal weights
 * the lower position, and a NaN counts as less than any weight. kept holds them in increasing
 * order, -1 behind them.
 *
 * new_page_offsets, new_last_page_len and new_page_ids describe the sequences once their kept rows
 * lie at positions 0 .. keep - 1: the first pages of each, without gaps; -1 behind the last id
 * (and in place of ids of a sequence whose table is invalid, which keeps no page). Where
 * sequences share entries of page_ids and the new table would be longer than that array, this is
 * reported, and the new table invalid from there on.
 */
typedef struct {
  int batch;              /* as in hstu_kv_cache */
  int num_heads_kv;
  int page_size;
  int index_is_int64;
  long long num_pages;
  const void* page_offsets;
  const void* page_ids;
  const void* last_page_len;
  long long num_page_ids;
  const float* weights;   /* [num_pages, Nk, page_size], 16-byte aligned */
  int budget;             /* in [1, 2^30] */
  int recent;             /* in [0, 2^30] */
  int max_seqlen_k;       /* bound on Lk, in [1, 2^30] */
  int reserved;           /* must be 0 */
  int* kept;              /* [B, Nk, budget] */
  void* new_page_offsets; /* [B + 1], [num_page_ids] and [B], of the index type; */
  void* new_page_ids;     /* none of them may overlap the table that is read */
  void* new_last_page_len;
  int* status;
} hstu_select_args;

HSTU_API hstu_status hstu_kv_select(const hstu_select_args* args, void* stream);

/*
 * Move rows together, in place: position r of every sequence and kv head takes the K and V row
 * (scales and factors too, and its entry of weights, if given) that position kept[b, hk, r] holds,
 * for r = 0, 1, .. as long as kept[b, hk, r] >= 0 (at most budget). cache describes the sequences as
 * they were. Positions increase with r (hstu_kv_select's do); a list where they do not, or pass the
 * sequence's length, is reported and ends there. Other rows are left as they are, and so are their
 * entries of weights: hstu_kv_append sets those of the rows that come next to 0. Where *status becomes
 * HSTU_DEVERR_TIMEOUT, rows are moved in part: what the sequences hold is lost.
 */
typedef struct {
  const int* kept;        /* [B, Nk, budget], 4-byte aligned */
  int budget;             /* in [1, 2^30] */
  int max_seqlen_k;       /* bound on Lk, in [1, 2^30] */
  float* weights;         /* [num_pages, Nk, page_size], 16-byte aligned, or NULL */
  void* workspace;        /* hstu_compact_workspace bytes, 16-byte aligned; NULL if that is 0. Not
                             shared by calls that may run at the same time */
  long long workspace_bytes;
  int reserved;           /* must be 0 */
} hstu_compact_args;

/* Bytes of workspace that hstu_kv_compact needs for these sizes (pointers are not read). */
HSTU_API hstu_status hstu_compact_workspace(const hstu_kv_cache* cache,
                                            const hstu_compact_args* args, long long* bytes);

HSTU_API hstu_status hstu_kv_compact(const hstu_kv_cache* cache, const hstu_compact_args* args,
                                     void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HSTU_EVICT_H_ */
