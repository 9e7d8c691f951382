/*
 * hstu_kv.h — C ABI of the paged KV cache operators (GB300, sm_103a): writing new rows
 * into the cache that hstu_fwd_run_kv reads, reading a sequence's rows back, and softmax
 * attention of new tokens over the cache.
 *
 * The cache ("RecOps Running Case Documentation", Inputs and Outputs table, kv_cache /
 * page_offsets / page_ids / last_page_len rows): kv_cache [num_pages, 2, page_size, Nk, D],
 * plane 0 of a page holds K rows, plane 1 V rows. The pages of sequence b are
 * page_ids[page_offsets[b] .. page_offsets[b + 1]), in order, and its length is
 *   Lk = (pages - 1) * page_size + last_page_len[b]   (0 without pages).
 * For these operators the table describes the sequences with their new rows: the n rows
 * seq_offsets gives a sequence are its last n positions, Lk - n .. Lk - 1.
 *
 * Element types of the cache: fp32, fp16, bf16, or FP8 E4M3 in one of three forms,
 *   plain cast      the value of an element is its E4M3 value;
 *   static factors  k_descale / v_descale of hstu_fwd_descale's TENSOR, BATCH or HEAD
 *                   granularity: value = factor * E4M3 value (the form hstu_fwd reads);
 *   row scales      kv_scale [num_pages, 2, Nk, page_size], one unsigned byte s per page,
 *                   plane, head and row, 1 <= s <= 253: value = 2^(s - 127) * E4M3 value.
 *
 * Ownership: the caller owns every tensor, workspaces included; no entry point allocates,
 * synchronises or keeps anything between calls, so calls on different streams, and captured
 * graphs, share nothing unless the caller's tensors do. All tensor arguments are DEVICE
 * pointers on the current device. Every call is asynchronous on `stream` (a cudaStream_t;
 * NULL = legacy default stream).
 *
 * Errors are returned as hstu_status codes; nothing aborts, throws or traps. What only the
 * device can see (offsets that decrease or pass their tensors, a last_page_len outside
 * [1, page_size], more new rows than the sequence has, a length above its bound, a page id
 * outside the cache) never leads to an access outside the tensors. A sequence whose offsets
 * or lengths are invalid is left out: nothing of it is written. A row whose page id is
 * invalid is left unwritten (append, read); a sequence with such an id among its pages gets
 * unspecified attention outputs. Each sets *status (if given) to HSTU_DEVERR_OFFSETS, and a
 * pipeline wait of hstu_softmax_fwd that ran past its limit sets it to HSTU_DEVERR_TIMEOUT
 * (outputs incomplete); *status is left alone otherwise (the caller zeroes it). A call without
 * sequences or without rows (total_tokens = 0) has nothing to do and looks at nothing.
 */
#ifndef HSTU_KV_H_
#define HSTU_KV_H_

#include "hstu_fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A cache with its page table. Index arrays are int32 or int64 (index_is_int64), and so are
 * the seq_offsets that come with it. */
typedef struct {
  int dtype;             /* hstu_dtype of kv_cache */
  int batch;             /* B in [0, 2^20]; 0 = nothing to do */
  int num_heads_kv;      /* Nk in [1, 65536] */
  int head_dim;          /* D: a multiple of 16 in [16, 256] */
  int page_size;         /* 32, 128 or 256 */
  int index_is_int64;    /* 0 or 1 */
  int descale;           /* E4M3: hstu_descale_granularity of k_descale and v_descale: CAST
                            (none), TENSOR, BATCH or HEAD; CAST with kv_scale */
  int reserved;          /* must be 0 */
  void* kv_cache;        /* 16-byte aligned */
  void* kv_scale;        /* E4M3 with row scales, 16-byte aligned, or NULL */
  long long num_pages;   /* in [1, 2^30] */
  const void* page_offsets;   /* [B + 1] */
  const void* page_ids;       /* [num_page_ids], each in [0, num_pages) */
  const void* last_page_len;  /* [B], each in [1, page_size] (unused without pages) */
  long long num_page_ids;
  const float* k_descale;     /* fp32, 4-byte aligned, non-zero; [1], [B] or [B, Nk] */
  const float* v_descale;
  int* status;                /* device word for what the device finds, or NULL */
} hstu_kv_cache;

/* Rows of k and v: row t of k starts at k + t * k_stride elements and holds [Nk, D]
 * contiguously (a slice of a fused projection's output, for instance). Rows start on 16-byte
 * boundaries. seq_offsets [B + 1]: increasing from >= 0, last <= total_tokens. */
typedef struct {
  void* k;
  void* v;
  long long k_stride;     /* elements between rows, >= Nk * D */
  long long v_stride;
  const void* seq_offsets;
  long long total_tokens; /* rows of k and v; rows of no sequence are left alone */
  int dtype;              /* HSTU_F32, HSTU_F16 or HSTU_BF16; the cache's, unless that is E4M3 */
  int reserved;           /* must be 0 */
} hstu_kv_rows;

/*
 * Write the rows of k and v into the cache (k and v are only read). Rows of an E4M3 cache
 * are quantised: with row scales, s - 127 is the smallest e >= -100 for which the largest
 * finite magnitude of the row's D values is at most 448 * 2^e (-100 for a row of zeros), and
 * the code is x * 2^-e rounded to E4M3; with static factors it is x / factor rounded, and with
 * a plain cast x rounded. Rounding is to nearest even; what lies beyond +-448 (infinities
 * included) becomes +-448, a NaN stays a NaN. No page may belong to two sequences that
 * append to it in one call (the order of their writes is not defined).
 */
HSTU_API hstu_status hstu_kv_append(const hstu_kv_cache* cache, const hstu_kv_rows* rows,
                                    void* stream);

/* Read rows of the cache into k and v, dequantised and rounded to rows->dtype: the last n
 * positions of every sequence, n = its seq_offsets difference (its whole length Lk for the
 * whole sequence). k and v must not overlap. A value beyond the type's range becomes infinite:
 * quantisation may have rounded a row's largest up to 2^16 (fp16, from 63488 on) or 2^128 (bf16
 * and fp32, from 248 * 2^120 on). */
HSTU_API hstu_status hstu_kv_read(const hstu_kv_cache* cache, const hstu_kv_rows* rows,
                                  void* stream);

/*
 * Softmax attention of the queries over the cached keys. For query row i of a sequence with
 * n query rows (its position is Lk - n + i), query head h and kv head hk = h / (Nq / Nk):
 *   x_j  = alpha * sum_d q[i, h, d] * k[j, hk, d]      j < Lk, and j <= Lk - n + i if causal
 *   out[i, h, :] = sum_j exp(x_j) v[j, hk, :] / sum_j exp(x_j),   lse[i, h] = ln sum_j exp(x_j)
 * A row that sees no key (Lk = 0, or n > Lk with the causal mask) gets out = 0, lse = -inf.
 * n may exceed Lk: with causal = 0 the cached rows may be those of another sequence, of any
 * length (cross attention). The keys and values of the sequence itself are finite; rows of a
 * page beyond the sequence's end may hold anything. Rows of out and lse that belong to no
 * sequence are left alone.
 *
 * Statistics and sums are fp32. fp16 and bf16: the weights are rounded to the type of q for the
 * product with V, or to fp16 over an E4M3 cache (bf16 weights of at most 16 rows of a kv head over
 * a bf16 cache, single tokens for instance, come in two parts, whose sum is exact to 2^-16).
 * fp16 holds what is 2^-24 of the largest of the weights, or, over an E4M3 cache, of the weights
 * times their rows' scales. Rows of an E4M3 cache keep their bits whatever the scales of others,
 * but those of scale 2^-100 or less (rows of zeros) may count as zeros, and their weights with the
 * largest scale of the 127 rows around them. bf16 queries over an E4M3 cache are products of fp16
 * with a power of two of their row: elements below 2^-38 of its largest vanish.
 */
typedef struct {
  const void* q;          /* [T, Nq, D]: row t at q + t * q_stride elements, 16-byte aligned */
  long long q_stride;     /* elements, >= Nq * D, a multiple of 16 bytes */
  const void* seq_offsets;/* [B + 1] */
  long long total_tokens; /* T */
  int dtype;              /* of q and out: HSTU_F32, HSTU_F16 or HSTU_BF16; the cache's, or the
                             cache is E4M3 */
  int num_heads_q;        /* Nq >= 0, a multiple of Nk, Nq / Nk <= 128 */
  int max_seqlen;         /* bound on n, in [1, 2^24] */
  int max_seqlen_k;       /* bound on Lk, in [1, 2^30] */
  int causal;             /* 0 or 1 */
  float alpha;            /* in (0, 2e38] */
  void* out;              /* [T, Nq, D] contiguous, 16-byte aligned */
  float* lse;             /* [T, Nq], or NULL */
  void* workspace;        /* hstu_softmax_workspace bytes, 16-byte aligned; NULL if that is 0.
                             Not shared by calls that may run at the same time */
  long long workspace_bytes;
  int reserved;           /* must be 0 */
} hstu_softmax_args;

/* Bytes of workspace that hstu_softmax_fwd needs for these sizes (pointers are not read). */
HSTU_API hstu_status hstu_softmax_workspace(const hstu_kv_cache* cache,
                                            const hstu_softmax_args* args, long long* bytes);

HSTU_API hstu_status hstu_softmax_fwd(const hstu_kv_cache* cache, const hstu_softmax_args* args,
                                      void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HSTU_KV_H_ */
