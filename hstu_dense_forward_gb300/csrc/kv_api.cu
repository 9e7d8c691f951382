// C ABI of the paged KV cache operators: argument checks, the choice of kernel and of the
// number of key ranges, and launches. See include/hstu_kv.h for the contracts.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/hstu_kv.h"
#include "kv_cache.cuh"
#include "kv_checks.h"
#include "kv_kernels.h"

using namespace hstu;

namespace {

hstu_status copy_rows(const hstu_kv_cache* c, const hstu_kv_rows* r, bool append, void* stream) {
  const hstu_status st = check_cache(c);
  if (st != HSTU_OK) return st;
  if (!r || !row_dtype_ok(c, r->dtype)) return HSTU_ERR_INVALID_ARG;
  const bool more = append && r->reserved == HSTU_ROWS_WEIGHTS;  // (fields behind `reserved`)
  if (r->reserved && !more) return HSTU_ERR_INVALID_ARG;
  float* weights = more ? r->weights : nullptr;
  if (r->total_tokens < 0 || r->total_tokens > 0x7fffffffll) return HSTU_ERR_INVALID_ARG;
  if (c->batch == 0 || r->total_tokens == 0) return HSTU_OK;
  const long long width = (long long)c->num_heads_kv * c->head_dim;
  const int eb = elem_bytes(r->dtype);
  if (!r->k || !r->v || !aligned(r->k, 16) || !aligned(r->v, 16) || !r->seq_offsets ||
      !aligned(r->seq_offsets, c->index_is_int64 ? 8 : 4) || r->k_stride < width ||
      r->v_stride < width || r->k_stride * eb % 16 != 0 || r->v_stride * eb % 16 != 0 ||
      r->k_stride > (1ll << 40) || r->v_stride > (1ll << 40) || !cache_pointers_ok(c) ||
      !aligned(weights, 16) || (!append && r->k == r->v))  // (one place for both planes)
    return HSTU_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !device_sms(dev, &sms)) return HSTU_ERR_CUDA;
  const hstu::CacheView v = cache_view(c, r->seq_offsets, r->total_tokens);
  return hstu::launch_kv_copy(v, r->k, r->v, r->k_stride, r->v_stride, weights, r->dtype,
                              cache_format(c->dtype), append, sms,
                              static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? HSTU_OK
             : HSTU_ERR_CUDA;
}

// How a call runs: query rows of one CTA, key ranges, grid and workspace.
struct AttnPlan {
  enum { SIMT, TC, ROWS } kernel;
  int qtiles, ctas;    // query tiles of one CTA, CTAs of one SM (TC)
  int rows;            // query rows of one item (SIMT, ROWS)
  int cluster;         // CTAs that divide the keys of one item (ROWS)
  int by_length;       // CTAs of a round (ROWS)
  int balanced;        // CTAs share the items' key tiles (TC)
  int splits, min_range;
  long long tiles, blocks, workspace, parts_bytes;
};

// Whether CTAs share few items' key tiles: one CTA per SM takes an equal share. With a CTA for each
// item the longest takes its keys times the rounds of CTAs that the items make; shared out the
// work takes the part of that which the SMs have in the mean (three quarters: sequences are
// shorter than the bound), plus some 15 us for the items' table, for what borders part, and for
// the second kernel, the time of 2000 keys (head dims above 128, whose key tiles hold half as
// many: 3200). Measured so: two sequences of 300 tokens over 1300 keys 29 us alone, 32 shared,
// over 2300 43 and 35, over 4400 72 and 41; 208 items of 8000 keys 128 and 107; but 270 items of
// 3000 97 and 105: from 1.5 rounds on the SMs are filled well enough.
bool parting_pays(long long keys, long long items, long long sms, int head_dim) {
  const long long rounds = (items + sms - 1) / sms;
  return items * 2 < 3 * sms &&
         keys * (4 * rounds * sms - 3 * items) >= (head_dim > 128 ? 3200 : 2000) * 4 * sms;
}

// Row tiles and CTAs of the tensor-core kernel (times of bf16, D = 128, unless they say more).
template <typename SetRows>
void plan_tiles(const hstu_kv_cache* c, const hstu_softmax_args* a, long long most, long long G,
                long long sms, const SetRows& set_rows, const long long& bm,
                const long long& items, AttnPlan* pl) {
  const long long tile = 128 / G * G;
  const bool codes = cache_format(c->dtype) != hstu::kSame, small = c->head_dim <= 128;
  // Two query tiles share the loads of K and V and keep the tensor pipe busier, if there are rows
  // for both (4096 tokens over 4096, 16 heads of 4: 660 us with two, 712 with one; 64 sequences of
  // some 200 rows over 2500 keys: 141 and 126)
  pl->qtiles = small && most > 128 / G && a->total_tokens * G / c->batch >= 256 ? 2 : 1;
  pl->ctas = 1;
  set_rows(pl->qtiles * tile);
  if (c->batch <= hstu::kMaxSeqs && a->total_tokens * G / bm + c->batch <= hstu::kMaxItems &&
      parting_pays(a->max_seqlen_k, items, sms, c->head_dim)) {
    pl->balanced = 1;
    pl->blocks = sms;
    pl->parts_bytes = 2 * pl->blocks * pl->qtiles * 128 * (c->head_dim + 1) * 4;
    pl->workspace = pl->parts_bytes + pl->blocks * (long long)sizeof(hstu::JoinRecord);
    return;
  }
  if (small && !codes && (pl->qtiles == 1 || a->max_seqlen_k <= 4096)) {
    // A CTA for each item, two on an SM if there are as many: with short keys what hides an item's
    // first and last steps is another item (24 sequences of some 500 rows over 900 keys, D = 64:
    // 49 us with two query tiles, 46 with two CTAs; 32 of 400 over 1400 120 and 109; with longer
    // keys they come out even: 16 of 2048 over 4600 146 and 146). With no more items than SMs one
    // CTA with two score buffers is faster (8 sequences of 200 rows over 600 keys: 13.2 and 14.8).
    pl->qtiles = 1;
    set_rows(tile);
    pl->ctas = items > sms ? 2 : 1;
  }
  // Short keys: a CTA takes several items, whose first loads and last stores overlap, too (155
  // sequences of up to 21 rows over 120 keys, eight heads: 33 us, with a CTA for each item 43;
  // but of up to 600 keys, uneven items, 60 sequences of 400 rows 59 and 54)
  if (pl->qtiles == 1 && a->max_seqlen_k <= 256 && pl->blocks > sms * pl->ctas)
    pl->blocks = sms * pl->ctas;
}

hstu_status plan_attention(const hstu_kv_cache* c, const hstu_softmax_args* a, AttnPlan* pl) {
  const hstu_status st = check_cache(c);
  if (st != HSTU_OK) return st;
  if (!a || a->reserved || !row_dtype_ok(c, a->dtype)) return HSTU_ERR_INVALID_ARG;
  if (a->total_tokens < 0 || a->total_tokens > 0x7fffffffll || a->num_heads_q < 0 ||
      a->num_heads_q % c->num_heads_kv != 0)
    return HSTU_ERR_INVALID_ARG;
  if (a->max_seqlen < 1 || a->max_seqlen > (1 << 24) || a->max_seqlen_k < 1 ||
      a->max_seqlen_k > (1 << 30) || (a->causal != 0 && a->causal != 1) ||
      !(a->alpha > 0.0f) || !(a->alpha <= 2e38f))  // (times log2 e it stays finite)
    return HSTU_ERR_INVALID_ARG;
  const long long G = a->num_heads_q / c->num_heads_kv;
  if (G > 128) return HSTU_ERR_UNSUPPORTED;
  *pl = AttnPlan{};
  pl->splits = 1;
  pl->min_range = 128;
  if (c->batch == 0 || a->total_tokens == 0 || G == 0) return HSTU_OK;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !device_sms(dev, &sms)) return HSTU_ERR_CUDA;
  const long long most = a->max_seqlen < a->total_tokens ? a->max_seqlen : a->total_tokens;
  // query rows (token, head) of one item (a CTA's, or a cluster's); row tiles that hold rows: at
  // most one partly filled tile a sequence
  long long bm = 0, items = 0;
  auto set_rows = [&](long long rows) {
    bm = rows;
    pl->tiles = (most * G + bm - 1) / bm;
    pl->blocks = c->batch * pl->tiles * c->num_heads_kv;
    items = a->total_tokens * G / bm + c->batch;
    if (items > c->batch * pl->tiles) items = c->batch * pl->tiles;
    items *= c->num_heads_kv;
  };
  if (a->dtype == HSTU_F32) {
    // up to 16 rows in CTAs of four, which read the keys' rows straight into registers (tiles of
    // 16 rows in shared memory instead: 128 sequences of one token and eight heads 1334 us, now
    // 288; with 16 rows a kv head 235 and 136, over E4M3 221 and 145)
    pl->kernel = AttnPlan::SIMT;
    pl->rows = most * G <= 16 ? 4 : 64;
    set_rows(pl->rows);
  } else if (most * G <= 16) {
    pl->kernel = AttnPlan::ROWS;
    pl->rows = most * G <= 8 ? 8 : 16;
    set_rows(pl->rows);
  } else {
    pl->kernel = AttnPlan::TC;
    plan_tiles(c, a, most, G, sms, set_rows, bm, items, pl);
  }
  if (c->batch * pl->tiles * c->num_heads_kv > 0x7fffffffll / 8) return HSTU_ERR_UNSUPPORTED;
  pl->cluster = 1;
  if (pl->kernel == AttnPlan::ROWS) {
    // at most one wave of CTAs: more of them, of fewer keys each, measured slower (four sequences
    // of 100k bf16 keys: 74.5 us with one wave, 83.8 with two, 101 with four; 400 items of up to
    // 500 E4M3 keys on 456 places: 13.7 us alone, 20.2 in pairs)
    const long long slots =
        (long long)hstu::softmax_rows_ctas(c->head_dim, cache_format(c->dtype), pl->rows) * sms;
    const long long can = (a->max_seqlen_k + 127) / 128;  // two tiles of 64 keys each
    long long want = slots / items < can ? slots / items : can;
    if (want < 1) want = 1;
    while (pl->cluster < 8 && pl->cluster * 2 <= want) pl->cluster *= 2;
    pl->splits = (int)(want / pl->cluster);
    // E2M1: a cluster's CTAs lie in one group of SMs, whose number eight CTAs do not divide, so that the
    // last clusters of a full wave wait for a second one. Seven eighths of the wave fit (eight items of
    // 100k keys: 8 x 7 CTAs each 73 us, 8 x 6 53; one 40 and 31, four 43 and 32). Of few CTAs an item that
    // may be half of them, and those of clusters of two all fit, but their many ranges cost some 2 us to
    // join (items of 100k keys: 12 with 8 x 4 CTAs each 72, 2 x 19 65; 16 8 x 3 91, 2 x 14 81; 25 8 x 1
    // 186, 8 x 2 128, 2 x 9 118; 28 8 x 1 179, 8 x 2 183, 2 x 8 126; 36 8 x 1 179, 2 x 6 168. Of 40k keys:
    // 16 36 and 35, 25 67 and 49; of 20k: 16 25.1 and 25.8, 24 29 and 30, 28 36 and 31). The bf16
    // kernel's numbers are multiples that fit as they are.
    if (c->dtype == HSTU_FP4_E2M1 && pl->cluster == 8) {
      if (a->max_seqlen_k >= 32768 && want >= 12 && want < 48) {
        pl->cluster = 2;
        pl->splits = (int)(want / 2);
      } else if (pl->splits > 1) {
        pl->splits = (int)(want * 7 / 64);
      }
    }
    pl->min_range = 128 * pl->cluster;
    if (pl->cluster == 1 && pl->splits == 1 && pl->rows == 8 && c->head_dim <= 128)
      pl->by_length = rows_by_length(c->batch, pl->blocks, sms, c->num_page_ids, c->page_size,
                                     a->max_seqlen_k);
  } else if (pl->kernel == AttnPlan::SIMT) {
    pl->min_range = 128;
    // resident CTAs: four an SM; of four rows three, in two waves (25 sequences of some 7500 keys,
    // five rows: 166 us with one wave, 142 with two, 146 with four)
    const long long want = ((pl->rows == 64 ? 4ll : 6ll) * sms + items - 1) / items;
    const long long can = (a->max_seqlen_k + pl->min_range - 1) / pl->min_range;
    pl->splits = (int)(want < can ? want : can);
  }
  if (pl->splits > 1) {
    pl->parts_bytes = (long long)pl->splits * a->total_tokens * a->num_heads_q *
                      (c->head_dim + 1) * 4;
    pl->workspace = pl->parts_bytes;
  }
  return HSTU_OK;
}

// An E2M1 cache whose pages are turned into bf16 ones first (see expand.cu): for bf16 queries of 768
// packed rows a sequence in the mean, three of the attention kernel's items (16 sequences of 256
// tokens, four heads to a kv head: 121 us so, 147 without; of 128 tokens 88 and 86; one head to a kv head,
// of 768 tokens over 8000 keys at D = 64 116 and 150), and of 2048 rows above D = 128, whose kernel waits
// less for the conversion (16 sequences of 768 rows over 8000 keys, D = 256: 374 us so, 266 without; four
// of 1536 over 30,000 518 and 425, 16 over 8000 484 and 547, of 4096 980 and 1220), as long as the pages that batch and max_seqlen_k allow take a gigabyte at most. (What page_ids holds besides has no
// part in it: the weights are bf16 here and fp16 without.)
struct Expanded {
  long long ids, pages;  // bytes
  long long per;         // pages of a sequence at most
  bool by_entry;         // a place for every entry of page_ids; or `per` for every sequence
  hstu_kv_cache cache;
};
bool expand_pays(const hstu_kv_cache* c, const hstu_softmax_args* a, Expanded* e) {
  if (!c || !a || c->dtype != HSTU_FP4_E2M1 || a->dtype != HSTU_BF16 || c->batch < 1 ||
      c->num_heads_kv < 1 || a->num_heads_q < 1 || c->num_page_ids < 1 ||
      c->num_page_ids > (1ll << 40) || a->total_tokens > 0x7fffffffll || a->max_seqlen_k < 1 ||
      check_cache(c) != HSTU_OK)
    return false;
  const long long rows = a->total_tokens * (a->num_heads_q / c->num_heads_kv);
  const long long page = 4ll * c->page_size * c->num_heads_kv * c->head_dim;
  e->per = ((long long)a->max_seqlen_k + c->page_size - 1) / c->page_size;
  const long long most = c->batch * e->per;
  if (rows < (c->head_dim > 128 ? 2048ll : 768ll) * c->batch || most > (1ll << 30) / page)
    return false;
  e->by_entry = c->num_page_ids <= most;
  e->ids = (c->num_page_ids * (c->index_is_int64 ? 8 : 4) + 15) / 16 * 16;
  e->cache = *c;
  e->cache.dtype = HSTU_BF16;
  e->cache.kv_scale = nullptr;
  e->cache.num_pages = e->by_entry ? c->num_page_ids : most;
  e->pages = e->cache.num_pages * page;
  return true;
}

hstu_status softmax_over(const hstu_kv_cache* c, const hstu_softmax_args* a, void* stream);

// The rows' tensors (not the workspace).
bool attn_pointers_ok(const hstu_kv_cache* c, const hstu_softmax_args* a) {
  return a->q && a->out && a->seq_offsets && aligned(a->q, 16) && aligned(a->out, 16) &&
         aligned(a->lse, 4) && aligned(a->seq_offsets, c->index_is_int64 ? 8 : 4) &&
         a->q_stride >= (long long)a->num_heads_q * c->head_dim && a->q_stride <= (1ll << 36) &&
         a->q_stride * elem_bytes(a->dtype) % 16 == 0;
}

}  // namespace

extern "C" {

hstu_status hstu_kv_append(const hstu_kv_cache* cache, const hstu_kv_rows* rows, void* stream) {
  return copy_rows(cache, rows, true, stream);
}

hstu_status hstu_kv_read(const hstu_kv_cache* cache, const hstu_kv_rows* rows, void* stream) {
  return copy_rows(cache, rows, false, stream);
}

hstu_status hstu_softmax_workspace(const hstu_kv_cache* cache, const hstu_softmax_args* args,
                                   long long* bytes) {
  if (!bytes) return HSTU_ERR_INVALID_ARG;
  *bytes = 0;
  AttnPlan pl;
  hstu_status st = plan_attention(cache, args, &pl);
  Expanded e;
  if (st == HSTU_OK && pl.blocks > 0 && expand_pays(cache, args, &e)) {
    st = plan_attention(&e.cache, args, &pl);
    pl.workspace += e.ids + e.pages;
  }
  if (st == HSTU_OK) *bytes = pl.workspace;
  return st;
}

hstu_status hstu_softmax_fwd(const hstu_kv_cache* c, const hstu_softmax_args* a, void* stream) {
  Expanded e;
  long long need = 0;
  if (!expand_pays(c, a, &e)) return softmax_over(c, a, stream);
  const hstu_status st = hstu_softmax_workspace(c, a, &need);
  if (st != HSTU_OK) return st;
  if (a->workspace_bytes < need) return softmax_over(c, a, stream);  // (the caller's choice)
  if (!cache_pointers_ok(c) || !attn_pointers_ok(c, a) || !a->workspace ||
      !aligned(a->workspace, 16))
    return HSTU_ERR_INVALID_ARG;
  hstu_softmax_args b = *a;
  char* at = static_cast<char*>(a->workspace);
  e.cache.page_ids = at;
  e.cache.kv_cache = at + e.ids;
  b.workspace = need > e.ids + e.pages ? at + e.ids + e.pages : nullptr;
  b.workspace_bytes = a->workspace_bytes - e.ids - e.pages;
  if (launch_expand(cache_view(c, a->seq_offsets, a->total_tokens), e.cache.kv_cache, at, e.per,
                    e.by_entry, static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return HSTU_ERR_CUDA;
  return softmax_over(&e.cache, &b, stream);
}

}  // extern "C"

namespace {

hstu_status softmax_over(const hstu_kv_cache* c, const hstu_softmax_args* a, void* stream) {
  AttnPlan pl;
  const hstu_status st = plan_attention(c, a, &pl);
  if (st != HSTU_OK) return st;
  if (pl.blocks == 0) return HSTU_OK;  // empty input
  if (!attn_pointers_ok(c, a) || !cache_pointers_ok(c)) return HSTU_ERR_INVALID_ARG;
  if (pl.workspace > 0 &&
      (!a->workspace || !aligned(a->workspace, 16) || a->workspace_bytes < pl.workspace))
    return HSTU_ERR_INVALID_ARG;
  hstu::SoftmaxParams p = {};
  p.c = cache_view(c, a->seq_offsets, a->total_tokens);
  p.q = a->q;
  p.out = a->out;
  p.lse = a->lse;
  p.q_stride = a->q_stride;
  p.Nq = a->num_heads_q;
  p.G = a->num_heads_q / c->num_heads_kv;
  p.max_q = a->max_seqlen;
  p.max_k = a->max_seqlen_k;
  p.causal = a->causal;
  p.scale_log2 = (float)((double)a->alpha * 1.4426950408889634);
  p.splits = pl.splits;
  p.min_range = pl.min_range;
  p.timeout_ns = 1000000000ll;
  p.balanced = pl.balanced;
  p.by_length = pl.by_length;
  // workspace: outputs of the parts, their sums, the table of items
  p.part_o = static_cast<float*>(a->workspace);
  p.part_lse = p.part_o + pl.parts_bytes / 4 / (c->head_dim + 1) * c->head_dim;
  p.joins =
      reinterpret_cast<hstu::JoinRecord*>(static_cast<char*>(a->workspace) + pl.parts_bytes);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int fmt = cache_format(c->dtype);
  cudaError_t e =
      pl.kernel == AttnPlan::ROWS
          ? hstu::launch_softmax_rows(p, a->dtype, fmt, pl.rows, pl.tiles, pl.blocks,
                                      pl.cluster, s)
      : pl.kernel == AttnPlan::TC
          ? hstu::launch_softmax_tc(p, a->dtype, fmt, pl.qtiles, pl.ctas, pl.tiles, pl.blocks, s)
          : hstu::launch_softmax_simt(p, fmt, pl.rows, pl.tiles, pl.blocks, s);
  if (e == cudaSuccess && (pl.splits > 1 || pl.balanced))
    e = hstu::launch_softmax_join(p, a->dtype, 128 / p.G, pl.qtiles, (int)pl.blocks, s);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // namespace
