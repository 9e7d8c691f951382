// C ABI of the paged KV cache operators: argument checks, the choice of kernel and of the
// number of key ranges, and launches. See include/hstu_kv.h for the contracts.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/hstu_kv.h"
#include "kv_cache.cuh"
#include "kv_kernels.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int elem_bytes(int dtype) { return dtype == HSTU_F32 ? 4 : dtype == HSTU_FP8_E4M3 ? 1 : 2; }

// Sizes of a cache descriptor; pointers are checked by cache_pointers_ok.
hstu_status check_cache(const hstu_kv_cache* c) {
  if (!c || c->reserved) return HSTU_ERR_INVALID_ARG;
  if (c->dtype < HSTU_F32 || c->dtype > HSTU_FP8_E4M3) return HSTU_ERR_INVALID_ARG;
  if (c->batch < 0 || c->batch > (1 << 20)) return HSTU_ERR_INVALID_ARG;
  if (c->num_heads_kv < 1 || c->num_heads_kv > 65536) return HSTU_ERR_INVALID_ARG;
  if (c->head_dim < 1) return HSTU_ERR_INVALID_ARG;
  if (c->head_dim % 16 != 0 || c->head_dim > 256) return HSTU_ERR_UNSUPPORTED;
  if (c->page_size != 32 && c->page_size != 128 && c->page_size != 256)
    return HSTU_ERR_INVALID_ARG;
  if (c->index_is_int64 != 0 && c->index_is_int64 != 1) return HSTU_ERR_INVALID_ARG;
  if (c->descale < HSTU_DESCALE_CAST || c->descale > HSTU_DESCALE_BLOCK)
    return HSTU_ERR_INVALID_ARG;
  if (c->descale == HSTU_DESCALE_BLOCK) return HSTU_ERR_UNSUPPORTED;
  const bool fp8 = c->dtype == HSTU_FP8_E4M3;
  if (!fp8 && (c->descale != HSTU_DESCALE_CAST || c->kv_scale)) return HSTU_ERR_INVALID_ARG;
  if (c->descale != HSTU_DESCALE_CAST && c->kv_scale) return HSTU_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->num_pages > (1ll << 30) || c->num_page_ids < 0)
    return HSTU_ERR_INVALID_ARG;
  return HSTU_OK;
}

bool cache_pointers_ok(const hstu_kv_cache* c) {
  if (!c->kv_cache || !aligned(c->kv_cache, 16) || !c->page_offsets || !c->last_page_len ||
      (!c->page_ids && c->num_page_ids > 0))
    return false;
  const uintptr_t ib = c->index_is_int64 ? 8 : 4;
  if (!aligned(c->page_offsets, ib) || !aligned(c->last_page_len, ib) ||
      !aligned(c->page_ids, ib) || !aligned(c->status, 4) || !aligned(c->kv_scale, 16))
    return false;
  const bool factors = c->descale != HSTU_DESCALE_CAST;
  if (factors != (c->k_descale != nullptr) || factors != (c->v_descale != nullptr)) return false;
  return aligned(c->k_descale, 4) && aligned(c->v_descale, 4);
}

hstu::CacheView cache_view(const hstu_kv_cache* c, const void* seq_offsets, long long T) {
  hstu::CacheView v = {};
  v.cache = c->kv_cache;
  v.scale = static_cast<uint8_t*>(c->kv_scale);
  v.page_offsets = c->page_offsets;
  v.page_ids = c->page_ids;
  v.last_page_len = c->last_page_len;
  v.seq_offsets = seq_offsets;
  v.k_ds = c->k_descale;
  v.v_ds = c->v_descale;
  v.status = c->status;
  v.num_pages = c->num_pages;
  v.num_page_ids = c->num_page_ids;
  v.T = T;
  v.index64 = c->index_is_int64;
  v.B = c->batch;
  v.Nk = c->num_heads_kv;
  v.D = c->head_dim;
  v.page_shift = c->page_size == 32 ? 5 : c->page_size == 128 ? 7 : 8;
  v.ds_b = c->descale == HSTU_DESCALE_BATCH ? 1
           : c->descale == HSTU_DESCALE_HEAD ? c->num_heads_kv : 0;
  v.ds_h = c->descale == HSTU_DESCALE_HEAD ? 1 : 0;
  return v;
}

// Row dtype against the cache's: the same, or any 32- or 16-bit type with an E4M3 cache.
bool row_dtype_ok(const hstu_kv_cache* c, int dtype) {
  if (dtype < HSTU_F32 || dtype > HSTU_BF16) return false;
  return c->dtype == HSTU_FP8_E4M3 || c->dtype == dtype;
}

// Streaming multiprocessors of a device, asked for once.
bool device_sms(int dev, int* sms) {
  static std::atomic<int> known[64];
  const bool keep = dev >= 0 && dev < 64;
  if (keep && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return true;
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return false;
  if (keep) known[dev].store(*sms, std::memory_order_relaxed);
  return true;
}

hstu_status copy_rows(const hstu_kv_cache* c, const hstu_kv_rows* r, bool append, void* stream) {
  const hstu_status st = check_cache(c);
  if (st != HSTU_OK) return st;
  if (!r || r->reserved || !row_dtype_ok(c, r->dtype)) return HSTU_ERR_INVALID_ARG;
  if (r->total_tokens < 0 || r->total_tokens > 0x7fffffffll) return HSTU_ERR_INVALID_ARG;
  if (c->batch == 0 || r->total_tokens == 0) return HSTU_OK;
  const long long width = (long long)c->num_heads_kv * c->head_dim;
  const int eb = elem_bytes(r->dtype);
  if (!r->k || !r->v || !aligned(r->k, 16) || !aligned(r->v, 16) || !r->seq_offsets ||
      !aligned(r->seq_offsets, c->index_is_int64 ? 8 : 4) || r->k_stride < width ||
      r->v_stride < width || r->k_stride * eb % 16 != 0 || r->v_stride * eb % 16 != 0 ||
      r->k_stride > (1ll << 40) || r->v_stride > (1ll << 40) || !cache_pointers_ok(c) ||
      (!append && r->k == r->v))  // (one place for both planes)
    return HSTU_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !device_sms(dev, &sms)) return HSTU_ERR_CUDA;
  const hstu::CacheView v = cache_view(c, r->seq_offsets, r->total_tokens);
  return hstu::launch_kv_copy(v, r->k, r->v, r->k_stride, r->v_stride, r->dtype,
                              c->dtype == HSTU_FP8_E4M3, append, sms,
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
  const bool fp8 = c->dtype == HSTU_FP8_E4M3, small = c->head_dim <= 128;
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
  if (small && !fp8 && (pl->qtiles == 1 || a->max_seqlen_k <= 4096)) {
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
        (long long)hstu::softmax_rows_ctas(c->head_dim, c->dtype == HSTU_FP8_E4M3, pl->rows) * sms;
    const long long can = (a->max_seqlen_k + 127) / 128;  // two tiles of 64 keys each
    long long want = slots / items < can ? slots / items : can;
    if (want < 1) want = 1;
    while (pl->cluster < 8 && pl->cluster * 2 <= want) pl->cluster *= 2;
    pl->splits = (int)(want / pl->cluster);
    pl->min_range = 128 * pl->cluster;
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
  const hstu_status st = plan_attention(cache, args, &pl);
  if (st == HSTU_OK) *bytes = pl.workspace;
  return st;
}

hstu_status hstu_softmax_fwd(const hstu_kv_cache* c, const hstu_softmax_args* a, void* stream) {
  AttnPlan pl;
  const hstu_status st = plan_attention(c, a, &pl);
  if (st != HSTU_OK) return st;
  if (pl.blocks == 0) return HSTU_OK;  // empty input
  if (!a->q || !a->out || !a->seq_offsets || !aligned(a->q, 16) || !aligned(a->out, 16) ||
      !aligned(a->lse, 4) || !aligned(a->seq_offsets, c->index_is_int64 ? 8 : 4) ||
      a->q_stride < (long long)a->num_heads_q * c->head_dim || a->q_stride > (1ll << 36) ||
      a->q_stride * elem_bytes(a->dtype) % 16 != 0 || !cache_pointers_ok(c))
    return HSTU_ERR_INVALID_ARG;
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
  // workspace: outputs of the parts, their sums, the table of items
  p.part_o = static_cast<float*>(a->workspace);
  p.part_lse = p.part_o + pl.parts_bytes / 4 / (c->head_dim + 1) * c->head_dim;
  p.joins =
      reinterpret_cast<hstu::JoinRecord*>(static_cast<char*>(a->workspace) + pl.parts_bytes);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool fp8 = c->dtype == HSTU_FP8_E4M3;
  cudaError_t e =
      pl.kernel == AttnPlan::ROWS
          ? hstu::launch_softmax_rows(p, a->dtype, fp8, pl.rows, pl.tiles, pl.blocks,
                                      pl.cluster, s)
      : pl.kernel == AttnPlan::TC
          ? hstu::launch_softmax_tc(p, a->dtype, fp8, pl.qtiles, pl.ctas, pl.tiles, pl.blocks, s)
          : hstu::launch_softmax_simt(p, fp8, pl.rows, pl.tiles, pl.blocks, s);
  if (e == cudaSuccess && (pl.splits > 1 || pl.balanced))
    e = hstu::launch_softmax_join(p, a->dtype, 128 / p.G, pl.qtiles, (int)pl.blocks, s);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // extern "C"
