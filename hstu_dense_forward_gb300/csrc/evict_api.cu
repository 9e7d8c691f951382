// C ABI of eviction from the paged KV cache: argument checks, the choice of kernels, launches. See
// include/hstu_evict.h for the contracts.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/hstu_evict.h"
#include "evict_kernels.h"
#include "kv_checks.h"
#include "kv_kernels.h"

using namespace hstu;

namespace {

bool bad_bound(int x) { return x < 1 || x > (1 << 30); }

int row_bytes(const hstu_kv_cache* c) {
  const int fmt = cache_format(c->dtype);
  return fmt == kE2m1   ? c->head_dim / 2
         : fmt == kE4m3 ? c->head_dim
                        : c->head_dim * elem_bytes(c->dtype);
}

// Chunks of the ranks of a sequence and kv head.
long long compact_chunks(const hstu_kv_cache* c, const hstu_compact_args* a) {
  const long long ranks = a->budget < a->max_seqlen_k ? a->budget : a->max_seqlen_k;
  const int rows = compact_rows(row_bytes(c));
  return (ranks + rows - 1) / rows;
}

}  // namespace

extern "C" {

hstu_status hstu_kv_weights(const hstu_kv_cache* c, const hstu_weights_args* a, void* stream) {
  const hstu_status st = check_cache(c);
  if (st != HSTU_OK) return st;
  if (!a || a->reserved || !row_dtype_ok(c, a->dtype)) return HSTU_ERR_INVALID_ARG;
  if (a->total_tokens < 0 || a->total_tokens > 0x7fffffffll || a->num_heads_q < 0 ||
      a->num_heads_q % c->num_heads_kv != 0)
    return HSTU_ERR_INVALID_ARG;
  if (a->max_seqlen < 1 || a->max_seqlen > (1 << 24) || bad_bound(a->max_seqlen_k) ||
      (a->causal != 0 && a->causal != 1) || (a->accumulate != 0 && a->accumulate != 1) ||
      !(a->alpha > 0.0f) || !(a->alpha <= 2e38f))
    return HSTU_ERR_INVALID_ARG;
  const long long G = a->num_heads_q / c->num_heads_kv;
  if (G > 128) return HSTU_ERR_UNSUPPORTED;
  const bool none = a->total_tokens == 0 || G == 0;  // no queries: only 0 to add or to store
  if (c->batch == 0 || (none && a->accumulate)) return HSTU_OK;
  if (!a->seq_offsets || !aligned(a->seq_offsets, c->index_is_int64 ? 8 : 4) || !a->weights ||
      !aligned(a->weights, 16) || !cache_pointers_ok(c))
    return HSTU_ERR_INVALID_ARG;
  if (!none &&
      (!a->q || !a->lse || !aligned(a->q, 16) || !aligned(a->lse, 4) ||
       a->q_stride < (long long)a->num_heads_q * c->head_dim || a->q_stride > (1ll << 36) ||
       a->q_stride * elem_bytes(a->dtype) % 16 != 0))
    return HSTU_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !device_sms(dev, &sms)) return HSTU_ERR_CUDA;
  WeightsParams w = {};
  w.a.c = cache_view(c, a->seq_offsets, a->total_tokens);
  w.a.q = a->q;
  w.a.q_stride = a->q_stride;
  w.a.Nq = a->num_heads_q;
  w.a.G = (int)(G > 0 ? G : 1);
  w.a.max_q = a->max_seqlen;
  w.a.max_k = a->max_seqlen_k;
  w.a.causal = a->causal;
  w.a.scale_log2 = (float)((double)a->alpha * 1.4426950408889634);
  w.a.splits = 1;
  w.a.min_range = 128;
  w.a.timeout_ns = 1000000000ll;
  w.lse = a->lse;
  w.weights = a->weights;
  w.accumulate = a->accumulate;
  const int fmt = cache_format(c->dtype);
  const long long most = a->max_seqlen < a->total_tokens ? a->max_seqlen : a->total_tokens;
  const long long pairs = (long long)c->batch * c->num_heads_kv;
  if (pairs > 0x7fffffffll / 8) return HSTU_ERR_UNSUPPORTED;
  // CTAs that take turns at the keys of a sequence and kv head, `keys` at a time
  auto slots_for = [&](long long ctas, int keys) {
    const long long can = ((long long)a->max_seqlen_k + keys - 1) / keys;
    long long want = (ctas + pairs - 1) / pairs;
    if (want > can) want = can;
    if (want * pairs > 0x7fffffffll) want = 0x7fffffffll / pairs;
    return (int)(want < 1 ? 1 : want);
  };
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a->dtype == HSTU_F32) {
    const bool few = none || most * G <= 16;
    const int slots = slots_for((few ? 16ll : 4ll) * sms, few ? 128 : kWeightsSimtKeys);
    if (few) w.a.splits = slots;
    e = launch_weights_simt(w, fmt, few ? 0 : slots, s);
  } else if (none || most * G <= 16) {
    // one wave of CTAs, each with a stretch of the keys
    const int rows = none || most * G <= 8 ? 8 : 16;
    const long long ctas = (long long)weights_rows_ctas(c->head_dim, fmt, rows) * sms;
    const long long can = (a->max_seqlen_k + 127) / 128, want = ctas / pairs;
    w.a.splits = (int)(want < 1 ? 1 : want < can ? want : can);
    if (w.a.splits == 1)
      w.a.by_length = rows_by_length(c->batch, pairs, sms, c->num_page_ids, c->page_size,
                                     a->max_seqlen_k);
    e = launch_weights_rows(w, a->dtype, fmt, rows, s);
  } else {
    const int keys = weights_tc_keys(c->head_dim);
    const long long steps = ((long long)a->max_seqlen_k + keys - 1) / keys;
    const long long tiles = (most + 128 / G - 1) / (128 / G);  // of query rows
    int slots = slots_for(2ll * sms, keys), cluster = 1;
    if (slots == steps)
      while (cluster < 8 && slots * pairs * cluster * 2 <= 2ll * sms && tiles >= 8 * cluster)
        cluster *= 2;
    e = launch_weights_tc(w, a->dtype, fmt, slots, cluster, s);
  }
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

hstu_status hstu_kv_select(const hstu_select_args* a, void* stream) {
  if (!a || a->reserved) return HSTU_ERR_INVALID_ARG;
  if (a->batch < 0 || a->batch > (1 << 20) || a->num_heads_kv < 1 || a->num_heads_kv > 65536 ||
      (a->page_size != 32 && a->page_size != 128 && a->page_size != 256) ||
      (a->index_is_int64 != 0 && a->index_is_int64 != 1) || a->num_pages < 1 ||
      a->num_pages > (1ll << 30) || a->num_page_ids < 0 || bad_bound(a->budget) ||
      a->recent < 0 || a->recent > (1 << 30) || bad_bound(a->max_seqlen_k))
    return HSTU_ERR_INVALID_ARG;
  const long long pairs = (long long)a->batch * a->num_heads_kv;
  if (pairs > 0x7fffffffll) return HSTU_ERR_UNSUPPORTED;
  if (a->batch == 0) return HSTU_OK;
  const uintptr_t ib = a->index_is_int64 ? 8 : 4;
  const bool ids = a->num_page_ids > 0;
  if (!a->page_offsets || !a->last_page_len || !a->weights || !a->kept || !a->new_page_offsets ||
      !a->new_last_page_len || (ids && (!a->page_ids || !a->new_page_ids)) ||
      !aligned(a->page_offsets, ib) || !aligned(a->page_ids, ib) ||
      !aligned(a->last_page_len, ib) || !aligned(a->new_page_offsets, ib) ||
      !aligned(a->new_page_ids, ib) || !aligned(a->new_last_page_len, ib) ||
      !aligned(a->weights, 16) || !aligned(a->kept, 4) || !aligned(a->status, 4) ||
      a->new_page_offsets == a->page_offsets || a->new_last_page_len == a->last_page_len ||
      (ids && a->new_page_ids == a->page_ids))
    return HSTU_ERR_INVALID_ARG;
  SelectParams p = {};
  p.c.page_offsets = a->page_offsets;
  p.c.page_ids = a->page_ids;
  p.c.last_page_len = a->last_page_len;
  p.c.status = a->status;
  p.c.num_pages = a->num_pages;
  p.c.num_page_ids = a->num_page_ids;
  p.c.index64 = a->index_is_int64;
  p.c.B = a->batch;
  p.c.Nk = a->num_heads_kv;
  p.c.page_shift = page_shift(a->page_size);
  p.weights = a->weights;
  p.budget = a->budget;
  p.recent = a->recent;
  p.max_k = a->max_seqlen_k;
  p.kept = a->kept;
  p.new_page_offsets = a->new_page_offsets;
  p.new_page_ids = a->new_page_ids;
  p.new_last_page_len = a->new_last_page_len;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !device_sms(dev, &sms)) return HSTU_ERR_CUDA;
  return launch_select(p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? HSTU_OK
                                                                                 : HSTU_ERR_CUDA;
}

hstu_status hstu_compact_workspace(const hstu_kv_cache* c, const hstu_compact_args* a,
                                   long long* bytes) {
  if (!bytes) return HSTU_ERR_INVALID_ARG;
  *bytes = 0;
  const hstu_status st = check_cache(c);
  if (st != HSTU_OK) return st;
  if (!a || a->reserved || bad_bound(a->budget) || bad_bound(a->max_seqlen_k))
    return HSTU_ERR_INVALID_ARG;
  const long long tickets = (long long)c->batch * c->num_heads_kv * compact_chunks(c, a);
  if (tickets > 0x70000000ll) return HSTU_ERR_UNSUPPORTED;  // (they are counted in 32 bits)
  const long long pairs = (long long)c->batch * c->num_heads_kv;
  *bytes = tickets ? (4 + pairs + 2 * tickets) * (long long)sizeof(int) : 0;
  return HSTU_OK;
}

hstu_status hstu_kv_compact(const hstu_kv_cache* c, const hstu_compact_args* a, void* stream) {
  long long need = 0;
  const hstu_status st = hstu_compact_workspace(c, a, &need);
  if (st != HSTU_OK) return st;
  if (c->batch == 0) return HSTU_OK;
  if (!a->kept || !aligned(a->kept, 4) || !aligned(a->weights, 16) || !cache_pointers_ok(c))
    return HSTU_ERR_INVALID_ARG;
  if (need > 0 && (!a->workspace || !aligned(a->workspace, 16) || a->workspace_bytes < need))
    return HSTU_ERR_INVALID_ARG;
  CompactParams p = {};
  p.c = cache_view(c, nullptr, 0);
  p.kept = a->kept;
  p.budget = a->budget;
  p.max_k = a->max_seqlen_k;
  p.weights = a->weights;
  p.row_bytes = row_bytes(c);
  p.by_head = cache_format(c->dtype) == kE2m1;
  p.counter = static_cast<int*>(a->workspace);
  p.ends = p.counter + 4;
  p.loaded = p.ends + (long long)c->batch * c->num_heads_kv;
  p.fronts = p.loaded + (long long)c->batch * c->num_heads_kv * compact_chunks(c, a);
  p.timeout_ns = 1000000000ll;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !device_sms(dev, &sms)) return HSTU_ERR_CUDA;
  return launch_compact(p, (int)compact_chunks(c, a), sms, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? HSTU_OK
             : HSTU_ERR_CUDA;
}

}  // extern "C"
