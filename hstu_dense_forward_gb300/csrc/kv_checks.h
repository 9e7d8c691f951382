// Checks of the arguments that the entry points over a paged KV cache share.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/hstu_kv.h"
#include "kv_cache.cuh"

namespace hstu {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline int elem_bytes(int dtype) { return dtype == HSTU_F32 ? 4 : 2; }

inline int cache_format(int dtype) {
  return dtype == HSTU_FP8_E4M3   ? kE4m3
         : dtype == HSTU_FP4_E2M1 ? kE2m1
                                  : kSame;
}

// Sizes of a cache descriptor; pointers are checked by cache_pointers_ok.
inline hstu_status check_cache(const hstu_kv_cache* c) {
  if (!c || c->reserved) return HSTU_ERR_INVALID_ARG;
  const bool fp8 = c->dtype == HSTU_FP8_E4M3, fp4 = c->dtype == HSTU_FP4_E2M1;
  if (!fp4 && (c->dtype < HSTU_F32 || c->dtype > HSTU_FP8_E4M3)) return HSTU_ERR_INVALID_ARG;
  if (c->batch < 0 || c->batch > (1 << 20)) return HSTU_ERR_INVALID_ARG;
  if (c->num_heads_kv < 1 || c->num_heads_kv > 65536) return HSTU_ERR_INVALID_ARG;
  if (c->head_dim < 1) return HSTU_ERR_INVALID_ARG;
  if (c->head_dim % (fp4 ? 32 : 16) != 0 || c->head_dim > 256) return HSTU_ERR_UNSUPPORTED;
  if (c->page_size != 32 && c->page_size != 128 && c->page_size != 256)
    return HSTU_ERR_INVALID_ARG;
  if (c->index_is_int64 != 0 && c->index_is_int64 != 1) return HSTU_ERR_INVALID_ARG;
  if (c->descale < HSTU_DESCALE_CAST || c->descale > HSTU_DESCALE_BLOCK)
    return HSTU_ERR_INVALID_ARG;
  if (c->descale == HSTU_DESCALE_BLOCK) return HSTU_ERR_UNSUPPORTED;
  if (!fp8 && (c->descale != HSTU_DESCALE_CAST || (c->kv_scale && !fp4)))
    return HSTU_ERR_INVALID_ARG;
  if (c->descale != HSTU_DESCALE_CAST && c->kv_scale) return HSTU_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->num_pages > (1ll << 30) || c->num_page_ids < 0)
    return HSTU_ERR_INVALID_ARG;
  return HSTU_OK;
}

inline bool cache_pointers_ok(const hstu_kv_cache* c) {
  if (!c->kv_cache || !aligned(c->kv_cache, 16) || !c->page_offsets || !c->last_page_len ||
      (!c->page_ids && c->num_page_ids > 0))
    return false;
  const uintptr_t ib = c->index_is_int64 ? 8 : 4;
  if (!aligned(c->page_offsets, ib) || !aligned(c->last_page_len, ib) ||
      !aligned(c->page_ids, ib) || !aligned(c->status, 4) || !aligned(c->kv_scale, 16))
    return false;
  if (c->dtype == HSTU_FP4_E2M1 &&
      (!c->kv_scale || !c->kv_group_scale || !aligned(c->kv_group_scale, 16)))
    return false;
  const bool factors = c->descale != HSTU_DESCALE_CAST;
  if (factors != (c->k_descale != nullptr) || factors != (c->v_descale != nullptr)) return false;
  return aligned(c->k_descale, 4) && aligned(c->v_descale, 4);
}

inline int page_shift(int page_size) { return page_size == 32 ? 5 : page_size == 128 ? 7 : 8; }

inline CacheView cache_view(const hstu_kv_cache* c, const void* seq_offsets, long long T) {
  CacheView v = {};
  v.cache = c->kv_cache;
  v.scale = static_cast<uint8_t*>(c->kv_scale);
  // (a field that callers of the other forms may not have)
  v.group = c->dtype == HSTU_FP4_E2M1 ? static_cast<uint8_t*>(c->kv_group_scale) : nullptr;
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
  v.page_shift = page_shift(c->page_size);
  v.ds_b = c->descale == HSTU_DESCALE_BATCH ? 1
           : c->descale == HSTU_DESCALE_HEAD ? c->num_heads_kv : 0;
  v.ds_h = c->descale == HSTU_DESCALE_HEAD ? 1 : 0;
  return v;
}

// Row dtype against the cache's: the same, or any 32- or 16-bit type with a cache of codes.
inline bool row_dtype_ok(const hstu_kv_cache* c, int dtype) {
  if (dtype < HSTU_F32 || dtype > HSTU_BF16) return false;
  return cache_format(c->dtype) != kSame || c->dtype == dtype;
}

// Streaming multiprocessors of a device, asked for once.
inline bool device_sms(int dev, int* sms) {
  static std::atomic<int> known[64];
  const bool keep = dev >= 0 && dev < 64;
  if (keep && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return true;
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return false;
  if (keep) known[dev].store(*sms, std::memory_order_relaxed);
  return true;
}

}  // namespace hstu
