// Which rows of a paged cache to keep: per sequence and kv head the last ones and those of the largest
// attention weights among the others (hstu_kv_select).
//
// Weights become unsigned keys of the same order, a NaN the smallest. A CTA per (sequence, kv head)
// finds the smallest key that is kept by eight bits at a time, each time counting the next eight bits
// of the keys that agree with what is known, then writes the positions in order: all of larger keys
// and of that key as many, from the first on, as the budget leaves.
#include "common.cuh"
#include "evict_kernels.h"
#include "kernels.h"
#include "kv_cache.cuh"

namespace hstu {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;

__device__ __forceinline__ void store_index(void* p, long long i, int index64, long long x) {
  if (index64)
    static_cast<long long*>(p)[i] = x;
  else
    static_cast<int*>(p)[i] = (int)x;
}

__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);  // (-0 becomes +0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ bool table_ok(const SelectParams& p, const PagedSeq& s) {
  return s.ok && s.Lk <= p.max_k;
}

// Exclusive sum of x over the CTA, in order of the threads; total: all of it.
__device__ __forceinline__ long long block_scan(long long x, long long* warps, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long v = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += y;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = v;
  __syncthreads();
  long long before = 0;
  total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warps[w];
    total += warps[w];
  }
  return before + v - x;
}

// Page offsets and last pages' lengths of the shorter sequences, by one CTA.
__global__ void __launch_bounds__(kThreads) new_table_kernel(const SelectParams p) {
  __shared__ long long warps[kWarps];
  long long carry = 0;
  for (int b0 = 0; b0 < p.c.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    long long pages = 0;
    if (b < p.c.B) {
      const PagedSeq s = paged_table(p.c, b);
      const bool ok = table_ok(p, s);
      if (!ok) report(p.c, HSTU_DEVERR_OFFSETS);
      const long long keep = ok ? min(s.Lk, (long long)p.budget) : 0;
      pages = (keep + page_size(p.c) - 1) >> p.c.page_shift;
      store_index(p.new_last_page_len, b, p.c.index64,
                  pages ? keep - ((pages - 1) << p.c.page_shift) : 1);
    }
    long long total;
    const long long before = block_scan(pages, warps, total);
    if (b < p.c.B) store_index(p.new_page_offsets, b, p.c.index64, carry + before);
    carry += total;
  }
  if (threadIdx.x == 0) store_index(p.new_page_offsets, p.c.B, p.c.index64, carry);
}

__global__ void __launch_bounds__(kThreads) select_kernel(const SelectParams p) {
  __shared__ int count[256];
  __shared__ long long warps[kWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left;
  const int hk = (int)(blockIdx.x % (unsigned)p.c.Nk), b = (int)(blockIdx.x / (unsigned)p.c.Nk);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const PagedSeq s = paged_table(p.c, b);
  const bool ok = table_ok(p, s);
  const long long Lk = ok ? s.Lk : 0;
  int* kept = p.kept + ((long long)b * p.c.Nk + hk) * p.budget;
  const int keep = (int)min(Lk, (long long)p.budget), recent = min(p.recent, keep);
  const int others = (int)Lk - recent;  // positions that weights decide on
  const int take = keep - recent;       // of which so many are kept

  if (hk == 0) {  // the sequence's page ids, and -1 behind the last sequence's
    const long long first = load_index(p.new_page_offsets, b, p.c.index64);
    const long long pages = load_index(p.new_page_offsets, b + 1, p.c.index64) - first;
    for (long long i = tid; i < pages; i += kThreads)
      store_index(p.new_page_ids, first + i, p.c.index64,
                  load_index(p.c.page_ids, s.po + i, p.c.index64));
    const long long end = load_index(p.new_page_offsets, p.c.B, p.c.index64);
    for (long long i = end + (long long)b * kThreads + tid; i < p.c.num_page_ids;
         i += (long long)p.c.B * kThreads)
      store_index(p.new_page_ids, i, p.c.index64, -1);
  }

  auto key_at = [&](int pos) {
    const long long page = page_at(p.c, s, pos);
    if (page < 0) {
      report(p.c, HSTU_DEVERR_OFFSETS);
      return 0u;
    }
    return order_key(p.weights[((page * p.c.Nk + hk) << p.c.page_shift) +
                               (pos & ((1 << p.c.page_shift) - 1))]);
  };
  // the key of the last row that is kept by its weight, and how many of that key are
  uint32_t edge = 0;
  int left = take;
  if (take > 0 && take < others) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) count[tid] = 0;
      __syncthreads();
      for (int pos = tid; pos < others; pos += kThreads) {
        const uint32_t k = key_at(pos);
        if (shift == 24 || (k >> (shift + 8)) == (edge >> (shift + 8)))
          atomicAdd(&count[k >> shift & 255u], 1);
      }
      __syncthreads();
      if (warp == 0) {  // the digit at which the keys from the largest on reach `left`
        int mine[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += mine[i] = count[255 - (lane * 8 + i)];
        int before = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, before, d);
          if (lane >= d) before += y;
        }
        before -= sum;
        if (before < left && before + sum >= left) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (before < left && before + mine[i] >= left) {
              s_prefix = edge | (uint32_t)(255 - (lane * 8 + i)) << shift;
              s_left = left - before;
            }
            before += mine[i];
          }
        }
      }
      __syncthreads();
      edge = s_prefix;
      left = s_left;
    }
  }
  // positions in order
  int written = 0, equal = 0;  // kept, and of the edge's key, before this round
  for (int p0 = 0; p0 < (int)Lk && written < keep; p0 += kThreads) {
    const int pos = p0 + tid;
    bool larger = false, same = false;
    if (pos < (int)Lk) {
      if (pos >= others || take == others) {
        larger = true;
      } else if (take > 0) {
        const uint32_t k = key_at(pos);
        larger = k > edge;
        same = k == edge;
      }
    }
    // (both counts in one scan)
    long long total;
    const long long before = block_scan((long long)larger | (long long)same << 32, warps, total);
    const int larger_before = (int)(before & 0xffffffff), same_before = equal + (int)(before >> 32);
    const int same_taken = min(same_before, left) - min(equal, left);  // in this round, before me
    if (larger || (same && same_before < left))
      kept[written + larger_before + same_taken] = pos;
    const int same_all = equal + (int)(total >> 32);
    written += (int)(total & 0xffffffff) + min(same_all, left) - min(equal, left);
    equal = same_all;
  }
  for (int r = keep + tid; r < p.budget; r += kThreads) kept[r] = -1;
}

}  // namespace

cudaError_t launch_select(const SelectParams& p, cudaStream_t stream) {
  new_table_kernel<<<1, kThreads, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  select_kernel<<<(unsigned)((long long)p.c.B * p.c.Nk), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace hstu
