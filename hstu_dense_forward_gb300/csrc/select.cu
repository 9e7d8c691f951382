// Which rows of a paged cache to keep: per sequence and kv head the last ones and those of the largest
// attention weights among the others (hstu_kv_select).
//
// Weights become unsigned keys of the same order, a NaN the smallest. A cluster of CTAs per (sequence,
// kv head) reads them once into shared memory, a stretch of the positions each, and finds the smallest
// key that is kept by eleven bits at a time, each time counting the next eleven bits of the keys that
// agree with what is known (eight at a time, whose first are a sign and seven of an exponent, crowd
// few counters). Then it writes the positions in order: all of larger keys and, of that
// key, as many as the budget leaves, from the first on. Warps own stretches of the positions, so that a
// count before the writes gives every warp its first rank. Two CTAs share an SM (one, with all of its
// registers: 31 us in place of 26 for 128 lists of 4k-16k positions). (Keys that were read anew in
// each of the five passes, by one CTA: 58 us, and one list of 100,000 350.)
#include <cooperative_groups.h>

#include "common.cuh"
#include "evict_kernels.h"
#include "kernels.h"
#include "kv_cache.cuh"
#include "kv_kernels.h"

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

// Pages that sequence b keeps. (store: its last page's length is written, a bad table reported.)
__device__ __forceinline__ long long kept_pages(const SelectParams& p, int b, bool store) {
  const PagedSeq s = paged_table(p.c, b);
  const bool ok = table_ok(p, s);
  const long long keep = ok ? min(s.Lk, (long long)p.budget) : 0;
  const long long pages = (keep + page_size(p.c) - 1) >> p.c.page_shift;
  if (store) {
    if (!ok) report(p.c, HSTU_DEVERR_OFFSETS);
    store_index(p.new_last_page_len, b, p.c.index64,
                pages ? keep - ((pages - 1) << p.c.page_shift) : 1);
  }
  return pages;
}

// What the new page offsets stop at. (Sequences whose entries of page_ids overlap can have more pages
// than new_page_ids holds: the offsets stop behind its end, where they are no valid table's.)
__device__ __forceinline__ long long most_pages(const SelectParams& p) {
  return p.c.index64 ? p.c.num_page_ids + 1 : min(p.c.num_page_ids + 1, 0x7fffffffll);
}

// Page offsets and last pages' lengths of the shorter sequences, by one CTA (of more sequences than a
// CTA has threads; of fewer select_kernel's CTAs find their offsets by themselves, a launch less: five
// sequences of up to 300 rows 9.0 us in place of 10.0).
__global__ void __launch_bounds__(kThreads) new_table_kernel(const SelectParams p) {
  __shared__ long long warps[kWarps];
  const long long most = most_pages(p);
  long long carry = 0;
  for (int b0 = 0; b0 < p.c.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    const long long pages = b < p.c.B ? kept_pages(p, b, true) : 0;
    long long total;
    const long long before = block_scan(pages, warps, total);
    if (b < p.c.B) store_index(p.new_page_offsets, b, p.c.index64, min(carry + before, most));
    carry += total;
  }
  if (threadIdx.x == 0) store_index(p.new_page_offsets, p.c.B, p.c.index64, min(carry, most));
}

constexpr int kMaxKeys = 49152;  // of a CTA that shared memory holds; others are read anew
constexpr int kBins = 2 * kThreads;  // of eleven bits
constexpr int kLoads = 8;        // of a lane at a time

__global__ void __launch_bounds__(kThreads, 2) select_kernel(const SelectParams p, int cluster,
                                                          int capacity) {
  namespace cg = cooperative_groups;
  extern __shared__ uint32_t keys[];  // [capacity]
  __shared__ __align__(8) int count[2][kBins];
  __shared__ int w_larger[kWarps], w_equal[kWarps];
  __shared__ int totals[2];  // of the CTA's keys: larger than the edge, equal to it
  __shared__ uint32_t s_edge;
  __shared__ int s_left;
  const unsigned pair = blockIdx.x / (unsigned)cluster;
  const int rank = (int)(blockIdx.x % (unsigned)cluster);
  const int hk = (int)(pair % (unsigned)p.c.Nk), b = (int)(pair / (unsigned)p.c.Nk);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const PagedSeq s = paged_table(p.c, b);
  const bool ok = table_ok(p, s);
  const int Lk = ok ? (int)s.Lk : 0;
  int* kept = p.kept + (long long)pair * p.budget;
  const int keep = min(Lk, p.budget), recent = min(p.recent, keep);
  const int others = Lk - recent;  // positions that weights decide on
  const int take = keep - recent;  // of which so many are kept
  const bool decide = take > 0 && take < others;

  if (hk == 0 && rank == 0) {  // the sequence's page ids, and -1 behind the last sequence's
    long long first, end;
    if (p.c.B <= kThreads) {
      __shared__ long long scan[kWarps], s_first;
      const long long x = tid < p.c.B ? kept_pages(p, tid, b == 0) : 0, most = most_pages(p);
      const long long before = min(block_scan(x, scan, end), most);
      end = min(end, most);
      if (tid == b) s_first = before;
      if (b == 0) {
        if (tid < p.c.B) store_index(p.new_page_offsets, tid, p.c.index64, before);
        if (tid == 0) store_index(p.new_page_offsets, p.c.B, p.c.index64, end);
      }
      __syncthreads();
      first = s_first;
    } else {
      first = load_index(p.new_page_offsets, b, p.c.index64);
      end = load_index(p.new_page_offsets, p.c.B, p.c.index64);
    }
    long long pages = ((long long)keep + page_size(p.c) - 1) >> p.c.page_shift;
    if (pages > p.c.num_page_ids - first) {  // (entries that overlap)
      if (tid == 0) report(p.c, HSTU_DEVERR_OFFSETS);
      pages = p.c.num_page_ids - first;
    }
    for (long long i = tid; i < pages; i += kThreads)
      store_index(p.new_page_ids, first + i, p.c.index64,
                  load_index(p.c.page_ids, s.po + i, p.c.index64));
    for (long long i = end + (long long)b * kThreads + tid; i < p.c.num_page_ids;
         i += (long long)p.c.B * kThreads)
      store_index(p.new_page_ids, i, p.c.index64, -1);
  }

  // This CTA's positions [p0, p0 + mine): a warp's are a stretch of `per` of them. (Pages hold whole
  // groups of 32 rows, so that a warp's 32 positions lie in one.)
  const int groups = (Lk + 31) / 32;
  const int g0 = (int)((long long)groups * rank / cluster);
  const int g1 = (int)((long long)groups * (rank + 1) / cluster);
  const int p0 = g0 * 32, mine = min(Lk, g1 * 32) - p0;
  const int per = (g1 - g0 + kWarps - 1) / kWarps;  // groups of a warp
  const int first = min(warp * per, g1 - g0), last = min(first + per, g1 - g0);
  auto key_from = [&](int at) {  // at: counted from p0
    const int pos = p0 + at;
    if (at >= mine) return 0u;
    const long long page = page_at(p.c, s, pos);
    if (page < 0) {
      report(p.c, HSTU_DEVERR_OFFSETS);
      return 0u;
    }
    return order_key(p.weights[((page * p.c.Nk + hk) << p.c.page_shift) +
                               (pos & ((1 << p.c.page_shift) - 1))]);
  };
  auto key_at = [&](int at) { return at < capacity ? keys[at] : key_from(at); };
  // the key of the last row that is kept by its weight, and how many of that key are
  uint32_t edge = 0;
  int left = take;
  if (decide) {  // (for the whole cluster)
    for (int g = first; g < last; g += kLoads) {
      uint32_t k[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) k[i] = g + i < last ? key_from((g + i) * 32 + lane) : 0u;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int at = (g + i) * 32 + lane;
        if (g + i < last && at < capacity) keys[at] = k[i];
      }
    }
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t bins = pass == 2 ? 1023u : 2047u;
      const uint32_t known = pass == 0 ? 0u : ~0u << (pass == 1 ? 21 : 10);
      int* mine_count = count[pass & 1];
      mine_count[tid] = mine_count[tid + kThreads] = 0;
      __syncthreads();
      for (int g = first; g < last; ++g) {
        const int at = g * 32 + lane;
        const uint32_t k = key_at(at);
        if (p0 + at < others && ((k ^ edge) & known) == 0)
          atomicAdd(&mine_count[k >> shift & bins], 1);
      }
      // the other CTAs' counts; this buffer is written again two passes on, when all have read it
      if (cluster > 1)
        cg::this_cluster().sync();
      else
        __syncthreads();
      // the digit at which the keys from the largest on reach `left`: two digits a thread
      int digit[2] = {0, 0};
      const int top = kBins - 2 * tid;
      for (int r = 0; r < cluster; ++r) {
        const int* c = cluster > 1 ? cg::this_cluster().map_shared_rank(mine_count, r) : mine_count;
        const int2 two = *reinterpret_cast<const int2*>(c + top - 2);
        digit[0] += two.y;
        digit[1] += two.x;
      }
      const int sum = digit[0] + digit[1];
      int before = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += y;
      }
      if (lane == 31) w_larger[warp] = before;
      __syncthreads();
      int warps_before = lane < warp ? w_larger[lane] : 0;
      warps_before = __reduce_add_sync(0xffffffffu, warps_before);
      before += warps_before - sum;
      if (before < left && before + sum >= left) {  // one thread
        const bool second = before + digit[0] < left;
        s_edge = edge | (uint32_t)(top - (second ? 2 : 1)) << shift;
        s_left = left - before - (second ? digit[0] : 0);
      }
      __syncthreads();
      edge = s_edge;
      left = s_left;
    }
  }
  // larger: kept; same: of the edge's key, of which the first `left` are kept
  auto look = [&](int g, bool& larger, bool& same) {
    const int at = g * 32 + lane, pos = p0 + at;
    larger = pos < Lk && (pos >= others || take == others);
    same = false;
    if (decide && at < mine && pos < others) {
      const uint32_t k = key_at(at);
      larger = k > edge;
      same = k == edge;
    }
  };
  int larger_sum = 0, equal_sum = 0;
  for (int g = first; g < last; ++g) {
    bool larger, same;
    look(g, larger, same);
    larger_sum += __popc(__ballot_sync(0xffffffffu, larger));
    equal_sum += __popc(__ballot_sync(0xffffffffu, same));
  }
  if (lane == 0) {
    w_larger[warp] = larger_sum;
    w_equal[warp] = equal_sum;
  }
  __syncthreads();
  int larger_before = 0, equal_before = 0;
  if (cluster > 1) {
    if (warp < 2) {
      const int sum = __reduce_add_sync(0xffffffffu, (warp ? w_equal : w_larger)[lane]);
      if (lane == 0) totals[warp] = sum;
    }
    cg::this_cluster().sync();
    for (int r = 0; r < rank; ++r) {
      const int* t = cg::this_cluster().map_shared_rank(totals, r);
      larger_before += t[0];
      equal_before += t[1];
    }
  }
  larger_before += __reduce_add_sync(0xffffffffu, lane < warp ? w_larger[lane] : 0);
  equal_before += __reduce_add_sync(0xffffffffu, lane < warp ? w_equal[lane] : 0);
  for (int g = first; g < last; ++g) {
    bool larger, same;
    look(g, larger, same);
    const uint32_t l = __ballot_sync(0xffffffffu, larger), e = __ballot_sync(0xffffffffu, same);
    const uint32_t below = (1u << lane) - 1u;
    const int eq = equal_before + __popc(e & below);
    if (larger || (same && eq < left))
      kept[larger_before + __popc(l & below) + min(eq, left)] = p0 + g * 32 + lane;
    larger_before += __popc(l);
    equal_before += __popc(e);
  }
  for (int r = keep + rank * kThreads + tid; r < p.budget; r += cluster * kThreads) kept[r] = -1;
  if (cluster > 1) cg::this_cluster().sync();  // the others have read this CTA's shared memory
}

}  // namespace

cudaError_t launch_select(const SelectParams& p, int sms, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (p.c.B > kThreads) {
    new_table_kernel<<<1, kThreads, 0, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const long long pairs = (long long)p.c.B * p.c.Nk;
  // as many CTAs a list as the SMs have room for, of 2048 positions at least
  int cluster = 1;
  while (cluster < 8 && pairs * cluster * 2 <= 2ll * sms && p.max_k > 2048ll * cluster) cluster *= 2;
  long long capacity = (p.max_k + cluster - 1) / cluster + 64;
  if (capacity > kMaxKeys) capacity = kMaxKeys;
  static std::atomic<unsigned long long> done;
  e = allow_smem(reinterpret_cast<const void*>(select_kernel), kMaxKeys * 4, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(pairs * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)capacity * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, select_kernel, p, cluster, (int)capacity);
}

}  // namespace hstu
