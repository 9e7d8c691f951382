// The pages of an E2M1 cache that sequences with queries have as bf16, in the layout of a bf16 cache,
// for attention of many query rows over them. Every CTA of that kernel would turn the keys and values of
// its items into 16 bits by itself, and its softmax waits for the warps that do: with several items a kv
// head and sequence it is faster to convert them once, a pass that is bound by memory (16 sequences of
// 100-512 tokens over some 4500 keys, two kv heads of four: 191 us, with this 145; four of 4096 over 4096
// 965 and 672). The products of codes, factors and powers of two have seven bits, so that bf16 holds them.
#include "kernels.h"
#include "kv_cache.cuh"
#include "kv_kernels.h"

namespace hstu {

namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads)
    expand_kernel(const CacheView c, __nv_bfloat16* pages, void* ids, unsigned per, bool by_entry) {
  const unsigned b = blockIdx.x / per, i = blockIdx.x % per;
  const PagedSeq s = paged_seq(c, b);
  if (!s.ok || s.n == 0 || i >= s.pages || s.pages > per) return;  // (nothing reads its pages)
  const long long entry = s.po + i, slot = by_entry ? entry : blockIdx.x;
  const long long page = load_index(c.page_ids, entry, c.index64);
  const bool ok = page >= 0 && page < c.num_pages;
  if (threadIdx.x == 0 && blockIdx.y == 0) {  // (an id outside the cache stays one)
    if (c.index64)
      static_cast<long long*>(ids)[entry] = ok ? slot : -1;
    else
      static_cast<int*>(ids)[entry] = ok ? (int)slot : -1;
  }
  if (!ok) return;
  const int groups = c.D / 16, ps = 1 << c.page_shift;
  const int chunks = 2 * ps * c.Nk * groups;  // of sixteen elements, in the order of their places
  uint4* to = reinterpret_cast<uint4*>(pages) + slot * chunks * 2;
  // group, kv head, and plane and row of a chunk; of those further on, by addition
  const int first = blockIdx.y * kThreads + threadIdx.x, step = gridDim.y * kThreads;
  int g = first % groups, hk = first / groups % c.Nk, r = first / groups / c.Nk;
  const int dg = step % groups, dh = step / groups % c.Nk, dr = step / groups / c.Nk;
#pragma unroll 4
  for (int x = first; x < chunks; x += step) {
    const long long row = scale_row(c, page, r >> c.page_shift, r & (ps - 1), hk);
    const float f = scale_value(c.scale[row]) * e4m3_value(c.group[row * groups + g]);
    float v[16];
    load16_e2m1(static_cast<const uint8_t*>(c.cache) + (row * groups + g) * 8, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= f;
    store16(reinterpret_cast<__nv_bfloat16*>(to + x * 2), v);
    g += dg;
    hk += dh + (g >= groups ? 1 : 0);
    r += dr + (hk >= c.Nk ? 1 : 0);
    g -= g >= groups ? groups : 0;
    hk -= hk >= c.Nk ? c.Nk : 0;
  }
}

}  // namespace

cudaError_t launch_expand(const CacheView& c, void* pages, void* ids, long long per, bool by_entry,
                          cudaStream_t stream) {
  // four chunks a thread, if a page has as many
  const long long chunks = (2ll * c.Nk * (c.D / 16)) << c.page_shift;
  const long long parts = chunks / (4 * kThreads);
  expand_kernel<<<dim3((unsigned)(c.B * per), parts < 1 ? 1 : parts < 1024 ? (unsigned)parts : 1024),
                  kThreads, 0, stream>>>(c, static_cast<__nv_bfloat16*>(pages), ids, (unsigned)per,
                                         by_entry);
  return cudaGetLastError();
}

}  // namespace hstu
