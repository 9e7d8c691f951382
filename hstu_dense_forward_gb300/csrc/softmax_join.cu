// Joins the parts of outputs that several CTAs worked on: key ranges of a sequence (CUDA-core and
// few-row kernels), or pieces of the items of a balanced run (tensor-core kernel).
//
// out = sum_s 2^(e_s - max e) O_s / sum_s 2^(e_s - max e) over the parts s of a row, e_s the base-2
// logarithm of part s's sum and O_s its output. One group of D / 4 lanes (rounded up to a power
// of two, one warp at most) per (row, head), four consecutive elements a lane and step.
// Launched with programmatic dependent launch: it waits for the kernel before it.
#include <math_constants.h>

#include "kernels.h"
#include "kv_cache.cuh"
#include "kv_kernels.h"
#include "ptx.cuh"

namespace hstu {

namespace {

constexpr int kThreads = 256;
constexpr float kLn2 = 0.69314718055994530942f;

template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&x)[4]);
template <>
__device__ __forceinline__ void store4<float>(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
template <>
__device__ __forceinline__ void store4<__half>(__half* p, const float (&x)[4]) {
  const __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* p, const float (&x)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}

// The parts of a row: `count` of them, part i at row number at(i) of part_o and part_lse.
struct Ranges {
  long long row, all;
  int count;
  __device__ long long at(int i) const { return i * all + row; }
};
// Pieces of an item: the first ends CTA c's share inside the item (slot 2 c + 1), the others
// begin inside it (slots 2 (c + i)).
struct Pieces {
  int c, count, slot_rows, row;  // (rows of a slot, the row's place in it)
  __device__ long long at(int i) const {
    return (long long)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * slot_rows + row;
  }
};

template <typename T, typename Parts>
__device__ __forceinline__ void join(const SoftmaxParams& p, const Parts& parts, long long row,
                                     int first, int step) {
  float top = -CUDART_INF_F;
  for (int i = 0; i < parts.count; ++i) top = fmaxf(top, p.part_lse[parts.at(i)]);
  const float base = top == -CUDART_INF_F ? 0.f : top;
  float sum = 0.f;
  for (int i = 0; i < parts.count; ++i) sum += exp2f(p.part_lse[parts.at(i)] - base);
  const int D = p.c.D;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  for (int d = first; d < D; d += step) {
    float o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < parts.count; ++i) {
      const long long at = parts.at(i);
      const float w = exp2f(p.part_lse[at] - base) * inv;
      if (w == 0.f) continue;  // a part without keys for this row holds nothing
      const float4 f = *reinterpret_cast<const float4*>(p.part_o + at * D + d);
      o[0] = fmaf(w, f.x, o[0]);
      o[1] = fmaf(w, f.y, o[1]);
      o[2] = fmaf(w, f.z, o[2]);
      o[3] = fmaf(w, f.w, o[3]);
    }
    store4(static_cast<T*>(p.out) + row * D + d, o);
  }
  if (p.lse && first == 0) p.lse[row] = (top + log2f(sum)) * kLn2;
}

// Key ranges: every row of a sequence with more than one.
template <typename T>
__global__ void __launch_bounds__(kThreads) join_ranges_kernel(const SoftmaxParams p,
                                                               int lane_shift) {
  ptx::grid_dependency_wait();
  const long long lane = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long row = lane >> lane_shift, t = row / p.Nq;
  if (t >= p.c.T) return;
  const PagedSeq s = paged_seq(p.c, seq_of_row(p.c, t));
  if (!attn_seq_ok(p, s) || t < s.t0 || t >= s.t0 + s.n) return;
  const int count = key_ranges(p, s.Lk).count;
  if (count < 2) return;  // written by the attention kernel
  join<T>(p, Ranges{row, p.c.T * p.Nq, count}, row, (int)(lane & ((1 << lane_shift) - 1)) * 4,
          4 << lane_shift);
}

// Pieces of a balanced run. Block (c, y) looks at the border between the shares of CTAs c and
// c + 1: if it is the first that parts an item's key tiles, the block joins kJoinRows of its
// rows. tile_tokens: tokens of one query tile, query_tiles of an item.
constexpr int kJoinRows = 32;

template <typename T>
__global__ void __launch_bounds__(kThreads) join_pieces_kernel(const SoftmaxParams p,
                                                               int tile_tokens, int query_tiles,
                                                               int grid) {
  ptx::grid_dependency_wait();
  const PlanTable& pl = *p.plan;
  const int c = blockIdx.x, e = pl.begin_item[c + 1], hk = pl.begin_head[c + 1];
  const long long units = pl.cost[pl.items] * p.c.Nk;
  const int ctas = share_ctas(units, grid);
  if (units == 0 || c + 1 >= ctas) return;
  const long long cost = pl.cost[e + 1] - pl.cost[e], base = pl.cost[e] * p.c.Nk + hk * cost;
  // shares end at u1 (CTA c - 1) and u2; a border in front of the item's tiles parts nothing
  const long long u1 = share(units, ctas, c), u2 = share(units, ctas, c + 1);
  if (u2 <= base + kItemCost || u1 > base + kItemCost) return;
  int last = c + 1;
  while (share(units, ctas, last + 1) < base + cost) ++last;
  const int b = pl.seq[e];
  const PagedSeq s = paged_seq(p.c, b);
  const int rows = query_tiles * 128;
  for (int x = blockIdx.y * kJoinRows + (threadIdx.x >> 5);
       x < min(rows, (int)(blockIdx.y + 1) * kJoinRows); x += kThreads / 32) {
    const int q = x / 128, r = x % 128;
    const long long tok = ((long long)(e - pl.first[b]) * query_tiles + q) * tile_tokens + r / p.G;
    if (r >= tile_tokens * p.G || tok >= s.n) continue;
    const long long row = (s.t0 + tok) * p.Nq + hk * p.G + r % p.G;
    join<T>(p, Pieces{c, last - c + 1, rows, x}, row, (threadIdx.x & 31) * 4, 128);
  }
}

template <typename T>
cudaError_t launch(const SoftmaxParams& p, int tile_tokens, int query_tiles, int grid,
                   cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.balanced) {
    cfg.gridDim = dim3((unsigned)grid, (unsigned)(query_tiles * 128 / kJoinRows));
    return cudaLaunchKernelEx(&cfg, join_pieces_kernel<T>, p, tile_tokens, query_tiles, grid);
  }
  int shift = 0;
  while (shift < 5 && (4 << shift) < p.c.D) ++shift;
  const long long lanes = p.c.T * p.Nq << shift;
  cfg.gridDim = dim3((unsigned)((lanes + kThreads - 1) / kThreads));
  return cudaLaunchKernelEx(&cfg, join_ranges_kernel<T>, p, shift);
}

}  // namespace

cudaError_t launch_softmax_join(const SoftmaxParams& p, int dtype, int tile_tokens,
                                int query_tiles, int grid, cudaStream_t stream) {
  if (dtype == HSTU_F32) return launch<float>(p, tile_tokens, query_tiles, grid, stream);
  if (dtype == HSTU_BF16) return launch<__nv_bfloat16>(p, tile_tokens, query_tiles, grid, stream);
  return launch<__half>(p, tile_tokens, query_tiles, grid, stream);
}

}  // namespace hstu
