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

template <typename T>
__device__ __forceinline__ void join(const SoftmaxParams& p, int count, long long row, int first,
                                     int step) {
  const long long all = p.c.T * p.Nq;  // part i of the row is number i * all + row
  float top = -CUDART_INF_F;
  for (int i = 0; i < count; ++i) top = fmaxf(top, p.part_lse[i * all + row]);
  const float base = top == -CUDART_INF_F ? 0.f : top;
  float sum = 0.f;
  for (int i = 0; i < count; ++i) sum += exp2f(p.part_lse[i * all + row] - base);
  const int D = p.c.D;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  for (int d = first; d < D; d += step) {
    float o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < count; ++i) {
      const long long at = i * all + row;
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
  join<T>(p, count, row, (int)(lane & ((1 << lane_shift) - 1)) * 4, 4 << lane_shift);
}

// Pieces of a balanced run: block (c, y) joins kJoinRows rows of the item that CTA c + 1's record
// names, a warp four of them (what bounds it is the latency of its few dependent loads: one row
// after the other, found from the table of items, took 20 us a call, this 6). An item's rows are
// packed, `tile_rows` to a query tile of 128 slot rows; its first piece lies in slot
// 2 first + 1 of the CTAs' slots, piece i in slot 2 (first + i).
constexpr int kWarpRows = 4, kJoinRows = kWarpRows * kThreads / 32;

template <typename T>
__global__ void __launch_bounds__(kThreads) join_pieces_kernel(const SoftmaxParams p,
                                                               int tile_rows, int query_tiles) {
  ptx::grid_dependency_wait();
  const JoinRecord j = p.joins[blockIdx.x + 1];
  const int first = blockIdx.x, lane = threadIdx.x & 31;
  const int row0 = (int)blockIdx.y * kJoinRows + (int)(threadIdx.x >> 5) * kWarpRows;
  if (j.count == 0 || row0 >= j.rows) return;
  auto at = [&](int i, int row) {
    const long long slot = i == 0 ? 2 * first + 1 : 2 * (first + i);
    return slot * (query_tiles * 128) + row / tile_rows * 128 + row % tile_rows;
  };
  // lane 8 r + i: part i (and 8 + i, ...) of row r
  const int mine = min(row0 + lane / 8, j.rows - 1), part = lane % 8;
  auto log_sum = [&](int i) { return i < j.count ? p.part_lse[at(i, mine)] : -CUDART_INF_F; };
  const float e0 = log_sum(part);
  float top = e0;
  for (int i = 8; i < j.count; i += 8) top = fmaxf(top, log_sum(i + part));
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  const float base = top == -CUDART_INF_F ? 0.f : top;
  float sum = exp2f(e0 - base);
  for (int i = 8; i < j.count; i += 8) sum += exp2f(log_sum(i + part) - base);
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  auto out_row = [&](int row) { return (j.t0 + row / p.G) * p.Nq + j.hk * p.G + row % p.G; };
  if (p.lse && part == 0 && row0 + lane / 8 < j.rows)
    p.lse[out_row(mine)] = (top + log2f(sum)) * kLn2;
  const int D = p.c.D;
  for (int d0 = 0; d0 < D; d0 += 128) {  // (every lane stays for the shuffles)
    const int d = d0 + lane * 4;
    float o[kWarpRows][4] = {};
    for (int i0 = 0; i0 < j.count; i0 += 8) {
      const float w = exp2f((i0 ? log_sum(i0 + part) : e0) - base) * inv;
      for (int i = i0; i < min(j.count, i0 + 8); ++i) {
        float4 f[kWarpRows];
        float wr[kWarpRows];
#pragma unroll
        for (int r = 0; r < kWarpRows; ++r) {
          wr[r] = __shfl_sync(0xffffffffu, w, r * 8 + i - i0);
          f[r] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (wr[r] != 0.f && d < D)  // a part without keys for this row holds nothing
            f[r] = *reinterpret_cast<const float4*>(
                p.part_o + at(i, min(row0 + r, j.rows - 1)) * D + d);
        }
#pragma unroll
        for (int r = 0; r < kWarpRows; ++r) {
          o[r][0] = fmaf(wr[r], f[r].x, o[r][0]);
          o[r][1] = fmaf(wr[r], f[r].y, o[r][1]);
          o[r][2] = fmaf(wr[r], f[r].z, o[r][2]);
          o[r][3] = fmaf(wr[r], f[r].w, o[r][3]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kWarpRows; ++r)
      if (row0 + r < j.rows && d < D)
        store4(static_cast<T*>(p.out) + out_row(row0 + r) * D + d, o[r]);
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
    if (grid < 2) return cudaSuccess;  // (one CTA: nothing is parted)
    cfg.gridDim = dim3((unsigned)grid - 1, (unsigned)(query_tiles * 128 / kJoinRows));
    return cudaLaunchKernelEx(&cfg, join_pieces_kernel<T>, p, tile_tokens * p.G, query_tiles);
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
