// Launch interface between the entry points of the KV cache operators (kv_api.cu) and their
// kernels.
#pragma once
#include <cuda_runtime.h>

#include <atomic>

namespace hstu {

// Allows a kernel `bytes` of dynamic shared memory, once per device (`done`: one bit each).
inline cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit & done.load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

struct CacheView;
struct SoftmaxParams;

// Append (append = true) or read back; dtype of k and v, e4m3: the cache holds E4M3.
cudaError_t launch_kv_copy(const CacheView& c, void* k, void* v, long long k_stride,
                           long long v_stride, int dtype, bool e4m3, bool append, int sms,
                           cudaStream_t stream);

// fp32 attention on CUDA cores: `rows` (4 or 64) packed query rows of one kv head per CTA.
cudaError_t launch_softmax_simt(const SoftmaxParams& p, bool e4m3, int rows, long long tiles,
                                long long blocks, cudaStream_t stream);

// Tensor-core attention (bf16, fp16). A CTA takes qtiles tiles of 128 / G tokens, two where
// D <= 128 only; an SM holds `ctas` CTAs, two where D <= 128 with one tile and no E4M3.
cudaError_t launch_softmax_tc(const SoftmaxParams& p, int dtype, bool e4m3, int qtiles, int ctas,
                              long long tiles, long long blocks, cudaStream_t stream);

// Attention of few rows (bf16, fp16): `rows` (8 or 16) packed rows of one kv head per cluster
// of CTAs; CTAs of it that an SM holds.
int softmax_rows_ctas(int D, bool e4m3, int rows);
cudaError_t launch_softmax_rows(const SoftmaxParams& p, int dtype, bool e4m3, int rows,
                                long long tiles, long long blocks, int cluster,
                                cudaStream_t stream);

// Joins the parts of outputs that several CTAs worked on (balanced runs of the tensor-core
// kernel: tokens of a query tile, query tiles of an item, CTAs of the run).
cudaError_t launch_softmax_join(const SoftmaxParams& p, int dtype, int tile_tokens,
                                int query_tiles, int grid, cudaStream_t stream);

}  // namespace hstu
