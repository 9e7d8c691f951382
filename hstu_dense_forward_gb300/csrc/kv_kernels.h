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

// Append (append = true) or read back; dtype of k and v, fmt: what the cache holds (kSame, ..).
// weights: of the rows' entries, which an append sets to 0, or nullptr.
cudaError_t launch_kv_copy(const CacheView& c, void* k, void* v, long long k_stride,
                           long long v_stride, float* weights, int dtype, int fmt, bool append, int sms,
                           cudaStream_t stream);

// The pages of an E2M1 cache that sequences with queries have, as bf16 [.., 2, page_size, Nk, D], and
// the entries of a table of them for theirs (-1 for an id outside the cache). Page i of sequence b comes
// to the place of its entry of page_ids (by_entry), or to b * per + i; sequences have `per` pages at most
// (longer ones are left out).
cudaError_t launch_expand(const CacheView& c, void* pages, void* ids, long long per, bool by_entry,
                          cudaStream_t stream);

// fp32 attention on CUDA cores: `rows` (4 or 64) packed query rows of one kv head per CTA.
cudaError_t launch_softmax_simt(const SoftmaxParams& p, int fmt, int rows, long long tiles,
                                long long blocks, cudaStream_t stream);

// Tensor-core attention (bf16, fp16). A CTA takes qtiles tiles of 128 / G tokens, two where
// D <= 128 only; an SM holds `ctas` CTAs, two where D <= 128 with one tile and no codes.
cudaError_t launch_softmax_tc(const SoftmaxParams& p, int dtype, int fmt, int qtiles, int ctas,
                              long long tiles, long long blocks, cudaStream_t stream);

// Items of one tile each, `ctas` of them, are taken by the sequences' lengths (see softmax_rows.cuh)
// where that pays: CTAs of a round, or 0. A CTA finds its sequence in some 2 us, for up to 256 of them;
// what it saves is that an SM's items are long ones together. So there have to be two an SM at least,
// the mean length (as far as the host sees it: of as many pages as page_ids has entries) must be 2048
// keys and more, and the longest a quarter longer. Measured with four heads over 16-bit, E4M3 and E2M1
// caches: 128 sequences of 1024-4096 keys 112 -> 104 us, 73 -> 62 and 79 -> 62, 80 of them 79 -> 73,
// 50 -> 46 and 61 -> 52. Where the rule says 0: 160 of 200-500 keys 30 -> 32, 19 -> 23 and 23 -> 26, 128
// of 4096 each 153 -> 156, 109 -> 116 and 106 -> 110, 40 of 1024-4096 (one item an SM, 16 bits) 44 -> 46,
// 200 of 10-100 and one head 6.4 -> 8.3, 6.8 -> 9.0 and 7.3 -> 9.3.
inline int rows_by_length(long long batch, long long ctas, long long sms, long long num_page_ids,
                          int page_size, long long max_keys) {
  const long long keys = (num_page_ids < (1ll << 32) ? num_page_ids : 1ll << 32) * page_size;
  return batch > 1 && batch <= 256 && ctas >= 2 * sms && keys >= 2048 * batch &&
                 5 * keys <= 4 * max_keys * batch
             ? (int)sms
             : 0;
}

// Attention of few rows (bf16, fp16): `rows` (8 or 16) packed rows of one kv head per cluster
// of CTAs; CTAs of it that an SM holds.
int softmax_rows_ctas(int D, int fmt, int rows);
cudaError_t launch_softmax_rows(const SoftmaxParams& p, int dtype, int fmt, int rows,
                                long long tiles, long long blocks, int cluster,
                                cudaStream_t stream);

// Joins the parts of outputs that several CTAs worked on (balanced runs of the tensor-core
// kernel: tokens of a query tile, query tiles of an item, CTAs of the run).
cudaError_t launch_softmax_join(const SoftmaxParams& p, int dtype, int tile_tokens,
                                int query_tiles, int grid, cudaStream_t stream);

}  // namespace hstu
