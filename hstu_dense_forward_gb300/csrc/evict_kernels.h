// Launch interface between the entry points of eviction (evict_api.cu) and their kernels.
#pragma once
#include <cuda_runtime.h>

#include "kv_cache.cuh"

namespace hstu {

// Attention weights of the cached keys: a.q .. a.causal as in the attention.
struct WeightsParams {
  SoftmaxParams a;
  const float* lse;  // [T, Nq]
  float* weights;    // [num_pages, Nk, page_size]
  int accumulate;
};

// Few rows (16-bit; at most `rows`, 8 or 16, of a kv head and sequence); CTAs that an SM holds.
int weights_rows_ctas(int D, int fmt, int rows);
cudaError_t launch_weights_rows(const WeightsParams& w, int dtype, int fmt, int rows,
                                cudaStream_t stream);

// More rows, on the tensor cores; `slots` CTAs take turns at the key steps of a sequence and kv head.
// Or clusters of `cluster` CTAs, which divide the query rows; they have a step each.
int weights_tc_keys(int D);  // keys of a step
cudaError_t launch_weights_tc(const WeightsParams& w, int dtype, int fmt, int slots, int cluster,
                              cudaStream_t stream);

// fp32 rows, on CUDA cores; slots = 0: at most 16 of a kv head and sequence, whose keys a.splits CTAs
// divide.
cudaError_t launch_weights_simt(const WeightsParams& w, int fmt, int slots, cudaStream_t stream);
constexpr int kWeightsSimtKeys = 64;  // keys of a step

struct SelectParams {
  CacheView c;  // the table and Nk alone
  const float* weights;
  int budget, recent;
  long long max_k;
  int* kept;
  void* new_page_offsets;
  void* new_page_ids;
  void* new_last_page_len;
};
cudaError_t launch_select(const SelectParams& p, int sms, cudaStream_t stream);

struct CompactParams {
  CacheView c;
  const int* kept;
  int budget;
  long long max_k;
  float* weights;  // or nullptr
  int row_bytes;   // of a head's row in one plane of the cache
  int by_head;     // the cache has its heads before the rows (E2M1)
  int* counter;    // of the chunks that have been handed out
  int* ends;       // [B, Nk]: where lists end
  int* loaded;     // [B, Nk, chunks]: the chunk's rows have been read
  int* fronts;     // [B, Nk, chunks]: the chunks in front that a chunk waits for
  long long timeout_ns;
};
constexpr int kCompactRows = 256;  // most ranks of a chunk
int compact_rows(int row_bytes);   // ranks of a chunk
cudaError_t launch_compact(const CompactParams& p, int chunks, int sms, cudaStream_t stream);

}  // namespace hstu
