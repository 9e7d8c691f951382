// Writing rows into the paged KV cache and reading them back (hstu_kv_append, hstu_kv_read).
//
// Both move every element once: a group of LG lanes (the power of two at or above D / 16)
// takes one (row, kv head) of both planes, sixteen elements a lane in 16-byte accesses. The
// row's place (sequence by bisection, then page table, then page id) is found by every lane
// for itself: the loads hit in L1 and their latency is hidden by the other warps.
// Quantisation with row scales: the largest magnitude of the D values is found by shuffles,
// and the scale is a power of two, so that scaling is exact and the rounding to E4M3 is the
// only one (an arbitrary factor would add one, and E4M3 is a floating-point format: it gains
// nothing by it).
#include "kernels.h"
#include "kv_cache.cuh"
#include "kv_kernels.h"
#include "ptx.cuh"

namespace hstu {

namespace {

constexpr int kThreads = 256;
constexpr int kMinExp = -100;  // smallest exponent of a row scale

struct CopyParams {
  CacheView c;
  void* k;
  void* v;
  long long k_stride, v_stride;  // elements
  int lane_shift;                // log2(LG)
};

enum : int { kCopy = 0, kCast = 1, kStatic = 2, kScale = 3 };

// Place of one (row, head) group, shared by both kernels.
struct Place {
  int b, hk, d0;       // sequence, kv head, first element of this lane
  long long t, page, row;
  bool lane_ok;        // this lane holds elements (d0 < D) of a row that exists
  bool ok;             // ... whose sequence and page are valid
};

__device__ __forceinline__ Place find_place(const CopyParams& p) {
  Place w;
  const long long lane = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (p.c.status) {  // every sequence is checked by some thread, those without rows too
    const long long threads = (long long)gridDim.x * kThreads;
    for (long long b = lane; b < p.c.B; b += threads) {
      const PagedSeq s = paged_seq(p.c, b);
      if (!s.ok || s.n > s.Lk) report(p.c, HSTU_DEVERR_OFFSETS);
    }
  }
  const long long group = lane >> p.lane_shift;
  w.d0 = (int)(lane & ((1 << p.lane_shift) - 1)) * 16;
  w.t = group / p.c.Nk;
  w.hk = (int)(group - w.t * p.c.Nk);
  w.lane_ok = w.t < p.c.T && w.d0 < p.c.D;
  w.ok = false;
  w.page = w.row = 0;
  w.b = 0;
  if (w.t >= p.c.T) return w;
  w.b = seq_of_row(p.c, w.t);
  const PagedSeq s = paged_seq(p.c, w.b);
  if (!s.ok || s.n > s.Lk || w.t < s.t0 || w.t >= s.t0 + s.n) return w;
  const long long pos = s.Lk - s.n + (w.t - s.t0);
  w.page = page_at(p.c, s, pos);
  w.row = pos & (page_size(p.c) - 1);
  if (w.page < 0) {
    report(p.c, HSTU_DEVERR_OFFSETS);
    return w;
  }
  w.ok = true;
  return w;
}

__device__ __forceinline__ float factor(const CacheView& c, const float* f, int b, int hk) {
  return f[(long long)b * c.ds_b + (long long)hk * c.ds_h];
}

// Exponent of the row scale from the bits of the row's largest finite magnitude
// m 2^k (1 <= m < 2): 448 = 1.75 * 2^8, so e = k - 8, or k - 7 above m = 1.75.
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < kMinExp ? kMinExp : e;
}

__device__ __forceinline__ void store_codes(uint8_t* dst, const float (&x)[16], float mul) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = ptx::cvt_e4m3x2_f32(x[4 * i] * mul, x[4 * i + 1] * mul) |
           ptx::cvt_e4m3x2_f32(x[4 * i + 2] * mul, x[4 * i + 3] * mul) << 16;
  *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Largest magnitude of a row over its lane group, as fp32 bits. Magnitudes order like their
// bits; infinities and NaN (bits from 0x7f800000 on) are left out.
__device__ __forceinline__ uint32_t row_max(const float (&x)[16], bool lane_ok, int lanes) {
  uint32_t m = 0;
  if (lane_ok) {
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    if (m >= 0x7f800000u) {
      m = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t u = __float_as_uint(x[i]) & 0x7fffffffu;
        if (u < 0x7f800000u) m = max(m, u);
      }
    }
  }
  for (int d = 1; d < lanes; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  return m;
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const CopyParams p) {
  const Place w = find_place(p);
  float x[2][16];
  if (w.ok && w.lane_ok) {
    load16(static_cast<const T*>(p.k) + w.t * p.k_stride + (long long)w.hk * p.c.D + w.d0, x[0]);
    load16(static_cast<const T*>(p.v) + w.t * p.v_stride + (long long)w.hk * p.c.D + w.d0, x[1]);
  }
#pragma unroll
  for (int plane = 0; plane < 2; ++plane) {
    uint32_t top = 0;
    if constexpr (MODE == kScale)  // (every lane of the warp takes part in the shuffles)
      top = row_max(x[plane], w.ok && w.lane_ok, 1 << p.lane_shift);
    if (!w.ok || !w.lane_ok) continue;
    const long long at = cache_row(p.c, w.page, plane, w.row, w.hk) + w.d0;
    if constexpr (MODE == kCopy) {
      store16(static_cast<T*>(p.c.cache) + at, x[plane]);
    } else {
      uint8_t* dst = static_cast<uint8_t*>(p.c.cache) + at;
      if constexpr (MODE == kScale) {
        const int e = scale_exponent(top);
        store_codes(dst, x[plane], __uint_as_float((uint32_t)(127 - e) << 23));
        if (w.d0 == 0) p.c.scale[scale_row(p.c, w.page, plane, w.row, w.hk)] = (uint8_t)(e + 127);
      } else if constexpr (MODE == kStatic) {
        const float f = factor(p.c, plane ? p.c.v_ds : p.c.k_ds, w.b, w.hk);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[plane][i] /= f;
        store_codes(dst, x[plane], 1.0f);
      } else {
        store_codes(dst, x[plane], 1.0f);
      }
    }
  }
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const CopyParams p) {
  const Place w = find_place(p);
  if (!w.ok || !w.lane_ok) return;
  float x[2][16];
#pragma unroll
  for (int plane = 0; plane < 2; ++plane) {
    const long long at = cache_row(p.c, w.page, plane, w.row, w.hk) + w.d0;
    if constexpr (MODE == kCopy)
      load16(static_cast<const T*>(p.c.cache) + at, x[plane]);
    else
      load16(static_cast<const uint8_t*>(p.c.cache) + at, x[plane]);
  }
#pragma unroll
  for (int plane = 0; plane < 2; ++plane) {
    float f = 1.0f;
    if constexpr (MODE == kScale)
      f = scale_value(p.c.scale[scale_row(p.c, w.page, plane, w.row, w.hk)]);
    if constexpr (MODE == kStatic) f = factor(p.c, plane ? p.c.v_ds : p.c.k_ds, w.b, w.hk);
    if constexpr (MODE == kScale || MODE == kStatic) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[plane][i] *= f;
    }
    T* dst = static_cast<T*>(plane ? p.v : p.k) + w.t * (plane ? p.v_stride : p.k_stride) +
             (long long)w.hk * p.c.D + w.d0;
    store16(dst, x[plane]);
  }
}

template <typename T>
cudaError_t launch(const CopyParams& p, bool append, int mode, unsigned grid, cudaStream_t st) {
#define HSTU_COPY(M)                                            \
  if (append)                                                   \
    kv_append_kernel<T, M><<<grid, kThreads, 0, st>>>(p);       \
  else                                                          \
    kv_read_kernel<T, M><<<grid, kThreads, 0, st>>>(p);         \
  break
  switch (mode) {
    case kCopy: HSTU_COPY(kCopy);
    case kCast: HSTU_COPY(kCast);
    case kStatic: HSTU_COPY(kStatic);
    default: HSTU_COPY(kScale);
  }
#undef HSTU_COPY
  return cudaGetLastError();
}

}  // namespace

long long kv_copy_blocks(long long T, int Nk, int D) {
  int shift = 0;
  while ((16 << shift) < D) ++shift;
  return ((T * Nk << shift) + kThreads - 1) / kThreads;
}

cudaError_t launch_kv_copy(const CacheView& c, void* k, void* v, long long k_stride,
                           long long v_stride, int dtype, bool e4m3, bool append,
                           cudaStream_t stream) {
  CopyParams p = {};
  p.c = c;
  p.k = k;
  p.v = v;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  while ((16 << p.lane_shift) < c.D) ++p.lane_shift;
  const unsigned grid = (unsigned)kv_copy_blocks(c.T, c.Nk, c.D);
  const int mode = !e4m3 ? kCopy : c.scale ? kScale : c.k_ds ? kStatic : kCast;
  if (dtype == HSTU_F32) return launch<float>(p, append, mode, grid, stream);
  if (dtype == HSTU_BF16) return launch<__nv_bfloat16>(p, append, mode, grid, stream);
  return launch<__half>(p, append, mode, grid, stream);
}

}  // namespace hstu
