// Writing rows into the paged KV cache and reading them back (hstu_kv_append, hstu_kv_read).
//
// Both move every element once. A block takes 2^row_shift consecutive rows and every kv head of
// them. First one thread per row finds the row's place (sequence by bisection, page table, page
// id: a chain of dependent loads, whose latency a block pays once); then groups of LG lanes (the
// power of two at or above D / 16) take one (row, head) after the other, both planes, sixteen
// elements a lane in 16-byte accesses, the rows of one head side by side (their scales are
// adjacent bytes). The loads of an append need no place and are issued before it is known.
// Quantisation with row scales: the largest magnitude of the D values is found by shuffles,
// and the scale is a power of two, so that scaling is exact and the rounding to E4M3 is the
// only one (an arbitrary factor would add one, and E4M3 is a floating-point format: it gains
// nothing by it).
// E2M1 has one bit behind the leading one and six powers of two less, so there each group of
// sixteen elements, which is what a lane holds, has a factor besides, rounded to E4M3. Codes are
// roundings of exact quotients: a quotient in fp32 falls on the middle of two codes only if the
// exact one does, since element, factor (4 bits) and middle (3 bits) all are fp32 values. Writing
// 68,000 rows of eight heads (D = 128, bf16) takes 90 us, 4.0 TB/s: warps wait for loads, of which each
// has one unit ahead, and convert meanwhile (57 % of issue slots). Reading them back takes 73.5, 4.9 TB/s.
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
  float* weights;                // [num_pages, Nk, page_size]: 0 for the rows of an append; or nullptr
  int lane_shift;                // log2(LG)
  int row_shift;                 // log2(rows of a block)
};

enum : int { kCopy = 0, kCast = 1, kStatic = 2, kScale = 3, kGroup = 4 };

constexpr int kMaxRows = 32;  // rows of a block

// Where a row lies in the cache: its sequence, page (-1: nowhere) and row of the page.
struct Place {
  long long page;
  int b, row;
};

__device__ __forceinline__ Place find_place(const CopyParams& p, long long t) {
  Place w;
  w.page = -1;
  w.b = w.row = 0;
  if (t >= p.c.T) return w;
  w.b = seq_of_row(p.c, t);
  const PagedSeq s = paged_seq(p.c, w.b);
  if (!s.ok || s.n > s.Lk || t < s.t0 || t >= s.t0 + s.n) return w;
  const long long pos = s.Lk - s.n + (t - s.t0);
  w.page = page_at(p.c, s, pos);
  w.row = (int)(pos & (page_size(p.c) - 1));
  if (w.page < 0) report(p.c, HSTU_DEVERR_OFFSETS);
  return w;
}

// The places of the block's rows, and (with a status word) a check of every sequence, those
// without rows too.
__device__ __forceinline__ void find_places(const CopyParams& p, Place* places) {
  if (threadIdx.x < (1u << p.row_shift))
    places[threadIdx.x] = find_place(p, ((long long)blockIdx.x << p.row_shift) + threadIdx.x);
  if (p.c.status) {
    const long long threads = (long long)gridDim.x * kThreads;
    for (long long b = (long long)blockIdx.x * kThreads + threadIdx.x; b < p.c.B; b += threads) {
      const PagedSeq s = paged_seq(p.c, b);
      if (!s.ok || s.n > s.Lk) report(p.c, HSTU_DEVERR_OFFSETS);
    }
  }
  __syncthreads();
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

// The same for E2M1 rows: 2688 = 1.3125 * 2^11 (448 times 6).
__device__ __forceinline__ int group_exponent(uint32_t bits) {
  const int e = (int)(bits >> 23) - 127 - 11 + ((bits & 0x7fffffu) > 0x280000u ? 1 : 0);
  return e < kMinExp ? kMinExp : e;
}

// Sixteen elements times 2^-e as E2M1 codes and their factor's E4M3 code. own: the largest magnitude's
// bits, infinities and NaN included. A NaN makes the factor one. Quotients are products with the
// factor's reciprocal, corrected once by the exact residual, which rounds them as a division does
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990): two
// of them in three packed instructions (68,000 rows of eight heads 90 us, with sixteen divisions a lane
// 154).
__device__ __forceinline__ uint2 group_codes(const float (&x)[16], uint32_t own, int e,
                                             uint32_t& factor) {
  const float mul = __uint_as_float((uint32_t)(127 - e) << 23);
  float top = __uint_as_float(own) * mul;
  float y[16];
#pragma unroll
  for (int i = 0; i < 16; i += 2) ptx::mul_f32x2(y[i], y[i + 1], x[i], x[i + 1], mul, mul);
  bool nan = false;
  if (own >= 0x7f800000u) {
    top = 2688.0f;  // (an infinity; a NaN alone counts as one, too)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      nan |= x[i] != x[i];
      y[i] = fminf(fmaxf(y[i], -2688.0f), 2688.0f);
    }
  }
  factor = ptx::cvt_e4m3x2_f32(top / 6.0f, 0.0f) & 0xffu;
  const float f = e4m3_value(factor), r = factor ? 1.0f / f : 0.0f;
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    float q0, q1, d0, d1;
    ptx::mul_f32x2(q0, q1, y[i], y[i + 1], r, r);
    ptx::fma_f32x2(d0, d1, q0, q1, -f, -f, y[i], y[i + 1]);
    ptx::fma_f32x2(y[i], y[i + 1], d0, d1, r, r, q0, q1);
  }
  if (nan) factor = 0x7fu;
  return make_uint2(f32x8_to_e2m1(y), f32x8_to_e2m1(y + 8));
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
// bits; infinities and NaN (bits from 0x7f800000 on) are left out. own: the lane's, with those.
__device__ __forceinline__ uint32_t row_max(const float (&x)[16], bool lane_ok, int lanes,
                                            uint32_t& own) {
  uint32_t m = 0;
  own = 0;
  if (lane_ok) {
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    own = m;
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

// One (row, head) of a block: group x takes row x mod rows of head x / rows.
struct Unit {
  int r, hk;
  long long t;
  bool ok;  // the row exists and this lane holds elements of it
};
__device__ __forceinline__ Unit unit_at(const CopyParams& p, int x, int d0) {
  Unit u;
  u.r = x & ((1 << p.row_shift) - 1);
  u.hk = x >> p.row_shift;
  u.t = ((long long)blockIdx.x << p.row_shift) + u.r;
  u.ok = u.hk < p.c.Nk && u.t < p.c.T && d0 < p.c.D;
  return u;
}

template <typename T>
__device__ __forceinline__ void load_rows(const CopyParams& p, const Unit& u, int d0,
                                          float (&x)[2][16]) {
  if (!u.ok) return;
  load16(static_cast<const T*>(p.k) + u.t * p.k_stride + (long long)u.hk * p.c.D + d0, x[0]);
  load16(static_cast<const T*>(p.v) + u.t * p.v_stride + (long long)u.hk * p.c.D + d0, x[1]);
}

// CLEAR: the rows' entries of the weights become 0. (As a branch on the pointer, every append was
// 0.1 us slower, of prompts 0.4.)
template <typename T, int MODE, bool CLEAR>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const CopyParams p) {
  __shared__ Place places[kMaxRows];
  const int groups = kThreads >> p.lane_shift, units = p.c.Nk << p.row_shift;
  const int d0 = (threadIdx.x & ((1 << p.lane_shift) - 1)) * 16;
  int i = threadIdx.x >> p.lane_shift;
  float x[2][16];
  Unit u = unit_at(p, i, d0);
  load_rows<T>(p, u, d0, x);
  find_places(p, places);
  if constexpr (CLEAR) {
    for (int x = threadIdx.x; x < units; x += kThreads) {
      const Place w = places[x & ((1 << p.row_shift) - 1)];
      if (w.page >= 0)
        p.weights[((w.page * p.c.Nk + (x >> p.row_shift)) << p.c.page_shift) + w.row] = 0.f;
    }
  }
  // every lane of a warp makes the same number of rounds (the shuffles)
  for (int base = 0; base < units; base += groups, i += groups) {
    const Place w = places[u.r];
    const bool ok = u.ok && w.page >= 0;
#pragma unroll
    for (int plane = 0; plane < 2; ++plane) {
      uint32_t top = 0, own = 0;
      if constexpr (MODE == kScale || MODE == kGroup)
        top = row_max(x[plane], ok, 1 << p.lane_shift, own);
      if (!ok) continue;
      if constexpr (MODE == kGroup) {
        const int e = group_exponent(top);
        const long long r = scale_row(p.c, w.page, plane, w.row, u.hk);
        uint32_t factor;
        const uint2 codes = group_codes(x[plane], own, e, factor);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.c.cache) + (r * p.c.D + d0) / 2) = codes;
        p.c.group[(r * p.c.D + d0) / 16] = (uint8_t)factor;
        if (d0 == 0) p.c.scale[r] = (uint8_t)(e + 127);
        continue;
      }
      const long long at = cache_row(p.c, w.page, plane, w.row, u.hk) + d0;
      if constexpr (MODE == kCopy) {
        store16(static_cast<T*>(p.c.cache) + at, x[plane]);
      } else {
        uint8_t* dst = static_cast<uint8_t*>(p.c.cache) + at;
        if constexpr (MODE == kScale) {
          const int e = scale_exponent(top);
          store_codes(dst, x[plane], __uint_as_float((uint32_t)(127 - e) << 23));
          if (d0 == 0) p.c.scale[scale_row(p.c, w.page, plane, w.row, u.hk)] = (uint8_t)(e + 127);
        } else if constexpr (MODE == kStatic) {
          const float f = factor(p.c, plane ? p.c.v_ds : p.c.k_ds, w.b, u.hk);
#pragma unroll
          for (int e = 0; e < 16; ++e) x[plane][e] /= f;
          store_codes(dst, x[plane], 1.0f);
        } else {
          store_codes(dst, x[plane], 1.0f);
        }
      }
    }
    u = unit_at(p, i + groups, d0);
    load_rows<T>(p, u, d0, x);
  }
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const CopyParams p) {
  __shared__ Place places[kMaxRows];
  find_places(p, places);
  const int groups = kThreads >> p.lane_shift, units = p.c.Nk << p.row_shift;
  const int d0 = (threadIdx.x & ((1 << p.lane_shift) - 1)) * 16;
#pragma unroll 2
  for (int i = threadIdx.x >> p.lane_shift; i < units; i += groups) {
    const Unit u = unit_at(p, i, d0);
    const Place w = places[u.r];
    if (!u.ok || w.page < 0) continue;
    float x[2][16], f[2] = {1.0f, 1.0f};
#pragma unroll
    for (int plane = 0; plane < 2; ++plane) {
      if constexpr (MODE == kGroup) {
        const long long r = scale_row(p.c, w.page, plane, w.row, u.hk);
        f[plane] = scale_value(p.c.scale[r]) * e4m3_value(p.c.group[(r * p.c.D + d0) / 16]);
        load16_e2m1(static_cast<const uint8_t*>(p.c.cache) + (r * p.c.D + d0) / 2, x[plane]);
        continue;
      }
      const long long at = cache_row(p.c, w.page, plane, w.row, u.hk) + d0;
      if constexpr (MODE == kScale)
        f[plane] = scale_value(p.c.scale[scale_row(p.c, w.page, plane, w.row, u.hk)]);
      if constexpr (MODE == kStatic)
        f[plane] = factor(p.c, plane ? p.c.v_ds : p.c.k_ds, w.b, u.hk);
      if constexpr (MODE == kCopy)
        load16(static_cast<const T*>(p.c.cache) + at, x[plane]);
      else
        load16(static_cast<const uint8_t*>(p.c.cache) + at, x[plane]);
    }
#pragma unroll
    for (int plane = 0; plane < 2; ++plane) {
      if constexpr (MODE == kScale || MODE == kStatic || MODE == kGroup) {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[plane][e] *= f[plane];
      }
      store16(static_cast<T*>(plane ? p.v : p.k) + u.t * (plane ? p.v_stride : p.k_stride) +
                  (long long)u.hk * p.c.D + d0,
              x[plane]);
    }
  }
}

template <typename T>
cudaError_t launch(const CopyParams& p, bool append, int mode, unsigned grid, cudaStream_t st) {
#define HSTU_COPY(M)                                            \
  if (append && p.weights)                                      \
    kv_append_kernel<T, M, true><<<grid, kThreads, 0, st>>>(p); \
  else if (append)                                              \
    kv_append_kernel<T, M, false><<<grid, kThreads, 0, st>>>(p);\
  else                                                          \
    kv_read_kernel<T, M><<<grid, kThreads, 0, st>>>(p);         \
  break
  switch (mode) {
    case kCopy: HSTU_COPY(kCopy);
    case kCast: HSTU_COPY(kCast);
    case kStatic: HSTU_COPY(kStatic);
    case kGroup: HSTU_COPY(kGroup);
    default: HSTU_COPY(kScale);
  }
#undef HSTU_COPY
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_copy(const CacheView& c, void* k, void* v, long long k_stride,
                           long long v_stride, float* weights, int dtype, int fmt, bool append, int sms,
                           cudaStream_t stream) {
  CopyParams p = {};
  p.c = c;
  p.k = k;
  p.v = v;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.weights = weights;
  while ((16 << p.lane_shift) < c.D) ++p.lane_shift;
  // rows of a block: enough to give every group of lanes work, as few as keep the SMs busy
  const int groups = kThreads >> p.lane_shift;
  while ((1 << p.row_shift) < kMaxRows &&
         ((c.Nk << p.row_shift) < groups || (c.T >> p.row_shift) > 16ll * sms))
    ++p.row_shift;
  const long long blocks = (c.T + (1 << p.row_shift) - 1) >> p.row_shift;
  const unsigned grid = (unsigned)blocks;
  const int mode = fmt == kSame    ? kCopy
                   : fmt == kE2m1 ? kGroup
                   : c.scale      ? kScale
                   : c.k_ds       ? kStatic
                                  : kCast;
  if (dtype == HSTU_F32) return launch<float>(p, append, mode, grid, stream);
  if (dtype == HSTU_BF16) return launch<__nv_bfloat16>(p, append, mode, grid, stream);
  return launch<__half>(p, append, mode, grid, stream);
}

}  // namespace hstu
