// Rows of the paged KV cache as fp32 operands of the CUDA-core kernels.
#pragma once
#include "kv_cache.cuh"

namespace hstu {

// A cached row: the place of its K elements, and of their scale. V's lie a plane further on.
struct RowAt {
  long long elems;  // -1: no such row
  long long scale;
};

// What one access of a thread takes from the cache, until it is written to shared memory: four
// fp32 elements, or eight codes with their row's scale (and their group's factor).
template <int FMT>
struct Piece;
template <>
struct Piece<kSame> {
  static constexpr int N = 4;
  float4 x;
  __device__ __forceinline__ void none() { x = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const CacheView& c, long long elems, long long) {
    x = *reinterpret_cast<const float4*>(static_cast<const float*>(c.cache) + elems);
  }
  __device__ __forceinline__ void store(float* at) const { *reinterpret_cast<float4*>(at) = x; }
};
template <>
struct Piece<kE4m3> {
  static constexpr int N = 8;
  uint2 x;
  uint8_t scale;
  __device__ __forceinline__ void none() {
    x = make_uint2(0u, 0u);
    scale = 127;
  }
  __device__ __forceinline__ void load(const CacheView& c, long long elems, long long at) {
    x = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.cache) + elems);
    scale = c.scale ? c.scale[at] : 127;
  }
  // (every second four lanes write their second half first: eight lanes, one access of shared
  // memory, then lie in different banks)
  __device__ __forceinline__ void store(float* at) const {
    const float e = scale_value(scale);
    float4 f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t lo, hi;
      e4m3x4_to_f16x2(i ? x.y : x.x, lo, hi);
      const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&lo));
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      f[i] = make_float4(u.x * e, u.y * e, v.x * e, v.y * e);
    }
    const bool turn = threadIdx.x & 4;
    *reinterpret_cast<float4*>(at + (turn ? 4 : 0)) = turn ? f[1] : f[0];
    *reinterpret_cast<float4*>(at + (turn ? 0 : 4)) = turn ? f[0] : f[1];
  }
};

template <>
struct Piece<kE2m1> {
  static constexpr int N = 8;
  uint32_t x;
  uint8_t scale, group;
  __device__ __forceinline__ void none() {
    x = 0u;
    scale = 127;
    group = 0;
  }
  // (elems: the row's first element, plus d, in a layout of heads before rows)
  __device__ __forceinline__ void load(const CacheView& c, long long elems, long long at) {
    x = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(c.cache) + elems / 2);
    group = c.group[elems / 16];
    scale = c.scale[at];
  }
  __device__ __forceinline__ void store(float* at) const {
    const float e = scale_value(scale) * e4m3_value(group);
    uint32_t h[4];
    e2m1x8_to_f16x2(x, h);
    float4 f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&h[2 * i]));
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[2 * i + 1]));
      f[i] = make_float4(u.x * e, u.y * e, v.x * e, v.y * e);
    }
    const bool turn = threadIdx.x & 4;
    *reinterpret_cast<float4*>(at + (turn ? 4 : 0)) = turn ? f[1] : f[0];
    *reinterpret_cast<float4*>(at + (turn ? 0 : 4)) = turn ? f[0] : f[1];
  }
};

// Sixteen elements of a key that lane j of its group holds, as four float4: E4M3 elements
// 16 j .., fp32 ones 4 (j + i D / 16) .. in piece i, so that a group's loads are contiguous.
// E4M3 elements stay codes until they are used (with their row's scale, which multiplies a score
// and a weight instead of every element), so that more of them are on their way at a time.
template <int FMT>
struct FewRow;
template <>
struct FewRow<kSame> {
  float4 x[4];
  template <int D_>
  __device__ __forceinline__ void load(const CacheView& c, int page, int plane, int row,
                                       int hk, int j) {
    const float* at = static_cast<const float*>(c.cache) + cache_row(c, page, plane, row, hk);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = 4 * (j + i * (D_ / 16));
      x[i] = page >= 0 && d < c.D ? *reinterpret_cast<const float4*>(at + d)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __device__ __forceinline__ void get(float4 (&f)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = x[i];
  }
  __device__ __forceinline__ float factor() const { return 1.f; }
};
template <>
struct FewRow<kE4m3> {
  uint4 x;
  uint8_t scale;
  template <int D_>
  __device__ __forceinline__ void load(const CacheView& c, int page, int plane, int row,
                                       int hk, int j) {
    x = make_uint4(0u, 0u, 0u, 0u);
    scale = 127;
    if (page < 0) return;
    if (16 * j < c.D)
      x = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(c.cache) +
                                          cache_row(c, page, plane, row, hk) + 16 * j);
    if (c.scale) scale = c.scale[scale_row(c, page, plane, row, hk)];
  }
  __device__ __forceinline__ void get(float4 (&f)[4]) const {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t lo, hi;
      e4m3x4_to_f16x2(w[i], lo, hi);
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
      const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      f[i] = make_float4(a.x, a.y, b.x, b.y);
    }
  }
  __device__ __forceinline__ float factor() const { return scale_value(scale); }
};
template <>
struct FewRow<kE2m1> {
  uint2 x;
  uint8_t scale, group;
  template <int D_>
  __device__ __forceinline__ void load(const CacheView& c, int page, int plane, int row,
                                       int hk, int j) {
    x = make_uint2(0u, 0u);
    scale = 127;
    group = 0;
    if (page < 0) return;
    const long long r = scale_row(c, page, plane, row, hk);
    if (16 * j < c.D) {
      x = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.cache) +
                                          r * (c.D / 2) + 8 * j);
      group = c.group[r * (c.D / 16) + j];
    }
    scale = c.scale[r];
  }
  __device__ __forceinline__ void get(float4 (&f)[4]) const {
    const float g = e4m3_value(group);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      uint32_t h[4];
      e2m1x8_to_f16x2(w ? x.y : x.x, h);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h[2 * i]));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h[2 * i + 1]));
        f[2 * w + i] = make_float4(a.x * g, a.y * g, b.x * g, b.y * g);
      }
    }
  }
  __device__ __forceinline__ float factor() const { return scale_value(scale); }
};
// First of the four elements in piece i of lane j.
template <int D_, int FMT>
__device__ __forceinline__ int few_dim(int i, int j) {
  return FMT != kSame ? 16 * j + 4 * i : 4 * (j + i * (D_ / 16));
}

__device__ __forceinline__ float dot4(const float4& a, const float4& b, float s) {
  return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, s))));
}

}  // namespace hstu
