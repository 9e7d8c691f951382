// fp32 softmax attention over the paged KV cache on CUDA cores (FFMA), with the running maximum m
// and sum l of the softmax in base 2:
//   x = scale_log2 * Q K^T, m' = max(m, x), P = 2^(x - m'), l = 2^(m - m') l + sum P,
//   O = 2^(m - m') O + P V,                        out = O / l, log2 of the sum = m + log2 l.
// A CTA takes packed query rows of one kv head (packed row r of a sequence is query token r / G,
// head hk * G + r % G, so that the G heads that share a kv head share its loads) and one range of
// the keys; a second kernel joins the ranges.
//
// softmax_simt_kernel: 64 rows, 256 threads (16 x 16), in steps of BN keys. A thread owns rows
// ty + 16 a, of the scores keys tx + 16 c and of the output columns 4 tx + 64 u .. + 3; every
// operand comes from shared memory in float4 (four elements of the head dim, or four keys), so
// that a step spends four times as many FMAs as loads. What bounds it is shared memory: 773 tokens
// over 2275 cached ones, 20 heads of 4, D = 256, take 1171 us, 36 TFLOP/s, D = 128 639.
//
// softmax_few_kernel: 4 rows, for calls of at most 16, where reading the cache is what counts:
// D / 16 lanes hold a key, two keys at a time, straight from the cache in registers, and every
// group of lanes keeps a softmax of its own keys until the end. 128 sequences of one token over
// some 1500 keys of eight heads, D = 128: 288 us, 5.6 TB/s; over E4M3 rows, a quarter of the
// bytes, the instructions bound it: 281 us (with two keys at a time 546, its loads too few).
#include <math_constants.h>

#include "common.cuh"
#include "kernels.h"
#include "kv_cache.cuh"
#include "kv_kernels.h"
#include "ptx.cuh"

namespace hstu {

namespace {

constexpr int kThreads = 256;
constexpr float kLn2 = 0.69314718055994530942f;

// A cached row: the place of its K elements, and of their scale. V's lie a plane further on.
struct RowAt {
  long long elems;  // -1: no such row
  long long scale;
};

template <int D_, bool E4M3>
struct Cfg {
  static constexpr int D = D_, BM = 64;
  // Keys of a step: 64 spend more FMAs per load of the scores' operands, 32 leave an SM a second
  // CTA at D = 128, which E4M3 rows, whose conversion waits, need more (773 tokens over 2275, 20
  // heads, with the slower loads of sixteen elements a thread: D = 256 1479 us with 32 and 1336
  // with 64, D = 128 773 and 716, over E4M3 725 and 730).
  static constexpr int BN = D == 128 && E4M3 ? 32 : 64;
  static constexpr int RA = BM / 16, CK = BN / 16, U = D / 64;
  static constexpr int LD = D + 4, LDP = BN + 4;  // padded rows: conflict-free float4 reads
  static constexpr int OFF_K = BM * LD, OFF_V = OFF_K + BN * LD, OFF_P = OFF_V + BN * D;
  static constexpr int OFF_ROW = OFF_P + BM * LDP;  // where the step's rows lie
  static constexpr int SMEM = 4 * OFF_ROW + BN * (int)sizeof(RowAt);
};

// What one access of a thread takes from the cache, until it is written to shared memory: four
// fp32 elements, or eight E4M3 codes with their row's scale.
template <bool E4M3>
struct Piece;
template <>
struct Piece<false> {
  static constexpr int N = 4;
  float4 x;
  __device__ __forceinline__ void none() { x = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const CacheView& c, long long elems, long long) {
    x = *reinterpret_cast<const float4*>(static_cast<const float*>(c.cache) + elems);
  }
  __device__ __forceinline__ void store(float* at) const { *reinterpret_cast<float4*>(at) = x; }
};
template <>
struct Piece<true> {
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

__device__ __forceinline__ float dot4(const float4& a, const float4& b, float s) {
  return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, s))));
}

template <int D_, bool E4M3>
__global__ void __launch_bounds__(kThreads) softmax_simt_kernel(const SoftmaxParams p, int tiles) {
  using C = Cfg<D_, E4M3>;
  constexpr int BM = C::BM, BN = C::BN;
  extern __shared__ float sm[];
  const int D = p.c.D;
  float* Qs = sm;             // [BM][LD]
  float* Ks = sm + C::OFF_K;  // [BN][LD]
  float* Vs = sm + C::OFF_V;  // [BN][D_]
  float* Ps = sm + C::OFF_P;  // [BM][LDP]
  RowAt* rows_at = reinterpret_cast<RowAt*>(sm + C::OFF_ROW);  // [BN]
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;

  // block: sequence b, row tile (later tiles first: with the causal mask they see more
  // keys), kv head; blockIdx.y: key range
  const long long blk = blockIdx.x;
  const int hk = (int)(blk % p.c.Nk);
  const int tile = tiles - 1 - (int)(blk / p.c.Nk % tiles);
  const int b = (int)(blk / p.c.Nk / tiles);
  const int split = blockIdx.y;
  const PagedSeq s = paged_seq(p.c, b);
  if (!attn_seq_ok(p, s)) {
    if (threadIdx.x == 0) report(p.c, HSTU_DEVERR_OFFSETS);
    return;
  }
  const long long rows = s.n * p.G, m0 = (long long)tile * BM;
  const KeyRanges kr = key_ranges(p, s.Lk);
  const int nsplit = kr.count;
  if (m0 >= rows || split >= nsplit) return;
  // keys any row of the tile may see, within the range
  const long long last = (min(m0 + BM, rows) - 1) / p.G;  // last query token of the tile
  long long kend = s.Lk;
  if (p.causal) kend = min(kend, s.Lk - s.n + last + 1);
  const long long k0 = split * kr.keys;
  kend = min(kend, k0 + kr.keys);

  // rows of zeros and columns of zeros where there are none
  const float* q = static_cast<const float*>(p.q);
  for (int x = threadIdx.x; x < BM * (D_ / 4); x += kThreads) {
    const int r = x / (D_ / 4), d = x % (D_ / 4) * 4;
    const long long pr = m0 + r;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (pr < rows && d < D)
      f = *reinterpret_cast<const float4*>(q + (s.t0 + pr / p.G) * p.q_stride +
                                           (hk * p.G + pr % p.G) * (long long)D + d);
    *reinterpret_cast<float4*>(Qs + r * C::LD + d) = f;
  }
  float fk = p.scale_log2, fv = 1.f;  // static factors fold into the scale and the output
  if (p.c.k_ds) {
    fk *= p.c.k_ds[(long long)b * p.c.ds_b + (long long)hk * p.c.ds_h];
    fv = p.c.v_ds[(long long)b * p.c.ds_b + (long long)hk * p.c.ds_h];
  }
  float4 acc[C::RA][C::U];
  float m[C::RA], l[C::RA];
  long long lim[C::RA];  // keys that each row sees: [0, lim)
#pragma unroll
  for (int a = 0; a < C::RA; ++a) {
    m[a] = -CUDART_INF_F;
    l[a] = 0.f;
    const long long pr = m0 + ty + 16 * a;
    lim[a] = pr >= rows ? 0 : p.causal ? s.Lk - s.n + pr / p.G + 1 : s.Lk;
    lim[a] = min(lim[a], kend);
#pragma unroll
    for (int u = 0; u < C::U; ++u) acc[a][u] = make_float4(0.f, 0.f, 0.f, 0.f);
  }

  // One thread a row loads the next step's page id before this step's products and looks at it
  // behind them.
  const long long plane = (long long)p.c.Nk * D << p.c.page_shift;
  const long long scale_plane = (long long)p.c.Nk << p.c.page_shift;
  long long id64 = 0;
  int id32 = 0;
  auto load_id = [&](long long n) {
    if (threadIdx.x >= BN || n >= kend) return;
    const long long at = s.po + (n >> p.c.page_shift);
    if (p.c.index64)
      id64 = static_cast<const long long*>(p.c.page_ids)[at];
    else
      id32 = static_cast<const int*>(p.c.page_ids)[at];
  };
  load_id(k0 + threadIdx.x);
  for (long long n0 = k0; n0 < kend; n0 += BN) {
    __syncthreads();  // previous step finished with Ks/Vs/Ps
    if (threadIdx.x < BN) {
      const long long n = n0 + threadIdx.x, page = p.c.index64 ? id64 : id32;
      RowAt w = {-1, 0};
      if (n < kend) {
        if (page >= 0 && page < p.c.num_pages) {
          w.elems = cache_row(p.c, page, 0, n & (page_size(p.c) - 1), hk);
          w.scale = scale_row(p.c, page, 0, n & (page_size(p.c) - 1), hk);
        } else {
          report(p.c, HSTU_DEVERR_OFFSETS);  // (a row of zeros then)
        }
      }
      rows_at[threadIdx.x] = w;
    }
    __syncthreads();
    // A warp's accesses to the cache and to shared memory are contiguous (with sixteen elements a
    // thread a fifth of all cycles of shared memory were bank conflicts: D = 256 1336 us instead
    // of 1171), and up to sixteen of a thread are on their way at a time.
    constexpr int NE = Piece<E4M3>::N, NX = BN * (D_ / NE) / kThreads, NB = NX < 8 ? NX : 8;
#pragma unroll 1
    for (int x0 = 0; x0 < NX; x0 += NB) {
      Piece<E4M3> kx[NB], vx[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int x = (x0 + i) * kThreads + threadIdx.x, r = x / (D_ / NE), d = x % (D_ / NE) * NE;
        const RowAt w = rows_at[r];
        kx[i].none();
        vx[i].none();
        if (w.elems >= 0 && d < D) {
          kx[i].load(p.c, w.elems + d, w.scale);
          vx[i].load(p.c, w.elems + plane + d, w.scale + scale_plane);
        }
      }
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int x = (x0 + i) * kThreads + threadIdx.x, r = x / (D_ / NE), d = x % (D_ / NE) * NE;
        kx[i].store(Ks + r * C::LD + d);
        vx[i].store(Vs + r * D_ + d);
      }
    }
    load_id(n0 + BN + threadIdx.x);
    __syncthreads();
    // scores of rows ty + 16a, keys tx + 16c
    float sc[C::RA][C::CK];
#pragma unroll
    for (int a = 0; a < C::RA; ++a)
#pragma unroll
      for (int c = 0; c < C::CK; ++c) sc[a][c] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D_; d += 4) {
      float4 qa[C::RA], kb[C::CK];
#pragma unroll
      for (int a = 0; a < C::RA; ++a)
        qa[a] = *reinterpret_cast<const float4*>(Qs + (ty + 16 * a) * C::LD + d);
#pragma unroll
      for (int c = 0; c < C::CK; ++c)
        kb[c] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * c) * C::LD + d);
#pragma unroll
      for (int a = 0; a < C::RA; ++a)
#pragma unroll
        for (int c = 0; c < C::CK; ++c) sc[a][c] = dot4(qa[a], kb[c], sc[a][c]);
    }
#pragma unroll
    for (int a = 0; a < C::RA; ++a) {
      float top = -CUDART_INF_F;
#pragma unroll
      for (int c = 0; c < C::CK; ++c) {
        sc[a][c] = n0 + tx + 16 * c < lim[a] ? sc[a][c] * fk : -CUDART_INF_F;
        top = fmaxf(top, sc[a][c]);
      }
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float mn = fmaxf(m[a], top);
      const float base = mn == -CUDART_INF_F ? 0.f : mn;  // no key yet: weights 2^-inf = 0
      const float corr = exp2f(m[a] - base);
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < C::CK; ++c) {
        const float w = exp2f(sc[a][c] - base);
        sum += w;
        Ps[(ty + 16 * a) * C::LDP + tx + 16 * c] = w;
      }
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      l[a] = l[a] * corr + sum;
      m[a] = mn;
#pragma unroll
      for (int u = 0; u < C::U; ++u) {
        acc[a][u].x *= corr;
        acc[a][u].y *= corr;
        acc[a][u].z *= corr;
        acc[a][u].w *= corr;
      }
    }
    __syncthreads();
#pragma unroll 2
    for (int j = 0; j < BN; j += 4) {
      float4 pa[C::RA];
#pragma unroll
      for (int a = 0; a < C::RA; ++a)
        pa[a] = *reinterpret_cast<const float4*>(Ps + (ty + 16 * a) * C::LDP + j);
#pragma unroll
      for (int u = 0; u < C::U; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(Vs + (j + i) * D_ + tx * 4 + 64 * u);
#pragma unroll
          for (int a = 0; a < C::RA; ++a) {
            const float w = i == 0 ? pa[a].x : i == 1 ? pa[a].y : i == 2 ? pa[a].z : pa[a].w;
            acc[a][u].x = fmaf(w, v.x, acc[a][u].x);
            acc[a][u].y = fmaf(w, v.y, acc[a][u].y);
            acc[a][u].z = fmaf(w, v.z, acc[a][u].z);
            acc[a][u].w = fmaf(w, v.w, acc[a][u].w);
          }
        }
    }
  }
#pragma unroll
  for (int a = 0; a < C::RA; ++a) {
    const long long pr = m0 + ty + 16 * a;
    if (pr >= rows) continue;
    const long long row = (s.t0 + pr / p.G) * p.Nq + hk * p.G + pr % p.G;  // of out and lse
    const float inv = l[a] > 0.f ? fv / l[a] : l[a];  // (a NaN sum stays one)
    const float log2sum = l[a] == 0.f ? -CUDART_INF_F : m[a] + log2f(l[a]);
    float* dst = nsplit > 1 ? p.part_o + ((long long)split * p.c.T * p.Nq + row) * D
                            : static_cast<float*>(p.out) + row * D;
#pragma unroll
    for (int u = 0; u < C::U; ++u) {
      const int d = tx * 4 + 64 * u;
      if (d < D)
        *reinterpret_cast<float4*>(dst + d) = make_float4(acc[a][u].x * inv, acc[a][u].y * inv,
                                                          acc[a][u].z * inv, acc[a][u].w * inv);
    }
    if (tx == 0) {
      if (nsplit > 1)
        p.part_lse[(long long)split * p.c.T * p.Nq + row] = log2sum;
      else if (p.lse)
        p.lse[row] = log2sum * kLn2;
    }
  }
}

constexpr int kFewRows = 4, kFewThreads = 128;

// Sixteen elements of a key that lane j of its group holds, as four float4: E4M3 elements
// 16 j .., fp32 ones 4 (j + i D / 16) .. in piece i, so that a group's loads are contiguous.
// E4M3 elements stay codes until they are used (with their row's scale, which multiplies a score
// and a weight instead of every element), so that more of them are on their way at a time.
template <bool E4M3>
struct FewRow;
template <>
struct FewRow<false> {
  float4 x[4];
  template <int D_>
  __device__ __forceinline__ void load(const SoftmaxParams& p, int page, int plane, int row,
                                       int hk, int j) {
    const float* at = static_cast<const float*>(p.c.cache) + cache_row(p.c, page, plane, row, hk);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = 4 * (j + i * (D_ / 16));
      x[i] = page >= 0 && d < p.c.D ? *reinterpret_cast<const float4*>(at + d)
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
struct FewRow<true> {
  uint4 x;
  uint8_t scale;
  template <int D_>
  __device__ __forceinline__ void load(const SoftmaxParams& p, int page, int plane, int row,
                                       int hk, int j) {
    x = make_uint4(0u, 0u, 0u, 0u);
    scale = 127;
    if (page < 0) return;
    if (16 * j < p.c.D)
      x = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.c.cache) +
                                          cache_row(p.c, page, plane, row, hk) + 16 * j);
    if (p.c.scale) scale = p.c.scale[scale_row(p.c, page, plane, row, hk)];
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
// First of the four elements in piece i of lane j.
template <int D_, bool E4M3>
__device__ __forceinline__ int few_dim(int i, int j) {
  return E4M3 ? 16 * j + 4 * i : 4 * (j + i * (D_ / 16));
}

template <int D_, bool E4M3>
__global__ void __launch_bounds__(kFewThreads, 3) softmax_few_kernel(const SoftmaxParams p,
                                                                     int tiles) {
  constexpr int R = kFewRows, U = E4M3 ? 4 : 2, LPK = D_ / 16, KW = 32 / LPK;
  constexpr int WARPS = kFewThreads / 32, STEP = WARPS * U * KW;  // keys of a step
  __shared__ float4 qs[R][4][LPK];
  __shared__ float part_o[WARPS][R][D_], part_m[WARPS][R], part_l[WARPS][R];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = lane % LPK, g = lane / LPK;
  const uint32_t blk = blockIdx.x;
  const int hk = (int)(blk % (uint32_t)p.c.Nk);
  const int tile = tiles - 1 - (int)(blk / (uint32_t)p.c.Nk % (uint32_t)tiles);
  const int b = (int)(blk / (uint32_t)p.c.Nk / (uint32_t)tiles), split = blockIdx.y;
  const PagedSeq s = paged_seq(p.c, b);
  if (!attn_seq_ok(p, s)) {
    if (threadIdx.x == 0) report(p.c, HSTU_DEVERR_OFFSETS);
    return;
  }
  const long long rows = s.n * p.G, m0 = (long long)tile * R;
  const KeyRanges kr = key_ranges(p, s.Lk);
  if (m0 >= rows || split >= kr.count) return;
  // keys any row of the tile may see, within the range
  long long kend = s.Lk;
  if (p.causal) kend = min(kend, s.Lk - s.n + (min(m0 + R, rows) - 1) / p.G + 1);
  const long long k0 = split * kr.keys;
  kend = min(kend, k0 + kr.keys);

  const float* q = static_cast<const float*>(p.q);
  for (int x = threadIdx.x; x < R * 4 * LPK; x += kFewThreads) {
    const int r = x / (4 * LPK), i = x / LPK % 4, d = few_dim<D_, E4M3>(i, x % LPK);
    const long long pr = m0 + r;
    qs[r][i][x % LPK] = pr < rows && d < p.c.D
        ? *reinterpret_cast<const float4*>(q + (s.t0 + pr / p.G) * p.q_stride +
                                           (hk * p.G + pr % p.G) * (long long)p.c.D + d)
        : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float fk = p.scale_log2, fv = 1.f;  // static factors fold into the scale and the output
  if (p.c.k_ds) {
    fk *= p.c.k_ds[(long long)b * p.c.ds_b + (long long)hk * p.c.ds_h];
    fv = p.c.v_ds[(long long)b * p.c.ds_b + (long long)hk * p.c.ds_h];
  }
  __syncthreads();
  float m[R], l[R];
  float4 acc[R][4];
  const int keys = (int)(kend - k0);
  int lim[R];  // keys of the range that each row sees: [0, lim)
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = -CUDART_INF_F;
    l[r] = 0.f;
    const long long pr = m0 + r;
    const long long see = pr >= rows ? k0 : p.causal ? s.Lk - s.n + pr / p.G + 1 : s.Lk;
    lim[r] = (int)(min(see, kend) - k0);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[r][i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int mine = warp * U * KW + g;  // this group's keys of a step: mine, mine + KW
  auto page_of = [&](int n) { return n < keys ? (int)page_at(p.c, s, k0 + n) : -1; };
  int next[U];
#pragma unroll
  for (int u = 0; u < U; ++u) next[u] = page_of(mine + u * KW);
  for (int n0 = 0; n0 < keys; n0 += STEP) {
    FewRow<E4M3> k[U], v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int n = n0 + mine + u * KW, row = (int)(k0 + n) & (int)(page_size(p.c) - 1);
      const int page = next[u];
      if (page < 0 && n < keys) report(p.c, HSTU_DEVERR_OFFSETS);  // (a row of zeros then)
      k[u].template load<D_>(p, page, 0, row, hk, j);
      v[u].template load<D_>(p, page, 1, row, hk, j);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) next[u] = page_of(n0 + STEP + mine + u * KW);
    float x[U][R];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float4 f[4];
      k[u].get(f);
      const float fu = fk * k[u].factor();
#pragma unroll
      for (int r = 0; r < R; ++r) {
        x[u][r] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[u][r] = dot4(qs[r][i][j], f[i], x[u][r]);
#pragma unroll
        for (int d = 1; d < LPK; d <<= 1) x[u][r] += __shfl_xor_sync(0xffffffffu, x[u][r], d);
        x[u][r] = n0 + mine + u * KW < lim[r] ? x[u][r] * fu : -CUDART_INF_F;
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float top = m[r];
#pragma unroll
      for (int u = 0; u < U; ++u) top = fmaxf(top, x[u][r]);
      const float base = top == -CUDART_INF_F ? 0.f : top;  // no key yet: weights 2^-inf = 0
      if (__any_sync(0xffffffffu, top > m[r])) {
        const float corr = exp2f(m[r] - base);
        l[r] *= corr;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[r][i].x *= corr;
          acc[r][i].y *= corr;
          acc[r][i].z *= corr;
          acc[r][i].w *= corr;
        }
        m[r] = top;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        x[u][r] = exp2f(x[u][r] - base);
        l[r] += x[u][r];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float4 f[4];
      v[u].get(f);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float w = x[u][r] * v[u].factor();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[r][i].x = fmaf(w, f[i].x, acc[r][i].x);
          acc[r][i].y = fmaf(w, f[i].y, acc[r][i].y);
          acc[r][i].z = fmaf(w, f[i].z, acc[r][i].z);
          acc[r][i].w = fmaf(w, f[i].w, acc[r][i].w);
        }
      }
    }
  }
  // the warp's groups, then the CTA's warps
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float top = m[r];
#pragma unroll
    for (int d = LPK; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float corr = exp2f(m[r] - (top == -CUDART_INF_F ? 0.f : top));
    l[r] *= corr;
#pragma unroll
    for (int d = LPK; d < 32; d <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], d);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float e[4] = {acc[r][i].x * corr, acc[r][i].y * corr, acc[r][i].z * corr, acc[r][i].w * corr};
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int d = LPK; d < 32; d <<= 1) e[c] += __shfl_xor_sync(0xffffffffu, e[c], d);
      if (g == 0)
        *reinterpret_cast<float4*>(&part_o[warp][r][few_dim<D_, E4M3>(i, j)]) =
            make_float4(e[0], e[1], e[2], e[3]);
    }
    if (lane == 0) {
      part_m[warp][r] = top;
      part_l[warp][r] = l[r];
    }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < R * (D_ / 4); x += kFewThreads) {
    const int r = x / (D_ / 4), d = x % (D_ / 4) * 4;
    const long long pr = m0 + r;
    if (pr >= rows || d >= p.c.D) continue;
    float top = part_m[0][r];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) top = fmaxf(top, part_m[w][r]);
    float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float c = exp2f(part_m[w][r] - (top == -CUDART_INF_F ? 0.f : top));
      const float4 f = *reinterpret_cast<const float4*>(&part_o[w][r][d]);
      sum = fmaf(part_l[w][r], c, sum);
      o[0] = fmaf(f.x, c, o[0]);
      o[1] = fmaf(f.y, c, o[1]);
      o[2] = fmaf(f.z, c, o[2]);
      o[3] = fmaf(f.w, c, o[3]);
    }
    const long long row = (s.t0 + pr / p.G) * p.Nq + hk * p.G + pr % p.G;  // of out and lse
    const float inv = sum > 0.f ? fv / sum : sum;  // (a NaN sum stays one)
    float* dst = kr.count > 1 ? p.part_o + ((long long)split * p.c.T * p.Nq + row) * p.c.D
                              : static_cast<float*>(p.out) + row * p.c.D;
    *reinterpret_cast<float4*>(dst + d) =
        make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
    if (d == 0) {
      const float log2sum = sum == 0.f ? -CUDART_INF_F : top + log2f(sum);
      if (kr.count > 1)
        p.part_lse[(long long)split * p.c.T * p.Nq + row] = log2sum;
      else if (p.lse)
        p.lse[row] = log2sum * kLn2;
    }
  }
}

template <int D, bool E4M3>
cudaError_t launch(const SoftmaxParams& p, int rows, long long tiles, long long blocks,
                   cudaStream_t stream) {
  if (rows == kFewRows) {
    softmax_few_kernel<D, E4M3>
        <<<dim3((unsigned)blocks, p.splits), kFewThreads, 0, stream>>>(p, (int)tiles);
    return cudaGetLastError();
  }
  using C = Cfg<D, E4M3>;
  auto* kernel = softmax_simt_kernel<D, E4M3>;
  static std::atomic<unsigned long long> done;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), C::SMEM, done);
  if (e != cudaSuccess) return e;
  kernel<<<dim3((unsigned)blocks, p.splits), kThreads, C::SMEM, stream>>>(p, (int)tiles);
  return cudaGetLastError();
}

template <bool E4M3>
cudaError_t launch_dim(const SoftmaxParams& p, int rows, long long tiles, long long blocks,
                       cudaStream_t stream) {
  if (p.c.D > 128) return launch<256, E4M3>(p, rows, tiles, blocks, stream);
  if (p.c.D > 64) return launch<128, E4M3>(p, rows, tiles, blocks, stream);
  return launch<64, E4M3>(p, rows, tiles, blocks, stream);
}

}  // namespace

cudaError_t launch_softmax_simt(const SoftmaxParams& p, bool e4m3, int rows, long long tiles,
                                long long blocks, cudaStream_t stream) {
  return e4m3 ? launch_dim<true>(p, rows, tiles, blocks, stream)
              : launch_dim<false>(p, rows, tiles, blocks, stream);
}

}  // namespace hstu
