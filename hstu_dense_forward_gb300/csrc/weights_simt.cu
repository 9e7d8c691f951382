// Attention weights of the cached keys from fp32 query rows, on CUDA cores (FFMA). A CTA holds 64 keys
// of one kv head in shared memory and passes over the packed query rows that see any of them, 64 at a
// time: a thread owns keys tx + 16 c and rows ty + 16 a, whose weights it adds up over the rows; the
// sums of the sixteen ty are joined in order at the end. Then the next 64 keys of its share.
#include <math_constants.h>

#include "common.cuh"
#include "evict_kernels.h"
#include "kernels.h"
#include "kv_cache.cuh"
#include "kv_kernels.h"
#include "rows_fp32.cuh"

namespace hstu {

namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.44269504088896340736f;

template <int D_>
struct Cfg {
  static constexpr int D = D_, BM = 64, BN = kWeightsSimtKeys, LD = D + 4;
  static constexpr int OFF_K = BM * LD, OFF_L = OFF_K + BN * LD, OFF_S = OFF_L + BM;
  static constexpr int OFF_ROW = OFF_S + 16 * BN;
  static constexpr int SMEM = 4 * OFF_ROW + BN * (int)sizeof(RowAt);
};

template <int D_, int FMT>
__global__ void __launch_bounds__(kThreads) weights_simt_kernel(const WeightsParams w, int slots) {
  using C = Cfg<D_>;
  constexpr int BM = C::BM, BN = C::BN, LD = C::LD;
  const SoftmaxParams& p = w.a;
  extern __shared__ float sm[];
  float* Qs = sm;             // [BM][LD]
  float* Ks = sm + C::OFF_K;  // [BN][LD]
  float* Ls = sm + C::OFF_L;  // [BM] base-2 logarithms of the rows' sums
  float* Ss = sm + C::OFF_S;  // [16][BN]
  RowAt* rows_at = reinterpret_cast<RowAt*>(sm + C::OFF_ROW);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, D = p.c.D;
  // (first keys first: with the causal mask more rows see them)
  const unsigned pairs = (unsigned)p.c.B * p.c.Nk;
  const int hk = (int)(blockIdx.x % pairs % p.c.Nk), b = (int)(blockIdx.x % pairs / p.c.Nk);
  const PagedSeq s = paged_seq(p.c, b);
  if (!attn_seq_ok(p, s)) {
    if (threadIdx.x == 0) report(p.c, HSTU_DEVERR_OFFSETS);
    return;
  }
  const long long rows = p.Nq ? s.n * p.G : 0;
  if (rows == 0 && w.accumulate) return;
  float fk = p.scale_log2;
  if (p.c.k_ds) fk *= p.c.k_ds[(long long)b * p.c.ds_b + (long long)hk * p.c.ds_h];
  const float* q = static_cast<const float*>(p.q);
  for (long long k0 = (long long)(blockIdx.x / pairs) * BN; k0 < s.Lk;
       k0 += (long long)slots * BN) {
    __syncthreads();  // the step before has been read
    if (threadIdx.x < BN) {
      const long long n = k0 + threadIdx.x;
      RowAt at = {-1, 0};
      if (n < s.Lk) {
        const long long page = page_at(p.c, s, n), row = n & (page_size(p.c) - 1);
        if (page >= 0) {
          at.scale = scale_row(p.c, page, 0, row, hk);
          at.elems = FMT == kE2m1 ? at.scale * D : cache_row(p.c, page, 0, row, hk);
        } else {
          report(p.c, HSTU_DEVERR_OFFSETS);
        }
      }
      rows_at[threadIdx.x] = at;
    }
    __syncthreads();
    constexpr int NE = Piece<FMT>::N;
#pragma unroll 4
    for (int x = threadIdx.x; x < BN * (D_ / NE); x += kThreads) {
      const int r = x / (D_ / NE), d = x % (D_ / NE) * NE;
      const RowAt at = rows_at[r];
      Piece<FMT> k;
      k.none();
      if (at.elems >= 0 && d < D) k.load(p.c, at.elems + d, at.scale);
      k.store(Ks + r * LD + d);
    }
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    // rows that see key k0 or a later one
    long long m0 = 0;
    if (p.causal) m0 = max(0ll, k0 - (s.Lk - s.n)) * p.G / BM * BM;
    for (; m0 < rows; m0 += BM) {
      __syncthreads();
      const int have = (int)min((long long)BM, rows - m0);
      for (int x = threadIdx.x; x < (have + 15) / 16 * 16 * (D_ / 4); x += kThreads) {
        const int r = x / (D_ / 4), d = x % (D_ / 4) * 4;
        const long long pr = m0 + r;
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < have && d < D)
          f = *reinterpret_cast<const float4*>(q + (s.t0 + pr / p.G) * p.q_stride +
                                               (hk * p.G + pr % p.G) * (long long)D + d);
        *reinterpret_cast<float4*>(Qs + r * LD + d) = f;
      }
      if (threadIdx.x < have) {
        const long long pr = m0 + threadIdx.x;
        Ls[threadIdx.x] = w.lse[(s.t0 + pr / p.G) * p.Nq + hk * p.G + pr % p.G] * kLog2e;
      }
      __syncthreads();
      // (sixteen rows at a time: single tokens have few)
      auto product = [&](auto tag, int a0) {
        constexpr int RA = decltype(tag)::value;
        float sc[RA][4] = {};
#pragma unroll 4
        for (int d = 0; d < D_; d += 4) {
          float4 qa[RA], kb[4];
#pragma unroll
          for (int a = 0; a < RA; ++a)
            qa[a] = *reinterpret_cast<const float4*>(Qs + (ty + 16 * (a0 + a)) * LD + d);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            kb[c] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * c) * LD + d);
#pragma unroll
          for (int a = 0; a < RA; ++a)
#pragma unroll
            for (int c = 0; c < 4; ++c) sc[a][c] = dot4(qa[a], kb[c], sc[a][c]);
        }
#pragma unroll
        for (int a = 0; a < RA; ++a) {
          const int r = ty + 16 * (a0 + a);
          if (r >= have) continue;
          const long long lim = p.causal ? s.Lk - s.n + (m0 + r) / p.G + 1 : s.Lk;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (k0 + tx + 16 * c < lim) sum[c] += exp2f(fmaf(sc[a][c], fk, -Ls[r]));
        }
      };
      if (have > 16)
        product(std::integral_constant<int, 4>{}, 0);
      else
        product(std::integral_constant<int, 1>{}, 0);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) Ss[ty * BN + tx + 16 * c] = sum[c];
    __syncthreads();
    if (threadIdx.x < BN && rows_at[threadIdx.x].elems >= 0) {
      float total = 0.f;
#pragma unroll
      for (int y = 0; y < 16; ++y) total += Ss[y * BN + threadIdx.x];
      const long long n = k0 + threadIdx.x;
      float* to = w.weights + ((page_at(p.c, s, n) * p.c.Nk + hk) << p.c.page_shift) +
                  (n & (page_size(p.c) - 1));
      *to = w.accumulate ? *to + total : total;
    }
  }
}

template <int D, int FMT>
cudaError_t launch(const WeightsParams& w, int slots, cudaStream_t stream) {
  using C = Cfg<D>;
  auto* kernel = weights_simt_kernel<D, FMT>;
  static std::atomic<unsigned long long> done;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), C::SMEM, done);
  if (e != cudaSuccess) return e;
  const long long blocks = (long long)w.a.c.B * w.a.c.Nk * slots;
  kernel<<<dim3((unsigned)blocks), kThreads, C::SMEM, stream>>>(w, slots);
  return cudaGetLastError();
}

template <int FMT>
cudaError_t launch_dim(const WeightsParams& w, int slots, cudaStream_t stream) {
  if (w.a.c.D > 128) return launch<256, FMT>(w, slots, stream);
  if (w.a.c.D > 64) return launch<128, FMT>(w, slots, stream);
  return launch<64, FMT>(w, slots, stream);
}

}  // namespace

cudaError_t launch_weights_simt(const WeightsParams& w, int fmt, int slots, cudaStream_t stream) {
  return fmt == kE4m3   ? launch_dim<kE4m3>(w, slots, stream)
         : fmt == kE2m1 ? launch_dim<kE2m1>(w, slots, stream)
                        : launch_dim<kSame>(w, slots, stream);
}

}  // namespace hstu
