// Attention weights of the cached keys from fp32 query rows, on CUDA cores (FFMA).
//
// weights_simt_kernel: a CTA holds 64 keys of one kv head in shared memory and passes over the packed
// query rows that see any of them, 64 at a time: a thread owns keys tx + 16 c and rows ty + 16 a, whose
// weights it adds up over the rows; the sums of the sixteen ty are joined in order at the end. Then
// the next 64 keys of its share. Shared memory's loads of the operands bound it (the last 64 tokens of
// two sequences of some 10,000, two kv heads of four: 105 us, 23 TFLOP/s).
//
// weights_few_kernel: calls of at most 16 rows, where reading the keys counts: D / 16 lanes hold a key,
// straight from the cache in registers, and go through the rows (64 sequences of one token over some
// 2500 keys of four heads, D = 128: 67 us, 5.1 TB/s, with the kernel above 380).
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

constexpr int kFewRows = 16, kFewThreads = 128;

template <int D_, int FMT>
__global__ void __launch_bounds__(kFewThreads) weights_few_kernel(const WeightsParams w) {
  constexpr int U = FMT != kSame ? 4 : 2, LPK = D_ / 16, KW = 32 / LPK;
  constexpr int WARPS = kFewThreads / 32, STEP = WARPS * U * KW;  // keys of a step
  __shared__ float4 qs[kFewRows][4][LPK];
  __shared__ float logs[kFewRows];
  __shared__ int lims[kFewRows];  // keys of the range that each row sees: [0, lim)
  const SoftmaxParams& p = w.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = lane % LPK, g = lane / LPK;
  const int hk = (int)(blockIdx.x % (unsigned)p.c.Nk), b = (int)(blockIdx.x / (unsigned)p.c.Nk);
  const PagedSeq s = paged_seq(p.c, b);
  const long long all = p.Nq ? s.n * p.G : 0;
  if (!attn_seq_ok(p, s) || all > kFewRows) {
    if (threadIdx.x == 0) report(p.c, HSTU_DEVERR_OFFSETS);
    return;
  }
  const KeyRanges kr = key_ranges(p, s.Lk);
  const long long k0 = blockIdx.y * kr.keys, kend = min(s.Lk, k0 + kr.keys);
  const int rows = (int)all, keys = (int)(kend - k0);
  if (k0 >= kend || (rows == 0 && w.accumulate)) return;
  const float* q = static_cast<const float*>(p.q);
  for (int x = threadIdx.x; x < rows * 4 * LPK; x += kFewThreads) {
    const int r = x / (4 * LPK), i = x / LPK % 4, d = few_dim<D_, FMT>(i, x % LPK);
    qs[r][i][x % LPK] = d < p.c.D
        ? *reinterpret_cast<const float4*>(q + (s.t0 + r / p.G) * p.q_stride +
                                           (hk * p.G + r % p.G) * (long long)p.c.D + d)
        : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (threadIdx.x < rows) {
    const int r = threadIdx.x;
    logs[r] = w.lse[(s.t0 + r / p.G) * p.Nq + hk * p.G + r % p.G] * kLog2e;
    const long long see = p.causal ? s.Lk - s.n + r / p.G + 1 : s.Lk;
    lims[r] = (int)(min(see, kend) - k0);
  }
  float fk = p.scale_log2;
  if (p.c.k_ds) fk *= p.c.k_ds[(long long)b * p.c.ds_b + (long long)hk * p.c.ds_h];
  __syncthreads();
  const int mine = warp * U * KW + g;  // this group's keys of a step: mine, mine + KW ..
  auto page_of = [&](int n) { return n < keys ? (int)page_at(p.c, s, k0 + n) : -1; };
  int next[U];
#pragma unroll
  for (int u = 0; u < U; ++u) next[u] = page_of(mine + u * KW);
  for (int n0 = 0; n0 < keys; n0 += STEP) {
    FewRow<FMT> k[U];
    float* to[U];
    float old[U], sum[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int n = n0 + mine + u * KW, row = (int)(k0 + n) & (int)(page_size(p.c) - 1);
      const int page = next[u];
      if (page < 0 && n < keys) report(p.c, HSTU_DEVERR_OFFSETS);
      k[u].template load<D_>(p.c, page, 0, row, hk, j);
      to[u] = page >= 0 && j == 0
                  ? w.weights + (((long long)page * p.c.Nk + hk) << p.c.page_shift) + row
                  : nullptr;
      old[u] = w.accumulate && to[u] ? *to[u] : 0.f;
      sum[u] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) next[u] = page_of(n0 + STEP + mine + u * KW);
    float4 f[U][4];
    float fu[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      k[u].get(f[u]);
      fu[u] = fk * k[u].factor();
    }
    for (int r = 0; r < rows; ++r) {
      float4 qr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) qr[i] = qs[r][i][j];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) x = dot4(qr[i], f[u][i], x);
#pragma unroll
        for (int d = 1; d < LPK; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        if (n0 + mine + u * KW < lims[r]) sum[u] += exp2f(fmaf(x, fu[u], -logs[r]));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (to[u]) *to[u] = old[u] + sum[u];
  }
}

template <int D, int FMT>
cudaError_t launch(const WeightsParams& w, int slots, cudaStream_t stream) {
  if (slots == 0) {
    weights_few_kernel<D, FMT>
        <<<dim3((unsigned)(w.a.c.B * (long long)w.a.c.Nk), w.a.splits), kFewThreads, 0, stream>>>(w);
    return cudaGetLastError();
  }
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
