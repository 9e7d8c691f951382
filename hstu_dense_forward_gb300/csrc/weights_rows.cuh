// Attention weights of the cached keys from few query rows (single tokens), bf16 / fp16:
//   weights[j] (+)= sum_r 2^(x_rj - lse_r log2 e),   x_rj in base 2 as in softmax_rows.cuh,
// over the up to 16 packed rows r of a sequence and kv head. The scores are those of the attention of
// few rows, over the same ring of TMA loads without the values; a lane's four (eight) scores of two
// keys are summed over the rows by itself and then with the three lanes that hold the other rows.
// Nothing is kept between keys, so any number of CTAs divides them. 128 tokens over 1k-4k keys of four
// heads, D = 128: over bf16 keys 60 us, 6.0 TB/s with the weights, bound by reading; E4M3 42 (4.4 TB/s),
// where the fullest SM issues in 82 % of its cycles and the mean one in 64 %; E2M1 50.
#pragma once
#include "evict_kernels.h"
#include "softmax_rows.cuh"

namespace hstu {
namespace rows {

constexpr float kLog2e = 1.44269504088896340736f;

template <int D, int NT, bool BF16, int FMT>
__global__ void __launch_bounds__(Cfg<D, NT, BF16, FMT, 1>::THREADS, Cfg<D, NT, BF16, FMT, 1>::CTAS)
    weights_rows_kernel(const __grid_constant__ CUtensorMap tm_c, const WeightsParams w) {
  using C = Cfg<D, NT, BF16, FMT, 1>;
  const SoftmaxParams& p = w.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Item it;
  long long blk = blockIdx.x;
  if (p.by_length)
    blk = item_by_length(p, blk, gridDim.x, C::THREADS, reinterpret_cast<LengthOrder*>(smem));
  it.hk = (int)(blk % p.c.Nk);
  it.b = (int)(blk / p.c.Nk);
  it.split = blockIdx.y;
  it.s = paged_seq(p.c, it.b);
  it.rows = p.Nq ? it.s.n * p.G : 0;  // (of queries without heads none, however many tokens)
  if (!attn_seq_ok(p, it.s) || it.rows > C::RT) {
    if (threadIdx.x == 0) report(p.c, HSTU_DEVERR_OFFSETS);
    return;
  }
  const KeyRanges kr = key_ranges(p, it.s.Lk);
  it.nsplit = kr.count;
  it.m0 = 0;
  it.k0 = it.split * kr.keys;
  it.kend = min(it.s.Lk, it.k0 + kr.keys);
  if (it.k0 >= it.kend || (it.rows == 0 && w.accumulate)) return;
  Bars* bars = reinterpret_cast<Bars*>(smem + C::OFF_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int keys = (int)(it.kend - it.k0), n = (keys + C::KT - 1) / C::KT;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NST; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bars->full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->empty[s]), C::CW);
    }
    bars->abort = 0;
    ptx::fence_barrier_init();
    ptx::fence_proxy_async_smem();
  }
  __syncthreads();
  const int g = lane >> 2, c = lane & 3;
  if (warp == C::CW) {
    if (lane == 0) load_role<C>(p, bars, smem, it, n, &tm_c);
  } else {
    Queries<C> qs;
    load_queries<C>(p, it, keys, g, c, qs);
    float l2[NT][2];  // base-2 logarithms of the sums of rows 2c, 2c + 1; no row: its weights are 0
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const long long r = 8 * i + 2 * c + y;
        l2[i][y] = CUDART_INF_F;
        if (r < it.rows)
          l2[i][y] = w.lse[(it.s.t0 + r / p.G) * p.Nq + it.hk * p.G + r % p.G] * kLog2e;
      }
    const int mine = g + 8 * (c & 1);  // of the warp's sixteen keys, the one that this lane writes
    // the page of the lane's key in a tile, loaded a tile ahead: what its place holds is then loaded
    // while the tile is waited for
    auto page_of = [&](int t) {
      const int at = t * C::KT + warp * 16 + mine;
      return at < keys ? page_at(p.c, it.s, it.k0 + at) : -1ll;
    };
    long long next = page_of(0);
    int st = 0;
    uint32_t phase = 0;
    for (int t = 0; t < n; ++t) {
      const int at = t * C::KT + warp * 16;  // first of the warp's keys
      const long long pos = it.k0 + at + mine, page = next;
      float* to = w.weights;
      float old = 0.f;
      if (page >= 0) {
        to += ((page * p.c.Nk + it.hk) << p.c.page_shift) + (pos & (page_size(p.c) - 1));
        if (w.accumulate && c < 2) old = *to;
      }
      next = page_of(t + 1);
      if (!__all_sync(0xffffffffu, wait_bar(p, bars, &bars->full[st], phase))) break;
      if (at < keys) {
        float sc[NT][4], ev[2], sum[2] = {0.f, 0.f};
        tile_scores<C>(p, smem, st, warp * 16, g, c, qs, sc, ev);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float e = ex2(sc[i][2 * x + y] - l2[i][y]);
              sum[x] += at + g + 8 * x < qs.lim[i][y] ? e : 0.f;
            }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 1);
          sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 2);
        }
        if (page >= 0 && c < 2) *to = old + (c ? sum[1] : sum[0]);
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->empty[st]));
      if (++st == C::NST) {
        st = 0;
        phase ^= 1u;
      }
    }
  }
  __syncthreads();
  if (bars->abort) {
    // copies that were issued but never consumed land before the shared memory is given up
    const uint64_t start = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - start < 200000ull) {
    }
  }
}

template <int D, int NT, bool BF16, int FMT>
cudaError_t launch_weights(const WeightsParams& w, const CUtensorMap& tc, cudaStream_t stream) {
  using C = Cfg<D, NT, BF16, FMT, 1>;
  auto* kernel = weights_rows_kernel<D, NT, BF16, FMT>;
  static std::atomic<unsigned long long> done;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), C::USED, done);
  if (e != cudaSuccess) return e;
  kernel<<<dim3((unsigned)(w.a.c.B * (long long)w.a.c.Nk), w.a.splits), C::THREADS, C::USED,
           stream>>>(tc, w);
  return cudaGetLastError();
}

template <bool BF16, int FMT, int NT>
cudaError_t launch_weights_dim(const WeightsParams& w, const CUtensorMap& tc, cudaStream_t s) {
  if (w.a.c.D > 128) return launch_weights<256, NT, BF16, FMT>(w, tc, s);
  if (w.a.c.D > 64) return launch_weights<128, NT, BF16, FMT>(w, tc, s);
  return launch_weights<64, NT, BF16, FMT>(w, tc, s);
}

template <bool BF16, int FMT>
cudaError_t launch_weights_fmt(const WeightsParams& w, const CUtensorMap& tc, int rows,
                               cudaStream_t s) {
  return rows == 8 ? launch_weights_dim<BF16, FMT, 1>(w, tc, s)
                   : launch_weights_dim<BF16, FMT, 2>(w, tc, s);
}

}  // namespace rows
}  // namespace hstu
