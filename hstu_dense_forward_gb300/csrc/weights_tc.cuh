// Attention weights of the cached keys on the 5th-generation tensor cores, bf16 / fp16:
//   weights[j] (+)= sum_r 2^(f_j s_rj - lse_r log2 e),   s = K Q^T (fp32, TMEM),
// over the packed query rows r of a sequence and kv head (row r: token r / G, head hk * G + r % G)
// that see key j; f_j is alpha log2 e times the key's row scale. Keys are the M side of the products,
// so that a thread of the epilogue owns a key, a TMEM lane, and adds up along its columns: no step of
// the sum crosses threads, and what belongs to a row is the same in all lanes.
//
// A CTA keeps a step of KT keys (one or two tiles of 128) in shared memory and passes over the query
// tiles (128 / G tokens each) that see any of them, then takes the next step of its share; the first
// keys, which with the causal mask the most rows see, come first in the grid. Where there are few
// steps, a cluster of CTAs divides the query tiles of one and adds its sums up in the first of them
// (one prompt of 4096 tokens, two kv heads: 138 us alone). Warp roles:
//   warps 0 .. 7          the sums, a warpgroup for each half of the columns, a thread for a key of
//                         every tile: what belongs to a row is read once for both keys;
//   next warp             issues every tcgen05.mma; owns TMEM;
//   next warp             TMA loads: query tiles, and the keys of a cache of the queries' type;
//   next warp             the rows' logarithms, into shared memory;
//   codes: four warps     load the keys and turn them into the queries' type (E4M3 codes and
//                         products of an E2M1 code and factor have 4 and 7 bits: exact in both).
// The scores have two buffers in TMEM: the next products run while one is summed up. An exponential
// takes four cycles of a scheduler, so that a step of 256 keys and 128 rows takes 1024 cycles, as long
// as its products at D = 128; 1850 are reached: four prompts of 4096 tokens, 16 heads of 4, take 125 us
// (1097 TFLOP/s), D = 64 119, D = 256 200, over E4M3 and E2M1 keys 136 and 138.
//
// Every wait is bounded (timeout_ns): on expiry the CTA reports HSTU_DEVERR_TIMEOUT, every role
// leaves its loop, the MMAs in flight are waited for, TMEM is freed and the kernel returns.
#pragma once
#include <cooperative_groups.h>
#include <cuda.h>
#include <math_constants.h>

#include <type_traits>

#include "common.cuh"
#include "evict_kernels.h"
#include "kernels.h"
#include "kv_cache.cuh"
#include "kv_kernels.h"
#include "pipeline.cuh"
#include "ptx.cuh"

namespace hstu {
namespace wt {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kMaxCluster = 8;

template <int D_, int FMT_>
struct Cfg {
  static constexpr int D = D_, FMT = FMT_;
  static constexpr bool CODES = FMT != kSame, FP4 = FMT == kE2m1;
  static constexpr int NT = D == 256 ? 1 : 2, KT = 128 * NT;  // key tiles, keys of a step
  static constexpr int SWB = 128, EPC = 64, NCB = D / EPC;    // swizzled blocks of a row
  static constexpr int K_CB = KT * SWB, K_STEP = NCB * K_CB;
  static constexpr int Q_CB = 128 * SWB, Q_TILE = NCB * Q_CB;
  // (D = 256: with two steps of keys and one query tile four prompts of 4096 tokens took 334 us)
  static constexpr int NK = D == 64 ? 3 : D == 128 ? 2 : 1, NQ = D == 64 ? 4 : 2;
  static constexpr int OFF_Q = NK * K_STEP, OFF_L = OFF_Q + NQ * Q_TILE;
  static constexpr int OFF_S = OFF_L + 4 * 128 * 4;         // rows' logarithms, of four tiles
  static constexpr int OFF_R = OFF_S + 2 * KT * 4;          // half the columns' sums, of two steps
  static constexpr int OFF_BAR = OFF_R + (kMaxCluster - 1) * KT * 4;  // the other CTAs' sums
  static constexpr int USED = OFF_BAR + 512 + 1024;
  // (one CTA per SM, which takes its share of TMEM: no second one may come to wait for it)
  static constexpr int SMEM = USED < 120 * 1024 ? 120 * 1024 : USED;
  static_assert(SMEM <= 232448, "shared memory");
  static constexpr int SUM_WARPS = 8, MMA_WARP = 8, LOAD_WARP = 9, LOG_WARP = 10;
  static constexpr int CONV_WARP = 12;  // (a warpgroup's boundary)
  static constexpr int THREADS = (CODES ? CONV_WARP + 4 : LOG_WARP + 1) * 32;
  static constexpr uint32_t TMEM_COLS = NT * 2 * 128;
};

struct Bars {
  uint64_t k_full[3], k_empty[3], q_full[4], q_empty[4];
  uint64_t s_full[2], s_empty[2], joined, drain;
  uint32_t tmem_base;
  volatile int abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block");

// The cluster's other CTAs have stored their sums.
__device__ __forceinline__ bool wait_joined(const SoftmaxParams& p, Bars* bars) {
  const uint32_t a = ptx::smem_u32(&bars->joined);
  const uint64_t start = ptx::globaltimer_ns();
  while (!ptx::mbar_try_wait_cluster(a, 0)) {
    if (bars->abort || (long long)(ptx::globaltimer_ns() - start) > p.timeout_ns) {
      bars->abort = 1;
      report(p.c, HSTU_DEVERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

// A CTA's work: steps first, first + slots, .. of one sequence and kv head; of the query tiles, those
// of its rank in the cluster, every cluster-th.
struct Work {
  PagedSeq s;
  int b, hk, steps, first, tpt;
  int tiles;  // query tiles of the sequence
  int rank, cluster;
};

// First query tile of the CTA that sees a key of the step from k0 on.
__device__ __forceinline__ int first_tile(const SoftmaxParams& p, const Work& w, long long k0) {
  const long long tok = p.causal ? k0 - (w.s.Lk - w.s.n) : 0;
  const int t = tok > 0 ? (int)min(tok / w.tpt, (long long)w.tiles) : 0;
  return t + (w.rank - t % w.cluster + w.cluster) % w.cluster;
}

// ------------------------------------------------------------------ loads
template <class C>
__device__ void load_role(const SoftmaxParams& p, Bars* bars, uint8_t* smem, const Work& w,
                          int slots, const CUtensorMap* tq, const CUtensorMap* tc) {
  const uint32_t sbase = ptx::smem_u32(smem);
  const int ps = 1 << p.c.page_shift, rows = ps < 128 ? ps : 128;  // rows of a box
  const uint32_t q_bytes = (uint32_t)(w.tpt * p.G) * C::SWB * C::NCB;
  uint32_t ki = 0, qi = 0;
  for (int step = w.first; step < w.steps; step += slots, ++ki) {
    const long long k0 = (long long)step * C::KT;
    if constexpr (!C::CODES) {
      const int slot = ki % C::NK;
      if (!wait_bar(p, bars, &bars->k_empty[slot], ((ki / C::NK) & 1) ^ 1)) return;
      const uint32_t bar = ptx::smem_u32(&bars->k_full[slot]);
      ptx::mbar_arrive_expect_tx(bar, C::K_STEP);
      for (int r = 0; r < C::KT; r += rows) {
        // (behind the sequence's last page that page again: those rows are not written)
        long long page = page_at(p.c, w.s, min(k0 + r, w.s.Lk - 1));
        if (page < 0) {
          report(p.c, HSTU_DEVERR_OFFSETS);
          page = 0;
        }
#pragma unroll
        for (int cb = 0; cb < C::NCB; ++cb)
          ptx::tma_load_4d(sbase + slot * C::K_STEP + cb * C::K_CB + r * C::SWB, tc, bar,
                           cb * C::EPC, w.hk, (int)((k0 + r) & (ps - 1)), (int)(2 * page));
      }
    }
    for (int t = first_tile(p, w, k0); t < w.tiles; t += w.cluster, ++qi) {
      const int slot = qi % C::NQ;
      if (!wait_bar(p, bars, &bars->q_empty[slot], ((qi / C::NQ) & 1) ^ 1)) return;
      const uint32_t bar = ptx::smem_u32(&bars->q_full[slot]);
      ptx::mbar_arrive_expect_tx(bar, q_bytes);
#pragma unroll
      for (int cb = 0; cb < C::NCB; ++cb)
        ptx::tma_load_3d(sbase + C::OFF_Q + slot * C::Q_TILE + cb * C::Q_CB, tq, bar, cb * C::EPC,
                         w.hk * p.G, (int)(w.s.t0 + (long long)t * w.tpt));
    }
  }
}

// Two fp16 values as bf16 ones (exact: at most 8 bits, in range).
__device__ __forceinline__ uint32_t half_to_bf16(uint32_t h) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A thread converts sixteen codes of a row at a time. Rows beyond the sequence become zeros.
template <class C, bool BF16>
__device__ void convert_role(const SoftmaxParams& p, Bars* bars, uint8_t* smem, const Work& w,
                             int slots, int tid) {
  constexpr int CPR = C::D / 16, CHUNKS = C::KT * CPR / 128;  // of a row, of a thread
  constexpr int FLY = CHUNKS < 8 ? CHUNKS : 8;                // on their way at a time
  uint32_t ki = 0;
  for (int step = w.first; step < w.steps; step += slots, ++ki) {
    const long long k0 = (long long)step * C::KT;
    const int slot = ki % C::NK, have = (int)min((long long)C::KT, w.s.Lk - k0);
    if (!warp_wait(p, bars, &bars->k_empty[slot], ((ki / C::NK) & 1) ^ 1)) return;
    uint8_t* dst = smem + slot * C::K_STEP;
#pragma unroll 1
    for (int i0 = 0; i0 < CHUNKS; i0 += FLY) {
      uint4 u[FLY];
#pragma unroll
      for (int i = 0; i < FLY; ++i) {
        const int x = (i0 + i) * 128 + tid, r = x / CPR, chunk = x % CPR;
        u[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= have || chunk * 16 >= p.c.D) continue;
        const long long pos = k0 + r, page = page_at(p.c, w.s, pos);
        if (page < 0) {
          report(p.c, HSTU_DEVERR_OFFSETS);
          continue;
        }
        const long long row = pos & (page_size(p.c) - 1);
        const uint8_t* codes = static_cast<const uint8_t*>(p.c.cache);
        if constexpr (C::FP4) {
          const long long e = scale_row(p.c, page, 0, row, w.hk) * p.c.D + chunk * 16;
          const uint2 v = *reinterpret_cast<const uint2*>(codes + e / 2);
          u[i] = make_uint4(v.x, v.y, p.c.group[e / 16], 0u);
        } else {
          u[i] = *reinterpret_cast<const uint4*>(codes + cache_row(p.c, page, 0, row, w.hk) +
                                                 chunk * 16);
        }
      }
#pragma unroll
      for (int i = 0; i < FLY; ++i) {
        const int x = (i0 + i) * 128 + tid, r = x / CPR, chunk = x % CPR;
        const uint32_t in[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
        uint32_t h[8];
        if constexpr (C::FP4) {
          const uint32_t f = e4m3x2_to_f16x2(in[2] * 0x101u);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            uint32_t v[4];
            e2m1x8_to_f16x2(in[y], v);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __half2 m = __hmul2(*reinterpret_cast<const __half2*>(&v[e]),
                                        *reinterpret_cast<const __half2*>(&f));
              h[4 * y + e] = *reinterpret_cast<const uint32_t*>(&m);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) e4m3x4_to_f16x2(in[e], h[2 * e], h[2 * e + 1]);
        }
        if constexpr (BF16) {
#pragma unroll
          for (int e = 0; e < 8; ++e) h[e] = half_to_bf16(h[e]);
        }
        uint8_t* row = dst + chunk / 4 * C::K_CB + r * C::SWB;
        const int c16 = chunk % 4 * 2;
        *reinterpret_cast<uint4*>(row + ((c16 ^ (r & 7)) * 16)) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(row + (((c16 + 1) ^ (r & 7)) * 16)) =
            make_uint4(h[4], h[5], h[6], h[7]);
      }
    }
    ptx::fence_proxy_async_smem();
    ptx::mbar_arrive(ptx::smem_u32(&bars->k_full[slot]));
  }
}

// ------------------------------------------------------------------ products
template <class C, bool BF16>
__device__ void mma_role(const SoftmaxParams& p, Bars* bars, uint32_t sbase, uint32_t tmem,
                         const Work& w, int slots) {
  constexpr uint32_t IDESC = ptx::idesc_f16(BF16 ? 1u : 0u, 128, 128, 0);
  uint32_t ki = 0, qi = 0;
  for (int step = w.first; step < w.steps; step += slots, ++ki) {
    const int t0 = first_tile(p, w, (long long)step * C::KT), kslot = ki % C::NK;
    if (!warp_wait(p, bars, &bars->k_full[kslot], (ki / C::NK) & 1)) return;
    for (int t = t0; t < w.tiles; t += w.cluster, ++qi) {
      const int qslot = qi % C::NQ, sb = qi & 1;
      if (!warp_wait(p, bars, &bars->q_full[qslot], (qi / C::NQ) & 1)) return;
      const uint64_t bd0 = ptx::smem_desc(sbase + C::OFF_Q + qslot * C::Q_TILE, 16, 8 * C::SWB, 2);
      if (!warp_wait(p, bars, &bars->s_empty[sb], ((qi >> 1) & 1) ^ 1)) return;
      ptx::tc_fence_after();
      const uint64_t ad0 = ptx::smem_desc(sbase + kslot * C::K_STEP, 16, 8 * C::SWB, 2);
      if (ptx::elect_one()) {
#pragma unroll
        for (int m = 0; m < C::NT; ++m)
#pragma unroll
          for (int kk = 0; kk < C::D / 16; ++kk) {
            const uint32_t in = (kk % 4) * 32;
            ptx::mma_ss(tmem + (sb * C::NT + m) * 128,
                        ptx::desc_add(ad0, (kk / 4) * C::K_CB + m * 128 * C::SWB + in),
                        ptx::desc_add(bd0, (kk / 4) * C::Q_CB + in), IDESC, kk > 0 ? 1u : 0u);
          }
        ptx::mma_commit(ptx::smem_u32(&bars->s_full[sb]));
        ptx::mma_commit(ptx::smem_u32(&bars->q_empty[qslot]));
      }
      __syncwarp();
    }
    if (ptx::elect_one()) ptx::mma_commit(ptx::smem_u32(&bars->k_empty[kslot]));
    __syncwarp();
  }
}

// Waits for the MMAs issued so far, whatever ended the role: TMEM is freed after this.
__device__ __forceinline__ void mma_drain(const SoftmaxParams& p, Bars* bars) {
  __syncwarp();
  if (ptx::elect_one()) ptx::mma_commit(ptx::smem_u32(&bars->drain));
  __syncwarp();
  const uint64_t start = ptx::globaltimer_ns();
  while (!ptx::mbar_try_wait(ptx::smem_u32(&bars->drain), 0)) {
    if ((long long)(ptx::globaltimer_ns() - start) > p.timeout_ns) {
      bars->abort = 1;
      report(p.c, HSTU_DEVERR_TIMEOUT);
      return;
    }
  }
}

// ------------------------------------------------------------------ logarithms
// -lse log2 e of a query tile's columns, four a lane; columns without a row: their weights are 0. A
// tile's scores count as there once these are. Slots are written again four tiles on: two tiles after
// their own the warps that sum have told that they are done with the one between.
template <class C>
__device__ void log_role(const WeightsParams& wp, Bars* bars, uint8_t* smem, const Work& w,
                         int slots, int lane) {
  const SoftmaxParams& p = wp.a;
  float4* logs = reinterpret_cast<float4*>(smem + C::OFF_L);
  const int columns = w.tpt * p.G;
  int off[4];  // lse of the lane's columns, counted from the tile's first
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = min(4 * lane + i, columns - 1);
    off[i] = c / p.G * p.Nq + c % p.G;
  }
  auto load = [&](int t) {
    const float* at = wp.lse + (w.s.t0 + (long long)t * w.tpt) * p.Nq + w.hk * p.G;
    const int rows = (int)min((long long)w.tpt, w.s.n - (long long)t * w.tpt) * p.G;
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = 4 * lane + i < rows ? at[off[i]] * -kLog2e : -CUDART_INF_F;
    return make_float4(x[0], x[1], x[2], x[3]);
  };
  uint32_t qi = 0;
  for (int step = w.first; step < w.steps; step += slots) {
    const int t0 = first_tile(p, w, (long long)step * C::KT);
    float4 x = t0 < w.tiles ? load(t0) : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int t = t0; t < w.tiles; t += w.cluster, ++qi) {
      if (!warp_wait(p, bars, &bars->s_empty[qi & 1], ((qi >> 1) & 1) ^ 1)) return;
      logs[(qi & 3) * 32 + lane] = x;
      ptx::mbar_arrive(ptx::smem_u32(&bars->s_full[qi & 1]));
      if (t + w.cluster < w.tiles) x = load(t + w.cluster);
    }
  }
}

// ------------------------------------------------------------------ sums
// A thread takes its columns of its NT keys in four chunks, each of which it loads from TMEM while it
// sums up the one before; the first chunk of a tile is loaded behind the last one of the tile before
// if its products are done by then (their barrier is looked at a chunk earlier: an answer takes some
// hundred cycles). So a tile's buffer is free again before its last chunk is summed up.
template <class C>
__device__ void sum_role(const WeightsParams& wp, Bars* bars, uint8_t* smem, uint32_t tmem,
                         const Work& w, int slots, int warp, int lane) {
  constexpr int NT = C::NT, CH = 16;  // columns of a chunk
  const SoftmaxParams& p = wp.a;
  const int half = warp / 4, r = (warp & 3) * 32 + lane;  // key of a tile, TMEM lane
  const uint32_t s_col = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * 64;
  const float* logs = reinterpret_cast<const float*>(smem + C::OFF_L) + half * 64;  // [4][128]
  float* sums = reinterpret_cast<float*>(smem + C::OFF_S) + r;                      // [2][KT]
  const int full_tiles = (int)(w.s.n / w.tpt);  // whose tokens are all there
  uint32_t qi = 0, si = 0;
  uint32_t s[2][NT][CH];
  bool ok = true;  // no wait has run out; if one has, the warps still meet at every barrier
  auto load_chunk = [&](int b, uint32_t col) {
#pragma unroll
    for (int m = 0; m < NT; ++m) ptx::tmem_ld16_issue(col + m * 128, s[b][m]);
  };
  for (int step = w.first; step < w.steps; step += slots, ++si) {
    const long long k0 = (long long)step * C::KT;
    const int t0 = first_tile(p, w, k0);
    float f[NT], old[NT];
    float* to[NT];
    float2 sum[NT];
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      const long long pos = k0 + m * 128 + r;
      const long long page = pos < w.s.Lk ? page_at(p.c, w.s, pos) : -1;
      f[m] = p.scale_log2;
      old[m] = 0.f;
      to[m] = nullptr;
      sum[m] = make_float2(0.f, 0.f);
      if (page >= 0) {
        const long long row = pos & (page_size(p.c) - 1);
        if (C::CODES && p.c.scale)
          f[m] *= scale_value(p.c.scale[scale_row(p.c, page, 0, row, w.hk)]);
        to[m] = wp.weights + ((page * p.c.Nk + w.hk) << p.c.page_shift) + row;
        if (wp.accumulate && half == 0) old[m] = *to[m];
      }
      if (C::CODES && p.c.k_ds)
        f[m] *= p.c.k_ds[(long long)w.b * p.c.ds_b + (long long)w.hk * p.c.ds_h];
      f[m] = fminf(fmaxf(f[m], -3e38f), 3e38f);  // (finite: columns without a row have scores of 0)
    }
    // tiles from `seen` on see every key of the step
    int seen = 0;
    if (p.causal) {
      const long long tok = k0 + C::KT - 1 - (w.s.Lk - w.s.n);
      seen = tok > 0 ? (int)min((tok + w.tpt - 1) / w.tpt, (long long)w.tiles) : 0;
    }
    if (t0 < w.tiles) {
      ok = ok && warp_wait(p, bars, &bars->s_full[qi & 1], (qi >> 1) & 1);
      ptx::tc_fence_after();
      if (ok) load_chunk(0, s_col + (qi & 1) * NT * 128);
    }
    for (int t = t0; t < w.tiles && ok; t += w.cluster, ++qi) {
      const int sb = qi & 1;
      const uint32_t col = s_col + sb * NT * 128, next_col = s_col + (sb ^ 1) * NT * 128;
      const uint32_t next_full = ptx::smem_u32(&bars->s_full[sb ^ 1]);
      const uint32_t next_parity = ((qi + 1) >> 1) & 1;
      const bool more = t + w.cluster < w.tiles;
      const float* ls = logs + (qi & 3) * 128;
      const bool whole = t >= seen && t < full_tiles;
      // columns [lo, hi) of this half see the key; those of the warp's first key, and of its last
      int lo[NT], first[NT], last[NT], hi = 64;
#pragma unroll
      for (int m = 0; m < NT; ++m) lo[m] = first[m] = last[m] = 0;
      if (!whole) {
        const long long tok0 = (long long)t * w.tpt;
        hi = (int)min((long long)w.tpt, w.s.n - tok0) * p.G - half * 64;
        if (p.causal) {
#pragma unroll
          for (int m = 0; m < NT; ++m) {
            const long long tok = k0 + m * 128 + r - (w.s.Lk - w.s.n) - tok0;
            lo[m] = (tok > 0 ? (int)min(tok * p.G, 128ll) : 0) - half * 64;
            first[m] = __shfl_sync(0xffffffffu, lo[m], 0);
            last[m] = __shfl_sync(0xffffffffu, lo[m], 31);
          }
        }
      }
      bool ready = false;
      // (a loop of its own for tiles that are seen whole: branches in it cost 15 % of prompts)
      auto sum_up = [&](auto masked) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t(&v)[NT][CH] = s[c & 1];
          ptx::tmem_ld_wait(v[0]);
          if constexpr (NT == 2) ptx::reg_fence(v[1]);
          if (c < 3) {
            load_chunk((c + 1) & 1, col + CH * (c + 1));
          } else {  // the buffer is free
            ptx::tc_fence_before();
            ptx::mbar_arrive(ptx::smem_u32(&bars->s_empty[sb]));
            if (__all_sync(0xffffffffu, ready)) {
              ptx::tc_fence_after();
              load_chunk(0, next_col);
            }
          }
          if (c == 2 && more) ready = ptx::mbar_test(next_full, next_parity);
          // x of four columns of key tile m; the sum of their weights
          auto exponents = [&](int m, int e, const float4& l, float (&x)[4]) {
            ptx::fma_f32x2(x[0], x[1], __uint_as_float(v[m][e]), __uint_as_float(v[m][e + 1]), f[m],
                           f[m], l.x, l.y);
            ptx::fma_f32x2(x[2], x[3], __uint_as_float(v[m][e + 2]), __uint_as_float(v[m][e + 3]),
                           f[m], f[m], l.z, l.w);
          };
          auto add = [&](int m, const float (&x)[4]) {
            ptx::add_f32x2(sum[m].x, sum[m].y, ex2(x[0]), ex2(x[1]));
            ptx::add_f32x2(sum[m].x, sum[m].y, ex2(x[2]), ex2(x[3]));
          };
          bool all = true;  // every column of the chunk sees the warp's keys
          if constexpr (decltype(masked)::value) {
            all = CH * (c + 1) <= hi;
#pragma unroll
            for (int m = 0; m < NT; ++m) all = all && CH * c >= last[m];
          }
          if (all) {
#pragma unroll
            for (int e = 0; e < CH; e += 4) {
              const float4 l = *reinterpret_cast<const float4*>(ls + CH * c + e);
              float x[4];
#pragma unroll
              for (int m = 0; m < NT; ++m) {
                exponents(m, e, l, x);
                add(m, x);
              }
            }
          } else if constexpr (decltype(masked)::value) {
#pragma unroll
            for (int m = 0; m < NT; ++m) {
              if (CH * (c + 1) <= first[m] || CH * c >= hi) continue;  // none does
#pragma unroll
              for (int e = 0; e < CH; e += 4) {
                float x[4];
                exponents(m, e, *reinterpret_cast<const float4*>(ls + CH * c + e), x);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (CH * c + e + i < lo[m] || CH * c + e + i >= hi) x[i] = -CUDART_INF_F;
                add(m, x);
              }
            }
          }
        }
      };
      if (whole)
        sum_up(std::false_type{});
      else
        sum_up(std::true_type{});
      if (more && !__all_sync(0xffffffffu, ready)) {
        ok = warp_wait(p, bars, &bars->s_full[sb ^ 1], next_parity);
        ptx::tc_fence_after();
        if (ok) load_chunk(0, next_col);
      }
    }
    if (half) {
#pragma unroll
      for (int m = 0; m < NT; ++m) sums[(si & 1) * C::KT + m * 128] = sum[m].x + sum[m].y;
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (half == 0 && ok) {
      float total[NT];
#pragma unroll
      for (int m = 0; m < NT; ++m)
        total[m] = sum[m].x + sum[m].y + sums[(si & 1) * C::KT + m * 128];
      if (w.cluster > 1) {  // (one step: the first CTA adds the others' sums, in their order)
        const uint32_t red = ptx::smem_u32(smem + C::OFF_R) + r * 4;
        if (w.rank) {
#pragma unroll
          for (int m = 0; m < NT; ++m)
            ptx::store_remote(red + ((w.rank - 1) * C::KT + m * 128) * 4, 0, total[m]);
          ptx::arrive_remote(ptx::smem_u32(&bars->joined), 0);
          continue;
        }
        if (!wait_joined(p, bars)) continue;
        for (int c = 1; c < w.cluster; ++c)
#pragma unroll
          for (int m = 0; m < NT; ++m)
            total[m] += reinterpret_cast<const float*>(
                smem + C::OFF_R)[(c - 1) * C::KT + m * 128 + r];
      }
#pragma unroll
      for (int m = 0; m < NT; ++m)
        if (to[m]) *to[m] = old[m] + total[m];
    }
  }
}

// ------------------------------------------------------------------ kernel
template <int D, bool BF16, int FMT>
__global__ void __launch_bounds__(Cfg<D, FMT>::THREADS, 1)
    weights_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_c, const WeightsParams wp,
                      int slots, int cluster) {
  using C = Cfg<D, FMT>;
  const SoftmaxParams& p = wp.a;
  extern __shared__ uint8_t smem_raw[];
  Work w;
  const unsigned pairs = (unsigned)p.c.B * p.c.Nk, blk = blockIdx.x / cluster, pair = blk % pairs;
  w.hk = (int)(pair % p.c.Nk);
  w.b = (int)(pair / p.c.Nk);
  w.first = (int)(blk / pairs);
  w.cluster = cluster;
  w.rank = (int)(blockIdx.x % cluster);
  w.s = paged_seq(p.c, w.b);
  if (!attn_seq_ok(p, w.s)) {
    if (threadIdx.x == 0) report(p.c, HSTU_DEVERR_OFFSETS);
    return;
  }
  w.tpt = 128 / p.G;
  w.tiles = (int)((w.s.n + w.tpt - 1) / w.tpt);
  w.steps = (int)((w.s.Lk + C::KT - 1) / C::KT);
  if (w.first >= w.steps || (w.tiles == 0 && wp.accumulate)) return;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + C::OFF_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 3; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bars->k_full[s]), C::CODES ? 128 : 1);
      ptx::mbar_init(ptx::smem_u32(&bars->k_empty[s]), 1);
    }
    for (int s = 0; s < 4; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bars->q_full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->q_empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bars->s_full[s]), 1 + 32);  // (the products, the logarithms)
      ptx::mbar_init(ptx::smem_u32(&bars->s_empty[s]), 256);
    }
    ptx::mbar_init(ptx::smem_u32(&bars->drain), 1);
    ptx::mbar_init(ptx::smem_u32(&bars->joined), 128 * (cluster > 1 ? cluster - 1 : 1));
    bars->abort = 0;
    ptx::fence_barrier_init();
  }
  if (warp == C::MMA_WARP) {
    ptx::tmem_alloc(ptx::smem_u32(&bars->tmem_base), C::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  // columns of a query tile that no head has (G does not divide 128): zeros
  const int empty = 128 - w.tpt * p.G;
  for (int x = threadIdx.x; x < C::NQ * C::NCB * empty * 8; x += C::THREADS) {
    const int row = w.tpt * p.G + x / 8 % empty, block = x / 8 / empty;
    *reinterpret_cast<uint4*>(smem + C::OFF_Q + block * C::Q_CB + row * C::SWB + x % 8 * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  ptx::fence_proxy_async_smem();
  ptx::tc_fence_before();
  if (cluster > 1)  // (the others' barriers are there)
    cooperative_groups::this_cluster().sync();
  else
    __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  if (warp < C::SUM_WARPS) {
    sum_role<C>(wp, bars, smem, tmem, w, slots, warp, lane);
  } else if (warp == C::MMA_WARP) {
    mma_role<C, BF16>(p, bars, ptx::smem_u32(smem), __shfl_sync(0xffffffffu, tmem, 0), w, slots);
    mma_drain(p, bars);
  } else if (warp == C::LOAD_WARP) {
    if (lane == 0) load_role<C>(p, bars, smem, w, slots, &tm_q, &tm_c);
  } else if (warp == C::LOG_WARP) {
    log_role<C>(wp, bars, smem, w, slots, lane);
  } else if (C::CODES && warp >= C::CONV_WARP) {
    convert_role<C, BF16>(p, bars, smem, w, slots, threadIdx.x - C::CONV_WARP * 32);
  }
  __syncwarp();
  ptx::tc_fence_before();
  if (cluster > 1)  // (the first CTA stays until the others have stored their sums there)
    cooperative_groups::this_cluster().sync();
  else
    __syncthreads();
  if (bars->abort) {
    // copies that were issued but never consumed land before the CTA exits
    const uint64_t start = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - start < 200000ull) {
    }
  }
  ptx::tc_fence_after();
  if (warp == C::MMA_WARP) {
    __syncwarp();
    ptx::tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int D, bool BF16, int FMT>
cudaError_t launch_variant(const WeightsParams& w, const CUtensorMap& tq, const CUtensorMap& tc,
                           int slots, int cluster, cudaStream_t stream) {
  using C = Cfg<D, FMT>;
  auto* kernel = weights_tc_kernel<D, BF16, FMT>;
  static std::atomic<unsigned long long> done;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), C::SMEM, done);
  if (e != cudaSuccess) return e;
  const long long blocks = (long long)w.a.c.B * w.a.c.Nk * slots * cluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, tq, tc, w, slots, cluster);
}

template <bool BF16, int FMT>
cudaError_t launch_dim(const WeightsParams& w, const CUtensorMap& tq, const CUtensorMap& tc,
                       int slots, int cluster, cudaStream_t s) {
  if (w.a.c.D > 128) return launch_variant<256, BF16, FMT>(w, tq, tc, slots, cluster, s);
  if (w.a.c.D > 64) return launch_variant<128, BF16, FMT>(w, tq, tc, slots, cluster, s);
  return launch_variant<64, BF16, FMT>(w, tq, tc, slots, cluster, s);
}

}  // namespace wt
}  // namespace hstu
