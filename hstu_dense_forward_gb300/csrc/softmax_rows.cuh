// bf16 / fp16 softmax attention of few query rows (single tokens) over the paged KV cache:
// bound by reading the cache once.
//
// One CTA takes up to sixteen packed query rows (row r of a sequence is query token r / G and
// head hk * G + r % G) of one kv head and a stretch of its keys, in tiles of 64 keys that one
// warp loads by TMA into a ring; each of the other warps takes sixteen keys of every tile and
// keeps its own running maximum m, sum l and output O (registers) over them:
//   S = Q K^T, O += P V   with mma.sync m16n8k16: the sixteen rows are the M side, so that a
// single token of a GQA group fills it; tcgen05's smallest M of 64 would waste the products of
// 48 rows and more, and its operands' way through TMEM costs latency that so few rows cannot
// hide. K and V go from shared memory to the fragments without ldmatrix: both products are
// sums over, or independent in, the head dim, so the head dim may be permuted as long as Q and
// O follow. A lane reads whole 16-byte pieces of a key's row for the scores, and the same piece
// of four keys for the output, which byte permutes turn into pairs of keys.
//
// E4M3 caches: codes become fp16 by one conversion (exact) and the products run in fp16. A
// row scale 2^e of K multiplies the score. One of V would leave fp16's range if it multiplied a
// weight, so it enters the exponent instead: with u_j = x_j + e_j (base 2) and m = max u,
//   P_j = 2^(u_j - m) is at most 1 (times 2^kLazy), O = sum P_j code_j, l = sum P_j 2^-e_j,
// and O / l is the output (2^m cancels). bf16 queries become fp16 times a power of two of their
// row, chosen so that the row's largest lies in [2^14, 2^15): what drops below fp16's smallest
// value is 2^-38 of that.
//
// The warps of a CTA join their (m, l, O) in shared memory, the CTAs of a cluster, which share
// the item and divide its keys, through distributed shared memory; ranges beyond a cluster's
// eight go through the workspace as in the other kernels.
#pragma once
#include <cooperative_groups.h>
#include <cuda.h>
#include <math_constants.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "kv_cache.cuh"
#include "kv_kernels.h"
#include "ptx.cuh"

namespace hstu {
namespace rows {

constexpr int KT = 64;     // keys of one tile
constexpr int RT = 16;     // packed query rows of one CTA
constexpr float kLazy = 8.0f;
constexpr float kLn2 = 0.69314718055994530942f;

template <int D_, bool BF16_, bool E4M3_>
struct Cfg {
  static constexpr int D = D_;
  static constexpr bool BF16 = BF16_, E4M3 = E4M3_;
  static constexpr bool MMA_BF16 = BF16 && !E4M3;
  static constexpr int EB = E4M3 ? 1 : 2;
  static constexpr int SWB = D * EB < 128 ? D * EB : 128;  // bytes of one swizzled row block
  static constexpr int NCB = D * EB / SWB;                 // blocks of a key's row
  static constexpr int CB = KT * SWB;                      // one block of a tile
  static constexpr int CPB = SWB / 16;                     // 16-byte pieces of a block's row
  static constexpr int LPC = CPB / 4;                      // pieces per lane (scores)
  static constexpr int NV = SWB / EB / 8;                  // output columns per lane and block
  // D = 256: two warps share sixteen keys and take half of the output columns each
  static constexpr int HALVES = D == 256 ? 2 : 1;
  static constexpr int OB = NCB / HALVES;                  // output blocks of one warp
  static constexpr int KW = KT / 16;                       // groups of sixteen keys
  static constexpr int CW = KW * HALVES, THREADS = (CW + 1) * 32;
  static constexpr int PLANE = KT * D * EB, STAGE = 2 * PLANE;
  static constexpr int MIN_CTAS = D == 256 ? 1 : 2;  // CTAs per SM
  // ring depth: 96 KB a CTA, two CTAs per SM (D = 256: 192 KB, one)
  static constexpr int NST = (MIN_CTAS == 1 ? 196608 : 98304) / STAGE;
  static constexpr int OFF_SC = NST * STAGE;               // row scales: 2 KT bytes a stage
  static constexpr int OFF_ML = OFF_SC + (E4M3 ? NST * 2 * KT : 0);
  static constexpr int OFF_BAR = OFF_ML + (2 * KW + 2) * RT * 4;
  static constexpr int USED = OFF_BAR + 256 + 1024;
  static_assert(KW * RT * D * 4 <= NST * STAGE, "the joined outputs reuse the ring");
  static_assert(USED <= 232448 / MIN_CTAS - 1024, "shared memory");
};

struct Bars {
  uint64_t full[12], empty[12];
  volatile int abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

__device__ __forceinline__ bool wait_bar(const SoftmaxParams& p, Bars* bars, uint64_t* bar,
                                         uint32_t parity) {
  const uint32_t a = ptx::smem_u32(bar);
  if (ptx::mbar_try_wait(a, parity)) return true;
  const uint64_t start = ptx::globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (ptx::mbar_try_wait(a, parity)) return true;
    if ((i & 15u) == 0) {
      if (bars->abort) return false;
      if ((long long)(ptx::globaltimer_ns() - start) > p.timeout_ns) {
        bars->abort = 1;
        report(p.c, HSTU_DEVERR_TIMEOUT);
        return false;
      }
    }
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// d += a b, m16n8k16.
template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte piece `piece` of row r inside a block with SWB-byte swizzled rows.
template <int SWB>
__device__ __forceinline__ uint32_t piece_at(int r, int piece) {
  const uint32_t o = r * SWB + piece * 16;
  return SWB == 128 ? o ^ ((o >> 3) & 0x70u) : SWB == 64 ? o ^ ((o >> 3) & 0x30u) : o;
}

struct Item {
  PagedSeq s;
  int b, hk, split, nsplit;
  long long m0, rows;   // first packed row, packed rows of the sequence
  long long k0, kend;   // keys of this CTA
};

__device__ __forceinline__ bool make_item(const SoftmaxParams& p, int tiles, int cluster,
                                          Item& it) {
  const long long blk = blockIdx.x / cluster;
  const int rank = blockIdx.x % cluster;
  it.hk = (int)(blk % p.c.Nk);
  const int tile = (int)(blk / p.c.Nk % tiles);
  it.b = (int)(blk / p.c.Nk / tiles);
  it.split = blockIdx.y;
  it.s = paged_seq(p.c, it.b);
  if (!attn_seq_ok(p, it.s)) {
    if (threadIdx.x == 0) report(p.c, HSTU_DEVERR_OFFSETS);
    return false;
  }
  it.rows = it.s.n * p.G;
  it.m0 = (long long)tile * RT;
  const KeyRanges kr = key_ranges(p, it.s.Lk);
  it.nsplit = kr.count;
  if (it.m0 >= it.rows || it.split >= kr.count) return false;
  const long long last = (min(it.m0 + RT, it.rows) - 1) / p.G;  // last token of the tile
  long long e = min(it.s.Lk, (it.split + 1) * kr.keys);
  if (p.causal) e = min(e, it.s.Lk - it.s.n + last + 1);
  const long long k0 = it.split * kr.keys;
  const long long nt = e > k0 ? (e - k0 + KT - 1) / KT : 0;
  const long long per = (nt + cluster - 1) / cluster;  // tiles of one CTA of the cluster
  it.k0 = min(e, k0 + rank * per * KT);
  it.kend = min(e, k0 + (rank + 1) * per * KT);
  return true;
}

template <class C>
__device__ void load_role(const SoftmaxParams& p, Bars* bars, uint8_t* smem, const Item& it,
                          int tiles, const CUtensorMap* tc) {
  const uint32_t sbase = ptx::smem_u32(smem);
  const int ps = 1 << p.c.page_shift;
  const int boxes = ps >= KT ? 1 : KT / 32, brows = ps >= KT ? KT : 32;
  for (int t = 0; t < tiles; ++t) {
    const long long n0 = it.k0 + (long long)t * KT;
    long long page[KT / 32];
#pragma unroll
    for (int m = 0; m < KT / 32; ++m) {
      if (m >= boxes) break;
      page[m] = page_at(p.c, it.s, min(n0 + 32 * m, it.s.Lk - 1));
      if (page[m] < 0) {  // unspecified outputs, but a valid access
        report(p.c, HSTU_DEVERR_OFFSETS);
        page[m] = 0;
      }
    }
    const int st = t % C::NST;
    if (!wait_bar(p, bars, &bars->empty[st], ((t / C::NST) & 1) ^ 1)) return;
    const uint32_t bar = ptx::smem_u32(&bars->full[st]);
    const bool scales = C::E4M3 && p.c.scale;
    ptx::mbar_arrive_expect_tx(bar, C::STAGE + (scales ? 2 * KT : 0));
    const int row0 = ps >= KT ? (int)(n0 & (ps - 1)) : 0;
#pragma unroll
    for (int m = 0; m < KT / 32; ++m) {
      if (m >= boxes) break;
#pragma unroll
      for (int plane = 0; plane < 2; ++plane) {
#pragma unroll
        for (int cb = 0; cb < C::NCB; ++cb)
          ptx::tma_load_4d(sbase + st * C::STAGE + plane * C::PLANE + cb * C::CB + m * 32 * C::SWB,
                           tc, bar, cb * (C::SWB / C::EB), it.hk, row0,
                           (int)(2 * page[m]) + plane);
        if (scales)
          ptx::bulk_load(sbase + C::OFF_SC + st * 2 * KT + plane * KT + m * 32,
                         p.c.scale + scale_row(p.c, page[m], plane, row0, it.hk), brows, bar);
      }
    }
  }
}

// Joins results of a row: reference, sum and weights of n parts.
__device__ __forceinline__ float part_weight(float m, float top) {
  return m == -CUDART_INF_F ? 0.0f : ex2(m - top);
}

template <int D, bool BF16, bool E4M3>
__global__ void __launch_bounds__(Cfg<D, BF16, E4M3>::THREADS, Cfg<D, BF16, E4M3>::MIN_CTAS)
    softmax_rows_kernel(const __grid_constant__ CUtensorMap tm_c, const SoftmaxParams p, int tiles,
                        int cluster) {
  using C = Cfg<D, BF16, E4M3>;
  using T16 = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  namespace cg = cooperative_groups;
  extern __shared__ uint8_t smem_raw[];
  Item it;
  if (!make_item(p, tiles, cluster, it)) return;  // (the whole cluster)
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + C::OFF_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = (int)((it.kend - it.k0 + KT - 1) / KT);
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
  const int kg = warp % C::KW, half = warp / C::KW;  // keys and output half of a warp
  float o[C::OB * C::NV][4];
  float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};
  if (warp == C::CW) {
    if (lane == 0) load_role<C>(p, bars, smem, it, n, &tm_c);
  } else {
    // Q fragments in the scores' order of the head dim: piece j of block cb holds, for lane
    // c, elements e0 .. of which each k-step takes four (two registers per row)
    constexpr int EPP = 16 / C::EB;  // elements of one piece
    uint32_t qa[C::NCB * C::LPC * EPP / 4][4];
    float fr[2];        // score factor of rows g and g + 8
    long long lim[2];   // keys that they see, counted from this CTA's first
    float fk = p.scale_log2;
    if (E4M3 && p.c.k_ds)
      fk *= p.c.k_ds[(long long)it.b * p.c.ds_b + (long long)it.hk * p.c.ds_h];
    long long see = it.kend - it.k0;  // fewest of them
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long pr = it.m0 + g + 8 * h;
      const bool real = pr < it.rows;
      const long long tok = real ? pr / p.G : 0;
      lim[h] = it.kend - it.k0;
      if (p.causal && real) lim[h] = min(lim[h], it.s.Lk - it.s.n + tok + 1 - it.k0);
      see = min(see, lim[h]);
      const T16* q = static_cast<const T16*>(p.q) + (it.s.t0 + tok) * p.q_stride +
                     (it.hk * p.G + (real ? pr % p.G : 0)) * (long long)p.c.D;
      uint32_t top = 0;  // largest magnitude of the row, as 16-bit patterns
#pragma unroll
      for (int cb = 0; cb < C::NCB; ++cb)
#pragma unroll
        for (int j = 0; j < C::LPC; ++j) {
          const int e0 = cb * (C::SWB / C::EB) + (c * C::LPC + j) * EPP;
#pragma unroll
          for (int x = 0; x < EPP / 8; ++x) {
            uint4 u = make_uint4(0u, 0u, 0u, 0u);
            if (real && e0 + 8 * x < p.c.D) u = *reinterpret_cast<const uint4*>(q + e0 + 8 * x);
            const int k = ((cb * C::LPC + j) * EPP + 8 * x) / 4;
            qa[k][h] = u.x;
            qa[k][2 + h] = u.y;
            qa[k + 1][h] = u.z;
            qa[k + 1][2 + h] = u.w;
            if constexpr (E4M3 && BF16) {
              const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
            }
          }
        }
      fr[h] = fk;
      if constexpr (E4M3 && BF16) {  // the row as fp16, times 2^(14 - exponent of its largest)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int sh = min(14 - ((int)(top >> 7) - 127), 126);
        const float mul = __uint_as_float((uint32_t)(sh + 127) << 23);
        fr[h] = fk * __uint_as_float((uint32_t)(127 - sh) << 23);
#pragma unroll
        for (int k = 0; k < C::NCB * C::LPC * EPP / 4; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t w = qa[k][2 * x + h];
            qa[k][2 * x + h] = pack2<false>(__uint_as_float(w << 16) * mul,
                                            __uint_as_float(w & 0xffff0000u) * mul);
          }
      }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) see = min(see, __shfl_xor_sync(0xffffffffu, see, d));
#pragma unroll
    for (int i = 0; i < C::OB * C::NV; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    for (int t = 0; t < n; ++t) {
      const int st = t % C::NST;
      if (!__all_sync(0xffffffffu, wait_bar(p, bars, &bars->full[st], (t / C::NST) & 1))) break;
      const long long at = (long long)t * KT + kg * 16;  // first of the warp's keys
      const long long left = it.kend - it.k0 - at;       // of them, keys of this CTA
      if (left > 0) {
        const uint8_t* kt = smem + st * C::STAGE;
        float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int cb = 0; cb < C::NCB; ++cb)
#pragma unroll
          for (int j = 0; j < C::LPC; ++j) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {  // keys g and g + 8
              const uint4 u = *reinterpret_cast<const uint4*>(
                  kt + cb * C::CB + piece_at<C::SWB>(kg * 16 + 8 * x + g, c * C::LPC + j));
              const uint32_t w[4] = {u.x, u.y, u.z, u.w};
              const int k = (cb * C::LPC + j) * EPP / 4;
              if constexpr (E4M3) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  mma<false>(sc[x], qa[k + e], e4m3x2_to_f16x2(w[e]),
                             e4m3x2_to_f16x2(w[e] >> 16));
              } else {
                mma<C::MMA_BF16>(sc[x], qa[k], w[0], w[1]);
                mma<C::MMA_BF16>(sc[x], qa[k + 1], w[2], w[3]);
              }
            }
          }
        // u = x + exponent of V's row scale; key 8 x + 2 c + e of the warp's is sc[x][e]
        // (row g) and sc[x][2 + e] (row g + 8)
        float ve[2][2];  // 2^-e of V's row scales
        if constexpr (E4M3) {
          if (p.c.scale) {
            const uint8_t* sp = smem + C::OFF_SC + st * 2 * KT + kg * 16 + 2 * c;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t ks = *reinterpret_cast<const uint16_t*>(sp + 8 * x);
              const uint32_t vs = *reinterpret_cast<const uint16_t*>(sp + KT + 8 * x);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float f = scale_value((ks >> (8 * e)) & 0xffu);
                const int ev = (int)((vs >> (8 * e)) & 0xffu) - 127;
                ve[x][e] = __uint_as_float((uint32_t)(127 - ev) << 23);
                sc[x][e] = fmaf(sc[x][e] * f, fr[0], (float)ev);
                sc[x][2 + e] = fmaf(sc[x][2 + e] * f, fr[1], (float)ev);
              }
            }
          }
        }
        if (!E4M3 || !p.c.scale) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              ve[x][e] = 1.0f;
              sc[x][e] *= fr[0];
              sc[x][2 + e] *= fr[1];
            }
        }
        if (at + 16 > see) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const long long j = at + 8 * x + 2 * c + e;
              if (j >= lim[0]) sc[x][e] = -CUDART_INF_F;
              if (j >= lim[1]) sc[x][2 + e] = -CUDART_INF_F;
              if (j >= it.kend - it.k0) ve[x][e] = 0.0f;  // (an unused scale may be anything)
            }
        }
        float mx[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[h] = fmaxf(fmaxf(sc[0][2 * h], sc[0][2 * h + 1]), fmaxf(sc[1][2 * h], sc[1][2 * h + 1]));
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
        }
        // the reference follows the maximum when that lies more than kLazy above it
        if (__any_sync(0xffffffffu, mx[0] > m[0] + kLazy || mx[1] > m[1] + kLazy)) {
          float corr[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bool up = mx[h] > m[h] + kLazy;
            corr[h] = up ? ex2(m[h] - mx[h]) : 1.0f;  // (0 at the first visible key)
            if (up) m[h] = mx[h];
            l[h] *= corr[h];
          }
#pragma unroll
          for (int i = 0; i < C::OB * C::NV; ++i) {
            o[i][0] *= corr[0];
            o[i][1] *= corr[0];
            o[i][2] *= corr[1];
            o[i][3] *= corr[1];
          }
        }
        uint32_t pa[4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float base = m[h] == -CUDART_INF_F ? 0.0f : m[h];
            const float p0 = ex2(sc[x][2 * h] - base), p1 = ex2(sc[x][2 * h + 1] - base);
            l[h] = fmaf(p0, ve[x][0], l[h]);
            l[h] = fmaf(p1, ve[x][1], l[h]);
            pa[2 * x + h] = pack2<C::MMA_BF16>(p0, p1);
          }
        const uint8_t* vt = kt + C::PLANE;
#pragma unroll
        for (int ob = 0; ob < C::OB; ++ob) {
          const uint8_t* blk = vt + (half * C::OB + ob) * C::CB;
          constexpr int NW = C::NV * C::EB / 4;  // words of a lane's piece: 4, or 2 (64 codes a row)
          uint32_t v[4][NW];                     // keys 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int key = 2 * c + (y & 1) + 8 * (y >> 1), r = kg * 16 + key;
            if constexpr (NW == 4) {
              const uint4 u = *reinterpret_cast<const uint4*>(blk + piece_at<C::SWB>(r, g));
              v[y][0] = u.x;
              v[y][1] = u.y;
              v[y][2] = u.z;
              v[y][3] = u.w;
            } else {
              const uint2 u = *reinterpret_cast<const uint2*>(blk + piece_at<C::SWB>(r, g >> 1) +
                                                              (g & 1) * 8);
              v[y][0] = u.x;
              v[y][1] = u.y;
            }
            if (left < 16 && key >= left) {  // beyond the keys: a page's unused rows, maybe NaN
#pragma unroll
              for (int w = 0; w < NW; ++w) v[y][w] = 0u;
            }
          }
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            if constexpr (E4M3) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint32_t b0 = __byte_perm(v[0][w], v[1][w], e ? 0x7362 : 0x5140);
                const uint32_t b1 = __byte_perm(v[2][w], v[3][w], e ? 0x7362 : 0x5140);
                float(&lo)[4] = o[ob * C::NV + 4 * w + 2 * e];
                float(&hi)[4] = o[ob * C::NV + 4 * w + 2 * e + 1];
                mma<false>(lo, pa, e4m3x2_to_f16x2(b0), e4m3x2_to_f16x2(b1));
                mma<false>(hi, pa, e4m3x2_to_f16x2(b0 >> 16), e4m3x2_to_f16x2(b1 >> 16));
              }
            } else {
              mma<C::MMA_BF16>(o[ob * C::NV + 2 * w], pa, __byte_perm(v[0][w], v[1][w], 0x5410),
                               __byte_perm(v[2][w], v[3][w], 0x5410));
              mma<C::MMA_BF16>(o[ob * C::NV + 2 * w + 1], pa,
                               __byte_perm(v[0][w], v[1][w], 0x7632),
                               __byte_perm(v[2][w], v[3][w], 0x7632));
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->empty[st]));
    }
  }

  // ---- join the warps: m and l of every (key group, row), then O relative to the largest m
  float* wm = reinterpret_cast<float*>(smem + C::OFF_ML);  // [KW][RT]
  float* wl = wm + C::KW * RT;                             // [KW][RT]
  float* cm = wl + C::KW * RT;                             // [RT]
  float* cl = cm + RT;                                     // [RT]
  float* part = reinterpret_cast<float*>(smem);            // [KW][RT][D] over the ring
  if (warp < C::CW) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (c == 0 && half == 0) {
        wm[kg * RT + g + 8 * h] = m[h];
        wl[kg * RT + g + 8 * h] = l[h];
      }
    }
  }
  __syncthreads();  // every warp is done with the ring, too
  if (bars->abort) {
    // copies that were issued but never consumed land before the shared memory is given up
    const uint64_t start = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - start < 200000ull) {
    }
    __syncthreads();
  }
  if (warp < C::CW) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = g + 8 * h;
      if (it.m0 + r >= it.rows) continue;
      float top = -CUDART_INF_F;
#pragma unroll
      for (int w = 0; w < C::KW; ++w) top = fmaxf(top, wm[w * RT + r]);
      const float f = part_weight(m[h], top);
#pragma unroll
      for (int ob = 0; ob < C::OB; ++ob)
#pragma unroll
        for (int x = 0; x < 2; ++x) {  // columns NV * (2 c + x) + i of the block
          float* dst = part + (kg * RT + r) * D + (half * C::OB + ob) * (C::SWB / C::EB) +
                       C::NV * (2 * c + x);
#pragma unroll
          for (int i = 0; i < C::NV; i += 4)
            *reinterpret_cast<float4*>(dst + i) = make_float4(
                o[ob * C::NV + i][2 * h + x] * f, o[ob * C::NV + i + 1][2 * h + x] * f,
                o[ob * C::NV + i + 2][2 * h + x] * f, o[ob * C::NV + i + 3][2 * h + x] * f);
        }
    }
  }
  if (threadIdx.x < RT) {
    const int r = threadIdx.x;
    float top = -CUDART_INF_F, sum = 0.f;
    for (int w = 0; w < C::KW; ++w) top = fmaxf(top, wm[w * RT + r]);
    for (int w = 0; w < C::KW; ++w) sum = fmaf(part_weight(wm[w * RT + r], top), wl[w * RT + r], sum);
    cm[r] = top;
    cl[r] = sum;
  }
  __syncthreads();

  // ---- join the CTAs of the cluster and write
  const int nrows = (int)min((long long)RT, it.rows - it.m0);
  const int pieces = p.c.D / 4;  // four columns each
  if (cluster > 1) {  // this CTA's sum over its warps, in place, for the others to read
    for (int x = threadIdx.x; x < nrows * pieces; x += C::THREADS) {
      const int r = x / pieces, d = x % pieces * 4;
      float4 a = *reinterpret_cast<const float4*>(part + r * D + d);
#pragma unroll
      for (int w = 1; w < C::KW; ++w) {
        const float4 b = *reinterpret_cast<const float4*>(part + (w * RT + r) * D + d);
        a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
      }
      *reinterpret_cast<float4*>(part + r * D + d) = a;
    }
    cg::this_cluster().sync();
  }
  const int rank = blockIdx.x % cluster;
  const int parts = cluster > 1 ? cluster : C::KW;
  const float fv = E4M3 && p.c.v_ds
                       ? p.c.v_ds[(long long)it.b * p.c.ds_b + (long long)it.hk * p.c.ds_h]
                       : 1.0f;
  for (int x = rank * C::THREADS + threadIdx.x; x < nrows * pieces; x += cluster * C::THREADS) {
    const int r = x / pieces, d = x % pieces * 4;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float top = cm[r], sum = cl[r];
    if (cluster > 1) {
      top = -CUDART_INF_F;
      sum = 0.f;
      for (int w = 0; w < parts; ++w) top = fmaxf(top, cg::this_cluster().map_shared_rank(cm, w)[r]);
    }
    for (int w = 0; w < parts; ++w) {
      float f = 1.0f;
      const float* src = part + (w * RT + r) * D + d;
      if (cluster > 1) {
        f = part_weight(cg::this_cluster().map_shared_rank(cm, w)[r], top);
        sum = fmaf(f, cg::this_cluster().map_shared_rank(cl, w)[r], sum);
        src = cg::this_cluster().map_shared_rank(part, w) + r * D + d;
      }
      const float4 b = *reinterpret_cast<const float4*>(src);
      a = make_float4(fmaf(f, b.x, a.x), fmaf(f, b.y, a.y), fmaf(f, b.z, a.z), fmaf(f, b.w, a.w));
    }
    const long long pr = it.m0 + r;
    const long long row = (it.s.t0 + pr / p.G) * p.Nq + it.hk * p.G + pr % p.G;  // of out and lse
    const float inv = sum == 0.0f ? 0.0f : fv / sum;
    a = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    if (it.nsplit > 1) {
      *reinterpret_cast<float4*>(
          p.part_o + ((long long)it.split * p.c.T * p.Nq + row) * p.c.D + d) = a;
    } else {
      *reinterpret_cast<uint2*>(static_cast<T16*>(p.out) + row * p.c.D + d) =
          make_uint2(pack2<BF16>(a.x, a.y), pack2<BF16>(a.z, a.w));
    }
    if (d == 0) {
      const float log2sum = sum == 0.0f ? -CUDART_INF_F : top + log2f(sum);
      if (it.nsplit > 1)
        p.part_lse[(long long)it.split * p.c.T * p.Nq + row] = log2sum;
      else if (p.lse)
        p.lse[row] = log2sum * kLn2;
    }
  }
  if (cluster > 1) cg::this_cluster().sync();  // the others have read this CTA's shared memory
}

template <int D, bool BF16, bool E4M3>
cudaError_t launch_variant(const SoftmaxParams& p, const CUtensorMap& tc, long long tiles,
                           long long blocks, int cluster, cudaStream_t stream) {
  using C = Cfg<D, BF16, E4M3>;
  auto* kernel = softmax_rows_kernel<D, BF16, E4M3>;
  static std::atomic<unsigned long long> done;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), C::USED, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks * cluster), p.splits);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::USED;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)cluster, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, tc, p, (int)tiles, cluster);
}

template <bool BF16, bool E4M3>
cudaError_t launch_rows(const SoftmaxParams& p, const CUtensorMap& tc, long long tiles,
                        long long blocks, int cluster, cudaStream_t s) {
  if (p.c.D > 128) return launch_variant<256, BF16, E4M3>(p, tc, tiles, blocks, cluster, s);
  if (p.c.D > 64) return launch_variant<128, BF16, E4M3>(p, tc, tiles, blocks, cluster, s);
  return launch_variant<64, BF16, E4M3>(p, tc, tiles, blocks, cluster, s);
}

}  // namespace rows
}  // namespace hstu
