// bf16 / fp16 softmax attention of few query rows (single tokens) over the paged KV cache:
// bound by reading the cache once.
//
// One CTA takes 8 or 16 packed query rows (row r of a sequence is query token r / G and head
// hk * G + r % G) of one kv head and a stretch of its keys, in tiles of 64 keys that one warp
// loads by TMA into a ring; each of the other warps takes sixteen keys of every tile and keeps
// its own running maximum m, sum l and output O (registers) over them. Both products are
// transposed, so that keys and head dim are the M side and the few query rows the N side, of
// which mma.sync m16n8k16 has as few as eight:
//   S^T = K Q^T,   O^T += V^T P^T.
// tcgen05's smallest M of 64 (rows) would waste most of its products, and its operands' way
// through TMEM costs latency that so few rows cannot hide. K and V go from shared memory to the
// fragments without ldmatrix: the scores are sums over the head dim, and the output's columns
// are independent of each other, so the head dim may be permuted as long as Q and O follow. A
// lane reads whole 16-byte pieces of a key's row for the scores, and the same piece of four
// keys for the output, which byte permutes turn into pairs of keys.
//
// E4M3 caches: codes become fp16 by one conversion (exact) and the products run in fp16. A
// row scale 2^e of K multiplies the score. One of V would leave fp16's range if it multiplied a
// weight, so it enters the exponent instead, relative to a reference of its own: with m = max x
// and m + d = max (x_j + e_j) (base 2),
//   P_j = 2^(x_j + e_j - m - d) is at most 1 (times 2^kLazy), O = sum P_j code_j,
//   l = sum 2^(x_j - m),
// and 2^d O / l is the output. (With one reference for both, weights would vanish from l beside
// values 2^126 larger than theirs: a row of zeros has e = -100.) bf16 queries become fp16 times a
// power of two of their row, chosen so that the row's largest lies in [2^14, 2^15): what drops
// below fp16's smallest value is 2^-38 of that.
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
constexpr float kLazy = 8.0f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNoKey = -1e38f;  // E4M3: reference of a row that has seen no key

template <int D_, int NT_, bool BF16_, bool E4M3_>
struct Cfg {
  static constexpr int D = D_, NT = NT_, RT = 8 * NT;      // packed query rows of one CTA
  static constexpr bool BF16 = BF16_, E4M3 = E4M3_;
  static constexpr bool MMA_BF16 = BF16 && !E4M3;
  static constexpr int EB = E4M3 ? 1 : 2;
  static constexpr int SWB = D * EB < 128 ? D * EB : 128;  // bytes of one swizzled row block
  static constexpr int NCB = D * EB / SWB;                 // blocks of a key's row
  static constexpr int BE = SWB / EB;                      // elements of a block
  static constexpr int CB = KT * SWB;                      // one block of a tile
  static constexpr int EPP = 16 / EB;                      // elements of a 16-byte piece
  static constexpr int LPC = SWB / 64;                     // pieces per lane and block (scores)
  static constexpr int KS = D / 16;                        // k-steps of the scores
  static constexpr int NV = BE / 8;                        // output columns per lane and block
  static constexpr int CW = KT / 16, THREADS = (CW + 1) * 32;
  static constexpr int PLANE = KT * D * EB, STAGE = 2 * PLANE;
  // CTAs per SM: what their registers (O and Q) and a ring of at least three stages leave. E4M3
  // spends more instructions per byte and needs the warps of a third CTA.
  static constexpr int CTAS = D == 256 ? (E4M3 && NT == 1 ? 2 : 1) : (E4M3 && NT == 1 ? 3 : 2);
  static constexpr int NST = (CTAS == 1 ? 196608 : CTAS == 2 ? 98304 : 65536) / STAGE;
  static constexpr int OFF_SC = NST * STAGE;               // row scales: 2 KT bytes a stage
  static constexpr int OFF_ML = OFF_SC + (E4M3 ? NST * 2 * KT : 0);
  static constexpr int OFF_BAR = OFF_ML + (E4M3 ? 3 : 2) * (CW + 1) * RT * 4;
  static constexpr int USED = OFF_BAR + 256 + 1024;
  static_assert(NST >= 3 && NST <= 12, "ring");
  static_assert(CW * RT * D * 4 <= NST * STAGE, "the joined outputs reuse the ring");
  static_assert(USED <= 232448 / CTAS - 1024, "shared memory");
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
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit elements, two of a row per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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

template <int RT>
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
// The unit of a part's output (E4M3), from that of the parts' joint sum.
__device__ __forceinline__ float part_unit(float m, float d, float top) { return (m - top) + d; }
__device__ __forceinline__ float part_weight(float m, float top) {
  return m == -CUDART_INF_F ? 0.0f : ex2(m - top);
}

template <int D, int NT, bool BF16, bool E4M3>
__global__ void __launch_bounds__(Cfg<D, NT, BF16, E4M3>::THREADS, Cfg<D, NT, BF16, E4M3>::CTAS)
    softmax_rows_kernel(const __grid_constant__ CUtensorMap tm_c, const SoftmaxParams p, int tiles,
                        int cluster) {
  using C = Cfg<D, NT, BF16, E4M3>;
  using T16 = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  namespace cg = cooperative_groups;
  constexpr int RT = C::RT;
  extern __shared__ uint8_t smem_raw[];
  Item it;
  if (!make_item<RT>(p, tiles, cluster, it)) return;  // (the whole cluster)
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

  // Lane (g, c) of a warp holds, of S^T, keys g and g + 8 against rows 2c and 2c + 1 of each
  // row tile; of O^T, columns NV g .. NV g + NV - 1 of every block against the same rows.
  const int g = lane >> 2, c = lane & 3;
  float o[NT][C::KS][4];  // [..][x]: columns 2x (elements 0, 1) and 2x + 1 of the lane's
  float m[NT][2], l[NT][2];
  float dv[NT][2];  // E4M3: O's unit is 2^(m + dv)
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    m[i][0] = m[i][1] = E4M3 ? kNoKey : -CUDART_INF_F;
    l[i][0] = l[i][1] = dv[i][0] = dv[i][1] = 0.f;
#pragma unroll
    for (int x = 0; x < C::KS; ++x) o[i][x][0] = o[i][x][1] = o[i][x][2] = o[i][x][3] = 0.f;
  }
  if (warp == C::CW) {
    if (lane == 0) load_role<C>(p, bars, smem, it, n, &tm_c);
  } else {
    float fk = p.scale_log2;
    if (E4M3 && p.c.k_ds)
      fk *= p.c.k_ds[(long long)it.b * p.c.ds_b + (long long)it.hk * p.c.ds_h];
    const int keys = (int)(it.kend - it.k0);
    // Q fragments in the scores' order of the head dim: of piece j of block cb, lane c's
    // elements in fours, two registers each (rows g)
    uint32_t qb[NT][C::KS][2];
    float fr[NT][2];  // score factor of rows 2c and 2c + 1
    int lim[NT][2];   // keys that they see, counted from this CTA's first (maybe < 0)
    int see = keys;   // fewest of them
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const long long pr = it.m0 + 8 * i + g;
      const bool real = pr < it.rows;
      const long long tok = real ? pr / p.G : 0;
      const T16* q = static_cast<const T16*>(p.q) + (it.s.t0 + tok) * p.q_stride +
                     (it.hk * p.G + (real ? pr % p.G : 0)) * (long long)p.c.D;
      uint32_t top = 0;  // largest magnitude of the row, as 16-bit patterns
#pragma unroll
      for (int cb = 0; cb < C::NCB; ++cb)
#pragma unroll
        for (int j = 0; j < C::LPC; ++j) {
          const int e0 = cb * C::BE + (c * C::LPC + j) * C::EPP;
#pragma unroll
          for (int x = 0; x < C::EPP / 8; ++x) {
            uint4 u = make_uint4(0u, 0u, 0u, 0u);
            if (real && e0 + 8 * x < p.c.D) u = *reinterpret_cast<const uint4*>(q + e0 + 8 * x);
            const int k = ((cb * C::LPC + j) * C::EPP + 8 * x) / 4;
            qb[i][k][0] = u.x;
            qb[i][k][1] = u.y;
            qb[i][k + 1][0] = u.z;
            qb[i][k + 1][1] = u.w;
            if constexpr (E4M3 && BF16) {
              const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
            }
          }
        }
      float f = fk;
      if constexpr (E4M3 && BF16) {  // the row as fp16, times 2^(14 - exponent of its largest)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int sh = min(14 - ((int)(top >> 7) - 127), 126);
        const float mul = __uint_as_float((uint32_t)(sh + 127) << 23);
        f = fk * __uint_as_float((uint32_t)(127 - sh) << 23);
#pragma unroll
        for (int k = 0; k < C::KS; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t w = qb[i][k][x];
            qb[i][k][x] = pack2<false>(__uint_as_float(w << 16) * mul,
                                       __uint_as_float(w & 0xffff0000u) * mul);
          }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        fr[i][y] = __shfl_sync(0xffffffffu, f, 4 * (2 * c + y));
        const long long row = it.m0 + 8 * i + 2 * c + y;
        lim[i][y] = keys;
        if (p.causal && row < it.rows)
          lim[i][y] = (int)min((long long)keys, it.s.Lk - it.s.n + row / p.G + 1 - it.k0);
        see = min(see, lim[i][y]);
      }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) see = min(see, __shfl_xor_sync(0xffffffffu, see, d));

    for (int t = 0; t < n; ++t) {
      const int st = t % C::NST;
      if (!__all_sync(0xffffffffu, wait_bar(p, bars, &bars->full[st], (t / C::NST) & 1))) break;
      const int at = t * KT + warp * 16;  // first of the warp's keys
      const int left = keys - at;         // of them, keys of this CTA
      if (left > 0) {
        const uint8_t* kt = smem + st * C::STAGE;
        // two sums per score, of alternate k-steps: a product's latency is some 35 cycles, and
        // each waits for the one before it in its sum
        float sc[NT][4], sd[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[i][e] = sd[i][e] = 0.f;
#pragma unroll
        for (int cb = 0; cb < C::NCB; ++cb)
#pragma unroll
          for (int j = 0; j < C::LPC; ++j) {
            const uint4 u0 = *reinterpret_cast<const uint4*>(
                kt + cb * C::CB + piece_at<C::SWB>(warp * 16 + g, c * C::LPC + j));
            const uint4 u1 = *reinterpret_cast<const uint4*>(
                kt + cb * C::CB + piece_at<C::SWB>(warp * 16 + 8 + g, c * C::LPC + j));
            const uint32_t w0[4] = {u0.x, u0.y, u0.z, u0.w}, w1[4] = {u1.x, u1.y, u1.z, u1.w};
            const int k = (cb * C::LPC + j) * C::EPP / 4;
            if constexpr (E4M3) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t a0, a1, a2, a3;
                e4m3x4_to_f16x2(w0[e], a0, a2);
                e4m3x4_to_f16x2(w1[e], a1, a3);
#pragma unroll
                for (int i = 0; i < NT; ++i)
                  mma<false>(e & 1 ? sd[i] : sc[i], a0, a1, a2, a3, qb[i][k + e][0],
                             qb[i][k + e][1]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                mma<C::MMA_BF16>(sc[i], w0[0], w1[0], w0[1], w1[1], qb[i][k][0], qb[i][k][1]);
                mma<C::MMA_BF16>(sd[i], w0[2], w1[2], w0[3], w1[3], qb[i][k + 1][0],
                                 qb[i][k + 1][1]);
              }
            }
          }
        // scores in base 2; sc[i][2 x + y]: key g + 8 x, row 2 c + y
        float ev[2] = {0.f, 0.f};  // exponents of V's row scales (of a key beyond the last, any)
        if (E4M3 && p.c.scale) {
          const uint8_t* sp = smem + C::OFF_SC + st * 2 * KT + warp * 16 + g;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float f = scale_value(sp[8 * x]);
            ev[x] = (float)((int)sp[KT + 8 * x] - 127);
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int y = 0; y < 2; ++y)
                // (the factors first: their product is in range where the score is)
                sc[i][2 * x + y] = (sc[i][2 * x + y] + sd[i][2 * x + y]) * (f * fr[i][y]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[i][e] = (sc[i][e] + sd[i][e]) * fr[i][e & 1];
        }
        if (at + 16 > see) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int j = at + 8 * x + g;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int y = 0; y < 2; ++y)
                if (j >= lim[i][y]) sc[i][2 * x + y] = -CUDART_INF_F;
          }
        }
        // the references follow their maxima when those lie more than kLazy above them (E4M3: whole
        // numbers, so that their differences are exact)
        bool over = false;
        float xs[NT][4], xw[NT][4];  // E4M3: logarithms of what the sum takes, and of the weights
        auto relative = [&] {
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              xs[i][2 * x] = sc[i][2 * x];
              xs[i][2 * x + 1] = sc[i][2 * x + 1];
              ptx::add_f32x2(xs[i][2 * x], xs[i][2 * x + 1], -m[i][0], -m[i][1]);
              xw[i][2 * x] = xw[i][2 * x + 1] = ev[x];
              ptx::add_f32x2(xw[i][2 * x], xw[i][2 * x + 1], -dv[i][0], -dv[i][1]);
              ptx::add_f32x2(xw[i][2 * x], xw[i][2 * x + 1], xs[i][2 * x], xs[i][2 * x + 1]);
            }
        };
        if constexpr (E4M3) relative();
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            over |= E4M3 ? fmaxf(xs[i][e], xw[i][e]) > kLazy : sc[i][e] > m[i][e & 1] + kLazy;
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            float corr[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float mx = fmaxf(sc[i][y], sc[i][2 + y]);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
              const bool up = mx > m[i][y] + kLazy;
              const float to = E4M3 ? ceilf(mx) : mx;
              corr[y] = up ? ex2(m[i][y] - to) : 1.0f;  // (0 at the first visible key)
              l[i][y] *= corr[y];
              if constexpr (E4M3) {
                if (up) dv[i][y] += m[i][y] - to;
                if (up) m[i][y] = to;
                float u = fmaxf((sc[i][y] - m[i][y]) + ev[0], (sc[i][2 + y] - m[i][y]) + ev[1]);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, d));
                const bool wide = u > dv[i][y] + kLazy;
                corr[y] = wide ? ex2(dv[i][y] - ceilf(u)) : 1.0f;
                if (wide) dv[i][y] = ceilf(u);
              } else if (up) {
                m[i][y] = to;
              }
            }
#pragma unroll
            for (int x = 0; x < C::KS; ++x)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[i][x][e] *= corr[e & 1];
          }
          if constexpr (E4M3) relative();
        }
        // P^T fragments: keys 2c, 2c + 1 (and + 8) of row g. bf16 weights come with what their
        // rounding leaves, for a product of its own: rounded to 2^-8 alone they are as far off as
        // the output's rounding, and the cache's loads leave time for twice the products (four
        // sequences of 100k keys: 74.0 us with one, 74.1 with both; 32 of 2500 keys and eight
        // heads 55.6 and 57.0).
        constexpr int PARTS = C::MMA_BF16 ? 2 : 1;
        uint32_t pb[PARTS][NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const float b0 = m[i][0] == -CUDART_INF_F ? 0.0f : m[i][0];
          const float b1 = m[i][1] == -CUDART_INF_F ? 0.0f : m[i][1];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float p0 = ex2(E4M3 ? xs[i][2 * x] : sc[i][2 * x] - b0);
            float p1 = ex2(E4M3 ? xs[i][2 * x + 1] : sc[i][2 * x + 1] - b1);
            l[i][0] += p0;
            l[i][1] += p1;
            if constexpr (E4M3) {
              p0 = ex2(xw[i][2 * x]);
              p1 = ex2(xw[i][2 * x + 1]);
            }
            const uint32_t w = pack2<C::MMA_BF16>(p0, p1);
            pb[0][i][x] = transpose8(w);
            if constexpr (C::MMA_BF16)
              pb[1][i][x] = transpose8(pack2<true>(p0 - __uint_as_float(w << 16),
                                                   p1 - __uint_as_float(w & 0xffff0000u)));
          }
        }
        const uint8_t* vt = kt + C::PLANE;
#pragma unroll
        for (int cb = 0; cb < C::NCB; ++cb) {
          const uint8_t* blk = vt + cb * C::CB;
          constexpr int NW = C::NV * C::EB / 4;  // words of a lane's piece: 4, or 2 (64 codes a row)
          uint32_t v[4][NW];                     // keys 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int key = 2 * c + (y & 1) + 8 * (y >> 1), r = warp * 16 + key;
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
          }
          if (left < 16) {  // beyond the keys: a page's unused rows, maybe NaN
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (2 * c + (y & 1) + 8 * (y >> 1) >= left) {
#pragma unroll
                for (int w = 0; w < NW; ++w) v[y][w] = 0u;
              }
          }
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            if constexpr (E4M3) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint32_t a0, a1, a2, a3;
                e4m3x4_to_f16x2(__byte_perm(v[0][w], v[1][w], e ? 0x7362 : 0x5140), a0, a1);
                e4m3x4_to_f16x2(__byte_perm(v[2][w], v[3][w], e ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
                for (int i = 0; i < NT; ++i)
                  mma<false>(o[i][cb * C::NV / 2 + 2 * w + e], a0, a1, a2, a3, pb[0][i][0],
                             pb[0][i][1]);
              }
            } else {
              const uint32_t a0 = __byte_perm(v[0][w], v[1][w], 0x5410);
              const uint32_t a1 = __byte_perm(v[0][w], v[1][w], 0x7632);
              const uint32_t a2 = __byte_perm(v[2][w], v[3][w], 0x5410);
              const uint32_t a3 = __byte_perm(v[2][w], v[3][w], 0x7632);
#pragma unroll
              for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int h = 0; h < PARTS; ++h)
                  mma<C::MMA_BF16>(o[i][cb * C::NV / 2 + w], a0, a1, a2, a3, pb[h][i][0],
                                   pb[h][i][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->empty[st]));
    }
  }

  // ---- join the warps: m and l of every (warp, row), then O relative to the largest m
  float* wm = reinterpret_cast<float*>(smem + C::OFF_ML);  // [CW][RT]
  float* wl = wm + C::CW * RT;                             // [CW][RT]
  float* cm = wl + C::CW * RT;                             // [RT]
  float* cl = cm + RT;                                     // [RT]
  float* wd = cl + RT;                                     // [CW][RT], E4M3: units of O
  float* cd = wd + C::CW * RT;                             // [RT]
  float* part = reinterpret_cast<float*>(smem);            // [CW][RT][D] over the ring
  if (warp < C::CW) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[i][y] += __shfl_xor_sync(0xffffffffu, l[i][y], d);
        if (g == 0) {
          wm[warp * RT + 8 * i + 2 * c + y] = m[i][y];
          wl[warp * RT + 8 * i + 2 * c + y] = l[i][y];
          if constexpr (E4M3) wd[warp * RT + 8 * i + 2 * c + y] = dv[i][y];
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
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int r = 8 * i + 2 * c + y;
        if (it.m0 + r >= it.rows) continue;
        float top = -CUDART_INF_F;
#pragma unroll
        for (int w = 0; w < C::CW; ++w) top = fmaxf(top, wm[w * RT + r]);
        float f;
        if constexpr (E4M3) {
          float unit = -CUDART_INF_F;
#pragma unroll
          for (int w = 0; w < C::CW; ++w)
            unit = fmaxf(unit, part_unit(wm[w * RT + r], wd[w * RT + r], top));
          f = part_weight(part_unit(m[i][y], dv[i][y], top), unit);
        } else {
          f = part_weight(m[i][y], top);
        }
#pragma unroll
        for (int cb = 0; cb < C::NCB; ++cb) {
          float* dst = part + (warp * RT + r) * D + cb * C::BE + C::NV * g;
          const int x = cb * C::NV / 2;
#pragma unroll
          for (int e = 0; e < C::NV / 2; e += 2)
            *reinterpret_cast<float4*>(dst + 2 * e) =
                make_float4(o[i][x + e][y] * f, o[i][x + e][2 + y] * f, o[i][x + e + 1][y] * f,
                            o[i][x + e + 1][2 + y] * f);
        }
      }
  }
  if (threadIdx.x < RT) {
    const int r = threadIdx.x;
    float top = -CUDART_INF_F, sum = 0.f;
    for (int w = 0; w < C::CW; ++w) top = fmaxf(top, wm[w * RT + r]);
    for (int w = 0; w < C::CW; ++w) sum = fmaf(part_weight(wm[w * RT + r], top), wl[w * RT + r], sum);
    cm[r] = top;
    cl[r] = sum;
    if constexpr (E4M3) {
      float unit = -CUDART_INF_F;
      for (int w = 0; w < C::CW; ++w)
        unit = fmaxf(unit, part_unit(wm[w * RT + r], wd[w * RT + r], top));
      cd[r] = unit;
    }
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
      for (int w = 1; w < C::CW; ++w) {
        const float4 b = *reinterpret_cast<const float4*>(part + (w * RT + r) * D + d);
        a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
      }
      *reinterpret_cast<float4*>(part + r * D + d) = a;
    }
    cg::this_cluster().sync();
  }
  const int rank = blockIdx.x % cluster;
  const int parts = cluster > 1 ? cluster : C::CW;
  const float fv = E4M3 && p.c.v_ds
                       ? p.c.v_ds[(long long)it.b * p.c.ds_b + (long long)it.hk * p.c.ds_h]
                       : 1.0f;
  for (int x = rank * C::THREADS + threadIdx.x; x < nrows * pieces; x += cluster * C::THREADS) {
    const int r = x / pieces, d = x % pieces * 4;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float top = cm[r], sum = cl[r], unit = E4M3 ? cd[r] : 0.f;
    if (cluster > 1) {
      top = -CUDART_INF_F;
      sum = 0.f;
      for (int w = 0; w < parts; ++w) top = fmaxf(top, cg::this_cluster().map_shared_rank(cm, w)[r]);
      if constexpr (E4M3) {
        unit = -CUDART_INF_F;
        for (int w = 0; w < parts; ++w)
          unit = fmaxf(unit, part_unit(cg::this_cluster().map_shared_rank(cm, w)[r],
                                       cg::this_cluster().map_shared_rank(cd, w)[r], top));
      }
    }
    for (int w = 0; w < parts; ++w) {
      float f = 1.0f;
      const float* src = part + (w * RT + r) * D + d;
      if (cluster > 1) {
        const float mw = cg::this_cluster().map_shared_rank(cm, w)[r];
        f = part_weight(mw, top);
        sum = fmaf(f, cg::this_cluster().map_shared_rank(cl, w)[r], sum);
        if constexpr (E4M3)
          f = part_weight(part_unit(mw, cg::this_cluster().map_shared_rank(cd, w)[r], top), unit);
        src = cg::this_cluster().map_shared_rank(part, w) + r * D + d;
      }
      const float4 b = *reinterpret_cast<const float4*>(src);
      a = make_float4(fmaf(f, b.x, a.x), fmaf(f, b.y, a.y), fmaf(f, b.z, a.z), fmaf(f, b.w, a.w));
    }
    const long long pr = it.m0 + r;
    const long long row = (it.s.t0 + pr / p.G) * p.Nq + it.hk * p.G + pr % p.G;  // of out and lse
    float inv = sum == 0.0f ? 0.0f : fv / sum;
    if constexpr (E4M3) {  // 2^unit in two factors: it may pass fp32's range
      const float half = truncf(unit * 0.5f), rest = ex2(unit - half);
      inv *= ex2(half);
      a = make_float4(a.x * rest, a.y * rest, a.z * rest, a.w * rest);
    }
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

template <int D, int NT, bool BF16, bool E4M3>
cudaError_t launch_variant(const SoftmaxParams& p, const CUtensorMap& tc, long long tiles,
                           long long blocks, int cluster, cudaStream_t stream) {
  using C = Cfg<D, NT, BF16, E4M3>;
  auto* kernel = softmax_rows_kernel<D, NT, BF16, E4M3>;
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

template <bool BF16, bool E4M3, int NT>
cudaError_t launch_dim(const SoftmaxParams& p, const CUtensorMap& tc, long long tiles,
                       long long blocks, int cluster, cudaStream_t s) {
  if (p.c.D > 128) return launch_variant<256, NT, BF16, E4M3>(p, tc, tiles, blocks, cluster, s);
  if (p.c.D > 64) return launch_variant<128, NT, BF16, E4M3>(p, tc, tiles, blocks, cluster, s);
  return launch_variant<64, NT, BF16, E4M3>(p, tc, tiles, blocks, cluster, s);
}

// rows: packed query rows of one item, 8 or 16.
template <bool BF16, bool E4M3>
cudaError_t launch_rows(const SoftmaxParams& p, const CUtensorMap& tc, int rows, long long tiles,
                        long long blocks, int cluster, cudaStream_t s) {
  return rows == 8 ? launch_dim<BF16, E4M3, 1>(p, tc, tiles, blocks, cluster, s)
                   : launch_dim<BF16, E4M3, 2>(p, tc, tiles, blocks, cluster, s);
}

}  // namespace rows
}  // namespace hstu
