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
// E2M1 caches: a lane's sixteen consecutive elements of a key are a group, whose factor multiplies
// them in fp16; factor times code has seven bits, 2^-10 .. 2688, and is exact. What follows holds for
// them as for E4M3 codes. What bounds them is a warp's chain over sixteen keys, some 460 instructions
// (128 tokens over 1k-4k keys of four heads, D = 128: 62 us, 3.2 TB/s of codes, 59 % of issue slots).
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
#include "pipeline.cuh"
#include "ptx.cuh"

namespace hstu {
namespace rows {

constexpr float kLazy = 8.0f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNoKey = -1e38f;  // E4M3: reference of a row that has seen no key

// PLANES: of the cache that the kernel reads (both, or the keys alone).
template <int D_, int NT_, bool BF16_, int FMT_, int PLANES_ = 2>
struct Cfg {
  static constexpr int D = D_, NT = NT_, RT = 8 * NT;      // packed query rows of one CTA
  static constexpr int FMT = FMT_, PLANES = PLANES_;
  static constexpr bool BF16 = BF16_, CODES = FMT != kSame, FP4 = FMT == kE2m1;
  static constexpr bool MMA_BF16 = BF16 && !CODES;
  static constexpr int RB = FP4 ? D / 2 : CODES ? D : 2 * D;  // bytes of a key's row
  static constexpr int SWB = RB < 128 ? RB : 128;          // bytes of one swizzled row block
  static constexpr int NCB = RB / SWB;                     // blocks of a key's row
  static constexpr int BE = D / NCB;                       // elements of a block
  // Keys of a tile, sixteen a warp. A CTA's time is its longest sequence's, tile after tile: more
  // warps shorten that where registers allow as many on an SM (weights of 128 tokens over 1k-4k keys
  // of four heads: bf16 69 us with 64 keys, 61 with 128; E4M3 49 and 46. Attention over E2M1 keys, two
  // CTAs an SM then instead of three, 65 and 76).
  static constexpr int KT = PLANES == 1 ? 128 : 64;
  static constexpr int CB = KT * SWB;                      // one block of a tile
  static constexpr int EPP = 16 * D / RB;                  // elements of a 16-byte piece
  static constexpr int LPC = SWB / 64;                     // pieces per lane and block (scores)
  static constexpr int LE = BE / 4;                        // elements per lane and block (scores)
  static constexpr int KS = D / 16;                        // k-steps of the scores
  static constexpr int NV = BE / 8;                        // output columns per lane and block
  static constexpr int CW = KT / 16, THREADS = (CW + 1) * 32;
  static constexpr int PLANE = KT * RB, STAGE = PLANES * PLANE;
  // CTAs per SM: what their registers (O and Q) and a ring of at least three stages leave. E4M3
  // spends more instructions per byte and needs the warps of a third CTA.
  static constexpr int CTAS = PLANES == 1 ? (RB == 512 || (D == 256 && NT == 2)        ? 1
                                             : RB > 128 || D == 256 || NT == 2 ? 2
                                                                               : 3)
                              : D == 256  ? (CODES && NT == 1 ? 2 : 1)
                                          : (CODES && NT == 1 ? 3 : 2);
  static constexpr int RING = CTAS == 1 ? 196608 : CTAS == 2 ? 98304 : FP4 || PLANES == 1 ? 57344 : 65536;
  static constexpr int NST = RING / STAGE < 12 ? RING / STAGE : 12;
  // the tile's stage is counted where registers allow it (16 rows, D = 256, E4M3: 319 us so, 298
  // with a division)
  static constexpr bool COUNTED = NT == 1 && D <= 128;
  static constexpr int OFF_SC = NST * STAGE;               // row scales: KT bytes a plane and stage
  static constexpr int GPLANE = KT * (D / 16);             // E2M1: factors of a plane's tile
  static constexpr int OFF_GR = OFF_SC + (CODES ? NST * PLANES * KT : 0);
  static constexpr int OFF_ML = OFF_GR + (FP4 ? NST * PLANES * GPLANE : 0);
  static constexpr int OFF_BAR =
      OFF_ML + (PLANES == 1 ? 0 : (CODES ? 3 : 2) * (CW + 1) * RT * 4);
  static constexpr int USED = OFF_BAR + 256 + 1024;
  static_assert(NST >= 3 && NST <= 12, "ring");
  static_assert(PLANES == 1 || CW * RT * D * 4 <= NST * STAGE, "the joined outputs reuse the ring");
  static_assert(USED <= 232448 / CTAS - 1024, "shared memory");
};

struct Bars {
  uint64_t full[12], empty[12];
  volatile int abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

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

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Two factors of E2M1 groups as fp16.
__device__ __forceinline__ uint32_t group_pair(uint32_t lo, uint32_t hi) {
  return e4m3x2_to_f16x2(lo | hi << 8);
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

// The sequence that is number `rank` by length, the longest first, by the whole CTA. Lengths count in
// 256ths of their bound, equal ones in order. (Ranks by comparing every length with every other took
// 4 us of a CTA at 200 sequences, where this takes 2.)
constexpr int kMaxSorted = 256;
struct LengthOrder {
  int bins[256];  // sequences of a length
  uint8_t bin[kMaxSorted];
  int found;
};
__device__ __forceinline__ int sequence_by_length(const SoftmaxParams& p, int rank, int threads,
                                                  LengthOrder* w) {
  const int tid = threadIdx.x, lane = tid & 31;
  const float per_key = 256.0f / ((float)p.max_k + 1.0f);
  for (int i = tid; i < 256; i += threads) w->bins[i] = 0;
  for (int b = tid; b < p.c.B; b += threads)
    w->bin[b] = (uint8_t)min(255, (int)((float)min(paged_table(p.c, b).Lk, p.max_k) * per_key));
  __syncthreads();
  for (int b = tid; b < p.c.B; b += threads) atomicAdd(&w->bins[w->bin[b]], 1);
  __syncthreads();
  if (tid < 32) {
    // lane l has bins 255 - 8 l .. 248 - 8 l; the one that rank falls into, and its number there
    int count[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += count[i] = w->bins[255 - 8 * lane - i];
    int before = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, d);
      if (lane >= d) before += y;
    }
    int left = rank - (before - sum), bin = 255 - 8 * lane;
    const uint32_t has = __ballot_sync(0xffffffffu, left >= 0 && left < sum);
#pragma unroll
    for (int i = 0; i < 7; ++i) {
      const bool on = left >= count[i] && bin == 255 - 8 * lane - i;
      left -= on ? count[i] : 0;
      bin -= on ? 1 : 0;
    }
    const int owner = __ffs(has) - 1;
    left = __shfl_sync(0xffffffffu, left, owner);
    bin = __shfl_sync(0xffffffffu, bin, owner);
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
      const uint32_t in = __ballot_sync(0xffffffffu, b0 + lane < p.c.B && w->bin[b0 + lane] == bin);
      if ((in >> lane & 1u) && __popc(in & ((1u << lane) - 1u)) == left) w->found = b0 + lane;
      left -= __popc(in);
    }
  }
  ptx::fence_proxy_async_smem();  // (TMA writes there next)
  __syncthreads();
  return w->found;
}

// Place of the CTA's item in the order of the lengths. A round of by_length CTAs, one an SM, goes
// through it forwards, the next backwards, so that an SM's share of long and short sequences evens out
// (128 sequences of 1k-4k keys and four heads on 456 places: 79 us in the sequences' order, 62 so).
__device__ __forceinline__ long long place_by_length(const SoftmaxParams& p, long long blk,
                                                     long long blocks) {
  const long long round = blk / p.by_length, first = round * p.by_length;
  if (!(round & 1) || first + p.by_length > blocks) return blk;
  return 2 * first + p.by_length - 1 - blk;
}

__device__ __forceinline__ long long item_by_length(const SoftmaxParams& p, long long blk,
                                                    long long blocks, int threads, LengthOrder* w) {
  blk = place_by_length(p, blk, blocks);
  const int b = sequence_by_length(p, (int)(blk / p.c.Nk), threads, w);
  return (long long)b * p.c.Nk + blk % p.c.Nk;
}

struct Item {
  PagedSeq s;
  int b, hk, split, nsplit;
  long long m0, rows;   // first packed row, packed rows of the sequence
  long long k0, kend;   // keys of this CTA
};

template <class C, bool ORDER>
__device__ __forceinline__ bool make_item(const SoftmaxParams& p, int tiles, int cluster,
                                          Item& it, uint8_t* smem) {
  long long blk = blockIdx.x / cluster;
  const int rank = blockIdx.x % cluster;
  if constexpr (ORDER) {  // (one tile, no clusters)
    blk = item_by_length(p, blk, gridDim.x, C::THREADS, reinterpret_cast<LengthOrder*>(smem));
  }
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
  it.m0 = (long long)tile * C::RT;
  const KeyRanges kr = key_ranges(p, it.s.Lk);
  it.nsplit = kr.count;
  if (it.m0 >= it.rows || it.split >= kr.count) return false;
  const long long last = (min(it.m0 + C::RT, it.rows) - 1) / p.G;  // last token of the tile
  long long e = min(it.s.Lk, (it.split + 1) * kr.keys);
  if (p.causal) e = min(e, it.s.Lk - it.s.n + last + 1);
  const long long k0 = it.split * kr.keys;
  const long long nt = e > k0 ? (e - k0 + C::KT - 1) / C::KT : 0;
  const long long per = (nt + cluster - 1) / cluster;  // tiles of one CTA of the cluster
  it.k0 = min(e, k0 + rank * per * C::KT);
  it.kend = min(e, k0 + (rank + 1) * per * C::KT);
  return true;
}

template <class C>
__device__ void load_role(const SoftmaxParams& p, Bars* bars, uint8_t* smem, const Item& it,
                          int tiles, const CUtensorMap* tc) {
  const uint32_t sbase = ptx::smem_u32(smem);
  const int ps = 1 << p.c.page_shift;
  const int boxes = ps >= C::KT ? 1 : C::KT / 32, brows = ps >= C::KT ? C::KT : 32;
  for (int t = 0; t < tiles; ++t) {
    const long long n0 = it.k0 + (long long)t * C::KT;
    long long page[C::KT / 32];
#pragma unroll
    for (int m = 0; m < C::KT / 32; ++m) {
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
    const bool scales = C::CODES && p.c.scale;
    const int gb = p.c.D / 16;  // E2M1: factors of a row
    ptx::mbar_arrive_expect_tx(
        bar, C::STAGE + (scales ? C::PLANES * C::KT : 0) + (C::FP4 ? C::PLANES * C::KT * gb : 0));
    const int row0 = ps >= C::KT ? (int)(n0 & (ps - 1)) : 0;
#pragma unroll
    for (int m = 0; m < C::KT / 32; ++m) {
      if (m >= boxes) break;
#pragma unroll
      for (int plane = 0; plane < C::PLANES; ++plane) {
#pragma unroll
        for (int cb = 0; cb < C::NCB; ++cb) {
          const uint32_t dst =
              sbase + st * C::STAGE + plane * C::PLANE + cb * C::CB + m * 32 * C::SWB;
          if constexpr (C::FP4)
            ptx::tma_load_4d(dst, tc, bar, 0, row0, it.hk, (int)(2 * page[m]) + plane);
          else
            ptx::tma_load_4d(dst, tc, bar, cb * C::BE, it.hk, row0, (int)(2 * page[m]) + plane);
        }
        if constexpr (C::FP4)
          ptx::bulk_load(sbase + C::OFF_GR + (C::PLANES * st + plane) * C::GPLANE + m * 32 * gb,
                         p.c.group + scale_row(p.c, page[m], plane, row0, it.hk) * gb, brows * gb,
                         bar);
        if (scales)
          ptx::bulk_load(sbase + C::OFF_SC + (C::PLANES * st + plane) * C::KT + m * 32,
                         p.c.scale + scale_row(p.c, page[m], plane, row0, it.hk), brows, bar);
      }
    }
  }
}

// What a warp holds of the item's query rows. Lane (g, c): the products' fragments of rows g of
// each row tile, in the scores' order of the head dim (of block cb, lane c's elements in fours, two
// registers each), and what the scores of rows 2c and 2c + 1 need.
template <class C>
struct Queries {
  uint32_t qb[C::NT][C::KS][2];
  float fr[C::NT][2];  // the score's factor
  int lim[C::NT][2];   // keys that they see, counted from this CTA's first (maybe < 0)
  int see;             // fewest of them
};

template <class C>
__device__ __forceinline__ void load_queries(const SoftmaxParams& p, const Item& it, int keys,
                                             int g, int c, Queries<C>& qs) {
  using T16 = typename std::conditional<C::BF16, __nv_bfloat16, __half>::type;
  float fk = p.scale_log2;
  if (C::CODES && p.c.k_ds)
    fk *= p.c.k_ds[(long long)it.b * p.c.ds_b + (long long)it.hk * p.c.ds_h];
  auto& qb = qs.qb;
  qs.see = keys;
#pragma unroll
  for (int i = 0; i < C::NT; ++i) {
    const long long pr = it.m0 + 8 * i + g;
    const bool real = pr < it.rows;
    const long long tok = real ? pr / p.G : 0;
    const T16* q = static_cast<const T16*>(p.q) + (it.s.t0 + tok) * p.q_stride +
                   (it.hk * p.G + (real ? pr % p.G : 0)) * (long long)p.c.D;
    uint32_t top = 0;  // largest magnitude of the row, as 16-bit patterns
#pragma unroll
    for (int cb = 0; cb < C::NCB; ++cb)
#pragma unroll
      for (int x = 0; x < C::LE / 8; ++x) {
        const int e0 = cb * C::BE + c * C::LE + 8 * x;
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (real && e0 < p.c.D) u = *reinterpret_cast<const uint4*>(q + e0);
        const int k = (cb * C::LE + 8 * x) / 4;
        qb[i][k][0] = u.x;
        qb[i][k][1] = u.y;
        qb[i][k + 1][0] = u.z;
        qb[i][k + 1][1] = u.w;
        if constexpr (C::CODES && C::BF16) {
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
        }
      }
    float f = fk;
    if constexpr (C::CODES && C::BF16) {  // the row as fp16, times 2^(14 - exponent of its largest)
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
      qs.fr[i][y] = __shfl_sync(0xffffffffu, f, 4 * (2 * c + y));
      const long long row = it.m0 + 8 * i + 2 * c + y;
      qs.lim[i][y] = keys;
      if (p.causal && row < it.rows)
        qs.lim[i][y] = (int)min((long long)keys, it.s.Lk - it.s.n + row / p.G + 1 - it.k0);
      qs.see = min(qs.see, qs.lim[i][y]);
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) qs.see = min(qs.see, __shfl_xor_sync(0xffffffffu, qs.see, d));
}

// Scores of a tile's keys r16 .. r16 + 15 in base 2; sc[i][2 x + y]: key g + 8 x, row 2 c + y. ev:
// exponents of V's row scales (unless they are 0).
template <class C>
__device__ __forceinline__ void tile_scores(const SoftmaxParams& p, const uint8_t* smem, int st,
                                            int r16, int g, int c, const Queries<C>& qs,
                                            float (&sc)[C::NT][4], float (&ev)[2]) {
  constexpr int NT = C::NT;
  const uint8_t* kt = smem + st * C::STAGE;
  // two sums per score, of alternate k-steps: a product's latency is some 35 cycles, and
  // each waits for the one before it in its sum
  float sd[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) sc[i][e] = sd[i][e] = 0.f;
  if constexpr (C::FP4) {
    const int gb = p.c.D / 16, r0 = r16 + g;
    const uint8_t* gp = smem + C::OFF_GR + C::PLANES * st * C::GPLANE + r0 * gb;
    constexpr int LU = C::LE / 16;  // groups of sixteen elements that the lane holds
    uint32_t w[2][2 * LU];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      if constexpr (LU == 1) {
        const uint2 u = *reinterpret_cast<const uint2*>(kt + (r0 + 8 * y) * C::SWB + c * 8);
        w[y][0] = u.x;
        w[y][1] = u.y;
      } else {
#pragma unroll
        for (int j = 0; j < LU / 2; ++j) {
          const uint4 u = *reinterpret_cast<const uint4*>(
              kt + piece_at<C::SWB>(r0 + 8 * y, c * (LU / 2) + j));
          w[y][4 * j] = u.x;
          w[y][4 * j + 1] = u.y;
          w[y][4 * j + 2] = u.z;
          w[y][4 * j + 3] = u.w;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < LU; ++u) {
      uint32_t f[2] = {0u, 0u};  // (behind the head dim another row's, or nothing)
      if (c * LU + u < gb) {
        f[0] = group_pair(gp[c * LU + u], gp[c * LU + u]);
        f[1] = group_pair(gp[8 * gb + c * LU + u], gp[8 * gb + c * LU + u]);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t h[2][4];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          e2m1x8_to_f16x2(w[y][2 * u + x], h[y]);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[y][e] = mul_f16x2(h[y][e], f[y]);
        }
        const int k = 4 * u + 2 * x;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          mma<false>(sc[i], h[0][0], h[1][0], h[0][1], h[1][1], qs.qb[i][k][0], qs.qb[i][k][1]);
          mma<false>(sd[i], h[0][2], h[1][2], h[0][3], h[1][3], qs.qb[i][k + 1][0],
                     qs.qb[i][k + 1][1]);
        }
      }
    }
  } else {
#pragma unroll
    for (int cb = 0; cb < C::NCB; ++cb)
#pragma unroll
      for (int j = 0; j < C::LPC; ++j) {
        const uint4 u0 = *reinterpret_cast<const uint4*>(
            kt + cb * C::CB + piece_at<C::SWB>(r16 + g, c * C::LPC + j));
        const uint4 u1 = *reinterpret_cast<const uint4*>(
            kt + cb * C::CB + piece_at<C::SWB>(r16 + 8 + g, c * C::LPC + j));
        const uint32_t w0[4] = {u0.x, u0.y, u0.z, u0.w}, w1[4] = {u1.x, u1.y, u1.z, u1.w};
        const int k = (cb * C::LPC + j) * C::EPP / 4;
        if constexpr (C::CODES) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x2(w0[e], a0, a2);
            e4m3x4_to_f16x2(w1[e], a1, a3);
#pragma unroll
            for (int i = 0; i < NT; ++i)
              mma<false>(e & 1 ? sd[i] : sc[i], a0, a1, a2, a3, qs.qb[i][k + e][0],
                         qs.qb[i][k + e][1]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            mma<C::MMA_BF16>(sc[i], w0[0], w1[0], w0[1], w1[1], qs.qb[i][k][0], qs.qb[i][k][1]);
            mma<C::MMA_BF16>(sd[i], w0[2], w1[2], w0[3], w1[3], qs.qb[i][k + 1][0],
                             qs.qb[i][k + 1][1]);
          }
        }
      }
  }
  // scores in base 2; sc[i][2 x + y]: key g + 8 x, row 2 c + y
  if (C::CODES && p.c.scale) {
    const uint8_t* sp = smem + C::OFF_SC + st * C::PLANES * C::KT + r16 + g;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float f = scale_value(sp[8 * x]);
      if (C::PLANES == 2) ev[x] = (float)((int)sp[C::KT + 8 * x] - 127);
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          // (the factors first: their product is in range where the score is)
          sc[i][2 * x + y] = (sc[i][2 * x + y] + sd[i][2 * x + y]) * (f * qs.fr[i][y]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[i][e] = (sc[i][e] + sd[i][e]) * qs.fr[i][e & 1];
  }
}

// Parts of a row: the unit of one's output (codes), and its weight, against those of all (top).
__device__ __forceinline__ float part_unit(float m, float d, float top) { return (m - top) + d; }
__device__ __forceinline__ float part_weight(float m, float top) {
  return m == -CUDART_INF_F ? 0.0f : ex2(m - top);
}

// ORDER: CTAs take the sequences by length. (A kernel of its own: as a branch in one kernel it cost
// registers that those of 16 rows and of D = 256 have not got, and 0.2 us of every call.)
template <int D, int NT, bool BF16, int FMT, bool ORDER>
__global__ void __launch_bounds__(Cfg<D, NT, BF16, FMT>::THREADS, Cfg<D, NT, BF16, FMT>::CTAS)
    softmax_rows_kernel(const __grid_constant__ CUtensorMap tm_c, const SoftmaxParams p, int tiles,
                        int cluster) {
  using C = Cfg<D, NT, BF16, FMT>;
  using T16 = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr bool CODES = C::CODES;
  namespace cg = cooperative_groups;
  constexpr int RT = C::RT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Item it;
  if (!make_item<C, ORDER>(p, tiles, cluster, it, smem)) return;  // (the whole cluster)
  Bars* bars = reinterpret_cast<Bars*>(smem + C::OFF_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = (int)((it.kend - it.k0 + C::KT - 1) / C::KT);
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
    m[i][0] = m[i][1] = CODES ? kNoKey : -CUDART_INF_F;
    l[i][0] = l[i][1] = dv[i][0] = dv[i][1] = 0.f;
#pragma unroll
    for (int x = 0; x < C::KS; ++x) o[i][x][0] = o[i][x][1] = o[i][x][2] = o[i][x][3] = 0.f;
  }
  if (warp == C::CW) {
    if (lane == 0) load_role<C>(p, bars, smem, it, n, &tm_c);
  } else {
    const int keys = (int)(it.kend - it.k0);
    Queries<C> qs;
    load_queries<C>(p, it, keys, g, c, qs);
    auto& lim = qs.lim;
    const int see = qs.see;

    int stage = 0;  // of the ring
    uint32_t phase = 0;
    for (int t = 0; t < n; ++t) {
      const int st = C::COUNTED ? stage : t % C::NST;
      const uint32_t parity = C::COUNTED ? phase : (t / C::NST) & 1;
      if (!__all_sync(0xffffffffu, wait_bar(p, bars, &bars->full[st], parity))) break;
      const int at = t * C::KT + warp * 16;  // first of the warp's keys
      const int left = keys - at;         // of them, keys of this CTA
      if (left > 0) {
        const uint8_t* kt = smem + st * C::STAGE;
        float sc[NT][4], ev[2] = {0.f, 0.f};  // exponents of V's row scales (of a key beyond the last, any)
        tile_scores<C>(p, smem, st, warp * 16, g, c, qs, sc, ev);
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
        if constexpr (CODES) relative();
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            over |= CODES ? fmaxf(xs[i][e], xw[i][e]) > kLazy : sc[i][e] > m[i][e & 1] + kLazy;
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
              const float to = CODES ? ceilf(mx) : mx;
              corr[y] = up ? ex2(m[i][y] - to) : 1.0f;  // (0 at the first visible key)
              l[i][y] *= corr[y];
              if constexpr (CODES) {
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
          if constexpr (CODES) relative();
        }
        // P^T fragments: keys 2c, 2c + 1 (and + 8) of row g. bf16 weights come with what their
        // rounding leaves, for a product of its own: rounded to 2^-8 alone they are as far off as
        // the output's rounding, and the cache's loads leave time for twice the products (four
        // sequences of 100k keys: 74.0 us with one, 74.1 with both; 32 of 2500 keys and eight
        // heads 55.6 and 57.0).
        // So do fp16 weights over E2M1 keys, for fp16 outputs (tokens over 70,000 keys in the mean: error
        // against 64 bits 0.00033 with one part, 0.00021 with both; the output's rounding is 0.00021).
        constexpr int PARTS = C::MMA_BF16 || (C::FP4 && !BF16) ? 2 : 1;
        uint32_t pb[PARTS][NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const float b0 = m[i][0] == -CUDART_INF_F ? 0.0f : m[i][0];
          const float b1 = m[i][1] == -CUDART_INF_F ? 0.0f : m[i][1];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float p0 = ex2(CODES ? xs[i][2 * x] : sc[i][2 * x] - b0);
            float p1 = ex2(CODES ? xs[i][2 * x + 1] : sc[i][2 * x + 1] - b1);
            l[i][0] += p0;
            l[i][1] += p1;
            if constexpr (CODES) {
              p0 = ex2(xw[i][2 * x]);
              p1 = ex2(xw[i][2 * x + 1]);
            }
            const uint32_t w = pack2<C::MMA_BF16>(p0, p1);
            pb[0][i][x] = transpose8(w);
            if constexpr (C::MMA_BF16)
              pb[1][i][x] = transpose8(pack2<true>(p0 - __uint_as_float(w << 16),
                                                   p1 - __uint_as_float(w & 0xffff0000u)));
            else if constexpr (PARTS == 2)
              pb[1][i][x] = transpose8(
                  pack2<false>(p0 - __low2float(*reinterpret_cast<const __half2*>(&w)),
                               p1 - __high2float(*reinterpret_cast<const __half2*>(&w))));
          }
        }
        const uint8_t* vt = kt + C::PLANE;
        if constexpr (C::FP4) {
          constexpr int NW = C::NV / 8;  // words of the lane's columns of a key
          const int gb = p.c.D / 16;
          const uint8_t* gp = smem + C::OFF_GR + (2 * st + 1) * C::GPLANE + warp * 16 * gb;
          uint32_t v[4][NW];  // keys 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int key = 2 * c + (y & 1) + 8 * (y >> 1), r = warp * 16 + key;
            if constexpr (NW == 1) {
              v[y][0] = *reinterpret_cast<const uint32_t*>(vt + r * C::SWB + g * 4);
            } else if constexpr (NW == 2) {
              const uint2 u = *reinterpret_cast<const uint2*>(vt + piece_at<C::SWB>(r, g >> 1) +
                                                              (g & 1) * 8);
              v[y][0] = u.x;
              v[y][1] = u.y;
            } else {
              const uint4 u = *reinterpret_cast<const uint4*>(vt + piece_at<C::SWB>(r, g));
              v[y][0] = u.x;
              v[y][1] = u.y;
              v[y][2] = u.z;
              v[y][3] = u.w;
            }
          }
          constexpr int GW = NW > 2 ? 2 : 1;  // groups of the lane's columns
#pragma unroll
          for (int u = 0; u < GW; ++u) {
            const int gr = g * C::NV / 16 + u;
            uint32_t b[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {  // (beyond the keys: a page's unused rows, maybe NaN)
              const int key = 2 * c + (y & 1) + 8 * (y >> 1);
              b[y] = gr < gb && key < left ? gp[key * gb + gr] : 0u;
            }
            const uint32_t f01 = group_pair(b[0], b[1]), f23 = group_pair(b[2], b[3]);
#pragma unroll
            for (int w = u * (NW / GW); w < (u + 1) * (NW / GW); ++w) {
              // byte t of e (o): the codes of both keys in column 2 t (2 t + 1) of the word's eight
              constexpr uint32_t M = 0x0f0f0f0fu;
              uint32_t e0[4], o0[4], e1[4], o1[4];
              e2m1x8_to_f16x2((v[0][w] & M) | ((v[1][w] << 4) & ~M), e0);
              e2m1x8_to_f16x2(((v[0][w] >> 4) & M) | (v[1][w] & ~M), o0);
              e2m1x8_to_f16x2((v[2][w] & M) | ((v[3][w] << 4) & ~M), e1);
              e2m1x8_to_f16x2(((v[2][w] >> 4) & M) | (v[3][w] & ~M), o1);
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                const uint32_t a0 = mul_f16x2(e0[t], f01), a1 = mul_f16x2(o0[t], f01);
                const uint32_t a2 = mul_f16x2(e1[t], f23), a3 = mul_f16x2(o1[t], f23);
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                  for (int h = 0; h < PARTS; ++h)
                    mma<false>(o[i][4 * w + t], a0, a1, a2, a3, pb[h][i][0], pb[h][i][1]);
              }
            }
          }
        } else {
#pragma unroll
          for (int cb = 0; cb < C::NCB; ++cb) {
            const uint8_t* blk = vt + cb * C::CB;
            constexpr int NW = C::NV * (C::CODES ? 1 : 2) / 4;  // words of a lane's piece: 4, or 2
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
              if constexpr (CODES) {
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
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&bars->empty[st]));
      if (C::COUNTED && ++stage == C::NST) {
        stage = 0;
        phase ^= 1u;
      }
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
          if constexpr (CODES) wd[warp * RT + 8 * i + 2 * c + y] = dv[i][y];
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
        if constexpr (CODES) {
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
    if constexpr (CODES) {
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
  const float fv = CODES && p.c.v_ds
                       ? p.c.v_ds[(long long)it.b * p.c.ds_b + (long long)it.hk * p.c.ds_h]
                       : 1.0f;
  for (int x = rank * C::THREADS + threadIdx.x; x < nrows * pieces; x += cluster * C::THREADS) {
    const int r = x / pieces, d = x % pieces * 4;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float top = cm[r], sum = cl[r], unit = CODES ? cd[r] : 0.f;
    if (cluster > 1) {
      top = -CUDART_INF_F;
      sum = 0.f;
      for (int w = 0; w < parts; ++w) top = fmaxf(top, cg::this_cluster().map_shared_rank(cm, w)[r]);
      if constexpr (CODES) {
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
        if constexpr (CODES)
          f = part_weight(part_unit(mw, cg::this_cluster().map_shared_rank(cd, w)[r], top), unit);
        src = cg::this_cluster().map_shared_rank(part, w) + r * D + d;
      }
      const float4 b = *reinterpret_cast<const float4*>(src);
      a = make_float4(fmaf(f, b.x, a.x), fmaf(f, b.y, a.y), fmaf(f, b.z, a.z), fmaf(f, b.w, a.w));
    }
    const long long pr = it.m0 + r;
    const long long row = (it.s.t0 + pr / p.G) * p.Nq + it.hk * p.G + pr % p.G;  // of out and lse
    float inv = sum == 0.0f ? 0.0f : fv / sum;
    if constexpr (CODES) {  // 2^unit in two factors: it may pass fp32's range
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

template <int D, int NT, bool BF16, int FMT, bool ORDER = false>
cudaError_t launch_variant(const SoftmaxParams& p, const CUtensorMap& tc, long long tiles,
                           long long blocks, int cluster, cudaStream_t stream) {
  using C = Cfg<D, NT, BF16, FMT>;
  auto* kernel = softmax_rows_kernel<D, NT, BF16, FMT, ORDER>;
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

template <bool BF16, int FMT, int NT>
cudaError_t launch_dim(const SoftmaxParams& p, const CUtensorMap& tc, long long tiles,
                       long long blocks, int cluster, cudaStream_t s) {
  if (p.c.D > 128) return launch_variant<256, NT, BF16, FMT>(p, tc, tiles, blocks, cluster, s);
  if constexpr (NT == 1) {
    if (p.by_length)
      return p.c.D > 64 ? launch_variant<128, NT, BF16, FMT, true>(p, tc, tiles, blocks, 1, s)
                        : launch_variant<64, NT, BF16, FMT, true>(p, tc, tiles, blocks, 1, s);
  }
  if (p.c.D > 64) return launch_variant<128, NT, BF16, FMT>(p, tc, tiles, blocks, cluster, s);
  return launch_variant<64, NT, BF16, FMT>(p, tc, tiles, blocks, cluster, s);
}

// rows: packed query rows of one item, 8 or 16.
template <bool BF16, int FMT>
cudaError_t launch_rows(const SoftmaxParams& p, const CUtensorMap& tc, int rows, long long tiles,
                        long long blocks, int cluster, cudaStream_t s) {
  return rows == 8 ? launch_dim<BF16, FMT, 1>(p, tc, tiles, blocks, cluster, s)
                   : launch_dim<BF16, FMT, 2>(p, tc, tiles, blocks, cluster, s);
}

}  // namespace rows
}  // namespace hstu
