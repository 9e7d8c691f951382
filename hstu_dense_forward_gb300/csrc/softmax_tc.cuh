// bf16 / fp16 softmax attention over the paged KV cache on the 5th-generation tensor cores.
//
// Per query row and tile of KT keys, in base 2 with the running reference m and sum l:
//   S = Q K^T (fp32, TMEM), x = scale_log2 * S, P = 2^(x - m) (16-bit, TMEM, over S),
//   l += sum P, O += P V (fp32, TMEM);  out = O / l.
// m is raised to the row's running maximum only when that lies more than kLazy above it: P then
// stays at or below 2^kLazy, which 16-bit weights and fp32 sums hold with the same relative
// precision, and O (in TMEM) has to be rescaled a few times per row instead of once per tile.
//
// An item is a kv head and NQT tiles of up to 128 packed query rows (row r of a tile is token
// r / G and query head hk * G + r % G, so that the G heads that share keys share their loads),
// with all the keys that they see. Small numbers of items do not fill the SMs evenly, so then
// one CTA per SM takes an equal share of all items' key tiles: every CTA computes the same
// running sum of the items' tiles (plus kItemCost for what an item costs by itself) and works on
// one contiguous piece of it, which may begin and end inside an item. An item in several pieces
// leaves its pieces' outputs and sums in the workspace, and a second kernel joins them. With
// many items each CTA takes one (over short keys several). Warp roles:
//   warps 0 .. 4 NQT - 1   softmax, one warpgroup per query tile, one thread per row; they also
//                          write Q to TMEM (where it does not come by TMA) and the output;
//   next warp              issues every tcgen05.mma; owns TMEM;
//   next warp              TMA loads: K and V tiles through one ring, in the order in which the
//                          products need them (and Q where TMEM has no room for it);
//   next warp              a balanced run's record for the joining kernel;
//   E4M3: eight more warps turn E4M3 tiles (staged by TMA) into fp16 ones in the ring, four
//                          the keys and four the values (one warpgroup for both took 2750
//                          cycles a tile, longer than the products).
// With two query tiles, one tile's products run while the softmax of the other does. With one
// (few rows, or D = 256, whose O takes half of TMEM) the scores have two buffers instead, or an SM
// holds two CTAs with one buffer each, which also hide each other's first and last steps.
//
// E4M3 caches: both products run in fp16, which holds every code exactly. A tile's rows are taken
// relative to the largest of its row scales, 2^EK (K) or 2^EV (V): a code becomes fp16 by one
// conversion and one product with 2^(e - EK). 2^EK multiplies the scores. 2^EV would leave fp16's
// range as a factor of the weights, so it enters their exponent, and O has a unit of its own: with
// m following max x, as ever, and m + d following max (x + EV),
//   P = 2^(x + EV - m - d), O += P V in units of 2^(m + d), l += 2^(d - EV) sum P in units of 2^m,
// and 2^d O / l is the output. (With one reference for both, weights would vanish from l beside
// values 2^126 larger than theirs; a tile of zeros has EV = -100.) The references are whole
// numbers, so that 2^d and EV - d - m are exact. bf16 queries become fp16 in place, times a power
// of two of their row, chosen so that the row's largest lies in [2^14, 2^15): what drops below
// fp16's smallest value is 2^-38 of that. (Dequantising to q's type instead took twice the
// instructions: 1028 us where this took 837, 4096 tokens over 4096.)
//
// That is exact for keys within 2^14 of each other (a code's last bit is 2^-9, fp16's 2^-24), and
// for values it keeps the weights' bits within 2^7: max (x + EV) is at most 2^7 above the largest
// of weight times scale, and O's unit lies 2^7 below that, so that weights keep 2^-31 of it. Tiles
// whose rows lie farther apart (outliers) keep their codes, and every column its row's exponents:
//   x_j = 2^ek_j (q . code_j), P_j = 2^(x_j + ev_j - m - d).
// So a row's weight and value keep their bits whatever other rows of its tile hold, seen or not.
// (Prompts of which every tile has an outlier take longer: 2048 tokens over 2048, four of 16 heads,
// D = 64 708 instead of 218 us, D = 128 741 and 266, D = 256 843 and 480.) Rows of the smallest
// scale that is written, 2^-100, are left out of this: they are zeros, or count as such beside rows
// of 2^-85. Their scores do raise O's unit, like those of a row of the tile's largest scale, and
// weights keep 2^-31 of theirs. (Telling such rows apart where the unit is raised took 20-30 % of
// prompts with a row of zeros in every tile.)
//
// E2M1 caches: a code becomes fp16 times its group's factor (and 2^(e - EK)); factor times code has
// seven bits, 2^-10 .. 2688. All the rest is as for E4M3, with 2688 in the place of 448.
//
// Every wait is bounded (timeout_ns): on expiry the CTA reports HSTU_DEVERR_TIMEOUT, every role
// leaves its loop, the MMAs in flight are waited for, TMEM is freed and the kernel returns.
#pragma once
#include <cuda.h>

#include <math_constants.h>
#include <stddef.h>

#include "common.cuh"
#include "kernels.h"
#include "kv_cache.cuh"
#include "kv_kernels.h"
#include "pipeline.cuh"
#include "ptx.cuh"

namespace hstu {
namespace sm {

constexpr float kLazy = 8.0f;  // log2 of the largest weight
constexpr float kLn2 = 0.69314718055994530942f;
// References beyond 2^22 are rounded by 1/4 and more, and what is relative to them is computed so
// that the largest score is 0 all the same.
constexpr float kLargeScore = 4194304.0f;
// E4M3:
constexpr float kTiny = 1.17549435e-38f;    // 2^-126
constexpr float kNoKey = -1e38f;            // reference of a row that has seen no key
constexpr float kHead = 7.0f;               // log2 of the largest weight when O's unit is set
constexpr int kSpreadK = 14, kSpreadV = 7;  // spread of exponents that are taken relative to one
constexpr uint32_t kLeast = 27;             // smallest row scale that is written
constexpr float kApart = 96.0f;             // d - EV of tiles whose sums are computed apart

template <int D_, int NQT_, int CTAS_, int FMT_>
struct Cfg {
  static constexpr int D = D_, NQT = NQT_, CTAS = CTAS_;  // CTAS: of an SM
  static constexpr bool CODES = FMT_ != kSame, FP4 = FMT_ == kE2m1;
  static_assert(D == 64 || D == 128 || D == 256, "head dim of the kernel");
  static_assert(NQT == 1 || (NQT == 2 && D <= 128), "query tiles");
  static_assert(CTAS == 1 || (CTAS == 2 && NQT == 1 && D <= 128 && FMT_ == kSame), "CTAs per SM");
  static constexpr int KT = D == 256 ? 64 : 128;  // keys of one tile
  static constexpr int NSB = NQT == 1 && CTAS == 1 ? 2 : 1;  // score buffers of a query tile
  static constexpr int SWB = 128, EPC = 64;       // swizzled row bytes and elements of a block
  static constexpr int NCB = D / EPC;             // column blocks of a row
  static constexpr int Q_CB = 128 * SWB, Q_TILE = NCB * Q_CB;
  static constexpr int KV_CB = KT * SWB, KV_TILE = NCB * KV_CB;
  static constexpr int ST_ROW = FP4 ? D / 2 : D, ST_TILE = KT * ST_ROW;  // staged tile of codes
  static constexpr int GR_TILE = FP4 ? KT * (D / 16) : 0;  // E2M1: its factors
  // The scores' A operand, Q, comes from TMEM where that has room: from shared memory it takes,
  // with K, all of the latter's bandwidth, and threads wait for their barriers meanwhile.
  static constexpr bool QT = NSB == 2 || D == 64;
  // ring depths: what 227 KB of shared memory holds
  static constexpr int NSLOT = CTAS == 2  ? (D == 64 ? 6 : 2)
                               : D == 64  ? (CODES ? 4 : 8)
                               : QT       ? (CODES ? 4 : 6)
                                          : (CODES ? 3 : 4);
  static constexpr int NST = !CODES ? 0 : QT ? 4 : 3;
  static constexpr int SM_WARPS = 4 * NQT;
  static constexpr int MMA_WARP = SM_WARPS, LOAD_WARP = SM_WARPS + 1;
  static constexpr int CONV_WARP = SM_WARPS + 4;  // (a warpgroup each for K and V)
  static constexpr int THREADS = (SM_WARPS + 4 + (CODES ? 8 : 0)) * 32;
  // columns of S that a softmax thread holds at a time, half a row (loaded twice: for the maximum
  // and for the weights): loops over halves stay small enough for the instruction cache
  static constexpr int SC = KT / 2;
  // TMEM: score buffers of KT columns (P over them), O, Q (two elements a column)
  static constexpr uint32_t O_COL = NQT * NSB * KT, Q_COL = O_COL + NQT * D;
  static constexpr uint32_t TMEM_COLS = 512 / CTAS;
  static_assert(Q_COL + (QT ? NQT * D / 2 : 0) <= TMEM_COLS, "TMEM");
  static constexpr int OFF_Q = 0, OFF_KV = QT ? 0 : NQT * Q_TILE;
  static constexpr int OFF_ST = OFF_KV + NSLOT * KV_TILE;
  static constexpr int OFF_SC = OFF_ST + NST * ST_TILE;  // row scales of the staged tiles
  static constexpr int OFF_GR = OFF_SC + NST * 128;
  static constexpr int OFF_BAR = OFF_GR + NST * GR_TILE;
  static constexpr int OFF_PLAN = OFF_BAR + (CODES ? 4096 : 2048);
  static constexpr int USED = OFF_PLAN + kPlanSharedBytes + 1024;  // (alignment of the base)
  // (one CTA per SM, which takes all of TMEM: no second one may come to wait for it)
  static constexpr int SMEM = CTAS == 1 && USED < 120 * 1024 ? 120 * 1024 : USED;
  static_assert(SMEM <= 232448 / CTAS - (CTAS - 1) * 1024, "shared memory");
};

constexpr int kExpDepth = 8;  // tiles whose exponents are kept (the conversion is fewer ahead)

struct Bars {
  uint64_t q_ready[2], q_empty, o_empty[2], exp_full[kExpDepth];
  uint64_t q_full, kv_full[8], kv_empty[8], st_full[4], st_empty[4];
  uint64_t s_full[2], p_half[2], p_full[2], pv_done[2], drain;
  uint32_t tmem_base;
  volatile int abort;
  // E4M3: 2^EK, EV, and whether the rows of K, of V have exponents of their own; then what the
  // softmax takes for every row's, biased by 127
  alignas(16) float tile_exp[kExpDepth][4];
  uint8_t row_exp[kExpDepth][2][128];
};
static_assert(offsetof(Bars, tile_exp) <= 2048 && sizeof(Bars) <= 4096, "barrier block");

// A piece of one item: key tiles [a, b) of it.
struct Seg {
  PagedSeq s;
  int b, hk;
  int nq;              // query tiles that hold rows
  long long tok0;      // first token of tile 0
  long long k0, kend;  // keys of the piece
  int n[2];            // key tiles of each query tile (n[0] <= n[1], at most one apart)
  int nmax;
  int slot;            // workspace slot, or -1: the piece is the whole item
};

// Key tiles that query tile q (tokens from first) of a sequence sees, counted from key 0.
template <class C>
__device__ __forceinline__ int tiles_seen(const SoftmaxParams& p, const PagedSeq& s,
                                          long long first, int tpt) {
  long long e = s.Lk;
  if (p.causal) e = min(e, s.Lk - s.n + min(first + tpt, s.n));
  return e > 0 ? (int)((e + C::KT - 1) / C::KT) : 0;
}
// The same for an item: its last query tile that holds rows sees the most.
template <class C>
__device__ __forceinline__ int item_tiles(const SoftmaxParams& p, const PagedSeq& s, int tile) {
  const int tpt = 128 / p.G;
  long long first = (long long)tile * C::NQT * tpt;
  if (C::NQT == 2 && first + tpt < s.n) first += tpt;
  return tiles_seen<C>(p, s, first, tpt);
}

template <class C>
__device__ __forceinline__ void fill_seg(const SoftmaxParams& p, int b, int tile, int hk, int from,
                                         int to, int slot, Seg& g) {
  const int tpt = 128 / p.G;
  g.s = paged_seq(p.c, b);
  g.b = b;
  g.hk = hk;
  g.slot = slot;
  g.tok0 = (long long)tile * C::NQT * tpt;
  g.k0 = (long long)from * C::KT;
  g.kend = min(g.s.Lk, (long long)to * C::KT);
  g.nq = 1;
  g.n[0] = max(0, min(tiles_seen<C>(p, g.s, g.tok0, tpt), to) - from);
  g.n[1] = 0;
  g.nmax = g.n[0];
  if (C::NQT == 2 && g.tok0 + tpt < g.s.n) {
    g.nq = 2;
    g.nmax = g.n[1] = max(0, min(tiles_seen<C>(p, g.s, g.tok0 + tpt, tpt), to) - from);
  }
}

// The pieces that this CTA works on, in order. Every role walks them by itself.
struct Walk {
  long long u, end;  // units (of a share) or items left
  int e, hk;         // of a share: item pair (sequence, tile) and kv head at u
};

template <class C>
__device__ __forceinline__ void walk_begin(const SoftmaxParams& p, const PlanTable& pl, int tiles,
                                           Walk& w) {
  w.u = blockIdx.x;  // items of their own: every gridDim.x-th
  w.end = (long long)p.c.B * tiles * p.c.Nk;
  w.e = w.hk = 0;
  if (!p.balanced) return;
  const int items = pl.items;
  const long long units = pl.cost[items] * p.c.Nk;
  const int ctas = share_ctas(units, gridDim.x);
  w.end = 0;
  if (units == 0 || (int)blockIdx.x >= ctas) return;
  w.u = share(units, ctas, blockIdx.x);
  w.end = share(units, ctas, blockIdx.x + 1);
  int lo = 0, hi = items;  // the last e with cost[e] Nk <= u
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pl.cost[mid] * p.c.Nk <= w.u)
      lo = mid;
    else
      hi = mid;
  }
  w.e = lo;
  w.hk = (int)((w.u - pl.cost[lo] * p.c.Nk) / (pl.cost[lo + 1] - pl.cost[lo]));
}

template <class C>
__device__ __forceinline__ bool walk_next(const SoftmaxParams& p, const PlanTable& pl, Walk& w,
                                          int tiles, Seg& g) {
  if (!p.balanced) {
    while (w.u < w.end) {
      const uint32_t blk = (uint32_t)w.u, pair = blk / (uint32_t)p.c.Nk;  // (fit 31 bits)
      w.u += gridDim.x;
      const int tile = tiles - 1 - (int)(pair % tiles);  // later tiles see more keys: first
      const int b = (int)(pair / tiles), hk = (int)(blk - pair * p.c.Nk);
      const PagedSeq s = paged_seq(p.c, b);
      if (!attn_seq_ok(p, s)) {
        if (threadIdx.x == 0) report(p.c, HSTU_DEVERR_OFFSETS);
        continue;
      }
      if ((long long)tile * C::NQT * (128 / p.G) >= s.n) continue;
      fill_seg<C>(p, b, tile, hk, 0, item_tiles<C>(p, s, tile), -1, g);
      return true;
    }
    return false;
  }
  while (w.u < w.end) {
    const long long cost = pl.cost[w.e + 1] - pl.cost[w.e];
    const long long base = pl.cost[w.e] * p.c.Nk + w.hk * cost;
    const long long o1 = w.u - base, o2 = min(cost, w.end - base);
    const int n = (int)cost - kItemCost;
    const KeyTiles k = piece_tiles(o1, o2);
    const int e = w.e, hk = w.hk;
    w.u = base + o2;
    if (o2 == cost && ++w.hk == p.c.Nk) {
      w.hk = 0;
      ++w.e;
    }
    if (k.to > k.from || (n == 0 && o1 == 0)) {
      const int b = pl.seq[e];
      const bool whole = k.from == 0 && k.to == n;
      fill_seg<C>(p, b, e - pl.first[b], hk, k.from, k.to,
                  whole ? -1 : 2 * (int)blockIdx.x + (k.from > 0 ? 0 : 1), g);
      return true;
    }
  }
  return false;
}

// Inclusive running sums of x[1 .. n] by one warp (x[0] stays).
template <typename T>
__device__ void warp_scan(T* x, int n, int lane) {
  T carry = x[0];
  for (int base = 1; base <= n; base += 32) {
    T v = base + lane <= n ? x[base + lane] : T(0);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += y;
    }
    if (base + lane <= n) x[base + lane] = carry + v;
    carry += __shfl_sync(0xffffffffu, v, 31);
  }
}

// The table of items (balanced runs), by the whole CTA. The host has made sure that sequences and
// items fit.
template <class C>
__device__ void make_plan(const SoftmaxParams& p, PlanTable& pl) {
  const int tid = threadIdx.x, tokens = C::NQT * (128 / p.G);
  if (tid == 0) {
    pl.first[0] = 0;
    pl.cost[0] = 0;
  }
  for (int b = tid; b < p.c.B; b += C::THREADS) {
    const PagedSeq s = paged_seq(p.c, b);
    const bool ok = attn_seq_ok(p, s);
    if (!ok) report(p.c, HSTU_DEVERR_OFFSETS);
    pl.first[b + 1] = ok ? (int)((s.n + tokens - 1) / tokens) : 0;
  }
  __syncthreads();
  if (tid < 32) warp_scan(pl.first, p.c.B, tid);
  __syncthreads();
  // (offsets that overlap could name more rows than there are: what does not fit is left out)
  const int items = min(pl.first[p.c.B], kMaxItems);
  for (int e = tid; e < items; e += C::THREADS) {
    int lo = 0, hi = p.c.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pl.first[mid] <= e)
        lo = mid;
      else
        hi = mid;
    }
    pl.seq[e] = (uint16_t)lo;
    pl.cost[e + 1] = kItemCost + item_tiles<C>(p, paged_seq(p.c, lo), e - pl.first[lo]);
  }
  __syncthreads();
  if (tid < 32) warp_scan(pl.cost, items, tid);
  if (tid == 32) pl.items = items;
  __syncthreads();
}

// Whether an item is parted at the border in front of this CTA's share, and first there: what the
// kernel that joins the pieces needs to know then.
template <class C>
__device__ JoinRecord join_record(const SoftmaxParams& p, const PlanTable& pl, int tiles) {
  JoinRecord j = {0, 0, 0, 0};
  const int c = blockIdx.x;
  const long long units = pl.cost[pl.items] * p.c.Nk;
  const int ctas = share_ctas(units, gridDim.x);
  if (units == 0 || c == 0 || c >= ctas) return j;
  Walk w;
  walk_begin<C>(p, pl, tiles, w);
  const long long cost = pl.cost[w.e + 1] - pl.cost[w.e];
  const long long base = pl.cost[w.e] * p.c.Nk + w.hk * cost;
  // (a border in front of the item's tiles parts nothing)
  if (w.u <= base + kItemCost || share(units, ctas, c - 1) > base + kItemCost) return j;
  int last = c;
  while (share(units, ctas, last + 1) < base + cost) ++last;
  const int b = pl.seq[w.e], tokens = C::NQT * (128 / p.G);
  const PagedSeq s = paged_seq(p.c, b);
  const long long tok0 = (long long)(w.e - pl.first[b]) * tokens;
  j.count = last - c + 2;
  j.hk = w.hk;
  j.rows = (int)min((long long)tokens, s.n - tok0) * p.G;
  j.t0 = s.t0 + tok0;
  return j;
}

// Place of K and V tiles in the ring's order: the order in which the MMA warp needs them.
// One query tile: K0 K1 V0 K2 V1 ... (the scores run a tile ahead); two: K0 V0 K1 V1 ...
template <class C>
__device__ __forceinline__ int k_index(int t) {
  return C::NSB == 2 ? (t == 0 ? 0 : 2 * t - 1) : 2 * t;
}
template <class C>
__device__ __forceinline__ int v_index(int t, int n) {
  return C::NSB == 2 ? (t + 1 < n ? 2 * t + 2 : 2 * t + 1) : 2 * t + 1;
}
// The tile behind place i: its number, and whether it is a V tile.
template <class C>
__device__ __forceinline__ bool ring_tile(int i, int n, int& t) {
  if (C::NSB == 1) {
    t = i >> 1;
    return i & 1;
  }
  if (i == 0 || (i & 1)) {
    t = (i + 1) >> 1;
    if (t < n) return false;  // K
    t = n - 1;                // the last place
    return true;
  }
  t = (i - 2) >> 1;
  return true;
}

// 2^-d as an fp16 pattern, d in [0, 14]; beyond, 0 (rows of the smallest scale).
__device__ __forceinline__ uint32_t half_power(int d) {
  return d < 15 ? (uint32_t)(15 - d) << 10 : 0u;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float power2(int e) {  // e in [-126, 127]
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if one is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
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

// ------------------------------------------------------------------ loads
// Every role takes the CTA's pieces one after the other; its ring places and barrier phases run
// on (ring: places before the piece, tiles: key tiles before it, and so on).
template <class C>
__device__ void load_role(const SoftmaxParams& p, Bars* bars, uint8_t* smem, const PlanTable& pl,
                          int tiles, const CUtensorMap* tq, const CUtensorMap* tc) {
  const uint32_t sbase = ptx::smem_u32(smem);
  const int tpt = 128 / p.G, ps = 1 << p.c.page_shift;
  const uint32_t q_bytes = (uint32_t)(tpt * p.G) * C::SWB * C::NCB;
  constexpr int DEPTH = C::CODES ? C::NST : C::NSLOT;
  uint64_t* full = C::CODES ? bars->st_full : bars->kv_full;
  uint64_t* empty = C::CODES ? bars->st_empty : bars->kv_empty;
  const int boxes = ps >= C::KT ? 1 : C::KT / 32;
  uint32_t ring = 0, queries = 0;
  Walk w;
  Seg it;
  walk_begin<C>(p, pl, tiles, w);
  while (walk_next<C>(p, pl, w, tiles, it)) {
    const int nmax = it.nmax;
    for (int i = 0; i < 2 * nmax; ++i) {
      int t;
      const bool v = ring_tile<C>(i, nmax, t);
      const long long n0 = it.k0 + (long long)t * C::KT;
      // page ids first: their latency passes while the slot is waited for. Places past the
      // sequence's last page repeat that page (their rows are masked).
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
      const int slot = (ring + i) % DEPTH;
      if (!wait_bar(p, bars, &empty[slot], (((ring + i) / DEPTH) & 1) ^ 1)) return;
      const uint32_t bar = ptx::smem_u32(&full[slot]);
      const bool scales = C::CODES && p.c.scale;
      const int gb = p.c.D / 16;  // E2M1: factors of a row
      ptx::mbar_arrive_expect_tx(bar, C::CODES ? C::ST_TILE + (scales ? C::KT : 0) +
                                                     (C::FP4 ? C::KT * gb : 0)
                                               : C::KV_TILE);
      const int row0 = ps >= C::KT ? (int)(n0 & (ps - 1)) : 0;
#pragma unroll
      for (int m = 0; m < C::KT / 32; ++m) {
        if (m >= boxes) break;
        const int plane = (int)(2 * page[m]) + (v ? 1 : 0);
        if constexpr (C::CODES) {
          const uint32_t dst = sbase + C::OFF_ST + slot * C::ST_TILE + m * 32 * C::ST_ROW;
          if constexpr (C::FP4) {
            ptx::tma_load_4d(dst, tc, bar, 0, row0, it.hk, plane);
            ptx::bulk_load(sbase + C::OFF_GR + slot * C::GR_TILE + m * 32 * gb,
                           p.c.group + scale_row(p.c, page[m], v ? 1 : 0, row0, it.hk) * gb,
                           (boxes == 1 ? C::KT : 32) * gb, bar);
          } else {
            ptx::tma_load_4d(dst, tc, bar, 0, it.hk, row0, plane);
          }
          if (scales)
            ptx::bulk_load(sbase + C::OFF_SC + slot * 128 + m * 32,
                           p.c.scale + scale_row(p.c, page[m], v ? 1 : 0, row0, it.hk),
                           boxes == 1 ? C::KT : 32, bar);
        } else {
#pragma unroll
          for (int cb = 0; cb < C::NCB; ++cb)
            ptx::tma_load_4d(
                sbase + C::OFF_KV + slot * C::KV_TILE + cb * C::KV_CB + m * 32 * C::SWB, tc, bar,
                cb * C::EPC, it.hk, row0, plane);
        }
      }
      if (!C::QT && i == 0) {  // the piece's queries, once the previous piece's scores are done
        if (!wait_bar(p, bars, &bars->q_empty, (queries & 1) ^ 1)) return;
        ptx::mbar_arrive_expect_tx(ptx::smem_u32(&bars->q_full), it.nq * q_bytes);
        for (int q = 0; q < it.nq; ++q)
#pragma unroll
          for (int cb = 0; cb < C::NCB; ++cb)
            ptx::tma_load_3d(sbase + C::OFF_Q + q * C::Q_TILE + cb * C::Q_CB, tq,
                             ptx::smem_u32(&bars->q_full), cb * C::EPC, it.hk * p.G,
                             (int)(it.s.t0 + it.tok0 + q * tpt));
        ++queries;
      }
    }
    ring += 2 * nmax;
  }
}

// ------------------------------------------------------------------ codes -> fp16
// A thread converts sixteen codes of a row at a time (of E2M1 a group). Rows beyond the sequence become zeros
// (what an unused row of a page holds, NaN included, does not reach the products).
template <class C>
__device__ void convert_role(const SoftmaxParams& p, Bars* bars, uint8_t* smem,
                             const PlanTable& pl, int tiles, bool values, int warp, int lane) {
  constexpr int CPR = C::D / 16;  // chunks of a row
  constexpr int STEP = 128 / CPR, PASSES = C::KT / STEP;  // rows of one pass of the four warps
  constexpr int RPW = 32 / CPR;  // rows of one pass of a warp
  const int chunk = lane % CPR, r0 = warp * RPW + lane / CPR;
  // the row whose factor this lane holds for its warp (PASSES of RPW rows, 32 at most)
  const int my_row = warp * RPW + lane % RPW + STEP * (lane / RPW % PASSES);
  const int cb = chunk / 4, c16 = (chunk % 4) * 2;  // column block, first 16-byte piece in it
  uint32_t ring = 0, done = 0;
  Walk walk;
  Seg it;
  walk_begin<C>(p, pl, tiles, walk);
  while (walk_next<C>(p, pl, walk, tiles, it)) {
    uint32_t one = 0x3c003c00u;  // 1.0 twice; keys change sign if their static factor is negative
    if (!values && p.c.k_ds &&
        p.c.k_ds[(long long)it.b * p.c.ds_b + (long long)it.hk * p.c.ds_h] < 0.0f)
      one ^= 0x80008000u;
    for (int x = 0; x < 2 * it.nmax; ++x) {
      int t;
      if (ring_tile<C>(x, it.nmax, t) != values) continue;
      const uint32_t i = ring + x, te = (done + t) % kExpDepth;
      const int have = (int)min((long long)C::KT, it.s.Lk - it.k0 - (long long)t * C::KT);
      const int st = i % C::NST, slot = i % C::NSLOT;
      if (!warp_wait(p, bars, &bars->st_full[st], (i / C::NST) & 1)) return;
      const uint8_t* scale = smem + C::OFF_SC + st * 128;
      int top = 127;  // the largest scale of the tile's rows
      uint32_t exps = 0x7f7f7f7fu;
      bool own = false;  // the rows keep exponents of their own
      if (p.c.scale) {
        if (lane * 4 < C::KT) exps = *reinterpret_cast<const uint32_t*>(scale + lane * 4);
        uint32_t b[4], high = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          b[e] = lane * 4 + e < have ? (exps >> (8 * e)) & 0xffu : kLeast;
          high = max(high, b[e]);
        }
        top = (int)__reduce_max_sync(0xffffffffu, high);
        // scales in (kLeast, top - spread) lie apart
        const int spread = values ? kSpreadV : kSpreadK;
        const uint32_t least = kLeast + 1, range = (uint32_t)max(top - spread - (int)least, 0);
        own = __any_sync(0xffffffffu, b[0] - least < range || b[1] - least < range ||
                                          b[2] - least < range || b[3] - least < range);
        if (!own) exps = (uint32_t)top * 0x01010101u;
      }
      if (warp == 0) {
        if (lane * 4 < C::KT)
          *reinterpret_cast<uint32_t*>(&bars->row_exp[te][values ? 1 : 0][lane * 4]) = exps;
        __syncwarp();
        if (lane == 0) {
          bars->tile_exp[te][values ? 1 : 0] = values ? (float)(top - 127) : power2(top - 127);
          bars->tile_exp[te][values ? 3 : 2] = own ? 1.0f : 0.0f;
          ptx::mbar_arrive(ptx::smem_u32(&bars->exp_full[te]));
        }
      }
      const uint8_t* src = smem + C::OFF_ST + st * C::ST_TILE + chunk * (C::FP4 ? 8 : 16);
      uint8_t* dst = smem + C::OFF_KV + slot * C::KV_TILE + cb * C::KV_CB;
      uint32_t mine = one;  // factor of row my_row, twice (0 beyond the sequence)
      if (p.c.scale && !own) mine = half_power(top - (int)scale[my_row]) * 0x10001u;
      if (my_row >= have) mine = 0u;
      uint4 u[PASSES];
#pragma unroll
      for (int k = 0; k < PASSES; ++k) {
        if constexpr (C::FP4) {  // (and the group's factor)
          const uint2 x = *reinterpret_cast<const uint2*>(src + (r0 + STEP * k) * C::ST_ROW);
          u[k] = make_uint4(x.x, x.y, 0u, 0u);
          if (chunk < p.c.D / 16)
            u[k].z = smem[C::OFF_GR + st * C::GR_TILE + (r0 + STEP * k) * (p.c.D / 16) + chunk];
        } else {
          u[k] = *reinterpret_cast<const uint4*>(src + (r0 + STEP * k) * C::ST_ROW);
        }
        if (r0 + STEP * k >= have) u[k] = make_uint4(0u, 0u, 0u, 0u);
      }
      if (!warp_wait(p, bars, &bars->kv_empty[slot], ((i / C::NSLOT) & 1) ^ 1)) return;
#pragma unroll
      for (int k = 0; k < PASSES; ++k) {
        const int r = r0 + STEP * k;
        const uint32_t in[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
        const uint32_t f = __shfl_sync(0xffffffffu, mine, lane / CPR + RPW * k);
        uint32_t w[8];
        if constexpr (C::FP4) {
          // (factor 2^-9 .. 448 times 2^-14 .. 1 and code: multiples of 2^-24, at most 2688)
          const uint32_t fg = mul_f16x2(f, e4m3x2_to_f16x2(in[2] * 0x101u));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t x[4];
            e2m1x8_to_f16x2(in[h], x);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[4 * h + e] = mul_f16x2(x[e], fg);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            e4m3x4_to_f16x2(in[e], w[2 * e], w[2 * e + 1]);
            w[2 * e] = mul_f16x2(w[2 * e], f);
            w[2 * e + 1] = mul_f16x2(w[2 * e + 1], f);
          }
        }
        uint8_t* row = dst + r * C::SWB;
        *reinterpret_cast<uint4*>(row + ((c16 ^ (r & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(row + (((c16 + 1) ^ (r & 7)) * 16)) =
            make_uint4(w[4], w[5], w[6], w[7]);
      }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(ptx::smem_u32(&bars->kv_full[slot]));
      ptx::mbar_arrive(ptx::smem_u32(&bars->st_empty[st]));
    }
    ring += 2 * it.nmax;
    done += it.nmax;
  }
}

// The power of two that takes a bf16 row with `top` (a magnitude's pattern) as its largest
// into [2^14, 2^15).
__device__ __forceinline__ int row_shift(uint32_t top) {
  return min(14 - ((int)(top >> 7) - 127), 126);
}
__device__ __forceinline__ uint32_t larger_magnitude(uint32_t top, const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
  return top;
}
// Two bf16 values as fp16 ones, times `mul`.
__device__ __forceinline__ uint32_t bf16_to_half(uint32_t w, float mul) {
  return pack2<false>(__uint_as_float(w << 16) * mul, __uint_as_float(w & 0xffff0000u) * mul);
}

// The query row at p.q + at to a thread's TMEM lane; for E4M3 keys a bf16 row becomes fp16 times
// 2^sh, and 2^-sh is returned. By a whole warp; rows without a query are zeros.
template <class C, bool BF16>
__device__ float query_to_tmem(const SoftmaxParams& p, uint32_t col, bool any, bool valid,
                               long long at) {
  if (!any) return 1.0f;
  const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at);
  const int pieces = valid ? p.c.D / 8 : 0;  // of 16 bytes, eight at a time in flight
  int sh = 0;
  if constexpr (BF16 && C::CODES) {
    uint32_t top = 0;
#pragma unroll 1
    for (int x0 = 0; x0 < C::D / 8; x0 += 8) {
      uint4 u[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) u[x] = x0 + x < pieces ? q[x0 + x] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int x = 0; x < 8; ++x) top = larger_magnitude(top, u[x]);
    }
    sh = row_shift(top);
  }
  const float mul = power2(sh);
#pragma unroll 1
  for (int x0 = 0; x0 < C::D / 8; x0 += 8) {
    uint4 u[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) u[x] = x0 + x < pieces ? q[x0 + x] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int x = 0; x < 8; x += 2) {
      uint32_t w[8] = {u[x].x,     u[x].y,     u[x].z,     u[x].w,
                       u[x + 1].x, u[x + 1].y, u[x + 1].z, u[x + 1].w};
      if constexpr (BF16 && C::CODES) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = bf16_to_half(w[e], mul);
      }
      ptx::tmem_st8(col + (x0 + x) * 4, w);
    }
  }
  ptx::tmem_st_wait();
  return power2(-sh);
}

// Row r of a bf16 query tile (swizzled shared memory) becomes fp16 times 2^sh; returns 2^-sh.
template <class C>
__device__ float query_to_half(uint8_t* tile, int r) {
  uint32_t top = 0;
#pragma unroll 4
  for (int x = 0; x < C::NCB * 8; ++x)
    top = larger_magnitude(top, *reinterpret_cast<const uint4*>(
                                    tile + (x >> 3) * C::Q_CB + r * C::SWB +
                                    ((x & 7) ^ (r & 7)) * 16));
  const int sh = row_shift(top);
  const float mul = power2(sh);
#pragma unroll 4
  for (int x = 0; x < C::NCB * 8; ++x) {
    uint4* at = reinterpret_cast<uint4*>(tile + (x >> 3) * C::Q_CB + r * C::SWB +
                                         ((x & 7) ^ (r & 7)) * 16);
    const uint4 u = *at;
    *at = make_uint4(bf16_to_half(u.x, mul), bf16_to_half(u.y, mul), bf16_to_half(u.z, mul),
                     bf16_to_half(u.w, mul));
  }
  return power2(-sh);
}

// ------------------------------------------------------------------ products
template <class C, bool BF16>
struct Issuer {
  const SoftmaxParams& p;
  Bars* bars;
  uint32_t sbase, tmem;
  static constexpr uint32_t AB = BF16 && !C::CODES ? 1u : 0u;  // operands: bf16, or fp16
  static constexpr uint32_t IDESC_S = ptx::idesc_f16(AB, 128, C::KT, 0);
  static constexpr uint32_t IDESC_O = ptx::idesc_f16(AB, 128, C::D, 1);

  __device__ __forceinline__ bool kv_ready(int slot, uint32_t phase) {
    return warp_wait(p, bars, &bars->kv_full[slot], phase);
  }
  // scores of query tile q into buffer sb; `last`: the K tile is free after them
  __device__ __forceinline__ void scores(int q, int sb, int slot, bool last) {
    const uint64_t ad0 = ptx::smem_desc(sbase + C::OFF_Q + q * C::Q_TILE, 16, 8 * C::SWB, 2);
    const uint64_t bd0 = ptx::smem_desc(sbase + C::OFF_KV + slot * C::KV_TILE, 16, 8 * C::SWB, 2);
    const uint32_t full = ptx::smem_u32(&bars->s_full[sb]);
    const uint32_t empty = ptx::smem_u32(&bars->kv_empty[slot]);
    if (ptx::elect_one()) {
#pragma unroll
      for (int kk = 0; kk < C::D / 16; ++kk) {
        const uint32_t in = (kk % 4) * 32;
        const uint64_t bd = ptx::desc_add(bd0, (kk / 4) * C::KV_CB + in);
        if constexpr (C::QT)
          ptx::mma_ts(tmem + sb * C::KT, tmem + C::Q_COL + q * (C::D / 2) + kk * 8, bd, IDESC_S,
                      kk > 0 ? 1u : 0u);
        else
          ptx::mma_ss(tmem + sb * C::KT, ptx::desc_add(ad0, (kk / 4) * C::Q_CB + in), bd, IDESC_S,
                      kk > 0 ? 1u : 0u);
      }
      ptx::mma_commit(full);
      if (last) ptx::mma_commit(empty);
    }
    __syncwarp();
  }
  // O of query tile q += P (over score buffer sb) V, for one half of the keys: the first half's
  // product runs while the second half's weights are computed. `last`: the V tile is free after
  // the second one
  __device__ __forceinline__ void accumulate(int q, int sb, int slot, int half, bool first,
                                             bool last) {
    const uint64_t bd0 =
        ptx::smem_desc(sbase + C::OFF_KV + slot * C::KV_TILE, C::KV_CB, 8 * C::SWB, 2);
    const uint32_t done = ptx::smem_u32(&bars->pv_done[q]);
    const uint32_t empty = ptx::smem_u32(&bars->kv_empty[slot]);
    if (ptx::elect_one()) {
#pragma unroll
      for (int x = 0; x < C::KT / 32; ++x) {
        const int kk = half * (C::KT / 32) + x;
        ptx::mma_ts(tmem + C::O_COL + q * C::D, tmem + sb * C::KT + kk * 8,
                    ptx::desc_add(bd0, kk * 16 * C::SWB), IDESC_O, (!first || kk > 0) ? 1u : 0u);
      }
      if (half) {
        ptx::mma_commit(done);
        if (last) ptx::mma_commit(empty);
      }
    }
    __syncwarp();
  }
};

// The ring's places in their order.
template <class C>
struct Place {
  int slot;
  uint32_t phase;
  __device__ __forceinline__ void next() {
    if (++slot == C::NSLOT) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// By a whole warp, of which one lane issues: its values are uniform, what the products'
// instructions want (in one lane's own branch each value went to the uniform registers by itself:
// 4096 tokens over 4096 took 724 us instead of 660, with a head dim of 256 940 instead of 773).
template <class C, bool BF16>
__device__ void mma_role(const SoftmaxParams& p, Issuer<C, BF16>& is, Bars* bars,
                         const PlanTable& pl, int tiles) {
  Place<C> at{0, 0u};
  uint32_t queries = 0;
  uint32_t g[2] = {0, 0};        // key tiles of each query tile before the piece
  uint32_t outputs[2] = {0, 0};  // pieces of it that had any
  Walk w;
  Seg it;
  walk_begin<C>(p, pl, tiles, w);
  while (walk_next<C>(p, pl, w, tiles, it)) {
    const int n = __shfl_sync(0xffffffffu, it.nmax, 0);
    if (n == 0) continue;
    const int nq[2] = {__shfl_sync(0xffffffffu, it.n[0], 0),
                       C::NQT == 2 ? __shfl_sync(0xffffffffu, it.n[1], 0) : 0};
    // Queries that the warpgroups write: those with tiles of the piece arrive (another could run
    // any number of pieces ahead). Queries that they convert: all arrive, and none can fall
    // behind the loads.
#pragma unroll
    for (int q = 0; q < C::NQT; ++q) {
      if (C::QT ? nq[q] > 0 : BF16 && C::CODES)
        if (!warp_wait(p, bars, &bars->q_ready[q], (C::QT ? outputs[q] : queries) & 1)) return;
    }
    if (!C::QT && !(BF16 && C::CODES) && !warp_wait(p, bars, &bars->q_full, queries & 1)) return;
    ++queries;
    // Scores of the first NSB tiles, over weights of the piece before: its last product must be
    // done. (Those before it are: the softmax hands over a piece's last weights only then, so
    // that this wait, too, cannot take one phase for another.)
    for (int t = 0; t < C::NSB && t < n; ++t) {
      if (!is.kv_ready(at.slot, at.phase)) return;
#pragma unroll
      for (int q = 0; q < C::NQT; ++q) {
        if (t >= nq[q]) continue;
        const uint32_t gt = g[q] + t;
        if (t == 0 && gt > 0 && !warp_wait(p, bars, &bars->pv_done[q], (gt - 1) & 1)) return;
        ptx::tc_fence_after();
        is.scores(q, C::NSB == 2 ? gt & 1 : q, at.slot, q == 1 || t >= nq[1]);
      }
      at.next();
    }
    if (!C::QT && n <= C::NSB) {
      if (ptx::elect_one()) ptx::mma_commit(ptx::smem_u32(&bars->q_empty));
      __syncwarp();
    }
    // the piece's first products overwrite O: the previous output has been read
#pragma unroll
    for (int q = 0; q < C::NQT; ++q)
      if (nq[q] > 0 && !warp_wait(p, bars, &bars->o_empty[q], (outputs[q]++ & 1) ^ 1)) return;
    // Then per tile and query tile: O += P(t) V, and the scores of tile t + NSB over P(t), which
    // that product must have read. With two query tiles the softmax of one runs meanwhile. One
    // look at all barriers first: a test takes some 100 cycles, in which the tensor pipe may run
    // empty.
    for (int t = 0; t < n; ++t) {
      const Place<C> v = at;
      at.next();
      const Place<C> k = at;
      uint32_t kv = 0u;  // 4, 8: V(t), K(t + NSB) are known to be there
#pragma unroll
      for (int q = 0; q < C::NQT; ++q) {
        if (t >= nq[q]) continue;
        const uint32_t gt = g[q] + t;
        const int sb = C::NSB == 2 ? gt & 1 : q;
        const uint32_t par = C::NSB == 2 ? (gt >> 1) & 1 : gt & 1;
        uint32_t ready = q == 0
            ? ptx::mbar_tests(ptx::smem_u32(&bars->p_half[sb]), par,
                              ptx::smem_u32(&bars->p_full[sb]), par,
                              ptx::smem_u32(&bars->kv_full[v.slot]), v.phase,
                              ptx::smem_u32(&bars->kv_full[k.slot]), k.phase)
            : ptx::mbar_tests(ptx::smem_u32(&bars->p_half[sb]), par,
                              ptx::smem_u32(&bars->p_full[sb]), par);
        ready = __reduce_and_sync(0xffffffffu, ready);
        if (q == 0) kv = ready;
        if (!(kv & 4u) && !is.kv_ready(v.slot, v.phase)) return;
        kv |= 4u;
        if (!(ready & 1u) && !warp_wait(p, bars, &bars->p_half[sb], par)) return;
        ptx::tc_fence_after();
        is.accumulate(q, sb, v.slot, 0, t == 0, false);
        if (!(ready & 2u) && !warp_wait(p, bars, &bars->p_full[sb], par)) return;
        ptx::tc_fence_after();
        is.accumulate(q, sb, v.slot, 1, false, q == 1 || t >= nq[1]);
        if (t + C::NSB < nq[q]) {
          if (!(kv & 8u) && !is.kv_ready(k.slot, k.phase)) return;
          kv |= 8u;
          if (!warp_wait(p, bars, &bars->pv_done[q], gt & 1)) return;
          ptx::tc_fence_after();
          is.scores(q, sb, k.slot, q == 1 || t + C::NSB >= nq[1]);
        }
      }
      if (t + C::NSB < n) {
        at.next();
        if (!C::QT && t + C::NSB + 1 == n) {
          if (ptx::elect_one()) ptx::mma_commit(ptx::smem_u32(&bars->q_empty));
          __syncwarp();
        }
      }
    }
    g[0] += nq[0];
    g[1] += nq[1];
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

// ------------------------------------------------------------------ softmax
template <class C, bool BF16>
__device__ void softmax_role(const SoftmaxParams& p, Bars* bars, uint8_t* smem, uint32_t tmem,
                             const PlanTable& pl, int tiles, int q, int warp, int lane) {
  constexpr int KT = C::KT;
  const int r = (warp & 3) * 32 + lane;  // row of the tile, TMEM lane
  const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
  const int tpt = 128 / p.G;
  const uint32_t o_col = tmem + lane_off + C::O_COL + q * C::D;
  uint32_t ring = 0, queries = 0, done = 0;  // places, pieces with keys, key tiles before this one
  uint32_t g = 0;                            // key tiles of this query tile before this piece
  Walk walk;
  Seg it;
  walk_begin<C>(p, pl, tiles, walk);
  for (; walk_next<C>(p, pl, walk, tiles, it); ring += 2 * it.nmax, done += it.nmax) {
    float fk = p.scale_log2, fv = 1.0f;  // static factors fold into the scale and the output
    const long long tok = it.tok0 + (long long)q * tpt + r / p.G;
    const bool valid = q < it.nq && r < tpt * p.G && tok < it.s.n;
    const bool any = __any_sync(0xffffffffu, valid);
    if (C::CODES && p.c.k_ds) {
      fk *= p.c.k_ds[(long long)it.b * p.c.ds_b + (long long)it.hk * p.c.ds_h];
      fv = p.c.v_ds[(long long)it.b * p.c.ds_b + (long long)it.hk * p.c.ds_h];
    }
    const int n = C::NQT == 2 && q ? it.n[1] : it.n[0];
    if constexpr (C::QT) {
      if (n > 0) {  // (this tile's scores of the piece before are done: its last have been seen)
        fk *= query_to_tmem<C, BF16>(
            p, tmem + lane_off + C::Q_COL + q * (C::D / 2), any, valid,
            (it.s.t0 + tok) * p.q_stride + (it.hk * p.G + r % p.G) * (long long)p.c.D);
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_u32(&bars->q_ready[q]));
      }
    } else if (BF16 && C::CODES && it.nmax > 0) {
      if (!warp_wait(p, bars, &bars->q_full, queries++ & 1)) return;
      if (valid) fk *= query_to_half<C>(smem + C::OFF_Q + q * C::Q_TILE, r);
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(ptx::smem_u32(&bars->q_ready[q]));
    }
    if (q >= it.nq) continue;
    // keys that the row sees: positions [k0, k0 + lim); rows without a token follow the widest
    long long see = it.kend;
    if (p.causal && valid) see = min(see, it.s.Lk - it.s.n + tok + 1);
    const int lim = (int)max(see - it.k0, 0ll);
    const int rest = (int)min(it.s.Lk - it.k0, 0x7fffffffll);  // keys of the sequence from k0 on
    float m = C::CODES ? kNoKey : -CUDART_INF_F, l = 0.0f;
    float d = 0.0f, o_ref = m;        // E4M3: O's unit is 2^(m + d)
    float lowest = -CUDART_INF_F;     // EV below which a tile's sum is computed apart
    float high = -CUDART_INF_F;       // a score above it raises a reference
    for (int t = 0; t < n; ++t, ++g) {
      const int sb = C::NSB == 2 ? (g & 1) : q;
      const uint32_t par = C::NSB == 2 ? (g >> 1) & 1 : g & 1;
      if (!warp_wait(p, bars, &bars->s_full[sb], par)) return;
      ptx::tc_fence_after();
      float ek = 1.0f, ev = 0.0f;  // the tile's 2^EK and EV
      bool own = false;            // its rows have exponents of their own
      if constexpr (C::CODES) {
        // (with the scores there the conversion has come to this tile; a warpgroup without tiles
        // of the last piece could otherwise be here phases ahead of it)
        const uint32_t te = done + t;
        if (!warp_wait(p, bars, &bars->exp_full[te % kExpDepth], (te / kExpDepth) & 1)) return;
        const float4 x = *reinterpret_cast<const float4*>(bars->tile_exp[te % kExpDepth]);
        ek = x.x;
        ev = x.y;
        own = x.z + x.w > 0.0f;
      }
      // Factor of the scores. For a query of zeros (or nearly) over small keys it would be 0, and
      // a masked score, -inf, NaN by it: the smallest normal value instead leaves scores below
      // 2^-90 (a NaN stays one).
      const float fa = C::CODES ? max_nan(fabsf(fk) * ek, kTiny) : fk;
      const uint32_t s_col = tmem + lane_off + sb * KT;
      constexpr int NC = C::SC / 32;  // chunks held at a time
      uint32_t sv[NC][32];
      float neg = 0.0f;
      if constexpr (C::CODES) {
        neg = ev - o_ref;
        high = fminf(m, kHead - neg) + kLazy;
      }
      const int left = lim - t * KT;  // keys of the tile that the row sees
      const bool masked = !__all_sync(0xffffffffu, left >= KT);
      // columns [c0, c0 + SC) of S: masked scores are -inf (fa is positive: a negative static
      // factor has changed the keys' signs)
      auto load_scores = [&](int c0) {
#pragma unroll
        for (int c = 0; c < NC; ++c) ptx::tmem_ld32_issue(s_col + c0 + c * 32, sv[c]);
        ptx::tmem_ld_wait(sv[0]);
#pragma unroll
        for (int c = 1; c < NC; ++c) ptx::reg_fence(sv[c]);
        if (masked) {
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c0 + c * 32 + e >= left) sv[c][e] = 0xff800000u;
        }
      };
      // V rows beyond the sequence (their pages may hold anything) become zeros: 0 * NaN. (E4M3:
      // the conversion has done that.)
      auto clear_values = [&] {
        const int have = rest - t * KT;
        if (C::CODES || have >= KT) return true;
        const uint32_t vi = ring + v_index<C>(t, it.nmax);
        if (!warp_wait(p, bars, &bars->kv_full[vi % C::NSLOT], (vi / C::NSLOT) & 1)) return false;
        uint8_t* v = smem + C::OFF_KV + (vi % C::NSLOT) * C::KV_TILE;
        const int pieces = (KT - have) * (C::SWB / 16);  // of one column block
        for (int x = r; x < C::NCB * pieces; x += 128)
          *reinterpret_cast<uint4*>(v + (x / pieces) * C::KV_CB + have * C::SWB +
                                    (x % pieces) * 16) = make_uint4(0u, 0u, 0u, 0u);
        ptx::fence_proxy_async_smem();
        return true;
      };
      auto rescale = [&](float corr) {  // O, by a factor
        // (S(t) was issued after PV(t - 2) was done: this phase is the next one)
        if (!warp_wait(p, bars, &bars->pv_done[q], (g - 1) & 1)) return false;
        ptx::tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < C::D; c += 16) {
          uint32_t o[16];
          ptx::tmem_ld16(o_col + c, o);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
          ptx::tmem_st16(o_col + c, o);
        }
        return true;
      };
      if (any) {
        float top[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll 1
        for (int c0 = 0; c0 < KT; c0 += C::SC) {
          load_scores(c0);
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              top[(e >> 1) & 3] = ptx::max3(top[(e >> 1) & 3], __uint_as_float(sv[c][e]),
                                            __uint_as_float(sv[c][e + 1]));
        }
        const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * fa;
        // raise the reference: at the first visible key, and when weights would pass 2^kLazy
        // (any key is above -inf)
        const bool raise = valid && (mx > high || (C::CODES && ev < lowest));
        if (__any_sync(0xffffffffu, raise || own)) {
          float corr = 1.0f;  // (0 at the first visible key)
          bool apart;
          // f(score relative to `ref`, exponent of the value row) of 16 keys from c on
          auto columns = [&](int c, float ref, auto f) {
            uint32_t s[16];
            ptx::tmem_ld16(s_col + c, s);
            uint4 ku = {}, vu = {};
            if constexpr (C::CODES) {
              const uint8_t* rows = bars->row_exp[(done + t) % kExpDepth][0];
              ku = *reinterpret_cast<const uint4*>(rows + c);
              vu = *reinterpret_cast<const uint4*>(rows + 128 + c);
            }
            const uint32_t kw[4] = {ku.x, ku.y, ku.z, ku.w}, vw[4] = {vu.x, vu.y, vu.z, vu.w};
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint32_t kb = (kw[e >> 2] >> (8 * (e & 3))) & 0xffu;
              const int vb = (int)((vw[e >> 2] >> (8 * (e & 3))) & 0xffu) - 127;
              const float k = C::CODES ? fabsf(fk) * scale_value(kb) : fa;
              // (rounded like m: an exact product may be far from a large one's rounding)
              const float y = __fmul_rn(__uint_as_float(s[e]), k) - ref;
              f(e, c + e < left ? y : -CUDART_INF_F, C::CODES ? (float)vb : 0.0f);
            }
          };
          if constexpr (C::CODES) {
            float top = mx;
            if (own) {  // (mx took codes for keys)
              top = -CUDART_INF_F;
#pragma unroll 1
              for (int c = 0; c < KT; c += 16)
                columns(c, 0.0f, [&](int, float y, float) { top = fmaxf(top, y); });
            }
            if (valid && top > m + kLazy) {
              const float to = ceilf(top);
              l *= ex2(m - to);
              d += m - to;
              m = to;
            }
            float u = (top - m) + ev;
            if (own) {
              u = -CUDART_INF_F;
#pragma unroll 1
              for (int c = 0; c < KT; c += 16)
                columns(c, m, [&](int, float y, float e) { u = fmaxf(u, y + e); });
            }
            if (valid && u > d + (kHead + kLazy)) {
              const float to = ceilf(u) - kHead;
              corr = ex2(d - to);
              d = to;
            }
            // The sum cannot take this tile's weights: 2^-30 of its unit is below 2^-126 of O's, or
            // neg loses bits.
            if (valid && m != kNoKey) lowest = fabsf(m) > kLargeScore ? CUDART_INF_F : d - kApart;
            apart = __any_sync(0xffffffffu, ev < lowest) || own;
            o_ref = m + d;
            neg = ev - o_ref;
          } else {
            if (valid && mx > m + kLazy) {
              corr = ex2(m - mx);
              m = mx;
              l *= corr;
              high = fabsf(m) > kLargeScore ? -CUDART_INF_F : m + kLazy;
            }
            apart = __any_sync(0xffffffffu, high < m);
          }
          // Such tiles in two steps: each score relative to m first, which is what the sum takes,
          // then the weight. (Few calls come here. 16 columns at a time, in this branch that few
          // tiles take, cost the others nothing; beside the loop below this took 4-8 % of prompts.)
          if (apart) {
            if (t > 0 && __any_sync(0xffffffffu, corr != 1.0f) && !rescale(corr)) return;
            if (!clear_values()) return;
#pragma unroll 1
            for (int c = 0; c < KT; c += 16) {
              uint32_t pk[8];
              float w[16];
              columns(c, !C::CODES && m == -CUDART_INF_F ? 0.0f : m, [&](int i, float y, float e) {
                l += ex2(y);
                w[i] = ex2(C::CODES ? y + (e - d) : y);
              });
#pragma unroll
              for (int e = 0; e < 8; ++e)
                pk[e] = pack2<BF16 && !C::CODES>(w[2 * e], w[2 * e + 1]);
              ptx::tmem_st8(s_col + c / 2, pk);
              if (c == KT / 2 - 16) {
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                ptx::mbar_arrive(ptx::smem_u32(&bars->p_half[sb]));
              }
            }
            ptx::tmem_st_wait();
            if (C::NSB > 1 && t > 0 && t == n - 1 &&
                !warp_wait(p, bars, &bars->pv_done[q], (g - 1) & 1))
              return;
            ptx::tc_fence_before();
            ptx::mbar_arrive(ptx::smem_u32(&bars->p_full[sb]));
            continue;
          }
          if (t > 0 && !rescale(corr)) return;
        }
        if constexpr (!C::CODES) neg = m == -CUDART_INF_F ? 0.0f : -m;
      }
      if (!clear_values()) return;
      float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
      // weights of chunk `at` held in sv[i], summed and stored as columns of P
      auto weights = [&](int i, int at) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float x0, x1;
          ptx::fma_f32x2(x0, x1, __uint_as_float(sv[i][2 * e]), __uint_as_float(sv[i][2 * e + 1]),
                         fa, fa, neg, neg);
          const float p0 = ex2(x0), p1 = ex2(x1);
          ptx::add_f32x2(sum[e & 1][0], sum[e & 1][1], p0, p1);
          pk[e] = pack2<BF16 && !C::CODES>(p0, p1);
        }
        ptx::tmem_st16(s_col + at * 16, pk);
      };
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        if (any) {
          load_scores(half * C::SC);
#pragma unroll
          for (int c = 0; c < NC; ++c) weights(c, half * NC + c);
          ptx::tmem_st_wait();
        }
        if (half == 0) {
          ptx::tc_fence_before();
          ptx::mbar_arrive(ptx::smem_u32(&bars->p_half[sb]));
        }
      }
      const float tile_sum = (sum[0][0] + sum[0][1]) + (sum[1][0] + sum[1][1]);
      // (the sum's unit is 2^m, the weights' 2^(m + d - ev))
      l = C::CODES ? fmaf(tile_sum, ex2(-neg - m), l) : l + tile_sum;
      // A parity wait cannot tell a phase from the one two before it. The wait for PV(n - 1)
      // below needs PV(n - 2) to be done (of the piece before, it is); S(n - 1) was issued after
      // PV(n - 1 - NSB) only, and once P(n - 1) is handed over both may complete at any time.
      if (C::NSB > 1 && t > 0 && t == n - 1 &&
          !warp_wait(p, bars, &bars->pv_done[q], (g - 1) & 1))
        return;
      ptx::tc_fence_before();
      ptx::mbar_arrive(ptx::smem_u32(&bars->p_full[sb]));
    }
    if (n > 0) {
      if (!warp_wait(p, bars, &bars->pv_done[q], (g - 1) & 1)) return;
      ptx::tc_fence_after();
    }
    // out and lse of the row, or its place in the workspace
    const long long row = (it.s.t0 + tok) * p.Nq + it.hk * p.G + r % p.G;
    const long long part = (long long)it.slot * (C::NQT * 128) + q * 128 + r;
    float inv = l > 0.0f ? fv / l : l;  // (a NaN sum stays one)
    float unit = 1.0f;  // 2^d in two factors: it may pass fp32's range where the output does not
    if constexpr (C::CODES) {
      const int e = (int)d;
      inv *= power2(e / 2);
      unit = power2(e - e / 2);
    }
    const int D = p.c.D;
#pragma unroll 1
    for (int c = 0; any && c < D; c += 16) {
      uint32_t o[16];
      if (n > 0) {
        ptx::tmem_ld16(o_col + c, o);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = 0u;
      }
      if (!valid) continue;
      float f[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) f[e] = l == 0.0f ? 0.0f : __uint_as_float(o[e]) * inv * unit;
      if (it.slot >= 0) {
        store16(p.part_o + part * D + c, f);
      } else if constexpr (BF16) {
        store16(static_cast<__nv_bfloat16*>(p.out) + row * D + c, f);
      } else {
        store16(static_cast<__half*>(p.out) + row * D + c, f);
      }
    }
    if (valid) {
      const float log2sum = l == 0.0f ? -CUDART_INF_F : m + log2f(l);
      if (it.slot >= 0)
        p.part_lse[part] = log2sum;
      else if (p.lse)
        p.lse[row] = log2sum * kLn2;
    }
    if (n > 0) {  // O has been read: the next piece's products may overwrite it
      ptx::tc_fence_before();
      ptx::mbar_arrive(ptx::smem_u32(&bars->o_empty[q]));
    }
  }
}

// ------------------------------------------------------------------ kernel
template <int D, int NQT, int CTAS, bool BF16, int FMT>
__global__ void __launch_bounds__(Cfg<D, NQT, CTAS, FMT>::THREADS, CTAS)
    softmax_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_c, const SoftmaxParams p,
                      int tiles) {
  using C = Cfg<D, NQT, CTAS, FMT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + C::OFF_BAR);
  PlanTable& pl = *reinterpret_cast<PlanTable*>(smem + C::OFF_PLAN);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == C::LOAD_WARP && lane == 0) {
    ptx::mbar_init(ptx::smem_u32(&bars->q_full), 1);
    ptx::mbar_init(ptx::smem_u32(&bars->q_empty), 1);
    ptx::mbar_init(ptx::smem_u32(&bars->drain), 1);
    for (int s = 0; s < kExpDepth; ++s) ptx::mbar_init(ptx::smem_u32(&bars->exp_full[s]), 2);
    for (int s = 0; s < C::NSLOT; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bars->kv_full[s]), C::CODES ? 128 : 1);
      ptx::mbar_init(ptx::smem_u32(&bars->kv_empty[s]), 1);
    }
    for (int s = 0; s < 4; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bars->st_full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->st_empty[s]), 128);
    }
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(ptx::smem_u32(&bars->s_full[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->p_half[s]), 128);
      ptx::mbar_init(ptx::smem_u32(&bars->p_full[s]), 128);
      ptx::mbar_init(ptx::smem_u32(&bars->pv_done[s]), 1);
      ptx::mbar_init(ptx::smem_u32(&bars->o_empty[s]), 128);
      ptx::mbar_init(ptx::smem_u32(&bars->q_ready[s]), 128);
    }
    bars->abort = 0;
    ptx::fence_barrier_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == C::MMA_WARP) {
    ptx::tmem_alloc(ptx::smem_u32(&bars->tmem_base), C::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  if (p.balanced) make_plan<C>(p, pl);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  // With E4M3's conversion warps the launch leaves the softmax too few registers. 512 threads
  // launch with 128 each (65,536): 208 for its warps and 96 for the others are 63,488. 640 launch
  // with 96 (61,440): 120 and 80 are as many.
  if constexpr (C::CODES) {
    if (warp < C::SM_WARPS)
      ptx::regs_inc<C::NQT == 2 ? 120 : 208>();
    else
      ptx::regs_dec<C::NQT == 2 ? 80 : 96>();
  }
  if (warp < C::SM_WARPS) {
    softmax_role<C, BF16>(p, bars, smem, tmem, pl, tiles, warp / 4, warp, lane);
  } else if (warp == C::MMA_WARP) {
    Issuer<C, BF16> is{p, bars, ptx::smem_u32(smem), __shfl_sync(0xffffffffu, tmem, 0)};
    mma_role<C, BF16>(p, is, bars, pl, tiles);
    mma_drain(p, bars);
  } else if (warp == C::LOAD_WARP) {
    if (lane == 0) load_role<C>(p, bars, smem, pl, tiles, &tm_q, &tm_c);
  } else if (warp == C::LOAD_WARP + 1) {
    if (p.balanced && lane == 0) p.joins[blockIdx.x] = join_record<C>(p, pl, tiles);
  } else if (C::CODES && warp >= C::CONV_WARP) {
    const int w = warp - C::CONV_WARP;
    convert_role<C>(p, bars, smem, pl, tiles, w >= 4, w & 3, lane);
  }
  __syncwarp();
  ptx::tc_fence_before();
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

template <int D, int NQT, int CTAS, bool BF16, int FMT>
cudaError_t launch_variant(const SoftmaxParams& p, const CUtensorMap& tq, const CUtensorMap& tc,
                           long long tiles, long long blocks, cudaStream_t stream) {
  using C = Cfg<D, NQT, CTAS, FMT>;
  auto* kernel = softmax_tc_kernel<D, NQT, CTAS, BF16, FMT>;
  static std::atomic<unsigned long long> done;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), C::SMEM, done);
  if (e != cudaSuccess) return e;
  kernel<<<dim3((unsigned)blocks), C::THREADS, C::SMEM, stream>>>(tq, tc, p, (int)tiles);
  return cudaGetLastError();
}

// Kernel for the head dim, the number of query tiles and the CTAs of an SM.
template <int D, bool BF16, int FMT>
cudaError_t launch_dim(const SoftmaxParams& p, const CUtensorMap& tq, const CUtensorMap& tc,
                       int qtiles, int ctas, long long tiles, long long blocks, cudaStream_t s) {
  if constexpr (FMT == kSame) {
    if (ctas == 2) return launch_variant<D, 1, 2, BF16, FMT>(p, tq, tc, tiles, blocks, s);
  }
  return qtiles == 2 ? launch_variant<D, 2, 1, BF16, FMT>(p, tq, tc, tiles, blocks, s)
                     : launch_variant<D, 1, 1, BF16, FMT>(p, tq, tc, tiles, blocks, s);
}
template <bool BF16, int FMT>
cudaError_t launch_tc(const SoftmaxParams& p, const CUtensorMap& tq, const CUtensorMap& tc,
                      int qtiles, int ctas, long long tiles, long long blocks, cudaStream_t s) {
  if (p.c.D > 128) return launch_variant<256, 1, 1, BF16, FMT>(p, tq, tc, tiles, blocks, s);
  if (p.c.D > 64) return launch_dim<128, BF16, FMT>(p, tq, tc, qtiles, ctas, tiles, blocks, s);
  return launch_dim<64, BF16, FMT>(p, tq, tc, qtiles, ctas, tiles, blocks, s);
}

}  // namespace sm
}  // namespace hstu
