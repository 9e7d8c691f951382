// Paged KV cache as the cache operators' kernels see it: the page table, a sequence's
// geometry with the checks of it, and conversions of E4M3 elements.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/hstu_kv.h"
#include "kernels.h"

namespace hstu {

// Device view of hstu_kv_cache (see include/hstu_kv.h).
struct CacheView {
  void* cache;              // [num_pages, 2, page_size, Nk, D]
  uint8_t* scale;           // [num_pages, 2, Nk, page_size] or nullptr
  const void* page_offsets;
  const void* page_ids;
  const void* last_page_len;
  const void* seq_offsets;  // [B + 1] rows of the call's q, or of its k and v
  const float* k_ds;        // static factors: entry b * ds_b + hk * ds_h, or nullptr
  const float* v_ds;
  int* status;
  long long num_pages, num_page_ids, T;
  int index64, B, Nk, D;
  int page_shift;           // log2(page_size)
  int ds_b, ds_h;
};

__device__ __forceinline__ long long page_size(const CacheView& c) { return 1ll << c.page_shift; }

__device__ __forceinline__ void report(const CacheView& c, int what) {
  if (c.status) atomicCAS(c.status, HSTU_DEVERR_NONE, what);
}

// A sequence: query (or new) rows [t0, t0 + n), Lk cached rows in pages [po, po + pages).
struct PagedSeq {
  long long t0, n, Lk, po, pages;
  bool ok;  // offsets and lengths are valid; the page ids are checked where they are used
};

__device__ __forceinline__ PagedSeq paged_seq(const CacheView& c, long long b) {
  PagedSeq s;
  s.t0 = load_index(c.seq_offsets, b, c.index64);
  const long long t1 = load_index(c.seq_offsets, b + 1, c.index64);
  s.po = load_index(c.page_offsets, b, c.index64);
  const long long pe = load_index(c.page_offsets, b + 1, c.index64);
  const long long last = load_index(c.last_page_len, b, c.index64);
  s.n = t1 - s.t0;
  s.pages = pe - s.po;
  s.ok = s.t0 >= 0 && s.n >= 0 && t1 <= c.T && s.po >= 0 && s.pages >= 0 && pe <= c.num_page_ids &&
         (s.pages == 0 || (last >= 1 && last <= page_size(c)));
  s.Lk = s.ok && s.pages > 0 ? ((s.pages - 1) << c.page_shift) + last : 0;
  return s;
}

// Page that holds position pos of a valid sequence (pos < Lk), or -1 if its id is outside
// the cache.
__device__ __forceinline__ long long page_at(const CacheView& c, const PagedSeq& s,
                                             long long pos) {
  const long long id = load_index(c.page_ids, s.po + (pos >> c.page_shift), c.index64);
  return id >= 0 && id < c.num_pages ? id : -1;
}

// First element of (page, plane, row of the page, kv head) in the cache.
__device__ __forceinline__ long long cache_row(const CacheView& c, long long page, int plane,
                                               long long row, int hk) {
  return ((((page * 2 + plane) << c.page_shift) + row) * c.Nk + hk) * c.D;
}
__device__ __forceinline__ long long scale_row(const CacheView& c, long long page, int plane,
                                               long long row, int hk) {
  return (((page * 2 + plane) * c.Nk + hk) << c.page_shift) + row;
}

// The sequence that row t belongs to by seq_offsets (the last b with seq_offsets[b] <= t), by
// bisection; offsets that decrease give some b in range, whose rows the caller compares.
__device__ __forceinline__ int seq_of_row(const CacheView& c, long long t) {
  int lo = 0, hi = c.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (load_index(c.seq_offsets, mid, c.index64) <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// 2^(s - 127): the exponent field itself.
__device__ __forceinline__ float scale_value(uint32_t s) { return __uint_as_float(s << 23); }

// Two E4M3 codes (the low 16 bits of x) as two fp16 values (exact: E4M3's range and
// precision lie inside fp16's).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)x));
  return r;
}

// Four codes as two pairs.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}

// Sixteen consecutive elements as fp32 values (exact).
template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&x)[16]);
template <>
__device__ __forceinline__ void load16<float>(const float* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 f = reinterpret_cast<const float4*>(p)[i];
    x[4 * i] = f.x;
    x[4 * i + 1] = f.y;
    x[4 * i + 2] = f.z;
    x[4 * i + 3] = f.w;
  }
}
template <>
__device__ __forceinline__ void load16<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 u = reinterpret_cast<const uint4*>(p)[i];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[8 * i + 2 * e] = __uint_as_float(w[e] << 16);
      x[8 * i + 2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
}
template <>
__device__ __forceinline__ void load16<__half>(const __half* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 u = reinterpret_cast<const uint4*>(p)[i];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
      x[8 * i + 2 * e] = f.x;
      x[8 * i + 2 * e + 1] = f.y;
    }
  }
}
template <>
__device__ __forceinline__ void load16<uint8_t>(const uint8_t* p, float (&x)[16]) {  // E4M3
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t h = e4m3x2_to_f16x2(w[i >> 1] >> (16 * (i & 1)));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// Sixteen fp32 values rounded once to T and stored.
template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&x)[16]);
template <>
__device__ __forceinline__ void store16<float>(float* p, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4*>(p)[i] =
        make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* p, const float (&x)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
template <>
__device__ __forceinline__ void store16<__half>(__half* p, const float (&x)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2 v = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// ------------------------------------------------------------- softmax attention
// Items of a balanced run of the tensor-core kernel: (sequence, tile of query tokens) pairs in
// order, each of them once per kv head.
constexpr int kMaxItems = 512, kMaxSeqs = 512;
struct PlanTable {
  long long cost[kMaxItems + 1];  // running sum of the pairs' costs, in key tiles
  int first[kMaxSeqs + 1];        // first pair of each sequence
  uint16_t seq[kMaxItems];        // sequence of each pair
  int items;
};
constexpr int kPlanSharedBytes = sizeof(PlanTable);

// What to join at the border in front of CTA c's share, written by CTA c: pieces of CTAs
// c - 1 .. c - 2 + count make up the outputs of one item (count 0: nothing to join here).
struct JoinRecord {
  int count, hk;
  int rows;      // of the item (its tokens times G)
  long long t0;  // its first token
};

// An item costs its key tiles and kItemCost for what it needs besides (its queries' load, the
// first products' and the output's latency). These units, all heads' of a pair in a row, are
// shared out equally: CTA c takes units [share(c), share(c + 1)).
constexpr int kItemCost = 2;
constexpr int kMinUnits = 4;  // fewest units worth a CTA
__host__ __device__ inline long long share(long long units, int ctas, int c) {
  return units * c / ctas;
}
__host__ __device__ inline int share_ctas(long long units, int grid) {
  const long long c = units / kMinUnits;
  return c < 1 ? 1 : c < grid ? (int)c : grid;
}
// Key tiles [from, to) of an item of `cost` units that its units [o1, o2) stand for. A piece
// from 0 to the last is the whole item; others lie in workspace slot 2 c (a piece that CTA c
// begins inside an item) or 2 c + 1 (one that it ends inside).
struct KeyTiles {
  int from, to;
};
__host__ __device__ inline KeyTiles piece_tiles(long long o1, long long o2) {
  KeyTiles k;
  k.from = o1 > kItemCost ? (int)(o1 - kItemCost) : 0;
  k.to = o2 > kItemCost ? (int)(o2 - kItemCost) : 0;
  return k;
}

struct SoftmaxParams {
  CacheView c;
  const void* q;
  void* out;
  float* lse;              // [T, Nq] or nullptr
  float* part_o;           // [splits][T, Nq, D]: each key range's normalised output, or (balanced)
                           // [2 per CTA][rows of an item][D]: each piece's
  float* part_lse;         // the same without D: log2 of the sums (-inf: no key)
  JoinRecord* joins;       // [CTAs] what to join at each share's border (balanced)
  int balanced;            // tensor-core kernel: CTAs share the items' key tiles equally
  long long q_stride;      // elements
  int Nq, G;               // query heads, query heads of one kv head
  int max_q;               // bound on n
  long long max_k;         // bound on Lk
  int causal;
  float scale_log2;        // alpha * log2(e): scores in powers of two
  int splits;              // most key ranges of one sequence (1: outputs are written at once)
  int min_range;           // fewest keys worth a range of their own (a multiple of 128)
  long long timeout_ns;
};

// Key ranges of a sequence of Lk keys: `count` ranges of `keys` keys each (a multiple of 128;
// the last may be shorter). They follow from the sequence's own length, not from the bound on
// it, so that a loose bound costs no parallelism.
struct KeyRanges {
  long long keys;
  int count;
};
__device__ __forceinline__ KeyRanges key_ranges(const SoftmaxParams& p, long long Lk) {
  KeyRanges r;
  r.keys = ((Lk + p.splits - 1) / p.splits + 127) & ~127ll;
  if (r.keys < p.min_range) r.keys = p.min_range;
  r.count = Lk > 0 ? (int)((Lk + r.keys - 1) / r.keys) : 1;
  return r;
}

__device__ __forceinline__ bool attn_seq_ok(const SoftmaxParams& p, const PagedSeq& s) {
  return s.ok && s.n <= p.max_q && s.Lk <= p.max_k;
}

}  // namespace hstu
