// Moving the kept rows of a paged cache together, in place (hstu_kv_compact).
//
// Positions increase in the list of kept rows, so that rank r never lies behind its source: a CTA per
// (sequence, kv head) takes the ranks in order, some at a time, whose rows it holds in registers
// between its loads and its stores.
#include "common.cuh"
#include "evict_kernels.h"
#include "kernels.h"
#include "kv_cache.cuh"

namespace hstu {

namespace {

constexpr int kThreads = 256, kPieces = 8;  // 16-byte pieces that a thread holds
constexpr int kMaxRows = 256;               // ranks of a round

// Rows of one head in plane 0 (the other lies `plane` rows further on).
struct Move {
  long long from, to;        // rows of the cache, -1: nothing to move
  long long sfrom, sto;      // of the scales
};

__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactParams p, int rows) {
  __shared__ Move moves[kMaxRows];
  __shared__ int s_any;
  const int hk = (int)(blockIdx.x % (unsigned)p.c.Nk), b = (int)(blockIdx.x / (unsigned)p.c.Nk);
  const int tid = threadIdx.x;
  const PagedSeq s = paged_table(p.c, b);
  if (!s.ok || s.Lk > p.max_k) {
    if (tid == 0) report(p.c, HSTU_DEVERR_OFFSETS);
    return;
  }
  const int* kept = p.kept + ((long long)b * p.c.Nk + hk) * p.budget;
  const int most = (int)min(s.Lk, (long long)p.budget);
  const int pieces = p.row_bytes / 16, gb = p.c.D / 16;
  const long long plane = (long long)p.c.Nk << p.c.page_shift;  // rows of a plane
  auto row_of = [&](long long page, long long pos, bool by_head) {
    const long long row = pos & (page_size(p.c) - 1);
    return by_head ? scale_row(p.c, page, 0, row, hk)
                   : (((page * 2) << p.c.page_shift) + row) * p.c.Nk + hk;
  };
  for (int r0 = 0; r0 < most; r0 += rows) {
    const int n = min(rows, most - r0);
    __syncthreads();  // the stores of the round before are done with `moves`
    if (tid == 0) s_any = 0;
    __syncthreads();
    if (tid < n) {
      const int r = r0 + tid, src = kept[r];
      Move m = {-1, -1, -1, -1};
      if (src > r && src < s.Lk) {
        const long long a = page_at(p.c, s, src), d = page_at(p.c, s, r);
        if (a >= 0 && d >= 0) {
          m.from = row_of(a, src, p.by_head);
          m.to = row_of(d, r, p.by_head);
          m.sfrom = row_of(a, src, true);
          m.sto = row_of(d, r, true);
          s_any = 1;
        } else {
          report(p.c, HSTU_DEVERR_OFFSETS);
        }
      } else if (src >= 0 && src != r) {
        report(p.c, HSTU_DEVERR_OFFSETS);
      }
      moves[tid] = m;
    }
    __syncthreads();
    if (!s_any) continue;
    const int all = n * 2 * pieces;  // at most kThreads * kPieces
    uint4* cache = static_cast<uint4*>(p.c.cache);
    uint4 u[kPieces];
    uint16_t group[kPieces];
    uint8_t scale[2];
    float weight = 0.f;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int x = i * kThreads + tid, r = x / (2 * pieces), y = x % (2 * pieces);
      if (x < all && moves[r].from >= 0)
        u[i] = cache[(moves[r].from + (y >= pieces ? plane : 0)) * pieces + y % pieces];
      if (p.c.group) {
        const int gr = x / gb, gy = x % gb;  // pairs of factors, of both planes
        if (gr < n && moves[gr].from >= 0)
          group[i] = reinterpret_cast<const uint16_t*>(
              p.c.group)[(moves[gr].sfrom + (gy >= gb / 2 ? plane : 0)) * (gb / 2) + gy % (gb / 2)];
      }
    }
    if (p.c.scale) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (tid < n && moves[tid].from >= 0) scale[i] = p.c.scale[moves[tid].sfrom + i * plane];
    }
    // (a scale row of plane 0 lies in page 2 * page: half of it is the weights' place)
    auto weight_at = [&](long long srow) {
      const long long page = srow / (2 * plane);
      return page * plane + (srow - page * 2 * plane);
    };
    if (p.weights && tid < n && moves[tid].from >= 0) weight = p.weights[weight_at(moves[tid].sfrom)];
    __syncthreads();  // every row of the round is in registers
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int x = i * kThreads + tid, r = x / (2 * pieces), y = x % (2 * pieces);
      if (x < all && moves[r].from >= 0)
        cache[(moves[r].to + (y >= pieces ? plane : 0)) * pieces + y % pieces] = u[i];
      if (p.c.group) {
        const int gr = x / gb, gy = x % gb;
        if (gr < n && moves[gr].from >= 0)
          reinterpret_cast<uint16_t*>(
              p.c.group)[(moves[gr].sto + (gy >= gb / 2 ? plane : 0)) * (gb / 2) + gy % (gb / 2)] =
              group[i];
      }
    }
    if (tid < n && moves[tid].from >= 0) {
      if (p.c.scale) {
#pragma unroll
        for (int i = 0; i < 2; ++i) p.c.scale[moves[tid].sto + i * plane] = scale[i];
      }
      if (p.weights) p.weights[weight_at(moves[tid].sto)] = weight;
    }
  }
}

}  // namespace

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream) {
  // as many rows as the registers hold, of both planes (the factors of an E2M1 row are an eighth
  // of it, a 16-bit piece of them for each of its own)
  int rows = kThreads * kPieces / (2 * (p.row_bytes / 16));
  if (rows > kMaxRows) rows = kMaxRows;
  compact_kernel<<<(unsigned)((long long)p.c.B * p.c.Nk), kThreads, 0, stream>>>(p, rows);
  return cudaGetLastError();
}

}  // namespace hstu
