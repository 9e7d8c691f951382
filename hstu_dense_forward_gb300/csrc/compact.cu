// Moving the kept rows of a paged cache together, in place (hstu_kv_compact).
//
// Rank r of a (sequence, kv head) takes the row at position kept[r] >= r. Ranks are moved in chunks,
// each by a CTA that holds the chunk's rows in registers between its loads and its stores. Positions
// increase with the ranks, so that what a chunk overwrites can be a source of that chunk and of those
// in front of it only, two of them at most: it stores once those have loaded. Chunks are handed out by a
// counter, in order for every (sequence, kv head). A CTA takes its next chunk's number before it is done
// with the one it has, so that the CTA that has a chunk in front may still wait itself; but waits are
// for lower numbers only, and the lowest one that is not done has nothing to wait for. (One CTA for all
// of a (sequence, kv head), chunk after chunk: 128 of 4096 ranks of 256-byte rows took 312 us, one of
// 50,000 3355; now 94 and 20.) Lists that do not increase end there, and which chunks one waits for
// follows from the list, too: a launch of its own finds both. (Chunks that asked all in front of them for
// the list's end waited for CTAs at an earlier chunk: eight lists that keep 40,000 of 100,000 rows took
// 105 us in place of 79, now 64.) Bound by memory: a kept row is read once and written once (rows of
// 256 bytes 94 us for 32 sequences, 4096 of 4k-16k rows of four heads, 5.7 TB/s; E4M3 59, E2M1 51).
#include "common.cuh"
#include "evict_kernels.h"
#include "kernels.h"
#include "kv_cache.cuh"
#include "ptx.cuh"

namespace hstu {

namespace {

constexpr int kThreads = 256, kPieces = 8;  // 16-byte pieces that a thread holds
constexpr int kCtas = 4;                    // of an SM

// A row of one head in plane 0: its first 16-byte piece in the cache, and the row among those of what
// has its heads before the rows (the other plane lies a plane further on).
struct Move {
  long long from, to;  // -1: nothing to move
  long long sfrom, sto;
};

__device__ __forceinline__ int load_acquire(const int* p) {
  int x;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(x) : "l"(p) : "memory");
  return x;
}
__device__ __forceinline__ void store_release(int* p, int x) {
  asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(x) : "memory");
}

// Whether rank r is none of the list's, whose positions increase.
__device__ __forceinline__ bool ends_at(const int* kept, int r, long long Lk) {
  const int src = kept[r];
  return src >= Lk || src <= (r ? kept[r - 1] : -1);
}

// Where lists end: ends[pair] becomes kNoEnd - the first rank that is none of the list's, and stays 0
// where all are. And which chunks in front have sources where a chunk stores, two at most, next to each
// other: fronts[..] is four times the first, plus how many. Positions increase up to the list's end, so
// that the lanes' looks at the ends of 32 parts of the chunks leave one part. (All of them looked at by
// every chunk: a list of a million rows of 256 bytes took 721 us, now 181; of 100,000 fp32 rows of
// D = 256, 6250 chunks, 120 and 77.) A warp for each chunk.
constexpr int kNoEnd = 0x7fffffff;
__global__ void __launch_bounds__(kThreads) lists_kernel(const CompactParams p, int rows, int chunks) {
  const long long ticket = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (ticket >= (long long)p.c.B * p.c.Nk * chunks) return;
  const long long pair = ticket / chunks;
  const PagedSeq s = paged_table(p.c, pair / p.c.Nk);
  const int* kept = p.kept + pair * p.budget;
  const int most = s.ok && s.Lk <= p.max_k ? (int)min(s.Lk, (long long)p.budget) : 0;
  const int chunk = (int)(ticket % chunks), r0 = chunk * rows, last = min(r0 + rows, most);
  const int lane = threadIdx.x & 31;
  if (r0 >= most) return;
  int lo = 0, len = chunk;  // the first with a source at r0 or behind is one of [lo, lo + len]
  while (len > 30) {
    const int step = (len + 31) / 32;
    const int end = lo + min((lane + 1) * step, len) - 1;  // of the lane's part
    const int before = min(len, step * __popc(__ballot_sync(
        0xffffffffu, lane * step < len && kept[end * rows + rows - 1] < r0)));
    lo += before;
    len = max(min(step, len - before) - 1, 0);  // (the part's last one is at r0 or behind)
  }
  const int c = lo + lane;  // (and the one behind it)
  const bool look = lane <= len + 1 && c < chunk;
  const int c_first = look ? kept[c * rows] : r0 + rows, c_last = look ? kept[c * rows + rows - 1] : 0;
  int end = kNoEnd;
#pragma unroll
  for (int i = 0; i < kCompactRows / 32; ++i) {
    const int r = r0 + lane + 32 * i;
    if (r < last && ends_at(kept, r, s.Lk)) end = min(end, r);
  }
  if (end < kNoEnd) atomicMax(p.ends + pair, kNoEnd - end);
  const uint32_t with = __ballot_sync(0xffffffffu, c_first < r0 + rows && c_last >= r0);
  if (lane == 0) p.fronts[ticket] = with ? 4 * (lo + __ffs(with) - 1) + min(__popc(with), 2) : 0;
}

__global__ void __launch_bounds__(kThreads, kCtas)
    compact_kernel(const CompactParams p, int rows, int chunks, int lanes_shift) {
  __shared__ Move moves[kCompactRows];
  __shared__ int s_ticket, s_any, s_late, s_end, s_front;
  const int tid = threadIdx.x;
  const int pieces = p.row_bytes / 16;
  const long long plane = (long long)p.c.Nk << p.c.page_shift;  // rows of a plane
  const unsigned pairs = (unsigned)p.c.B * p.c.Nk;
  const long long tickets = (long long)pairs * chunks;
  uint4* cache = static_cast<uint4*>(p.c.cache);
  // (a row among those with heads before rows, without the planes: the weights' place)
  auto weight_at = [&](long long srow) {
    const long long page = srow / (2 * plane);
    return srow - page * plane;
  };
  // 2^lanes_shift lanes take the pieces of a row, of plane 0 and then of plane 1: of each round's
  // rows, this thread one piece. An E2M1 row has as many 16-bit pieces of factors.
  const int y = tid & ((1 << lanes_shift) - 1), step = kThreads >> lanes_shift;
  const int row0 = y < 2 * pieces ? tid >> lanes_shift : kCompactRows;  // (a lane too many: no row)
  const long long off = y >= pieces ? plane * pieces + y - pieces : y;
  uint16_t* factors = reinterpret_cast<uint16_t*>(p.c.group);
  // (one chunk each: they are not handed out, and none waits)
  if (tid == 0) s_ticket = chunks > 1 ? atomicAdd(p.counter, 1) : (int)blockIdx.x;
  __syncthreads();
  for (;;) {
    const unsigned ticket = (unsigned)s_ticket;
    if ((long long)ticket >= tickets) return;
    const int chunk = (int)(ticket / pairs), pair = (int)(ticket % pairs);
    const int hk = pair % p.c.Nk, b = pair / p.c.Nk;
    const PagedSeq s = paged_table(p.c, b);
    const bool ok = s.ok && s.Lk <= p.max_k;
    const int* kept = p.kept + ((long long)b * p.c.Nk + hk) * p.budget;
    const int most = ok ? (int)min(s.Lk, (long long)p.budget) : 0;
    // ranks of the list (of one chunk, whose end is not known yet: that it may have)
    const int end = chunks > 1 ? min(most, kNoEnd - p.ends[pair]) : most;
    const int r0 = chunk * rows;
    int n = max(0, min(rows, end - r0));
    int* loaded = p.loaded + (long long)pair * chunks;  // chunks that have loaded
    auto goes_on = [&](int end) {  // (lists end at negative positions, or with the budget)
      return ok ? end < p.budget && kept[end] >= 0 : hk == 0;
    };
    if (tid == 0 && chunk == 0 && (chunks > 1 || n == 0) && goes_on(end))
      report(p.c, HSTU_DEVERR_OFFSETS);
    __syncthreads();  // everyone has the ticket, and the chunk before is done with `moves`
    if (tid == 0) {
      // (its latency passes meanwhile)
      s_ticket = chunks > 1 ? atomicAdd(p.counter, 1) : (int)(ticket + gridDim.x);
      s_front = chunks > 1 && n > 0 ? p.fronts[(long long)pair * chunks + chunk] : 0;
      s_any = s_late = 0;
      s_end = n;
    }
    __syncthreads();
    if (n > 0) {
      for (int x = tid; x < n; x += kThreads) {
        const int r = r0 + x, src = kept[r];
        Move m = {-1, -1, -1, -1};
        if (chunks == 1 && ends_at(kept, r, s.Lk)) {
          atomicMin(&s_end, r);
        } else if (src > r) {
          const long long a = page_at(p.c, s, src), d = page_at(p.c, s, r);
          if (a >= 0 && d >= 0) {
            const long long mask = page_size(p.c) - 1;
            m.sfrom = scale_row(p.c, a, 0, src & mask, hk);
            m.sto = scale_row(p.c, d, 0, r & mask, hk);
            m.from = p.by_head ? m.sfrom
                               : (((a * 2) << p.c.page_shift) + (src & mask)) * p.c.Nk + hk;
            m.to = p.by_head ? m.sto : (((d * 2) << p.c.page_shift) + (r & mask)) * p.c.Nk + hk;
            m.from *= pieces;
            m.to *= pieces;
            s_any = 1;
          } else {
            report(p.c, HSTU_DEVERR_OFFSETS);
          }
        }
        moves[x] = m;
      }
      __syncthreads();
      if (chunks == 1) {
        n = s_end;
        if (tid == 0 && goes_on(n)) report(p.c, HSTU_DEVERR_OFFSETS);
      }
    }
    uint4 u[kPieces];
    uint16_t group[kPieces];
    uint8_t scale[2];
    float weight = 0.f;
    const bool mine = tid < n && moves[tid].from >= 0;
    const bool any = n > 0 && s_any;
    if (any) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int r = row0 + i * step;
        if (r < n && moves[r].from >= 0) {
          u[i] = cache[moves[r].from + off];
          if (factors) group[i] = factors[moves[r].from + off];
        }
      }
      if (mine) {
        if (p.c.scale) {
#pragma unroll
          for (int i = 0; i < 2; ++i) scale[i] = p.c.scale[moves[tid].sfrom + i * plane];
        }
        if (p.weights) weight = p.weights[weight_at(moves[tid].sfrom)];
      }
    }
    __syncthreads();  // every row of the chunk is in registers
    if (n > 0 && tid == 0 && chunks > 1) store_release(loaded + chunk, 1);
    if (!any) continue;
    if (tid < (s_front & 3)) {
      const int* flag = loaded + (s_front >> 2) + tid;
      if (!load_acquire(flag)) {
        const uint64_t start = ptx::globaltimer_ns();
        while (!load_acquire(flag)) {
          if ((long long)(ptx::globaltimer_ns() - start) > p.timeout_ns) {
            s_late = 1;
            report(p.c, HSTU_DEVERR_TIMEOUT);
            break;
          }
        }
      }
    }
    __syncthreads();
    if (s_late) continue;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int r = row0 + i * step;
      if (r < n && moves[r].from >= 0) {
        cache[moves[r].to + off] = u[i];
        if (factors) factors[moves[r].to + off] = group[i];
      }
    }
    if (mine) {
      if (p.c.scale) {
#pragma unroll
        for (int i = 0; i < 2; ++i) p.c.scale[moves[tid].sto + i * plane] = scale[i];
      }
      if (p.weights) p.weights[weight_at(moves[tid].sto)] = weight;
    }
  }
}

}  // namespace

namespace {
int lanes_shift(int row_bytes) {
  int s = 0;
  while ((1 << s) < 2 * (row_bytes / 16)) ++s;
  return s;
}
}  // namespace

int compact_rows(int row_bytes) {
  // as many rows of both planes as the registers hold
  const int rows = kThreads * kPieces >> lanes_shift(row_bytes);
  return rows < kCompactRows ? rows : kCompactRows;
}

cudaError_t launch_compact(const CompactParams& p, int chunks, int sms, cudaStream_t stream) {
  const long long tickets = (long long)p.c.B * p.c.Nk * chunks;
  const int rows = compact_rows(p.row_bytes);
  if (chunks > 1) {
    const size_t ints = 4 + (size_t)p.c.B * p.c.Nk + tickets;
    cudaError_t e = cudaMemsetAsync(p.counter, 0, sizeof(int) * ints, stream);
    if (e != cudaSuccess) return e;
    const long long warps = kThreads / 32;
    lists_kernel<<<(unsigned)((tickets + warps - 1) / warps), kThreads, 0, stream>>>(p, rows, chunks);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const long long most = (long long)kCtas * sms;
  compact_kernel<<<(unsigned)(tickets < most ? tickets : most), kThreads, 0, stream>>>(
      p, rows, chunks, lanes_shift(p.row_bytes));
  return cudaGetLastError();
}

}  // namespace hstu
