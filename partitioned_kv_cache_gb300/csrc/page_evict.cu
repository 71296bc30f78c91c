// page_evict.cu -- eviction from a paged cache by accumulated attention weight.
//
// Of a stream that holds n > budget keys, each K/V head keeps the first `sink`,
// the last `recent`, and of those between them the budget - sink - recent with
// the largest weight (ties: the earlier key).  Kept keys keep their order and
// close up: new place i holds old place kept[i].
//
// Two launches.  select_kernel, one CTA per (stream, head), finds the weight of
// the last key that still fits by a radix search over the weights' ordered bit
// patterns, eight bits a pass, ended early where all keys with the digits found are
// kept, and writes kept[] in a second look at the keys, a warp's consecutive ones
// each: some 32 us for 512 heads of 3000 to 9000 keys (50 with one key of a thread
// asked for at a time, no early end and an ordered scan with a barrier for every 512
// keys; 512 threads: 256 and 1024 are slower).  The move is bound by memory:
// kept keys and values are read and written once.  64 streams of 8 heads cut to
// 4096 keys of 128: 322 us, 6.4 TB/s.  Into other pages all rows
// move at once (copy_kernel); within the same pages a CTA owns 64 bytes of every
// row of its head and takes rows in ascending order, reading a batch of rows
// before it writes one: new places never lie behind old ones, so what a later
// batch reads is not yet overwritten (close_up_kernel).  The call above in place, 1.76
// GB read and written: 610 us, one CTA's turn of reads and writes behind the other.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pages.h"
#include "rx_internal.h"
#include "sm103_ptx.cuh"

namespace rx {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
// Keys whose ordered weights a select CTA keeps in shared memory; beyond, it
// reads them from the pool again in each of its passes (four at most, and two to write kept[]).
constexpr int kSelHeld = 24576;

struct EvictParams {
  PagePool pool;
  int Hkv;
  const int* len;
  int sink, recent, budget;
  const int* to;          // table of the new places [B][to_max_pages]
  int to_max_pages;
  int* new_len;
  int* kept;              // [B][Hkv][budget]
  int* overflow;
};

// Orders like the weight; NaN and keys without a page come last.
__device__ __forceinline__ uint32_t ordered(float w) {
  if (!(w == w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);   // -0 is 0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t s_key[];   // [min(candidates, kSelHeld)]
  __shared__ unsigned int s_hist[256];
  __shared__ int s_pick[3];             // the digit found, how many keys remain to be found in it, and are in it
  __shared__ int s_warp[2][kSelWarps];
  const int b = blockIdx.x / p.Hkv, h = blockIdx.x - b * p.Hkv;
  grid_dependency_wait();
  grid_launch_dependents();
  const int n = held_keys(p.pool, p.len, b);
  int* kept = p.kept + static_cast<size_t>(blockIdx.x) * p.budget;
  if (n <= p.budget) {
    for (int i = threadIdx.x; i < p.budget; i += kSelThreads) kept[i] = i < n ? i : -1;
    return;
  }
  const int lo = p.sink, hi = n - p.recent, m = hi - lo;
  int want = p.budget - p.sink - p.recent;   // of the m between
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool held = m <= kSelHeld;
  auto read = [&](int i) {
    const long long row = pool_row(p.pool, b, lo + i);
    return row < 0 ? 0u : ordered(__ldg(p.pool.weight + row * p.Hkv + h));
  };
  if (held) {
    // Eight keys of a thread at a time: their table entries, then their weights.
    constexpr int kAhead = 8;
    for (int i0 = threadIdx.x; i0 < m; i0 += kSelThreads * kAhead) {
      long long row[kAhead];
      float w[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kSelThreads;
        row[u] = i < m ? pool_row(p.pool, b, lo + i) : -1;
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) w[u] = row[u] < 0 ? __uint_as_float(0x7FFFFFFFu) : __ldg(p.pool.weight + row[u] * p.Hkv + h);
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (i0 + u * kSelThreads < m) s_key[i0 + u * kSelThreads] = ordered(w[u]);
    }
  }
  // The want-th largest pattern, eight bits at a time from the top.
  uint32_t found = 0u;
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += kSelThreads) s_hist[i] = 0u;
      __syncthreads();
      for (int i0 = 0; i0 < m; i0 += kSelThreads) {
        const int i = i0 + threadIdx.x;
        const uint32_t key = i < m ? (held ? s_key[i] : read(i)) : 0u;
        const bool in = i < m && (shift == 24 || (key >> (shift + 8)) == (found >> (shift + 8)));
        const unsigned int digit = in ? (key >> shift) & 255u : 256u;
        if (__popc(__ballot_sync(0xffffffffu, in)) <= 8) {
          if (in) atomicAdd(&s_hist[digit], 1u);
        } else {   // lanes with the same digit add once
          const unsigned int same = __match_any_sync(0xffffffffu, digit);
          if (in && lane == __ffs(same) - 1) atomicAdd(&s_hist[digit], static_cast<unsigned int>(__popc(same)));
        }
      }
      __syncthreads();
      if (warp == 0) {   // lane l: digits 255 - 8 l down to 248 - 8 l
        unsigned int mine = 0u;
#pragma unroll
        for (int d = 0; d < 8; ++d) mine += s_hist[255 - 8 * lane - d];
        unsigned int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned int x = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += x;
        }
        unsigned int above = upto - mine;
        if (above < static_cast<unsigned int>(want) && upto >= static_cast<unsigned int>(want)) {
          for (int d = 0; d < 8; ++d) {
            const unsigned int c = s_hist[255 - 8 * lane - d];
            if (above + c >= static_cast<unsigned int>(want)) {
              s_pick[0] = 255 - 8 * lane - d;
              s_pick[1] = want - static_cast<int>(above);
              s_pick[2] = static_cast<int>(c);
              break;
            }
            above += c;
          }
        }
      }
      __syncthreads();
      found |= static_cast<uint32_t>(s_pick[0]) << shift;
      want = s_pick[1];
      if (want == s_pick[2]) break;   // all of them are kept: whatever is at or above `found`
    }
  }
  // Kept: above `found`, and the first `want` of those equal to it (or all of them).
  const bool any = p.budget > p.sink + p.recent;
  const bool all = any && want == s_pick[2];
  for (int i = threadIdx.x; i < p.sink; i += kSelThreads) kept[i] = i;
  for (int i = threadIdx.x; i < p.recent; i += kSelThreads) kept[p.budget - p.recent + i] = hi + i;
  if (!any) return;
  // A warp takes consecutive keys: it counts them, and with the counts of the warps
  // before it knows their places.
  const int per = (m + kSelThreads - 1) / kSelThreads * 32;
  const int w0 = warp * per, w1 = min(m, w0 + per);
  auto look = [&](int i, unsigned int* over, unsigned int* same) {
    const uint32_t key = i < w1 ? (held ? s_key[i] : read(i)) : 0u;
    *over = __ballot_sync(0xffffffffu, i < w1 && (all ? key >= found : key > found));
    *same = __ballot_sync(0xffffffffu, i < w1 && !all && key == found);
  };
  int n_over = 0, n_same = 0;
  unsigned int over, same;
#pragma unroll 4
  for (int i0 = w0; i0 < w1; i0 += 32) {
    look(i0 + lane, &over, &same);
    n_over += __popc(over);
    n_same += __popc(same);
  }
  if (lane == 0) {
    s_warp[0][warp] = n_over;
    s_warp[1][warp] = n_same;
  }
  __syncthreads();
  n_over = n_same = 0;
  for (int w = 0; w < warp; ++w) {
    n_over += s_warp[0][w];
    n_same += s_warp[1][w];
  }
  const unsigned int below = (1u << lane) - 1u;
#pragma unroll 4
  for (int i0 = w0; i0 < w1; i0 += 32) {
    look(i0 + lane, &over, &same);
    const int o = n_over + __popc(over & below), e = n_same + __popc(same & below);
    if ((over >> lane & 1) || ((same >> lane & 1) && e < want)) kept[p.sink + o + min(e, want)] = lo + i0 + lane;
    n_over += __popc(over);
    n_same += __popc(same);
  }
}

// The lengths are written by the move: the selection of every head has read
// them by then, so that new_len may be len.
__device__ __forceinline__ void write_len(const EvictParams& p, int b, int h) {
  if (p.new_len && h == 0 && blockIdx.y == 0 && threadIdx.x == 0) p.new_len[b] = min(held_keys(p.pool, p.len, b), p.budget);
}

__device__ __forceinline__ long long to_row(const EvictParams& p, int b, int i) {
  const int slot = i >> p.pool.log_page;
  if (slot >= p.to_max_pages) return -1;
  const int pg = __ldg(p.to + static_cast<long long>(b) * p.to_max_pages + slot);
  if (static_cast<unsigned int>(pg) >= static_cast<unsigned int>(p.pool.n_pages)) return -1;
  return (static_cast<long long>(pg) << p.pool.log_page) + (i & ((1 << p.pool.log_page) - 1));
}

// D/8 lanes move a row of K and of V; a thread has two rows of each in flight (64
// streams of 8 heads cut to 4096 keys: a call took 362 us so, 368 with four).
// Rows: blockIdx.x over (stream, head), blockIdx.y over places.
constexpr int kCopyThreads = 256;
constexpr int kCopyRows = 2;

template <int D>
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ EvictParams p) {
  constexpr int L = D / 8, kRows = kCopyThreads / L * kCopyRows;
  const int b = blockIdx.x / p.Hkv, h = blockIdx.x - b * p.Hkv;
  grid_dependency_wait();
  grid_launch_dependents();
  write_len(p, b, h);
  const int sub = threadIdx.x % L;
  const int* kept = p.kept + static_cast<size_t>(blockIdx.x) * p.budget;
  const uint4* ks = static_cast<const uint4*>(p.pool.k);
  const uint4* vs = static_cast<const uint4*>(p.pool.v);
  for (int r0 = blockIdx.y * kRows; r0 < p.budget; r0 += gridDim.y * kRows) {
    if (__ldg(kept + r0) < 0) break;   // behind the last kept key
    long long src[kCopyRows], dst[kCopyRows];
    uint4 kx[kCopyRows], vx[kCopyRows];
    float w[kCopyRows];
#pragma unroll
    for (int u = 0; u < kCopyRows; ++u) {
      const int i = r0 + u * (kCopyThreads / L) + static_cast<int>(threadIdx.x) / L;
      src[u] = i < p.budget ? __ldg(kept + i) : -1;
      dst[u] = src[u] >= 0 ? to_row(p, b, i) : -1;
    }
#pragma unroll
    for (int u = 0; u < kCopyRows; ++u) {
      const bool asked = src[u] >= 0;
      if (asked) src[u] = pool_row(p.pool, b, static_cast<int>(src[u]));
      if (asked && (src[u] < 0 || dst[u] < 0) && sub == 0 && p.overflow) atomicOr(p.overflow, 1);
      if (src[u] < 0) dst[u] = -1;
    }
#pragma unroll
    for (int u = 0; u < kCopyRows; ++u) {
      if (dst[u] < 0) continue;
      const size_t row = static_cast<size_t>(src[u]) * p.Hkv + h;
      kx[u] = __ldg(ks + row * L + sub);
      vx[u] = __ldg(vs + row * L + sub);
      w[u] = __ldg(p.pool.weight + row);
    }
#pragma unroll
    for (int u = 0; u < kCopyRows; ++u) {
      if (dst[u] < 0) continue;
      const size_t row = static_cast<size_t>(dst[u]) * p.Hkv + h;
      static_cast<uint4*>(p.pool.k)[row * L + sub] = kx[u];
      static_cast<uint4*>(p.pool.v)[row * L + sub] = vx[u];
      if (sub == 0) p.pool.weight[row] = w[u];
    }
  }
}

// Within the same pages.  blockIdx.y: 64-byte column pieces of K, then of V,
// then the weights.  Four lanes hold a piece of a row; kCloseRows rows of a
// lane are read before any of the batch is written, and the next batch's reads
// are issued before this one's writes.
constexpr int kCloseThreads = 256;
constexpr int kCloseRows = 4;

template <int D>
__global__ void __launch_bounds__(kCloseThreads) close_up_kernel(const __grid_constant__ EvictParams p) {
  constexpr int kPieces = D / 32;                      // 64-byte pieces of a row
  constexpr int kBatch = kCloseThreads / 4 * kCloseRows;
  const int b = blockIdx.x / p.Hkv, h = blockIdx.x - b * p.Hkv;
  grid_dependency_wait();
  grid_launch_dependents();
  write_len(p, b, h);
  const int* kept = p.kept + static_cast<size_t>(blockIdx.x) * p.budget;
  const int piece = blockIdx.y;
  const bool weights = piece == 2 * kPieces;
  if (weights && p.overflow) {
    // Keys that stay are the first ones, so a page that holds any begins with one.
    const int slots = ((p.budget - 1) >> p.pool.log_page) + 1;
    for (int slot = threadIdx.x; slot < slots; slot += kCloseThreads) {
      const int i = slot << p.pool.log_page;
      if (__ldcg(kept + i) == i && pool_row(p.pool, b, i) < 0) atomicOr(p.overflow, 1);
    }
  }
  if (kept[p.budget - 1] <= p.budget - 1) return;      // nothing was dropped (or the stream is shorter: -1)
  uint4* base = static_cast<uint4*>(piece < kPieces ? p.pool.k : p.pool.v) + (piece % kPieces) * 4 + (threadIdx.x & 3);
  uint4 x[2][kCloseRows];
  long long dst[2][kCloseRows];
  auto read = [&](int buf, int r0) {
#pragma unroll
    for (int u = 0; u < kCloseRows; ++u) {
      const int i = r0 + u * (kCloseThreads / 4) + static_cast<int>(threadIdx.x >> 2);
      dst[buf][u] = -1;
      const int j = i < p.budget ? __ldcg(kept + i) : i;
      if (j == i) continue;                            // stays where it is
      const long long src = pool_row(p.pool, b, j);
      dst[buf][u] = pool_row(p.pool, b, i);
      if (src < 0 || dst[buf][u] < 0) {
        dst[buf][u] = -1;
        if (weights && (threadIdx.x & 3) == 0 && p.overflow) atomicOr(p.overflow, 1);
        continue;
      }
      if (weights) x[buf][u].x = __float_as_uint(__ldcg(p.pool.weight + src * p.Hkv + h));
      else x[buf][u] = __ldcg(base + (src * p.Hkv + h) * (D / 8));
    }
  };
  auto write = [&](int buf) {
#pragma unroll
    for (int u = 0; u < kCloseRows; ++u) {
      if (dst[buf][u] < 0) continue;
      if (!weights) base[(dst[buf][u] * p.Hkv + h) * (D / 8)] = x[buf][u];
      else if ((threadIdx.x & 3) == 0) p.pool.weight[dst[buf][u] * p.Hkv + h] = __uint_as_float(x[buf][u].x);
    }
  };
  read(0, 0);
  for (int r0 = 0; r0 < p.budget; r0 += 2 * kBatch) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int at = r0 + half * kBatch;
      if (at >= p.budget) break;
      read(half ^ 1, at + kBatch);                     // (past the budget: nothing)
      __syncthreads();                                 // all reads of this batch and the next are done
      write(half);
    }
  }
}

template <int D>
cudaError_t launch_d(const EvictParams& p, bool in_place, cudaStream_t s) {
  const int units = p.pool.B * p.Hkv;
  if (in_place) {
    const cudaError_t e = launch_k(close_up_kernel<D>, dim3(units, 2 * (D / 32) + 1), dim3(kCloseThreads), 0, s, p);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  constexpr int kRows = kCopyThreads / (D / 8) * kCopyRows;
  const int most = (p.budget + kRows - 1) / kRows;
  const cudaError_t e = launch_k(copy_kernel<D>, dim3(units, most < 65535 ? most : 65535), dim3(kCopyThreads), 0, s, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict_pages(const PagePool& pool, int Hkv, int D, const int* len, int sink, int recent, int budget,
                               const int* to, int to_max_pages, int* new_len, int* kept, int* overflow,
                               cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  EvictParams p{};
  p.pool = pool;
  p.Hkv = Hkv;
  p.len = len;
  p.sink = sink;
  p.recent = recent;
  p.budget = budget;
  p.to = to ? to : pool.table;
  p.to_max_pages = to ? to_max_pages : pool.max_pages;
  p.new_len = new_len;
  p.kept = kept;
  p.overflow = overflow;
  const int cap = pool_capacity(pool) - sink - recent;   // most candidates
  const int held = cap < 1 ? 1 : cap < kSelHeld ? cap : kSelHeld;
  static std::atomic<unsigned long long> ready{0};
  e = once_per_device(ready, dev, [] {
    return cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelHeld * 4);
  });
  if (e != cudaSuccess) return e;
  e = launch_k(select_kernel, dim3(pool.B * Hkv), dim3(kSelThreads), static_cast<size_t>(held) * 4, s, p);
  if (e != cudaSuccess) return e;
  switch (D) {
    case 64: return launch_d<64>(p, !to, s);
    case 128: return launch_d<128>(p, !to, s);
    case 256: return launch_d<256>(p, !to, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace rx
