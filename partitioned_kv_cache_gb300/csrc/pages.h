// pages.h -- a paged cache of language streams as the kernels see it.
//
// Keys and values live in a pool of pages [n_pages][page][Hkv][D]; place j of
// stream b is row j % page of page table[b][j / page].  The new tokens of a
// step are packed: stream b's are [q_start[b], q_start[b+1]) of N.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "rx_internal.h"

namespace rx {

// Runs `set` (a function's attributes, which a device keeps) once for each device.
template <typename Set>
cudaError_t once_per_device(std::atomic<unsigned long long>& done, int dev, Set set) {
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  const cudaError_t e = set();
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

struct PagePool {
  void* k;
  void* v;
  float* weight;       // [n_pages][page][Hkv]; may be null
  const int* table;    // [B][max_pages]
  int n_pages;
  int log_page;        // page = 1 << log_page, 16 to 256
  int max_pages;
  int B;
};

// The row of the pool that place j of stream b names, or -1 where the table's
// entry is no page.
__device__ __forceinline__ long long pool_row(const PagePool& p, int b, int j) {
  const int pg = __ldg(p.table + static_cast<long long>(b) * p.max_pages + (j >> p.log_page));
  if (static_cast<unsigned int>(pg) >= static_cast<unsigned int>(p.n_pages)) return -1;
  return (static_cast<long long>(pg) << p.log_page) + (j & ((1 << p.log_page) - 1));
}

// What a stream's table can hold (2^30 keys at most), and a length clamped to it.
__host__ __device__ __forceinline__ int pool_capacity(const PagePool& p) {
  const long long c = static_cast<long long>(p.max_pages) << p.log_page;
  return c > (1 << 30) ? (1 << 30) : static_cast<int>(c);
}
__device__ __forceinline__ int held_keys(const PagePool& p, const int* len, int b) {
  return max(0, min(__ldg(len + b), pool_capacity(p)));
}

// Tensor-map encoding for bf16 with the 128-byte swizzle.
bool encode_tmap_5d(CUtensorMap* tm, const void* base, const uint64_t dims[5], const uint64_t strides_bytes[4],
                    const uint32_t box[5]);

// Copies by tensor map cost the copy engine some 3 cycles for each row of 128
// bytes and 100 to 200 each, so one copy takes all column blocks of a page's
// tokens.  In shared memory they lie as [8 tokens][D/64 column blocks][8 rows of
// 128 bytes, swizzled]: whatever the page's size, an operand of any number of
// tokens has one stride between groups of 8, D/64 KB.
inline bool encode_page_map(CUtensorMap* tm, const void* pool, const PagePool& p, int Hkv, int D, int most) {
  const uint64_t kb = D / 64, row = static_cast<uint64_t>(Hkv) * D * 2, page = 1ull << p.log_page;
  const uint64_t dims[5] = {64, 8, Hkv * kb, page / 8, static_cast<uint64_t>(p.n_pages)};
  const uint64_t strides[4] = {row, 128, 8 * row, page * row};
  const uint32_t tokens = static_cast<uint32_t>(page) < static_cast<uint32_t>(most) ? static_cast<uint32_t>(page) : static_cast<uint32_t>(most);
  const uint32_t box[5] = {64, 8, static_cast<uint32_t>(kb), tokens / 8, 1};
  return encode_tmap_5d(tm, pool, dims, strides, box);
}

// Query rows (token, head of the group) of packed tokens q [N][Hq][D]: a copy
// brings `rows` of them as [D/64 column blocks][rows][128 bytes, swizzled];
// coordinates (0, head within the group, token, first head of the group * D/64).
inline bool encode_query_map(CUtensorMap* tm, const void* q, int N, int Hq, int Hkv, int D, int rows) {
  const uint64_t kb = D / 64, G = Hq / Hkv;
  const uint64_t dims[4] = {64, G, static_cast<uint64_t>(N), Hq * kb};
  const uint64_t strides[3] = {static_cast<uint64_t>(D) * 2, static_cast<uint64_t>(Hq) * D * 2, 128};
  const uint32_t g = static_cast<uint32_t>(G < static_cast<uint64_t>(rows) ? G : rows);
  const uint32_t box[4] = {64, g, static_cast<uint32_t>(rows) / g, static_cast<uint32_t>(kb)};
  return encode_tmap_4d(tm, q, dims, strides, box);
}

constexpr int kMaxAxes = 4;

struct HeadRotation {
  const float* freq;       // [pairs]
  const float* q_weight;   // [D] or null: no norm
  const float* k_weight;
  int Hq, Hkv, D;
  int pairs;               // rotated pairs of a head, sum of the sections
  int axes;
  int section_end[kMaxAxes];   // pairs [section_end[a-1], section_end[a]) turn with axis a
  int adjacent;            // pair i: elements 2i, 2i+1; else i, i + pairs
  float eps;
};

// Dense keys and values (k, v) or, with them null, into `pool`.
cudaError_t launch_rotate_heads(const void* x, long long row_stride, int N, const HeadRotation& r, const int* pos,
                                void* q, void* k, void* v, const PagePool& pool, const int* q_start, const int* held,
                                int* new_len, int* overflow, cudaStream_t s);

cudaError_t launch_evict_pages(const PagePool& pool, int Hkv, int D, const int* len, int sink, int recent, int budget,
                               const int* to, int to_max_pages, int* new_len, int* kept, int* overflow,
                               cudaStream_t s);

// Attention of packed new tokens over the pages and, where `al` is not null,
// one layer of the shared store in front of them.
struct PageAttention {
  const void* q;          // bf16 [N][Hq][D]
  void* out;              // bf16 [N][Hq][D]
  float* lse;             // [N][Hq] or null
  const int* q_start;     // [B+1]
  const int* len;         // [B]
  const int* prefix;      // [B] or null
  int N, Hq, Hkv, D;
};
cudaError_t launch_attend_pages(const PageAttention& a, const PagePool& pool, const AttnLaunch* al, void* ws,
                                cudaStream_t s);
size_t attend_pages_workspace(int N, int Hq, int Hkv, int D, int num_sms);

// The weight that keys gather from packed new tokens.
struct PageWeights {
  const void* q;          // bf16 [N][Hq][D]
  const float* lse;       // [N][Hq]
  const int* q_start;
  const int* len;
  const int* prefix;
  float* out;             // [n_pages][page][Hkv], may be the pool's weight
  float decay;
  int N, Hq, Hkv, D;
};
size_t weigh_pages_workspace(int N, int G, int num_sms);
cudaError_t launch_weigh_pages(const PageWeights& a, const PagePool& pool, void* ws, cudaStream_t s);

constexpr int kMaxPagedStreams = 1024;   // of one call: their plans go through shared memory

}  // namespace rx
