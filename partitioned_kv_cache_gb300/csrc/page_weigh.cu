// page_weigh.cu -- the attention weight that the keys of a paged cache gather
// from a step's new tokens (sm_103a).
//
//   out[j][h] = decay * weight[j][h] + sum over the stream's new tokens t that
//               see place j, and the query heads of group h, of exp(s - lse)
// with s = q . k_j / sqrt(D) and lse the attention's own, so that what the
// shared store took is not counted here.
//
// The keys are the M side: scores^T = K Q^T puts one key on each softmax thread,
// whose sum over the rows (the columns of its lane) needs no exchange and no
// atomics: the same inputs give the same bits.  A unit is (stream, K/V head, 128
// keys); it reads its keys once and all row tiles (64 rows: tokens x heads of the
// group) that see one of them.  CTAs take units in turn, grid apart, since later
// keys are seen by fewer rows.  One token per stream is bound by the keys' bytes;
// a chunk by Q K^T (both operands from shared memory) and, at D = 64, by the
// exponentials.
//
// Warps (224 threads): 0 = copies (lane 0 keys, lane 1 queries), 1 = tensor
// memory and K Q^T, 2..5 = exponentials and sums, 6 = the rows' lse.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "pages.h"
#include "rx_internal.h"
#include "sm103_ptx.cuh"

namespace rx {
namespace {

constexpr int kThreads = 224;
constexpr int kKeys = 128;   // of a unit
constexpr int kRows = 64;    // of a row tile
constexpr int kBufs = 4;     // score tiles in tensor memory

template <int D>
struct Layout {
  static constexpr int KB = D / 64;
  static constexpr int CTAS = D == 256 ? 1 : 2;
  static constexpr int K_BLOCK = kKeys * 128, Q_BLOCK = kRows * 128;
  static constexpr int K_TILE = KB * K_BLOCK, Q_TILE = KB * Q_BLOCK;
  static constexpr int NK = D == 64 ? 3 : 2, NQ = D == 64 ? 4 : 2;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_Q = NK * K_TILE;
  static constexpr int OFF_BAR = OFF_Q + NQ * Q_TILE;
  static constexpr int OFF_LSE = OFF_BAR + 32 * 8;              // [4][64] floats
  static constexpr int OFF_MISC = OFF_LSE + 4 * kRows * 4;
  static constexpr int OFF_BEFORE = OFF_MISC + 32;              // long long [B + 1]
  static constexpr int BYTES = OFF_BEFORE;
  static_assert(CTAS * (BYTES + 1024 + 1024 + (kMaxPagedStreams + 1) * 8) <= 233472, "shared memory");
};

// Barriers: K full / empty [3], Q full / empty [4], scores full / empty [4],
// lse full / empty [4], drained.
enum : int { B_KF = 0, B_KE = 3, B_QF = 6, B_QE = 10, B_SF = 14, B_SE = 18, B_LF = 22, B_LE = 26, B_DRAIN = 30 };

struct WeighParams {
  CUtensorMap tm_k;   // (D, Hkv, page, n_pages), box (64, 1, min(page, 128), 1)
  CUtensorMap tm_q;   // (D, G, Hkv, N), box (64, min(G, 64), 1, max(1, 64 / G))
  PagePool pool;
  const float* lse;
  const int* q_start;
  const int* len;
  const int* prefix;
  float* out;
  int N, Hq, Hkv, log_g;
  float decay;
  float scale_log2;
};

// One unit: keys [k0, k0 + 128) of a stream, row tiles [r0, r1).
struct Unit {
  int b, h, k0, q0, n, len, prefix, x0, r0, r1;
};

__device__ __forceinline__ int new_tokens(const WeighParams& p, int b, int* q0) {
  *q0 = max(0, min(__ldg(p.q_start + b), p.N));
  return max(0, max(0, min(__ldg(p.q_start + b + 1), p.N)) - *q0);
}

__device__ __forceinline__ Unit unit_at(const WeighParams& p, const long long* before, long long u) {
  int lo = 0, hi = p.pool.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (before[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  Unit x;
  x.b = lo;
  x.n = new_tokens(p, lo, &x.q0);
  x.len = held_keys(p.pool, p.len, lo);
  x.prefix = p.prefix ? max(0, min(__ldg(p.prefix + lo), x.len)) : 0;
  const int blocks = (x.len + kKeys - 1) / kKeys;
  const long long o = u - before[lo];
  x.h = static_cast<int>(o / blocks);
  x.k0 = static_cast<int>(o - static_cast<long long>(x.h) * blocks) * kKeys;
  x.x0 = x.len - x.n;
  const int first = x.k0 < x.prefix ? 0 : max(0, x.k0 - x.x0);   // first token that sees one of the keys
  x.r0 = (first << p.log_g) / kRows;
  x.r1 = ((x.n << p.log_g) + kRows - 1) / kRows;
  return x;
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  const bool ok = mbar_wait(bar, parity, abort);
  return __all_sync(0xffffffffu, ok);
}

// A ring position: slot and how often the ring has gone round.
struct Turn {
  int slot = 0, round = 0;
  __device__ __forceinline__ void step(int n) {
    if (++slot == n) {
      slot = 0;
      ++round;
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, Layout<D>::CTAS) page_weigh_kernel(const __grid_constant__ WeighParams p) {
  using Lay = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sK = base + Lay::OFF_K, sQ = base + Lay::OFF_Q, sBar = base + Lay::OFF_BAR;
  float* s_lse = reinterpret_cast<float*>(gbase + Lay::OFF_LSE);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + Lay::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + Lay::OFF_MISC + 4);
  long long* before = reinterpret_cast<long long*>(gbase + Lay::OFF_BEFORE);
  auto BAR = [&](int i) { return sBar + 8u * static_cast<uint32_t>(i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 31; ++i) {
      const int count = (i >= B_SE && i < B_SE + 4) || (i >= B_LE && i < B_LE + 4) ? 128 : i >= B_LF && i < B_LF + 4 ? 32 : 1;
      mbar_init(BAR(i), count);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kBufs * kRows);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();
  grid_launch_dependents();
  for (int b = threadIdx.x; b < p.pool.B; b += kThreads) {
    int q0;
    const int n = new_tokens(p, b, &q0);   // streams without new tokens have no work
    before[b + 1] = n > 0 ? static_cast<long long>(p.Hkv) * ((held_keys(p.pool, p.len, b) + kKeys - 1) / kKeys) : 0;
  }
  __syncthreads();
  if (warp == 0) {
    long long sum = 0;
    for (int b0 = 0; b0 < p.pool.B; b0 += 32) {
      long long x = b0 + lane < p.pool.B ? before[b0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b0 + lane < p.pool.B) before[b0 + lane + 1] = sum + x;
      sum += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) before[0] = 0;
  }
  __syncthreads();
  const long long units = before[p.pool.B];
  const uint32_t tmem = *tmem_slot;
  const int lp = p.pool.log_page;
  const int box = lp < 7 ? 1 << lp : kKeys;
  const bool some = static_cast<long long>(blockIdx.x) < units;

  if (some && warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------- keys
      Turn at;
      int issued = 0;
      for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const Unit x = unit_at(p, before, u);
        const int* table = p.pool.table + static_cast<long long>(x.b) * p.pool.max_pages;
        int pg[8];
        uint32_t named = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int place = x.k0 + i * box;
          pg[i] = i * box < kKeys && place < x.len ? __ldg(table + (place >> lp)) : -1;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) named += static_cast<unsigned int>(pg[i]) < static_cast<unsigned int>(p.pool.n_pages);
        if (at.round > 0 && !mbar_wait(BAR(B_KE + at.slot), (at.round - 1) & 1, abort_flag)) break;
        const uint32_t bar = BAR(B_KF + at.slot);
        mbar_arrive_expect_tx(bar, named * box * (D * 2));
        const int row = lp > 7 ? x.k0 & ((1 << lp) - 1) : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (static_cast<unsigned int>(pg[i]) >= static_cast<unsigned int>(p.pool.n_pages)) continue;
          for (int kb = 0; kb < Lay::KB; ++kb)
            tma_load_4d(sK + at.slot * Lay::K_TILE + kb * Lay::K_BLOCK + i * box * 128, &p.tm_k, kb * 64, x.h, row, pg[i], bar);
        }
        ++issued;
        at.step(Lay::NK);
      }
      volatile int no_abort = 0;
      for (int i = max(0, issued - Lay::NK); i < issued; ++i) mbar_wait(BAR(B_KF + i % Lay::NK), (i / Lay::NK) & 1, &no_abort);
    } else if (lane == 1) {
      // ---------------------------------------------------------- queries
      Turn at;
      int issued = 0;
      bool ok = true;
      for (long long u = blockIdx.x; ok && u < units; u += gridDim.x) {
        const Unit x = unit_at(p, before, u);
        for (int r = x.r0; r < x.r1; ++r) {
          if (at.round > 0 && !mbar_wait(BAR(B_QE + at.slot), (at.round - 1) & 1, abort_flag)) { ok = false; break; }
          const uint32_t bar = BAR(B_QF + at.slot);
          mbar_arrive_expect_tx(bar, Lay::Q_TILE);
          const int row = r * kRows;
          for (int kb = 0; kb < Lay::KB; ++kb)
            tma_load_4d(sQ + at.slot * Lay::Q_TILE + kb * Lay::Q_BLOCK, &p.tm_q, kb * 64, row & ((1 << p.log_g) - 1), x.h,
                        x.q0 + (row >> p.log_g), bar);
          ++issued;
          at.step(Lay::NQ);
        }
      }
      volatile int no_abort = 0;
      for (int i = max(0, issued - Lay::NQ); i < issued; ++i) mbar_wait(BAR(B_QF + i % Lay::NQ), (i / Lay::NQ) & 1, &no_abort);
    }
  } else if (some && warp == 1) {
    // ------------------------------------------------------------ K Q^T
    if (lane == 0) {
      constexpr uint32_t kIdesc = idesc_bf16_f32(kKeys, kRows, false, false);
      Turn k, q, s;
      bool ok = true;
      for (long long u = blockIdx.x; ok && u < units; u += gridDim.x) {
        const Unit x = unit_at(p, before, u);
        if (!mbar_wait(BAR(B_KF + k.slot), k.round & 1, abort_flag)) break;
        for (int r = x.r0; r < x.r1; ++r) {
          if (!mbar_wait(BAR(B_QF + q.slot), q.round & 1, abort_flag) ||
              (s.round > 0 && !mbar_wait(BAR(B_SE + s.slot), (s.round - 1) & 1, abort_flag))) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t kb = kk >> 2, ko = (kk & 3) * 32;
            umma_bf16(tmem + s.slot * kRows, sdesc_sw128(sK + k.slot * Lay::K_TILE + kb * Lay::K_BLOCK + ko, 16, 1024),
                      sdesc_sw128(sQ + q.slot * Lay::Q_TILE + kb * Lay::Q_BLOCK + ko, 16, 1024), kIdesc, kk > 0 ? 1u : 0u);
          }
          umma_commit(BAR(B_QE + q.slot));
          umma_commit(BAR(B_SF + s.slot));
          q.step(Lay::NQ);
          s.step(kBufs);
        }
        if (ok) umma_commit(BAR(B_KE + k.slot));
        k.step(Lay::NK);
      }
      umma_commit(BAR(B_DRAIN));
      volatile int no_abort = 0;
      mbar_wait(BAR(B_DRAIN), 0, &no_abort);
    }
  } else if (some && warp == 6) {
    // ------------------------------------------------------------ lse, in log2 units
    Turn at;
    bool ok = true;
    for (long long u = blockIdx.x; ok && u < units; u += gridDim.x) {
      const Unit x = unit_at(p, before, u);
      const int rows = x.n << p.log_g, gm = (1 << p.log_g) - 1;
      for (int r = x.r0; r < x.r1; ++r) {
        if (at.round > 0 && !warp_wait(BAR(B_LE + at.slot), (at.round - 1) & 1, abort_flag)) { ok = false; break; }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = r * kRows + i * 32 + lane;
          float v = INFINITY;   // rows behind the stream's, and rows that saw nothing, weigh nothing
          if (row < rows) {
            v = __ldg(p.lse + static_cast<size_t>(x.q0 + (row >> p.log_g)) * p.Hq + (x.h << p.log_g) + (row & gm));
            if (v == -INFINITY) v = INFINITY;
          }
          s_lse[at.slot * kRows + i * 32 + lane] = v * 1.44269504088896341f;
        }
        mbar_arrive(BAR(B_LF + at.slot));
        at.step(4);
      }
    }
  } else if (some) {
    // ------------------------------------------------------------ exponentials
    const int quarter = warp & 3, key = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    Turn at;   // of score and lse tiles, four of each
    bool ok = true;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
      const Unit x = unit_at(p, before, u);
      const int j = x.k0 + key;
      const long long row = j < x.len ? pool_row(p.pool, x.b, j) : -1;
      // First row that sees the key.
      const int first = j < x.prefix ? 0 : max(0, j - x.x0) << p.log_g;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      for (int r = x.r0; ok && r < x.r1; ++r) {
        if (!warp_wait(BAR(B_SF + at.slot), at.round & 1, abort_flag) ||
            !warp_wait(BAR(B_LF + at.slot), at.round & 1, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float s[kRows];
        tmem_ld64(tmem + at.slot * kRows + lane_off, s);
        tc_fence_before();
        mbar_arrive(BAR(B_SE + at.slot));
        const int hidden = first - r * kRows;   // leading rows of the tile that do not see the key
        if (__any_sync(0xffffffffu, hidden > 0)) {
#pragma unroll
          for (int c = 0; c < kRows; ++c)
            if (c < hidden) s[c] = -INFINITY;
        }
        const float4* lse = reinterpret_cast<const float4*>(s_lse + at.slot * kRows);
#pragma unroll
        for (int c = 0; c < kRows / 4; ++c) {
          const float4 e = lse[c];
          sum[0] += exp2f(fmaf(s[4 * c], p.scale_log2, -e.x));
          sum[1] += exp2f(fmaf(s[4 * c + 1], p.scale_log2, -e.y));
          sum[2] += exp2f(fmaf(s[4 * c + 2], p.scale_log2, -e.z));
          sum[3] += exp2f(fmaf(s[4 * c + 3], p.scale_log2, -e.w));
        }
        mbar_arrive(BAR(B_LE + at.slot));
        at.step(4);
      }
      if (row >= 0) {
        const size_t i = static_cast<size_t>(row) * p.Hkv + x.h;
        float got = (sum[0] + sum[1]) + (sum[2] + sum[3]);
        if (!ok) got = NAN;   // a wait gave up
        p.out[i] = p.decay == 0.f ? got : fmaf(p.decay, p.pool.weight[i], got);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kBufs * kRows);
}

template <int D>
cudaError_t launch_d(const WeighParams& p, int dev, int sms, cudaStream_t s) {
  using Lay = Layout<D>;
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = once_per_device(ready, dev, [] {
    return cudaFuncSetAttribute(page_weigh_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Lay::BYTES + 1024 + (kMaxPagedStreams + 1) * 8);
  });
  if (e != cudaSuccess) return e;
  e = launch_k(page_weigh_kernel<D>, dim3(sms * Lay::CTAS), dim3(kThreads), Lay::BYTES + 1024 + (p.pool.B + 1) * 8, s, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_weigh_pages(const PageWeights& a, const PagePool& pool, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = device_sm_count(dev, &sms);
  if (e != cudaSuccess) return e;
  const int G = a.Hq / a.Hkv, D = a.D, page = 1 << pool.log_page;
  WeighParams p;
  std::memset(&p, 0, sizeof(p));
  const uint64_t u = 2, dims[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(G), static_cast<uint64_t>(a.Hkv), static_cast<uint64_t>(a.N)};
  const uint64_t strides[3] = {D * u, D * u * G, D * u * a.Hq};
  const uint32_t box[4] = {64, static_cast<uint32_t>(G < kRows ? G : kRows), 1, static_cast<uint32_t>(G < kRows ? kRows / G : 1)};
  const uint64_t pd[4] = {static_cast<uint64_t>(D), static_cast<uint64_t>(a.Hkv), static_cast<uint64_t>(page), static_cast<uint64_t>(pool.n_pages)};
  const uint64_t ps[3] = {D * u, D * u * a.Hkv, D * u * a.Hkv * page};
  const uint32_t pb[4] = {64, 1, static_cast<uint32_t>(page < kKeys ? page : kKeys), 1};
  if (!encode_tmap_4d(&p.tm_q, a.q, dims, strides, box) || !encode_tmap_4d(&p.tm_k, pool.k, pd, ps, pb))
    return cudaErrorInvalidValue;
  p.pool = pool;
  p.lse = a.lse;
  p.q_start = a.q_start;
  p.len = a.len;
  p.prefix = a.prefix;
  p.out = a.out;
  p.N = a.N;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  while ((1 << p.log_g) < G) ++p.log_g;
  p.decay = a.decay;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D)));
  switch (D) {
    case 64: return launch_d<64>(p, dev, sms, s);
    case 128: return launch_d<128>(p, dev, sms, s);
    case 256: return launch_d<256>(p, dev, sms, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace rx
