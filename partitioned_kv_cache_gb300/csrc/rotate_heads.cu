// rotate_heads.cu -- what turns a layer's projection into the queries, keys and
// values that the attention entry points take: RMS norm of each query and key
// head, rotation by the token's position, and the keys' and values' way into
// dense buffers or into a stream's pages, in one pass.
//
// For one head x of D values with weight w (optional):
//   y_i = x_i * rsqrt(mean(x^2) + eps) * w_i
// and for every pair (a, b) = (y_i, y_{i+R/2}) (or (y_{2i}, y_{2i+1})), i < R/2,
// with the angle t = pos[axis(i)] * freq[i]:
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t).
// Values are copied.
//
// Angles.  pos * freq loses the whole angle in fp32 once it is large (half a
// unit in the last place of 10^6 is 0.03 rad).  Here freq / (2 pi) is a 64-bit
// fraction of a turn, so pos times it modulo 2^64 is the angle modulo one turn
// with no rounding but the fraction's own: 2^-53 of freq / (2 pi) times |pos|,
// below 10^-7 rad over all 32-bit positions at freq 1.  Its upper 32 bits feed
// sincospi.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pages.h"
#include "rx_internal.h"
#include "sm103_ptx.cuh"

namespace rx {
namespace {

constexpr int kThreads = 256;

struct RotateParams {
  const uint4* x;
  long long row_vecs;     // 16-byte vectors from one token's row to the next
  int N;
  HeadRotation r;
  const int* pos;         // [axes][N]
  uint4* q;               // [N][Hq][D]
  uint4* k;               // [N][Hkv][D], or null: into the pool
  uint4* v;
  PagePool pool;
  const int* q_start;
  const int* held;
  int* new_len;
  int* overflow;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// freq / (2 pi) as a fraction of 2^64, whole turns dropped.
__device__ __forceinline__ unsigned long long turn_fraction(float freq) {
  const double t = static_cast<double>(freq) * 0.15915494309189533577;
  return static_cast<unsigned long long>((t - floor(t)) * 18446744073709551616.0);
}

// A CTA takes TB tokens at a time.  D/8 lanes hold a head, eight values each;
// their cosines and sines are computed once per token into shared memory and
// serve all its heads.  Up to kFlight heads of a lane group are loaded before
// the first is worked on.
template <int D, int TB>
__global__ void __launch_bounds__(kThreads) rotate_heads_kernel(const __grid_constant__ RotateParams p) {
  constexpr int L = D / 8;
  constexpr int kGroups = kThreads / L;
  constexpr int kFlight = 4;
  __shared__ float2 s_turn[TB * (D / 2)];            // (cos, sin) of every pair
  __shared__ unsigned long long s_freq[D / 2];
  __shared__ float s_w[2][D];
  __shared__ int s_stream[TB];
  __shared__ long long s_row[TB];                    // pool row of the token's key and value, -1: dropped
  const int Hq = p.r.Hq, Hkv = p.r.Hkv, H = Hq + 2 * Hkv, pairs = p.r.pairs;
  const bool paged = p.k == nullptr;
  grid_dependency_wait();
  grid_launch_dependents();
  for (int i = threadIdx.x; i < pairs; i += kThreads) s_freq[i] = turn_fraction(p.r.freq[i]);
  for (int i = threadIdx.x; i < D; i += kThreads) {
    if (p.r.q_weight) s_w[0][i] = p.r.q_weight[i];
    if (p.r.k_weight) s_w[1][i] = p.r.k_weight[i];
  }
  if (paged && p.new_len) {
    for (int b = blockIdx.x * kThreads + threadIdx.x; b < p.pool.B; b += gridDim.x * kThreads) {
      const int s0 = max(0, min(p.q_start[b], p.N)), s1 = max(0, min(p.q_start[b + 1], p.N));
      const int len = p.held[b], cap = pool_capacity(p.pool);
      p.new_len[b] = len < 0 || len > cap ? len : len + min(max(0, s1 - s0), cap - len);
    }
  }
  const int sub = threadIdx.x % L, group = threadIdx.x / L;
  // Half pairs: the lane that holds the other halves of this lane's pairs.
  const int hl = pairs / 8;                                    // lanes that hold first halves
  const int lane = threadIdx.x & 31;
  const int other = (lane - sub) + (sub < hl ? sub + hl : sub < 2 * hl ? sub - hl : sub);
  const bool turned = p.r.adjacent ? sub * 8 < 2 * pairs : sub < 2 * hl;
  for (int n0 = blockIdx.x * TB; n0 < p.N; n0 += gridDim.x * TB) {
    __syncthreads();                                           // the last tokens' shared values are done with
    if (threadIdx.x < TB) s_stream[threadIdx.x] = paged ? -1 : 0;
    __syncthreads();
    if (paged) {
      for (int b = threadIdx.x; b < p.pool.B; b += kThreads) {
        const int s0 = p.q_start[b], s1 = p.q_start[b + 1];
#pragma unroll
        for (int t = 0; t < TB; ++t)
          if (n0 + t >= s0 && n0 + t < s1) s_stream[t] = b;
      }
    }
    for (int i = threadIdx.x; i < TB * pairs; i += kThreads) {
      const int t = i / pairs, c = i - t * pairs;
      if (n0 + t >= p.N) break;
      int axis = 0;
#pragma unroll
      for (int a = 0; a < kMaxAxes - 1; ++a) axis += a < p.r.axes - 1 && c >= p.r.section_end[a];
      const long long at = __ldg(p.pos + static_cast<size_t>(axis) * p.N + n0 + t);
      const int turn = static_cast<int>((static_cast<unsigned long long>(at) * s_freq[c]) >> 32);
      float sn, cs;
      sincospif(static_cast<float>(turn) * 4.656612873077392578125e-10f, &sn, &cs);   // 2^-31: half turns
      s_turn[t * (D / 2) + c] = make_float2(cs, sn);
    }
    __syncthreads();
    if (paged && threadIdx.x < TB) {
      const int t = threadIdx.x, b = s_stream[t];
      long long row = -1;
      if (b >= 0) {
        const int len = p.held[b], cap = pool_capacity(p.pool);
        const long long place = static_cast<long long>(len) + (n0 + t - p.q_start[b]);
        if (len >= 0 && len <= cap && place < cap) row = pool_row(p.pool, b, static_cast<int>(place));
        if (row < 0 && p.overflow) atomicOr(p.overflow, 1);
      }
      s_row[t] = row;
    }
    __syncthreads();
    const int vectors = min(TB, p.N - n0) * H;
    for (int base = 0; base < vectors; base += kGroups * kFlight) {   // the same turns for every lane
      const int v0 = base + group;
      uint4 raw[kFlight];
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const int i = v0 + f * kGroups;
        raw[f] = make_uint4(0u, 0u, 0u, 0u);
        if (i < vectors) {
          const int t = i / H;
          raw[f] = __ldg(p.x + static_cast<size_t>(n0 + t) * p.row_vecs + static_cast<size_t>(i - t * H) * L + sub);
        }
      }
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        if (base + f * kGroups >= vectors) break;              // the same for the whole CTA
        const int i = v0 + f * kGroups;
        const int t = min(i, vectors - 1) / H, h = i - t * H;
        const bool isq = h < Hq, isk = !isq && h < Hq + Hkv;
        uint32_t w[4] = {raw[f].x, raw[f].y, raw[f].z, raw[f].w};
        float y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[2 * e] = __uint_as_float(w[e] << 16);
          y[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
        const float* weight = isq ? p.r.q_weight : isk ? p.r.k_weight : nullptr;
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (weight) {
          const float r = rsqrtf(ss * (1.f / D) + p.r.eps);
          const float* ws = s_w[isq ? 0 : 1] + sub * 8;
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = y[e] * r * ws[e];
        }
        float z[8];
        if (p.r.adjacent) {
          const float2* cs = s_turn + t * (D / 2) + min(sub * 4, max(pairs - 4, 0));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 c = cs[e];
            z[2 * e] = y[2 * e] * c.x - y[2 * e + 1] * c.y;
            z[2 * e + 1] = y[2 * e + 1] * c.x + y[2 * e] * c.y;
          }
        } else {
          const float2* cs = s_turn + t * (D / 2) + (sub < hl ? sub : turned ? sub - hl : 0) * 8;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float o = __shfl_sync(0xffffffffu, y[e], other);
            const float2 c = cs[e];
            z[e] = y[e] * c.x + (sub < hl ? -o : o) * c.y;
          }
        }
        if (i >= vectors) continue;
        if (isq || isk) {
          if (turned) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = z[e];
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = pack2(y[2 * e], y[2 * e + 1]);
        }
        const uint4 done = make_uint4(w[0], w[1], w[2], w[3]);
        const size_t n = n0 + t;
        const int kv = isq ? 0 : isk ? h - Hq : h - Hq - Hkv;
        if (isq) {
          if (!paged || s_stream[t] >= 0) p.q[(n * Hq + h) * L + sub] = done;
        } else if (!paged) {
          (isk ? p.k : p.v)[(n * Hkv + kv) * L + sub] = done;
        } else if (s_row[t] >= 0) {
          const size_t row = static_cast<size_t>(s_row[t]) * Hkv + kv;
          static_cast<uint4*>(isk ? p.pool.k : p.pool.v)[row * L + sub] = done;
          if (isk && sub == 0 && p.pool.weight) p.pool.weight[row] = 0.f;
        }
      }
    }
  }
}

template <int D, int TB>
cudaError_t launch_tb(const RotateParams& p, int sms, cudaStream_t s) {
  const int blocks = p.N > 0 ? (p.N + TB - 1) / TB : 1;   // (without tokens: the lengths)
  const int most = sms * 8;
  const cudaError_t e = launch_k(rotate_heads_kernel<D, TB>, dim3(blocks < most ? blocks : most), dim3(kThreads), 0, s, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const RotateParams& p, int sms, cudaStream_t s) {
  // One token a CTA while the GPU holds them all at once, else four.
  return p.N <= sms * 8 ? launch_tb<D, 1>(p, sms, s) : launch_tb<D, 4>(p, sms, s);
}

}  // namespace

cudaError_t launch_rotate_heads(const void* x, long long row_stride, int N, const HeadRotation& r, const int* pos,
                                void* q, void* k, void* v, const PagePool& pool, const int* q_start, const int* held,
                                int* new_len, int* overflow, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = device_sm_count(dev, &sms);
  if (e != cudaSuccess) return e;
  RotateParams p{};
  p.x = static_cast<const uint4*>(x);
  p.row_vecs = row_stride / 8;
  p.N = N;
  p.r = r;
  p.pos = pos;
  p.q = static_cast<uint4*>(q);
  p.k = static_cast<uint4*>(k);
  p.v = static_cast<uint4*>(v);
  p.pool = pool;
  p.q_start = q_start;
  p.held = held;
  p.new_len = new_len;
  p.overflow = overflow;
  switch (r.D) {
    case 64: return launch_d<64>(p, sms, s);
    case 128: return launch_d<128>(p, sms, s);
    case 256: return launch_d<256>(p, sms, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace rx
