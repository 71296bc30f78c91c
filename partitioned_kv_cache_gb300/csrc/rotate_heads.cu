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
// fraction of a turn, so pos times it modulo 2^64 is the angle modulo one turn, off
// by |pos| times the fraction's own error: two roundings to double, 2^-52 of freq /
// (2 pi), so 5 10^-7 rad at most at freq 1 and the farthest positions (and 2^-54 of a
// turn for a negative freq, whose fraction is its distance from a whole turn).  Its
// upper 32 bits, rounded to fp32, feed sincospi: another 2^-26 of a turn, 10^-7 rad.
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

// bf16's values reach as far as fp32's, their squares do not stay within it.  Where
// the mean of a head's squares is not near enough to 1, the lanes that hold the head
// bring its values to the scale of the larger of their largest and sqrt(eps), a power
// of two, and get the mean (eps in it) in that scale.  All lanes of a warp call it;
// heads that are near or not `normed` stay as they are.  The vote on it costs 95 us for
// 93 (13600 tokens of 48 heads of 128).
constexpr float kNear = 8.6736173798840355e-19f;   // 2^-60
template <int D>
__device__ __forceinline__ float scaled_mean(float (&y)[16], float eps, float mean, bool normed) {
  constexpr int L = D / 16;
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(y[e]));
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float base = fmaxf(top, sqrtf(eps));
  // (zeros without eps, and a head with an infinity, have no scale)
  const bool far = normed && !(mean >= kNear && mean <= 1.f / kNear) && base > 0.f && base < INFINITY;
  const int k = far ? ilogbf(base) : 0;
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    y[e] = scalbnf(y[e], -k);
    ss = fmaf(y[e], y[e], ss);
  }
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  return far ? ss * (1.f / D) + scalbnf(eps, -2 * k) : mean;
}

// A CTA takes TB tokens at a time; the pairs' cosines and sines are computed once
// per token into shared memory and serve all its heads.  D/16 lanes hold a head,
// 16 values each as two chunks of eight, R/16 chunks apart: in half pairs a lane
// then has both values of its pairs and nothing is exchanged but the norm's sum.
// (With eight values a lane and the partners fetched from other lanes
// the prompts below took 129 us; with two groups of four, whose loads are 8 bytes
// wide, 192.)  A lane asks for kFlight heads at a time, the first of them before
// the angles are computed.  Bound by the loads in flight: 13600 tokens of 48 heads
// of 128 take 95 us, 4.7 TB/s.  More threads on an SM (64 registers cut to 48 or 40:
// 117 us), four heads in flight (104) and blocks of 512 threads (105) are slower,
// blocks of 128 as fast (91; 9.9 for 8.7 us at 2048 tokens).
template <int D, int TB>
__global__ void __launch_bounds__(kThreads) rotate_heads_kernel(const __grid_constant__ RotateParams p) {
  constexpr int L = D / 16;              // lanes of a head
  constexpr int kChunks = D / 8;         // 16-byte chunks of a head
  constexpr int kGroups = kThreads / L;
  constexpr int kFlight = 2;
  __shared__ __align__(16) float2 s_turn[TB * (D / 2)];   // (cos, sin) of every pair
  __shared__ __align__(16) float s_w[2][D];               // norm weights of queries and keys
  __shared__ unsigned long long s_freq[D / 2];
  __shared__ int s_stream[TB];
  __shared__ long long s_row[TB];                    // pool row of the token's key and value, -1: dropped
  const int Hq = p.r.Hq, Hkv = p.r.Hkv, H = Hq + 2 * Hkv, pairs = p.r.pairs;
  const bool paged = p.k == nullptr, adjacent = p.r.adjacent != 0;
  const int sub = threadIdx.x % L, group = threadIdx.x / L;
  const int half = pairs / 8;            // chunks of the first halves
  const bool turned = sub < half;
  const int c0 = turned ? sub : 2 * half + 2 * (sub - half), c1 = turned ? sub + half : c0 + 1;
  const bool norm_q = p.r.q_weight != nullptr, norm_k = p.r.k_weight != nullptr;
  grid_dependency_wait();
  grid_launch_dependents();
  for (int i = threadIdx.x; i < pairs; i += kThreads) s_freq[i] = turn_fraction(__ldg(p.r.freq + i));
  for (int i = threadIdx.x; i < D; i += kThreads) {
    if (norm_q) s_w[0][i] = __ldg(p.r.q_weight + i);
    if (norm_k) s_w[1][i] = __ldg(p.r.k_weight + i);
  }
  if (paged && p.new_len) {
    for (int b = blockIdx.x * kThreads + threadIdx.x; b < p.pool.B; b += gridDim.x * kThreads) {
      const int s0 = max(0, min(p.q_start[b], p.N)), s1 = max(0, min(p.q_start[b + 1], p.N));
      const int len = p.held[b], cap = pool_capacity(p.pool);
      p.new_len[b] = len < 0 || len > cap ? len : len + min(max(0, s1 - s0), cap - len);
    }
  }
  for (int n0 = blockIdx.x * TB; n0 < p.N; n0 += gridDim.x * TB) {
    const int tokens = min(TB, p.N - n0);
    // This lane group's heads in turn: (t, h), kGroups on each time.
    int lt = group / H, lh = group - lt * H;         // to load next
    int pt = lt, ph = lh;                            // to work on next
    uint4 raw[kFlight][2];
    auto load = [&]() {
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        if (lt < tokens) {
          const uint4* x = p.x + (n0 + lt) * p.row_vecs + lh * kChunks;
          raw[f][0] = __ldg(x + c0);
          raw[f][1] = __ldg(x + c1);
        }
        lh += kGroups;
        while (lh >= H) {
          lh -= H;
          ++lt;
        }
      }
    };
    load();
    __syncthreads();                                 // the last tokens' shared values are done with
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
    for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
      const int t = i / pairs, c = i - t * pairs;
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
    if (paged) {
      if (threadIdx.x < TB) {
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
    }
    const int vectors = tokens * H;
    for (int base = 0; base < vectors; base += kGroups * kFlight) {   // the same turns for every lane
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        if (base + f * kGroups >= vectors) break;
        const int t = pt, h = ph;
        ph += kGroups;
        while (ph >= H) {
          ph -= H;
          ++pt;
        }
        const bool there = t < tokens, isq = h < Hq, isv = h >= Hq + Hkv;
        uint32_t w[8] = {raw[f][0].x, raw[f][0].y, raw[f][0].z, raw[f][0].w, raw[f][1].x, raw[f][1].y, raw[f][1].z, raw[f][1].w};
        if (__any_sync(0xffffffffu, there && !isv)) {
          float y[16];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[2 * e] = __uint_as_float(w[e] << 16);
            y[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
          }
          if (norm_q || norm_k) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const bool normed = isq ? norm_q : norm_k;
            float mean = ss * (1.f / D) + p.r.eps;
            if (__any_sync(0xffffffffu, !(mean >= kNear && mean <= 1.f / kNear))) mean = scaled_mean<D>(y, p.r.eps, mean, normed);
            if (normed) {
              const float r = rsqrtf(mean);
              const float4* ws = reinterpret_cast<const float4*>(s_w[isq ? 0 : 1]);
              const float4 g[4] = {ws[2 * c0], ws[2 * c0 + 1], ws[2 * c1], ws[2 * c1 + 1]};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                y[4 * e] *= r * g[e].x;
                y[4 * e + 1] *= r * g[e].y;
                y[4 * e + 2] *= r * g[e].z;
                y[4 * e + 3] *= r * g[e].w;
              }
            }
          }
          if (turned) {
            // (cos, sin) of two pairs at a time.
            const float4* cs = reinterpret_cast<const float4*>(s_turn + (there ? t : 0) * (D / 2));
            if (adjacent) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 c = cs[2 * (i < 2 ? c0 : c1) + (i & 1)];
                float* z = y + 4 * i;
                const float a0 = z[0], b0 = z[1], a1 = z[2], b1 = z[3];
                z[0] = a0 * c.x - b0 * c.y;
                z[1] = b0 * c.x + a0 * c.y;
                z[2] = a1 * c.z - b1 * c.w;
                z[3] = b1 * c.z + a1 * c.w;
              }
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 c = cs[4 * sub + i];
                const float a0 = y[2 * i], a1 = y[2 * i + 1], b0 = y[2 * i + 8], b1 = y[2 * i + 9];
                y[2 * i] = a0 * c.x - b0 * c.y;
                y[2 * i + 8] = b0 * c.x + a0 * c.y;
                y[2 * i + 1] = a1 * c.z - b1 * c.w;
                y[2 * i + 9] = b1 * c.z + a1 * c.w;
              }
            }
          }
          if (!isv) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = pack2(y[2 * e], y[2 * e + 1]);
          }
        }
        if (!there) continue;
        uint4* dst = nullptr;
        if (isq) {
          if (s_stream[t] >= 0) dst = p.q + (static_cast<size_t>(n0 + t) * Hq + h) * kChunks;
        } else {
          const int kv = isv ? h - Hq - Hkv : h - Hq;
          if (!paged) {
            dst = (isv ? p.v : p.k) + (static_cast<size_t>(n0 + t) * Hkv + kv) * kChunks;
          } else if (s_row[t] >= 0) {
            const size_t row = static_cast<size_t>(s_row[t]) * Hkv + kv;
            dst = static_cast<uint4*>(isv ? p.pool.v : p.pool.k) + row * kChunks;
            if (!isv && sub == 0 && p.pool.weight) p.pool.weight[row] = 0.f;
          }
        }
        if (dst) {
          dst[c0] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[c1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
      if (base + kGroups * kFlight < vectors) load();
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
  // One token a CTA while an SM holds all of its CTAs at once (four), else four
  // tokens, whose angles and streams are looked up together.  With one and with four:
  // 16 tokens of 10 heads of 256 3.1 and 4.5 us, 600 4.4 and 4.8, 1208 7.5 and 5.9,
  // 4096 16.5 and 14.1; of 48 heads of 128 600 5.6 and 7.5, 1208 9.9 and 9.0, 4096
  // 28.2 and 25.0.
  return p.N <= sms * 4 ? launch_tb<D, 1>(p, sms, s) : launch_tb<D, 4>(p, sms, s);
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
