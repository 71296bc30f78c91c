// quant_attn.cu -- language streams' attention over the shared store and their
// own 8-bit tails.
//
// For query token t of stream b (its n_new[b] query tokens are the newest ones
// of its tail, of len keys) and query head h:
//   out = softmax_j(q . K_j / sqrt(D)) V_j over the keys
//   [pinned P; the window's frames; tail_b[0, len - n_new[b] + t + 1)]
// with one softmax ("Reflex: Real-Time VLA Control through Streaming
// Inference", §III "Core formulas", Proposition A.1: the parts may be taken
// apart and merged).  A tail key is 2^(k_exp - 127) times its e4m3 codes, a
// value likewise (quant_tail.cu).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "rx_internal.h"
#include "sm103_ptx.cuh"

namespace rx {
namespace {

constexpr int kRowThreads = 256;

// 2^(byte - 127); byte 255 stands for NaN.
__device__ __forceinline__ float exp_scale(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  float2 f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(f.x), "=f"(f.y) : "r"(h));
  return f;
}

// One CTA per (stream, query token, query head): its warps walk the keys in
// turn, each with a running maximum and sum, and meet at the end.
template <int D>
__global__ void __launch_bounds__(kRowThreads) stream_rows_kernel(const QuantStreams a) {
  constexpr int E = D / 32;   // elements per lane
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.x % a.Hq;
  const long long bt = blockIdx.x / a.Hq;
  const int t = static_cast<int>(bt % a.T), b = static_cast<int>(bt / a.T);
  const int g = h / (a.Hq / a.Hkv);
  const int n = a.n_new ? min(a.n_new[b], a.T) : a.T;
  if (t >= n) return;
  const int len = min(max(a.tail_len[b], 0), a.tail_cap);
  const int seen = max(0, min(len, len - n + t + 1));
  int head = 0, valid = 0;
  load_ring_state(a.st, &head, &valid);
  const bool hole = a.slots > a.N && valid == a.N;
  const int win = valid * a.F;
  const long long row = (bt * a.Hq + h) * D;
  float q[E];
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = __bfloat162float(a.q[row + lane * E + e]);
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  const int total = a.P + win + seen;
  for (int j = warp; j < total; j += kRowThreads / 32) {
    float k[E], v[E];
    if (j < a.P + win) {
      const bool pin = j < a.P;
      int tok = pin ? j : j - a.P;
      if (!pin && hole && tok >= head * a.F) tok += a.F;
      const int c = lane * E / 8, r = tok & 63;
      const long long off = g * (pin ? a.pin_head_stride : a.win_head_stride) + (tok >> 6) * tile_bytes(D) +
                            (c >> 3) * 8192 + r * 128 + (((c & 7) ^ (r & 7)) << 4) + (lane * E % 8) * 2;
      const __nv_bfloat16* kp = reinterpret_cast<const __nv_bfloat16*>((pin ? a.pin_k : a.win_k) + off);
      const __nv_bfloat16* vp = reinterpret_cast<const __nv_bfloat16*>((pin ? a.pin_v : a.win_v) + off);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        k[e] = __bfloat162float(kp[e]);
        v[e] = __bfloat162float(vp[e]);
      }
    } else {
      const long long at = (static_cast<long long>(b) * a.tail_cap + (j - a.P - win)) * a.Hkv + g;
      const uint16_t* kp = reinterpret_cast<const uint16_t*>(a.k_tail + at * D) + lane * E / 2;
      const uint16_t* vp = reinterpret_cast<const uint16_t*>(a.v_tail + at * D) + lane * E / 2;
      const float ks = exp_scale(a.k_exp[at]), vs = exp_scale(a.v_exp[at]);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 kf = e4m3x2_to_float2(kp[e / 2]), vf = e4m3x2_to_float2(vp[e / 2]);
        k[e] = kf.x * ks;
        k[e + 1] = kf.y * ks;
        v[e] = vf.x * vs;
        v[e + 1] = vf.y * vs;
      }
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float p = mn == -INFINITY ? 0.f : exp2f(s - mn);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * v[e];
    m = mn;
  }
  __shared__ float sm[kRowThreads / 32], sl[kRowThreads / 32], so[kRowThreads / 32][D];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += kRowThreads) {
    float M = -INFINITY, L = 0.f, O = 0.f;
    for (int w = 0; w < kRowThreads / 32; ++w) M = fmaxf(M, sm[w]);
    for (int w = 0; w < kRowThreads / 32; ++w) {
      const float f = sm[w] == -INFINITY && sl[w] == 0.f ? 0.f : exp2f(sm[w] - M);
      L += f * sl[w];
      O += f * so[w][e];
    }
    a.out[row + e] = __float2bfloat16_rn(L == 0.f ? 0.f : O / L);   // a row with no key at all gets zeros
  }
}

}  // namespace

cudaError_t launch_streams_quant(const QuantStreams& a, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned int>(a.B) * a.T * a.Hq);
  cudaError_t e;
  switch (a.D) {
    case 64: e = launch_k(stream_rows_kernel<64>, grid, dim3(kRowThreads), 0, s, a); break;
    case 128: e = launch_k(stream_rows_kernel<128>, grid, dim3(kRowThreads), 0, s, a); break;
    case 256: e = launch_k(stream_rows_kernel<256>, grid, dim3(kRowThreads), 0, s, a); break;
    default: return cudaErrorInvalidValue;
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace rx
