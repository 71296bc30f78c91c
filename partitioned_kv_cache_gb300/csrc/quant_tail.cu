// quant_tail.cu -- appending tokens to the language streams' 8-bit tails.
//
// "OxyGen: Unified KV Cache Management for Vision-Language-Action Models under
// Multi-Task Parallelism", §"Core method": every stream appends its own keys
// and values to a private tail.  Here a token's vector x of one K/V head is
// kept as D e4m3 codes and one byte, the exponent of a power-of-two scale
// 2^(byte - 127):
//   e    = the smallest integer >= -127 with max_i |x_i| <= 448 * 2^e
//   code = x_i * 2^-e rounded to e4m3 (nearest, ties to even), byte = e + 127
// so the largest code uses the top of the e4m3 range (448 is its largest
// value) and the scaling itself is exact: the code's rounding, at most 2^-4 of
// the value, is the only one.  An all-zero vector gets byte 0; a vector with
// an infinity or a NaN gets byte 255, which stands for NaN, and zero codes:
// it reads back as NaN without putting NaN codes where a masked product
// would meet them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rx_internal.h"
#include "sm103_ptx.cuh"

namespace rx {
namespace {

constexpr int kAppendThreads = 256;

// Quantise the vector that L = D/8 consecutive lanes hold, eight bf16 values
// each: *codes = this lane's eight codes, returns the vector's exponent byte.
// Every lane of the warp calls it.
template <int L>
__device__ __forceinline__ uint32_t quantise8(const uint4& x, uint2* codes) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
  // The magnitudes' bf16 bits order like the magnitudes; two at a time.
  const uint32_t two = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
  uint32_t top = max(two & 0xFFFFu, two >> 16);
  if constexpr (L == 32) {
    top = __reduce_max_sync(0xffffffffu, top);
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  // 1.m * 2^(E-127) <= 448 * 2^e = 1.75 * 2^(8+e): e = E - 135, one more
  // when the mantissa is above .75 (96/128), which adding 31 carries into E.
  const bool poison = top >= 0x7F80u;
  const uint32_t byte = poison ? 255u : static_cast<uint32_t>(max(static_cast<int>((top + 31u) >> 7) - 8, 0));
  // 2^-e; a poisoned vector's codes are zeros.
  const float up = __uint_as_float((254u - min(byte, 254u)) << 23);
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (poison) w[i] = 0u;
    f[2 * i] = __uint_as_float(w[i] << 16) * up;
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u) * up;
  }
  *codes = make_uint2(to_e4m3x2(f[0], f[1]) | (to_e4m3x2(f[2], f[3]) << 16), to_e4m3x2(f[4], f[5]) | (to_e4m3x2(f[6], f[7]) << 16));
  return byte;
}

// D/8 lanes per vector (token and head) of a stream; each lane moves 16 bytes
// of K and of V for kPerThread vectors, all loads in flight before the first
// conversion.  A CTA's vectors are consecutive in the stream's new tokens, so
// their codes land in consecutive places too.  Bound by memory: 24 prompts of
// up to 8191 tokens at D = 256 (170 MB) take 28.2 us, 6.0 TB/s, with four
// vectors a thread, 29.3 with two and 33.3 with one; calls that fit on the GPU
// at once are bound by latency and faster with one (16 tokens: 1.7 against
// 1.9 us, 61 x 8 tokens of 8 heads: 2.5 against 3.1 us).
template <int D, int kPerThread>
__global__ void __launch_bounds__(kAppendThreads) tail_append_quant_kernel(
    uint2* __restrict__ k_tail, uint2* __restrict__ v_tail, uint8_t* __restrict__ k_exp,
    uint8_t* __restrict__ v_exp, const int* __restrict__ tail_len, int* __restrict__ new_len,
    const uint4* __restrict__ k_new, const uint4* __restrict__ v_new, const int* __restrict__ n_new, int T,
    int tail_cap, int Hkv, unsigned int ctas, int* overflow) {
  constexpr int L = D / 8;                       // lanes of a vector
  constexpr unsigned int VB = kAppendThreads / L;   // vectors a CTA takes at a time
  grid_dependency_wait();
  grid_launch_dependents();
  const unsigned int b = blockIdx.x / ctas, part = blockIdx.x - b * ctas;   // ctas per stream
  const int len = tail_len[b];
  const int n = n_new ? max(0, min(n_new[b], T)) : T;
  const bool fine = len >= 0 && len <= tail_cap;
  const int keep = fine ? min(n, tail_cap - len) : 0;   // tokens stored
  if (part == 0 && threadIdx.x == 0) {
    if (keep < n && overflow) atomicOr(overflow, 1);
    if (new_len) new_len[b] = fine ? len + keep : len;
  }
  const unsigned int end = static_cast<unsigned int>(keep) * Hkv;   // the stream's vectors
  const unsigned int sub = threadIdx.x % L;
  const unsigned int v0 = part * (VB * kPerThread) + threadIdx.x / L;
  if (part * (VB * kPerThread) >= end) return;
  uint4 kx[kPerThread], vx[kPerThread];
  const size_t src = static_cast<size_t>(b) * T * Hkv;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const unsigned int v = v0 + i * VB;
    kx[i] = vx[i] = make_uint4(0u, 0u, 0u, 0u);
    if (v < end) {
      kx[i] = __ldg(k_new + (src + v) * L + sub);
      vx[i] = __ldg(v_new + (src + v) * L + sub);
    }
  }
  const size_t dst = (static_cast<size_t>(b) * tail_cap + len) * Hkv;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const unsigned int v = v0 + i * VB;
    uint2 kc, vc;
    const uint32_t kb = quantise8<L>(kx[i], &kc), vb = quantise8<L>(vx[i], &vc);
    if (v < end) {
      k_tail[(dst + v) * L + sub] = kc;
      v_tail[(dst + v) * L + sub] = vc;
      if (sub == 0) {
        k_exp[dst + v] = static_cast<uint8_t>(kb);
        v_exp[dst + v] = static_cast<uint8_t>(vb);
      }
    }
  }
}

template <int D, int kPerThread>
cudaError_t launch_per(void* k_tail, void* v_tail, uint8_t* k_exp, uint8_t* v_exp, const int* tail_len, int* new_len,
                     const void* k_new, const void* v_new, const int* n_new, int B, int T, int tail_cap, int Hkv,
                     int* overflow, cudaStream_t s) {
  constexpr unsigned int per = kAppendThreads / (D / 8) * kPerThread;   // vectors of a CTA
  const unsigned int ctas = (static_cast<unsigned int>(T) * Hkv + per - 1) / per;
  const cudaError_t e = launch_k(tail_append_quant_kernel<D, kPerThread>, dim3(ctas * B), dim3(kAppendThreads), 0, s,
                                 static_cast<uint2*>(k_tail), static_cast<uint2*>(v_tail), k_exp, v_exp, tail_len,
                                 new_len, static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), n_new,
                                 T, tail_cap, Hkv, ctas, overflow);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D>
cudaError_t launch_d(void* k_tail, void* v_tail, uint8_t* k_exp, uint8_t* v_exp, const int* tail_len, int* new_len,
                     const void* k_new, const void* v_new, const int* n_new, int B, int T, int tail_cap, int Hkv,
                     int* overflow, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = device_sm_count(dev, &sms);
  if (e != cudaSuccess) return e;
  // One vector a thread while all of them are resident together (2048 threads per SM).
  const bool once = static_cast<long long>(B) * T * Hkv * (D / 8) <= static_cast<long long>(sms) * 2048;
  return once ? launch_per<D, 1>(k_tail, v_tail, k_exp, v_exp, tail_len, new_len, k_new, v_new, n_new, B, T, tail_cap, Hkv, overflow, s)
              : launch_per<D, 4>(k_tail, v_tail, k_exp, v_exp, tail_len, new_len, k_new, v_new, n_new, B, T, tail_cap, Hkv, overflow, s);
}

}  // namespace

cudaError_t launch_tail_append_quant(void* k_tail, void* v_tail, uint8_t* k_exp, uint8_t* v_exp, const int* tail_len,
                                     int* new_len, const void* k_new, const void* v_new, const int* n_new, int B,
                                     int T, int tail_cap, int Hkv, int D, int* overflow, cudaStream_t s) {
  switch (D) {
    case 64: return launch_d<64>(k_tail, v_tail, k_exp, v_exp, tail_len, new_len, k_new, v_new, n_new, B, T, tail_cap, Hkv, overflow, s);
    case 128: return launch_d<128>(k_tail, v_tail, k_exp, v_exp, tail_len, new_len, k_new, v_new, n_new, B, T, tail_cap, Hkv, overflow, s);
    case 256: return launch_d<256>(k_tail, v_tail, k_exp, v_exp, tail_len, new_len, k_new, v_new, n_new, B, T, tail_cap, Hkv, overflow, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace rx
