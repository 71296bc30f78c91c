// verify_drafts.cu -- which of a stream's drafted tokens stay, and the token
// that follows them.
//
// A draft model proposes tokens x_0 .. x_{n-1} with probabilities q_t(x_t);
// the target model's probabilities after each of them are p_0 .. p_n.  With
// given uniform numbers u_t and r in [0, 1):
//   x_t is accepted while u_t * q_t(x_t) < p_t(x_t); a = the first refused
//   position, or n;
//   w_i = max(p_a(i) - q_a(i), 0) if a < n, else p_a(i); if no w_i is
//   positive, w = p_a;
//   next token = the smallest i with w_0 + .. + w_i > r * (w_0 + .. + w_{V-1}).
// The accepted tokens and the next one are then distributed as if the target
// had been sampled token by token.  Differences and sums are in 64 bits: the
// choice of i compares a sum over V terms with a threshold, and 32 bits would
// move its border by more than a token's probability.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rx_internal.h"
#include "sm103_ptx.cuh"

namespace rx {
namespace {

constexpr int kVerifyThreads = 1024;

__device__ __forceinline__ float prob(const float* p, long long i) { return p[i]; }
__device__ __forceinline__ float prob(const __nv_bfloat16* p, long long i) { return __bfloat162float(p[i]); }

// Inclusive sum over the block's threads in thread order.
__device__ __forceinline__ double block_scan(double v, double* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  for (int w = 0; w < warp; ++w) v += warp_sums[w];
  return v;
}

template <typename P>
__global__ void __launch_bounds__(kVerifyThreads) verify_drafts_kernel(const P* __restrict__ p, const P* __restrict__ q,
                                                                      const int* __restrict__ draft,
                                                                      const float* __restrict__ u,
                                                                      const float* __restrict__ r,
                                                                      const int* __restrict__ n_draft, int T, int V,
                                                                      const int* tail_len, int* __restrict__ tokens,
                                                                      int* __restrict__ n_accept, int* new_len) {
  grid_dependency_wait();
  grid_launch_dependents();
  __shared__ double sums[32];
  __shared__ double s_total, s_base;
  __shared__ int s_a, s_next, s_last;
  const int b = blockIdx.x;
  const int n = n_draft ? min(n_draft[b], T) : T;
  if (n < 0) {   // an idle slot
    for (int i = threadIdx.x; i <= T; i += kVerifyThreads) tokens[static_cast<long long>(b) * (T + 1) + i] = -1;
    if (threadIdx.x == 0) {
      n_accept[b] = -1;
      if (new_len) new_len[b] = tail_len[b];
    }
    return;
  }
  if (threadIdx.x == 0) {
    int a = 0;
    for (; a < n; ++a) {
      const long long bt = static_cast<long long>(b) * T + a;
      const int x = draft[bt];
      if (x < 0 || x >= V) break;
      const double px = prob(p, (bt + b) * V + x);
      const double qx = q ? prob(q, bt * V + x) : 1.0;
      if (!(static_cast<double>(u[bt]) * qx < px)) break;
    }
    s_a = a;
    s_next = -1;
    s_last = -1;
    s_base = 0.0;
  }
  __syncthreads();
  const int a = s_a;
  const P* pr = p + (static_cast<long long>(b) * (T + 1) + a) * V;
  const P* qr = a < n && q ? q + (static_cast<long long>(b) * T + a) * V : nullptr;
  const int out = a < n && !q ? draft[static_cast<long long>(b) * T + a] : -1;
  for (int form = 0; form < 2; ++form) {   // 1: no positive difference, the plain probabilities
    auto weight = [&](int i) {
      double w = prob(pr, i);
      if (form == 0) {
        if (qr) w -= prob(qr, i);
        if (i == out) w = 0.0;
      }
      return w > 0.0 && w < INFINITY ? w : 0.0;
    };
    double t = 0.0;
    for (int i = threadIdx.x; i < V; i += kVerifyThreads) t += weight(i);
    t = block_scan(t, sums);
    if (threadIdx.x == kVerifyThreads - 1) s_total = t;
    __syncthreads();
    if (s_total > 0.0) {
      const double want = static_cast<double>(r[b]) * s_total;
      for (int i0 = 0; i0 < V && s_next < 0; i0 += kVerifyThreads) {
        const int i = i0 + threadIdx.x;
        const double w = i < V ? weight(i) : 0.0;
        const double c = s_base + block_scan(w, sums);
        if (w > 0.0) atomicMax(&s_last, i);
        if (w > 0.0 && c > want) atomicMin(reinterpret_cast<unsigned int*>(&s_next), static_cast<unsigned int>(i));
        __syncthreads();
        if (threadIdx.x == kVerifyThreads - 1) s_base = c;
        __syncthreads();
      }
      break;
    }
    __syncthreads();
  }
  __syncthreads();
  const int next = s_next >= 0 ? s_next : s_last;   // rounding may leave the last sum at the threshold
  for (int i = threadIdx.x; i <= T; i += kVerifyThreads)
    tokens[static_cast<long long>(b) * (T + 1) + i] = i < a ? draft[static_cast<long long>(b) * T + i] : i == a ? next : -1;
  if (threadIdx.x == 0) {
    n_accept[b] = a;
    if (new_len) new_len[b] = tail_len[b] + 1 + a;
  }
}

}  // namespace

cudaError_t launch_verify_drafts(const void* p, const void* q, bool bf16, const int* draft, const float* u,
                                 const float* r, const int* n_draft, int B, int T, int V, const int* tail_len,
                                 int* tokens, int* n_accept, int* new_len, cudaStream_t s) {
  if (B == 0) return cudaSuccess;
  cudaError_t e;
  if (bf16)
    e = launch_k(verify_drafts_kernel<__nv_bfloat16>, dim3(B), dim3(kVerifyThreads), 0, s,
                 static_cast<const __nv_bfloat16*>(p), static_cast<const __nv_bfloat16*>(q), draft, u, r, n_draft, T, V,
                 tail_len, tokens, n_accept, new_len);
  else
    e = launch_k(verify_drafts_kernel<float>, dim3(B), dim3(kVerifyThreads), 0, s, static_cast<const float*>(p),
                 static_cast<const float*>(q), draft, u, r, n_draft, T, V, tail_len, tokens, n_accept, new_len);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace rx
