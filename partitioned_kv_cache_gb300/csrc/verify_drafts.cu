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
// had been sampled token by token.  The choice of i compares a sum over V
// terms with a threshold, and plain fp32 sums would move its border by more
// than a token's probability: products and differences keep every bit, sums
// about 46.
//
// Of p and q only row a is read: once for the totals, the span of the warp that
// holds the threshold a second time and a sixteenth of that a third (and p's
// row again where no difference is positive).  A cluster of up to 8 CTAs shares
// a stream's row, each warp a contiguous span of it, so that one stream alone
// still uses 8 SMs' load bandwidth.  A difference p - q > 0 is two fp32 numbers
// (the rounded difference and its exact remainder) and a sum another two (each
// addition's rounding error is kept, in a sum of its own).  With n terms that
// second sum's roundings come to n^2 / 2 * 2^-48 of the first at worst, so a
// lane puts both away into a double every 128 terms: 2^-35 at worst; over terms
// of a softmax about 2^-47 (65536 in one pair: 2^-33).  Double additions run at
// 1/64 of the fp32 rate on this GPU: one for each term, or even one warp
// reduction in every warp, would take longer than the loads, so besides these
// they are kept to one warp's few totals.  The CTAs push their totals into each
// other's shared memory; the CTA whose interval holds the threshold cuts the
// crossing warp's span over its 16 warps, and the crossing warp of those walks
// its terms, four a lane.  Bound by memory for many streams (64 x 257152 fp32:
// 28 us, 4.7 TB/s, with 4 CTAs a stream so that all are resident; with 8 it is
// 31 us) and by the chain of dependent loads for few (8 us from 1000 to 32000
// terms).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "rx_internal.h"
#include "sm103_ptx.cuh"

namespace rx {
namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyMaxCluster = 8;

struct VerifyParams {
  const void* p;
  const void* q;
  const int* draft;
  const float* u;
  const float* r;
  const int* n_draft;
  const int* tail_len;
  int* tokens;
  int* n_accept;
  int* new_len;
  int T, V;
  int cluster;   // CTAs of one stream
  int span;      // terms of one warp: a multiple of 32, and so of a 16-byte load's
};

__device__ __forceinline__ float prob(const float* p, long long i) { return __ldg(p + i); }
__device__ __forceinline__ float prob(const __nv_bfloat16* p, long long i) { return __bfloat162float(__ldg(p + i)); }

// 16 bytes of probabilities as fp32.
__device__ __forceinline__ void widen(const uint4& v, float (&f)[4]) {
  f[0] = __uint_as_float(v.x);
  f[1] = __uint_as_float(v.y);
  f[2] = __uint_as_float(v.z);
  f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void widen(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// A sum of non-negative terms as sum + rest, both fp32.
struct TwoSum {
  float sum = 0.f, rest = 0.f;
  // Adds x >= 0 with its own remainder e.
  __device__ __forceinline__ void add(float x, float e) {
    const float s = sum + x;
    const float b = s - sum;
    rest += ((sum - (s - b)) + (x - b)) + e;   // the addition's exact error
    sum = s;
  }
  // Adds p - q if that is positive and finite (q = 0: p itself).
  __device__ __forceinline__ void add_difference(float p, float q) {
    const float d = p - q;
    const bool counts = d > 0.f && d < INFINITY;
    add(counts ? d : 0.f, counts ? (p - d) - q : 0.f);   // p >= q: the exact remainder
  }
  __device__ __forceinline__ void add_lanes() {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float x = __shfl_xor_sync(0xffffffffu, sum, o), e = __shfl_xor_sync(0xffffffffu, rest, o);
      add(x, e);
    }
  }
  __device__ __forceinline__ double value() const { return static_cast<double>(sum) + static_cast<double>(rest); }
  __device__ __forceinline__ void set(double v) {
    sum = static_cast<float>(v);
    rest = static_cast<float>(v - static_cast<double>(sum));
  }
};

__device__ __forceinline__ double weight(float p, float q) {
  const float d = p - q;
  return d > 0.f && d < INFINITY ? static_cast<double>(p) - static_cast<double>(q) : 0.0;
}

// Inclusive sum over the warp's lanes.
__device__ __forceinline__ double lane_scan(double v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// The total of warp `lane` of this CTA (0 past the last).
__device__ __forceinline__ double warp_total(const float2* s_warp, int lane) {
  const float2 t = lane < kVerifyWarps ? s_warp[lane] : make_float2(0.f, 0.f);
  return static_cast<double>(t.x) + static_cast<double>(t.y);
}

// The first lane with something of its own (own > 0) whose inclusive sum on
// top of `base` is above `want`; where rounding hides the crossing, the last
// one with something (-1: none).  *before: the sum in front of that lane, base
// included.
__device__ __forceinline__ int crossing(double own, double inclusive, double base, double want, int lane, double* before) {
  const uint32_t over = __ballot_sync(0xffffffffu, own > 0.0 && base + inclusive > want);
  const uint32_t some = __ballot_sync(0xffffffffu, own > 0.0);
  const int w = over ? __ffs(over) - 1 : 31 - __clz(some);
  const double in = __shfl_sync(0xffffffffu, inclusive, max(w, 1) - 1);
  *before = w > 0 ? base + in : base;
  return w;
}

__device__ __forceinline__ void st_cluster_f64(uint32_t local, int rank, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(cluster_peer(local, rank)), "d"(v) : "memory");
}

// This lane's terms of [v0, v1).  VEC: 16-byte loads (v0 and V are multiples of
// a load's terms).
template <typename P, bool VEC>
__device__ __forceinline__ TwoSum lane_sum(const P* pr, const P* qr, int out, int v0, int v1, int lane) {
  TwoSum t;
  if constexpr (VEC) {
    constexpr int E = 16 / sizeof(P);
    constexpr int U = 4;   // 16-byte loads of p (and of q) in flight
    for (int i = v0 + lane * E; i < v1; i += 32 * E * U) {
      uint4 pv[U], qv[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int at = i + k * 32 * E;
        pv[k] = qv[k] = make_uint4(0u, 0u, 0u, 0u);
        if (at < v1) {
          pv[k] = __ldg(reinterpret_cast<const uint4*>(pr + at));
          if (qr) qv[k] = __ldg(reinterpret_cast<const uint4*>(qr + at));
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int at = i + k * 32 * E;
        float pf[E], qf[E];
        widen(pv[k], pf);
        widen(qv[k], qf);
        if (static_cast<unsigned>(out) - static_cast<unsigned>(at) < static_cast<unsigned>(E)) {   // one vector of the row, if any
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (at + e == out) pf[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) t.add_difference(pf[e], qf[e]);
      }
    }
  } else {
    constexpr int U = 8;
    for (int i = v0 + lane; i < v1; i += 32 * U) {
      float pf[U], qf[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int at = i + k * 32;
        pf[k] = at < v1 && at != out ? prob(pr, at) : 0.f;
        qf[k] = at < v1 && qr ? prob(qr, at) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < U; ++k) t.add_difference(pf[k], qf[k]);
    }
  }
  return t;
}

// More than kFold terms a lane, a double for each kFold.  (In a function of its
// own: inline, its doubles were computed for short spans too, and took 2.5 us.)
constexpr int kFold = 128;
template <typename P, bool VEC>
__device__ __noinline__ float2 long_lane_sum(const P* pr, const P* qr, int out, int v0, int v1, int lane) {
  double away = 0.0;
  for (int c0 = v0; c0 < v1; c0 += 32 * kFold) away += lane_sum<P, VEC>(pr, qr, out, c0, min(c0 + 32 * kFold, v1), lane).value();
  TwoSum t;
  t.set(away);
  return make_float2(t.sum, t.rest);
}

// The pair sum of the terms [v0, v1) over the warp's lanes.
template <typename P, bool VEC>
__device__ __forceinline__ TwoSum span_sum(const P* pr, const P* qr, int out, int v0, int v1, int lane) {
  TwoSum t;
  if (v1 - v0 > 32 * kFold) {
    const float2 x = long_lane_sum<P, VEC>(pr, qr, out, v0, v1, lane);
    t.sum = x.x;
    t.rest = x.y;
  } else {
    t = lane_sum<P, VEC>(pr, qr, out, v0, v1, lane);
  }
  t.add_lanes();
  return t;
}

// VEC: rows start on 16-byte boundaries (p, q and V are aligned): 16-byte loads.
template <typename P, bool VEC>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_drafts_kernel(const VerifyParams a) {
  __shared__ float2 s_warp[kVerifyWarps];
  __shared__ double s_cta[2][kVerifyMaxCluster], s_base, s_want;
  __shared__ int s_accept, s_pick, s_any;
  grid_dependency_wait();
  grid_launch_dependents();
  const P* p = static_cast<const P*>(a.p);
  const P* q = static_cast<const P*>(a.q);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster;
  const int T = a.T, V = a.V;
  const int n = a.n_draft ? min(a.n_draft[b], T) : T;
  // The first 32 drafts are asked for beside n_draft, not after it.
  int x = -1;
  float ut = 0.f;
  if (warp == 0 && lane < T) {
    x = a.draft[static_cast<long long>(b) * T + lane];
    ut = a.u[static_cast<long long>(b) * T + lane];
  }
  int* tokens = a.tokens + static_cast<long long>(b) * (T + 1);
  if (n < 0) {   // an idle slot (every CTA of the cluster leaves)
    if (rank == 0) {
      for (int i = threadIdx.x; i <= T; i += kVerifyThreads) tokens[i] = -1;
      if (threadIdx.x == 0) {
        a.n_accept[b] = -1;
        if (a.new_len) a.new_len[b] = a.tail_len[b];
      }
    }
    return;
  }
  // Totals are pushed into the peers' shared memory below; the matching wait
  // in front of them guarantees that every CTA of the cluster has started.
  if (a.cluster > 1) cluster_arrive_started();
  // ---- accepted tokens, 32 positions at a time
  if (warp == 0) {
    int acc = n;
    for (int t0 = 0; t0 < n; t0 += 32) {
      const int t = t0 + lane;
      bool refuse = false;
      const long long bt = static_cast<long long>(b) * T + t;
      if (t0 > 0 && t < T) {
        x = a.draft[bt];
        ut = a.u[bt];
      }
      if (t < n) {
        refuse = true;
        if (x >= 0 && x < V) {
          const float px = prob(p, (bt + b) * V + x);
          const float qx = q ? prob(q, bt * V + x) : 1.f;
          // u * q < p with the product in full: 48 bits, whose exponent fits
          // a double whatever the factors are (fp32 with its rounding error
          // lost the error of products near the smallest subnormal).
          refuse = !(static_cast<double>(ut) * static_cast<double>(qx) < static_cast<double>(px));
        }
      }
      const uint32_t ballot = __ballot_sync(0xffffffffu, refuse);
      if (ballot) {
        acc = t0 + __ffs(ballot) - 1;
        break;
      }
    }
    if (lane == 0) s_accept = acc;
  }
  __syncthreads();
  const int acc = s_accept;
  const P* pr = p + (static_cast<long long>(b) * (T + 1) + acc) * V;
  const P* qr = acc < n && q ? q + (static_cast<long long>(b) * T + acc) * V : nullptr;
  // Without draft probabilities a refused token's weight is p - 1, never positive.
  int out = acc < n && !q ? a.draft[static_cast<long long>(b) * T + acc] : -1;
  const int v0 = (rank * kVerifyWarps + warp) * a.span, v1 = min(v0 + a.span, V);   // this warp's terms
  int next = -1;
  bool mine = false, any = false;   // this warp writes the answer; some weight is positive
  for (int form = 0; form < 2; ++form) {
    // ---- totals of the warps, the CTAs, the stream
    const TwoSum t = span_sum<P, VEC>(pr, qr, out, v0, v1, lane);
    if (lane == 0) s_warp[warp] = make_float2(t.sum, t.rest);
    __syncthreads();
    if (form == 0 && a.cluster > 1) cluster_wait_started();
    double own = 0.0, inclusive = 0.0;
    if (warp == 0) {
      own = warp_total(s_warp, lane);
      inclusive = lane_scan(own, lane);
      const double cta = __shfl_sync(0xffffffffu, inclusive, 31);
      if (lane < a.cluster) st_cluster_f64(smem_u32(&s_cta[form][rank]), lane, cta);
    }
    // The stores are seen, and nothing of this CTA is read remotely later.
    if (a.cluster > 1) cluster_sync_all(); else __syncthreads();
    // ---- which warp's span holds the threshold
    if (warp == 0) {
      const double r = fminf(fmaxf(a.r[b], 0.f), 0x1.fffffep-1f);   // [0, 1); NaN: 0
      const double cta = lane < a.cluster ? s_cta[form][lane] : 0.0, ctas = lane_scan(cta, lane);
      const double total = __shfl_sync(0xffffffffu, ctas, 31);
      const double want = r * total;
      double base, inner;
      const int c = crossing(cta, ctas, 0.0, want, lane, &base);
      const int w = crossing(own, inclusive, base, want, lane, &inner);   // meaningful in CTA c
      if (lane == 0) {
        s_any = total > 0.0;
        s_pick = c == rank ? w : -1;
        s_base = inner;
        s_want = want;
      }
    }
    __syncthreads();
    any = s_any;
    if (!any) {   // no positive difference: the plain probabilities (alike in the whole cluster)
      qr = nullptr;
      out = -1;
      __syncthreads();   // s_any is free
      continue;
    }
    const int pick = s_pick;
    if (pick < 0) return;   // another CTA's
    // ---- that span again, cut over the warps
    const int w0 = (rank * kVerifyWarps + pick) * a.span, w1 = min(w0 + a.span, V);
    const int part = ((w1 - w0 + kVerifyWarps - 1) / kVerifyWarps + 31) / 32 * 32;
    const int x0 = w0 + warp * part, x1 = min(x0 + part, w1);
    const TwoSum d = span_sum<P, false>(pr, qr, out, x0, x1, lane);
    if (lane == 0) s_warp[warp] = make_float2(d.sum, d.rest);
    __syncthreads();
    const double want = s_want;
    if (warp == 0) {
      double inner;
      const double own = warp_total(s_warp, lane);
      const int w = crossing(own, lane_scan(own, lane), s_base, want, lane, &inner);
      __syncwarp();
      if (lane == 0) {
        s_pick = w;
        s_base = inner;
      }
    }
    __syncthreads();
    if (s_pick != warp) return;
    mine = true;
    double base = s_base;
    int last = -1;
    for (int i0 = x0; i0 < x1 && next < 0; i0 += 128) {   // four terms a lane
      const int at = i0 + lane * 4;
      double x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[e] = at + e < x1 && at + e != out ? weight(prob(pr, at + e), qr ? prob(qr, at + e) : 0.f) : 0.0;
      const double sum = lane_scan((x[0] + x[1]) + (x[2] + x[3]), lane);
      double run = __shfl_up_sync(0xffffffffu, sum, 1);
      run = lane ? base + run : base;
      int hit = -1, some = -1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        run += x[e];
        if (x[e] > 0.0) {
          some = at + e;
          if (hit < 0 && run > want) hit = at + e;
        }
      }
      const uint32_t over = __ballot_sync(0xffffffffu, hit >= 0), adds = __ballot_sync(0xffffffffu, some >= 0);
      if (over) next = __shfl_sync(0xffffffffu, hit, __ffs(over) - 1);
      else if (adds) last = __shfl_sync(0xffffffffu, some, 31 - __clz(adds));
      base += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (next < 0) next = last;   // rounding left the last sum at the threshold
    break;
  }
  if (!any) mine = rank == 0 && warp == 0;   // no weight at all: next = -1
  if (!mine) return;
  for (int i = lane; i <= T; i += 32)
    tokens[i] = i < acc ? a.draft[static_cast<long long>(b) * T + i] : i == acc ? next : -1;
  if (lane == 0) {
    a.n_accept[b] = acc;
    if (a.new_len) a.new_len[b] = a.tail_len[b] + 1 + acc;
  }
}

template <typename P, bool VEC>
cudaError_t launch_typed(const VerifyParams& a, int B, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned int>(a.cluster) * B);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = a.cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, verify_drafts_kernel<P, VEC>, a);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_verify_drafts(const void* p, const void* q, bool bf16, const int* draft, const float* u,
                                 const float* r, const int* n_draft, int B, int T, int V, const int* tail_len,
                                 int* tokens, int* n_accept, int* new_len, cudaStream_t s) {
  if (B == 0) return cudaSuccess;
  VerifyParams a{p, q, draft, u, r, n_draft, tail_len, tokens, n_accept, new_len, T, V, 1, 0};
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = device_sm_count(dev, &sms);
  if (e != cudaSuccess) return e;
  // About 4096 terms a CTA (8 a thread), in at most 8 CTAs a stream and no
  // more than fit on the GPU at once (two per SM).
  while (a.cluster < kVerifyMaxCluster && V > 4096 * a.cluster && 2ll * a.cluster * B <= 2ll * sms) a.cluster *= 2;
  const int warps = a.cluster * kVerifyWarps;
  a.span = ((V + warps - 1) / warps + 31) / 32 * 32;
  const uintptr_t at = reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q);
  const bool vec = (at & 15u) == 0 && static_cast<long long>(V) * (bf16 ? 2 : 4) % 16 == 0;
  if (bf16) return vec ? launch_typed<__nv_bfloat16, true>(a, B, s) : launch_typed<__nv_bfloat16, false>(a, B, s);
  return vec ? launch_typed<float, true>(a, B, s) : launch_typed<float, false>(a, B, s);
}

}  // namespace rx
