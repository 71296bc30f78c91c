// quant_attn.cu -- language streams' attention over the shared store and their
// own 8-bit tails (tcgen05, sm_103a).
//
// For query token t of stream b (its n_new[b] query tokens are the newest ones
// of its tail, of len keys) and query head h:
//   out = softmax_j(q . K_j / sqrt(D)) V_j over the keys
//   [pinned P; the window's frames; tail_b[0, len - n_new[b] + t + 1)]
// with one softmax ("Reflex: Real-Time VLA Control through Streaming
// Inference", §III "Core formulas", Proposition A.1: the parts may be taken
// apart and merged).  A tail key is 2^(k_exp - 127) times its e4m3 codes, a
// value likewise (quant_tail.cu).
//
// Three launches:
//   1. the shared store against the query rows of all streams together, by
//      the partitioned attention kernel, which writes fp32 partials;
//   2. stream_tail_kernel: every tail against its own stream's rows;
//   3. stream_merge_kernel: one row's partials into its bf16 output.
//
// stream_tail_kernel.  A tail is read by the G * n_new rows of one stream and
// K/V head, so the keys are the M = 128 side of the tensor-core products and
// the rows the N side:
//   S^T [128 keys x N] = K [128 x D] . Q^T      (K codes as loaded)
//   O^T [D x N]       += V^T [D x 128] . W^T    (V codes as loaded, MN-major)
// and the codes go from TMA to kind::f8f6f4 products without a conversion.
// The bf16 queries and fp32 weights enter as sums of e4m3 terms whose products
// accumulate in one fp32 accumulator: a query row, scaled by a power of two, is
// hi + lo exactly (8 significant bits in two 4-bit terms; what lies 2^-18 below
// the row's largest entry is rounded away); a weight is hi + mid + lo, within
// 2^-12 of itself or 2^-18 of the row's largest weight, so it adds nothing
// visible to the bf16 rounding of the output.
//   x_jn = S_jn * 2^(k_exp_j - 127) * (row scale) * log2(e) / sqrt(D)
//   l_n  = sum_j 2^(x_jn - m_n),   w_jn = 2^(x_jn + v_exp_j - 127 - M_n + 8)
// m_n and M_n are running maxima of x_jn and of x_jn + v_exp_j - 127: the
// weights' own reference keeps them at the top of the e4m3 range whatever the
// values' scales are.
//
// Work is cut into tiles of 128 keys of one (stream, K/V head, row tile) unit;
// each CTA takes an equal run of consecutive tiles (lengths are read on the
// device), and writes one fp32 partial per unit that it touches, to slot
// cta + unit (distinct, because a run that moves to a later CTA or a later unit
// never moves back).  Inside a unit, CT tiles form a chunk with one pair of
// maxima, one rescale of O and one synchronisation of the softmax warps; the
// scores of the next chunk are computed meanwhile.
//
// Warp roles (192 threads): warp 0 = TMA producer, warp 1 = TMEM allocator and
// MMA issuer, warps 2..5 = softmax and epilogue (thread = key of the tile for
// S^T, output column for O^T; TMEM lane quarter = warp % 4).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "rx_internal.h"
#include "sm103_ptx.cuh"

namespace rx {
namespace {

constexpr int kTailThreads = 192;
constexpr int kTK = 128;            // keys per tile
constexpr int kTerms = 3;           // e4m3 terms of a weight
constexpr float kTop = 8.f;         // log2 of a row's largest weight in e4m3 units

// ------------------------------------------------------------------- helpers
// 2^(byte - 127); byte 255 stands for NaN.
__device__ __forceinline__ float exp_scale(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 values -> two e4m3 codes (the first in the low byte), and back.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  float2 f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// Largest value over the warp's lanes; NaN is passed over.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ void st_shared_u8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// 8 or 16 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&v)[8]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&v)[16]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const float (&v)[8]) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const float (&v)[16]) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 inputs, fp32 accumulation, K = 32.
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor, kind::f8f6f4 with e4m3 A/B and fp32 D.
constexpr uint32_t idesc_e4m3_f32(int M, int N, bool a_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// Shared-memory matrix descriptor with rows of ROW bytes, 128- or 64-byte
// swizzle: as sdesc_sw128, layout type 4 (SWIZZLE_64B) for 64-byte rows.
template <int ROW>
__device__ __forceinline__ uint64_t sdesc_rows(uint32_t saddr, uint32_t lbo_bytes) {
  uint64_t d = sdesc_sw128(saddr, lbo_bytes, 8 * ROW);
  if (ROW == 64) d ^= (2ull ^ 4ull) << 61;
  return d;
}
// Byte offset of byte c of row r in such a layout (rows of ROW bytes).
template <int ROW>
__device__ __forceinline__ uint32_t swizzled(uint32_t r, uint32_t c) {
  const uint32_t x = ROW == 128 ? (r & 7u) : ((r >> 1) & 3u);
  return r * ROW + (((c >> 4) ^ x) << 4) + (c & 15u);
}

// ------------------------------------------------------------------ the work
struct TailParams {
  CUtensorMap tm_k;      // (D, Hkv, tail_cap, B) bytes, box (min(D, 128), 1, 128, 1)
  CUtensorMap tm_v;
  const __nv_bfloat16* q;
  const uint8_t* k_exp;
  const uint8_t* v_exp;
  const int* tail_len;
  const int* n_new;
  unsigned long long* head;   // [0] tiles of all streams, [1 + b] tiles before stream b
  float2* ml;                 // (m, l) [slot][RT]
  float* o;                   // [slot][RT][D], relative to m
  int* err;
  int B, T, G, Hkv, tail_cap;
  int row_tiles;              // row tiles of one stream and head: ceil(T * G / RT)
  int inject_tx;              // test aid: extra bytes CTA 0 expects on its first tile
  float scale_log2;
};

// Streams' keys and rows, from the lengths on the device.
struct StreamLen {
  int len, n;
};
__device__ __forceinline__ StreamLen stream_len(const int* tail_len, const int* n_new, int b, int T, int cap) {
  StreamLen s;
  s.len = min(max(tail_len[b], 0), cap);
  s.n = n_new ? min(max(n_new[b], 0), T) : T;
  return s;
}
// Tail keys that query token t sees.
__device__ __forceinline__ int keys_seen(const StreamLen& s, int t) { return max(0, min(s.len, s.len - s.n + t + 1)); }
// Key tiles of row tile rt: those its last row sees (none without a row).
__device__ __forceinline__ int unit_tiles(const StreamLen& s, int rt, int RT, int G) {
  if (rt * RT >= s.n * G) return 0;
  return (keys_seen(s, min(s.n - 1, (rt * RT + RT - 1) / G)) + kTK - 1) / kTK;
}
// Tiles of all row tiles of one stream and head.
__device__ __forceinline__ long long head_tiles(const StreamLen& s, int row_tiles, int RT, int G) {
  long long c = 0;
  for (int rt = 0; rt < row_tiles; ++rt) c += unit_tiles(s, rt, RT, G);
  return c;
}
// Active CTAs and the first tile of each: CTA c of A takes [c*C/A, (c+1)*C/A).
__device__ __forceinline__ unsigned long long first_tile(unsigned long long c, unsigned long long C, unsigned long long A) {
  return c * C / A;
}
__device__ __forceinline__ unsigned long long cta_of_tile(unsigned long long x, unsigned long long C, unsigned long long A) {
  return ((x + 1) * A - 1) / C;
}

// A CTA's run of tiles, unit by unit.  Every role walks it for itself.
struct Walk {
  int b, g, rt;         // the unit
  int skip;             // tiles of the unit before this run
  long long left;       // tiles of the run from here on
  StreamLen s;
  int tile0, ntiles;    // the segment: tiles [tile0, tile0 + ntiles) of the unit

  __device__ __forceinline__ bool next(const TailParams& p, int RT) {
    while (left > 0 && b < p.B) {
      const int ut = unit_tiles(s, rt, RT, p.G);
      if (ut > skip) {
        tile0 = skip;
        ntiles = static_cast<int>(min(static_cast<long long>(ut - skip), left));
        left -= ntiles;
        return true;
      }
      skip -= ut;
      advance(p);
    }
    return false;
  }
  __device__ __forceinline__ void advance(const TailParams& p) {
    if (++rt == p.row_tiles) {
      rt = 0;
      if (++g == p.Hkv) {
        g = 0;
        ++b;   // a run ends at the last tile, so b < B whenever tiles are left
        if (b < p.B) s = stream_len(p.tail_len, p.n_new, b, p.T, p.tail_cap);
      }
    }
  }
  // After a segment: the unit is finished for this run.
  __device__ __forceinline__ void done(const TailParams& p) {
    skip = 0;
    advance(p);
  }
};

template <int D, int RT>
struct TailLayout {
  static constexpr int N = RT < 16 ? 16 : RT;             // MMA N (a multiple of 16 at M = 128)
  static constexpr int ROW = D < 128 ? D : 128;           // bytes of a stored row (one column block)
  static constexpr int KB = D / ROW;                      // column blocks of a tile
  static constexpr int TILE = kTK * D;
  static constexpr int BLOCK = kTK * ROW;                 // one column block of a tile
  static constexpr int OB = D == 256 ? 2 : 1;             // 128-row blocks of O^T
  // Tiles per chunk, so that two chunks of scores and O fit in 512 columns of
  // TMEM (D = 256: one CTA per SM) or 256 (two CTAs per SM).
  static constexpr int CT = RT <= 16 ? 4 : RT == 32 ? (D == 256 ? 4 : 2) : (D == 256 ? 2 : 1);
  static constexpr int TM_O = 2 * CT * N;
  static constexpr int TM_USED = TM_O + OB * N;
  static constexpr int TM_COLS = TM_USED <= 128 ? 128 : TM_USED <= 256 ? 256 : 512;
  static constexpr int CTAS = D == 256 ? 1 : 2;           // per SM
  static constexpr int Q_BLOCK = N * ROW;                 // one column block of one term
  static constexpr int Q_BYTES = 2 * KB * Q_BLOCK;
  static constexpr int W_BLOCK = N * kTK;                 // one term of one tile's weights
  static constexpr int W_BYTES = CT * kTerms * W_BLOCK;
  static constexpr int MISC = 5120;
  static constexpr int BUDGET = (CTAS == 1 ? 227 : 113) * 1024 - 1024;   // less the alignment slack
  static constexpr int NS_FIT = (BUDGET - Q_BYTES - W_BYTES - MISC) / TILE;
  static constexpr int NS = NS_FIT > 12 ? 12 : NS_FIT;    // ring slots of one K or V tile
  static constexpr int OFF_RING = 0;
  static constexpr int OFF_Q = NS * TILE;
  static constexpr int OFF_W = OFF_Q + Q_BYTES;
  static constexpr int OFF_MISC = OFF_W + W_BYTES;
  static constexpr int BYTES = OFF_MISC + MISC;
  static constexpr int ALLOC = BYTES + 1024;
  // A chunk's V tiles are all resident before its products begin.
  static_assert(NS >= 3 && NS >= CT, "ring depth");
  static_assert(TM_USED <= 512 / CTAS, "tensor memory");
};

// The MISC area.
template <int RT>
struct TailMisc {
  unsigned long long bar[12 + 12 + 6];   // full, empty, Q ready, S full[2], W ready, PV done, drain
  uint32_t tmem;
  int abort;
  int b0, skip_unit;                     // first unit of the run: stream, and unit within it
  int skip_tile;
  int pad0;
  long long left;
  long long scan[kTailThreads / 32 + 1];
  float qs[RT];                          // 2^e of the query rows
  int seen[RT];                          // tail keys each row sees
  float m[RT], mv[RT];                   // running maxima (m_n, M_n)
  float ms[RT], mvs[RT];                 // ... as subtracted: m, M - kTop (0 while -inf)
  float al[RT], ao[RT];                  // factors of l and O of this chunk
  float wm[4][RT], wv[4][RT];            // the warps' maxima, then their sums of l
  int rescale;
};

enum : int { TB_FULL = 0, TB_EMPTY = 12, TB_Q = 24, TB_S = 25, TB_W = 27, TB_PV = 28, TB_DRAIN = 29 };

__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <int D, int RT>
__global__ void __launch_bounds__(kTailThreads, TailLayout<D, RT>::CTAS)
    stream_tail_kernel(const __grid_constant__ TailParams p) {
  using L = TailLayout<D, RT>;
  constexpr int N = L::N, CT = L::CT, NS = L::NS, ROW = L::ROW;
  constexpr int CB = RT < 16 ? RT : 16;   // columns taken at a time
  extern __shared__ uint8_t tail_smem[];
  const uint32_t raw = smem_u32(tail_smem);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = tail_smem + (base - raw);
  const uint32_t sRing = base + L::OFF_RING, sQ = base + L::OFF_Q, sW = base + L::OFF_W;
  static_assert(sizeof(TailMisc<RT>) <= L::MISC, "misc area");
  TailMisc<RT>& ms = *reinterpret_cast<TailMisc<RT>*>(gbase + L::OFF_MISC);
  volatile int* abort_flag = &ms.abort;
  const uint32_t sBar = base + L::OFF_MISC;
  auto BAR = [&](int i) { return sBar + 8u * static_cast<uint32_t>(i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 12; ++i) {
      mbar_init(BAR(TB_FULL + i), 1);
      mbar_init(BAR(TB_EMPTY + i), 1);
    }
    mbar_init(BAR(TB_Q), 128);
    mbar_init(BAR(TB_S), 1);
    mbar_init(BAR(TB_S + 1), 1);
    mbar_init(BAR(TB_W), 128);
    mbar_init(BAR(TB_PV), 1);
    mbar_init(BAR(TB_DRAIN), 1);
    ms.abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ms.tmem), L::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem;
  grid_dependency_wait();
  grid_launch_dependents();

  // ------------------------------------------------------ this CTA's tiles
  // Tiles before each stream, by a scan over the block's threads, 192 streams
  // a round; with more streams a second sweep finds the run's first.
  {
    auto scan_round = [&](int b, long long carry, long long* mine) {   // returns the carry after the round
      long long c = 0;
      if (b < p.B) c = p.Hkv * head_tiles(stream_len(p.tail_len, p.n_new, b, p.T, p.tail_cap), p.row_tiles, RT, p.G);
      long long inc = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      __syncthreads();
      if (lane == 31) ms.scan[warp] = inc;
      __syncthreads();
      long long before = carry, total = carry;
      for (int w = 0; w < kTailThreads / 32; ++w) {
        if (w < warp) before += ms.scan[w];
        total += ms.scan[w];
      }
      mine[0] = before + inc - c;
      mine[1] = c;
      return total;
    };
    long long mine[2], total = 0;
    for (int b0 = 0; b0 < p.B; b0 += kTailThreads) total = scan_round(b0 + threadIdx.x, total, mine);
    const unsigned long long C = static_cast<unsigned long long>(total);
    const unsigned long long A = min(static_cast<unsigned long long>(gridDim.x), C);
    const bool active = blockIdx.x < A;
    const long long first = active ? static_cast<long long>(first_tile(blockIdx.x, C, A)) : 0;
    if (threadIdx.x == 0) {
      ms.left = active ? static_cast<long long>(first_tile(blockIdx.x + 1ull, C, A)) - first : 0;
      if (blockIdx.x == 0) p.head[0] = C;
    }
    long long carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += kTailThreads) {
      const int b = b0 + threadIdx.x;
      if (p.B > kTailThreads) carry = scan_round(b, carry, mine);
      if (b < p.B) {
        if (blockIdx.x == 0) p.head[1 + b] = static_cast<unsigned long long>(mine[0]);
        if (active && first >= mine[0] && first < mine[0] + mine[1]) {
          ms.b0 = b;
          long long off = first - mine[0];
          const StreamLen s = stream_len(p.tail_len, p.n_new, b, p.T, p.tail_cap);
          const long long per_head = mine[1] / p.Hkv;
          const int g = static_cast<int>(off / per_head);
          off -= g * per_head;
          int rt = 0;
          for (int ut; off >= (ut = unit_tiles(s, rt, RT, p.G)); ++rt) off -= ut;
          ms.skip_unit = g * p.row_tiles + rt;
          ms.skip_tile = static_cast<int>(off);
        }
      }
    }
    __syncthreads();
  }
  Walk wk;
  wk.left = ms.left;
  if (wk.left > 0) {
    wk.b = ms.b0;
    wk.g = ms.skip_unit / p.row_tiles;
    wk.rt = ms.skip_unit % p.row_tiles;
    wk.skip = ms.skip_tile;
    wk.s = stream_len(p.tail_len, p.n_new, wk.b, p.T, p.tail_cap);
  }

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // Per segment: K of chunk 0, then K of chunk c + 1 and V of chunk c in
    // turn, the order in which the MMA issuer takes them.
    if (lane == 0) {
      unsigned int item = 0;
      bool stop = false;
      auto load = [&](const CUtensorMap* tm, int tile) {
        const int slot = item % NS;
        if (item >= NS && !mbar_wait(BAR(TB_EMPTY + slot), (item / NS - 1) & 1, abort_flag)) {
          stop = true;
          return;
        }
        mbar_arrive_expect_tx(BAR(TB_FULL + slot), L::TILE + (item == 0 && blockIdx.x == 0 ? p.inject_tx : 0));
        for (int kb = 0; kb < L::KB; ++kb)
          tma_load_4d(sRing + slot * L::TILE + kb * L::BLOCK, tm, kb * ROW, wk.g, tile * kTK, wk.b, BAR(TB_FULL + slot));
        ++item;
      };
      while (!stop && wk.next(p, RT)) {
        const int nt = wk.ntiles;
        for (int i = 0; i < min(CT, nt) && !stop; ++i) load(&p.tm_k, wk.tile0 + i);
        for (int c0 = 0; c0 < nt && !stop; c0 += CT) {
          for (int i = c0 + CT; i < min(c0 + 2 * CT, nt) && !stop; ++i) load(&p.tm_k, wk.tile0 + i);
          for (int i = c0; i < min(c0 + CT, nt) && !stop; ++i) load(&p.tm_v, wk.tile0 + i);
        }
        wk.done(p);
      }
      // Every copy issued must land before the CTA exits, even after an abort.
      volatile int no_abort = 0;
      for (unsigned int it = item > NS ? item - NS : 0; it < item; ++it)
        mbar_wait(BAR(TB_FULL + it % NS), (it / NS) & 1, &no_abort);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t kIdescS = idesc_e4m3_f32(kTK, N, false);
      constexpr uint32_t kIdescO = idesc_e4m3_f32(128, N, true);
      unsigned int item = 0, chunk = 0, seg = 0;
      bool ok = true;
      auto scores = [&](unsigned int ck, int tiles) {   // S^T of one chunk
        for (int i = 0; i < tiles && ok; ++i) {
          const int slot = item % NS;
          if (!mbar_wait(BAR(TB_FULL + slot), (item / NS) & 1, abort_flag)) {
            ok = false;
            return;
          }
          tc_fence_after();
          const uint32_t kt = sRing + slot * L::TILE;
          const uint32_t d = tmem + ((ck & 1) * CT + i) * N;
#pragma unroll
          for (int term = 0; term < 2; ++term)
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk) {
              const uint32_t kb = kk * 32 / ROW, ko = kk * 32 % ROW;
              umma_e4m3(d, sdesc_rows<ROW>(kt + kb * L::BLOCK + ko, 16),
                        sdesc_rows<ROW>(sQ + (term * L::KB + kb) * L::Q_BLOCK + ko, 16), kIdescS, (term | kk) ? 1u : 0u);
            }
          umma_commit(BAR(TB_EMPTY + slot));
          ++item;
        }
        umma_commit(BAR(TB_S + (ck & 1)));
      };
      while (ok && wk.next(p, RT)) {
        const int nt = wk.ntiles;
        if (!mbar_wait(BAR(TB_Q), seg & 1, abort_flag)) break;
        tc_fence_after();
        scores(chunk, min(CT, nt));
        for (int c0 = 0; c0 < nt && ok; c0 += CT, ++chunk) {
          if (c0 + CT < nt) scores(chunk + 1, min(CT, nt - c0 - CT));
          if (!ok || !mbar_wait(BAR(TB_W), chunk & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          for (int i = 0; i < min(CT, nt - c0); ++i) {
            const int slot = item % NS;
            if (!mbar_wait(BAR(TB_FULL + slot), (item / NS) & 1, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t vt = sRing + slot * L::TILE;
#pragma unroll
            for (int ob = 0; ob < L::OB; ++ob)
#pragma unroll
              for (int term = 0; term < kTerms; ++term)
#pragma unroll
                for (int kk = 0; kk < kTK / 32; ++kk)
                  // A: V codes, D along the stored rows (MN-major), 8-key
                  // groups 8 * ROW apart.  At D = 64 the product's upper 64
                  // rows read the bytes one tile further on and are not used.
                  umma_e4m3(tmem + L::TM_O + ob * N, sdesc_rows<ROW>(vt + ob * L::BLOCK + kk * 32 * ROW, L::BLOCK),
                            sdesc_rows<128>(sW + (i * kTerms + term) * L::W_BLOCK + kk * 32, 16), kIdescO,
                            (c0 | i | term | kk) ? 1u : 0u);
            umma_commit(BAR(TB_EMPTY + slot));
            ++item;
          }
          umma_commit(BAR(TB_PV));
        }
        wk.done(p);
        ++seg;
      }
      // No tensor-core work may be in flight when TMEM is released.
      umma_commit(BAR(TB_DRAIN));
      volatile int no_abort = 0;
      mbar_wait(BAR(TB_DRAIN), 0, &no_abort);
    }
  } else {
    // ------------------------------------------------- softmax and epilogue
    // After a wait that gave up the loops run on (their waits return at once)
    // so that all four warps meet at every barrier; the results are void and
    // the error bit says so.
    const int quarter = warp & 3;
    const int st = threadIdx.x - 64;                        // 0..127
    const int key_in_tile = quarter * 32 + lane;            // TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    unsigned int item0 = 0, chunk = 0;
    if (RT < N)   // rows of the operands past RT stay zero
      for (int i = st * 16; i < L::Q_BYTES + L::W_BYTES; i += 128 * 16) st_shared_v4(sQ + i, 0u, 0u, 0u, 0u);
    while (wk.next(p, RT)) {
      const int nt = wk.ntiles;
      const int row0 = wk.rt * RT;
      const int rows = min(RT, wk.s.n * p.G - row0);        // rows with a query token
      const int kmax = keys_seen(wk.s, min(wk.s.n - 1, (row0 + RT - 1) / p.G));   // keys any row sees
      const int kmin = keys_seen(wk.s, row0 / p.G);                               // ... every row sees
      softmax_sync();   // the previous segment's row state is no longer read
      if (st < RT) {
        ms.seen[st] = st < rows ? keys_seen(wk.s, (row0 + st) / p.G) : 0;
        ms.m[st] = -INFINITY;
        ms.mv[st] = -INFINITY;
      }
      // Q rows: 2^-e q = hi + lo, e as the append chooses it.
      for (int n = st >> 5; n < RT; n += 4) {
        constexpr int E = D / 32;
        uint32_t bits[E];
        uint32_t top = 0;
        const int r = row0 + n;
        const __nv_bfloat16* src =
            p.q + ((static_cast<long long>(wk.b) * p.T + r / p.G) * p.Hkv * p.G + wk.g * p.G + r % p.G) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          bits[e] = n < rows ? __bfloat16_as_ushort(src[e]) : 0u;
          top = max(top, bits[e] & 0x7FFFu);
        }
        top = __reduce_max_sync(0xffffffffu, top);
        const int ex = max(static_cast<int>(top >> 7) - 8 + ((top & 0x7Fu) > 96u ? 1 : 0), 1);
        const bool poison = (top >> 7) == 255u;
        if (lane == 0) ms.qs[n] = poison ? __uint_as_float(0x7FC00000u) : __uint_as_float(static_cast<uint32_t>(ex) << 23);
        const float up = __uint_as_float(static_cast<uint32_t>(254 - min(ex, 253)) << 23);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float a = poison ? 0.f : __uint_as_float(bits[e] << 16) * up;
          const float b = poison ? 0.f : __uint_as_float(bits[e + 1] << 16) * up;
          const uint32_t hi = to_e4m3x2(a, b);
          const float2 h = from_e4m3x2(hi);
          const uint32_t lo = to_e4m3x2(a - h.x, b - h.y);
          const uint32_t d = static_cast<uint32_t>(lane * E + e);
          const uint32_t off = (d / ROW) * L::Q_BLOCK + swizzled<ROW>(n, d % ROW);
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(sQ + off), "h"(static_cast<uint16_t>(hi)) : "memory");
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(sQ + L::KB * L::Q_BLOCK + off), "h"(static_cast<uint16_t>(lo))
                       : "memory");
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();   // the previous segment's reads of O
      mbar_arrive(BAR(TB_Q));
      softmax_sync();      // row state visible

      float l[RT];
#pragma unroll
      for (int n = 0; n < RT; ++n) l[n] = 0.f;
      const long long exp_base = (static_cast<long long>(wk.b) * p.tail_cap) * p.Hkv + wk.g;
      for (int c0 = 0; c0 < nt; c0 += CT, ++chunk) {
        const int tiles = min(CT, nt - c0);
        const int buf = chunk & 1;
        const uint32_t tS = tmem + buf * CT * N + lane_off;
        const int key0 = (wk.tile0 + c0) * kTK + key_in_tile;
        float ks[CT], ev[CT];
#pragma unroll
        for (int i = 0; i < CT; ++i) {
          const int key = key0 + i * kTK;
          uint32_t kb = 0, vb = 0;
          if (i < tiles && key < kmax) {
            const long long at = exp_base + static_cast<long long>(key) * p.Hkv;
            kb = p.k_exp[at];
            vb = p.v_exp[at];
          }
          ks[i] = exp_scale(kb) * p.scale_log2;
          ev[i] = vb == 255u ? __uint_as_float(0x7FC00000u) : static_cast<float>(vb) - 127.f;
        }
        mbar_wait(BAR(TB_S + buf), (chunk >> 1) & 1, abort_flag);
        __syncwarp();
        tc_fence_after();
        // ---- maxima of the chunk
#pragma unroll
        for (int n0 = 0; n0 < RT; n0 += CB) {
          float mx[CB], my[CB];
#pragma unroll
          for (int j = 0; j < CB; ++j) mx[j] = my[j] = -INFINITY;
#pragma unroll
          for (int i = 0; i < CT; ++i) {
            if (i < tiles) {
              float s[CB];
              tmem_ld_cols(tS + i * N + n0, s);
              const bool masked = (wk.tile0 + c0 + i + 1) * kTK > kmin;
#pragma unroll
              for (int j = 0; j < CB; ++j) {
                float x = s[j] * (ks[i] * ms.qs[n0 + j]);
                if (masked && key0 + i * kTK >= ms.seen[n0 + j]) x = -INFINITY;
                mx[j] = fmaxf(mx[j], x);
                my[j] = fmaxf(my[j], x + ev[i]);
              }
            }
          }
          float hx = 0.f, hy = 0.f;
#pragma unroll
          for (int j = 0; j < CB; ++j) {
            const float a = warp_max(mx[j]), b = warp_max(my[j]);
            if (lane == j) {
              hx = a;
              hy = b;
            }
          }
          if (lane < CB) {
            ms.wm[quarter][n0 + lane] = hx;
            ms.wv[quarter][n0 + lane] = hy;
          }
        }
        softmax_sync();
        if (st < 32) {
          bool grow = false;
          for (int n = st; n < RT; n += 32) {
            const float mo = ms.m[n], vo = ms.mv[n];
            const float mn = fmaxf(fmaxf(fmaxf(ms.wm[0][n], ms.wm[1][n]), fmaxf(ms.wm[2][n], ms.wm[3][n])), mo);
            const float vn = fmaxf(fmaxf(fmaxf(ms.wv[0][n], ms.wv[1][n]), fmaxf(ms.wv[2][n], ms.wv[3][n])), vo);
            ms.m[n] = mn;
            ms.mv[n] = vn;
            ms.ms[n] = mn == -INFINITY ? 0.f : mn;
            ms.mvs[n] = vn == -INFINITY ? 0.f : vn - kTop;
            ms.al[n] = mo == -INFINITY ? 0.f : ex2(mo - mn);
            ms.ao[n] = vo == -INFINITY ? 1.f : ex2(vo - vn);   // nothing accumulated yet: zeros (or NaN) stay
            grow |= c0 > 0 && vo != vn && vo != -INFINITY;
          }
          const bool any = __any_sync(0xffffffffu, grow);
          if (st == 0) ms.rescale = any;
        }
        softmax_sync();
        // ---- the previous chunk's product: W is free, and O may be rescaled
        if (c0 > 0) {
          mbar_wait(BAR(TB_PV), (chunk - 1) & 1, abort_flag);
          __syncwarp();
          tc_fence_after();
          if (ms.rescale) {
#pragma unroll
            for (int ob = 0; ob < L::OB; ++ob)
#pragma unroll
              for (int n0 = 0; n0 < RT; n0 += CB) {
                float o[CB];
                tmem_ld_cols(tmem + L::TM_O + ob * N + n0 + lane_off, o);
#pragma unroll
                for (int j = 0; j < CB; ++j) o[j] *= ms.ao[n0 + j];
                tmem_st_cols(tmem + L::TM_O + ob * N + n0 + lane_off, o);
              }
          }
        }
        // ---- weights
#pragma unroll
        for (int n0 = 0; n0 < RT; n0 += CB) {
#pragma unroll
          for (int j = 0; j < CB; ++j) l[n0 + j] *= ms.al[n0 + j];
#pragma unroll
          for (int i = 0; i < CT; ++i) {
            if (i < tiles) {
              float s[CB];
              tmem_ld_cols(tS + i * N + n0, s);
              const bool masked = (wk.tile0 + c0 + i + 1) * kTK > kmin;
              const uint32_t wrow = sW + i * kTerms * L::W_BLOCK;
#pragma unroll
              for (int j = 0; j < CB; j += 2) {
                float w[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int n = n0 + j + e;
                  const float x = s[j + e] * (ks[i] * ms.qs[n]);
                  float pr = ex2(x - ms.ms[n]);
                  w[e] = ex2(x + ev[i] - ms.mvs[n]);
                  if (masked && key0 + i * kTK >= ms.seen[n]) pr = w[e] = 0.f;
                  l[n] += pr;
                }
                const uint32_t c1 = to_e4m3x2(w[0], w[1]);
                const float2 f1 = from_e4m3x2(c1);
                const float r0 = w[0] - f1.x, r1 = w[1] - f1.y;
                const uint32_t c2 = to_e4m3x2(r0, r1);
                const float2 f2 = from_e4m3x2(c2);
                const uint32_t c3 = to_e4m3x2(r0 - f2.x, r1 - f2.y);
                const uint32_t a0 = wrow + swizzled<128>(n0 + j, key_in_tile);
                const uint32_t a1 = wrow + swizzled<128>(n0 + j + 1, key_in_tile);
                st_shared_u8(a0, c1 & 0xFFu);
                st_shared_u8(a1, c1 >> 8);
                st_shared_u8(a0 + L::W_BLOCK, c2 & 0xFFu);
                st_shared_u8(a1 + L::W_BLOCK, c2 >> 8);
                st_shared_u8(a0 + 2 * L::W_BLOCK, c3 & 0xFFu);
                st_shared_u8(a1 + 2 * L::W_BLOCK, c3 >> 8);
              }
            }
          }
        }
        // ---- stored rows past the last key: whatever they hold (NaN codes
        // among it) would meet a zero weight in the product, so they become
        // zeros once the tile has landed.
        const int last = wk.tile0 + c0 + tiles - 1;
        if ((last + 1) * kTK > kmax) {
          const int vi = tiles - 1;
          const unsigned int it = item0 + min(c0 + 2 * CT, nt) + c0 + vi;
          const int slot = it % NS;
          mbar_wait(BAR(TB_FULL + slot), (it / NS) & 1, abort_flag);
          if (last * kTK + key_in_tile >= kmax) {
            for (int kb = 0; kb < L::KB; ++kb)
              for (int x = 0; x < ROW; x += 16)
                st_shared_v4(sRing + slot * L::TILE + kb * L::BLOCK + key_in_tile * ROW + x, 0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(BAR(TB_W));
      }
      // ---- the segment's partial: O relative to m, and (m, l)
      const long long unit = (static_cast<long long>(wk.b) * p.Hkv + wk.g) * p.row_tiles + wk.rt;
      const long long slot_row = (unit + blockIdx.x) * RT;
      softmax_sync();   // wm is free
#pragma unroll
      for (int n = 0; n < RT; ++n) {
        float v = l[n];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) ms.wm[quarter][n] = v;
      }
      softmax_sync();
      if (st < rows)
        p.ml[slot_row + st] = make_float2(ms.m[st], (ms.wm[0][st] + ms.wm[1][st]) + (ms.wm[2][st] + ms.wm[3][st]));
      if (st < RT) ms.ao[st] = ms.mv[st] == -INFINITY ? 1.f : exp2f(ms.mvs[st] - ms.ms[st]);
      softmax_sync();
      mbar_wait(BAR(TB_PV), (chunk - 1) & 1, abort_flag);
      __syncwarp();
      tc_fence_after();
      if (D >= 128 || quarter < D / 32) {
#pragma unroll
        for (int ob = 0; ob < L::OB; ++ob)
#pragma unroll
          for (int n0 = 0; n0 < RT; n0 += CB) {
            float o[CB];
            tmem_ld_cols(tmem + L::TM_O + ob * N + n0 + lane_off, o);
            float* dst = p.o + (slot_row + n0) * D + ob * 128 + key_in_tile;
#pragma unroll
            for (int j = 0; j < CB; ++j)
              if (n0 + j < rows) dst[j * D] = o[j] * ms.ao[n0 + j];
          }
      }
      item0 += 2 * nt;
      wk.done(p);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, L::TM_COLS);
  if (threadIdx.x == 0 && ms.abort) atomicOr(p.err, kErrStreamTimeout);
}

// ---------------------------------------------------------------- the merge
// out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s over a row's partials:
// those of the shared store (O_s / l_s, pieces of eight fp32 values
// [D/8][128 rows]) and those of its tail.  kRowWarps warps share a row: warp w
// takes the partials w, w + kRowWarps, ..., kMergeChunk of them in flight, and
// the warps' sums meet in shared memory.
struct MergeParams {
  const float* shared_o;      // [unit][split][D/8][128][8]
  const float2* shared_ml;    // [unit][split][128]
  const unsigned long long* head;
  const float2* tail_ml;
  const float* tail_o;
  const int* tail_len;
  const int* n_new;
  __nv_bfloat16* out;
  int B, T, Hq, Hkv, G, tail_cap, row_tiles, RT;
  int splits, m_tiles, tail_ctas;
};

constexpr int kRowWarps = 4;
constexpr int kMergeRows = 2;      // rows of one CTA
constexpr int kMergeChunk = 8;

template <int D>
__global__ void __launch_bounds__(kMergeRows * kRowWarps * 32) stream_merge_kernel(const MergeParams p) {
  constexpr int E = D / 32;   // elements per lane
  __shared__ float sm[kMergeRows][kRowWarps], sl[kMergeRows][kRowWarps], so[kMergeRows][kRowWarps][D];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int mine = warp / kRowWarps, part = warp % kRowWarps;
  const long long rr = static_cast<long long>(blockIdx.x) * kMergeRows + mine;   // (b * T + t) * Hq + h
  bool live = rr < static_cast<long long>(p.B) * p.T * p.Hq;
  float M = -INFINITY, L = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  if (live) {
    const int h = static_cast<int>(rr % p.Hq);
    const long long bt = rr / p.Hq;
    const int t = static_cast<int>(bt % p.T), b = static_cast<int>(bt / p.T);
    const int g = h / p.G, gh = h % p.G;
    const unsigned long long C = p.head[0];
    unsigned long long first = p.head[1 + b];
    const StreamLen s = stream_len(p.tail_len, p.n_new, b, p.T, p.tail_cap);
    live = t < s.n;
    const long long row = bt * p.G + gh;   // row of the shared segment
    const long long su = (g * static_cast<long long>(p.m_tiles) + (row >> 7)) * p.splits;
    const int si = static_cast<int>(row & 127);
    const int r = t * p.G + gh, rt = r / p.RT;
    const int ut = live ? unit_tiles(s, rt, p.RT, p.G) : 0;
    long long tail_row = 0;   // the first tail partial's row
    int tails = 0;
    if (ut > 0) {
      const unsigned long long A = min(static_cast<unsigned long long>(p.tail_ctas), C);
      if (g > 0) first += g * head_tiles(s, p.row_tiles, p.RT, p.G);
      for (int k = 0; k < rt; ++k) first += unit_tiles(s, k, p.RT, p.G);
      const long long c0 = static_cast<long long>(cta_of_tile(first, C, A));
      tails = static_cast<int>(static_cast<long long>(cta_of_tile(first + ut - 1, C, A)) - c0) + 1;
      tail_row = ((static_cast<long long>(b) * p.Hkv + g) * p.row_tiles + rt + c0) * p.RT + r % p.RT;
    }
    const int count = live ? p.splits + tails : 0;
    for (int i0 = part; i0 < count; i0 += kRowWarps * kMergeChunk) {
      float2 ml[kMergeChunk];
      float v[kMergeChunk][E];
#pragma unroll
      for (int u = 0; u < kMergeChunk; ++u) {
        const int i = i0 + u * kRowWarps;
        ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int e = 0; e < E; ++e) v[u][e] = 0.f;
        if (i < count) {
          const bool shared = i < p.splits;
          const long long tr = tail_row + static_cast<long long>(i - p.splits) * p.RT;
          ml[u] = __ldcg(shared ? p.shared_ml + (su + i) * 128 + si : p.tail_ml + tr);
          const float* src = shared ? p.shared_o + (((su + i) * (D / 8) + lane * E / 8) * 128 + si) * 8 + lane * E % 8
                                    : p.tail_o + tr * D + lane * E;
#pragma unroll
          for (int e = 0; e < E; e += E < 4 ? 2 : 4) {
            if constexpr (E < 4) {
              const float2 x = __ldcg(reinterpret_cast<const float2*>(src + e));
              v[u][e] = x.x;
              v[u][e + 1] = x.y;
            } else {
              const float4 x = __ldcg(reinterpret_cast<const float4*>(src + e));
              v[u][e] = x.x;
              v[u][e + 1] = x.y;
              v[u][e + 2] = x.z;
              v[u][e + 3] = x.w;
            }
          }
        }
      }
      float Mn = M;
#pragma unroll
      for (int u = 0; u < kMergeChunk; ++u) Mn = fmaxf(Mn, ml[u].x);
      const float keep = M == -INFINITY ? 1.f : exp2f(M - Mn);   // 1: zeros (or NaN) so far
      L *= keep;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= keep;
#pragma unroll
      for (int u = 0; u < kMergeChunk; ++u) {
        // A sum without a maximum is zero, or NaN, which has to stay.
        const float f = ml[u].x == -INFINITY ? (ml[u].y == 0.f ? 0.f : 1.f) : exp2f(ml[u].x - Mn);
        const float wl = f * ml[u].y;
        const float w = i0 + u * kRowWarps < p.splits ? wl : f;
        L += wl;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(w, v[u][e], acc[e]);
      }
      M = Mn;
    }
  }
  if (lane == 0) {
    sm[mine][part] = M;
    sl[mine][part] = L;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) so[mine][part][lane * E + e] = acc[e];
  __syncthreads();
  if (!live) return;
  float Mt = -INFINITY, Lt = 0.f;
#pragma unroll
  for (int w = 0; w < kRowWarps; ++w) Mt = fmaxf(Mt, sm[mine][w]);
  float f[kRowWarps];
#pragma unroll
  for (int w = 0; w < kRowWarps; ++w) {
    f[w] = sm[mine][w] == -INFINITY ? 1.f : exp2f(sm[mine][w] - Mt);   // 1: zeros (or NaN)
    Lt += f[w] * sl[mine][w];
  }
  const float inv = Lt == 0.f ? 0.f : 1.f / Lt;   // a row with no key at all gets zeros
  // The row's D values over its kRowWarps * 32 threads.
  const int d0 = (part * 32 + lane) * 2;
  if (d0 < D) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
      x = fmaf(f[w], so[mine][w][d0], x);
      y = fmaf(f[w], so[mine][w][d0 + 1], y);
    }
    *reinterpret_cast<__nv_bfloat162*>(p.out + rr * D + d0) = __floats2bfloat162_rn(x * inv, y * inv);
  }
}

// ------------------------------------------------------------------ launches
template <int D, int RT>
cudaError_t launch_tails(TailParams& p, int num_sms, int* ctas, cudaStream_t s) {
  using L = TailLayout<D, RT>;
  const cudaError_t e = cudaFuncSetAttribute(stream_tail_kernel<D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC);
  if (e != cudaSuccess) return e;
  *ctas = num_sms * L::CTAS;
  return launch_k(stream_tail_kernel<D, RT>, dim3(*ctas), dim3(kTailThreads), L::ALLOC, s, p);
}

template <int D>
cudaError_t launch_tails_d(TailParams& p, int RT, int num_sms, int* ctas, cudaStream_t s) {
  switch (RT) {
    case 8: return launch_tails<D, 8>(p, num_sms, ctas, s);
    case 16: return launch_tails<D, 16>(p, num_sms, ctas, s);
    case 32: return launch_tails<D, 32>(p, num_sms, ctas, s);
    default: return launch_tails<D, 64>(p, num_sms, ctas, s);
  }
}

// Rows of a unit: the smallest of 8, 16, 32, 64 that holds one stream and
// head's T * G rows, or tiles of 64.
int unit_rows(long long rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// Partial rows: each unit has at most 2 * T * G rows (or 8), and each CTA adds
// one unit's.
size_t streams_quant_workspace(int max_req, int Hkv, int G, int D, int num_sms) {
  const size_t mine = static_cast<size_t>(unit_rows(static_cast<long long>(max_req) * G));
  const size_t rows = static_cast<size_t>(max_req) * Hkv * (2 * G > 8 ? 2 * G : 8) + 2 * static_cast<size_t>(num_sms) * mine;
  return up256((static_cast<size_t>(max_req) + 1) * 8) + up256(rows * 8) + up256(rows * D * 4);
}

cudaError_t launch_streams_quant(const QuantStreams& a, const AttnLaunch& al, size_t xchg_bytes, void* ws, int max_req,
                                 cudaStream_t s) {
  const int G = a.Hq / a.Hkv;
  const int RT = unit_rows(static_cast<long long>(a.T) * G);
  // 1. the shared store
  int splits = 0, m_tiles = 0;
  cudaError_t e = launch_attention_partials(al, a.q, a.B * a.T, xchg_bytes, s, &splits, &m_tiles);
  if (e != cudaSuccess) return e;
  // 2. the tails
  TailParams tp;
  memset(&tp, 0, sizeof(tp));
  const uint64_t dims[4] = {static_cast<uint64_t>(a.D), static_cast<uint64_t>(a.Hkv), static_cast<uint64_t>(a.tail_cap),
                            static_cast<uint64_t>(a.B)};
  const uint64_t strides[3] = {static_cast<uint64_t>(a.D), static_cast<uint64_t>(a.D) * a.Hkv,
                               static_cast<uint64_t>(a.D) * a.Hkv * a.tail_cap};
  const uint32_t box[4] = {static_cast<uint32_t>(a.D < 128 ? a.D : 128), 1u, static_cast<uint32_t>(kTK), 1u};
  if (!encode_tmap_u8_4d(&tp.tm_k, a.k_tail, dims, strides, box) || !encode_tmap_u8_4d(&tp.tm_v, a.v_tail, dims, strides, box))
    return cudaErrorInvalidValue;
  const size_t mine = static_cast<size_t>(unit_rows(static_cast<long long>(max_req) * G));
  const size_t rows = static_cast<size_t>(max_req) * a.Hkv * (2 * G > 8 ? 2 * G : 8) + 2 * static_cast<size_t>(al.num_sms) * mine;
  char* w = static_cast<char*>(ws);
  tp.head = reinterpret_cast<unsigned long long*>(w);
  w += up256((static_cast<size_t>(max_req) + 1) * 8);
  tp.ml = reinterpret_cast<float2*>(w);
  w += up256(rows * 8);
  tp.o = reinterpret_cast<float*>(w);
  tp.q = a.q;
  tp.k_exp = a.k_exp;
  tp.v_exp = a.v_exp;
  tp.tail_len = a.tail_len;
  tp.n_new = a.n_new;
  tp.err = al.err;
  tp.B = a.B;
  tp.T = a.T;
  tp.G = G;
  tp.Hkv = a.Hkv;
  tp.tail_cap = a.tail_cap;
  tp.row_tiles = (a.T * G + RT - 1) / RT;
  tp.inject_tx = al.inject_tx;
  tp.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(a.D)));
  int ctas = 0;
  switch (a.D) {
    case 64: e = launch_tails_d<64>(tp, RT, al.num_sms, &ctas, s); break;
    case 128: e = launch_tails_d<128>(tp, RT, al.num_sms, &ctas, s); break;
    case 256: e = launch_tails_d<256>(tp, RT, al.num_sms, &ctas, s); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess) return e;
  // 3. the merge
  MergeParams mp;
  memset(&mp, 0, sizeof(mp));
  const size_t units = static_cast<size_t>(m_tiles) * a.Hkv;
  mp.shared_o = static_cast<const float*>(al.xchg);
  mp.shared_ml = reinterpret_cast<const float2*>(static_cast<const char*>(al.xchg) + units * splits * 128 * a.D * 4);
  mp.head = tp.head;
  mp.tail_ml = tp.ml;
  mp.tail_o = tp.o;
  mp.tail_len = a.tail_len;
  mp.n_new = a.n_new;
  mp.out = a.out;
  mp.B = a.B;
  mp.T = a.T;
  mp.Hq = a.Hq;
  mp.Hkv = a.Hkv;
  mp.G = G;
  mp.tail_cap = a.tail_cap;
  mp.row_tiles = tp.row_tiles;
  mp.RT = RT;
  mp.splits = splits;
  mp.m_tiles = m_tiles;
  mp.tail_ctas = ctas;
  const long long out_rows = static_cast<long long>(a.B) * a.T * a.Hq;
  const dim3 grid(static_cast<unsigned int>((out_rows + kMergeRows - 1) / kMergeRows));
  const dim3 block(kMergeRows * kRowWarps * 32);
  switch (a.D) {
    case 64: e = launch_k(stream_merge_kernel<64>, grid, block, 0, s, mp); break;
    case 128: e = launch_k(stream_merge_kernel<128>, grid, block, 0, s, mp); break;
    default: e = launch_k(stream_merge_kernel<256>, grid, block, 0, s, mp); break;
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace rx
