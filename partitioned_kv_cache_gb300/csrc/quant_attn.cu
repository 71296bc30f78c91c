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
//      the partitioned attention kernel, which writes fp32 partials (behind a
//      copy of the ring's state where pushes may run meanwhile);
//   2. stream_tail_kernel: every tail against its own stream's rows, at the
//      same time (partition.h shares out the SMs);
//   3. stream_merge_kernel: one row's partials into its bf16 output.
//
// stream_tail_kernel.  A tail is read by the G * n_new rows of one stream and
// K/V head, so the keys are the M = 128 side of the tensor-core products and
// the rows the N side:
//   S^T [128 keys x N] = K [128 x D] . Q^T      (K codes as loaded)
//   O^T [D x N]       += V^T [D x 128] . W^T    (V codes as loaded, MN-major)
// and the codes go from TMA to kind::f8f6f4 products without a conversion.
// The bf16 queries and fp32 weights enter as sums of e4m3 terms whose products
// meet in fp32: a query row, scaled by a power of two, is hi + lo exactly (8
// significant bits in two 4-bit terms) down to 2^-9 of the row's largest entry,
// and within 2^-17 of that (half of lo's smallest step) below.  A weight
// is hi + mid/16 + lo/256, each term the e4m3 rounding of what is left, so it is
// within 2^-12 of its value, a sixteenth of a bf16 rounding (rounded to f16
// first it was within 2^-11, and 64 x 8 queries took 113.9 instead of 114.8 us
// over tails to 16384), or within 2^-23 of the largest weight that its row has so far (half of lo's
// smallest step, 2^-17, below a reference of 2^5; weights are compared with
// their values' scales).  Equal small weights beside a large one all lose the
// same, so a sum of products is closed after kSegment tiles: 16384 keys lose at
// most 2^-9 of the largest weight together.
//   x_jn = S_jn * 2^(k_exp_j - 127) * (row scale) * log2(e) / sqrt(D)
//   l_n  = sum_j 2^(x_jn - m_n),   w_jn = 2^(x_jn + v_exp_j - 127 - M_n + 5)
// m_n and M_n are running maxima of x_jn and of x_jn + v_exp_j - 127: the
// weights' own reference keeps them in the upper e4m3 range whatever the
// values' scales are.  (M_n is held as M_n - m_n: scores may be large enough to
// round an exponent away.)  Both are kept until some exponent outgrows them by
// 3.5 or more, which after a segment's first tile is rare.
//
// Work is cut into tiles of 128 keys of one (stream, K/V head, row tile) unit.
// The tiles of one head, all streams' in a row, are cut into equal runs
// (lengths are read on the device); a CTA takes one run of one head, and the
// CTAs next to it the same run of the other heads, so that what a stored token
// holds for all heads, side by side in memory, is read at about the same time
// (8 heads of 128: 6.0 TB/s, against 4.1 when one head's tiles followed the
// other's).  A run leaves one fp32 partial per unit that it touches, in its
// head's slot run + unit (distinct, because going on to a later run or a later
// unit never goes back in the other).  The scores of tile i + 1 are computed
// while tile i is in the softmax, and the weights have two buffers, so that a
// tile's softmax does not wait for the product before it unless a maximum grew.
//
// What bounds it, over 0.54 GB of tails: memory at few rows a unit (D = 256: 6.0,
// 5.8 and 5.75 TB/s at 8, 16 and 32 rows; D = 128: 6.0, 5.85 and 5.2; D = 64, 8
// rows: 5.4 to 5.8); the softmax warps' issue slots beyond (64 rows at D = 256:
// a tile takes 3100 cycles, 2400 of them theirs, where its bytes would take
// 2760, 4.3 TB/s; at D = 128 3.0; D = 64: 3.8 at 16 rows, 1.8 at 64, where a
// tile is 16 KB and its softmax the same); for small calls the chain of loads and
// the code's own arrival: one tile takes 7 us from the lengths to its partial.
//
// Warp roles: warp 0 = TMA producer, warp 1 = TMEM allocator and MMA issuer,
// the others = softmax and epilogue, in warpgroups of 4 warps that share up to
// 16 query rows (thread = key of the tile for S^T, output column for O^T; TMEM
// lane quarter = warp % 4).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "rx_internal.h"
#include "sm103_ptx.cuh"

namespace rx {
namespace {

constexpr int kTK = 128;            // keys per tile
constexpr int kTerms = 3;           // e4m3 terms of a weight, each standing for 1/16 of the one before
constexpr float kTermStep = 16.f;
constexpr int kExpAhead = 4;        // tiles ahead that scale exponents are fetched into L2
constexpr int kSegment = 128;       // most tiles of one unit that are summed under one pair of references
// log2 of a row's largest weight, in e4m3 units, where its reference is taken,
// and the most it may grow to before a new one is (448 is the largest code).
constexpr float kTop = 5.f;
constexpr float kRoom = 8.5f;
// A running maximum before any key: below every score, and finite, so that its
// differences need no care (2^(-inf - kNoMax) = 2^(kNoMax - m) = 0).
constexpr float kNoMax = -3.0e38f;

// ------------------------------------------------------------------- helpers
// 2^(byte - 127); byte 255 stands for NaN.
__device__ __forceinline__ float exp_scale(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two e4m3 codes -> fp32.
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  float2 f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
// Two fp32 values -> f16x2, and f16x2 -> two e4m3 codes.
__device__ __forceinline__ uint32_t to_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(v));
  return r;
}
// 16 (x - c) for e4m3 codes c of the f16x2 values x: exact.
__device__ __forceinline__ uint32_t e4m3x2_rest(uint32_t x, uint32_t c) {
  uint32_t f, r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(static_cast<uint16_t>(c)));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(f));
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(0x4C004C00u));
  return r;
}

// Column-wise combination over the warp's lanes of N values a lane, halving
// the values with each exchange: lane l gets that of column l / (32 / N).
// (A redux for each column took longer: 32 of them in each of 16 warps held up
// a segment's first tile by about 2 us.)
template <int N, typename Op>
__device__ __forceinline__ float across_lanes(const float (&in)[N], int lane, Op op) {
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = in[i];
  int off = 16;
#pragma unroll
  for (int n = N / 2; n > 0; n /= 2, off /= 2) {
    const bool upper = lane & off;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = upper ? v[i] : v[i + n];
      v[i] = op(upper ? v[i + n] : v[i], __shfl_xor_sync(0xffffffffu, give, off));
    }
  }
#pragma unroll
  for (; off > 0; off /= 2) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], off));
  return v[0];
}
struct MaxOp {   // NaN is passed over
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct SumOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

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

// Instruction descriptor, kind::f8f6f4 with e4m3 A/B and fp32 D; mn: both
// operands MN-major.
constexpr uint32_t idesc_e4m3_f32(int M, int N, bool mn) {
  return (1u << 4) | ((mn ? 3u : 0u) << 15) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// Shared-memory matrix descriptor with rows of ROW bytes, swizzled over their
// length: as sdesc_sw128, layout type 4 (SWIZZLE_64B) or 6 (SWIZZLE_32B) for
// rows of 64 or 32 bytes.
template <int ROW>
__device__ __forceinline__ uint64_t sdesc_rows(uint32_t saddr, uint32_t lbo_bytes) {
  uint64_t d = sdesc_sw128(saddr, lbo_bytes, 8 * ROW);
  if (ROW == 64) d ^= (2ull ^ 4ull) << 61;
  if (ROW == 32) d ^= (2ull ^ 6ull) << 61;
  return d;
}
// Its low word is (address / 16) | ..., so a step of n bytes adds n / 16 there.
__device__ __forceinline__ uint64_t desc_step(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }
// Keep the compiler from computing a loop's descriptors ahead of it, all of
// them at once: the registers are the softmax warps'.
__device__ __forceinline__ uint32_t here(uint32_t x) {
  asm volatile("" : "+r"(x));
  return x;
}
// Byte offset of byte c of row r in such a layout (rows of ROW bytes).
template <int ROW>
__device__ __forceinline__ uint32_t swizzled(uint32_t r, uint32_t c) {
  const uint32_t x = ROW == 128 ? (r & 7u) : ROW == 64 ? ((r >> 1) & 3u) : ((r >> 2) & 1u);
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
  int2* runs_of;              // [unit] the first and the last run with a tile of it
  float2* ml;                 // (m, l) [slot][RT]
  float* o;                   // [slot][RT][D], relative to m
  int* err;
  int B, T, Hkv, tail_cap;
  int gs;                     // log2 of the query heads per K/V head G
  int row_tiles;              // row tiles of one stream and head: ceil(T * G / RT)
  int heads;                  // heads taken side by side: CTA c has run c / heads of head c % heads (and every
  int runs;                   // heads-th one after it); runs of one head
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
__device__ __forceinline__ int unit_tiles(const StreamLen& s, int rt, int RT, int gs) {
  if (rt * RT >= s.n << gs) return 0;
  return (keys_seen(s, min(s.n - 1, (rt * RT + RT - 1) >> gs)) + kTK - 1) / kTK;
}
// Tiles of all row tiles of one stream and head.
__device__ __forceinline__ long long head_tiles(const StreamLen& s, int row_tiles, int RT, int gs) {
  long long c = 0;
  for (int rt = 0; rt < row_tiles; ++rt) c += unit_tiles(s, rt, RT, gs);
  return c;
}
// The first tile of CTA c of A, which share C tiles: floor(c * C / A).  With
// C = q A + r it is c q + floor(c r / A), in 32 bits but for the product (C is
// below 2^32 unless the tails fill memory many times over).
__device__ __forceinline__ unsigned long long first_tile(unsigned int c, unsigned long long C, unsigned int A) {
  if (C >> 32) return c * C / A;
  const unsigned int q = static_cast<unsigned int>(C) / A, r = static_cast<unsigned int>(C) - q * A;
  return static_cast<unsigned long long>(c) * q + c * r / A;
}

// Where a run starts: the stream, row tile and tile, the stream's lengths, and
// the run's tiles.
struct RunStart {
  int b, rt, skip;
  StreamLen s;
  long long left;
};
// A CTA's run of tiles, unit by unit, for each of its heads.  Every role walks
// it for itself.
struct Walk {
  int b, g, rt;         // the unit
  int skip;             // tiles of the unit before this run
  long long left;       // tiles of the run from here on
  StreamLen s;
  int tile0, ntiles;    // the segment: tiles [tile0, tile0 + ntiles) of the unit, kSegment at most

  __device__ __forceinline__ void begin(const RunStart& r) {
    b = r.b;
    rt = r.rt;
    skip = r.skip;
    s = r.s;
    left = r.left;
  }
  __device__ __forceinline__ bool next(const TailParams& p, const RunStart& r, int RT) {
    while (true) {
      while (left > 0 && b < p.B) {
        const int ut = unit_tiles(s, rt, RT, p.gs);
        if (ut > skip) {
          tile0 = skip;
          ntiles = static_cast<int>(min(static_cast<long long>(min(ut - skip, kSegment)), left));
          left -= ntiles;
          return true;
        }
        skip -= ut;
        advance(p);
      }
      g += p.heads;
      if (g >= p.Hkv) return false;
      begin(r);
      if (left <= 0) return false;
    }
  }
  __device__ __forceinline__ void advance(const TailParams& p) {
    if (++rt == p.row_tiles) {
      rt = 0;
      ++b;   // a run ends at the last tile, so b < B whenever tiles are left
      if (b < p.B) s = stream_len(p.tail_len, p.n_new, b, p.T, p.tail_cap);
    }
  }
  // After a segment.
  __device__ __forceinline__ void done() { skip += ntiles; }
  // Whether the run's segment before this one ended inside the same unit.
  __device__ __forceinline__ bool again(const RunStart& r) const {
    return tile0 != (b == r.b && rt == r.rt ? r.skip : 0);
  }
};

template <int D, int RT>
struct TailLayout {
  // The e4m3 terms of Q and W are further rows of one operand.  These products
  // are bound by their operands' way out of shared memory, 64 bytes a clock:
  // one of 128 x 32 codes with N rows takes about (4096 + 32 N) / 64 clocks
  // (measured: 96 at N = 64, 72 at N = 16), so the codes are read once for all
  // terms.  At 64 rows that leaves TMEM one tile's scores instead of two.
  static constexpr int NQ = 2 * RT;                       // MMA N of the scores
  static constexpr int SB = RT == 64 ? 1 : 2;             // tiles of scores
  static constexpr int NW = RT == 64 ? 3 * RT : 4 * RT;   // MMA N of the output (up to 32 rows a term's place is spare)
  static constexpr int WROW = RT == 64 ? RT : NW;         // bytes of a key's stored weights in one block
  static constexpr int CW = RT < 16 ? RT : 16;            // rows of one softmax warpgroup
  static constexpr int WG = RT / CW;                      // softmax warpgroups
  static constexpr int THREADS = 64 + 128 * WG;
  static constexpr int ROW = D < 128 ? D : 128;           // bytes of a stored row (one column block)
  static constexpr int KB = D / ROW;                      // column blocks of a tile
  static constexpr int TILE = kTK * D;
  static constexpr int BLOCK = kTK * ROW;                 // one column block of a tile
  static constexpr int OB = D == 256 ? 2 : 1;             // 128-row blocks of O^T
  static constexpr int TM_O = SB * NQ;                    // TMEM: scores, then O
  static constexpr int TM_USED = TM_O + OB * NW;
  static constexpr int TM_COLS = TM_USED <= 128 ? 128 : TM_USED <= 256 ? 256 : 512;
  static constexpr int CTAS = D == 256 || RT == 64 ? 1 : 2;   // per SM (StreamWorkspace counts on it)
  static constexpr int Q_BLOCK = NQ * ROW;                // one column block of Q
  static constexpr int Q_BYTES = KB * Q_BLOCK;
  static constexpr int W_BLOCK = WROW * kTK;              // [key][WROW]: all terms, or at 64 rows one
  static constexpr int W_BYTES = NW * kTK;                // a tile's weights; two tiles are kept
  static constexpr int MISC = RT == 64 ? 9728 : 5632;
  static constexpr int BUDGET = (CTAS == 1 ? 227 : 113) * 1024 - 1024;   // less the alignment slack
  static constexpr int NS_FIT = (BUDGET - Q_BYTES - 2 * W_BYTES - MISC) / TILE;
  static constexpr int NS = NS_FIT > 12 ? 12 : NS_FIT;    // ring slots of one K or V tile
  static constexpr int OFF_RING = 0;
  static constexpr int OFF_Q = NS * TILE;
  static constexpr int OFF_W = OFF_Q + Q_BYTES;
  static constexpr int OFF_MISC = OFF_W + 2 * W_BYTES;
  static constexpr int BYTES = OFF_MISC + MISC;
  static constexpr int ALLOC = BYTES + 1024;
  static_assert(NS >= 3, "ring depth");
  static_assert(TM_USED <= 512 / CTAS && TM_COLS <= 512 / CTAS, "tensor memory");
};

// The MISC area.
template <int RT>
struct TailMisc {
  unsigned long long bar[12 + 12 + 10];  // full, empty, Q ready, S full[2], W ready[2], PV done[2], drain, S read
  uint32_t tmem;
  int abort;
  RunStart start;
  long long scan[32];
  // (read four at a time)
  alignas(16) float qs[RT];              // 2^e of the query rows, times log2(e) / sqrt(D)
  int seen[RT];                          // tail keys each row sees
  alignas(16) float wm[2][4][RT], wv[2][4][RT];   // the warps' maxima, for even and odd tiles
  // Per softmax warp, for its warpgroup's rows: m, d = m - M + kTop, and the
  // last factors of l and O.
  alignas(16) float row[RT < 16 ? 4 : RT / 4][4][RT < 16 ? RT : 16];
};

enum : int { TB_FULL = 0, TB_EMPTY = 12, TB_Q = 24, TB_S = 25, TB_W = 27, TB_PV = 29, TB_DRAIN = 31, TB_SR = 32 };

__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ... and whether any of its threads' predicates holds.
__device__ __forceinline__ bool named_any(int id, int threads, bool mine) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(mine)), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

template <int D, int RT>
__global__ void __launch_bounds__(TailLayout<D, RT>::THREADS, TailLayout<D, RT>::CTAS)
    stream_tail_kernel(const __grid_constant__ TailParams p) {
  using L = TailLayout<D, RT>;
  constexpr int NS = L::NS, ROW = L::ROW, CW = L::CW, THREADS = L::THREADS;
  extern __shared__ uint8_t tail_smem[];
  const uint32_t raw = smem_u32(tail_smem);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = tail_smem + (base - raw);
  const uint32_t sRing = base + L::OFF_RING, sQ = base + L::OFF_Q, sW = base + L::OFF_W;
  static_assert(sizeof(TailMisc<RT>) <= L::MISC && L::OFF_MISC % 16 == 0, "misc area");
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
    mbar_init(BAR(TB_Q), 128 * L::WG);
    for (int i = 0; i < 2; ++i) {
      mbar_init(BAR(TB_S + i), 1);
      mbar_init(BAR(TB_W + i), 128 * L::WG);
      mbar_init(BAR(TB_PV + i), 1);
    }
    mbar_init(BAR(TB_DRAIN), 1);
    mbar_init(BAR(TB_SR), 128 * L::WG);
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
  // The query rows are fetched into L2, an equal part by each CTA, before the
  // tiles' copies fill the memory's queues: behind those a row took 3 to 5 us.
  // (A hint with no effect on what a load returns: safe before the wait.)
  {
    const long long bytes = (static_cast<long long>(p.B) * p.T * p.Hkv << p.gs) * D * 2;
    const long long part = (bytes / gridDim.x + 127) / 128 * 128;
    for (long long at = blockIdx.x * part + threadIdx.x * 128ll; at < min(bytes, (blockIdx.x + 1) * part); at += THREADS * 128ll)
      prefetch_l2(reinterpret_cast<const char*>(p.q) + at);
  }
  grid_dependency_wait();
  grid_launch_dependents();

  // ------------------------------------------------------ this CTA's tiles
  // Tiles of one head before each stream, by a scan over the block's threads,
  // THREADS streams a round; with more streams a second sweep finds the run's
  // first.
  {
    // One round over the streams from b0 on; returns the carry after it.
    auto scan_round = [&](int b0, long long carry, long long* mine) {
      const int b = b0 + threadIdx.x;
      const int warps = (min(p.B - b0, THREADS) + 31) / 32;   // that have a stream
      long long c = 0;
      if (b < p.B) c = head_tiles(stream_len(p.tail_len, p.n_new, b, p.T, p.tail_cap), p.row_tiles, RT, p.gs);
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
#pragma unroll 1
      for (int w = 0; w < warps; ++w) {
        if (w < warp) before += ms.scan[w];
        total += ms.scan[w];
      }
      mine[0] = before + inc - c;
      mine[1] = c;
      return total;
    };
    long long mine[2], total = 0;
    for (int b0 = 0; b0 < p.B; b0 += THREADS) total = scan_round(b0, total, mine);
    const unsigned long long C = static_cast<unsigned long long>(total);
    const unsigned int A = static_cast<unsigned int>(min(static_cast<unsigned long long>(p.runs), C));
    const unsigned int run = blockIdx.x / p.heads;
    const bool active = run < A;
    const long long first = active ? static_cast<long long>(first_tile(run, C, A)) : 0;
    if (threadIdx.x == 0) ms.start.left = active ? static_cast<long long>(first_tile(run + 1, C, A)) - first : 0;
    long long carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += THREADS) {
      const int b = b0 + threadIdx.x;
      if (p.B > THREADS) carry = scan_round(b0, carry, mine);
      if (b < p.B && active && first >= mine[0] && first < mine[0] + mine[1]) {
        long long off = first - mine[0];
        const StreamLen s = stream_len(p.tail_len, p.n_new, b, p.T, p.tail_cap);
        int rt = 0;
        for (int ut; off >= (ut = unit_tiles(s, rt, RT, p.gs)); ++rt) off -= ut;
        ms.start.b = b;
        ms.start.rt = rt;
        ms.start.skip = static_cast<int>(off);
        ms.start.s = s;
      }
    }
    __syncthreads();
  }
  Walk wk;
  wk.g = blockIdx.x % p.heads;
  wk.left = ms.start.left;
  if (wk.left > 0) wk.begin(ms.start); else wk.g = p.Hkv;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // Per segment: K_0, then K_{i+1} and V_i in turn, the order in which the
    // MMA issuer takes them.
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
      while (!stop && wk.next(p, ms.start, RT)) {
        load(&p.tm_k, wk.tile0);
        for (int i = 0; i < wk.ntiles && !stop; ++i) {
          if (i + 1 < wk.ntiles) load(&p.tm_k, wk.tile0 + i + 1);
          if (!stop) load(&p.tm_v, wk.tile0 + i);
        }
        wk.done();
      }
      // Every copy issued must land before the CTA exits, even after an abort.
      volatile int no_abort = 0;
      for (unsigned int it = item > NS ? item - NS : 0; it < item; ++it)
        mbar_wait(BAR(TB_FULL + it % NS), (it / NS) & 1, &no_abort);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t kIdescS = idesc_e4m3_f32(kTK, L::NQ, false);
      constexpr uint32_t kIdescO = idesc_e4m3_f32(128, L::NW, true);
      unsigned int item = 0, tile = 0, seg = 0;
      bool ok = true;
      auto scores = [&](unsigned int t) {   // S^T of the tile whose K is the next item
        const int slot = item % NS;
        if (!mbar_wait(BAR(TB_FULL + slot), (item / NS) & 1, abort_flag)) {
          ok = false;
          return;
        }
        tc_fence_after();
        const uint64_t kd = sdesc_rows<ROW>(here(sRing + slot * L::TILE), 16);
        const uint64_t qd = sdesc_rows<ROW>(here(sQ), 16);
        const uint32_t acc = here(tmem + t % L::SB * L::NQ);
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) {
          const uint32_t kb = kk * 32 / ROW, ko = kk * 32 % ROW;
          umma_e4m3(acc, desc_step(kd, kb * L::BLOCK + ko), desc_step(qd, kb * L::Q_BLOCK + ko), kIdescS, kk ? 1u : 0u);
        }
        umma_commit(BAR(TB_EMPTY + slot));
        umma_commit(BAR(TB_S + t % L::SB));
        ++item;
      };
      while (ok && wk.next(p, ms.start, RT)) {
        if (!mbar_wait(BAR(TB_Q), seg & 1, abort_flag)) break;
        tc_fence_after();
        scores(tile);
        for (int i = 0; i < wk.ntiles && ok; ++i, ++tile) {
          // Of two S buffers, the next tile's was read before W of tile - 1 was
          // ready; a single one is free when this tile's scores are read.
          if (i + 1 < wk.ntiles) {
            if (L::SB == 1 && !mbar_wait(BAR(TB_SR), tile & 1, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            scores(tile + 1);
          }
          const int slot = item % NS;
          if (!ok || !mbar_wait(BAR(TB_W + (tile & 1)), (tile >> 1) & 1, abort_flag) ||
              !mbar_wait(BAR(TB_FULL + slot), (item / NS) & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // A: V codes, D along the stored rows (MN-major), 8-key groups
          // 8 * ROW apart.  At D = 64 the product's upper 64 rows read the
          // bytes one tile further on and are not used.
          const uint64_t vd = sdesc_rows<ROW>(here(sRing + slot * L::TILE), L::BLOCK);
          // B: weights, rows n along the stored bytes of a key, likewise (at
          // 64 rows, three blocks of them).
          const uint64_t wd = sdesc_rows<L::WROW>(here(sW + (tile & 1) * L::W_BYTES), L::W_BLOCK);
          const uint32_t acc = here(tmem + L::TM_O);
#pragma unroll
          for (int ob = 0; ob < L::OB; ++ob)
#pragma unroll
            for (int kk = 0; kk < kTK / 32; ++kk)
              umma_e4m3(acc + ob * L::NW, desc_step(vd, ob * L::BLOCK + kk * 32 * ROW),
                        desc_step(wd, kk * 32 * L::WROW), kIdescO, (i | kk) ? 1u : 0u);
          umma_commit(BAR(TB_EMPTY + slot));
          umma_commit(BAR(TB_PV + (tile & 1)));
          ++item;
        }
        wk.done();
        ++seg;
      }
      // No tensor-core work may be in flight when TMEM is released.
      umma_commit(BAR(TB_DRAIN));
      volatile int no_abort = 0;
      mbar_wait(BAR(TB_DRAIN), 0, &no_abort);
    }
  } else {
    // ------------------------------------------------- softmax and epilogue
    // Warpgroup wg has the rows n0 .. n0 + CW - 1; a thread one key of the tile
    // for all of them (TMEM lane = key), and at the end one output column.
    // After a wait that gave up the loops run on (their waits return at once)
    // so that the warps meet at every barrier; the results are void and the
    // error bit says so.
    const int quarter = warp & 3;
    const int st = threadIdx.x - 64;
    const int wg = st >> 7;
    const int n0 = wg * CW;
    const int in_wg = st & 127;
    const int key_in_tile = quarter * 32 + lane;            // TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    float (&row)[4][CW] = ms.row[st >> 5];
    unsigned int item0 = 0, tile = 0;
    if (L::NW > kTerms * RT)   // the spare rows of W stay zero
      for (int i = st * 16; i < 2 * L::W_BYTES; i += 128 * L::WG * 16) st_shared_v4(sW + i, 0u, 0u, 0u, 0u);
    while (wk.next(p, ms.start, RT)) {
      const int nt = wk.ntiles;
      const int row0 = wk.rt * RT;
      const int rows = min(RT, (wk.s.n << p.gs) - row0);        // rows with a query token
      const int kmax = keys_seen(wk.s, min(wk.s.n - 1, (row0 + RT - 1) >> p.gs));   // keys any row sees
      const int kmin = keys_seen(wk.s, row0 >> p.gs);                               // ... every row sees
      // The exponents of a thread's key, loaded a tile ahead of their use.
      const long long exp_base = (static_cast<long long>(wk.b) * p.tail_cap) * p.Hkv + wk.g;
      uint32_t kb, vb;
      auto load_exps = [&](int key) {
        kb = vb = 0;
        if (key < kmax) {
          const long long at = exp_base + static_cast<long long>(key) * p.Hkv;
          kb = p.k_exp[at];
          vb = p.v_exp[at];
        }
      };
      // ... and fetched into L2 some tiles before that: behind the tiles'
      // copies a load from DRAM takes longer than a tile.
      auto fetch_exps = [&](int tile_in_unit) {
        const int key = tile_in_unit * kTK + key_in_tile;
        if (wg == 0 && tile_in_unit < wk.tile0 + nt && key < kmax) {
          const long long at = exp_base + static_cast<long long>(key) * p.Hkv;
          prefetch_l2(p.k_exp + at);
          prefetch_l2(p.v_exp + at);
        }
      };
      load_exps(wk.tile0 * kTK + key_in_tile);
      for (int a = 1; a < kExpAhead; ++a) fetch_exps(wk.tile0 + a);
      named_sync(8, 128 * L::WG);   // the previous segment's row state is no longer read
      if (st < RT) ms.seen[st] = st < rows ? keys_seen(wk.s, (row0 + st) >> p.gs) : 0;
      // Q rows: 2^-e q = hi + lo, e as the append chooses it; the next row is
      // loaded while one is converted.
      {
        constexpr int E = D / 32;
        uint32_t ahead[E / 2];
        auto load_row = [&](int n) {
#pragma unroll
          for (int e = 0; e < E / 2; ++e) ahead[e] = 0u;
          if (n >= rows) return;
          const int r = row0 + n;
          const long long token = static_cast<long long>(wk.b) * p.T + (r >> p.gs);
          const __nv_bfloat16* src = p.q + (((token * p.Hkv + wk.g) << p.gs) + (r & ((1 << p.gs) - 1))) * D + lane * E;
          if constexpr (E == 8) {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(src));
            ahead[0] = x.x, ahead[1] = x.y, ahead[2] = x.z, ahead[3] = x.w;
          } else if constexpr (E == 4) {
            const uint2 x = __ldg(reinterpret_cast<const uint2*>(src));
            ahead[0] = x.x, ahead[1] = x.y;
          } else {
            ahead[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
          }
        };
        load_row(st >> 5);
#pragma unroll 1
        for (int n = st >> 5; n < RT; n += 4 * L::WG) {
          uint32_t w32[E / 2];
#pragma unroll
          for (int e = 0; e < E / 2; ++e) w32[e] = ahead[e];
          load_row(n + 4 * L::WG);
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < E / 2; ++e) top = max(top, max(w32[e] & 0x7FFFu, (w32[e] >> 16) & 0x7FFFu));
          top = __reduce_max_sync(0xffffffffu, top);
          const int ex = max(static_cast<int>(top >> 7) - 8 + ((top & 0x7Fu) > 96u ? 1 : 0), 1);
          const bool poison = (top >> 7) == 255u;
          if (lane == 0)
            ms.qs[n] = poison ? __uint_as_float(0x7FC00000u) : __uint_as_float(static_cast<uint32_t>(ex) << 23) * p.scale_log2;
          const float up = __uint_as_float(static_cast<uint32_t>(254 - min(ex, 253)) << 23);
          uint32_t hi[E / 2], lo[E / 2];
#pragma unroll
          for (int e = 0; e < E / 2; ++e) {
            const float a = poison ? 0.f : __uint_as_float(w32[e] << 16) * up;
            const float b = poison ? 0.f : __uint_as_float(w32[e] & 0xFFFF0000u) * up;
            hi[e] = to_e4m3x2(a, b);
            const float2 h = from_e4m3x2(hi[e]);
            lo[e] = to_e4m3x2(a - h.x, b - h.y);
          }
          // (a term's rows are a multiple of 8, so they keep the row's swizzle)
          const uint32_t d = static_cast<uint32_t>(lane * E);
          const uint32_t at = sQ + (d / ROW) * L::Q_BLOCK + swizzled<ROW>(n, d % ROW);
          if constexpr (E == 8) {
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(hi[0] | hi[1] << 16), "r"(hi[2] | hi[3] << 16) : "memory");
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + RT * ROW), "r"(lo[0] | lo[1] << 16), "r"(lo[2] | lo[3] << 16) : "memory");
          } else if constexpr (E == 4) {
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(hi[0] | hi[1] << 16) : "memory");
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + RT * ROW), "r"(lo[0] | lo[1] << 16) : "memory");
          } else {
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(static_cast<uint16_t>(hi[0])) : "memory");
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + RT * ROW), "h"(static_cast<uint16_t>(lo[0])) : "memory");
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();   // the previous segment's reads of O
      mbar_arrive(BAR(TB_Q));
      named_sync(8, 128 * L::WG);      // row state visible

      float l[CW];
#pragma unroll
      for (int j = 0; j < CW; ++j) l[j] = 0.f;
      float m = kNoMax, mv = 0.f;   // lane j < CW: row n0 + j's m and M - m
      float dmax = 0.f;                // the largest d
      if (lane < CW) {
        row[0][lane] = kNoMax;
        row[1][lane] = 0.f;
      }
      __syncwarp();
      for (int i = 0; i < nt; ++i, ++tile) {
        const int buf = tile & 1;
        const int key = (wk.tile0 + i) * kTK + key_in_tile;
        // A NaN value poisons the scores of the rows that see it, as a NaN key
        // does: the whole row is NaN either way, and ev stays finite.
        const float ks = exp_scale(vb == 255u ? 255u : kb);
        const float ev = static_cast<float>(vb) - 127.f;
        load_exps(i + 1 < nt ? key + kTK : kmax);   // the next tile's, a tile ahead
        fetch_exps(wk.tile0 + i + kExpAhead);
        const bool masked = (wk.tile0 + i + 1) * kTK > kmin;
        mbar_wait(BAR(TB_S + tile % L::SB), tile / L::SB & 1, abort_flag);
        __syncwarp();
        tc_fence_after();
        // x_n - c_n for this key and the warpgroup's rows; c: an array in shared memory.
        auto scores_less = [&](float (&x)[CW], const float* c) {
          const uint32_t at = tmem + tile % L::SB * L::NQ + n0 + lane_off;
          float lo[CW];
          tmem_ld_cols(at, x);
          tmem_ld_cols(at + RT, lo);
#pragma unroll
          for (int j = 0; j < CW; ++j) x[j] += lo[j];
#pragma unroll
          for (int j = 0; j < CW; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(&ms.qs[n0 + j]);
            const float4 g = c ? *reinterpret_cast<const float4*>(c + j) : make_float4(0.f, 0.f, 0.f, 0.f);
            x[j] = fmaf(x[j], ks * f.x, -g.x);
            x[j + 1] = fmaf(x[j + 1], ks * f.y, -g.y);
            x[j + 2] = fmaf(x[j + 2], ks * f.z, -g.z);
            x[j + 3] = fmaf(x[j + 3], ks * f.w, -g.w);
          }
          if (masked) {
#pragma unroll
            for (int j = 0; j < CW; ++j)
              if (key >= ms.seen[n0 + j]) x[j] = -INFINITY;
          }
        };
        // ---- references: those of the tile before serve while no exponent
        // rises above kRoom (weights up to 2^kRoom fit e4m3).  The largest
        // x - m of the thread's key, its value's exponent and the largest row
        // offset d bound them all; only where that bound fails the rows are
        // looked at one by one.  The first tile of a segment always takes
        // new references.
        float u[CW];
        scores_less(u, row[0]);
        float top = u[0];
#pragma unroll
        for (int j = 1; j < CW; ++j) top = fmaxf(top, u[j]);
        bool over = top > kRoom || top + (ev + dmax) > kRoom;
        if (__any_sync(0xffffffffu, over)) {
          float t = -INFINITY;
#pragma unroll
          for (int j = 0; j < CW; ++j) t = fmaxf(t, u[j] + row[1][j]);
          over = top > kRoom || t + ev > kRoom;
        }
        if (named_any(1 + wg, 128, over)) {
          // The tile's maxima: over the warp's keys, then over the four warps,
          // lane j for row n0 + j.  Those of the values' exponents are taken
          // beside what the scores lie below their maximum (the warp's, then
          // the new one): beside a score of 2^24 or more they would be rounded
          // away.  (A column without a key in this warp: -inf and NaN, which
          // the maxima pass over.)
          scores_less(u, nullptr);
          float* wm = &ms.wm[buf][quarter][n0];
          const float hx = across_lanes(u, lane, MaxOp());
          if (lane % (32 / CW) == 0) wm[lane / (32 / CW)] = hx;
          __syncwarp();
          float y[CW];
#pragma unroll
          for (int j = 0; j < CW; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(&wm[j]);
            y[j] = u[j] - f.x + ev;
            y[j + 1] = u[j + 1] - f.y + ev;
            y[j + 2] = u[j + 2] - f.z + ev;
            y[j + 3] = u[j + 3] - f.w + ev;
          }
          const float hy = across_lanes(y, lane, MaxOp());
          if (lane % (32 / CW) == 0) ms.wv[buf][quarter][n0 + lane / (32 / CW)] = hy;
          named_sync(1 + wg, 128);
          float mn = m, vn = mv;
          if (lane < CW) {
#pragma unroll
            for (int w = 0; w < 4; ++w) mn = fmaxf(mn, ms.wm[buf][w][n0 + lane]);
            vn += m - mn;   // a row without a key so far: 0
#pragma unroll
            for (int w = 0; w < 4; ++w) vn = fmaxf(vn, ms.wv[buf][w][n0 + lane] + (ms.wm[buf][w][n0 + lane] - mn));
            row[0][lane] = mn;
            row[1][lane] = kTop - vn;
            row[2][lane] = ex2(m - mn);
            row[3][lane] = ex2((m - mn) + (mv - vn));
          }
          dmax = lane < CW ? kTop - vn : -INFINITY;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) dmax = fmaxf(dmax, __shfl_xor_sync(0xffffffffu, dmax, o));
          m = mn;
          mv = vn;
          __syncwarp();
#pragma unroll
          for (int j = 0; j < CW; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(&row[2][j]);
            const float4 g = *reinterpret_cast<const float4*>(&row[0][j]);
            l[j] *= f.x;
            l[j + 1] *= f.y;
            l[j + 2] *= f.z;
            l[j + 3] *= f.w;
            u[j] -= g.x;
            u[j + 1] -= g.y;
            u[j + 2] -= g.z;
            u[j + 3] -= g.w;
          }
          if (i > 0) {
            // O holds the tiles before: wait for their last product, then rescale.
            mbar_wait(BAR(TB_PV + (buf ^ 1)), ((tile - 1) >> 1) & 1, abort_flag);
            __syncwarp();
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < L::OB * kTerms; ++c) {
              const uint32_t at = tmem + L::TM_O + (c % L::OB) * L::NW + (c / L::OB) * RT + n0 + lane_off;
              float o[CW];
              tmem_ld_cols(at, o);
#pragma unroll
              for (int j = 0; j < CW; ++j) o[j] *= row[3][j];
              tmem_st_cols(at, o);
            }
          }
        }
        if (L::SB == 1) {   // the next tile's scores may take this one's place
          tc_fence_before();
          mbar_arrive(BAR(TB_SR));
        }
        // ---- weights, once the product that read this W buffer is done
        if (i > 1) {
          mbar_wait(BAR(TB_PV + buf), ((tile - 2) >> 1) & 1, abort_flag);
          __syncwarp();
        }
        uint32_t codes[kTerms][CW / 4];
#pragma unroll
        for (int j = 0; j < CW; j += 4) {
          const float4 d4 = *reinterpret_cast<const float4*>(&row[1][j]);
          const float dj[4] = {d4.x, d4.y, d4.z, d4.w};
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            l[j + e] += ex2(u[j + e]);
            w[e] = ex2(u[j + e] + ev + dj[e]);
          }
          // Each term is what e4m3 left of the weight so far, 16 times larger;
          // what the first left fits f16's 11 bits but for 2^-15 of the weight.
          const uint32_t c01 = to_e4m3x2(w[0], w[1]), c23 = to_e4m3x2(w[2], w[3]);
          codes[0][j / 4] = c01 | c23 << 16;
          const float2 f01 = from_e4m3x2(c01), f23 = from_e4m3x2(c23);
          uint32_t h01 = to_f16x2((w[0] - f01.x) * kTermStep, (w[1] - f01.y) * kTermStep);
          uint32_t h23 = to_f16x2((w[2] - f23.x) * kTermStep, (w[3] - f23.y) * kTermStep);
#pragma unroll
          for (int term = 1; term < kTerms; ++term) {
            const uint32_t d01 = f16x2_to_e4m3x2(h01), d23 = f16x2_to_e4m3x2(h23);
            codes[term][j / 4] = d01 | d23 << 16;
            if (term + 1 < kTerms) {
              h01 = e4m3x2_rest(h01, d01);
              h23 = e4m3x2_rest(h23, d23);
            }
          }
        }
        // The CW bytes of each term side by side in the key's stored row.
        const uint32_t wb = sW + buf * L::W_BYTES;
#pragma unroll
        for (int term = 0; term < kTerms; ++term) {
          const uint32_t at = wb + (L::WROW == L::NW ? swizzled<L::WROW>(key_in_tile, term * RT + n0)
                                                     : term * L::W_BLOCK + swizzled<L::WROW>(key_in_tile, n0));
          if constexpr (CW == 16)
            st_shared_v4(at, codes[term][0], codes[term][1], codes[term][2], codes[term][3]);
          else
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(codes[term][0]), "r"(codes[term][1]) : "memory");
        }
        // ---- stored rows past the last key: whatever they hold (NaN codes
        // among it) would meet a zero weight in the product, so they become
        // zeros once the tile has landed.
        if (wg == 0 && (wk.tile0 + i + 1) * kTK > kmax) {
          const unsigned int it = item0 + min(i + 2, nt) + i;   // K_0, then K_{i+1} and V_i in turn
          const int slot = it % NS;
          mbar_wait(BAR(TB_FULL + slot), (it / NS) & 1, abort_flag);
          if (key >= kmax) {
#pragma unroll 1
            for (int c = 0; c < L::KB; ++c)
#pragma unroll
              for (int y = 0; y < ROW; y += 16)
                st_shared_v4(sRing + slot * L::TILE + c * L::BLOCK + key_in_tile * ROW + y, 0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(BAR(TB_W + buf));
      }
      // ---- the segment's partial: O relative to m, and (m, l)
      const int run = blockIdx.x / p.heads;
      const long long in_head = static_cast<long long>(wk.b) * p.row_tiles + wk.rt;   // the unit among its head's
      const long long slot_row = (wk.g * (static_cast<long long>(p.B) * p.row_tiles + p.runs) + in_head + run) * RT + n0;
      if (st == 0) {
        int2* r = p.runs_of + (static_cast<long long>(wk.b) * p.Hkv + wk.g) * p.row_tiles + wk.rt;
        if (wk.tile0 == 0) r->x = run;
        if (wk.tile0 + nt == unit_tiles(wk.s, wk.rt, RT, p.gs)) r->y = run;
      }
      auto finish = [&](auto more) {
        constexpr bool again = decltype(more)::value;
        named_sync(1 + wg, 128);   // wm is free
        const float sum = across_lanes(l, lane, SumOp());
        if (lane % (32 / CW) == 0) ms.wm[0][quarter][n0 + lane / (32 / CW)] = sum;
        const float top = m == kNoMax ? -INFINITY : m;
        float all = top, before = 0.f;
        if (lane < CW) row[2][lane] = exp2f(mv - kTop);   // O's reference to m
        // A segment that goes on from another adds to what that one left, which
        // this thread (or for (m, l) its warpgroup) has written.
        if (again && lane < CW) {
          const float2 old = n0 + lane < rows ? p.ml[slot_row + lane] : make_float2(-INFINITY, 0.f);
          all = fmaxf(top, old.x);
          // A sum without a maximum is zero, or NaN, which has to stay.
          const float f = top == -INFINITY ? 1.f : exp2f(top - all);
          const float g = old.x == -INFINITY ? 1.f : exp2f(old.x - all);
          before = old.y * g;
          row[2][lane] *= f;
          row[3][lane] = g;
          row[0][lane] = f;
        }
        named_sync(1 + wg, 128);
        if (in_wg < CW && n0 + in_wg < rows) {
          const float here = (ms.wm[0][0][n0 + in_wg] + ms.wm[0][1][n0 + in_wg]) + (ms.wm[0][2][n0 + in_wg] + ms.wm[0][3][n0 + in_wg]);
          p.ml[slot_row + in_wg] = make_float2(all, again ? fmaf(here, row[0][in_wg], before) : here);
        }
        mbar_wait(BAR(TB_PV + ((tile - 1) & 1)), ((tile - 1) >> 1) & 1, abort_flag);
        __syncwarp();
        tc_fence_after();
        if (D >= 128 || quarter < D / 32) {
#pragma unroll 1
          for (int ob = 0; ob < L::OB; ++ob) {
            float o[CW];
            const uint32_t at = tmem + L::TM_O + ob * L::NW + n0 + lane_off;
            tmem_ld_cols(at, o);
#pragma unroll
            for (int term = 1; term < kTerms; ++term) {
              float t[CW];
              tmem_ld_cols(at + term * RT, t);
              const float f = term == 1 ? 1.f / kTermStep : 1.f / (kTermStep * kTermStep);
#pragma unroll
              for (int j = 0; j < CW; ++j) o[j] = fmaf(t[j], f, o[j]);
            }
            float* dst = p.o + slot_row * D + ob * 128 + key_in_tile;
#pragma unroll
            for (int j = 0; j < CW; ++j) o[j] *= row[2][j];
            if (again) {
#pragma unroll
              for (int j = 0; j < CW; ++j)
                if (n0 + j < rows) o[j] = fmaf(dst[j * D], row[3][j], o[j]);
            }
#pragma unroll
            for (int j = 0; j < CW; ++j)
              if (n0 + j < rows) dst[j * D] = o[j];
          }
        }
      };
      if (wk.again(ms.start)) finish(std::true_type());   // (a copy of its own: most runs have none)
      else finish(std::false_type());
      item0 += 2 * nt;
      wk.done();
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
// [D/8][128 rows]) and those of its tail.  WPR warps share a row: warp w takes
// the partials w, w + WPR, ..., kMergeChunk of them in flight, and the warps'
// sums meet in shared memory.  Bound by the latency of dependent loads: the
// unit's runs, then its partials.
struct MergeParams {
  const float* shared_o;      // [unit][split][D/8][128][8]
  const float2* shared_ml;    // [unit][split][128]
  const int2* runs_of;
  const float2* tail_ml;
  const float* tail_o;
  const int* tail_len;
  const int* n_new;
  __nv_bfloat16* out;
  int rows;                   // B * T * Hq
  int T, Hq, Hkv, gs, tail_cap, row_tiles, RT;
  int splits, m_tiles;
  int head_slots;             // partial slots of one head: its units and runs
};

constexpr int kMergeWarps = 8;
constexpr int kMergeChunk = 8;

template <int D, int WPR>
__global__ void __launch_bounds__(kMergeWarps * 32) stream_merge_kernel(const MergeParams p) {
  constexpr int E = D / 32;   // elements per lane
  constexpr int ROWS = kMergeWarps / WPR;
  __shared__ float sm[ROWS][WPR], sl[ROWS][WPR], so[ROWS][WPR][WPR > 1 ? D : 1];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int mine = warp / WPR, part = warp % WPR;
  const int rr = blockIdx.x * ROWS + mine;   // (b * T + t) * Hq + h
  bool live = rr < p.rows;
  float M = -INFINITY, L = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  if (live) {
    const int bt = rr / p.Hq, h = rr - bt * p.Hq;
    const int b = bt / p.T, t = bt - b * p.T;
    const int g = h >> p.gs, gh = h & ((1 << p.gs) - 1);
    const int r = (t << p.gs) + gh, rt = r / p.RT;
    const int unit = (b * p.Hkv + g) * p.row_tiles + rt;
    const int2 runs = __ldcg(p.runs_of + unit);   // (read beside the lengths; used only where the unit has tiles)
    const StreamLen s = stream_len(p.tail_len, p.n_new, b, p.T, p.tail_cap);
    live = t < s.n;
    const int ut = live ? unit_tiles(s, rt, p.RT, p.gs) : 0;
    const int tails = ut > 0 ? runs.y - runs.x + 1 : 0;
    const long long tail_row =   // the first tail partial's row
        (static_cast<long long>(g) * p.head_slots + b * p.row_tiles + rt + runs.x) * p.RT + r % p.RT;
    const int row = (bt << p.gs) + gh;             // row of the shared segment
    const long long su = (g * static_cast<long long>(p.m_tiles) + (row >> 7)) * p.splits;
    const int si = row & 127;
    const int count = live ? p.splits + tails : 0;
    for (int i0 = part; i0 < count; i0 += WPR * kMergeChunk) {
      float2 ml[kMergeChunk];
      float v[kMergeChunk][E];
#pragma unroll
      for (int u = 0; u < kMergeChunk; ++u) {
        const int i = i0 + u * WPR;
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
        const float w = i0 + u * WPR < p.splits ? wl : f;
        L += wl;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(w, v[u][e], acc[e]);
      }
      M = Mn;
    }
  }
  if constexpr (WPR == 1) {
    if (!live) return;
    const float inv = L == 0.f ? 0.f : 1.f / L;   // a row with no key at all gets zeros
    __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(p.out + static_cast<long long>(rr) * D + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
  } else {
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
    for (int w = 0; w < WPR; ++w) Mt = fmaxf(Mt, sm[mine][w]);
    float f[WPR];
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      f[w] = sm[mine][w] == -INFINITY ? 1.f : exp2f(sm[mine][w] - Mt);   // 1: zeros (or NaN)
      Lt += f[w] * sl[mine][w];
    }
    const float inv = Lt == 0.f ? 0.f : 1.f / Lt;
    // The row's D values over its WPR * 32 threads.
    const int d0 = (part * 32 + lane) * 2;
    if (d0 < D) {
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) {
        x = fmaf(f[w], so[mine][w][d0], x);
        y = fmaf(f[w], so[mine][w][d0 + 1], y);
      }
      *reinterpret_cast<__nv_bfloat162*>(p.out + static_cast<long long>(rr) * D + d0) = __floats2bfloat162_rn(x * inv, y * inv);
    }
  }
}

// ------------------------------------------------------------------ launches
template <int D, int RT>
cudaError_t launch_tails(TailParams& p, int num_sms, cudaStream_t s) {
  using L = TailLayout<D, RT>;
  const cudaError_t e = cudaFuncSetAttribute(stream_tail_kernel<D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC);
  if (e != cudaSuccess) return e;
  const int ctas = num_sms * L::CTAS;
  p.heads = p.Hkv < ctas ? p.Hkv : ctas;
  p.runs = ctas / p.heads;
  return launch_k(stream_tail_kernel<D, RT>, dim3(p.runs * p.heads), dim3(L::THREADS), L::ALLOC, s, p);
}

template <int D>
cudaError_t launch_tails_d(TailParams& p, int RT, int num_sms, cudaStream_t s) {
  switch (RT) {
    case 8: return launch_tails<D, 8>(p, num_sms, s);
    case 16: return launch_tails<D, 16>(p, num_sms, s);
    case 32: return launch_tails<D, 32>(p, num_sms, s);
    default: return launch_tails<D, 64>(p, num_sms, s);
  }
}

// Rows of a unit: the smallest of 8, 16, 32, 64 that holds one stream and
// head's T * G rows, or tiles of 64.
int unit_rows(long long rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

template <int D>
cudaError_t launch_merge(const MergeParams& p, cudaStream_t s) {
  // Many rows keep the GPU's loads in flight by themselves; few, or many
  // partials a row, are shared out over four warps.
  if (p.rows > 2048 && p.splits <= kMergeChunk)
    return launch_k(stream_merge_kernel<D, 1>, dim3((p.rows + kMergeWarps - 1) / kMergeWarps), dim3(kMergeWarps * 32), 0, s, p);
  constexpr int rows = kMergeWarps / 4;
  return launch_k(stream_merge_kernel<D, 4>, dim3((p.rows + rows - 1) / rows), dim3(kMergeWarps * 32), 0, s, p);
}

// The workspace of a cache's stream calls.  A unit has at most 2 * T * G rows
// (or 8), so all units together 2 * max_req * G (or 8 * max_req) per K/V head,
// in units of 8 rows or more; each run adds the rows of one unit: as many runs
// as CTAs, or one a head if there are more heads.  (Units of 32 rows or fewer
// may have twice the CTAs of 64-row units, and take no more for it.)
struct StreamWorkspace {
  size_t runs_of, ml, o, bytes;   // offsets
  StreamWorkspace(int max_req, int Hkv, int G, int D, int num_sms) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t unit_rows_all = static_cast<size_t>(max_req) * Hkv * (2 * G > 8 ? 2 * G : 8);
    const int most_rows = unit_rows(static_cast<long long>(max_req) * G);
    const int ctas = num_sms * (D == 256 || most_rows == 64 ? 1 : 2);
    const size_t rows = unit_rows_all + static_cast<size_t>(ctas > Hkv ? ctas : Hkv) * most_rows;
    runs_of = 0;
    ml = up(unit_rows_all / 8 * sizeof(int2));
    o = ml + up(rows * sizeof(float2));
    bytes = o + up(rows * D * sizeof(float));
  }
};

}  // namespace

size_t streams_quant_workspace(int max_req, int Hkv, int G, int D, int num_sms) {
  return StreamWorkspace(max_req, Hkv, G, D, num_sms).bytes;
}

cudaError_t launch_streams_quant(const QuantStreams& a, const AttnLaunch& al, size_t xchg_bytes, void* ws, int max_req,
                                 const StreamFork& fork, cudaStream_t s) {
  const int G = a.Hq / a.Hkv;
  const int RT = unit_rows(static_cast<long long>(a.T) * G);
  TailParams tp;
  memset(&tp, 0, sizeof(tp));
  const uint64_t dims[4] = {static_cast<uint64_t>(a.D), static_cast<uint64_t>(a.Hkv), static_cast<uint64_t>(a.tail_cap),
                            static_cast<uint64_t>(a.B)};
  const uint64_t strides[3] = {static_cast<uint64_t>(a.D), static_cast<uint64_t>(a.D) * a.Hkv,
                               static_cast<uint64_t>(a.D) * a.Hkv * a.tail_cap};
  const uint32_t box[4] = {static_cast<uint32_t>(a.D < 128 ? a.D : 128), 1u, static_cast<uint32_t>(kTK), 1u};
  if (!encode_tmap_u8_4d(&tp.tm_k, a.k_tail, dims, strides, box) || !encode_tmap_u8_4d(&tp.tm_v, a.v_tail, dims, strides, box))
    return cudaErrorInvalidValue;
  const StreamWorkspace w(max_req, a.Hkv, G, a.D, al.num_sms);
  char* mem = static_cast<char*>(ws);
  tp.runs_of = reinterpret_cast<int2*>(mem + w.runs_of);
  tp.ml = reinterpret_cast<float2*>(mem + w.ml);
  tp.o = reinterpret_cast<float*>(mem + w.o);
  tp.q = a.q;
  tp.k_exp = a.k_exp;
  tp.v_exp = a.v_exp;
  tp.tail_len = a.tail_len;
  tp.n_new = a.n_new;
  tp.err = al.err;
  tp.B = a.B;
  tp.T = a.T;
  while (1 << tp.gs < G) ++tp.gs;   // G is a power of two
  tp.Hkv = a.Hkv;
  tp.tail_cap = a.tail_cap;
  tp.row_tiles = (a.T * G + RT - 1) / RT;
  tp.inject_tx = al.inject_tx < (1 << 19) ? al.inject_tx : 1 << 19;   // a barrier counts fewer than 2^20 bytes
  tp.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(a.D)));
  // The shared store on the cache's own stream, the tails beside it on the
  // caller's; joined again whatever happens, so that a capture stays whole.
  const long long tail_tiles =
      static_cast<long long>(a.B) * a.Hkv * tp.row_tiles * ((a.tail_cap + kTK - 1) / kTK);
  int splits = 0, m_tiles = 0, tail_sms = 0;
  cudaError_t e = cudaEventRecord(fork.forked, s);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(fork.side, fork.forked, 0);
  if (e != cudaSuccess) return e;
  // A push on another stream may publish a window at any time, and the CTAs of
  // a large batch start in several waves: all of them read the state of now.
  AttnLaunch store = al;
  if (fork.held) {
    store.st = fork.held;
    e = launch_hold_ring_state(al.st, fork.held, fork.side);
  }
  if (e == cudaSuccess)
    e = launch_attention_partials(store, a.q, a.B * a.T, tail_tiles, xchg_bytes, fork.side, &splits, &m_tiles, &tail_sms);
  if (e == cudaSuccess) {
    switch (a.D) {
      case 64: e = launch_tails_d<64>(tp, RT, tail_sms, s); break;
      case 128: e = launch_tails_d<128>(tp, RT, tail_sms, s); break;
      default: e = launch_tails_d<256>(tp, RT, tail_sms, s); break;
    }
  }
  cudaError_t j = cudaEventRecord(fork.joined, fork.side);
  if (j == cudaSuccess) j = cudaStreamWaitEvent(s, fork.joined, 0);
  if (e == cudaSuccess) e = j;
  if (e != cudaSuccess) return e;
  MergeParams mp;
  memset(&mp, 0, sizeof(mp));
  const size_t units = static_cast<size_t>(m_tiles) * a.Hkv;
  mp.shared_o = static_cast<const float*>(al.xchg);
  mp.shared_ml = reinterpret_cast<const float2*>(static_cast<const char*>(al.xchg) + units * splits * 128 * a.D * 4);
  mp.runs_of = tp.runs_of;
  mp.head_slots = a.B * tp.row_tiles + tp.runs;
  mp.tail_ml = tp.ml;
  mp.tail_o = tp.o;
  mp.tail_len = a.tail_len;
  mp.n_new = a.n_new;
  mp.out = a.out;
  mp.rows = a.B * a.T * a.Hq;
  mp.T = a.T;
  mp.Hq = a.Hq;
  mp.Hkv = a.Hkv;
  mp.gs = tp.gs;
  mp.tail_cap = a.tail_cap;
  mp.row_tiles = tp.row_tiles;
  mp.RT = RT;
  mp.splits = splits;
  mp.m_tiles = m_tiles;
  switch (a.D) {
    case 64: e = launch_merge<64>(mp, s); break;
    case 128: e = launch_merge<128>(mp, s); break;
    default: e = launch_merge<256>(mp, s); break;
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace rx
