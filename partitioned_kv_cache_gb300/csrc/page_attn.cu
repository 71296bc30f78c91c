// page_attn.cu -- attention of packed new tokens over a paged cache, behind the
// shared store, on tcgen05 (sm_103a).
//
// "OxyGen: Unified KV Cache Management for Vision-Language-Action Models under
// Multi-Task Parallelism", §"Core method": language streams share a read-only
// prefill cache and append keys of their own; here those keys live in pages,
// and a step may bring any number of new tokens to a stream (one when it
// decodes, a chunk when a prompt enters).  With n new tokens at the end of len
// keys, token t attends with one softmax over
//   [pinned; window; places below max(len - n + t + 1, min(prefix, len))],
// and lse = log of the sum of the exponentials of its scores.
//
// Work.  A unit is (stream, K/V head, 128 query rows), row r = token r / G, head
// r % G of the group.  All units' key tiles are numbered in a row
// (page_plan.h) and cut into equal runs, one per CTA; a CTA works its run off
// unit by unit, its rings of K and V tiles never stopping in between.  A unit
// that lies in one run is finished there; of a cut unit every CTA leaves its
// part (O, m, l) in fp32 in the workspace and merge_kernel joins the parts in
// the order of the keys.  Lengths are read on the device.
//
// Inside a CTA the steps are those of the suffix's attention: S = Q K^T and
// O += P V on tcgen05 with accumulators in tensor memory, Q and P (bf16) the A
// operands in tensor memory too, O rescaled only when a row's maximum grows by more
// than 2^8.  (With Q in shared memory a product of 128 x 64 or 128 x 128 takes a
// quarter longer, for its operand's way out of there.)  A weight enters P V rounded
// to bf16 (2^-9 of it at most): beside the output's own rounding, 0.0017 relative to
// the exact result over a call's rows, that makes 0.0023, and two terms would cost
// P V a second time.
//
// What bounds it, and what it took (GB300, a graph of calls):
//   8 chunks of 2048 tokens, 8 heads over 1 of 256, 8448 shared keys, tails to
//   8000: the tensor core, 945 us, 1770 TFLOP/s (0.92 of cuBLAS's; hot, at the power
//   limit, 1560); 1355 us with Q in shared memory and one issuing thread.
//   32 single tokens, 32/8 heads of 128, tails to 16000: memory, 170 us, 6.1 TB/s.
//   5 chunks of up to 999 tokens, 32/8 heads of 128, pages of 32: 153 us, 842
//   TFLOP/s; in the middle of a unit 1086.  A tile of 128 keys there takes some 2200
//   cycles of which the products are 1030 and the copies 1600 (some 3 cycles for
//   every 128 bytes of a row and 100 to 200 a copy, whatever the SM count); they
//   and the softmax's steps meet at every tile's barriers.  (V by 16-byte copies of a
//   warp of its own instead, beside K's tensor copies: 175 us, and the single tokens
//   above 202.)
//
// Long sums.  The tensor core drops what an addition has below fp32's last place, so a
// sum over n keys of one sign comes out too small by some 6 10^-9 n of itself: 8 10^-4
// at 2^17 keys, 3.3 10^-3 at 2^19, more than bf16's rounding.  After 16384 keys (8 10^-5)
// O and the row's sum are put away in fp32, in the slot that the unit's part has anyway,
// and start again.  (The first case above has up to 16 496 keys; its time is as without. One
// loop over all tiles that looks for a sum's end cost 3% at D = 256.)
//
// Masked places.  Scores are masked by selection, so whatever a place behind
// the stream's end, in a page that the table does not name, or after a token
// holds, it weighs nothing.  A weight of 0 times an infinity or NaN in V would
// still be NaN: in tiles where not every row sees every key the softmax warps
// read V's tile in shared memory first and write zeros over rows that are
// outside, or not finite and hidden from some row; outputs of rows that see one of
// the latter become NaN.
//
// Warps: 0 = copies of K, 1 = tensor memory, copies of Q and Q K^T, 2 = P V, 3 =
// copies of V, 4..11 = softmax and epilogue.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "page_plan.h"
#include "pages.h"
#include "rx_internal.h"
#include "pages_ptx.cuh"

namespace rx {
namespace {

constexpr float kRescale = 8.0f;   // log2 units
constexpr int kMinRunKeys = 256;   // keys of a CTA's run, at least
constexpr int kSegmentKeys = 16384;   // of a sum of products (see above)
constexpr int kUnitPad = 4;        // tiles that a unit's start and end cost: chunks with units of 11 to 59 tiles
                                   // take 161 us, and 203 with 0
constexpr int kMergeThreads = 256;
// The merge is bound by its instructions and the depth of its loads.  Up to kMergeFew
// parts one thread joins 16 columns of a row, two parts at a time: 153 us for the five
// chunks above, where a thread per four columns took 155, and 47 us for a chunk of 512
// beside 16 single tokens, where one part at a time took 48.5.  More parts are shared by
// eight warps, kMergeFlight of a warp's asked for together.
constexpr int kMergeFew = 8;
constexpr int kMergeFlight = 4;

constexpr int kThreads = 384;
constexpr int kSoftmax = 256;      // of them two per query row

template <int D>
struct Layout {
  static constexpr int KB = D / 64;
  static constexpr int Q_BLOCK = kBM * 128;
  static constexpr int Q_BYTES = KB * Q_BLOCK;
  // Keys of a tile.  A tile's waits, barriers and masks cost the softmax as much as
  // 64 columns do: 128 keys are better where tensor memory has room for their scores
  // (5 chunks of up to 999 tokens, D = 128: 215 us with 64, 208 with 128).
  static constexpr int BN = D == 256 ? 64 : 128;
  static constexpr int BLOCK = BN * 128;                    // 64 columns of a K or V tile
  static constexpr int TILE = KB * BLOCK;
  static constexpr int SEGMENT = kSegmentKeys / BN;         // tiles of a sum of products, a power of two
  static constexpr int NK = D == 64 ? 5 : 3;
  static constexpr int NV = D == 64 ? 5 : D == 128 ? 3 : 2;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = Q_BYTES;
  static constexpr int OFF_V = OFF_K + NK * TILE;
  static constexpr int OFF_BAR = OFF_V + NV * TILE;
  static constexpr int OFF_MISC = OFF_BAR + 64 * 8;
  static constexpr int OFF_SUM = OFF_MISC + 128;            // floats [2 halves][128 rows]
  static constexpr int BYTES = OFF_SUM + 2 * kBM * 4;
  static constexpr int ALLOC = BYTES + 1024;
  // Tensor memory: O, Q (bf16 pairs), scores and P (bf16 pairs); of the last two
  // one has room for two tiles: P at D = 256, else the scores.
  static constexpr int NS = D == 256 ? 1 : 2, NP = 3 - NS;
  static constexpr int T_Q = D, T_S = T_Q + D / 2, T_P = T_S + NS * BN;
  static_assert(T_P + NP * (BN / 2) <= 512, "tensor memory");
  static_assert(ALLOC <= 232448, "shared memory");
};

// Barriers: K full / empty [10], V full / empty [10], Q full / empty (shared
// memory), Q in tensor memory, scores full / read [2], P full [2], P V done [2],
// O read, values checked, row sums there, drained.
enum : int {
  B_KF = 0, B_KE = 10, B_VF = 20, B_VE = 30, B_QF = 40, B_QE = 41, B_QT = 42, B_SF = 43, B_SR = 45, B_PF = 47, B_PV = 49,
  B_OR = 51, B_CHK = 52, B_SUM = 53, B_DRAIN = 54, B_COUNT = 55
};

// The parts that merge_kernel joins: those of the unit that CTA c's run begins
// and does not end (rows 0: none).
struct CutUnit {
  int token;   // first of the row tile
  int rows;
  int head;    // K/V head
  int parts;
};

struct PageAttnParams {
  CUtensorMap tm_q;            // 128 query rows (encode_query_map)
  CUtensorMap tm_k;            // a page's keys, BN at most (encode_page_map)
  CUtensorMap tm_v;
  const uint8_t* k_tiles[2];   // store: pinned, window of (layer, head 0)
  const uint8_t* v_tiles[2];
  long long head_stride[2];
  const DevState* st;          // null: no store
  int P, F, frames, slots;
  PagePool pool;
  const int* q_start;
  const int* len;
  const int* prefix;
  int N, Hq, Hkv, log_g;
  __nv_bfloat16* out;
  float* lse;
  float4* part;                // [2 * grid][D/4][part_rows]
  float2* part_ml;             // [2 * grid][part_rows]
  CutUnit* cut;                // [grid]
  int part_rows;
  int* err;
  int inject_tx;
  float scale_log2;
};

// A bit for every key of a tile.
template <int BN>
struct Bits {
  uint64_t w[BN / 64];
};
// The first n of 64 bits (n may be below 0 or above 64).
__device__ __forceinline__ uint64_t first_bits(int n) { return n >= 64 ? ~0ull : n > 0 ? (1ull << n) - 1 : 0ull; }

// 32 values of an array.
template <int N>
__device__ __forceinline__ float (&part(float (&x)[N], int at))[32] {
  return *reinterpret_cast<float(*)[32]>(x + at);
}

// Scores of keys that the row does not see.
__device__ __forceinline__ void hide(float (&x)[32], uint32_t seen) {
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (!(seen >> c & 1)) x[c] = -INFINITY;
}

// The store's tiles of 64 keys: pinned, then the window in slot order, past the
// spare slot.  A tile of 128 keys is two of them in a row.
struct StoreTiles {
  int n_pin, n_win, P, win_len, hole0, hole_n;
  __device__ __forceinline__ int count() const { return n_pin + n_win; }
  // Keys of its tile t of 64 (0 behind the last).
  __device__ __forceinline__ int valid(int t) const {
    return max(0, min(kTileTok, t < n_pin ? P - t * kTileTok : win_len - (t - n_pin) * kTileTok));
  }
};

__device__ __forceinline__ StoreTiles store_tiles(const PageAttnParams& p, int head, int valid) {
  StoreTiles s{0, 0, 0, 0, 0, 0};
  if (!p.st) return s;
  const bool hole = p.slots > p.frames && valid == p.frames;
  s.P = p.P;
  s.win_len = hole ? (p.slots - 1) * p.F : valid * p.F;
  s.hole0 = hole ? head * p.F / kTileTok : 0;
  s.hole_n = hole ? p.F / kTileTok : 0;
  s.n_pin = (p.P + kTileTok - 1) / kTileTok;
  s.n_win = (s.win_len + kTileTok - 1) / kTileTok;
  return s;
}

struct Stream {
  StreamPlan plan;
  int q0;
  int prefix;   // min(prefix, len), 0 without one
};

__device__ __forceinline__ Stream load_stream(const PageAttnParams& p, int log_t, int shared, int b) {
  Stream s;
  s.q0 = max(0, min(__ldg(p.q_start + b), p.N));
  const int q1 = max(0, min(__ldg(p.q_start + b + 1), p.N));
  s.plan.n = max(0, q1 - s.q0);
  s.plan.len = held_keys(p.pool, p.len, b);
  s.prefix = p.prefix ? max(0, min(__ldg(p.prefix + b), s.plan.len)) : 0;
  s.plan.floor = max(1, s.prefix);
  s.plan.shared = shared;
  s.plan.log_a = 7 - p.log_g;
  s.plan.log_t = log_t;
  s.plan.pad = kUnitPad;
  return s;
}

// Where a run begins: tile `at` of stream b; `left` tiles from there.
struct RunStart {
  long long at;
  long long left;
  int b;
};

// A walk over the parts of units in a run.
struct Walk {
  Stream s;
  int b, h, rt;
  int t0, count, tiles;   // the part: tiles [t0, t0 + count) of the unit's `tiles`
  int taken;              // numbers of the run that it takes, pads among them
  long long left;

  __device__ __forceinline__ bool begin(const PageAttnParams& p, int log_t, int shared, const RunStart& r) {
    left = r.left;
    if (left <= 0) return false;
    b = r.b;
    s = load_stream(p, log_t, shared, b);
    const long long per_head = s.plan.tiles_before(s.plan.row_tiles());
    h = static_cast<int>(r.at / per_head);
    const long long o = r.at - h * per_head;
    rt = s.plan.row_tile_of(o);
    t0 = static_cast<int>(o - s.plan.tiles_before(rt));
    measure();
    return count > 0 || next(p);   // (a run may begin in a pad)
  }
  __device__ __forceinline__ void measure() {
    tiles = s.plan.tiles(rt);
    taken = static_cast<int>(min(left, static_cast<long long>(tiles + s.plan.pad - t0)));
    count = min(taken, tiles - t0);
  }
  __device__ __forceinline__ bool next(const PageAttnParams& p) {
    left -= taken;
    if (left <= 0) return false;
    t0 = 0;
    if (++rt == s.plan.row_tiles()) {
      rt = 0;
      if (++h == p.Hkv) {
        h = 0;
        do {
          if (++b >= p.pool.B) return false;
          s = load_stream(p, s.plan.log_t, s.plan.shared, b);
        } while (s.plan.n == 0);
      }
    }
    measure();
    return true;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) page_attn_kernel(const __grid_constant__ PageAttnParams p) {
  using Lay = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sQ = base + Lay::OFF_Q, sK = base + Lay::OFF_K, sV = base + Lay::OFF_V, sBar = base + Lay::OFF_BAR;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + Lay::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + Lay::OFF_MISC + 4);
  int* ring_word = reinterpret_cast<int*>(gbase + Lay::OFF_MISC + 8);
  RunStart* run_start = reinterpret_cast<RunStart*>(gbase + Lay::OFF_MISC + 16);      // 24 bytes
  int* run_len = reinterpret_cast<int*>(gbase + Lay::OFF_MISC + 40);
  uint8_t* not_finite = gbase + Lay::OFF_MISC + 64;                                    // [2][16]
  float* row_sum = reinterpret_cast<float*>(gbase + Lay::OFF_SUM);
  auto BAR = [&](int i) { return sBar + 8u * static_cast<uint32_t>(i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i) {
      const bool all = i == B_QE || i == B_QT || (i >= B_SR && i < B_SR + 2) || (i >= B_PF && i < B_PF + 2) ||
                       i == B_OR || i == B_CHK || i == B_SUM;
      mbar_init(BAR(i), all ? kSoftmax : i == B_DRAIN ? 2 : 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_k);
    tma_prefetch_desc(&p.tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();
  grid_launch_dependents();

  // ---- this CTA's run.  The streams' tiles go through shared memory that the
  // rings use afterwards.
  if (threadIdx.x == 0 && p.st) load_ring_state(p.st, ring_word, ring_word + 1);
  __syncthreads();
  const StoreTiles store = store_tiles(p, ring_word[0], ring_word[1]);
  constexpr int kLogT = Lay::BN == 128 ? 7 : 6;
  const int shared = (store.count() * kTileTok + Lay::BN - 1) >> kLogT;   // tiles
  long long* before = reinterpret_cast<long long*>(gbase + Lay::OFF_K);   // [B + 1]
  for (int b = threadIdx.x; b < p.pool.B; b += kThreads) {
    const Stream s = load_stream(p, kLogT, shared, b);
    before[b + 1] = p.Hkv * s.plan.tiles_before(s.plan.row_tiles());
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
    __syncwarp();
    if (lane == 0) {
      const long long each = max(static_cast<long long>(kMinRunKeys / Lay::BN), (sum + gridDim.x - 1) / gridDim.x);
      const long long w0 = each * blockIdx.x, w1 = min(sum, w0 + each);
      int lo = 0, hi = p.pool.B - 1;
      while (lo < hi) {   // the last stream that begins at or before w0
        const int mid = (lo + hi + 1) >> 1;
        if (before[mid] <= w0) lo = mid;
        else hi = mid - 1;
      }
      run_start->at = w0 - before[lo];
      run_start->left = w1 - w0;
      run_start->b = lo;
      *run_len = static_cast<int>(each);
    }
  }
  // The scratch was written by the generic proxy; copies will write it next.
  fence_proxy_async_smem();
  __syncthreads();
  const RunStart run = *run_start;

  const uint32_t tmem = *tmem_slot;
  const uint32_t tO = tmem, tQ = tmem + Lay::T_Q, tS = tmem + Lay::T_S, tP = tmem + Lay::T_P;
  const int lp = p.pool.log_page;
  const int box = lp < kLogT ? 1 << lp : Lay::BN;         // tokens of one page copy

  Walk w;
  const bool some = w.begin(p, kLogT, shared, run);
  if (some && (warp == 0 || warp == 3)) {
    // ------------------------------------------------------------ copies of K, of V
    // The lanes hold the table's next 64 entries, asked for a round ahead; one
    // issues (copies by several lanes of a warp go one after the other all the same).
    const bool leader = elect_one();
    const bool isv = warp == 3;
    const CUtensorMap* tm = isv ? &p.tm_v : &p.tm_k;
    const int slots = isv ? Lay::NV : Lay::NK;
    const int bf = isv ? B_VF : B_KF, be = isv ? B_VE : B_KE;
    const uint32_t ring = isv ? sV : sK;
    const int log_e = lp < kLogT ? kLogT - lp : 0;         // pages of a tile
    int slot = 0, round = 0, issued = 0;
    bool more = true, stop = false;
    do {
      const int* table = p.pool.table + static_cast<long long>(w.b) * p.pool.max_pages;
      const int len = w.s.plan.len;
      auto entry = [&](int e) { return (static_cast<long long>(e) << lp) < len ? __ldg(table + e) : -1; };
      const int t_end = w.t0 + w.count;
      int e_base = max(0, (w.t0 - shared) * Lay::BN) >> lp;
      int now = entry(e_base + lane), then = entry(e_base + 32 + lane);
      for (int t = w.t0; t < t_end; ++t) {
        const int key0 = (t - shared) * Lay::BN;
        if (round > 0 && !warp_wait(BAR(be + slot), (round - 1) & 1, abort_flag)) {
          stop = true;
          break;
        }
        const uint32_t dst = ring + slot * Lay::TILE, bar = BAR(bf + slot);
        const uint32_t extra = issued == 0 && !isv && blockIdx.x == 0 ? static_cast<uint32_t>(p.inject_tx) : 0u;
        if (t < shared) {
          // Two (at D = 256 one) tiles of the store.
          constexpr int kHalves = Lay::BN / kTileTok;
          if (leader) {
            mbar_arrive_expect_tx(bar, min(kHalves, store.count() - t * kHalves) * Lay::KB * 8192 + extra);
#pragma unroll
            for (int i = 0; i < kHalves; ++i) {
              const int t64 = t * kHalves + i;
              if (t64 >= store.count()) break;
              const int region = t64 < store.n_pin ? 0 : 1;
              int at = region ? t64 - store.n_pin : t64;
              if (region && at >= store.hole0) at += store.hole_n;
              const uint8_t* src = (isv ? p.v_tiles[region] : p.k_tiles[region]) + w.h * p.head_stride[region] +
                                   static_cast<long long>(at) * Lay::KB * 8192;
              if constexpr (kHalves == 1) {
                bulk_load(dst, src, Lay::TILE, bar);
              } else {
#pragma unroll
                for (int kb = 0; kb < Lay::KB; ++kb) bulk_load(dst + kb * Lay::BLOCK + i * 8192, src + kb * 8192, 8192, bar);
              }
            }
          }
        } else {
          const int e0 = key0 >> lp;
          if (e0 - e_base >= 32) {
            e_base += 32;
            now = then;
            then = entry(e_base + 32 + lane);
          }
          const int at = e0 - e_base, pages = 1 << log_e, row = lp > kLogT ? key0 & ((1 << lp) - 1) : 0;
          const uint32_t named = __ballot_sync(0xffffffffu, static_cast<unsigned int>(now) < static_cast<unsigned int>(p.pool.n_pages)) >> at & ((2u << (pages - 1)) - 1);
          if (leader) mbar_arrive_expect_tx(bar, __popc(named) * box * (D * 2) + extra);
          for (int i = 0; i < pages; ++i) {
            const int pg = __shfl_sync(0xffffffffu, now, at + i);
            if (leader && (named >> i & 1)) tma_load_5d(dst + i * box * Lay::KB * 128, tm, 0, 0, w.h * Lay::KB, row >> 3, pg, bar);
          }
        }
        __syncwarp();
        ++issued;
        if (++slot == slots) {
          slot = 0;
          ++round;
        }
      }
      more = !stop && w.next(p);
    } while (more);
    // Every copy issued lands before the CTA exits, after an abort too.
    volatile int no_abort = 0;
    for (int n = max(0, issued - slots); n < issued; ++n) mbar_wait(BAR(bf + n % slots), (n / slots) & 1, &no_abort);
  } else if (some && warp == 1) {
    // ------------------------------------------------------------ Q K^T
    // Q is the A operand from tensor memory.  All lanes run the loop, so that its
    // values are the same for the whole warp, and one issues the products.
    constexpr uint32_t kIdesc = idesc_bf16_f32(kBM, Lay::BN, false, false);
    const bool leader = elect_one();
    int j = 0, slot = 0, round = 0, u = 0, asked = 0;
    bool ok = true, more = true;
    auto ask_q = [&](const Walk& x) {        // a unit's Q into shared memory
      if (leader) {
        mbar_arrive_expect_tx(BAR(B_QF), Lay::Q_BYTES);
        tma_load_4d(sQ, &p.tm_q, 0, 0, x.s.q0 + (x.rt << x.s.plan.log_a), (x.h << p.log_g) * Lay::KB, BAR(B_QF));
      }
      __syncwarp();
      ++asked;
    };
    ask_q(w);
    while (more) {
      const int count = uniform(w.count), first_t = uniform(w.t0);
      Walk coming = w;
      more = coming.next(p);
      ok = warp_wait(BAR(B_QT), u & 1, abort_flag);
      // This unit's is in tensor memory: the next one's can come.
      if (ok && more) {
        ok = warp_wait(BAR(B_QE), u & 1, abort_flag);
        if (ok) ask_q(coming);
      }
      for (int t = 0; ok && t < count; ++t) {
        const int st = Lay::NS == 1 ? 0 : j & 1;
        // The softmax has read the scores of tile j - NS.
        if (j >= Lay::NS && !warp_wait(BAR(B_SR + st), (j / Lay::NS - 1) & 1, abort_flag)) { ok = false; break; }
        if (!warp_wait(BAR(B_KF + slot), round & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        // The store's tiles are [column block][token], the pages' [8 tokens][column block].
        const bool paged = first_t + t >= shared;
        const uint64_t desc = sdesc_sw128(sK + slot * Lay::TILE, 16, paged ? Lay::KB * 1024 : 1024);
        const uint32_t block = (paged ? 1024 : Lay::BLOCK) >> 4;
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16_ts(tS + st * Lay::BN, tQ + kk * 8, desc + ((kk >> 2) * block + (kk & 3) * 2), kIdesc, kk > 0 ? 1u : 0u);
          umma_commit(BAR(B_KE + slot));
          umma_commit(BAR(B_SF + st));
        }
        __syncwarp();
        ++j;
        if (++slot == Lay::NK) {
          slot = 0;
          ++round;
        }
      }
      ++u;
      w = coming;
      more = more && ok;
    }
    if (leader) umma_commit(BAR(B_DRAIN));
    volatile int no_abort = 0;
    mbar_wait(BAR(B_QF), (asked - 1) & 1, &no_abort);
    mbar_wait(BAR(B_DRAIN), 0, &no_abort);
  } else if (some && warp == 2) {
    // ------------------------------------------------------------ P V
    constexpr uint32_t kIdesc = idesc_bf16_f32(kBM, D, false, true);
    const bool leader = elect_one();
    int j = 0, slot = 0, round = 0, opened = 0;   // sums opened so far
    bool ok = true;
    do {
      const int end = uniform(w.t0) + uniform(w.count);
      for (int t0 = end - uniform(w.count), t = t0; t < end; ++t) {
        const int st = j & 1;
        if (t - t0 == Lay::SEGMENT) t0 = t;   // a sum's first tile
        if (!warp_wait(BAR(B_PF + st), (j >> 1) & 1, abort_flag)) { ok = false; break; }
        if (!warp_wait(BAR(B_VF + slot), round & 1, abort_flag)) { ok = false; break; }
        // O still holds the last sum until the softmax warps have read it.
        if (t == t0 && opened++ > 0 && !warp_wait(BAR(B_OR), opened & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const bool paged = t >= shared;
        const uint64_t desc = sdesc_sw128(sV + slot * Lay::TILE, paged ? 1024 : Lay::BLOCK, paged ? Lay::KB * 1024 : 1024);
        const uint32_t step = (paged ? Lay::KB * 2048 : 2048) >> 4;   // 16 keys
        const uint32_t more = t > t0 ? 1u : 0u;
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < Lay::BN / 16; ++kk)
            umma_bf16_ts(tO, tP + (Lay::NP == 2 ? st * (Lay::BN / 2) : 0) + kk * 8, desc + kk * step, kIdesc, kk > 0 ? 1u : more);
          umma_commit(BAR(B_VE + slot));
          umma_commit(BAR(B_PV + st));
        }
        __syncwarp();
        ++j;
        if (++slot == Lay::NV) {
          slot = 0;
          ++round;
        }
      }
    } while (ok && w.next(p));
    if (leader) umma_commit(BAR(B_DRAIN));
    volatile int no_abort = 0;
    mbar_wait(BAR(B_DRAIN), 0, &no_abort);
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax
    // A row has two threads, in warps w and w + 4 (a warp reaches the tensor memory
    // lanes of its quarter): each looks at all scores of the row for the maximum, so
    // that both arrive at the same reference without a word, takes the exponentials
    // of half of the columns and, later, its half of O's columns.
    constexpr int kOCols = D / 2, BN = Lay::BN;
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const int row = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const bool first_thread = threadIdx.x == 128;
    if (first_thread) p.cut[blockIdx.x] = CutUnit{0, 0, 0, 0};
    int j = 0, vslot = 0, vround = 0, checks = 0, u = 0;
    bool ok = true, more = some;
    const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
    // Unit n's Q from shared into tensor memory, this thread's half of its row.
    // The scores of the last unit's tiles are all done: this thread waited for them.
    auto load_q = [&](int n) {
      if (!warp_wait(BAR(B_QF), n & 1, abort_flag)) return false;
      constexpr int kChunks = D / 16;   // of 16 bytes
#pragma unroll
      for (int c0 = 0; c0 < kChunks; c0 += 4) {
        uint32_t x[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = half * kChunks + c0 + i;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x[4 * i]), "=r"(x[4 * i + 1]), "=r"(x[4 * i + 2]), "=r"(x[4 * i + 3])
                       : "r"(sQ + (c >> 3) * Lay::Q_BLOCK + row * 128 + (((c & 7) ^ (row & 7)) << 4)));
        }
        tmem_st16(tQ + (half * kChunks + c0) * 4 + lane_off, x);
      }
      tc_fence_before();
      mbar_arrive(BAR(B_QT));
      mbar_arrive(BAR(B_QE));
      return true;
    };
    // A lane's entry of the table of the first 32 from a part's start on (0: none).
    auto entry_of = [&](const Walk& x) {
      const int e = (max(0, (x.t0 - shared) * BN) >> lp) + lane;
      return (static_cast<long long>(e) << lp) < x.s.plan.len
                 ? __ldg(p.pool.table + static_cast<long long>(x.b) * p.pool.max_pages + e) : 0;
    };
    int first_entry = more ? entry_of(w) : 0;
    if (more) ok = load_q(0);
    while (more) {
      const int t_row = (w.rt << w.s.plan.log_a) + (row >> p.log_g);
      const bool row_valid = t_row < w.s.plan.n;
      const int x0 = w.s.plan.len - w.s.plan.n;
      // Places below lim are seen by this row, those below all by every row.
      const int lim = row_valid ? max(x0 + t_row + 1, w.s.prefix) : 0;
      const int all = max(x0 + (w.rt << w.s.plan.log_a) + 1, w.s.prefix);
      const int* table = p.pool.table + static_cast<long long>(w.b) * p.pool.max_pages;
      // Which of the 32 table entries from e_base on name a page (those behind the
      // stream's end pass), and the lanes' entries after them, on their way.
      const int log_e = lp < kLogT ? kLogT - lp : 0;                // pages of a tile
      const uint32_t tile_pages = (2u << ((1 << log_e) - 1)) - 1;   // a bit for each
      auto entry = [&](int e) { return (static_cast<long long>(e) << lp) < w.s.plan.len ? __ldg(table + e) : 0; };
      auto named_of = [&](int x) { return __ballot_sync(0xffffffffu, static_cast<unsigned int>(x) < static_cast<unsigned int>(p.pool.n_pages)); };
      int e_base = max(0, (w.t0 - shared) * BN) >> lp;
      uint32_t named32 = named_of(first_entry);
      int then = entry(e_base + 32 + lane);
      const int plain = min(w.s.plan.len, all);   // every row sees every key before it
      float m_used = -INFINITY;
      float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      bool poison = false;
      // What of closed sums lies in the part's place: O in the scale of m_kept.
      auto kept = [&](int column) {
        const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (w.t0 == 0 ? 1 : 0);
        return p.part + (slot * (D / 4) + column / 4) * p.part_rows + row;
      };
      float m_kept = -INFINITY, l_kept = 0.f;
      // 32 columns of O, with those of closed sums where there are any.
      auto read_o = [&](int c, float f, bool closed, float (&o)[32]) {
        tmem_ld32(tO + c + lane_off, o);
        if (closed && row_valid) {
          const float4* from = kept(c);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 x = from[static_cast<size_t>(i) * p.part_rows];
            o[4 * i] = fmaf(x.x, f, o[4 * i]);
            o[4 * i + 1] = fmaf(x.y, f, o[4 * i + 1]);
            o[4 * i + 2] = fmaf(x.z, f, o[4 * i + 2]);
            o[4 * i + 3] = fmaf(x.w, f, o[4 * i + 3]);
          }
        }
      };
      auto kept_scale = [&]() { return m_kept == m_used ? 1.f : exp2f(m_kept - m_used); };
      const int t_end = w.t0 + w.count;
      for (int sum_t = w.t0; ok && sum_t < t_end; sum_t += Lay::SEGMENT) {
        if (sum_t > w.t0) {   // close the last sums
          if (!warp_wait(BAR(B_PV + ((j - 1) & 1)), ((j - 1) >> 1) & 1, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const float f = kept_scale();
#pragma unroll 1
          for (int c = half * kOCols; c < (half + 1) * kOCols; c += 32) {
            float o[32];
            read_o(c, f, sum_t - w.t0 > Lay::SEGMENT, o);
            if (row_valid) {
              float4* to = kept(c);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                to[static_cast<size_t>(i) * p.part_rows] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
          }
          tc_fence_before();
          mbar_arrive(BAR(B_OR));
          l_kept = fmaf(l_kept, f, (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y));
          l2[0] = l2[1] = make_float2(0.f, 0.f);
          m_kept = m_used;
        }
        const int sum_end = min(t_end, sum_t + Lay::SEGMENT);
        for (int t = sum_t; ok && t < sum_end; ++t, ++j) {
          const int st = j & 1;
          // Keys of the tile that are there, and those that this row sees.
          Bits<BN> there, mine;
          bool check;
          if (t < shared) {
            constexpr int kHalves = BN / kTileTok;
            int nv[kHalves];
            check = false;
#pragma unroll
            for (int i = 0; i < kHalves; ++i) {
              nv[i] = store.valid(t * kHalves + i);
              check = check || nv[i] < kTileTok;
            }
            if (check) {
#pragma unroll
              for (int i = 0; i < kHalves; ++i) there.w[i] = first_bits(nv[i]);
              mine = there;
            }
          } else {
            const int key0 = (t - shared) * BN;
            const int e0 = key0 >> lp;
            if (e0 - e_base >= 32) {
              e_base += 32;
              named32 = named_of(then);
              then = entry(e_base + 32 + lane);
            }
            const uint32_t named = named32 >> (e0 - e_base) & tile_pages;
            check = named != tile_pages || key0 + BN > plain;
            if (check) {
              const int nv = w.s.plan.len - key0, seen = lim - key0;
#pragma unroll
              for (int i = 0; i < BN / 64; ++i) {
                uint64_t x = ~0ull;
                if (named != tile_pages) {
                  x = 0;
                  for (int e = 0; e < max(1, 64 >> lp); ++e) {   // lp >= 6: one page holds the 64 keys
                    const int page_of = lp < 6 ? (i << (6 - lp)) + e : lp < kLogT ? i : 0;
                    if (named >> page_of & 1) x |= lp < 6 ? ((1ull << (1 << lp)) - 1) << (e << lp) : ~0ull;
                  }
                }
                there.w[i] = x & first_bits(nv - 64 * i);
                mine.w[i] = there.w[i] & first_bits(seen - 64 * i);
              }
            }
          }
          const int sb = j % Lay::NS;
          if (!warp_wait(BAR(B_SF + sb), (j / Lay::NS) & 1, abort_flag)) { ok = false; break; }
          tc_fence_after();
          float s[BN / 2];   // this thread's columns; the others are looked at only
          float top;
          const uint32_t s_own = tS + sb * BN + half * (BN / 2) + lane_off, s_other = tS + sb * BN + (half ^ 1) * (BN / 2) + lane_off;
          if constexpr (BN == 64) {
            float r[32];
            tmem_ld32x2(s_own, s, s_other, r);
            if (check) {
              hide(s, static_cast<uint32_t>(mine.w[0] >> (32 * half)));
              hide(r, static_cast<uint32_t>(mine.w[0] >> (32 - 32 * half)));
            }
            top = fmaxf(max32(r), max32(s));
          } else {
            float r[64];
            tmem_ld64(s_other, r);
            const uint64_t seen_r = half ? mine.w[0] : mine.w[BN / 64 - 1], seen_s = half ? mine.w[BN / 64 - 1] : mine.w[0];
            if (check) {
              hide(part(r, 0), static_cast<uint32_t>(seen_r));
              hide(part(r, 32), static_cast<uint32_t>(seen_r >> 32));
            }
            top = fmaxf(max32(part(r, 0)), max32(part(r, 32)));
            tmem_ld64(s_own, s);
            if (check) {
              hide(part(s, 0), static_cast<uint32_t>(seen_s));
              hide(part(s, 32), static_cast<uint32_t>(seen_s >> 32));
            }
            top = fmaxf(top, fmaxf(max32(part(s, 0)), max32(part(s, 32))));
          }
          tc_fence_before();
          mbar_arrive(BAR(B_SR + sb));
          if (check) {
            // V's rows, some threads each.  P V of tile j - 2 first: until then
            // V's barrier may be one phase behind, and its parity would pass.
            if (j >= 2 && !warp_wait(BAR(B_PV + st), ((j - 2) >> 1) & 1, abort_flag)) { ok = false; break; }
            if (!warp_wait(BAR(B_VF + vslot), vround & 1, abort_flag)) { ok = false; break; }
            constexpr int kShare = kSoftmax / BN;   // threads of a V row: 2 or 4
            const int vr = (threadIdx.x - 128) / kShare;
            const uint32_t at = sV + vslot * Lay::TILE + (t < shared ? vr * 128 : (vr >> 3) * (Lay::KB * 1024) + (vr & 7) * 128);
            const uint32_t block = t < shared ? Lay::BLOCK : 1024;
            constexpr int kChunks = D / 8 / kShare;
            const int c0 = (lane & (kShare - 1)) * kChunks;
            const bool outside = !(there.w[vr >> 6] >> (vr & 63) & 1);
            uint32_t odd = 0;
            // (A value that every row sees may do to them what it does.)
            const int unseen = t < shared ? BN : all - (t - shared) * BN;   // keys before it are seen by all
            if (!outside && vr >= unseen) {
#pragma unroll
              for (int i = 0; i < kChunks; ++i) {
                const int c = c0 + i;
                uint32_t x[4];
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                             : "r"(at + (c >> 3) * block + (((c & 7) ^ (vr & 7)) << 4)));
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  odd |= ((x[e] & 0x7F80u) == 0x7F80u) | ((x[e] & 0x7F800000u) == 0x7F800000u);
              }
            }
            odd |= __shfl_xor_sync(0xffffffffu, odd, 1);
            if (kShare == 4) odd |= __shfl_xor_sync(0xffffffffu, odd, 2);
            if (outside || odd) {
#pragma unroll
              for (int i = 0; i < kChunks; ++i) st_shared_v4(at + ((c0 + i) >> 3) * block + (((c0 + i) & 7) << 4), 0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            if (unseen < BN) {
              // Every second or fourth lane's bit, close up.
              uint32_t rows = __ballot_sync(0xffffffffu, odd != 0);
              volatile uint8_t* bits = not_finite + (checks & 1) * 16;
              if constexpr (kShare == 4) {
                rows &= 0x11111111u;
                rows = (rows | rows >> 3) & 0x03030303u;
                rows = (rows | rows >> 6) & 0x000F000Fu;
                rows = (rows | rows >> 12) & 0x000000FFu;
                if (lane == 0) bits[warp - 4] = static_cast<uint8_t>(rows);
              } else {
                rows &= 0x55555555u;
                rows = (rows | rows >> 1) & 0x33333333u;
                rows = (rows | rows >> 2) & 0x0F0F0F0Fu;
                rows = (rows | rows >> 4) & 0x00FF00FFu;
                rows = (rows | rows >> 8) & 0x0000FFFFu;
                if (lane == 0) reinterpret_cast<volatile uint16_t*>(bits)[warp - 4] = static_cast<uint16_t>(rows);
              }
              mbar_arrive(BAR(B_CHK));
              if (!warp_wait(BAR(B_CHK), checks & 1, abort_flag)) { ok = false; break; }
              ++checks;
#pragma unroll
              for (int i = 0; i < BN / 64; ++i) poison = poison || (reinterpret_cast<volatile uint64_t*>(bits)[i] & mine.w[i]) != 0;
            }
          }
          if (++vslot == Lay::NV) {
            vslot = 0;
            ++vround;
          }
          const float m_new = fmaxf(m_used, top * p.scale_log2);
          const bool need = m_new > m_used + kRescale;
          float fac = 1.f;
          if (need) {
            fac = exp2f(m_used - m_new);
#pragma unroll
            for (int i = 0; i < 2; ++i) l2[i] = make_float2(l2[i].x * fac, l2[i].y * fac);
            m_used = m_new;
          }
          if (__any_sync(0xffffffffu, need && t > sum_t)) {
            if (!warp_wait(BAR(B_PV + ((j - 1) & 1)), ((j - 1) >> 1) & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int c = half * kOCols; c < (half + 1) * kOCols; c += 32) {
              float o[32];
              tmem_ld32(tO + c + lane_off, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= fac;
              tmem_st32(tO + c + lane_off, o);
            }
          }
          const float nmb = m_used == -INFINITY ? 0.f : -m_used;
          const float2 nmb2 = make_float2(nmb, nmb);
          uint32_t pk[BN / 4];
#pragma unroll
          for (int c = 0; c < BN / 4; ++c) {
            float2 e = fma2(make_float2(s[2 * c], s[2 * c + 1]), scale2, nmb2);
            e = make_float2(exp2f(e.x), exp2f(e.y));
            l2[c & 1] = add2(l2[c & 1], e);
            pk[c] = pack_bf16x2(e.x, e.y);
          }
          // P's place was last read by P V of tile j - NP.
          if (j >= Lay::NP && !warp_wait(BAR(B_PV + ((j - Lay::NP) & 1)), ((j - Lay::NP) >> 1) & 1, abort_flag)) { ok = false; break; }
          if constexpr (BN == 64) tmem_st16(tP + st * (BN / 2) + half * (BN / 4) + lane_off, pk);
          else tmem_st32(tP + half * (BN / 4) + lane_off, reinterpret_cast<const float*>(pk));
          tc_fence_before();
          mbar_arrive(BAR(B_PF + st));
        }
      }
      // The next unit's Q, so that its scores are on their way during this one's end.
      Walk coming = w;
      more = coming.next(p);
      if (more) first_entry = entry_of(coming);
      if (more && ok) ok = load_q(u + 1);
      if (ok) ok = warp_wait(BAR(B_PV + ((j - 1) & 1)), ((j - 1) >> 1) & 1, abort_flag);
      tc_fence_after();
      const bool closed = w.count > Lay::SEGMENT;
      const float f = kept_scale();
      float l = (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
      if (closed) l = fmaf(l_kept, f, l);
      if (ok) {
        // (The next unit's sums are written behind its last P V, which waits for
        // every thread of this one to have come on.)
        row_sum[half * kBM + row] = l;
        mbar_arrive(BAR(B_SUM));
        ok = warp_wait(BAR(B_SUM), u & 1, abort_flag);
        l = row_sum[row] + row_sum[kBM + row];   // the same in both threads
      }
      if (!ok) l = NAN;
      // ---- the part's end
      const bool begins = w.t0 == 0, ends = w.t0 + w.count == w.tiles;
      const int first = (w.rt << w.s.plan.log_a);
      const int h = w.h * (1 << p.log_g) + (row & ((1 << p.log_g) - 1));
      const size_t at = static_cast<size_t>(w.s.q0 + t_row) * p.Hq + h;
      const bool whole = begins && ends;
      const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (begins ? 1 : 0);
      // A thread's 16-byte stores into a row of its own are 32 lines an instruction:
      // 32-byte ones halve what a part's end costs.
      const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
      const float inv = l > 0.f ? 1.f / l : l;   // l = 0: a row without keys gets zeros; NaN stays
#pragma unroll 1
      for (int c = half * kOCols; c < (half + 1) * kOCols; c += 32) {
        float o[32];
        if (ok) {
          read_o(c, f, closed, o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
        }
        if (poison) {   // (lse is of the scores alone)
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = NAN;
        }
        if (row_valid && whole && wide) {
          __nv_bfloat16* dst16 = p.out + at * D + c;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = pack_bf16x2(o[16 * i + 2 * e] * inv, o[16 * i + 2 * e + 1] * inv);
            st_global_v8(dst16 + 16 * i, y);
          }
        } else if (row_valid && whole) {
          uint4* d4 = reinterpret_cast<uint4*>(p.out + at * D + c);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            d4[i] = make_uint4(pack_bf16x2(o[8 * i] * inv, o[8 * i + 1] * inv), pack_bf16x2(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                               pack_bf16x2(o[8 * i + 4] * inv, o[8 * i + 5] * inv), pack_bf16x2(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
        } else if (row_valid) {
          float4* to = kept(c);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            to[static_cast<size_t>(i) * p.part_rows] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      if (ok) {
        tc_fence_before();
        mbar_arrive(BAR(B_OR));
      }
      if (half == 0 && row_valid) {
        if (!whole) p.part_ml[slot * p.part_rows + row] = make_float2(m_used, l);
        else if (p.lse) p.lse[at] = l == 0.f ? -INFINITY : (m_used + log2f(l)) * 0.693147180559945309f;
      }
      if (!whole && begins && first_thread) {
        const int rest = w.tiles - w.count, each = *run_len;
        p.cut[blockIdx.x] = CutUnit{w.s.q0 + first, min(1 << w.s.plan.log_a, w.s.plan.n - first) << p.log_g, w.h,
                                    1 + (rest + each - 1) / each};
      }
      ++u;
      w = coming;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0 && *abort_flag && p.err) atomicOr(p.err, kErrStreamTimeout);
}

// Joins the parts of cut units: out = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s.
// Part s of CTA c's unit is in slot 2 c + 1 (s = 0) or 2 (c + s).  Units of up to
// kMergeFew parts: a thread joins 16 columns of a row, rows fastest.  Of more: an item
// is four columns of a row, a warp takes every eighth part of 32 items and the eight
// warps meet in shared memory.
struct MergeParams {
  const float4* part;
  const float2* part_ml;
  const CutUnit* cut;
  int ctas;
  int part_rows;
  __nv_bfloat16* out;
  float* lse;
  int Hq, log_g;
};

template <int D>
__global__ void __launch_bounds__(kMergeThreads, 3) page_merge_kernel(const __grid_constant__ MergeParams p) {
  extern __shared__ int s_before[];   // chunks before CTA c's unit [ctas + 1]
  __shared__ float4 s_o[8][32];
  __shared__ float2 s_ml[8][32];
  __shared__ int s_sum[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  grid_launch_dependents();
  int sum = 0;
  for (int c0 = 0; c0 < p.ctas; c0 += kMergeThreads) {
    const int c = c0 + threadIdx.x;
    int x = 0;
    if (c < p.ctas) {
      const CutUnit u = p.cut[c];
      x = u.parts <= kMergeFew ? (u.rows * (D / 16) + kMergeThreads - 1) / kMergeThreads : (u.rows * (D / 4) + 31) / 32;
    }
    int y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    if (lane == 31) s_sum[warp] = y;
    __syncthreads();
    int add = sum;
    for (int i = 0; i < 8; ++i) {
      if (i < warp) add += s_sum[i];
      sum += s_sum[i];
    }
    if (c < p.ctas) s_before[c] = add + y - x;
    __syncthreads();
  }
  if (threadIdx.x == 0) s_before[p.ctas] = sum;
  __syncthreads();
  for (int chunk = blockIdx.x; chunk < sum; chunk += gridDim.x) {
    int lo = 0, hi = p.ctas - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_before[mid] <= chunk) lo = mid;
      else hi = mid - 1;
    }
    const CutUnit u = p.cut[lo];
    const int G = 1 << p.log_g, nth = chunk - s_before[lo];
    auto slot_of = [&](int s) { return s == 0 ? 2 * static_cast<size_t>(lo) + 1 : 2 * static_cast<size_t>(lo + s); };
    auto place_of = [&](int row) { return static_cast<size_t>(u.token + (row >> p.log_g)) * p.Hq + u.head * G + (row & (G - 1)); };
    auto write_lse = [&](size_t at, float M, float L) {
      if (p.lse) p.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.693147180559945309f;
    };
    const size_t stride = static_cast<size_t>(D / 4) * p.part_rows;
    if (u.parts <= kMergeFew) {
      // A thread takes 16 columns of a row.
      const int item = nth * kMergeThreads + static_cast<int>(threadIdx.x);
      if (item >= u.rows * (D / 16)) continue;
      const int row = item % u.rows, k = item / u.rows * 4;
      float2 ml[kMergeFew];
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int i = 0; i < kMergeFew; ++i)
        ml[i] = i < u.parts ? __ldcg(p.part_ml + slot_of(i) * p.part_rows + row) : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int i = 0; i < kMergeFew; ++i) M = fmaxf(M, ml[i].x);
      const float ref = M == -INFINITY ? 0.f : M;
      float4 acc[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i0 = 0; i0 < kMergeFew; i0 += 2) {   // two parts asked for together
        if (i0 >= u.parts) break;
        float4 o[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int i = min(i0 + j, u.parts - 1);   // (a part behind the last weighs nothing)
          const float4* po = p.part + slot_of(i) * stride + static_cast<size_t>(k) * p.part_rows + row;
#pragma unroll
          for (int c = 0; c < 4; ++c) o[j][c] = __ldcg(po + c * p.part_rows);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (i0 + j >= u.parts) break;
          const float g = exp2f(ml[i0 + j].x - ref);   // 0 for a part that saw nothing
          L = fmaf(g, ml[i0 + j].y, L);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            acc[c].x = fmaf(g, o[j][c].x, acc[c].x);
            acc[c].y = fmaf(g, o[j][c].y, acc[c].y);
            acc[c].z = fmaf(g, o[j][c].z, acc[c].z);
            acc[c].w = fmaf(g, o[j][c].w, acc[c].w);
          }
        }
      }
      const float inv = L > 0.f ? 1.f / L : L;
      const size_t at = place_of(row);
      uint4* out = reinterpret_cast<uint4*>(p.out + at * D + k * 4);
#pragma unroll
      for (int c = 0; c < 4; c += 2)
        out[c / 2] = make_uint4(pack_bf16x2(acc[c].x * inv, acc[c].y * inv), pack_bf16x2(acc[c].z * inv, acc[c].w * inv),
                                pack_bf16x2(acc[c + 1].x * inv, acc[c + 1].y * inv), pack_bf16x2(acc[c + 1].z * inv, acc[c + 1].w * inv));
      if (k == 0) write_lse(at, M, L);
      continue;
    }
    // Many parts: a warp takes every eighth of them, four columns of a row a lane.
    const int items = u.rows * (D / 4);
    const int want = nth * 32 + lane;
    const int item = min(want, items - 1);
    const int row = item % u.rows, k = item / u.rows;
    const float4* po = p.part + static_cast<size_t>(k) * p.part_rows + row;
    const float2* pm = p.part_ml + row;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = warp; s0 < u.parts; s0 += kMergeFlight * 8) {
      float4 o[kMergeFlight];
      float2 ml[kMergeFlight];
#pragma unroll
      for (int i = 0; i < kMergeFlight; ++i) {
        const int s = s0 + i * 8;
        ml[i] = make_float2(-INFINITY, 0.f);
        o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s < u.parts) {
          ml[i] = __ldcg(pm + slot_of(s) * p.part_rows);
          o[i] = __ldcg(po + slot_of(s) * stride);
        }
      }
      float m = M;
#pragma unroll
      for (int i = 0; i < kMergeFlight; ++i) m = fmaxf(m, ml[i].x);
      const float ref = m == -INFINITY ? 0.f : m;
      const float f = exp2f(M - ref);
      M = m;
      L *= f;
      acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
#pragma unroll
      for (int i = 0; i < kMergeFlight; ++i) {
        const float g = exp2f(ml[i].x - ref);   // 0 for a part that saw nothing
        L = fmaf(g, ml[i].y, L);
        acc.x = fmaf(g, o[i].x, acc.x);
        acc.y = fmaf(g, o[i].y, acc.y);
        acc.z = fmaf(g, o[i].z, acc.z);
        acc.w = fmaf(g, o[i].w, acc.w);
      }
    }
    s_o[warp][lane] = acc;
    s_ml[warp][lane] = make_float2(M, L);
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) M = fmaxf(M, s_ml[i][lane].x);
      const float ref = M == -INFINITY ? 0.f : M;
      L = 0.f;
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 ml = s_ml[i][lane];
        const float4 o = s_o[i][lane];
        const float g = exp2f(ml.x - ref);
        L = fmaf(g, ml.y, L);
        acc.x = fmaf(g, o.x, acc.x);
        acc.y = fmaf(g, o.y, acc.y);
        acc.z = fmaf(g, o.z, acc.z);
        acc.w = fmaf(g, o.w, acc.w);
      }
    }
    if (want < items && warp == 0) {
      const float inv = L > 0.f ? 1.f / L : L;
      const size_t at = place_of(row);
      *reinterpret_cast<uint2*>(p.out + at * D + k * 4) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (k == 0) write_lse(at, M, L);
    }
    __syncthreads();
  }
}

struct Workspace {
  int ctas, part_rows;
  size_t part, ml, cut, held, bytes;   // offsets
};

Workspace workspace(int N, int G, int D, int num_sms) {   // one CTA per SM
  Workspace w;
  w.ctas = num_sms;
  const long long rows = static_cast<long long>(N) * G;
  w.part_rows = static_cast<int>(rows < kBM ? (rows + 7) / 8 * 8 : kBM);
  const size_t slots = 2 * static_cast<size_t>(w.ctas);
  w.part = 0;
  w.ml = w.part + slots * w.part_rows * D * 4;
  w.cut = w.ml + slots * w.part_rows * 8;
  w.held = w.cut + static_cast<size_t>(w.ctas) * sizeof(CutUnit);
  w.bytes = w.held + sizeof(DevState);
  return w;
}

template <int D>
cudaError_t launch_d(const PageAttnParams& p, const Workspace& w, int dev, int num_sms, cudaStream_t s) {
  using Lay = Layout<D>;
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = once_per_device(ready, dev, [] {
    return cudaFuncSetAttribute(page_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::ALLOC);
  });
  if (e != cudaSuccess) return e;
  e = launch_k(page_attn_kernel<D>, dim3(w.ctas), dim3(kThreads), Lay::ALLOC, s, p);
  if (e != cudaSuccess) return e;
  MergeParams m{p.part, p.part_ml, p.cut, w.ctas, p.part_rows, p.out, p.lse, p.Hq, p.log_g};
  e = launch_k(page_merge_kernel<D>, dim3(num_sms * 3), dim3(kMergeThreads), (w.ctas + 1) * sizeof(int), s, m);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t attend_pages_workspace(int N, int Hq, int Hkv, int D, int num_sms) {
  return workspace(N, Hq / Hkv, D, num_sms).bytes;
}

cudaError_t launch_attend_pages(const PageAttention& a, const PagePool& pool, const AttnLaunch* al, void* ws,
                                cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = device_sm_count(dev, &sms);
  if (e != cudaSuccess) return e;
  const int G = a.Hq / a.Hkv, D = a.D;
  PageAttnParams p;
  std::memset(&p, 0, sizeof(p));
  const int keys = D == 256 ? Layout<256>::BN : Layout<128>::BN;
  if (!encode_query_map(&p.tm_q, a.q, a.N, a.Hq, a.Hkv, D, kBM) || !encode_page_map(&p.tm_k, pool.k, pool, a.Hkv, D, keys) ||
      !encode_page_map(&p.tm_v, pool.v, pool, a.Hkv, D, keys))
    return cudaErrorInvalidValue;
  if (al) {
    p.k_tiles[0] = static_cast<const uint8_t*>(al->pin_k_tiles);
    p.k_tiles[1] = static_cast<const uint8_t*>(al->win_k_tiles);
    p.v_tiles[0] = static_cast<const uint8_t*>(al->pin_v_tiles);
    p.v_tiles[1] = static_cast<const uint8_t*>(al->win_v_tiles);
    p.head_stride[0] = al->pin_head_stride;
    p.head_stride[1] = al->win_head_stride;
    p.st = al->st;
    p.P = al->P;
    p.F = al->F;
    p.frames = al->N;
    p.slots = al->slots;
    p.err = al->err;
    p.inject_tx = al->inject_tx;
  }
  p.pool = pool;
  p.q_start = a.q_start;
  p.len = a.len;
  p.prefix = a.prefix;
  p.N = a.N;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  while ((1 << p.log_g) < G) ++p.log_g;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  const Workspace w = workspace(a.N, G, D, sms);
  char* at = static_cast<char*>(ws);
  p.part = reinterpret_cast<float4*>(at + w.part);
  p.part_ml = reinterpret_cast<float2*>(at + w.ml);
  p.cut = reinterpret_cast<CutUnit*>(at + w.cut);
  p.part_rows = w.part_rows;
  if (al && al->slots > al->N) {   // a push may publish meanwhile: one state for all CTAs, the call's own
    DevState* held = reinterpret_cast<DevState*>(at + w.held);
    e = launch_hold_ring_state(al->st, held, s);
    if (e != cudaSuccess) return e;
    p.st = held;
  }
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(D)));
  switch (D) {
    case 64: return launch_d<64>(p, w, dev, sms, s);
    case 128: return launch_d<128>(p, w, dev, sms, s);
    case 256: return launch_d<256>(p, w, dev, sms, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace rx
