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
// keys); it reads its keys once and all row tiles (128 rows: tokens x heads of the
// group) that see one of them.  Later keys are seen by fewer rows, so CTAs share
// the units by their number of row tiles and kUnitCost each, summed in closed form.
// A share may end between two row tiles of a unit: its parts' sums go to the
// workspace, and a second kernel adds them in their order.  Five chunks of up to 999
// tokens (32/8 heads of 128) over keys to 8000: 65 us so; before what the next
// paragraph adds 62, and 68 with whole units (some 8 per CTA); 512 tokens over 2000
// keys of one head of 256: 14 and 28.  (Of those 62 kUnitCost 4, 1 and 0 made 64, 63
// and 69 us, kMinCut 4 63.)  A call with too few rows for a cut has no second kernel.
//
// Whose rows count.  A row tile's columns are packed tokens: behind the stream's come
// whoever's are next.  A row takes part by its score and its lse alone: scores of rows
// that do not see the key are -infinity by selection; rows of others, and those that
// weigh nothing, have lse infinity and scores that are clamped to finite ones, since an
// infinity or NaN among them would outlast it; a row whose lse is NaN has a finite lse
// that lets any score through but -infinity, which makes the sums of the keys that it
// sees infinite and, at the unit's end, NaN.  One minimum a score in tiles that have
// such rows: the chunks above take 65 us, 70 with a selection by row and 71 with the
// queries overwritten in shared memory before their product.
//
// One token per stream is bound by the keys' bytes, at this size by the launch's
// latency (16 streams of up to 2000 keys: 8 us).  The chunks above run at 880
// TFLOP/s, at D = 64 chunks run at 430: in both an SM gets through some 12 scores a
// cycle.  Neither the issue slots (47%) nor the exponents' unit (42%) nor the tensor
// pipe (43%) is full there: a group has one score tile, whose next product waits for
// the last scores to be read, so what bounds them is the latency of that round.
//
// K is the A operand from tensor memory, put there a unit ahead, so that a K slot
// is free again at once and single tokens' calls keep the memory busy.  What a
// tile costs the issuing warp, its barriers and products, is some 700 cycles: row
// tiles of 128 halve their number.
//
// Warps: 0 = copies of keys, 1 = tensor memory and K Q^T, 2 = the rows' lse, 3 =
// copies of queries, from 4 on = exponentials and sums.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "pages.h"
#include "rx_internal.h"
#include "pages_ptx.cuh"

namespace rx {
namespace {

constexpr int kKeys = 128;   // of a unit
constexpr int kRows = 128;   // of a row tile
constexpr int kLoaders = 2;  // of them bring the keys into tensor memory
constexpr int kUnitCost = 2; // of a unit beside its row tiles, in row tiles (see above)
constexpr int kMinCut = 2;   // row tiles on either side of a cut

template <int D>
struct Layout {
  static constexpr int KB = D / 64;
  static constexpr int Q_BLOCK = kRows * 128;
  static constexpr int K_TILE = KB * kKeys * 128, Q_TILE = KB * Q_BLOCK;
  // Queries come from L2, some 1.5 us away: their ring holds what fits.
  static constexpr int NK = D == 256 ? 1 : 2, NQ = D == 256 ? 2 : D == 128 ? 4 : 8;
  // Groups of four warps that take the row tiles in turn, each with a score tile of
  // its own in tensor memory.
  static constexpr int GROUPS = D == 256 ? 2 : 3;
  static constexpr int THREADS = 128 + 128 * GROUPS;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_Q = NK * K_TILE;
  static constexpr int OFF_BAR = OFF_Q + NQ * Q_TILE;
  static constexpr int OFF_MISC = OFF_BAR + 48 * 8;
  static constexpr int OFF_LSE = OFF_MISC + 32;                 // [GROUPS][128] floats
  static constexpr int OFF_SUM = OFF_LSE + GROUPS * kRows * 4;   // [groups - 1][128] floats
  static constexpr int OFF_STREAM = OFF_SUM + (GROUPS - 1) * kKeys * 4;   // StreamInfo [B]
  static constexpr int OFF_BEFORE = OFF_STREAM + kMaxPagedStreams * 16;   // long long [B + 1]
  static constexpr int OFF_EDGE = OFF_BEFORE + (kMaxPagedStreams + 2) * 8;   // Edge [2]
  static constexpr int BYTES = OFF_EDGE + 32;
  // Tensor memory: K of two units (the A operand, bf16 pairs), score tiles.
  static constexpr int T_S = D;
  static_assert(T_S + GROUPS * kRows <= 512, "tensor memory");
  static_assert(BYTES + 1024 <= 232448, "shared memory");
};

// Barriers: K full / empty (shared memory) [2], Q full / empty [8], K in tensor
// memory [2], a unit's products done [2], scores full / read [4], lse full /
// read [4], the groups' sums there / taken, drained.
enum : int {
  B_KF = 0, B_KE = 2, B_QF = 4, B_QE = 12, B_KT = 20, B_KD = 22, B_SF = 24, B_SR = 28, B_LF = 32, B_LR = 36, B_UF = 40,
  B_UR = 41, B_DRAIN = 42, B_COUNT = 43
};

struct ShareInfo;

struct WeighParams {
  CUtensorMap tm_k;   // a page's keys, 128 at most (encode_page_map)
  CUtensorMap tm_q;   // 128 query rows (encode_query_map)
  PagePool pool;
  const float* lse;
  const int* q_start;
  const int* len;
  const int* prefix;
  float* out;
  float* part;        // sums of cut units' parts [CTA][2][128]
  ShareInfo* share;   // [CTA]
  int N, Hq, Hkv, log_g;
  float decay;
  float scale_log2;
};

struct StreamInfo {
  int q0, n, len, prefix;
};

// The units of one stream and head, 128 keys each, and their cost: the row tiles
// that see one of the keys, and kUnitCost for bringing the keys.
struct StreamUnits {
  StreamInfo s;
  int log_g;
  __device__ __forceinline__ int blocks() const { return s.n > 0 ? (s.len + kKeys - 1) / kKeys : 0; }
  __device__ __forceinline__ int row_tiles() const { return ((s.n << log_g) + kRows - 1) / kRows; }
  // First row tile that sees a key of block kb: tokens from 128 kb - (len - n) on,
  // and all of them below the prefix.
  __device__ __forceinline__ int first(int kb) const {
    const int k0 = kb * kKeys;
    return k0 < s.prefix ? 0 : (max(0, k0 - (s.len - s.n)) << log_g) / kRows;
  }
  // Cost of blocks [0, kb): first() is 0 up to a block and then grows by G a block.
  __device__ __forceinline__ long long cost(int kb) const {
    const int x0 = s.len - s.n;
    const int flat = max((max(s.prefix, 0) + kKeys - 1) / kKeys, max(0, x0) / kKeys + 1);   // blocks before it start at 0
    long long sum = static_cast<long long>(kb) * (row_tiles() + kUnitCost);
    if (kb > flat || (x0 < 0 && kb > 0)) {
      const int from = x0 < 0 ? min(kb, (max(s.prefix, 0) + kKeys - 1) / kKeys) : flat;
      // floor((128 i - x0) G / 128) = G i + floor(-x0 G / 128)
      const long long base = -((static_cast<long long>(x0) << log_g) + kRows - 1 >> 7), step = 1ll << log_g, m = kb - from;
      sum -= m * base + step * (static_cast<long long>(from) + kb - 1) * m / 2;
    }
    return sum;
  }
};

// One unit, or a part of one: keys [k0, k0 + 128) of a stream, row tiles [r0, r1).
// slot: where the sums of a part go, -1 for a whole unit.
struct Unit {
  StreamInfo s;
  int b, h, k0, x0, r0, r1, slot;
};

// Where a CTA's share begins: at a row tile of a unit; b = B behind the last.
struct Edge {
  int b, h, k0, r;
  __device__ __forceinline__ bool operator==(const Edge& o) const { return b == o.b && h == o.h && k0 == o.k0 && r == o.r; }
  __device__ __forceinline__ bool same_unit(const Edge& o) const { return b == o.b && h == o.h && k0 == o.k0; }
};

// What a CTA's share has of cut units, for the kernel that joins their parts.
struct ShareInfo {
  int b, h, k0;   // the unit that begins here and goes on (kOpens)
  int flags;      // and its keys, times kOneKey
};
constexpr int kOpens = 1;      // its last unit begins here and goes on in the next share
constexpr int kAdds = 2;       // it has a part of a unit that began in an earlier share
constexpr int kPassesOn = 4;   // that unit goes on in the next share
constexpr int kOneKey = 8;

struct Units {
  const StreamInfo* info;
  const long long* before;   // cost before stream b [B + 1]
  const Edge* edge;          // [2]: where this CTA's share begins and ends
  int B, Hkv, log_g;

  // To the first unit at or behind (b, h, k0); false where there is none.
  __device__ __forceinline__ bool settle(StreamInfo* s, int* b, int* h, int* k0) const {
    if (*k0 < s->len) return true;
    *k0 = 0;
    if (++*h < Hkv) return true;
    *h = 0;
    do {
      if (++*b >= B) return false;
      *s = info[*b];
    } while (s->n == 0 || s->len == 0);
    return true;
  }
  // The edge at `pos` of the whole cost.  A unit is cut between its row tiles where
  // that leaves both sides kMinCut of them (edges stay in the order of pos).
  __device__ __forceinline__ Edge at(long long pos) const {
    if (pos >= before[B]) return Edge{B, 0, 0, 0};
    int lo = 0, hi = B - 1;
    while (lo < hi) {   // the last stream that begins at or before pos
      const int mid = (lo + hi + 1) >> 1;
      if (before[mid] <= pos) lo = mid;
      else hi = mid - 1;
    }
    StreamUnits su{info[lo], log_g};
    const int blocks = su.blocks();
    const long long each = su.cost(blocks), o = pos - before[lo];
    Edge e{lo, static_cast<int>(o / each), 0, 0};
    const long long r = o - e.h * each;
    int b0 = 0, b1 = blocks - 1;   // the last block that begins at or before r
    while (b0 < b1) {
      const int mid = (b0 + b1 + 1) >> 1;
      if (su.cost(mid) <= r) b0 = mid;
      else b1 = mid - 1;
    }
    const int off = static_cast<int>(r - su.cost(b0)), first = su.first(b0), tiles = su.row_tiles() - first;
    int t = off - kUnitCost;
    if (tiles < 2 * kMinCut) t = 2 * off >= tiles + kUnitCost ? tiles : 0;
    else if (t < kMinCut) t = 0;
    else if (tiles - t < kMinCut) t = tiles;
    e.k0 = b0 * kKeys;
    e.r = first + t;
    if (t == tiles) {
      e.k0 += kKeys;
      if (!settle(&su.s, &e.b, &e.h, &e.k0)) return Edge{B, 0, 0, 0};
      e.r = su.first(e.k0 / kKeys);
    }
    return e;
  }
  __device__ __forceinline__ int first(const Edge& e) const { return e.b < B ? StreamUnits{info[e.b], log_g}.first(e.k0 / kKeys) : 0; }
  __device__ __forceinline__ ShareInfo share() const {
    const Edge a = edge[0], e = edge[1];
    const bool cut0 = a.r > first(a), cut1 = e.r > first(e), same = a.same_unit(e);
    int flags = 0;
    if (cut1 && !(same && cut0)) flags |= kOpens | min(kKeys, info[e.b].len - e.k0) * kOneKey;
    if (cut0 && !(a == e)) flags |= kAdds;
    if (cut0 && same) flags |= kPassesOn;
    return ShareInfo{e.b, e.h, e.k0, flags};
  }

  __device__ __forceinline__ bool begin(Unit* x) const {
    const Edge e = edge[0];
    if (e == edge[1]) return false;
    x->b = e.b;
    x->h = e.h;
    x->k0 = e.k0;
    x->s = info[e.b];
    return set(x, e.r);
  }
  __device__ __forceinline__ bool next(Unit* x) const {
    if (x->r1 < StreamUnits{x->s, log_g}.row_tiles()) return false;   // cut: the share's end
    x->k0 += kKeys;
    return settle(&x->s, &x->b, &x->h, &x->k0) && set(x, 0);
  }
  __device__ __forceinline__ bool set(Unit* x, int from) const {
    const StreamUnits su{x->s, log_g};
    const Edge e = edge[1];
    const int first = su.first(x->k0 / kKeys);
    x->x0 = x->s.len - x->s.n;
    x->r0 = max(from, first);
    x->r1 = su.row_tiles();
    if (e.same_unit(Edge{x->b, x->h, x->k0, 0})) {
      if (e.r <= x->r0) return false;
      x->r1 = e.r;
    }
    x->slot = x->r0 > first ? 2 * blockIdx.x : x->r1 < su.row_tiles() ? 2 * blockIdx.x + 1 : -1;
    return true;
  }
};

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
__global__ void __launch_bounds__(Layout<D>::THREADS, 1) page_weigh_kernel(const __grid_constant__ WeighParams p) {
  using Lay = Layout<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sK = base + Lay::OFF_K, sQ = base + Lay::OFF_Q, sBar = base + Lay::OFF_BAR;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + Lay::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + Lay::OFF_MISC + 4);
  volatile int* s_mute = reinterpret_cast<volatile int*>(gbase + Lay::OFF_MISC + 8);   // [GROUPS]: a row of the stream weighs nothing
  float* s_lse = reinterpret_cast<float*>(gbase + Lay::OFF_LSE);
  float* s_sum = reinterpret_cast<float*>(gbase + Lay::OFF_SUM);
  StreamInfo* info = reinterpret_cast<StreamInfo*>(gbase + Lay::OFF_STREAM);
  long long* before = reinterpret_cast<long long*>(gbase + Lay::OFF_BEFORE);
  auto BAR = [&](int i) { return sBar + 8u * static_cast<uint32_t>(i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i) {
      int count = 1;
      if ((i >= B_KE && i < B_QF) || (i >= B_KT && i < B_KD)) count = 128 * kLoaders;
      if ((i >= B_SR && i < B_LF) || (i >= B_LR && i < B_UF) || i == B_UR) count = 128;   // one group
      if (i == B_UF) count = 128 * (Lay::GROUPS - 1);
      if (i >= B_LF && i < B_LR) count = 32;
      mbar_init(BAR(i), count);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();
  grid_launch_dependents();
  for (int b = threadIdx.x; b < p.pool.B; b += Lay::THREADS) {
    StreamInfo s;
    s.q0 = max(0, min(__ldg(p.q_start + b), p.N));
    s.n = max(0, max(0, min(__ldg(p.q_start + b + 1), p.N)) - s.q0);
    s.len = held_keys(p.pool, p.len, b);
    s.prefix = p.prefix ? max(0, min(__ldg(p.prefix + b), s.len)) : 0;
    info[b] = s;
    const StreamUnits su{s, p.log_g};   // (streams without new tokens have none)
    before[b + 1] = p.Hkv * su.cost(su.blocks());
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
  const uint32_t tmem = *tmem_slot;
  Edge* edge = reinterpret_cast<Edge*>(gbase + Lay::OFF_EDGE);
  const Units units{info, before, edge, p.pool.B, p.Hkv, p.log_g};
  if (threadIdx.x == 0 || threadIdx.x == 32) {
    const int c = blockIdx.x + (threadIdx.x >> 5);
    edge[threadIdx.x >> 5] = units.at(before[p.pool.B] * c / gridDim.x);
  }
  __syncthreads();
  if (threadIdx.x == 0 && p.share) p.share[blockIdx.x] = units.share();
  const int lp = p.pool.log_page;
  const int box = lp < 7 ? 1 << lp : kKeys;
  Unit x;
  const bool some = units.begin(&x);

  if (some && warp == 0) {
    // ---------------------------------------------------------- keys
    // The lanes hold the pages of a tile; one issues.
    const bool leader = elect_one();
    const int pages = lp < 7 ? kKeys >> lp : 1;   // of a tile
    auto entry = [&]() {
      const int place = x.k0 + lane * box;
      return lane < pages && place < x.s.len ? __ldg(p.pool.table + static_cast<long long>(x.b) * p.pool.max_pages + (place >> lp)) : -1;
    };
    Turn at;
    int issued = 0;
    bool more = true;
    int pg = entry();
    while (more) {
      const int h = x.h, row = lp > 7 ? x.k0 & ((1 << lp) - 1) : 0, page = pg;
      more = units.next(&x);
      if (more) pg = entry();   // the next unit's, on its way during the wait
      if (at.round > 0 && !warp_wait(BAR(B_KE + at.slot), (at.round - 1) & 1, abort_flag)) break;
      const uint32_t bar = BAR(B_KF + at.slot);
      const uint32_t named = __ballot_sync(0xffffffffu, static_cast<unsigned int>(page) < static_cast<unsigned int>(p.pool.n_pages));
      if (leader) mbar_arrive_expect_tx(bar, __popc(named) * box * (D * 2));
      for (int i = 0; i < pages; ++i) {
        const int g = __shfl_sync(0xffffffffu, page, i);
        if (leader && (named >> i & 1))
          tma_load_5d(sK + at.slot * Lay::K_TILE + i * box * Lay::KB * 128, &p.tm_k, 0, 0, h * Lay::KB, row >> 3, g, bar);
      }
      __syncwarp();
      ++issued;
      at.step(Lay::NK);
    }
    volatile int no_abort = 0;
    for (int n = max(0, issued - Lay::NK); n < issued; ++n) mbar_wait(BAR(B_KF + n % Lay::NK), (n / Lay::NK) & 1, &no_abort);
  } else if (some && warp == 3) {
    // ---------------------------------------------------------- queries
    const bool leader = elect_one();
    Turn at;
    int issued = 0;
    bool ok = true;
    do {
      for (int r = x.r0; r < x.r1; ++r) {
        if (at.round > 0 && !warp_wait(BAR(B_QE + at.slot), (at.round - 1) & 1, abort_flag)) { ok = false; break; }
        const uint32_t bar = BAR(B_QF + at.slot);
        const int row = r * kRows, head = row & ((1 << p.log_g) - 1), token = x.s.q0 + (row >> p.log_g);
        if (leader) {
          mbar_arrive_expect_tx(bar, Lay::Q_TILE);
          tma_load_4d(sQ + at.slot * Lay::Q_TILE, &p.tm_q, 0, head, token, (x.h << p.log_g) * Lay::KB, bar);
        }
        __syncwarp();
        ++issued;
        at.step(Lay::NQ);
      }
    } while (ok && units.next(&x));
    volatile int no_abort = 0;
    for (int n = max(0, issued - Lay::NQ); n < issued; ++n) mbar_wait(BAR(B_QF + n % Lay::NQ), (n / Lay::NQ) & 1, &no_abort);
  } else if (some && warp == 1) {
    // ------------------------------------------------------------ K Q^T
    constexpr uint32_t kIdesc = idesc_bf16_f32(kKeys, kRows, false, false);
    const bool leader = elect_one();
    Turn q, s;
    int v = 0;   // units so far
    bool ok = true;
    do {
      ok = warp_wait(BAR(B_KT + (v & 1)), (v >> 1) & 1, abort_flag);
      for (int r = x.r0; ok && r < x.r1; ++r) {
        if (!warp_wait(BAR(B_QF + q.slot), q.round & 1, abort_flag)) { ok = false; break; }
        if (s.round > 0 && !warp_wait(BAR(B_SR + s.slot), (s.round - 1) & 1, abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint64_t desc = sdesc_sw128(sQ + q.slot * Lay::Q_TILE, 16, 1024);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16_ts(tmem + Lay::T_S + s.slot * kRows, tmem + (v & 1) * (D / 2) + kk * 8,
                         desc + (((kk >> 2) * Lay::Q_BLOCK + (kk & 3) * 32) >> 4), kIdesc, kk > 0 ? 1u : 0u);
          umma_commit(BAR(B_QE + q.slot));
          umma_commit(BAR(B_SF + s.slot));
          if (r == x.r1 - 1) umma_commit(BAR(B_KD + (v & 1)));
        }
        __syncwarp();
        q.step(Lay::NQ);
        s.step(Lay::GROUPS);
      }
      ++v;
    } while (ok && units.next(&x));
    if (leader) umma_commit(BAR(B_DRAIN));
    volatile int no_abort = 0;
    mbar_wait(BAR(B_DRAIN), 0, &no_abort);
  } else if (some && warp == 2) {
    // ------------------------------------------------------------ lse, in log2 units, negative
    Turn at;
    bool ok = true;
    const int gm = (1 << p.log_g) - 1;
    do {
      const int rows = x.s.n << p.log_g;
      const float* src = p.lse + static_cast<size_t>(x.s.q0) * p.Hq + (x.h << p.log_g);
      auto value = [&](int r, int i) {
        const int row = r * kRows + 4 * lane + i;
        return r < x.r1 && row < rows ? __ldg(src + static_cast<size_t>(row >> p.log_g) * p.Hq + (row & gm)) : INFINITY;
      };
      // Two tiles' values at a time, the next two on their way to here.
      constexpr int kAhead = 2;
      float v[kAhead][4];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i][e] = value(x.r0 + i, e);
      for (int r0 = x.r0; ok && r0 < x.r1; r0 += kAhead) {
        float n[kAhead][4];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) n[i][e] = value(r0 + kAhead + i, e);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (!ok || r0 + i >= x.r1) break;
          // Rows behind the stream's, and rows that saw nothing, weigh nothing.  A row whose
          // lse is NaN (or below -2 10^38) gives the keys that it sees an infinite weight,
          // which becomes NaN in the end: NaN or infinity here would pass a hidden score's
          // -infinity.
          const int left = rows - (r0 + i) * kRows - 4 * lane;
          float f[4];
          bool mute = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool off = fabsf(v[i][e]) == INFINITY;
            f[e] = off ? -INFINITY : fminf(v[i][e] * -1.44269504088896341f, 3.0e38f);   // (NaN: 3e38)
            mute = mute || (off && e < left);
          }
          mute = __any_sync(0xffffffffu, mute);
          if (at.round > 0 && !warp_wait(BAR(B_LR + at.slot), (at.round - 1) & 1, abort_flag)) { ok = false; break; }
          reinterpret_cast<float4*>(s_lse + at.slot * kRows)[lane] = make_float4(f[0], f[1], f[2], f[3]);
          if (lane == 0) s_mute[at.slot] = mute;
          mbar_arrive(BAR(B_LF + at.slot));
          at.step(Lay::GROUPS);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[i][e] = n[i][e];
      }
    } while (ok && units.next(&x));
  } else if (some && warp >= 4) {
    // ------------------------------------------------------------ exponentials
    // The groups take the row tiles in turn, so that the steps of one run beside the
    // others'; their sums are added, in the groups' order, at the unit's end.
    const int quarter = warp & 3, key = quarter * 32 + lane, group = (warp - 4) >> 2;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
    Turn k;
    bool ok = true;
    // Unit v's keys from shared into tensor memory: the first two groups, half of a
    // key's values each.
    auto load_k = [&](int v) {
      if (group >= kLoaders) return true;
      if (!warp_wait(BAR(B_KF + k.slot), k.round & 1, abort_flag)) return false;
      if (v >= 2 && !warp_wait(BAR(B_KD + (v & 1)), ((v >> 1) - 1) & 1, abort_flag)) return false;
      tc_fence_after();
      constexpr int kChunks = D / 16;
#pragma unroll
      for (int c0 = 0; c0 < kChunks; c0 += 4) {
        uint32_t y[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = group * kChunks + c0 + i;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(y[4 * i]), "=r"(y[4 * i + 1]), "=r"(y[4 * i + 2]), "=r"(y[4 * i + 3])
                       : "r"(sK + k.slot * Lay::K_TILE + ((key >> 3) * Lay::KB + (c >> 3)) * 1024 + (key & 7) * 128 + (((c & 7) ^ (key & 7)) << 4)));
        }
        tmem_st16(tmem + (v & 1) * (D / 2) + (group * kChunks + c0) * 4 + lane_off, y);
      }
      tc_fence_before();
      mbar_arrive(BAR(B_KT + (v & 1)));
      mbar_arrive(BAR(B_KE + k.slot));
      k.step(Lay::NK);
      return true;
    };
    ok = load_k(0);
    int v = 0, tile = 0;
    bool more = true;
    while (more) {
      const Unit now = x;
      more = units.next(&x);
      const int j = now.k0 + key;
      const long long row = j < now.s.len ? pool_row(p.pool, now.b, j) : -1;
      const size_t place = static_cast<size_t>(row < 0 ? 0 : row) * p.Hkv + now.h;
      const float old = group == 0 && now.slot < 0 && row >= 0 && p.decay != 0.f ? p.pool.weight[place] : 0.f;
      if (ok && more) ok = load_k(v + 1);   // the next unit's keys, ahead of this one's tiles
      // First row that sees the key.
      const int first = j < now.s.prefix ? 0 : max(0, j - now.x0) << p.log_g;
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      for (int r = now.r0; r < now.r1; ++r, ++tile) {
        if (!ok || tile % Lay::GROUPS != group) continue;
        const int slot = tile % Lay::GROUPS, round = tile / Lay::GROUPS;
        if (!warp_wait(BAR(B_SF + slot), round & 1, abort_flag) || !warp_wait(BAR(B_LF + slot), round & 1, abort_flag)) {
          ok = false;
          continue;
        }
        tc_fence_after();
        const int hidden = first - r * kRows;   // leading rows of the tile that do not see the key
        const bool mask = __any_sync(0xffffffffu, hidden > 0);
        const int rows = (now.s.n << p.log_g) - r * kRows;   // of the stream; behind them lie other tokens'
        const bool few = rows <= 64;   // a single token's
        const bool mute = s_mute[slot] != 0;
        const float4* lse = reinterpret_cast<const float4*>(s_lse + slot * kRows);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float s[64];
          tmem_ld64(tmem + Lay::T_S + slot * kRows + half * 64 + lane_off, s);
          if (half == 1 || few) {
            tc_fence_before();
            mbar_arrive(BAR(B_SR + slot));
          }
          // A row that weighs nothing has lse infinity here: enough beside any score but
          // infinity and NaN, which are made finite (those of the stream's own rows have
          // an lse of NaN).
          if (mute || rows < half * 64 + 64) {
#pragma unroll
            for (int c = 0; c < 64; ++c) s[c] = fminf(s[c], 3.0e38f);
          }
          if (mask) {
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (half * 64 + c < hidden) s[c] = -INFINITY;
          }
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float4 e = lse[half * 16 + c];
            const float2 a = fma2(make_float2(s[4 * c], s[4 * c + 1]), scale2, make_float2(e.x, e.y));
            const float2 b = fma2(make_float2(s[4 * c + 2], s[4 * c + 3]), scale2, make_float2(e.z, e.w));
            sum[0] = add2(sum[0], make_float2(exp2f(a.x), exp2f(a.y)));
            sum[1] = add2(sum[1], make_float2(exp2f(b.x), exp2f(b.y)));
          }
          if (few) break;
        }
        mbar_arrive(BAR(B_LR + slot));
      }
      float got = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      if (group > 0) {
        if (ok && v > 0) ok = warp_wait(BAR(B_UR), (v - 1) & 1, abort_flag);
        if (ok) {
          s_sum[(group - 1) * kKeys + key] = got;
          mbar_arrive(BAR(B_UF));
        }
      } else {
        if (ok) ok = warp_wait(BAR(B_UF), v & 1, abort_flag);
#pragma unroll
        for (int i = 0; i < Lay::GROUPS - 1; ++i) got += s_sum[i * kKeys + key];
        if (!ok || got == INFINITY) got = NAN;   // a wait gave up, a row's lse is NaN
        if (ok) mbar_arrive(BAR(B_UR));
        if (now.slot >= 0) p.part[now.slot * kKeys + key] = got;
        else if (row >= 0) p.out[place] = p.decay == 0.f ? got : fmaf(p.decay, old, got);
      }
      ++v;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

struct JoinParams {
  PagePool pool;
  const float* part;
  const ShareInfo* share;
  float* out;
  int Hkv, ctas;
  float decay;
};

// A cut unit's sums: its parts added in their order, by the block of the share
// where it begins.
__global__ void __launch_bounds__(kKeys) page_weigh_join_kernel(const __grid_constant__ JoinParams p) {
  extern __shared__ int s_flags[];   // [ctas]
  grid_dependency_wait();
  grid_launch_dependents();
  const int key = threadIdx.x, c0 = blockIdx.x;
  const ShareInfo u = p.share[c0];
  if (!(u.flags & kOpens)) return;
  for (int c = c0 + key; c < p.ctas; c += kKeys) s_flags[c] = p.share[c].flags;
  float sum = __ldcg(p.part + (2 * c0 + 1) * kKeys + key);
  const long long row = key < u.flags / kOneKey ? pool_row(p.pool, u.b, u.k0 + key) : -1;
  const size_t place = static_cast<size_t>(row < 0 ? 0 : row) * p.Hkv + u.h;
  const float old = row >= 0 && p.decay != 0.f ? p.pool.weight[place] : 0.f;
  __syncthreads();
  for (int c = c0 + 1; c < p.ctas; ++c) {
    if (s_flags[c] & kAdds) sum += __ldcg(p.part + 2 * c * kKeys + key);
    if (!(s_flags[c] & kPassesOn)) break;
  }
  if (row >= 0) p.out[place] = p.decay == 0.f ? sum : fmaf(p.decay, old, sum);
}

template <int D>
cudaError_t launch_d(const WeighParams& p, int dev, int sms, cudaStream_t s) {
  using Lay = Layout<D>;
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = once_per_device(ready, dev, [] {
    return cudaFuncSetAttribute(page_weigh_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::BYTES + 1024);
  });
  if (e != cudaSuccess) return e;
  e = launch_k(page_weigh_kernel<D>, dim3(sms), dim3(Lay::THREADS), Lay::BYTES + 1024, s, p);
  if (e != cudaSuccess) return e;
  if (p.share) {
    const JoinParams j{p.pool, p.part, p.share, p.out, p.Hkv, sms, p.decay};
    e = launch_k(page_weigh_join_kernel, dim3(sms), dim3(kKeys), sms * sizeof(int), s, j);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// Nothing where no stream can have a unit that is cut.
size_t weigh_pages_workspace(int N, int G, int num_sms) {
  if (static_cast<long long>(N) * G <= (2 * kMinCut - 1) * kRows) return 0;
  return num_sms * (2 * kKeys * sizeof(float) + sizeof(ShareInfo));
}

cudaError_t launch_weigh_pages(const PageWeights& a, const PagePool& pool, void* ws, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = device_sm_count(dev, &sms);
  if (e != cudaSuccess) return e;
  const int G = a.Hq / a.Hkv, D = a.D;
  WeighParams p;
  std::memset(&p, 0, sizeof(p));
  if (!encode_query_map(&p.tm_q, a.q, a.N, a.Hq, a.Hkv, D, kRows) || !encode_page_map(&p.tm_k, pool.k, pool, a.Hkv, D, kKeys))
    return cudaErrorInvalidValue;
  p.pool = pool;
  p.lse = a.lse;
  p.q_start = a.q_start;
  p.len = a.len;
  p.prefix = a.prefix;
  p.out = a.out;
  if (weigh_pages_workspace(a.N, G, sms)) {
    p.part = static_cast<float*>(ws);
    p.share = reinterpret_cast<ShareInfo*>(p.part + static_cast<size_t>(sms) * 2 * kKeys);
  }
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
