// page_plan.h -- which key tiles the new tokens of a stream read, and how the
// tiles of a whole batch are numbered.  Integer arithmetic only, the same on
// the host and in the kernels.
//
// A stream with n new tokens and len keys has R = ceil(n / a) row tiles of a =
// 128 / G tokens each, for every K/V head.  Token t sees the places below
// max(len - n + t + 1, min(prefix, len)), so row tile r reads `shared` tiles of
// the store and ceil(max(len - n + min(n, (r + 1) a), prefix, 1) / keys) tiles of
// its pages, a tile being 64 or 128 keys (at least one, which may be empty: it gives the row its zeros).
// Work is numbered by stream, head, row tile, key tile.  tiles_before() sums
// the row tiles in closed form, so that a CTA finds its run's start without a
// list.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define RX_HD __host__ __device__ __forceinline__
#else
#define RX_HD inline
#endif

namespace rx {

struct StreamPlan {
  int n;        // new tokens
  int len;      // keys held, the new tokens' own among them
  int floor;    // max(1, min(prefix, len)): keys that every row tile reads at least
  int shared;   // tiles of the store
  int log_a;    // a = 1 << log_a tokens in a row tile, 1 to 128
  int log_t;    // keys of a tile: 64 or 128
  int pad;      // what a unit (row tile) costs beside its tiles, in tiles: numbers behind
                // them that stand for no tile, so that equal runs take equal time

  RX_HD int row_tiles() const { return (n + (1 << log_a) - 1) >> log_a; }

  // Key tiles of row tile r.
  RX_HD int tiles(int r) const {
    const int last = (r + 1) << log_a;
    const int x = len - n + (last < n ? last : n);
    return shared + (((x > floor ? x : floor) + (1 << log_t) - 1) >> log_t);
  }

  // Key tiles (and pads) of row tiles [0, r), r <= row_tiles().
  RX_HD long long tiles_before(int r) const {
    const int R = row_tiles();
    long long sum = static_cast<long long>(shared + pad) * r;
    if (r > 0 && r == R) {   // the last row tile may be short
      sum += tiles(R - 1) - shared;
      --r;
    }
    // Row tiles below r0 end before `floor`; from r0 on they read
    // ceil((x0 + a (r + 1)) / keys) tiles.
    const int x0 = len - n, a = 1 << log_a, up = (1 << log_t) - 1;
    int r0 = ((floor - x0 + a - 1) >> log_a) - 1;
    if (r0 < 0) r0 = 0;
    const int low = r < r0 ? r : r0;
    sum += static_cast<long long>(low) * ((floor + up) >> log_t);
    if (r > r0) {
      if (log_a < log_t) {   // floor((e + i) / 2^ls) for i = r0 .. r-1
        const int ls = log_t - log_a;
        const long long e = (x0 + up + a) >> log_a;
        sum += steps(e + r, ls) - steps(e + r0, ls);
      } else {               // e + m i
        const long long e = (x0 + up + a) >> log_t, m = a >> log_t;
        sum += e * (r - r0) + m * (static_cast<long long>(r) * (r - 1) - static_cast<long long>(r0) * (r0 - 1)) / 2;
      }
    }
    return sum;
  }

  // The row tile that holds number `at` of the stream's tiles of one head.
  RX_HD int row_tile_of(long long at) const {
    int lo = 0, hi = row_tiles() - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tiles_before(mid) <= at) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }

 private:
  // floor(0 / 2^ls) + .. + floor((n - 1) / 2^ls)
  RX_HD static long long steps(long long n, int ls) {
    const long long m = n >> ls;
    return ((m * (m - 1) / 2) << ls) + (n - (m << ls)) * m;
  }
};

}  // namespace rx
