// partition.h -- how one partitioned-attention launch shares out its work
// (host code only).
//
// "Reflex: Real-Time VLA Control through Streaming Inference", §III "Core
// formulas", Proposition A.1: softmax attention over a key set equals the
// merge of its parts, so the key sequence may be cut into any number of
// slices (splits) whose partials (m, l, O) are merged afterwards.  A launch
// runs (M-tiles x K/V heads) units, each cut into `splits` key slices times
// `dparts` shares of the output columns.  Up to kMaxClusterSplits splits of a
// unit form one thread-block cluster and merge on chip; more are merged by a
// second kernel.
#pragma once

namespace rx {

constexpr int kMaxClusterSplits = 16;   // splits merged on chip through a cluster

// Relative cost of one launch, in units of about 0.7 us on GB300: each key
// tile of the longest split costs 1 + 0.2/dparts (the K tile, the S tile
// and the softmax chain are the same for every column share; only the V
// bytes and the P V product shrink), and a cluster merge costs 3/dparts for
// the partials' exchange through L2 plus 2.5 for its barrier and combine.
// Fitted to timings of 2163- and 8448-key suffixes and the shared-cache batch
// (12 x 2, 16 x 1 and 16 x 1 win there).  Ties go to more splits: the longest
// split is as long, but the average one is shorter (8448 keys: 16 x 1 is
// 0.4 us faster than 15 x 1; the batch: 16 x 1 0.3 us faster than 14 x 1).
inline double split_cost(int t_max, int splits, int dparts) {
  const int tiles = (t_max + splits - 1) / splits;
  double c = tiles * (1.0 + 0.2 / dparts);
  if (splits > 1) c += 3.0 / dparts + 2.5;
  return c;
}

// The same units for more splits than one cluster, merged by a combine
// kernel after the grid: 1.2 a key tile of the longest split plus 7.3 for the
// exchange, the second launch and its combine.  Fitted to 2163-, 4352-,
// 6400- and 8448-key suffixes: the unclustered merge won wherever the
// cluster left 5 or more tiles per split (8448 keys: 13.55 against 15.12 us;
// 4352: 11.04 against 11.42 us) and lost at 3 (c3 and the shared-cache
// batch: 9.09 against 8.82 us, 11.23 against 11.12 us).
inline double split_cost_unclustered(int t_max, int splits) {
  const int tiles = (t_max + splits - 1) / splits;
  return tiles * 1.2 + 7.3;
}

struct PartitionRequest {
  int t_max;           // key tiles (64 keys) of the longest query segment
  int units;           // M-tiles x K/V heads
  int D;               // head dimension (64, 128 or 256)
  int num_sms;
  int max_splits;      // splits the exchange workspace holds
  int forced_splits;   // 0 = automatic
  int forced_dparts;   // 0 = automatic, else 1, 2 or 4
  const int* cap;      // [kMaxClusterSplits + 1]: clusters of c CTAs the device holds at once
};

struct PartitionChoice {
  int splits;
  int dparts;
  bool fused;          // the splits of a unit form one cluster and merge on chip
};

// The automatic choice minimises split_cost over the partitions whose
// clusters all fit on the device at once (one wave), then compares one
// unclustered candidate: the splits that keep the grid within three quarters
// of the SMs, reduced to the fewest with the same longest split.  Forced
// values are kept (splits are clamped to [1, min(t_max, max_splits)]).
// Returns false for a column split that is not 1, 2 or 4 or does not divide D
// into 64-column blocks.
inline bool choose_partition(const PartitionRequest& r, PartitionChoice* out) {
  const int units = r.units > 0 ? r.units : 1;
  // A cluster merge exchanges its partials through the workspace, which
  // holds at most max_splits of them.
  auto fits = [&](int sp, int dp) {
    if (sp == 1) return units * dp <= r.num_sms;
    return sp <= kMaxClusterSplits && sp <= r.max_splits && units * dp <= r.cap[sp];
  };
  int splits = r.forced_splits > 0 ? r.forced_splits : 0;
  int dparts = r.forced_dparts > 0 ? r.forced_dparts : 0;
  if (splits == 0 || dparts == 0) {
    double best = 1e30;
    int bs = 1, bd = 1;
    const int s_hi = r.t_max < kMaxClusterSplits ? r.t_max : kMaxClusterSplits;
    for (int sp = 1; sp <= s_hi; ++sp) {
      if (splits > 0 && sp != splits) continue;
      for (int dp = 1; dp <= 4; dp *= 2) {
        if (dparts > 0 && dp != dparts) continue;
        if (r.D / dp < 64 || !fits(sp, dp)) continue;
        const double c = split_cost(r.t_max, sp, dp);
        if (c < best - 1e-9 || (c < best + 1e-9 && sp > bs)) {
          best = c;
          bs = sp;
          bd = dp;
        }
      }
    }
    int sp_nf = r.t_max < r.max_splits ? r.t_max : r.max_splits;
    const int sp_cap = 3 * r.num_sms / 4 / units;
    sp_nf = sp_nf < sp_cap ? sp_nf : sp_cap;
    // The fewest splits whose longest one is as short: every extra split
    // adds a CTA's Q load and a partial to merge (8448 keys: 27 splits of at
    // most 5 tiles 12.00 us, 28 12.22 us).
    if (sp_nf >= 1) {
      const int longest = (r.t_max + sp_nf - 1) / sp_nf;
      sp_nf = (r.t_max + longest - 1) / longest;
    }
    if (sp_nf > kMaxClusterSplits && (splits == 0 || splits == sp_nf) && dparts <= 1) {
      const double c = split_cost_unclustered(r.t_max, sp_nf);
      if (c < best - 1e-9) {
        best = c;
        bs = sp_nf;
        bd = 1;
      }
    }
    if (splits == 0) splits = bs;
    if (dparts == 0) dparts = bd;
  }
  splits = splits > r.t_max ? r.t_max : splits;
  splits = splits > r.max_splits ? r.max_splits : splits;
  splits = splits < 1 ? 1 : splits;
  if (dparts != 1 && dparts != 2 && dparts != 4) return false;
  if (r.D % (dparts * 64) != 0) return false;
  out->splits = splits;
  out->dparts = dparts;
  out->fused = splits >= 2 && splits <= kMaxClusterSplits && r.cap[splits] >= 1;
  return true;
}

// How a call over language streams shares the GPU between the two kernels that
// run at the same time: the shared store against all rows (units of 128 rows
// x K/V heads, each `t_max` key tiles of 64, cut into `splits`) and the tails.
// Both take one CTA an SM, so whatever SMs the first holds the second waits
// for.  A 64-key tile of the store takes about half as long as a 128-key tile
// of a tail, of which there are at most `tail_tiles`, or a little more.
//  * The store gets its share of the work in SMs, at most 5/8 of them; where
//    that share is small, enough for two or three tiles a CTA (the tails may be
//    much shorter than their capacity), at most half of the SMs; and one CTA a
//    unit at least.
//  * The tails get the other SMs, if those are at least three quarters of what
//    their own work is worth; otherwise, and where the store holds far more
//    than its share, they get all SMs, some after the store.
// Measured (SMs for the store / for the tails, us a call; the first is taken):
// 80 queries over 8448 shared keys and tails to 2000 tokens, 85/67 28.0, 75/77
// 28.7, 95/57 27.8, 60/92 30.1, 75/87 34.2; 64 x 8 queries over 2304 keys and
// tails to 16384, 64/152 114.0, 32/120 112.1, 96/152 114.7, 128/152 117.6; 32
// queries over 2112 keys and tails to 16000, 22/130 39.4, 34/118 40.6; 16
// queries over 2112 keys and tails to 30, 17/135 14.8, 33/119 16.6.  Before the
// store's weights had a second term: 72 x 4 queries of 64/8 heads (D = 128) over
// 8448 keys and tails to 512, 144/152 135.6, 144/8 333; 8 prompts of 302 tokens
// over 8448 keys, 151/152 204, 151/1 4043; and one kernel after the other, the
// first four took 38.5 (25.5 beside), 124.3 (108.4), 47.6 (40.5) and 21.0 (14.2).
struct StreamPartition {
  int splits;     // key slices of each unit of the store
  int tail_sms;   // SMs that the tails' grid is made for
};
inline StreamPartition choose_stream_partition(int units, int t_max, long long tail_tiles, int num_sms, int max_splits) {
  const long long store = static_cast<long long>(units) * t_max;
  const long long share = num_sms * store / (store + 2 * tail_tiles + 1);   // the store's SMs by work
  const bool heavy = share >= num_sms / 8;
  long long want = heavy ? share : (store + 1) / 2;
  const long long most = heavy ? num_sms * 5 / 8 : num_sms / 2;
  want = want < most ? want : most;
  long long sp = want / units;
  sp = sp < max_splits ? sp : max_splits;
  sp = sp < t_max ? sp : t_max;
  sp = sp > 1 ? sp : 1;
  if (t_max > 0) {   // the fewest splits whose longest is as short
    const long long longest = (t_max + sp - 1) / sp;
    sp = (t_max + longest - 1) / longest;
  }
  const long long held = sp * units;
  StreamPartition r;
  r.splits = static_cast<int>(sp);
  const long long rest = num_sms - held;
  const bool beside = held <= share + share / 4 || held <= num_sms / 4;
  r.tail_sms = static_cast<int>(beside && 4 * rest >= 3 * (num_sms - share) ? rest : num_sms);
  return r;
}

}  // namespace rx
