// How the sequences of an rlt_attend_paged call are cut into ranges of keys, and
// how many partial rows that can make: free of CUDA calls, so that a plain C++
// check can run it.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define RLT_PLAN_FN __host__ __device__ __forceinline__
#else
#define RLT_PLAN_FN inline
#endif

namespace rlt {

RLT_PLAN_FN int ceil_div(int a, int b) { return (a + b - 1) / b; }
RLT_PLAN_FN int plan_min(int a, int b) { return a < b ? a : b; }
RLT_PLAN_FN int plan_max(int a, int b) { return a > b ? a : b; }

constexpr int PA_TK = 16;            // keys of a tile
constexpr int PA_UNIT_ROWS = 32;     // rows of a unit in the split rule
constexpr int PA_SPLIT_UNITS = 256;  // units x splits aimed at per sequence
constexpr int PA_MAX_SPLITS = 16;
constexpr int PA_SHORT_SPLITS = 4;   // splits of ..
constexpr int PA_MIN_KEYS = 256;     // .. at least so many keys, and more of ..
constexpr int PA_LONG_KEYS = 2048;   // .. at least these
constexpr int PA_ROW_BYTES = 64;     // keys x element bytes of a split for each row of a unit
// The same of sequences that go to the tcgen05 kernel: tiles of 256 rows, one
// CTA per SM, splits long enough that writing O in fp32 stays below a tenth.
// Of sequences of at most PA_STREAM_ROWS rows both halves of a CTA take the same
// rows and every other key tile (two streams, two slices of the split).
constexpr int PA_WIDE_FROM = 33;     // rows from which a sequence goes there
constexpr int PA_WIDE_ROWS = 256;
constexpr int PA_WIDE_UNITS = 148;
constexpr int PA_WIDE_KEYS = 4096;
constexpr int PA_STREAM_ROWS = 128;
constexpr int PA_STREAM_KEYS = 2048;

// How one sequence is cut, from its own rows and length only.
struct SeqCut {
  int m, first;      // rows, position of the first
  int k_lo, k_hi;    // keys any of its rows sees; k_lo is a multiple of 16
  int ranges, keys;  // key ranges and keys of one (a multiple of 16)
  int splits;        // slices its results come in: ranges, or two of each
  bool wide, streams;
};

// m may be 0 (a sequence without rows in the call): one range, of no items.
RLT_PLAN_FN SeqCut cut_seq(int m, int len, int group, int kv_heads, int window, bool wide_kernel,
                           int es) {
  SeqCut s;
  s.m = m;
  s.first = len - m;
  s.k_hi = plan_max(len, 0);
  const int lo = window > 0 ? plan_max(0, plan_max(s.first, 0) - window + 1) : 0;
  s.k_lo = plan_min(lo, s.k_hi) & ~(PA_TK - 1);
  const int span = s.k_hi - s.k_lo, rows = m * group;
  s.wide = wide_kernel && rows >= PA_WIDE_FROM;
  s.streams = s.wide && rows <= PA_STREAM_ROWS;
  int n;
  if (s.streams) {
    n = span / PA_STREAM_KEYS;
  } else if (s.wide) {
    // a unit fills an SM: rounded down, as a second wave costs more than idle SMs
    n = plan_min(PA_WIDE_UNITS / (kv_heads * ceil_div(rows, PA_WIDE_ROWS)),
                 ceil_div(span, PA_WIDE_KEYS));
  } else {
    const int units = plan_max(1, kv_heads * ceil_div(rows, PA_UNIT_ROWS));
    // Up to four ranges of 256 keys and more for the latency of few sequences;
    // beyond that a range's own start and end (about 2 us) wants 2048 keys to
    // pay: 32 steps in 8 bits of 2000-4096 positions took 169, 145, 135, 155 us
    // with ranges of at least 256, 512, 1024, 2048. Writing and joining a slice
    // stays below a tenth of reading its keys.
    n = plan_max(plan_min(PA_SHORT_SPLITS, ceil_div(span, PA_MIN_KEYS)),
                 ceil_div(span, PA_LONG_KEYS));
    const int unit_rows = plan_max(1, plan_min(rows, PA_UNIT_ROWS));
    n = plan_min(plan_min(n, ceil_div(PA_SPLIT_UNITS, units)),
                 ceil_div(span, PA_ROW_BYTES / es * unit_rows));
  }
  n = plan_max(1, plan_min(n, PA_MAX_SPLITS));
  s.keys = plan_max(PA_TK, ceil_div(ceil_div(span, n), PA_TK) * PA_TK);
  s.ranges = plan_max(1, ceil_div(span, s.keys));
  s.splits = s.streams ? 2 * s.ranges : s.ranges;
  return s;
}

// Whether a sequence of at most max_rows rows may go to k_pattn_wide.
inline bool may_be_wide(bool wide_kernel, int kv_heads, int n_heads, int max_rows) {
  return wide_kernel && (int64_t)max_rows * (n_heads / kv_heads) >= PA_WIDE_FROM;
}

inline int64_t most_splits(int max_len, int min_keys) {
  const int64_t n = ((int64_t)max_len + PA_TK + min_keys - 1) / min_keys;
  return n < PA_MAX_SPLITS ? n : PA_MAX_SPLITS;
}

// Partial rows the split rule can make, at most. k_pattn: a sequence of m rows
// makes m * heads * splits, with splits below units aimed at / own units + 1 and
// own units at least m * heads / rows of a unit. k_pattn_wide: the same for
// tiles; streams: two slices a range of at most PA_STREAM_ROWS rows a kv head.
inline int64_t partial_rows(bool wide_kernel, int kv_heads, int n, int n_heads, int rows,
                            int max_rows, int max_len) {
  const int64_t cells = (int64_t)rows * n_heads, narrow = most_splits(max_len, PA_MIN_KEYS);
  int64_t most = narrow > 1 ? (int64_t)n * PA_SPLIT_UNITS * PA_UNIT_ROWS + cells : 0;
  if (most > narrow * cells) most = narrow * cells;
  if (wide_kernel && most > 0) {
    // only few rows are left to k_pattn
    const int64_t few = (int64_t)n * PA_WIDE_FROM * kv_heads * narrow;
    if (most > few) most = few;
  }
  if (may_be_wide(wide_kernel, kv_heads, n_heads, max_rows)) {
    const int64_t wide = most_splits(max_len, PA_WIDE_KEYS),
                  streams = 2 * most_splits(max_len, PA_STREAM_KEYS);
    int64_t a = 0, b = streams * cells;
    if (wide > 1) {
      // (sequences of more than PA_STREAM_ROWS stacked rows)
      int64_t seqs = (int64_t)rows * (n_heads / kv_heads) / PA_STREAM_ROWS;
      if (seqs > n) seqs = n;
      a = seqs * PA_WIDE_UNITS * PA_WIDE_ROWS + cells;
      if (a > wide * cells) a = wide * cells;
    }
    const int64_t few = (int64_t)n * PA_STREAM_ROWS * kv_heads * streams;
    if (b > few) b = few;
    most += a + b;
  }
  return most;
}

}  // namespace rlt
