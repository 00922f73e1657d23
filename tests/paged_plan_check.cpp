// Host-only check of how rlt_attend_paged cuts sequences (paged_plan.h): built
// with g++ by test_paged_plan.py, with its checks of undefined behaviour, no
// CUDA. Random batches, sequences without rows or positions among them; counts
// violated invariants:
//   * a sequence's ranges are 1 .. PA_MAX_SPLITS, begin on tiles of keys, and
//     cover every key that a row of it sees;
//   * what a sequence is cut into depends on nothing but itself (and its
//     window), so a window as long as the sequence cuts like none;
//   * the partial rows of all sequences fit into what the caller's workspace is
//     sized for, also with rows behind the last sequence and larger bounds;
//   * a sequence for the tcgen05 kernel is one the call launches it for.
// The argument takes so many rows off the workspace, so that the test can show
// that the bound bites.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "paged_plan.h"

using namespace rlt;

int main(int argc, char **argv) {
  const long long off = argc > 1 ? atoll(argv[1]) : 0;
  std::mt19937 g(1);
  auto log_int = [&](int lo, int hi) {  // over the logarithm, lo >= 0
    const double u = std::uniform_real_distribution<double>(0, 1)(g);
    double v = lo + 1, r = (double)(hi + 1) / v;
    for (int i = 0; i < 20; i++) {  // v * r^u by bits of u
      r = __builtin_sqrt(r);
      if ((long long)(u * (1 << 20)) >> (19 - i) & 1) v *= r;
    }
    return (int)v - 1;
  };
  int cases = 0, failing = 0;
  long long tightest = 1LL << 60;
  for (; cases < 20000; cases++) {
    const int n = 1 + log_int(0, cases % 10 ? 40 : 2047), group = 1 + log_int(0, 15);
    const int H = 1 + log_int(0, 1024 / group < 64 ? 1024 / group - 1 : 63), heads = H * group;
    const int most_rows = log_int(0, cases % 3 ? 64 : 4096), most_len = log_int(0, 1 << 20);
    const int es = 1 << (g() % 3), window = g() % 2 ? 1 + log_int(0, most_len) : 0;
    const bool wide = es < 4 && g() % 2;
    std::vector<int> m(n), len(n);
    int rows = 0, max_rows = 0, max_len = 0, bad = 0;
    for (int b = 0; b < n; b++) {
      m[b] = g() % 4 ? log_int(0, most_rows) : 0;
      len[b] = g() % 8 ? (g() % 2 ? most_len - log_int(0, most_len) : log_int(0, most_len)) : 0;
      rows += m[b];
      max_rows = plan_max(max_rows, m[b]);
      max_len = plan_max(max_len, len[b]);
    }
    if ((long long)rows * heads > 1 << 28) continue;
    const int pad = g() % 3 ? 0 : 17, more = g() % 3 ? 0 : 1000;
    long long parts = 0;
    for (int b = 0; b < n; b++) {
      const SeqCut s = cut_seq(m[b], len[b], group, H, window, wide, es);
      const SeqCut whole = cut_seq(m[b], len[b], group, H, 0, wide, es);
      const SeqCut same = cut_seq(m[b], len[b], group, H, plan_max(1, len[b]), wide, es);
      const int lo = window ? plan_max(0, plan_max(len[b] - m[b], 0) - window + 1) : 0;
      bad += s.ranges < 1 || s.ranges > PA_MAX_SPLITS || s.keys < PA_TK || s.keys % PA_TK ||
             s.k_lo % PA_TK || s.k_lo > lo || s.k_hi != len[b] ||
             (long long)s.k_lo + (long long)s.ranges * s.keys < s.k_hi ||
             s.splits != s.ranges * (s.streams ? 2 : 1) || s.m != m[b] || s.first != len[b] - m[b];
      bad += same.k_lo != whole.k_lo || same.keys != whole.keys || same.splits != whole.splits;
      bad += s.wide && !may_be_wide(wide, H, heads, max_rows);
      if (s.splits > 1) parts += (long long)m[b] * heads * s.splits;
    }
    const long long room =
        partial_rows(wide, H, n, heads, rows + pad, max_rows + more, max_len + more) - off;
    bad += parts > room;
    if (parts > 0 && room + off - parts < tightest) tightest = room + off - parts;
    if (bad) {
      if (failing++ < 5)
        printf("case %d: n %d heads %d/%d rows %d len %d window %d: parts %lld room %lld\n", cases,
               n, heads, H, rows, max_len, window, parts, room);
    }
  }
  printf("cases %d failing %d tightest %lld\n", cases, failing, tightest);
  return 0;
}
