// Verification of drafted tokens against the target's distribution
// (rlt_verify), with the caller's random numbers.
//
// A token is decided by comparisons of sums over the vocabulary, and the draw
// by where a running sum passes a point; a sum in 32 bits is off by about
// 1e-7 of the total, and with tens of thousands of steps per row that picks a
// neighbouring token every few dozen draws. So what decides holds 64 bits, and
// 32 bits only where a bound on their error shows that they decide alike:
//
// k_verify_rows reads every logit row once: a block takes VF_CHUNK logits of a
// row, finds their maximum and the sum of their weights relative to it, in 32
// bits. With the argument of 2^y rounded twice (2^-23 |y|), the special-function
// unit (2^-22) and sums of 16 + 8 terms, a row's sum is off by less than
// 2^-22 + 2^-23 * (mean of |y| under the weights, at most log2 of the
// vocabulary <= 24 bits) + 24 * 2^-24 < 2^-17.6 of itself.
//
// k_verify_draw, a cluster of eight blocks per sequence: every block joins the
// rows' partial sums and makes the tests u q(x) Zp < p(x) Zq with 64-bit
// weights of the drafted words; one whose sides are closer than VF_CLOSE (twice
// both sums' bounds) is decided by exact sums. Of the row to draw from each
// block weighs its eighth in 64 bits, stores its sum into every block's shared
// memory, and the one in whose part the point falls walks to it. No block reads
// another's memory, so none has to stay for its peers after the last barrier.
//
// A draw from max(p - q, 0) needs Zp / Zq before a word's weight, and would read
// and weigh both rows twice. Instead one pass adds up, next to both sums, the
// p and q weights of the words whose difference is surely positive under the
// 32-bit sums, and keeps the few words too close to tell (VF_NEAR) aside: with
// the exact ratio r the part's weight is (sum of p) - r (sum of q) + what the
// words aside give. Where more are close than there is room for (p and q nearly
// equal) the rows are weighed again.
//
// The 64-bit weight 2^y takes ten fp64 operations: y = n / 256 + f / 256 with
// |f| <= 1/2 (rounded by adding 1.5 * 2^52), 2^(n / 256) from a table of 256
// entries and the exponent field, 2^(f / 256) from the exponential series to
// the third power, whose next term is below (ln 2 / 512)^4 / 24 = 1.4e-13.
// The maximum's product is rounded for the whole row: one factor within 2^-32.5
// (products below 2^30; larger ones take exp2) on all its weights and sums, the
// drafted word's among them, that tests and draws divide out. Weights below
// 2^-1000 are nothing.
//
// Measured on a B200 (device time): 64 sequences, up to 5 drafts, 131072 words
// 94 us (k_verify_rows 33 us, 0.92 of the copy rate; k_verify_draw 61 us: 80
// registers leave three blocks an SM, 444 places for the 512 blocks, and fp64
// operations are slow to complete); 2 sequences of 4 drafts, 32768 words 16 us.
#include <cmath>

#include "paged.cuh"

namespace rlt {
namespace {

constexpr int VF_THREADS = 256, VF_WARPS = VF_THREADS / 32;
constexpr int VF_PER = 16;                       // logits of a thread
constexpr int VF_CHUNK = VF_THREADS * VF_PER;    // logits of a block
constexpr int VF_MAX_K = 32;
constexpr int VF_CLUSTER = 8;
constexpr int VF_AHEAD = 8;                      // logits of a row a lane fetches together
constexpr double VF_CLOSE = 1.0 / 32768;         // 2^-15 > 4 * 2^-17.6
constexpr double VF_NEAR = 1.0 / 16384;          // of p's weight
constexpr int VF_ASIDE = 16;                     // words of a warp kept aside

struct RowPart {
  double sum;  // of weights relative to max
  float max;
  int arg;     // its first place
};

struct VerifyArgs {
  const float *target, *draft;
  int64_t t_seq, t_pos, d_seq, d_pos;
  const int *tokens, *lens;
  const float *uniforms;
  int n, k, V, chunks;
  double per;    // log2(e) / temperature; 0: greedy
  double reach;  // 1000 / per: what lies further below the maximum weighs nothing
  float per32;   // the same
  RowPart *parts;  // [n][2 k + 1][chunks]: target rows 0 .. k, then draft rows
  int *out, *counts;
};

__device__ __forceinline__ int draft_len(const VerifyArgs &A, int b) {
  return A.lens ? min(max(A.lens[b], 0), A.k) : A.k;
}

// NaN has no weight.
__device__ __forceinline__ float logit(float x) { return x == x ? x : -INFINITY; }

__device__ __forceinline__ void fill_table(double table[256]) {
  table[threadIdx.x] = exp2(threadIdx.x / 256.0);  // blocks of 256 threads
}

// Weight of a logit relative to the row's maximum m, whatever they are.
__device__ __noinline__ double weight_of(float x, float m, double per) {
  if (isinf(m)) return m > 0.f && x == m ? 1.0 : 0.0;
  const double y = ((double)x - (double)m) * per;
  return y > -1000.0 ? exp2(y) : 0.0;
}

// The same for many logits of one row: the product of a logit is rounded once,
// with the maximum's product, which all share, so rows whose products are too
// large for that take weight_of, and so do rows of infinities and temperatures
// under which every finite logit weighs something (from about 5e35 on).
struct RowWeights {
  float m, lo;   // what lies at or below lo weighs nothing
  double c, per256;
  bool plain;
};
__device__ __forceinline__ RowWeights row_weights(float m, double per, double reach) {
  const double per256 = 256.0 * per, c = (double)m * per256;
  const float lo = (float)((double)m - reach);
  return {m, lo, c, per256, !isinf(m) && !isinf(lo) && fabs(c) < 1073741824.0};
}
// Of plain rows; clamped to lo's (about 2^-1000) from below, NaN too.
__device__ __forceinline__ double weight_fast(float x, const RowWeights &R, const double *table) {
  const double t = fma((double)fmaxf(x, R.lo), R.per256, -R.c);
  const double shift = 6755399441055744.0;  // 1.5 * 2^52
  const double r = t + shift;
  const int n = __double2loint(r);
  const double f = t - (r - shift);
  const double a = 0.0027076061740622863;  // ln 2 / 256
  double p = fma(a * a * a / 6, f, a * a / 2);
  p = fma(p, f, a);
  p = fma(p, f, 1.0);
  p *= table[n & 255];
  return __hiloint2double(__double2hiint(p) + ((n >> 8) << 20), __double2loint(p));
}
// Whether a logit weighs anything in its row.
__device__ __forceinline__ bool weighs(float x, const RowWeights &R) {
  return R.plain ? x > R.lo : x == x && x > -INFINITY && (!isinf(R.m) || x == R.m);
}
// A single logit's weight: the one the row's exact sums take it with. (The shared
// rounding of the maximum's product, up to 2^-32.5 of every weight of the row,
// then stands on both sides of a test.)
__device__ __forceinline__ double weight_in_row(float x, const RowWeights &R, double per,
                                                const double *table) {
  if (!weighs(x, R)) return 0.0;
  return R.plain ? weight_fast(x, R, table) : weight_of(x, R.m, per);
}

__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
  return v;
}

// The larger maximum, the lower place among equals.
__device__ __forceinline__ void take_max(float &m, int &arg, float m2, int a2) {
  if (m2 > m || (m2 == m && a2 < arg)) {
    m = m2;
    arg = a2;
  }
}

__device__ __forceinline__ float exp2_sfu(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool GREEDY>
__global__ void __launch_bounds__(VF_THREADS) k_verify_rows(const VerifyArgs A) {
  __shared__ float s_m[VF_WARPS], s_s[VF_WARPS];
  __shared__ int s_a[VF_WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.z, row = blockIdx.y, len = draft_len(A, b);
  const bool draft = row > A.k;
  const int i = draft ? row - A.k - 1 : row;
  if (draft ? i >= len : i > len) return;
  const float *src = draft ? A.draft + b * A.d_seq + i * A.d_pos : A.target + b * A.t_seq + i * A.t_pos;
  const int v0 = blockIdx.x * VF_CHUNK;
  float x[VF_PER];
  // place of x[j]: four neighbours a load where the row allows it
  const bool fours = ((uintptr_t)src & 15) == 0 && v0 + VF_CHUNK <= A.V;
  auto place = [&](int j) {
    return v0 + (fours ? ((j >> 2) * VF_THREADS + tid) * 4 + (j & 3) : j * VF_THREADS + tid);
  };
  if (fours) {
#pragma unroll
    for (int j = 0; j < VF_PER / 4; j++) {
      const float4 y = *reinterpret_cast<const float4 *>(src + v0 + (j * VF_THREADS + tid) * 4);
      x[4 * j] = y.x, x[4 * j + 1] = y.y, x[4 * j + 2] = y.z, x[4 * j + 3] = y.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < VF_PER; j++) x[j] = place(j) < A.V ? src[place(j)] : -INFINITY;
  }
  float m = -INFINITY;
  int arg = A.V;
#pragma unroll
  for (int j = 0; j < VF_PER; j++) {
    x[j] = fmaxf(x[j], -INFINITY);  // NaN: no weight
    if (!GREEDY)
      m = fmaxf(m, x[j]);
    else if (x[j] > m || (x[j] == m && place(j) < arg && m > -INFINITY)) {
      m = x[j];
      arg = place(j);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(FULL_MASK, m, o);
    if (GREEDY)
      take_max(m, arg, m2, __shfl_xor_sync(FULL_MASK, arg, o));
    else
      m = fmaxf(m, m2);
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_a[warp] = arg;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < VF_WARPS; w++) {
    if (GREEDY)
      take_max(m, arg, s_m[w], s_a[w]);
    else
      m = fmaxf(m, s_m[w]);
  }
  float sum = 0.f;
  if (!GREEDY) {
    if (isinf(m)) {
#pragma unroll
      for (int j = 0; j < VF_PER; j++) sum += m > 0.f && x[j] == m ? 1.f : 0.f;
    } else if (m > 1e30f) {
      // halves: the difference itself may pass fp32's range
      const float twice = 2.f * fminf(A.per32, 1.5e38f);
#pragma unroll
      for (int j = 0; j < VF_PER; j++) sum += exp2_sfu((0.5f * x[j] - 0.5f * m) * twice);
    } else {
#pragma unroll
      for (int j = 0; j < VF_PER; j++) sum += exp2_sfu((x[j] - m) * A.per32);
    }
    sum = warp_sum(sum);
    if (lane == 0) s_s[warp] = sum;
    __syncthreads();
  }
  if (tid == 0) {
    double total = 0.0;
    if (!GREEDY)
      for (int w = 0; w < VF_WARPS; w++) total += s_s[w];
    A.parts[((size_t)b * (2 * A.k + 1) + row) * A.chunks + blockIdx.x] = {total, m, arg};
  }
}

struct RowSum {
  double sum;
  float max;
  int arg;
};

// A row's partial sums joined, by one warp.
__device__ __forceinline__ RowSum join_row(const VerifyArgs &A, int b, int row) {
  const RowPart *p = A.parts + ((size_t)b * (2 * A.k + 1) + row) * A.chunks;
  const int lane = threadIdx.x & 31;
  float m = -INFINITY;
  int arg = A.V;
  for (int c = lane; c < A.chunks; c += 32) take_max(m, arg, p[c].max, p[c].arg);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    take_max(m, arg, __shfl_xor_sync(FULL_MASK, m, o), __shfl_xor_sync(FULL_MASK, arg, o));
  double s = 0.0;
  for (int c = lane; c < A.chunks; c += 32) {
    const float mc = p[c].max;
    if (A.per > 0.0)
      s += p[c].sum * (mc == m ? 1.0 : exp2(((double)mc - (double)m) * A.per));
  }
  return {m == -INFINITY ? 0.0 : warp_sum64(s), m, arg};
}

// All threads of every block of the cluster, each warp together; orders stores
// into the blocks' shared memory before it against reads behind it.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n"
      "barrier.cluster.wait.acquire.aligned;\n" ::
          : "memory");
}
// v into the same shared-memory place of block `rank` of the cluster.
__device__ __forceinline__ void store_in_block(double *place, int rank, double v) {
  uint32_t addr;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(addr) : "r"(smem_u32(place)), "r"(rank));
  asm volatile("st.shared::cluster.f64 [%0], %1;\n" ::"r"(addr), "d"(v) : "memory");
}

enum { VF_DRAWN = 0, VF_DRAFTED = 1, VF_GREEDY = 2 };

// MODE: greedy, or whether the draft's distribution takes part.
template <int MODE>
__global__ void __cluster_dims__(VF_CLUSTER, 1, 1) __launch_bounds__(VF_THREADS, 3)
    k_verify_draw(const VerifyArgs A) {
  constexpr bool DRAFT = MODE == VF_DRAFTED;
  __shared__ double table[256];
  __shared__ RowSum s_t[VF_MAX_K + 1], s_d[VF_MAX_K];
  __shared__ int s_first, s_len;
  __shared__ double s_w[3][VF_WARPS], s_all[2][3][VF_CLUSTER];
  __shared__ float s_u[VF_MAX_K], s_lt[VF_MAX_K], s_ld[VF_MAX_K];  // of the drafted words
  __shared__ double2 s_aside[VF_WARPS][VF_ASIDE];  // p and q weights
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / VF_CLUSTER, rank = blockIdx.x % VF_CLUSTER;
  // The caller's inputs are complete: k_verify_rows waited for them before it
  // let this kernel begin. Only its sums are waited for below.
  int len = draft_len(A, b);
  if (tid == 0) s_len = len;
  __syncthreads();
  // a drafted token that is none of the vocabulary ends the draft
  if (tid < len) {
    const int x = A.tokens[b * A.k + tid];
    if (x < 0 || x >= A.V) {
      atomicMin(&s_len, tid);
    } else if (MODE != VF_GREEDY) {
      s_u[tid] = A.uniforms[(size_t)b * (A.k + 1) + tid];
      s_lt[tid] = logit(A.target[b * A.t_seq + tid * A.t_pos + x]);
      if (DRAFT) s_ld[tid] = logit(A.draft[b * A.d_seq + tid * A.d_pos + x]);
    }
  }
  fill_table(table);
  __syncthreads();
  cluster_barrier();  // every block has begun: its shared memory may be written
  len = s_len;
  pdl_wait();
  for (int i = warp; i <= len; i += VF_WARPS) {
    const RowSum s = join_row(A, b, i);
    if (lane == 0) s_t[i] = s;
  }
  if (DRAFT)
    for (int i = warp; i < len; i += VF_WARPS) {
      const RowSum s = join_row(A, b, A.k + 1 + i);
      if (lane == 0) s_d[i] = s;
    }
  __syncthreads();

  // The two sides of test i, u q(x) Zp < p(x) Zq, without Zp and Zq: every lane
  // of every block computes the same.
  auto sides = [&](int i, double &l, double &r) {
    r = weight_in_row(s_lt[i], row_weights(s_t[i].max, A.per, A.reach), A.per, table);
    l = (double)s_u[i];
    if (DRAFT)
      l *= weight_in_row(s_ld[i], row_weights(s_d[i].max, A.per, A.reach), A.per, table);
  };
  // Lowest index from `from` on that is not surely accepted (len: none); `close`
  // where the 32-bit sums do not decide it.
  bool close = false;
  auto first_open = [&](int from) {
    if (tid == 0) s_first = 2 * len;
    __syncthreads();
    if (tid >= from && tid < len) {
      if (MODE == VF_GREEDY) {
        if (A.tokens[b * A.k + tid] != s_t[tid].arg) atomicMin(&s_first, 2 * tid);
      } else {
        double l, r;
        sides(tid, l, r);
        l *= s_t[tid].sum;
        if (DRAFT) r *= s_d[tid].sum > 0.0 ? s_d[tid].sum : 1.0;
        const bool near = fabs(l - r) <= VF_CLOSE * fmax(l, r) && fmax(l, r) > 0.0;
        if (near)
          atomicMin(&s_first, 2 * tid + 1);
        else if (!(l < r))
          atomicMin(&s_first, 2 * tid);
      }
    }
    __syncthreads();
    const int f = s_first;
    __syncthreads();
    close = f & 1;
    return f >> 1;
  };

  // this block's part of a row: warps side by side, 32 logits a step
  const int steps = (A.V + 31) / 32;
  const int per_warp = (steps + VF_CLUSTER * VF_WARPS - 1) / (VF_CLUSTER * VF_WARPS);
  const int first = (rank * VF_WARPS + warp) * per_warp, last = min(steps, first + per_warp);
  int exchange = 0;
  double all[3][VF_CLUSTER];
  // The blocks' sums of three values, from each lane's, to every block.
  auto share = [&](double v0, double v1, double v2) {
    const double v[3] = {warp_sum64(v0), warp_sum64(v1), warp_sum64(v2)};
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < 3; i++) s_w[i][warp] = v[i];
    }
    __syncthreads();
    const int e = exchange++ & 1;
    if (tid < 3 * VF_CLUSTER) {
      const int which = tid / VF_CLUSTER;
      double sum = 0.0;
      for (int w = 0; w < VF_WARPS; w++) sum += s_w[which][w];
      store_in_block(&s_all[e][which][rank], tid % VF_CLUSTER, sum);
    }
    __syncthreads();
    cluster_barrier();
#pragma unroll
    for (int i = 0; i < 3; i++)
#pragma unroll
      for (int c = 0; c < VF_CLUSTER; c++) all[i][c] = s_all[e][i][c];
  };
  auto total_of = [&](int i) {
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < VF_CLUSTER; c++) s += all[i][c];
    return s;
  };
  // VF_AHEAD steps of a row from s0 on
  auto fetch = [&](const float *row, int s0, float x[VF_AHEAD]) {
    if (s0 + VF_AHEAD <= last && (s0 + VF_AHEAD) * 32 <= A.V) {
#pragma unroll
      for (int e = 0; e < VF_AHEAD; e++) x[e] = row[(s0 + e) * 32 + lane];
    } else {
#pragma unroll
      for (int e = 0; e < VF_AHEAD; e++) {
        const int v = (s0 + e) * 32 + lane;
        x[e] = s0 + e < last && v < A.V ? row[v] : -INFINITY;
      }
    }
  };

  auto weights_of = [&](const float x[VF_AHEAD], const RowWeights &R, double w[VF_AHEAD]) {
    if (R.plain) {
#pragma unroll
      for (int e = 0; e < VF_AHEAD; e++) w[e] = weight_fast(x[e], R, table);
    } else {
#pragma unroll
      for (int e = 0; e < VF_AHEAD; e++) w[e] = weight_of(logit(x[e]), R.m, A.per);
    }
  };

  // tests; every block of the cluster takes the same turns
  int j = first_open(0);
  double zp = 0.0, zq = 0.0, surely = 0.0;  // surely: this lane's part of p - q, see above
  bool split = false;                       // whether it holds
  if (MODE != VF_GREEDY) {
    while (j < len && (DRAFT || close)) {
      // exact sums of row j: they decide a close test, and a draw from the
      // difference needs them
      const RowSum T = s_t[j], D = DRAFT ? s_d[j] : RowSum{0.0, -INFINITY, 0};
      const RowWeights P = row_weights(T.max, A.per, A.reach), Q = row_weights(D.max, A.per, A.reach);
      const float *tr = A.target + b * A.t_seq + j * A.t_pos;
      const float *dr = DRAFT ? A.draft + b * A.d_seq + j * A.d_pos : nullptr;
      const double ratio = DRAFT && D.sum > 0.0 ? T.sum / D.sum : 0.0;
      double a = 0.0, d = 0.0, sure_p = 0.0, sure_q = 0.0;
      int aside = 0;
      for (int s0 = first; s0 < last; s0 += VF_AHEAD) {
        float x[VF_AHEAD], y[VF_AHEAD];
        fetch(tr, s0, x);
        if (DRAFT) fetch(dr, s0, y);
        // all weights first: fp64 operations take long and overlap
        double wp[VF_AHEAD], wq[VF_AHEAD];
        weights_of(x, P, wp);
        if (DRAFT) weights_of(y, Q, wq);
        unsigned near = 0;
#pragma unroll
        for (int e = 0; e < VF_AHEAD; e++) {
          a += wp[e];
          if (DRAFT) {
            d += wq[e];
            const double gap = fma(-ratio, wq[e], wp[e]);
            if (weighs(x[e], P)) {
              if (fabs(gap) <= VF_NEAR * wp[e]) {
                near |= 1u << e;
              } else if (gap > 0.0) {
                sure_p += wp[e];
                sure_q += wq[e];
              }
            }
          }
        }
        if (DRAFT && __any_sync(FULL_MASK, near != 0)) {
#pragma unroll
          for (int e = 0; e < VF_AHEAD; e++) {
            const unsigned nears = __ballot_sync(FULL_MASK, near >> e & 1);
            const int at = aside + __popc(nears & ((1u << lane) - 1));
            if ((near >> e & 1) && at < VF_ASIDE) s_aside[warp][at] = make_double2(wp[e], wq[e]);
            aside += __popc(nears);
          }
        }
      }
      share(a, d, lane == 0 && aside > VF_ASIDE ? 1.0 : 0.0);
      zp = total_of(0);
      zq = total_of(1);
      split = DRAFT && total_of(2) == 0.0;
      if (close) {
        double l, r;
        sides(j, l, r);
        if (l * zp < r * (DRAFT && zq > 0.0 ? zq : 1.0)) {
          j = first_open(j + 1);
          continue;
        }
      }
      const double over = zq > 0.0 ? zp / zq : 0.0;
      surely = sure_p - over * sure_q;
      if (lane < aside && lane < VF_ASIDE) {
        const double2 w = s_aside[warp][lane];
        surely += fmax(w.x - w.y * over, 0.0);
      }
      break;
    }
  }

  const RowSum T = s_t[j];
  int *out = A.out + (size_t)b * (A.k + 1);
  if (rank == 0 && tid <= A.k) {
    if (tid < j) out[tid] = A.tokens[b * A.k + tid];
    if (tid > j) out[tid] = -1;
  }
  if (MODE == VF_GREEDY || T.max == -INFINITY) {  // the whole cluster: nothing to draw
    if (rank == 0 && tid == 0) {
      const bool none = T.max == -INFINITY;
      out[j] = none ? -1 : T.arg;
      A.counts[b] = j + (none ? 0 : 1);
    }
    return;
  }

  // A draft row is addressed whether or not it takes part: nvcc 12.9 compiled
  // `condition ? row : nullptr` here to an address that ignored the condition.
  const int dj = min(j, max(len - 1, 0));
  const float *tr = A.target + b * A.t_seq + j * A.t_pos;
  const float *dr = DRAFT ? A.draft + b * A.d_seq + dj * A.d_pos : nullptr;
  const int skip = !DRAFT && A.k > 0 ? A.tokens[b * A.k + min(j, A.k - 1)] : -1;
  const RowWeights P = row_weights(T.max, A.per, A.reach);
  const RowWeights Q = row_weights(DRAFT ? s_d[dj].max : -INFINITY, A.per, A.reach);
  const double over = DRAFT && zq > 0.0 ? zp / zq : 0.0;  // the draft's weights on the target's scale
  const double point01 = (double)A.uniforms[(size_t)b * (A.k + 1) + A.k];
  bool residual = j < len;
  for (int pass = 0; pass < 2; pass++) {
    // weights of VF_AHEAD steps from s0 on
    auto weights = [&](int s0, double w[VF_AHEAD]) {
      float x[VF_AHEAD], y[VF_AHEAD];
      fetch(tr, s0, x);
      if (DRAFT && residual) fetch(dr, s0, y);
      double q[VF_AHEAD];
      weights_of(x, P, w);
      if (DRAFT && residual) weights_of(y, Q, q);
#pragma unroll
      for (int e = 0; e < VF_AHEAD; e++) {
        if (!weighs(x[e], P) || (!DRAFT && residual && (s0 + e) * 32 + lane == skip)) w[e] = 0.0;
        if (DRAFT && residual) w[e] = fmax(w[e] - q[e] * over, 0.0);
      }
    };
    double mine = 0.0;
    if (residual && split) {
      mine = surely;
    } else {
      for (int s0 = first; s0 < last; s0 += VF_AHEAD) {
        double w[VF_AHEAD];
        weights(s0, w);
#pragma unroll
        for (int e = 0; e < VF_AHEAD; e++) mine += w[e];
      }
    }
    share(mine, 0.0, 0.0);
    // the first block whose running sum passes the point; rounding aside there is one
    const double total = total_of(0);
    double before = 0.0, base = 0.0;
    int owner = -1, heavy = -1;
#pragma unroll
    for (int c = 0; c < VF_CLUSTER; c++)
      if (all[0][c] > 0.0) heavy = c;
    const double point = point01 * total;
#pragma unroll
    for (int c = 0; c < VF_CLUSTER; c++) {
      if (owner < 0 && (base + all[0][c] > point || c == heavy)) {
        owner = c;
        before = base;
      }
      base += all[0][c];
    }
    if (total > 1e-280) {
      if (rank != owner) return;
      int ow = -1, hw = -1;
      double wb = before, at = before;
      for (int w = 0; w < VF_WARPS; w++)
        if (s_w[0][w] > 0.0) hw = w;
      for (int w = 0; w < VF_WARPS; w++) {
        if (ow < 0 && (wb + s_w[0][w] > point || w == hw)) {
          ow = w;
          at = wb;
        }
        wb += s_w[0][w];
      }
      if (warp != ow) return;
      // batch by batch to the one the point falls in, then step by step
      int token = -1, weighted = -1;
      for (int s0 = first; s0 < last && token < 0; s0 += VF_AHEAD) {
        double w[VF_AHEAD], sum = 0.0;
        weights(s0, w);
        bool some = false;
#pragma unroll
        for (int e = 0; e < VF_AHEAD; e++) {
          sum += w[e];
          some |= w[e] > 0.0;
        }
        sum = warp_sum64(sum);
        if (!__any_sync(FULL_MASK, some)) continue;
        double step[VF_AHEAD];
#pragma unroll
        for (int e = 0; e < VF_AHEAD; e++) {
          const unsigned some_e = __ballot_sync(FULL_MASK, w[e] > 0.0);
          if (some_e) weighted = (s0 + e) * 32 + 31 - __clz(some_e);
        }
        if (!(at + sum > point)) {
          at += sum;
          continue;
        }
#pragma unroll
        for (int e = 0; e < VF_AHEAD; e++) step[e] = warp_sum64(w[e]);
        // the step, then the word
        int es = -1;
        double mine_w = 0.0;
#pragma unroll
        for (int e = 0; e < VF_AHEAD; e++) {
          if (es < 0 && at + step[e] > point) {
            es = e;
            mine_w = w[e];
          }
          if (es < 0) at += step[e];
        }
        if (es < 0) continue;  // by rounding only: the last word that weighs
        double run = mine_w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(FULL_MASK, run, o);
          if (lane >= o) run += y;
        }
        const unsigned passed = __ballot_sync(FULL_MASK, mine_w > 0.0 && at + run > point);
        const unsigned some_s = __ballot_sync(FULL_MASK, mine_w > 0.0);
        token = (s0 + es) * 32 + (passed ? __ffs(passed) - 1 : 31 - __clz(some_s));
      }
      if (lane == 0) {
        out[j] = token >= 0 ? token : weighted;
        A.counts[b] = j + 1;
      }
      return;
    }
    __syncthreads();  // s_w is read before the second pass writes it
    residual = false;  // nothing left of the difference: the target's own weights
  }
}

bool verify_shape_ok(int n, int k, int vocab) {
  return n >= 1 && n <= 65535 && k >= 0 && k <= VF_MAX_K && vocab >= 1 && vocab <= (1 << 24);
}
int verify_chunks(int vocab) { return (vocab + VF_CHUNK - 1) / VF_CHUNK; }

}  // namespace
}  // namespace rlt

using namespace rlt;

extern "C" {

RLT_API size_t rlt_verify_workspace_bytes(int n, int k, int vocab) {
  if (!verify_shape_ok(n, k, vocab)) return 0;
  const size_t b = (size_t)n * (2 * k + 1) * verify_chunks(vocab) * sizeof(RowPart);
  return (b + 255) / 256 * 256;
}

RLT_API int rlt_verify(const float *target, int64_t target_seq, int64_t target_pos,
                       const float *draft, int64_t draft_seq, int64_t draft_pos,
                       const int32_t *draft_tokens, const int32_t *lens, int n, int k, int vocab,
                       float temperature, const float *uniforms, int32_t *tokens, int32_t *counts,
                       void *workspace, size_t workspace_bytes, rlt_stream stream) {
  const bool greedy = temperature == 0.0f;
  if (!verify_shape_ok(n, k, vocab) || !(temperature >= 0.0f) || !std::isfinite(temperature) ||
      !target || (k > 0 && !draft_tokens) || (!greedy && !uniforms) || !tokens || !counts ||
      !workspace || ((uintptr_t)workspace & 255) || target_seq < 0 || target_pos < 0 ||
      draft_seq < 0 || draft_pos < 0)
    return RLT_ERR_INVALID_ARG;
  if (workspace_bytes < rlt_verify_workspace_bytes(n, k, vocab)) return RLT_ERR_CAPACITY;
  const double per = greedy ? 0.0 : 1.4426950408889634 / (double)temperature;
  VerifyArgs A;
  A.target = target;
  A.draft = k > 0 ? draft : nullptr;
  A.t_seq = target_seq;
  A.t_pos = target_pos;
  A.d_seq = draft_seq;
  A.d_pos = draft_pos;
  A.tokens = draft_tokens;
  A.lens = lens;
  A.uniforms = uniforms;
  A.n = n;
  A.k = k;
  A.V = vocab;
  A.chunks = verify_chunks(vocab);
  A.per = per;
  A.reach = greedy ? 0.0 : 1000.0 / per;
  A.per32 = (float)(per < 3e38 ? per : 3e38);  // finite: zero differences stay zero
  A.parts = static_cast<RowPart *>(workspace);
  A.out = tokens;
  A.counts = counts;
  cudaStream_t st = (cudaStream_t)stream;
  const bool drafted = A.draft && !greedy;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(A.chunks, drafted ? 2 * k + 1 : k + 1, n);
  cfg.blockDim = dim3(VF_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = st == nullptr ? 0 : 1;
  cudaError_t e = greedy ? cudaLaunchKernelEx(&cfg, k_verify_rows<true>, A)
                         : cudaLaunchKernelEx(&cfg, k_verify_rows<false>, A);
  if (e == cudaSuccess) {
    cfg.gridDim = dim3(n * VF_CLUSTER);
    e = greedy    ? cudaLaunchKernelEx(&cfg, k_verify_draw<VF_GREEDY>, A)
        : drafted ? cudaLaunchKernelEx(&cfg, k_verify_draw<VF_DRAFTED>, A)
                  : cudaLaunchKernelEx(&cfg, k_verify_draw<VF_DRAWN>, A);
  }
  return cuda_status_internal(e, __LINE__);
}

}  // extern "C"
