// Attention of a chunk of new tokens over a paged cache: what its kernels
// share (which rows and keys an item of work covers), the warp-level kernel
// and the merge of split rows.
//
// The query heads that share a key head are stacked: row r of a (sequence, kv
// head) is token r / g, head kvh * g + r % g, so a chunk of m tokens is one
// block of m * g query rows against one stream of keys.
//
// k_pattn (all types, all head sizes): an item is (sequence, kv head, tile of
// 16 * MT rows, range of keys). Four warps take tiles of 16 keys in turn; each
// keeps its own ring of stages filled with cp.async (16 keys never leave a
// page, whose positions are a multiple of 16, so a tile's page is one table
// entry), its own running maximum and sum, and accumulates O in registers; the
// four are joined in shared memory. Products are mma.sync m16n8k16 on bf16
// operands with fp32 accumulation: the work per key is a vector's (up to 32
// rows), the kernel is bound by reading the cache, and 128-row tcgen05 tiles
// would be mostly padding. fp32 operands are taken as three bf16 parts whose
// sum holds 24 bits, and the six products of parts down to 2^-16 of the
// largest are added, so nothing is lost against fp32 arithmetic.
//
// The order of head entries within a product is free as long as both operands
// share it, and so is the order of O's columns: 8-bit and fp32 rows are read
// from shared memory in the widest pieces that give a lane its operands
// (head_order, col_of), bf16 rows with ldmatrix.
//
// Splits: the keys of a sequence are cut into up to 16 ranges when its own
// (kv head, row tile) pairs are few, by a rule on that sequence alone (cut_seq in
// paged_plan.h), so a row's result does not depend on its batch. Ranges are joined
// in order by k_pattn_merge.
//
// Weights meet V as bf16 where the operands are bf16: that is the matrix operand,
// and rounds a result by no more than its own rounding does (a row's heaviest
// weight so far is one exactly: error in the norm 1.8e-3 against 1.7e-3 of the
// result's rounding alone). Sums take the unrounded weights, in fp32.
//
// Measured on a B200 (device time): one step of 32 sequences of 2000-4096 keys,
// 16 heads of 128, 8 bits 134-142 us on two boxes (3 TB/s: bound by issue, about
// 700 instructions per 16 keys and head, half of them turning codes into bf16);
// five tokens of 48 sequences of 1000-8192 keys, 32 heads on 8 key heads of
// 128, bf16 254 us (3.5 TB/s: latency at 8 warps an SM, O of 32 rows takes 128
// registers); one step of 4 short sequences 10.7 us with the merge.
#pragma once

#include <type_traits>

#include "paged.cuh"
#include "paged_plan.h"

namespace rlt {

constexpr int PA_THREADS = 128;

struct AttnArgs {
  PagedView C;
  RowsView R;
  const void *q;
  void *out;
  float *lse;
  int64_t ldq, ldo;
  int heads, group;
  int max_rows, max_len, window;
  float scale_log2;  // log2(e) / sqrt(head_dim)
  float *part;       // [part_rows][DH + 2]: O (not divided), maximum (base 2), sum
  int part_rows;
  int wide;          // whether k_pattn_wide takes part (its types and head sizes)
  int es;            // bytes of a cache element
};

// What a block keeps of the call's sequences, in shared memory: 4 (n + 1) ints.
struct Plan {
  int *items, *parts;  // items and partial rows before sequence b
  int *cu, *len;       // as given; len -1 where the sequence takes no part
  __device__ Plan(int *at, int n)
      : items(at), parts(at + n + 1), cu(at + 2 * (n + 1)), len(at + 3 * (n + 1)) {}
  static __host__ __device__ int bytes(int n) { return 4 * (n + 1) * (int)sizeof(int); }
  __device__ SeqCut cut(const AttnArgs &A, int b) const {
    const int l = len[b], m = l < 0 ? 0 : cu[b + 1] - cu[b];
    return cut_seq(m, max(l, 0), A.group, A.C.H, A.window, A.wide, A.es);
  }
};

// Fills the plan. Every thread of the block calls it.
template <int THREADS, class Items>
__device__ void make_plan(const AttnArgs &A, const Plan &P, Items count) {
  __shared__ int s_i[THREADS / 32], s_p[THREADS / 32];
  const int per = ceil_div(A.R.n, THREADS), b0 = threadIdx.x * per, b1 = min(A.R.n, b0 + per);
  int ni = 0, np = 0, fine = 1;
  for (int b = b0; b < b1; b++) {
    int lo, hi, len = A.R.len[b];
    if (!seq_rows(A.R, b, lo, hi)) {
      fine = 0;
      len = -1;
    } else if (hi - lo > A.max_rows || len < 0 || len > A.max_len) {
      flag_rows(A.R, RLT_PAGED_BAD_ROWS);
      len = -1;
    }
    P.cu[b] = lo;
    P.cu[b + 1] = hi;  // the same number the owner of sequence b + 1 writes
    P.len[b] = len;
    const SeqCut s =
        cut_seq(len < 0 ? 0 : hi - lo, max(len, 0), A.group, A.C.H, A.window, A.wide, A.es);
    P.items[b] = ni;  // within this thread's sequences, completed below
    P.parts[b] = np;
    ni += s.m > 0 ? count(s) : 0;
    np += s.splits > 1 ? s.m * A.heads * s.splits : 0;
  }
  int ii = ni, pp = np;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(FULL_MASK, ii, o), z = __shfl_up_sync(FULL_MASK, pp, o);
    if (lane >= o) {
      ii += y;
      pp += z;
    }
  }
  if (lane == 31) {
    s_i[warp] = ii;
    s_p[warp] = pp;
  }
  // rows that overlap could make more work than the call's buffers hold: none is done
  fine = __syncthreads_and(fine);
  int wi = 0, wp = 0, ti = 0, tp = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; w++) {
    if (w < warp) {
      wi += s_i[w];
      wp += s_p[w];
    }
    ti += s_i[w];
    tp += s_p[w];
  }
  const int oi = wi + ii - ni, op = wp + pp - np;
  for (int b = b0; b < b1; b++) {
    P.items[b] += oi;
    P.parts[b] += op;
  }
  if (threadIdx.x == 0) {
    P.items[A.R.n] = fine ? ti : 0;
    P.parts[A.R.n] = tp;
  }
  __syncthreads();
}

// The sequence that item `it` belongs to: the last b with items[b] <= it.
__device__ __forceinline__ int find_seq(const int *items, int n, int it) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (items[mid] <= it)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------------- k_pattn
// KIND: element type of the cache and the number of bf16 parts of the queries.
enum { PA_BF16 = 0, PA_F32 = 1, PA_E4M3 = 2, PA_E4M3_F32 = 3 };

template <int KIND, int DH, int MT> struct PaCfg {
  static constexpr bool E4 = KIND == PA_E4M3 || KIND == PA_E4M3_F32;
  static constexpr int ES = E4 ? 1 : KIND == PA_F32 ? 4 : 2;
  static constexpr int QP = KIND == PA_F32 || KIND == PA_E4M3_F32 ? 3 : 1;  // parts of q and p
  static constexpr int KP = KIND == PA_F32 ? 3 : 1;                         // parts of k and v
  static constexpr int RB = DH * ES;       // bytes of a row
  static constexpr int CPR = RB / 16;      // 16-byte pieces of a row
  static constexpr int SB = !E4 ? 0 : DH < 32 ? 1 : DH / 32;  // scale bytes of a row
  static constexpr int KV = PA_TK * RB;
  static constexpr int STAGE = 2 * KV + (E4 ? 2 * PA_TK * SB : 0);
  // CTAs of an SM the registers are cut for, and stages that fit as often
  static constexpr int CTAS = MT == 1 && QP == 1 ? 3 : 2;
  static constexpr int STAGES = KIND == PA_E4M3 || (DH == 128 && (KIND == PA_F32 || MT == 1)) ? 2 : 3;
  static constexpr int RT = 16 * MT;
  static constexpr int RING = 4 * STAGES * STAGE;
  static constexpr int JOIN = 4 * RT * DH * 4;  // O of the four warps, over the ring
  static constexpr int MAIN = RING > JOIN ? RING : JOIN;
  static constexpr int ML = 2 * 4 * RT * 4;     // maxima and sums of the four warps
  static int bytes(int n) { return MAIN + ML + Plan::bytes(n); }
};

// Place of 16-byte piece c of row r in a tile, chosen so that the lanes that
// read together meet different banks.
template <class Cfg> __device__ __forceinline__ int pa_piece(int r, int c) {
  if (Cfg::ES == 2) {  // ldmatrix: eight rows, one piece of each
    if (Cfg::CPR >= 8) return r * Cfg::CPR + (c ^ (r & 7));
    const int line = r * Cfg::CPR / 8, slot = (r * Cfg::CPR + c) & 7;
    return line * 8 + (slot ^ (line & (Cfg::CPR - 1)));
  }
  // operands of K: two rows, four pieces of each; of V: rows 2t, pieces side by side
  if (Cfg::RB == 512) return r * Cfg::CPR + (c ^ ((r >> 1 & 3) ^ ((r & 1) << 2)));
  if (Cfg::RB == 256)
    return r * Cfg::CPR + (c ^ (((r >> 1 & 1) | (r >> 2 & 1) << 2) ^ ((r & 1) << 2)));
  if (Cfg::RB == 128) return r * Cfg::CPR + (c ^ ((r >> 1 & 3) << 1 ^ ((r & 1) << 2)));
  const int line = r * Cfg::CPR / 8, slot = (r * Cfg::CPR + c) & 7;
  return line * 8 + (slot ^ ((line & 3) << 1));
}

__device__ __forceinline__ void mma16816(float c[4], const uint32_t a[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 2^x on the special-function unit; results below 2^-126 are zeros, which
// weights relative to a maximum of one may be.
__device__ __forceinline__ float pa_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// (a, b) as bf16 to nearest; what lies beyond bf16's largest becomes that.
__device__ __forceinline__ uint32_t pack_bf16_finite(float a, float b) {
  uint32_t d;
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  return d;
}

// (a, b) as P pairs of bf16 whose sum is the pair to 8 * P bits. Of several parts
// the first is kept finite: fp32 values above bf16's largest (3.39e38) would round
// to an infinity, which a weight of zero turns into NaN for rows that do not see
// the key. Infinities and NaN reach the last part as NaN.
template <int P> __device__ __forceinline__ void split_pair(float a, float b, uint32_t out[P]) {
#pragma unroll
  for (int i = 0; i < P; i++) {
    if (P > 1 && i == 0) {
      out[i] = pack_bf16_finite(a, b);
    } else {
      const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
      out[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    if (i + 1 < P) {
      a -= __uint_as_float(out[i] << 16);
      b -= __uint_as_float(out[i] & 0xffff0000u);
    }
  }
}

// c += sum of the products of parts i of a and j of b with i + j < max(QP, KP).
// Products of parts are summed from zero, smallest first, and added to c with
// one rounding: the tensor cores cut what they add to, and dozens of cuts of a
// long sum cost more than fp32's own additions (1.3e-6 of the result against
// 7e-7 over 1024 keys).
template <int QP, int KP>
__device__ __forceinline__ void mma_parts(float c[4], const uint32_t a[][4], const uint32_t *b0,
                                          const uint32_t *b1) {
  constexpr int N = QP > KP ? QP : KP;
  if constexpr (N == 1) {
    mma16816(c, a[0], b0[0], b1[0]);
  } else {
    float sum[4] = {};
#pragma unroll
    for (int s = N - 1; s >= 0; s--)
#pragma unroll
      for (int j = 0; j < KP; j++) {
        const int i = s - j;
        if (i >= 0 && i < QP) mma16816(sum, a[i], b0[j], b1[j]);
      }
#pragma unroll
    for (int e = 0; e < 4; e++) c[e] += sum[e];
  }
}

// Two codes as bf16 values: scale2 is their scales, or with TWO unset 2^120 of them.
template <bool TWO> __device__ __forceinline__ uint32_t pa_codes(uint32_t w, uint32_t scale2) {
  return TWO ? e4m3x2_value(w, scale2) : bmul2(e4m3x2_raw(w), scale2);
}

// Head entry i = 0..3 of lane t's four in product step ks (the two of the
// operand's low half, then the two of its high half).
template <int KIND, int DH> __device__ __forceinline__ int head_order(int ks, int t, int i) {
  if (KIND == PA_BF16) return 16 * ks + 2 * t + (i & 1) + (i >> 1) * 8;
  if (KIND == PA_F32) return 16 * ks + 4 * t + i;
  constexpr int GK = DH / 16 < 4 ? DH / 16 : 4;
  // pairs (0, 2) and (1, 3) of a word of e4m3 codes
  return (ks / GK) * GK * 16 + t * GK * 4 + (ks % GK) * 4 + ((i & 1) * 2 + (i >> 1));
}
// Head entry of column e = 0, 1 of lane t's pair in O's column tile j.
template <int KIND, int DH> __device__ __forceinline__ int col_of(int j, int t, int e) {
  return KIND == PA_BF16 ? 8 * j + 2 * t + e : (2 * t + e) * (DH / 8) + j;
}

template <int KIND, int DH, int MT>
__global__ void __launch_bounds__(PA_THREADS, PaCfg<KIND, DH, MT>::CTAS) k_pattn(const AttnArgs A) {
  using Cfg = PaCfg<KIND, DH, MT>;
  using TQ = typename std::conditional<Cfg::QP == 3, float, bf16>::type;
  constexpr int RB = Cfg::RB, CPR = Cfg::CPR, SB = Cfg::SB, QP = Cfg::QP, KP = Cfg::KP;
  constexpr int RT = Cfg::RT, KS = DH / 16, NT = DH / 8;
  extern __shared__ __align__(128) uint8_t pa_sm[];
  float *s_m = reinterpret_cast<float *>(pa_sm + Cfg::MAIN), *s_l = s_m + 4 * RT;
  const Plan P(reinterpret_cast<int *>(s_l + 4 * RT), A.R.n);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t *ring = pa_sm + warp * Cfg::STAGES * Cfg::STAGE;
  const uint32_t ring_u = smem_u32(ring);

  pdl_wait();
  pdl_trigger();
  make_plan<PA_THREADS>(A, P, [&](const SeqCut &s) {
    return s.wide ? 0 : A.C.H * s.splits * ceil_div(s.m * A.group, RT);
  });
  const int total = P.items[A.R.n];

  for (int it = blockIdx.x; it < total; it += gridDim.x) {
    const int b = find_seq(P.items, A.R.n, it), row0 = P.cu[b];
    const SeqCut S = P.cut(A, b);
    const int tiles = ceil_div(S.m * A.group, RT);
    int j = it - P.items[b];
    const int rt = j % tiles;
    j /= tiles;
    const int split = j % S.splits, kvh = j / S.splits;
    if (S.splits > 1 && P.parts[b + 1] > A.part_rows) {
      if (threadIdx.x == 0) flag_rows(A.R, RLT_PAGED_BAD_ROWS);
      continue;
    }
    const int r0 = rt * RT, R = min(RT, S.m * A.group - r0);
    const int pos_lo = S.first + r0 / A.group, pos_hi = S.first + (r0 + R - 1) / A.group;
    // keys of this split that a row of this tile sees
    int k0 = S.k_lo + split * S.keys, k1 = min(S.k_hi, k0 + S.keys);
    if (A.window > 0) k0 = max(k0, (pos_lo - A.window + 1) & ~(PA_TK - 1));
    k1 = min(k1, pos_hi + 1);
    const int t0 = k0 / PA_TK, t1 = k1 > k0 ? ceil_div(k1, PA_TK) : t0;
    const int my = t1 - t0 > warp ? (t1 - t0 - warp + 3) / 4 : 0;  // this warp's tiles

    float o[MT][NT][4], m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; mt++) {
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int e = 0; e < 4; e++) o[mt][n][e] = 0.f;
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
    }

    // lane i holds the row of the cache's key plane where the warp's tile i of
    // the current 32 begins (as many 16-byte rows as 36 bits reach: any GPU's
    // memory), or NO_PAGE
    constexpr int64_t NO_PAGE = -1;
    int64_t cells = NO_PAGE;
    uint32_t absent = 0;  // tiles of the last 32 whose page does not exist
    const uint8_t *lane_src = A.C.pages + lane * 16;
    const size_t plane = (size_t)A.C.P * RB;
    auto load = [&](int i) {
      if ((i & 31) == 0) {
        const int key = (t0 + warp + 4 * (i + lane)) * PA_TK;
        cells = NO_PAGE;
        if (i + lane < my) {
          const int idx = key / A.C.P;
          int pid = -1;
          if (idx < A.R.width) pid = A.R.table[(size_t)b * A.R.width + idx];
          if (pid >= 0 && pid < A.C.n_pages)
            cells = ((int64_t)pid * A.C.H + kvh) * 2 * A.C.P + (key - idx * A.C.P);
          else
            flag_rows(A.R, RLT_PAGED_BAD_PAGE);
        }
      }
      const int64_t cell = __shfl_sync(FULL_MASK, cells, i & 31);
      const bool there = cell != NO_PAGE;
      const int left = there ? S.k_hi - (t0 + warp + 4 * i) * PA_TK : 0;  // keys of the tile
      absent = (absent & ~(1u << (i & 31))) | (uint32_t)!there << (i & 31);
      const uint8_t *ksrc = lane_src + (there ? cell * RB : 0), *vsrc = ksrc + plane;
      const uint32_t dst = ring_u + (i % Cfg::STAGES) * Cfg::STAGE;
      // rows behind the sequence hold anything: read as zeros
      auto copy = [&](int x, int bytes) {
        const int c = x * 32 + lane;
        const uint32_t at = dst + pa_piece<Cfg>(c / CPR, c % CPR) * 16;
        cp_async16(at, ksrc + x * 512, bytes);
        cp_async16(at + Cfg::KV, vsrc + x * 512, bytes);
      };
      if (left >= PA_TK && RB >= 32) {
#pragma unroll
        for (int x = 0; x < (RB + 31) / 32; x++) copy(x, 16);
      } else {
#pragma unroll
        for (int x = 0; x < (RB + 31) / 32; x++)
          if (RB >= 32 || lane < RB) copy(x, (x * 32 + lane) / CPR < left ? 16 : 0);
      }
      if constexpr (Cfg::E4) {
        if (lane < 2 * SB) {
          const int kv = lane / SB, c = lane % SB;
          const uint8_t *src = A.C.scales + (there ? (cell + (kv ? A.C.P : 0)) * SB + c * 16 : 0);
          cp_async16(dst + 2 * Cfg::KV + lane * 16, src, there ? 16 : 0);
        }
      }
    };

#pragma unroll
    for (int i = 0; i < Cfg::STAGES - 1; i++) {
      if (i < my) load(i);
      cp_async_commit();
    }
    // queries, in product order; rows behind the last are zeros
    uint32_t qf[MT][KS][QP][4];
    int pos[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int hrow = 0; hrow < 2; hrow++) {
        const int r = mt * 16 + hrow * 8 + g;
        const bool on = r < R;
        const int tok = (r0 + r) / A.group, head = kvh * A.group + (r0 + r) % A.group;
        pos[mt][hrow] = on ? S.first + tok : -1;
        const TQ *src =
            static_cast<const TQ *>(A.q) + (int64_t)(row0 + tok) * A.ldq + head * DH;
#pragma unroll
        for (int ks = 0; ks < KS; ks++)
#pragma unroll
          for (int half = 0; half < 2; half++) {
            const float x = on ? to_f(src[head_order<KIND, DH>(ks, t, 2 * half)]) : 0.f;
            const float y = on ? to_f(src[head_order<KIND, DH>(ks, t, 2 * half + 1)]) : 0.f;
            uint32_t p[QP];
            split_pair<QP>(x, y, p);
#pragma unroll
            for (int i = 0; i < QP; i++) qf[mt][ks][i][2 * half + hrow] = p[i];
          }
      }
    for (int i = 0; i < my; i++) {
      cp_async_wait<Cfg::STAGES - 2>();
      __syncwarp();
      if (i + Cfg::STAGES - 1 < my) load(i + Cfg::STAGES - 1);
      cp_async_commit();
      const int key0 = (t0 + warp + 4 * i) * PA_TK;
      uint8_t *st = ring + (i % Cfg::STAGES) * Cfg::STAGE;
      const uint32_t st_u = smem_u32(st);
      uint8_t *sck = st + 2 * Cfg::KV, *scv = sck + PA_TK * SB;
      const bool gone = absent >> (i & 31) & 1;
      // whether every row of the tile sees all of these keys
      const bool all = !gone && key0 + PA_TK - 1 <= pos_lo && key0 + PA_TK <= k1 &&
                       (A.window == 0 || key0 > pos_hi - A.window);
      uint32_t strange = 0;  // keys some row may not see whose values are not finite
      if (!all) {
        if constexpr (Cfg::E4) {
          for (int x = lane; x < 2 * PA_TK * SB; x += 32) {
            const int key = x % (PA_TK * SB) / SB;
            if (key0 + key >= S.k_hi || gone) sck[x] = 127;
            if (x >= PA_TK * SB && sck[x] == 255) {
              strange |= 1u << key;
              sck[x] = 127;  // its elements are zeros
            }
          }
        } else {
          for (int c = lane; c < PA_TK * CPR; c += 32) {
            uint4 *v = reinterpret_cast<uint4 *>(st + Cfg::KV + pa_piece<Cfg>(c / CPR, c % CPR) * 16);
            const uint4 x = *v;
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            bool bad = false;
#pragma unroll
            for (int y = 0; y < 4; y++) {
              if (KIND == PA_F32)
                bad |= (w[y] & 0x7f800000u) == 0x7f800000u;
              else
                bad |= (w[y] & 0x7f80u) == 0x7f80u || (w[y] & 0x7f800000u) == 0x7f800000u;
            }
            if (bad) {
              strange |= 1u << (c / CPR);
              *v = make_uint4(0, 0, 0, 0);
            }
          }
        }
        strange = __reduce_or_sync(FULL_MASK, strange);
        __syncwarp();
      }

      // 8 bits: one multiplication by 2^(120 + e) where that is finite for
      // every scale of the tile (e <= 7, magnitudes up to 448 * 128), else two
      bool large = false;
      if constexpr (Cfg::E4) {
        constexpr int WORDS = 2 * PA_TK * SB / 4;
        uint32_t over = 0;
        for (int x = lane; x < WORDS; x += 32)
          over |= __vcmpgtu4(reinterpret_cast<const uint32_t *>(sck)[x], 0x86868686u);
        large = __any_sync(FULL_MASK, over != 0);
      }

      // S = Q K^T: two column tiles of 8 keys
      float s[MT][2][4];
#pragma unroll
      for (int mt = 0; mt < MT; mt++)
#pragma unroll
        for (int n = 0; n < 2; n++)
#pragma unroll
          for (int e = 0; e < 4; e++) s[mt][n][e] = 0.f;
      if (KIND == PA_BF16) {
        const int r = (lane & 7) + ((lane >> 4) << 3), c = (lane >> 3) & 1;
#pragma unroll
        for (int ks = 0; ks < KS; ks++) {
          uint32_t kf[4];
          ldsm4(kf, st_u + pa_piece<Cfg>(r, 2 * ks + c) * 16);
#pragma unroll
          for (int mt = 0; mt < MT; mt++) {
            mma16816(s[mt][0], qf[mt][ks][0], kf[0], kf[1]);
            mma16816(s[mt][1], qf[mt][ks][0], kf[2], kf[3]);
          }
        }
      } else if (KIND == PA_F32) {
#pragma unroll
        for (int ks = 0; ks < KS; ks++)
#pragma unroll
          for (int n = 0; n < 2; n++) {
            const float4 x = *reinterpret_cast<const float4 *>(
                st + pa_piece<Cfg>(n * 8 + g, 4 * ks + t) * 16);
            uint32_t b0[KP], b1[KP];
            split_pair<KP>(x.x, x.y, b0);
            split_pair<KP>(x.z, x.w, b1);
#pragma unroll
            for (int mt = 0; mt < MT; mt++) mma_parts<QP, KP>(s[mt][n], qf[mt][ks], b0, b1);
          }
      } else {
        auto products = [&](auto two) {
          constexpr uint32_t up = decltype(two)::value ? 0 : 120;  // added to scale bytes
          constexpr int GK = KS < 4 ? KS : 4;  // steps served by one piece of 4 * GK codes
#pragma unroll
          for (int n = 0; n < 2; n++)
#pragma unroll
            for (int kg = 0; kg < KS / GK; kg++) {
              const int row = n * 8 + g, byte = kg * GK * 16 + t * GK * 4;
              const uint8_t *src = st + pa_piece<Cfg>(row, byte / 16) * 16 + byte % 16;
              uint32_t w[4];
              if (GK == 4) {
                const uint4 x = *reinterpret_cast<const uint4 *>(src);
                w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
              } else if (GK == 2) {
                const uint2 x = *reinterpret_cast<const uint2 *>(src);
                w[0] = x.x, w[1] = x.y;
              } else {
                w[0] = *reinterpret_cast<const uint32_t *>(src);
              }
              const uint32_t sb = sck[row * SB + (SB > 1 ? byte / 32 : 0)] + up;
              const uint32_t sc = scale_pair(sb, sb);
#pragma unroll
              for (int x = 0; x < GK; x++) {
                const uint32_t b0 = pa_codes<decltype(two)::value>(w[x] << 8, sc);
                const uint32_t b1 = pa_codes<decltype(two)::value>(w[x], sc);
#pragma unroll
                for (int mt = 0; mt < MT; mt++)
                  mma_parts<QP, 1>(s[mt][n], qf[mt][kg * GK + x], &b0, &b1);
              }
            }
        };
        if (large)
          products(std::true_type{});
        else
          products(std::false_type{});
      }

      // softmax: the lane holds rows g, g + 8, keys 2t, 2t + 1 of each column tile
      uint32_t pf[MT][QP][4];
      bool grew = false;
      float corr[MT][2];
#pragma unroll
      for (int mt = 0; mt < MT; mt++) {
#pragma unroll
        for (int hrow = 0; hrow < 2; hrow++) {
          float mx = -INFINITY;
#pragma unroll
          for (int n = 0; n < 2; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
              float &x = s[mt][n][2 * hrow + e];
              x *= A.scale_log2;
              if (!all) {
                const int rel = n * 8 + 2 * t + e, key = key0 + rel, p = pos[mt][hrow];
                const bool sees = !gone && key <= p && (A.window == 0 || key > p - A.window);
                if (!sees) x = -INFINITY;
                if (sees && (strange >> rel & 1)) l[mt][hrow] = NAN;
              }
              mx = fmaxf(mx, x);
            }
          mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(FULL_MASK, mx, 2));
          const float mn = fmaxf(m[mt][hrow], mx);
          grew |= mn > m[mt][hrow];
          const float base = mn == -INFINITY ? 0.f : mn;
          corr[mt][hrow] = pa_exp2(m[mt][hrow] - base);
          m[mt][hrow] = mn;
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < 2; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
              float &x = s[mt][n][2 * hrow + e];
              x = pa_exp2(x - base);
              sum += x;
            }
          l[mt][hrow] = l[mt][hrow] * corr[mt][hrow] + sum;
#pragma unroll
          for (int n = 0; n < 2; n++) {
            uint32_t p[QP];
            split_pair<QP>(s[mt][n][2 * hrow], s[mt][n][2 * hrow + 1], p);
#pragma unroll
            for (int x = 0; x < QP; x++) pf[mt][x][2 * n + hrow] = p[x];
          }
        }
      }
      if (__any_sync(FULL_MASK, grew)) {
#pragma unroll
        for (int mt = 0; mt < MT; mt++)
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) o[mt][n][e] *= corr[mt][e >> 1];
      }

      // O += P V
      if (KIND == PA_BF16) {
        const int r = lane & 15, c = lane >> 4;
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          uint32_t vf[4];
          ldsm4t(vf, st_u + Cfg::KV + pa_piece<Cfg>(r, n + c) * 16);
#pragma unroll
          for (int mt = 0; mt < MT; mt++) {
            mma16816(o[mt][n], pf[mt][0], vf[0], vf[1]);
            mma16816(o[mt][n + 1], pf[mt][0], vf[2], vf[3]);
          }
        }
      } else if (KIND == PA_F32) {
        // the lane's NT columns lie side by side: pieces of up to four of keys 2t, 2t + 1, + 8
        constexpr int W = NT < 4 ? NT : 4;
#pragma unroll
        for (int n0 = 0; n0 < NT; n0 += W) {
          float x[4][4];  // W of each key
#pragma unroll
          for (int k = 0; k < 4; k++) {
            const int row = 2 * t + (k & 1) + (k >> 1) * 8, byte = (g * NT + n0) * 4;
            const uint8_t *src = st + Cfg::KV + pa_piece<Cfg>(row, byte / 16) * 16 + byte % 16;
            if (W == 4) {
              const float4 y = *reinterpret_cast<const float4 *>(src);
              x[k][0] = y.x, x[k][1] = y.y, x[k][2] = y.z, x[k][3] = y.w;
            } else {
              const float2 y = *reinterpret_cast<const float2 *>(src);
              x[k][0] = y.x, x[k][1] = y.y;
            }
          }
#pragma unroll
          for (int n = 0; n < W; n++) {
            uint32_t b0[KP], b1[KP];
            split_pair<KP>(x[0][n], x[1][n], b0);
            split_pair<KP>(x[2][n], x[3][n], b1);
#pragma unroll
            for (int mt = 0; mt < MT; mt++) mma_parts<QP, KP>(o[mt][n0 + n], pf[mt], b0, b1);
          }
        }
      } else {
        auto products = [&](auto two) {
          // words of up to four codes: NT codes of keys 2t, 2t + 1, 2t + 8, 2t + 9
          constexpr uint32_t up = decltype(two)::value ? 0 : 120;
          constexpr int W = NT < 4 ? NT : 4;
          uint32_t sc[2];
#pragma unroll
          for (int k = 0; k < 2; k++) {
            const int row = 2 * t + 8 * k, blk = SB > 1 ? g * NT / 32 : 0;
            sc[k] = scale_pair(scv[row * SB + blk] + up, scv[(row + 1) * SB + blk] + up);
          }
#pragma unroll
          for (int n0 = 0; n0 < NT; n0 += W) {
            uint32_t x[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
              const int row = 2 * t + (k & 1) + (k >> 1) * 8, byte = g * NT + n0;
              const uint8_t *src = st + Cfg::KV + pa_piece<Cfg>(row, byte / 16) * 16 + byte % 16;
              x[k] = W == 4 ? *reinterpret_cast<const uint32_t *>(src)
                            : (uint32_t) * reinterpret_cast<const uint16_t *>(src);
            }
#pragma unroll
            for (int n = 0; n < W; n++) {
              const uint32_t sel = n | n << 4 | (4 + n) << 8 | (4 + n) << 12;
              const uint32_t b0 = pa_codes<decltype(two)::value>(__byte_perm(x[0], x[1], sel), sc[0]);
              const uint32_t b1 = pa_codes<decltype(two)::value>(__byte_perm(x[2], x[3], sel), sc[1]);
#pragma unroll
              for (int mt = 0; mt < MT; mt++)
                mma_parts<QP, 1>(o[mt][n0 + n], pf[mt], &b0, &b1);
            }
          }
        };
        if (large)
          products(std::true_type{});
        else
          products(std::false_type{});
      }
      __syncwarp();
    }
    cp_async_wait<0>();

    // join the four warps: everything relative to the largest maximum
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int hrow = 0; hrow < 2; hrow++) {
        l[mt][hrow] += __shfl_xor_sync(FULL_MASK, l[mt][hrow], 1);
        l[mt][hrow] += __shfl_xor_sync(FULL_MASK, l[mt][hrow], 2);
        if (t == 0) {
          const int r = mt * 16 + hrow * 8 + g;
          s_m[warp * RT + r] = m[mt][hrow];
          s_l[warp * RT + r] = l[mt][hrow];
        }
      }
    __syncthreads();  // also: every warp is done with its ring
    float *s_o = reinterpret_cast<float *>(pa_sm);
#pragma unroll
    for (int mt = 0; mt < MT; mt++)
#pragma unroll
      for (int hrow = 0; hrow < 2; hrow++) {
        const int r = mt * 16 + hrow * 8 + g;
        if (r < R) {
#pragma unroll
          for (int n = 0; n < NT; n++)
#pragma unroll
            for (int e = 0; e < 2; e++)
              s_o[(warp * RT + r) * DH + col_of<KIND, DH>(n, t, e)] = o[mt][n][2 * hrow + e];
        }
      }
    __syncthreads();
    for (int x = threadIdx.x; x < R * (DH / 4); x += PA_THREADS) {
      const int r = x / (DH / 4), d = (x % (DH / 4)) * 4;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; w++) M = fmaxf(M, s_m[w * RT + r]);
      const float base = M == -INFINITY ? 0.f : M;
      float L = 0.f, v[4] = {};
#pragma unroll
      for (int w = 0; w < 4; w++) {
        const float c = pa_exp2(s_m[w * RT + r] - base);
        L += s_l[w * RT + r] * c;
        const float4 y = *reinterpret_cast<const float4 *>(s_o + (w * RT + r) * DH + d);
        v[0] += y.x * c, v[1] += y.y * c, v[2] += y.z * c, v[3] += y.w * c;
      }
      const int tok = (r0 + r) / A.group, head = kvh * A.group + (r0 + r) % A.group;
      if (S.splits > 1) {
        const size_t p = (size_t)P.parts[b] + ((size_t)tok * A.heads + head) * S.splits + split;
        float *dst = A.part + p * (DH + 2);
#pragma unroll
        for (int e = 0; e < 4; e += 2)
          *reinterpret_cast<float2 *>(dst + d + e) = make_float2(v[e], v[e + 1]);
        if (d == 0) *reinterpret_cast<float2 *>(dst + DH) = make_float2(M, L);
      } else {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        TQ *dst = static_cast<TQ *>(A.out) + (int64_t)(row0 + tok) * A.ldo + head * DH + d;
        if (QP == 3) {
          *reinterpret_cast<float4 *>(dst) =
              make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
        } else {
          uint32_t a, c;
          split_pair<1>(v[0] * inv, v[1] * inv, &a);
          split_pair<1>(v[2] * inv, v[3] * inv, &c);
          *reinterpret_cast<uint2 *>(dst) = make_uint2(a, c);
        }
        if (A.lse && d == 0)
          A.lse[(size_t)(row0 + tok) * A.heads + head] = (M + log2f(L)) * 0.69314718055994531f;
      }
    }
    __syncthreads();
  }
}

// Joins the ranges of split rows, in order: a warp per (row, head).
template <typename T, int DH>
__global__ void __launch_bounds__(256) k_pattn_merge(const AttnArgs A) {
  extern __shared__ int pm_sm[];
  const Plan P(pm_sm, A.R.n);
  // (the caller's inputs are complete: the kernel before waited for them)
  make_plan<256>(A, P, [&](const SeqCut &s) { return s.splits > 1 ? s.m : 0; });
  pdl_wait();
  const int total = P.items[A.R.n] * A.heads;
  const int lane = threadIdx.x & 31;
  for (int x = blockIdx.x * 8 + (threadIdx.x >> 5); x < total; x += gridDim.x * 8) {
    const int head = x % A.heads, it = x / A.heads, b = find_seq(P.items, A.R.n, it);
    if (P.parts[b + 1] > A.part_rows) continue;
    const int row0 = P.cu[b];
    const SeqCut S = P.cut(A, b);
    const int tok = it - P.items[b];
    const float *src =
        A.part + ((size_t)P.parts[b] + ((size_t)tok * A.heads + head) * S.splits) * (DH + 2);
    // lane i holds the maximum and sum of slice i (at most 32)
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < S.splits) ml = *reinterpret_cast<const float2 *>(src + lane * (DH + 2) + DH);
    float M = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL_MASK, M, o));
    const float c = pa_exp2(ml.x - (M == -INFINITY ? 0.f : M));
    const float L = warp_sum(ml.y * c), inv = L == 0.f ? 0.f : 1.f / L;
    constexpr int W = DH / 32 < 1 ? 1 : DH / 32;  // entries of a lane
    float v[W] = {};
    for (int s = 0; s < S.splits; s++) {
      const float cs = __shfl_sync(FULL_MASK, c, s);
      if (lane * W < DH) {
#pragma unroll
        for (int e = 0; e < W; e++) v[e] += src[s * (DH + 2) + lane * W + e] * cs;
      }
    }
    T *dst = static_cast<T *>(A.out) + (int64_t)(row0 + tok) * A.ldo + head * DH;
    if (lane * W < DH) {
#pragma unroll
      for (int e = 0; e < W; e++) dst[lane * W + e] = from_f<T>(v[e] * inv);
    }
    if (A.lse && lane == 0)
      A.lse[(size_t)(row0 + tok) * A.heads + head] = (M + log2f(L)) * 0.69314718055994531f;
  }
}

}  // namespace rlt
