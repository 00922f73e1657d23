// Chunk attention over a paged cache on the tcgen05 tensor cores: sequences
// with many query rows per key head, bf16 queries, head sizes 64 and 128.
//
// An item is (sequence, kv head, 256 stacked query rows, range of keys), two
// tiles of 128 rows that share every key tile of 128 positions. One CTA per
// SM walks the items:
//   warps 0-3, 4-7  softmax of row tile 0, 1: a thread per row (tensor-memory
//                   lane = row)
//   warps 8-11      loaders: queries, keys, values into shared memory in the
//                   128-byte swizzle the MMA reads; bf16 rows with cp.async,
//                   8-bit rows through registers as bf16 values
//   warps 12, 13    issue the tcgen05.mma of row tile 0, 1
//   warp 14         one lane relays loaded stages (warp 15 only gives up registers)
// S_t = Q_t K^T goes to tensor memory (128 x 128 fp32); the softmax writes P
// over it as bf16 (packed two keys a column), and O_t += P_t V takes P from
// tensor memory and V as an MN-major operand as it lies in the cache. Each
// tile is a chain S(i), softmax, PV(i), S(i+1); the two chains run side by
// side, one tile's softmax under the other's products.
//
// Softmax: O is rescaled (in tensor memory, by the softmax warps) only when a
// row's maximum has grown by more than 2^8 since the reference it is scaled
// by; until then weights reach up to 2^8 (bf16 has the range, the sum is fp32)
// and the join divides by the same reference. P's rounding to bf16 is the
// precision of the matrix operand, and relative, so the reference does not change
// it; only that a row's heaviest weight is then rounded like the others, where
// relative to the maximum it would be one exactly. P's rounding and the result's
// own, 1.7e-3 in the norm each, make 2.2-2.3e-3 together. Sums take the unrounded
// weights.
//
// Values that some row of the item does not see are cleared of infinities and
// NaN by the loaders (0 * NaN would reach that row) and their keys flagged; a row
// that does see such a key, in a tile that its half may see whole, turns to NaN
// through its sum.
//
// Every mbarrier wait is bounded in device time; a CTA that gives up sets
// RLT_PAGED_TIMEOUT and leaves.
//
// Measured on a B200: 2048 rows behind 30 thousand positions, 16 heads of 128,
// bf16 610-625 us (850-870 TFLOP/s; 128 of the 148 SMs have a tile). A tile of
// 256 x 128 scores takes about 3900 clocks against 2048 of the matrix pipe: the
// chain of one row tile (softmax 1900, PV and scores 1500, hand-overs) sets the
// pace, not the exponentials or the loads (leaving either out gains 7 %).
#pragma once

#include "enc_attn.cuh"
#include "gemm_tc.cuh"
#include "paged_attn.cuh"

namespace rlt {

constexpr int PW_THREADS = 512, PW_LOADERS = 128;
// Registers of a thread of the softmax, loader and MMA warpgroups: 2 * 184 + 88
// + 56 = 4 * 128, what the block is launched with.
constexpr int PW_REGS_SOFTMAX = 184, PW_REGS_LOADER = 88, PW_REGS_MMA = 56;
constexpr int PW_TK = 128;                // keys of a tile
constexpr int PW_RT = 256;                // query rows of an item

template <int DH> struct PwCfg {
  static constexpr int STAGES = DH == 64 ? 4 : 2;  // of K and of V
  static constexpr int HALF = 128 * 128;           // 128 rows of 64 entries
  static constexpr int TILE = HALF * (DH / 64);
  static constexpr int INFO = 2 * STAGES;          // key tiles whose flags are kept
  static constexpr int Q = 0;
  static constexpr int K = 2 * TILE;
  static constexpr int V = K + STAGES * TILE;
  static constexpr int BARS = V + STAGES * TILE;
  static constexpr int NBARS = 3 + 6 * STAGES + 8;
  static constexpr int FLAGS = BARS + NBARS * 8;   // [INFO][8] words: unseen keys, strange keys
  static constexpr int SLOT = FLAGS + INFO * 8 * 4;
  static constexpr int PLAN = SLOT + 16;
  static int bytes(int n) { return PLAN + Plan::bytes(n) + 1024; }
};

// Warp-uniform bounded wait: the warp leaves together (what follows is often
// warp-collective). The clock is read only once the first polls have failed.
__device__ __forceinline__ bool pw_wait(uint64_t *bar, unsigned parity) {
#pragma unroll 1
  for (int i = 0; i < 64; i++)
    if (__all_sync(FULL_MASK, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (__all_sync(FULL_MASK, mbar_try_wait(bar, parity))) return true;
    if (__shfl_sync(FULL_MASK, globaltimer_ns() - t0 > WAIT_LIMIT_NS_TC, 0)) return false;
  }
}

__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// V: rows of 128 bytes along the keys, 8-key groups 1024 bytes apart, the
// second 64 head entries one half tile further.
__device__ __forceinline__ uint64_t pw_desc_v(uint32_t addr, int half) {
  uint64_t d = 0;
  d |= (uint64_t)(addr >> 4) & 0x3FFFull;
  d |= (uint64_t)(half >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void pw_ld32(uint32_t taddr, uint32_t r[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void pw_st32(uint32_t taddr, const uint32_t r[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void pw_st16(uint32_t taddr, const uint32_t r[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void pw_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void pw_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void pw_fence_async() {
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}
// An arrival once this thread's cp.async copies so far are complete.
__device__ __forceinline__ void arrive_behind_copies(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(smem_u32(bar))
               : "memory");
}
// `times` arrivals of a thread where `on` holds, without a branch: the warp stays
// together for the tensor-memory loads that follow.
__device__ __forceinline__ void arrive_if(bool on, uint64_t *bar, int times) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %0, 0;\n"
      " @p mbarrier.arrive.shared::cta.b64 _, [%1], %2;\n}\n" ::"r"((int)on),
      "r"(smem_u32(bar)), "r"(times)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(one));
  return one != 0;
}
template <int N> __device__ __forceinline__ void reg_shrink() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N> __device__ __forceinline__ void reg_grow() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
// Two fp32 multiply-adds, two additions.
__device__ __forceinline__ float2 ffma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t &>(d))
      : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)),
        "l"(reinterpret_cast<uint64_t &>(c)));
  return d;
}
__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t &>(d))
      : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
  return d;
}

// Byte offset of 16-byte piece c of a row's 64 entries in a half tile.
__device__ __forceinline__ int pw_piece(int row, int c) { return row * 128 + ((c ^ (row & 7)) << 4); }

// What every role needs of an item.
struct PwItem {
  SeqCut S;
  int b, row0, kvh, range, r0, R;  // R: rows of the item
  int k0, k1, nk;                  // first key, end, key tiles
};

__device__ __forceinline__ bool pw_item(const AttnArgs &A, const Plan &P, int it, PwItem &I) {
  I.b = find_seq(P.items, A.R.n, it);
  I.row0 = P.cu[I.b];
  I.S = P.cut(A, I.b);
  const int rows = I.S.m * A.group, tiles = ceil_div(rows, PW_RT);
  int j = it - P.items[I.b];
  const int rt = j % tiles;
  j /= tiles;
  I.range = j % I.S.ranges;
  I.kvh = j / I.S.ranges;
  I.r0 = rt * PW_RT;
  I.R = min(PW_RT, rows - I.r0);
  const int pos_lo = I.S.first + I.r0 / A.group, pos_hi = I.S.first + (I.r0 + I.R - 1) / A.group;
  int k0 = I.S.k_lo + I.range * I.S.keys, k1 = min(I.S.k_hi, k0 + I.S.keys);
  if (A.window > 0) k0 = max(k0, (pos_lo - A.window + 1) & ~(PA_TK - 1));
  k1 = min(k1, pos_hi + 1);
  I.k0 = k0;
  I.k1 = k1;
  I.nk = k1 > k0 ? ceil_div(k1 - k0, PW_TK) : 0;
  return !(I.S.splits > 1 && P.parts[I.b + 1] > A.part_rows);
}

// Key tiles i of the item that half t of the CTA takes: from, from + by, ..;
// none where the half is idle.
__device__ __forceinline__ bool pw_idle(const PwItem &I, int t) {
  return I.nk == 0 || (I.S.streams ? t >= I.nk : t * 128 >= I.R);
}

// Whether rows at positions lo .. hi all see keys key0 .. key0 + 127.
__device__ __forceinline__ bool pw_all_see(const AttnArgs &A, const PwItem &I, int key0, int lo,
                                           int hi) {
  return key0 + PW_TK - 1 <= lo && key0 + PW_TK <= I.k1 &&
         (A.window == 0 || key0 > hi - A.window);
}

template <bool E4, int DH>
__global__ void __launch_bounds__(PW_THREADS, 1) k_pattn_wide(const AttnArgs A) {
  using Cfg = PwCfg<DH>;
  constexpr int ST = Cfg::STAGES;
  extern __shared__ uint8_t pw_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(pw_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + Cfg::BARS);
  // *_in: counted by the loaders; *_full: passed on by the relay
  uint64_t *q_in = bars, *q_full = bars + 1, *q_empty = bars + 2, *k_in = bars + 3,
           *k_full = k_in + ST, *k_empty = k_full + ST, *v_in = k_empty + ST, *v_full = v_in + ST,
           *v_empty = v_full + ST, *s_full = v_empty + ST, *p_full = s_full + 2,
           *o_full = p_full + 4;  // p_full[t][part of the keys]
  uint32_t *flags = reinterpret_cast<uint32_t *>(sm + Cfg::FLAGS);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + Cfg::SLOT);
  const Plan P(reinterpret_cast<int *>(sm + Cfg::PLAN), A.R.n);
  __shared__ int s_fail;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    s_fail = 0;
    mbar_init(q_in, PW_LOADERS);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);  // one for each row tile
    for (int i = 0; i < ST; i++) {
      mbar_init(k_in + i, PW_LOADERS);
      mbar_init(k_full + i, 1);
      mbar_init(k_empty + i, 2);
      mbar_init(v_in + i, PW_LOADERS + 1);  // and the flags' writer
      mbar_init(v_full + i, 1);
      mbar_init(v_empty + i, 2);
    }
    for (int t = 0; t < 2; t++) {
      mbar_init(s_full + t, 1);
      mbar_init(p_full + 2 * t, 128);
      mbar_init(p_full + 2 * t + 1, 128);
      mbar_init(o_full + t, 1);
    }
    fence_mbar_init();
  }
  if (warp == 12) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  // k_pattn of the same call runs before: its predecessors' writes are complete (it
  // waited before it let this kernel start), its own are waited for at the end
  pdl_trigger();
  make_plan<PW_THREADS>(A, P, [&](const SeqCut &s) {
    return s.wide ? A.C.H * s.ranges * ceil_div(s.m * A.group, PW_RT) : 0;
  });
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int total = P.items[A.R.n];
  volatile int *fail = &s_fail;

  if (warp >= 8 && warp < 12) {
    // ------------------------------------------------------------- loaders
    reg_shrink<PW_REGS_LOADER>();
    const int tid = threadIdx.x - 256;
    uint32_t n_item = 0, n_tile = 0;  // items and key tiles so far (barrier phases)
    bool ok = true;
    for (int it = blockIdx.x; ok && it < total; it += gridDim.x) {
      PwItem I;
      if (!pw_item(A, P, it, I)) {
        if (tid == 0) flag_rows(A.R, RLT_PAGED_BAD_ROWS);
        continue;
      }
      if (I.nk == 0) continue;
      const int pos_lo = I.S.first + I.r0 / A.group,
                pos_hi = I.S.first + (I.r0 + I.R - 1) / A.group;
      // Queries, behind the item's first keys and values: those need no more than
      // their stages, the queries' place is in use until the last item is done.
      auto load_queries = [&]() {
        if (n_item > 0 && !pw_wait(q_empty, (n_item - 1) & 1)) return false;
        for (int x = tid; x < PW_RT * (DH / 8); x += PW_LOADERS) {
          const int r = x / (DH / 8), c = x % (DH / 8);
          if (I.R <= 128 && r >= 128) break;
          const int tok = (I.r0 + r) / A.group, head = I.kvh * A.group + (I.r0 + r) % A.group;
          const bf16 *src = static_cast<const bf16 *>(A.q) +
                            (r < I.R ? (int64_t)(I.row0 + tok) * A.ldq + head * DH + c * 8 : 0);
          cp_async16(smem_u32(sm + Cfg::Q + (r >> 7) * Cfg::TILE + (c >> 3) * Cfg::HALF +
                              pw_piece(r & 127, c & 7)),
                     src, r < I.R ? 16 : 0);
        }
        arrive_behind_copies(q_in);
        return true;
      };

      // pages of a key tile: lane j < 8 holds the row of the cache's key plane
      // where keys 16 j .. 16 j + 15 begin (rows of 64 bytes and more: 32 bits
      // reach over any GPU's memory), or NO_PAGE
      constexpr uint32_t NO_PAGE = 0xffffffffu;
      auto pages_of = [&](int i) {
        uint32_t cell = NO_PAGE;
        const int key = I.k0 + i * PW_TK + (lane & 7) * PA_TK;
        if (lane < 8 && key < I.k1) {
          const int idx = key / A.C.P;
          int pid = -1;
          if (idx < A.R.width) pid = A.R.table[(size_t)I.b * A.R.width + idx];
          if (pid >= 0 && pid < A.C.n_pages)
            cell = ((uint32_t)pid * A.C.H + I.kvh) * 2u * A.C.P + (key - idx * A.C.P);
          else
            flag_rows(A.R, RLT_PAGED_BAD_PAGE);
        }
        return cell;
      };
      // flags of tile i: keys that do not exist, keys whose values were cleared
      auto flag_word = [&](int i, int w) -> uint32_t * {
        return flags + ((n_tile + i) % Cfg::INFO) * 8 + w;
      };

      // by threads 0 .. 3: two groups of 16 keys a word
      auto write_flags = [&](int i, uint32_t gone) {
        const uint32_t g2 = gone >> (2 * tid);
        *flag_word(i, tid) = ((g2 & 1) ? 0xffffu : 0u) | ((g2 & 2) ? 0xffff0000u : 0u);
        *flag_word(i, 4 + tid) = 0;
      };

      if constexpr (!E4) {
        constexpr int PASSES = DH / 8;             // 128 * DH / 8 pieces by 128 threads
        constexpr int RPP = 128 / (DH / 8);        // rows of a pass: 8 or 16
        uint32_t cells = pages_of(0);
        const int c = tid % (DH / 8), row_in = tid / (DH / 8);
        const bf16 *thread_src = reinterpret_cast<const bf16 *>(A.C.pages) +
                                 (size_t)(row_in % PA_TK) * DH + c * 8;
        const uint32_t thread_dst = (c >> 3) * Cfg::HALF + pw_piece(row_in, c & 7);
        for (int i = 0; ok && i < I.nk; i++) {
          const int st = (n_tile + i) % ST, use = (n_tile + i) / ST;
          const int key0 = I.k0 + i * PW_TK;
          const uint32_t next = i + 1 < I.nk ? pages_of(i + 1) : NO_PAGE;
          const unsigned gone = __ballot_sync(FULL_MASK, lane < 8 && cells == NO_PAGE &&
                                                             key0 + lane * PA_TK < I.k1) & 0xffu;
#pragma unroll
          for (int kv = 0; kv < 2; kv++) {
            uint64_t *empty = (kv ? v_empty : k_empty) + st;
            if (use > 0 && !pw_wait(empty, (use - 1) & 1)) {
              ok = false;
              break;
            }
            const uint32_t dst =
                smem_u32(sm + (kv ? Cfg::V : Cfg::K) + st * Cfg::TILE) + thread_dst;
            const size_t plane = kv ? (size_t)A.C.P * DH : 0;
#pragma unroll
            for (int p = 0; p < PASSES; p++) {
              const uint32_t cell = __shfl_sync(FULL_MASK, cells, p * RPP / PA_TK);
              const bool on = cell != NO_PAGE && key0 + p * RPP + row_in < I.S.k_hi;
              const bf16 *src = thread_src + plane;
              if (on) src += (size_t)(cell + p * RPP % PA_TK) * DH;
              cp_async16(dst + p * RPP * 128, src, on ? 16 : 0);
            }
            if (kv == 0 || (!gone && pw_all_see(A, I, key0, pos_lo, pos_hi))) {
              // counted when the copies land
              if (kv == 1 && tid == 0) {
                for (int w = 0; w < 8; w++) *flag_word(i, w) = 0;
                tc_mbar_arrive(v_in + st);
              }
              arrive_behind_copies((kv ? v_in : k_in) + st);
              continue;
            }
            // values that some row does not see
            cp_async_commit();
            cp_async_wait<0>();
            if (tid < 4) write_flags(i, gone);
            asm volatile("bar.sync 1, 128;\n" ::: "memory");
#pragma unroll 1
            for (int p = 0; p < PASSES; p++) {
              const int row = p * RPP + row_in;
              uint4 *v = reinterpret_cast<uint4 *>(sm + Cfg::V + st * Cfg::TILE + thread_dst +
                                                   p * RPP * 128);
              const uint4 x = *v;
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
              bool bad = false;
#pragma unroll
              for (int y = 0; y < 4; y++)
                bad |= (w[y] & 0x7f80u) == 0x7f80u || (w[y] & 0x7f800000u) == 0x7f800000u;
              if (bad) {
                *v = make_uint4(0, 0, 0, 0);
                atomicOr(flag_word(i, 4 + (row >> 5)), 1u << (row & 31));
              }
            }
            tc_mbar_arrive(v_in + st);
            if (tid == 0) tc_mbar_arrive(v_in + st);
          }
          cells = next;
          if (i == 0 && ok) ok = load_queries();
        }
      } else {
        // codes through registers: the next unit's are fetched before this
        // thread waits for its stage
        constexpr int CPR = DH / 16;               // pieces of 16 codes of a row
        constexpr int RPP = 128 / CPR;             // rows of a pass: 16 or 32
        constexpr int PASSES = 128 / RPP;
        constexpr int SB = DH / 32;
        uint4 code[PASSES];
        uint32_t sbyte[PASSES];
        const int c = tid % CPR, row_in = tid / CPR;
        uint32_t cells = NO_PAGE, gone = 0;
        auto fetch = [&](int i, int kv) {
          const int key0 = I.k0 + i * PW_TK;
          if (kv == 0) {
            cells = pages_of(i);
            gone = __ballot_sync(FULL_MASK, lane < 8 && cells == NO_PAGE &&
                                                key0 + lane * PA_TK < I.k1) & 0xffu;
          }
#pragma unroll
          for (int p = 0; p < PASSES; p++) {
            const int row = p * RPP + row_in;
            const uint32_t first = __shfl_sync(FULL_MASK, cells, row / PA_TK);
            const bool on = first != NO_PAGE && key0 + row < I.S.k_hi;
            const size_t cell = (size_t)first + row % PA_TK + (kv ? A.C.P : 0);
            code[p] = make_uint4(0, 0, 0, 0);
            sbyte[p] = 127;
            if (on) {
              code[p] = *reinterpret_cast<const uint4 *>(A.C.pages + cell * DH + c * 16);
              sbyte[p] = A.C.scales[cell * SB + c / 2];
            }
          }
        };
        fetch(0, 0);
        for (int i = 0; ok && i < I.nk; i++) {
          const int st = (n_tile + i) % ST, use = (n_tile + i) / ST;
          const int key0 = I.k0 + i * PW_TK;
#pragma unroll
          for (int kv = 0; kv < 2; kv++) {
            if (use > 0 && !pw_wait((kv ? v_empty : k_empty) + st, (use - 1) & 1)) {
              ok = false;
              break;
            }
            const bool masked = kv == 1 && (gone || !pw_all_see(A, I, key0, pos_lo, pos_hi));
            if (masked) {
              if (tid < 4) write_flags(i, gone);
              asm volatile("bar.sync 1, 128;\n" ::: "memory");
            } else if (kv == 1 && tid == 0) {
              for (int w = 0; w < 8; w++) *flag_word(i, w) = 0;
            }
            uint8_t *dst = sm + (kv ? Cfg::V : Cfg::K) + st * Cfg::TILE + (c >> 2) * Cfg::HALF;
#pragma unroll
            for (int p = 0; p < PASSES; p++) {
              const int row = p * RPP + row_in;
              if (masked && sbyte[p] == 255) {
                atomicOr(flag_word(i, 4 + (row >> 5)), 1u << (row & 31));
                sbyte[p] = 127;  // its codes are zeros
              }
              const uint32_t sc = scale_pair(sbyte[p], sbyte[p]);
              const uint32_t w[4] = {code[p].x, code[p].y, code[p].z, code[p].w};
              uint32_t o[8];
#pragma unroll
              for (int y = 0; y < 4; y++) {
                // codes 0, 2 and 1, 3 of the word, then put in order
                const uint32_t even = e4m3x2_value(w[y] << 8, sc), odd = e4m3x2_value(w[y], sc);
                o[2 * y] = __byte_perm(even, odd, 0x5410);
                o[2 * y + 1] = __byte_perm(even, odd, 0x7632);
              }
              const int c8 = (c & 3) * 2;
              *reinterpret_cast<uint4 *>(dst + pw_piece(row, c8)) = make_uint4(o[0], o[1], o[2], o[3]);
              *reinterpret_cast<uint4 *>(dst + pw_piece(row, c8 + 1)) =
                  make_uint4(o[4], o[5], o[6], o[7]);
            }
            tc_mbar_arrive((kv ? v_in : k_in) + st);
            if (kv == 1 && tid == 0) tc_mbar_arrive(v_in + st);
            if (kv == 0)
              fetch(i, 1);
            else if (i + 1 < I.nk)
              fetch(i + 1, 0);
          }
          if (i == 0 && ok) ok = load_queries();
        }
      }
      n_item++;
      n_tile += I.nk;
    }
    cp_async_commit();
    cp_async_wait<0>();  // after a wait that gave up copies may be in flight
    if (!ok) *fail = 1;
  } else if (warp >= 12) {
    // ---------------------------------------------------------- MMA issuer
    reg_shrink<PW_REGS_MMA>();
    if (warp <= 13) {
      // One warp per row tile; the whole warp walks the loop, so that
      // descriptors stay uniform, and one elected lane issues.
      constexpr uint32_t idS = idesc_bf16_f32(128, PW_TK);
      constexpr uint32_t idO = idesc_bf16_f32(128, DH) | (1u << 16);  // V: MN-major
      const int t = warp - 12;
      const uint64_t q0 = smem_desc_sw128(sm + Cfg::Q), k0 = smem_desc_sw128(sm + Cfg::K);
      const uint64_t v0 = pw_desc_v(smem_u32(sm + Cfg::V), Cfg::HALF);
      const uint32_t tS = tmem + t * 128, tO = tmem + 256 + t * DH;
      uint32_t n_item = 0, n_tile = 0, n_t = 0;
      bool ok = true;
      for (int it = blockIdx.x; ok && it < total; it += gridDim.x) {
        PwItem I;
        if (!pw_item(A, P, it, I) || I.nk == 0) continue;
        // Every item's queries are waited for, by an idle half too, and its
        // arrival on q_empty comes from here: a warp that the phases overtook
        // would take an old phase for the next.
        ok = pw_wait(q_full, n_item & 1);
        if (!ok) break;
        if (pw_idle(I, t)) {
          if (lane == 0) tc_mbar_arrive(q_empty);
        } else {
          // streams: both halves have the queries of the first tile
          const uint64_t qd = q0 + (I.S.streams ? 0 : (uint64_t)(t * (Cfg::TILE >> 4)));
          const int from = I.S.streams ? t : 0, by = I.S.streams ? 2 : 1;
          auto scores = [&](int i) {
            const uint64_t kd = k0 + (uint64_t)(((n_tile + i) % ST) * (Cfg::TILE >> 4));
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < DH / 16; k++) {
                const uint64_t at = (uint64_t)((k >> 2) * (Cfg::HALF >> 4) + 2 * (k & 3));
                umma_bf16(tS, qd + at, kd + at, idS, k > 0 ? 1u : 0u);
              }
              umma_commit(s_full + t);
            }
            __syncwarp();
          };
          ok = pw_wait(k_full + (n_tile + from) % ST, (n_tile + from) / ST & 1);
          if (!ok) break;
          tc_fence_after();
          scores(from);
          for (int i = from; i < I.nk; i += by) {
            // PV of tile i in two parts as P comes, then the scores of the next
            // tile. The softmax has waited for V before it hands P on.
            const int st = (n_tile + i) % ST;
            const uint64_t vd = v0 + (uint64_t)(st * (Cfg::TILE >> 4));
            const int next = i + by;
            const bool more = next < I.nk;
            if (more) ok = pw_wait(k_full + (n_tile + next) % ST, (n_tile + next) / ST & 1);
            ok = ok && pw_wait(p_full + 2 * t, n_t & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 6; k++)
                umma_ts(tO, tS + k * 8, vd + (uint64_t)(k * (2048 >> 4)), idO,
                        (i > from || k > 0) ? 1u : 0u);
            }
            __syncwarp();
            ok = pw_wait(p_full + 2 * t + 1, n_t & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int k = 6; k < 8; k++)
                umma_ts(tO, tS + k * 8, vd + (uint64_t)(k * (2048 >> 4)), idO, 1u);
              if (by == 2) {  // for both halves
                umma_commit(v_empty + st);
                umma_commit(v_empty + st);
              }
              if (!more) umma_commit(o_full + t);
            }
            __syncwarp();
            n_t++;
            if (more) scores(next);
          }
          if (!ok) break;
        }
        n_item++;
        n_tile += I.nk;
      }
      if (!ok) *fail = 1;
    }
    if (warp == 14 && lane == 0) {
      // The relay: what the loaders wrote (through the generic proxy, some of it
      // by asynchronous copies that only the barrier knows of) is fenced for the
      // tensor core here, so that the issuing thread does not spend the fence.
      uint32_t n_item = 0, n_tile = 0;
      bool ok = true;
      auto pass_on = [&](uint64_t *in, uint64_t *full, unsigned parity) {
        if (ok && !mbar_wait_bounded(in, parity, WAIT_LIMIT_NS_TC)) ok = false;
        pw_fence_async();
        if (ok) tc_mbar_arrive(full);
      };
      for (int it = blockIdx.x; ok && it < total; it += gridDim.x) {
        PwItem I;
        if (!pw_item(A, P, it, I) || I.nk == 0) continue;
        for (int i = 0; ok && i < I.nk; i++) {
          const int st = (n_tile + i) % ST, use = (n_tile + i) / ST;
          pass_on(k_in + st, k_full + st, use & 1);
          pass_on(v_in + st, v_full + st, use & 1);
          if (i == 0) pass_on(q_in, q_full, n_item & 1);
        }
        n_item++;
        n_tile += I.nk;
      }
      if (!ok) *fail = 1;
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax
    reg_grow<PW_REGS_SOFTMAX>();
    const int t = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t tS = tmem + t * 128 + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t tO = tmem + 256 + t * DH + ((uint32_t)((warp & 3) * 32) << 16);
    const float lift = 8.f / A.scale_log2;
    uint32_t n_tile = 0, n_t = 0, n_item = 0;
    bool ok = true;
    for (int it = blockIdx.x; ok && it < total; it += gridDim.x) {
      PwItem I;
      if (!pw_item(A, P, it, I)) continue;
      // row of the item, and the half's key tiles: i = from, from + by, ..
      const int r = (I.S.streams ? 0 : t * 128) + row;
      const int from = I.S.streams ? t : 0, by = I.S.streams ? 2 : 1;
      const bool idle = pw_idle(I, t);
      const int tok = (I.r0 + r) / A.group, head = I.kvh * A.group + (I.r0 + r) % A.group;
      const int pos = r < I.R ? I.S.first + tok : -1;
      const int top = I.r0 + (I.S.streams ? 0 : t * 128);
      const int pos_lo = I.S.first + top / A.group;
      const int pos_hi = I.S.first + (min(I.r0 + I.R, top + 128) - 1) / A.group;
      if (idle && !I.S.streams && I.nk > 0) {  // no rows: the whole warpgroup skips
        n_tile += I.nk;
        continue;
      }
      float top_score = -INFINITY, l = 0.f;  // the reference, not scaled; the sum
      for (int i = from; !idle && i < I.nk; i += by) {
        const int st = (n_tile + i) % ST, use = (n_tile + i) / ST;
        const int key0 = I.k0 + i * PW_TK;
        // (in this order: V's phase is known to be this tile's once the scores are)
        if (!pw_wait(s_full + t, n_t & 1) || !pw_wait(v_full + st, use & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        n_t++;
        // Products complete in the order of their issue: with these scores K has
        // been read, and V of the tile before. One thread gives stages back, for
        // the other half too where that does not take the tile; V of a stream,
        // whose next scores are two tiles away, is given back by the issuer (a
        // commit a tile more took the other form from 579 to 694 us at 2048 rows
        // behind 30 thousand positions).
        const int times = by == 2 || I.R <= 128 ? 2 : 1;
        arrive_if(row == 0, k_empty + st, times);
        arrive_if(row == 0 && by == 1 && i > 0, v_empty + (n_tile + i - 1) % ST, times);
        const uint32_t *fl = flags + ((n_tile + i) % Cfg::INFO) * 8;
        // the loaders judge by the whole item: what they cleared counts here too
        // where this half sees the tile whole
        const bool all = pw_all_see(A, I, key0, pos_lo, pos_hi) &&
                         !(fl[0] | fl[1] | fl[2] | fl[3] | fl[4] | fl[5] | fl[6] | fl[7]);
        // the row of scores and its maximum
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 4; c++) pw_ld32(tS + 32 * c, s + 32 * c);
        pw_wait_ld();
        if (!all) {
#pragma unroll
          for (int c = 0; c < 4; c++) {
            // keys of the chunk the row sees, as bits
            const int k0 = key0 + 32 * c;
            const int hi = min(min(pos, I.k1 - 1) - k0, 31);                    // last seen
            const int lo = A.window > 0 ? max(pos - A.window + 1 - k0, 0) : 0;  // first seen
            uint32_t see = hi < 0 || lo > 31 ? 0u : (0xffffffffu >> (31 - hi)) & (0xffffffffu << lo);
            see &= ~fl[c];
            if (see & fl[4 + c]) l = NAN;
#pragma unroll
            for (int e = 0; e < 32; e++)
              if (!(see >> e & 1)) s[32 * c + e] = 0xff800000u;
          }
        }
        float mxs[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 128; e += 2)
          mxs[(e >> 1) & 3] = max3(mxs[(e >> 1) & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
        float mx = fmaxf(fmaxf(mxs[0], mxs[1]), fmaxf(mxs[2], mxs[3]));
        // O keeps its reference until the maximum has outgrown it by 2^8
        const bool grow = mx > top_score + lift || (top_score == -INFINITY && mx > top_score);
        if (i > from && __any_sync(FULL_MASK, grow)) {
          const float corr = grow ? pa_exp2((top_score - mx) * A.scale_log2) : 1.f;
#pragma unroll 1
          for (int c = 0; c < DH / 16; c++) {
            float v[16];
            tmem_ld16(tO + 16 * c, v);
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; e++) w[e] = __float_as_uint(v[e] * corr);
            pw_st16(tO + 16 * c, w);
          }
          pw_wait_st();
          l *= corr;
        }
        if (grow) top_score = mx;
        // A weight's argument is score * scale - base, one multiply-add: the product
        // is not rounded, the base was, so all weights of a row are off by the same
        // 2^d, |d| half a unit in the base's last place, which the sum undoes. From
        // 2^30 on 2^d could overflow, and neighbouring scores lie 2^-64 and more
        // apart in weight: there the difference of the scores themselves does.
        float sc = A.scale_log2, base = top_score == -INFINITY ? 0.f : top_score * A.scale_log2;
        if (fabsf(base) >= 1073741824.f) {
          sc = 1.f;
          base = top_score;
        }
        const float2 sc2 = make_float2(sc, sc), nb2 = make_float2(-base, -base);
        // weights, packed in place: pair e of keys becomes s[e]. P is handed on
        // in two parts, 96 keys and 32, so that most of PV runs under the last
        // exponentials; stores are waited for a few pairs after their issue.
        float2 sums[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        auto weigh = [&](int e) {
          float2 x = make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
          x = ffma2(x, sc2, nb2);
          x.x = pa_exp2(x.x);
          x.y = pa_exp2(x.y);
          sums[e & 1] = fadd2(sums[e & 1], x);
          s[e] = pack_bf16(x.x, x.y);
        };
        auto hand_on = [&](int part) {
          pw_wait_st();
          tc_fence_before();
          tc_mbar_arrive(p_full + 2 * t + part);
        };
#pragma unroll
        for (int e = 0; e < 32; e++) weigh(e);
        pw_st32(tS, s);
#pragma unroll
        for (int e = 32; e < 48; e++) weigh(e);
        pw_st16(tS + 32, s + 32);
#pragma unroll
        for (int e = 48; e < 52; e++) weigh(e);
        hand_on(0);
#pragma unroll
        for (int e = 52; e < 64; e++) weigh(e);
        pw_st16(tS + 48, s + 48);
        const float2 sum = fadd2(sums[0], sums[1]);
        hand_on(1);
        l += sum.x + sum.y;
      }
      if (!ok) break;
      if (!idle) {
        if (!pw_wait(o_full + t, n_item & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        arrive_if(row == 0, q_empty, 1);
        arrive_if(row == 0 && by == 1, v_empty + (n_tile + I.nk - 1) % ST, I.R <= 128 ? 2 : 1);
        n_item++;
      }
      n_tile += I.nk;
      const bool on = r < I.R;
      const float m = top_score * A.scale_log2;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      float *part = A.part + ((size_t)P.parts[I.b] + ((size_t)tok * A.heads + head) * I.S.splits +
                              (I.S.streams ? 2 * I.range + t : I.range)) * (DH + 2);
      bf16 *dst = static_cast<bf16 *>(A.out) + (int64_t)(I.row0 + tok) * A.ldo + head * DH;
#pragma unroll
      for (int c = 0; c < DH / 32; c++) {
        uint32_t s[32];
        if (!idle) {
          pw_ld32(tO + 32 * c, s);
          pw_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; e++) s[e] = 0;
        }
        if (on && I.S.splits > 1) {
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            *reinterpret_cast<float2 *>(part + 32 * c + e) =
                make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1]));
        } else if (on) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t w[4];
#pragma unroll
            for (int y = 0; y < 4; y++)
              w[y] = pack_bf16(__uint_as_float(s[e + 2 * y]) * inv,
                               __uint_as_float(s[e + 2 * y + 1]) * inv);
            *reinterpret_cast<uint4 *>(dst + 32 * c + e) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        __syncwarp();  // the warp loads O together
      }
      if (on) {
        if (I.S.splits > 1)
          *reinterpret_cast<float2 *>(part + DH) = make_float2(m, l);
        else if (A.lse)
          A.lse[(size_t)(I.row0 + tok) * A.heads + head] = (m + log2f(l)) * 0.69314718055994531f;
      }
      // O is read before the next item's first P lets it be written
      tc_fence_before();
    }
    if (!ok) *fail = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && s_fail) flag_rows(A.R, RLT_PAGED_TIMEOUT);
  if (warp == 12) tmem_dealloc(tmem, 512);
  pdl_wait();
}

}  // namespace rlt
