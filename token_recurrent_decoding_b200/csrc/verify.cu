// Verification of drafted tokens against the target's distribution
// (rlt_verify), with the caller's random numbers.
//
// A token is decided by comparisons of sums over the vocabulary, and the draw
// by where a running sum passes a point; a sum in 32 bits is off by about
// 1e-7 of the total, and with tens of thousands of steps per row that picks a
// neighbouring token every few dozen draws. So weights and sums hold 64 bits.
// The weight 2^y of a logit takes eleven fp64 operations: y = n / 64 + f / 64
// with |f| <= 1/2 (rounded by adding 1.5 * 2^52), 2^(n / 64) from a table of
// 64 entries and the exponent field, 2^(f / 64) from the exponential series to
// the fourth power, whose next term is below (ln 2 / 128)^5 / 120 = 4e-14.
//
// k_verify_rows reads every logit row once: a block takes VF_CHUNK logits of a
// row, finds their maximum and the sum of their weights relative to it. Bound
// by memory (the fp64 pipe needs about as long as the reads).
// k_verify_draw, a cluster of eight blocks per sequence: every block joins the
// rows' partial sums and makes the tests; then each weighs its eighth of the
// row to draw from and stores its sum into every block's shared memory, and the
// one in whose part the point falls walks to it. No block reads another's
// memory, so none has to stay for its peers after the last barrier.
#include <cmath>

#include "paged.cuh"

namespace rlt {
namespace {

constexpr int VF_THREADS = 256, VF_WARPS = VF_THREADS / 32;
constexpr int VF_PER = 16;                       // logits of a thread
constexpr int VF_CHUNK = VF_THREADS * VF_PER;    // logits of a block
constexpr int VF_MAX_K = 32;
constexpr int VF_CLUSTER = 8;

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
  double per64;  // 64 * log2(e) / temperature; 0: greedy
  RowPart *parts;  // [n][2 k + 1][chunks]: target rows 0 .. k, then draft rows
  int *out, *counts;
};

__device__ __forceinline__ int draft_len(const VerifyArgs &A, int b) {
  return A.lens ? min(max(A.lens[b], 0), A.k) : A.k;
}

// NaN has no weight.
__device__ __forceinline__ float logit(float x) { return x == x ? x : -INFINITY; }

__device__ __forceinline__ void fill_table(double *table) {
  if (threadIdx.x < 64) table[threadIdx.x] = exp2(threadIdx.x / 64.0);
}

// 2^(t / 64) for t <= 0.
__device__ __forceinline__ double weight64(double t, const double *table) {
  const double shift = 6755399441055744.0;  // 1.5 * 2^52
  const double r = t + shift;
  const int n = __double2loint(r);
  const double f = t - (r - shift);
  const double a = 0.010830424696249145;  // ln 2 / 64
  double p = a * a * a * a / 24;
  p = fma(p, f, a * a * a / 6);
  p = fma(p, f, a * a / 2);
  p = fma(p, f, a);
  p = fma(p, f, 1.0);
  p *= table[n & 63];
  p = __hiloint2double(__double2hiint(p) + ((n >> 6) << 20), __double2loint(p));
  return t > -65000.0 ? p : 0.0;  // 2^-1015: everything smaller counts as nothing
}

// Weight of x relative to the row's maximum m. The difference comes first: a
// product of a large logit would be rounded by more than one.
__device__ __forceinline__ double weight_of(float x, float m, double per64, const double *table) {
  if (isinf(m)) return m > 0.f && x == m ? 1.0 : 0.0;
  return weight64(((double)x - (double)m) * per64, table);
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

__global__ void __launch_bounds__(VF_THREADS) k_verify_rows(const VerifyArgs A) {
  __shared__ double table[64];
  __shared__ float s_m[VF_WARPS];
  __shared__ int s_a[VF_WARPS];
  __shared__ double s_s[VF_WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  fill_table(table);
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.z, row = blockIdx.y, len = draft_len(A, b);
  const bool draft = row > A.k;
  const int i = draft ? row - A.k - 1 : row;
  if (draft ? i >= len : i > len) return;
  const float *src = draft ? A.draft + b * A.d_seq + i * A.d_pos : A.target + b * A.t_seq + i * A.t_pos;
  const int v0 = blockIdx.x * VF_CHUNK + tid;
  float x[VF_PER];
#pragma unroll
  for (int j = 0; j < VF_PER; j++) {
    const int v = v0 + j * VF_THREADS;
    x[j] = v < A.V ? logit(src[v]) : -INFINITY;
  }
  float m = -INFINITY;
  int arg = A.V;
#pragma unroll
  for (int j = 0; j < VF_PER; j++)
    if (x[j] > m) {
      m = x[j];
      arg = v0 + j * VF_THREADS;
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    take_max(m, arg, __shfl_xor_sync(FULL_MASK, m, o), __shfl_xor_sync(FULL_MASK, arg, o));
  if (lane == 0) {
    s_m[warp] = m;
    s_a[warp] = arg;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < VF_WARPS; w++) take_max(m, arg, s_m[w], s_a[w]);
  double sum = 0.0;
  if (A.per64 > 0.0) {
#pragma unroll
    for (int j = 0; j < VF_PER; j++) sum += weight_of(x[j], m, A.per64, table);
    sum = warp_sum64(sum);
    if (lane == 0) s_s[warp] = sum;
    __syncthreads();
  }
  if (tid == 0) {
    double total = 0.0;
    if (A.per64 > 0.0)
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
    s += p[c].sum * (mc == m ? 1.0 : exp2(((double)mc - (double)m) * A.per64 / 64.0));
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

template <bool DRAFT>  // whether the draft's distribution takes part
__global__ void __cluster_dims__(VF_CLUSTER, 1, 1) __launch_bounds__(VF_THREADS)
    k_verify_draw(const VerifyArgs A) {
  __shared__ double table[64];
  __shared__ RowSum s_t[VF_MAX_K + 1], s_d[VF_MAX_K];
  __shared__ int s_first, s_len;
  __shared__ double s_w[VF_WARPS], s_all[2][VF_CLUSTER];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / VF_CLUSTER, rank = blockIdx.x % VF_CLUSTER;
  fill_table(table);
  __syncthreads();
  cluster_barrier();  // every block has begun: its shared memory may be written
  pdl_wait();
  int len = draft_len(A, b);
  if (tid == 0) s_len = len;
  __syncthreads();
  // a drafted token that is none of the vocabulary ends the draft
  if (tid < len) {
    const int x = A.tokens[b * A.k + tid];
    if (x < 0 || x >= A.V) atomicMin(&s_len, tid);
  }
  __syncthreads();
  len = s_len;
  if (tid == 0) s_first = len;
  const bool greedy = !(A.per64 > 0.0);
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
  if (tid < len) {
    const int x = A.tokens[b * A.k + tid];
    const RowSum T = s_t[tid];
    bool fine;
    if (greedy) {
      fine = x == T.arg;
    } else {
      const double wp = weight_of(logit(A.target[b * A.t_seq + tid * A.t_pos + x]), T.max,
                                  A.per64, table);
      double wq = 1.0, zq = 1.0;
      if (DRAFT) {
        const RowSum D = s_d[tid];
        wq = weight_of(logit(A.draft[b * A.d_seq + tid * A.d_pos + x]), D.max,
                       A.per64, table);
        zq = D.sum > 0.0 ? D.sum : 1.0;
      }
      fine = (double)A.uniforms[(size_t)b * (A.k + 1) + tid] * wq * T.sum < wp * zq;
    }
    if (!fine) atomicMin(&s_first, tid);
  }
  __syncthreads();
  const int j = s_first;
  const RowSum T = s_t[j];
  int *out = A.out + (size_t)b * (A.k + 1);
  if (rank == 0 && tid <= A.k) {
    if (tid < j) out[tid] = A.tokens[b * A.k + tid];
    if (tid > j) out[tid] = -1;
  }
  if (greedy || T.max == -INFINITY) {  // the whole cluster: nothing to draw
    if (rank == 0 && tid == 0) {
      const bool none = T.max == -INFINITY;
      out[j] = none ? -1 : T.arg;
      A.counts[b] = j + (none ? 0 : 1);
    }
    return;
  }

  // weights of this block's part of the row: warps side by side, 32 logits a step
  const bool refused = j < len;
  const float *tr = A.target + b * A.t_seq + j * A.t_pos;
  // A draft row is addressed whether or not it takes part: nvcc 12.9 compiled
  // `condition ? row : nullptr` here to an address that ignored the condition.
  const int dj = min(j, max(len - 1, 0));
  const float *dr = DRAFT ? A.draft + b * A.d_seq + dj * A.d_pos : nullptr;
  const int skip = !DRAFT && A.k > 0 ? A.tokens[b * A.k + min(j, A.k - 1)] : -1;
  const RowSum D = DRAFT ? s_d[dj] : RowSum{0.0, -INFINITY, 0};
  const double over = D.sum > 0.0 ? T.sum / D.sum : 0.0;  // the draft's weights on the target's scale
  const int steps = (A.V + 31) / 32;
  const int per_warp = (steps + VF_CLUSTER * VF_WARPS - 1) / (VF_CLUSTER * VF_WARPS);
  const int first = (rank * VF_WARPS + warp) * per_warp, last = min(steps, first + per_warp);
  const double point01 = (double)A.uniforms[(size_t)b * (A.k + 1) + A.k];
  bool residual = refused;
  for (int pass = 0; pass < 2; pass++) {
    auto weight = [&](int v) {
      if (v >= A.V || (!DRAFT && residual && v == skip)) return 0.0;
      double w = weight_of(logit(tr[v]), T.max, A.per64, table);
      if (DRAFT && residual)
        w = fmax(w - weight_of(logit(dr[v]), D.max, A.per64, table) * over, 0.0);
      return w;
    };
    double mine = 0.0;
#pragma unroll 4
    for (int s = first; s < last; s++) mine += weight(s * 32 + lane);
    mine = warp_sum64(mine);
    if (lane == 0) s_w[warp] = mine;
    __syncthreads();
    if (tid < VF_CLUSTER) {
      double sum = 0.0;
      for (int w = 0; w < VF_WARPS; w++) sum += s_w[w];
      store_in_block(&s_all[pass][rank], tid, sum);
    }
    __syncthreads();
    cluster_barrier();
    // the first block whose running sum passes the point; rounding aside there is one
    double total = 0.0, before = 0.0, base = 0.0;
    int owner = -1, heavy = -1;
    double all[VF_CLUSTER];
#pragma unroll
    for (int c = 0; c < VF_CLUSTER; c++) {
      all[c] = s_all[pass][c];
      total += all[c];
      if (all[c] > 0.0) heavy = c;
    }
    const double point = point01 * total;
#pragma unroll
    for (int c = 0; c < VF_CLUSTER; c++) {
      if (owner < 0 && (base + all[c] > point || c == heavy)) {
        owner = c;
        before = base;
      }
      base += all[c];
    }
    if (total > 0.0) {
      if (rank != owner) return;
      int ow = -1, hw = -1;
      double wb = before, at = before;
      for (int w = 0; w < VF_WARPS; w++)
        if (s_w[w] > 0.0) hw = w;
      for (int w = 0; w < VF_WARPS; w++) {
        if (ow < 0 && (wb + s_w[w] > point || w == hw)) {
          ow = w;
          at = wb;
        }
        wb += s_w[w];
      }
      if (warp != ow) return;
      int token = -1, weighted = -1;
      for (int s = first; s < last && token < 0; s++) {
        const double w = weight(s * 32 + lane);
        double run = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(FULL_MASK, run, o);
          if (lane >= o) run += y;
        }
        const unsigned passed = __ballot_sync(FULL_MASK, w > 0.0 && at + run > point);
        const unsigned some = __ballot_sync(FULL_MASK, w > 0.0);
        if (passed) token = s * 32 + __ffs(passed) - 1;
        if (some) weighted = s * 32 + 31 - __clz(some);
        at += __shfl_sync(FULL_MASK, run, 31);
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
  const double per64 = greedy ? 0.0 : 64.0 * 1.4426950408889634 / (double)temperature;
  if (!std::isfinite(per64 * 1e38)) return RLT_ERR_INVALID_ARG;
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
  A.per64 = per64;
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
  cudaError_t e = cudaLaunchKernelEx(&cfg, k_verify_rows, A);
  if (e == cudaSuccess) {
    cfg.gridDim = dim3(n * VF_CLUSTER);
    e = drafted ? cudaLaunchKernelEx(&cfg, k_verify_draw<true>, A)
                : cudaLaunchKernelEx(&cfg, k_verify_draw<false>, A);
  }
  return cuda_status_internal(e, __LINE__);
}

}  // extern "C"
