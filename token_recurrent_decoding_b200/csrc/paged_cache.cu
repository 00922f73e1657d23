// Rows of keys and values into a paged cache (rlt_paged_append) and out of it
// (rlt_paged_read), as they are or in 8 bits.
//
// One thread moves a piece of 8 or 16 elements of a row's head, four pieces in
// flight; in 8 bits the lanes of a block find its largest magnitude a together.
// The least e with a <= 448 * 2^e comes from a's own bits: for a = f * 2^x,
// 1 <= f < 2, it is x - 8, plus one where f > 1.75 (448 = 1.75 * 2^8). x * 2^-e
// is exact, so the conversion to e4m3 is the only rounding.
// Bound by memory; a block takes a few neighbouring rows and finds their
// sequences once. Measured on a B200 (device time): 16 thousand rows of 16 heads
// of 128 bf16 written in 8 bits and read back 93 us (4.3 TB/s), 73 thousand rows
// of 8 heads read 84 us (5.4 TB/s).
#include <cuda_fp8.h>

#include "paged.cuh"

namespace rlt {
namespace {

constexpr int PC_THREADS = 256;
constexpr int PC_MAX_ROWS = 16;  // rows of a block

struct RowPlace {
  int page, slot;  // page < 0: the row does not exist; -2: not a row of the call
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t *>(&v);
}

// N dense elements <-> fp32 (N a multiple of 8).
template <int N> __device__ __forceinline__ void load_row(const float *p, float f[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 a = *reinterpret_cast<const float4 *>(p + i);
    f[i] = a.x; f[i + 1] = a.y; f[i + 2] = a.z; f[i + 3] = a.w;
  }
}
template <int N> __device__ __forceinline__ void load_row(const bf16 *p, float f[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8) ld16_coherent(p + i, f + i);
}
template <int N> __device__ __forceinline__ void store_row(float *p, const float f[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4)
    *reinterpret_cast<float4 *>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
}
template <int N> __device__ __forceinline__ void store_row(bf16 *p, const float f[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8)
    *reinterpret_cast<uint4 *>(p + i) =
        make_uint4(pack2(f[i], f[i + 1]), pack2(f[i + 2], f[i + 3]), pack2(f[i + 4], f[i + 5]),
                   pack2(f[i + 6], f[i + 7]));
}

// N elements as e4m3 under a scale shared by LANES neighbouring lanes; returns
// the scale byte. The lanes of a block are all active. Under the largest scale,
// 2^120, elements from 248 * 2^120 on would round to 2^128, an infinity in fp32
// and bf16: they become 240 * 2^120, the largest below.
template <int N, int LANES>
__device__ __forceinline__ int quantise(const float f[N], uint32_t w[N / 4]) {
  // magnitudes as bits: ordered like the values, infinities and NaN above all
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < N; i++) a = max(a, __float_as_uint(f[i]) & 0x7fffffffu);
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(FULL_MASK, a, o));
  if (a >= 0x7f800000u) {
#pragma unroll
    for (int i = 0; i < N / 4; i++) w[i] = 0;
    return 255;
  }
  // subnormals (exponent field 0) lie far below the least scale
  int e = (int)(a >> 23) - 127 - 8 + ((a & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, E4M3_EMIN);
  const float inv = pow2f(-e);
#pragma unroll
  for (int i = 0; i < N / 4; i++) {
    const float2 x = make_float2(f[4 * i] * inv, f[4 * i + 1] * inv);
    const float2 y = make_float2(f[4 * i + 2] * inv, f[4 * i + 3] * inv);
    w[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3) |
           ((uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3) << 16);
  }
  if (e == E4M3_EMAX) {  // codes 0x78 (256) become 0x77 (240)
#pragma unroll
    for (int i = 0; i < N / 4; i++)
      w[i] = __vminu4(w[i] & 0x7f7f7f7fu, 0x77777777u) | (w[i] & 0x80808080u);
  }
  return e + 127;
}

template <int N>
__device__ __forceinline__ void dequantise(const uint32_t w[N / 4], int sb, float f[N]) {
  const float s = __uint_as_float((uint32_t)sb << 23);  // byte 255: infinity, times zero NaN
  const float p = __uint_as_float(0x7b800000u);         // 2^120
#pragma unroll
  for (int i = 0; i < N / 4; i++) {
    // elements 1, 3 of the word, then 0, 2; raw bf16 bits widened to fp32
    const uint32_t odd = e4m3x2_raw(w[i]), even = e4m3x2_raw(w[i] << 8);
    f[4 * i] = __uint_as_float(even << 16) * p * s;
    f[4 * i + 1] = __uint_as_float(odd << 16) * p * s;
    f[4 * i + 2] = __uint_as_float(even & 0xffff0000u) * p * s;
    f[4 * i + 3] = __uint_as_float(odd & 0xffff0000u) * p * s;
  }
}

// Places of the block's rows r0 .. r0 + nr - 1, by all threads of the block.
__device__ void find_rows(const PagedView &C, const RowsView &R, int r0, int nr, RowPlace *place) {
  // the sequences that end at or before the first row come before its own
  __shared__ int s_before;
  if (threadIdx.x == 0) s_before = 0;
  __syncthreads();
  int c = 0, bad = 0;
  for (int i = threadIdx.x; i < R.n; i += PC_THREADS) {
    int lo, hi;
    bad |= !seq_rows(R, i, lo, hi);
    c += hi <= r0;
  }
  c = __reduce_add_sync(FULL_MASK, c);
  if ((threadIdx.x & 31) == 0 && c) atomicAdd(&s_before, c);
  bad = __syncthreads_or(bad);  // then no row of the call is touched
  if (threadIdx.x < nr) {
    const int r = r0 + threadIdx.x;
    int b = s_before;
    while (b < R.n && R.cu[b + 1] <= r) b++;
    RowPlace p{-2, 0};
    if (!bad && b < R.n && r >= R.cu[b]) {
      const long pos = (long)R.len[b] - R.cu[b + 1] + r;
      p.page = -1;
      if (pos >= 0 && pos < (long)R.width * C.P) {
        const int i = (int)(pos / C.P);
        const int page = R.table[(size_t)b * R.width + i];
        if (page >= 0 && page < C.n_pages) p = {page, (int)(pos - (long)i * C.P)};
      }
      if (p.page < 0) flag_rows(R, RLT_PAGED_BAD_PAGE);
    }
    place[threadIdx.x] = p;
  }
  __syncthreads();
}

// Elements of a thread's piece: 16 where that is half a block of the scale (a
// 16-byte access on the stored side), else 8.
template <int KIND, int DH> constexpr int piece_of() {
  return KIND == RLT_KV_E4M3 && DH >= 32 ? 16 : 8;
}

template <typename T, int KIND, int DH, bool WRITE>
__global__ void __launch_bounds__(PC_THREADS)
    k_paged_rows(PagedView C, RowsView R, T *k, T *v, int64_t ld, int rows_per_block) {
  __shared__ RowPlace place[PC_MAX_ROWS];
  pdl_wait();
  const int r0 = blockIdx.x * rows_per_block, nr = min(rows_per_block, R.rows - r0);
  find_rows(C, R, r0, nr, place);
  constexpr int N = piece_of<KIND, DH>(), PIECES = DH / N;
  constexpr int BLOCK = DH < 32 ? DH : 32, LANES = BLOCK / N;
  constexpr int SB = DH / BLOCK;  // scale bytes of a row's head
  constexpr int U = 4;            // pieces of a thread in flight
  const int half = C.H * PIECES, per_row = 2 * half;
  // (row, j): this thread's next piece, j = (kv, head, piece). Every lane of a
  // warp takes every trip: a block's lanes exchange their maxima.
  int row = threadIdx.x / per_row, j = threadIdx.x - row * per_row;
  const int trips = (nr * per_row + PC_THREADS - 1) / PC_THREADS;
  for (int t = 0; t < trips; t += U) {
    T *dense[U];
    size_t cell[U];
    int page[U], piece[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const RowPlace p = row < nr ? place[row] : RowPlace{-2, 0};
      const int kv = j >= half, jj = j - kv * half, h = jj / PIECES;
      piece[u] = jj % PIECES;
      page[u] = p.page;
      dense[u] = (kv ? v : k) + (int64_t)(r0 + row) * ld + h * DH + piece[u] * N;
      cell[u] = (((size_t)max(p.page, 0) * C.H + h) * 2 + kv) * C.P + p.slot;
      for (j += PC_THREADS; j >= per_row; j -= per_row) row++;
    }
    if constexpr (KIND == RLT_KV_PLAIN) {
      constexpr int Q = N * sizeof(T) / 16;
      uint4 x[U][Q];
#pragma unroll
      for (int u = 0; u < U; u++)
        if (page[u] >= 0) {
          const T *held = reinterpret_cast<const T *>(C.pages) + cell[u] * DH + piece[u] * N;
#pragma unroll
          for (int y = 0; y < Q; y++)
            x[u][y] = reinterpret_cast<const uint4 *>(WRITE ? dense[u] : held)[y];
        } else {
#pragma unroll
          for (int y = 0; y < Q; y++) x[u][y] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
      for (int u = 0; u < U; u++)
        if (page[u] >= (WRITE ? 0 : -1)) {
          T *held = reinterpret_cast<T *>(C.pages) + cell[u] * DH + piece[u] * N;
#pragma unroll
          for (int y = 0; y < Q; y++)
            reinterpret_cast<uint4 *>(WRITE ? held : dense[u])[y] = x[u][y];
        }
    } else if constexpr (WRITE) {
      float f[U][N];
#pragma unroll
      for (int u = 0; u < U; u++) {
#pragma unroll
        for (int i = 0; i < N; i++) f[u][i] = 0.f;
        if (page[u] >= 0) load_row<N>(dense[u], f[u]);
      }
#pragma unroll
      for (int u = 0; u < U; u++) {
        uint32_t w[N / 4];
        const int sb = quantise<N, LANES>(f[u], w);
        if (page[u] >= 0) {
          uint8_t *dst = C.pages + cell[u] * DH + piece[u] * N;
          if constexpr (N == 16)
            *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
          else
            *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
          if (piece[u] % LANES == 0) C.scales[cell[u] * SB + piece[u] / LANES] = (uint8_t)sb;
        }
      }
    } else {
      uint32_t w[U][N / 4];
      int sb[U];
#pragma unroll
      for (int u = 0; u < U; u++) {
#pragma unroll
        for (int i = 0; i < N / 4; i++) w[u][i] = 0;
        sb[u] = 127;
        if (page[u] >= 0) {
          const uint8_t *src = C.pages + cell[u] * DH + piece[u] * N;
          if constexpr (N == 16) {
            const uint4 y = *reinterpret_cast<const uint4 *>(src);
            w[u][0] = y.x, w[u][1] = y.y, w[u][N / 4 - 2] = y.z, w[u][N / 4 - 1] = y.w;
          } else {
            const uint2 y = *reinterpret_cast<const uint2 *>(src);
            w[u][0] = y.x, w[u][1] = y.y;
          }
          sb[u] = C.scales[cell[u] * SB + piece[u] / LANES];
        }
      }
#pragma unroll
      for (int u = 0; u < U; u++) {
        float f[N];
        dequantise<N>(w[u], sb[u], f);
        if (page[u] >= -1) store_row<N>(dense[u], f);
      }
    }
  }
}

template <bool WRITE>
cudaError_t run_rows(const rlt_paged_kv *c, const rlt_paged_rows *w, void *k, void *v, int64_t ld,
                     cudaStream_t st) {
  const PagedView C = paged_view(c);
  const RowsView R = rows_view(w);
  // about 2048 pieces a block, but blocks for every SM first
  const int piece = c->kind == RLT_KV_E4M3 && c->head_dim >= 32 ? 16 : 8;
  const int per_row = 2 * c->n_kv_heads * c->head_dim / piece, sms = sm_count();
  int nr = 2048 / per_row;
  if (nr > w->rows / (2 * sms > 0 ? 2 * sms : 1)) nr = w->rows / (2 * sms > 0 ? 2 * sms : 1);
  nr = nr < 1 ? 1 : nr > PC_MAX_ROWS ? PC_MAX_ROWS : nr;
  const int grid = (w->rows + nr - 1) / nr;
#define RLT_PAGED_CASE(T, KIND, DH)                                                             \
  return launch_pdl(k_paged_rows<T, KIND, DH, WRITE>, grid, PC_THREADS, 0, st, C, R,            \
                    static_cast<T *>(k), static_cast<T *>(v), ld, nr)
#define RLT_PAGED_DH(T, KIND)                      \
  switch (c->head_dim) {                           \
    case 16: RLT_PAGED_CASE(T, KIND, 16);          \
    case 32: RLT_PAGED_CASE(T, KIND, 32);          \
    case 64: RLT_PAGED_CASE(T, KIND, 64);          \
    default: RLT_PAGED_CASE(T, KIND, 128);         \
  }
  if (c->dtype == RLT_BF16) {
    if (c->kind == RLT_KV_PLAIN) RLT_PAGED_DH(bf16, RLT_KV_PLAIN)
    RLT_PAGED_DH(bf16, RLT_KV_E4M3)
  }
  if (c->kind == RLT_KV_PLAIN) RLT_PAGED_DH(float, RLT_KV_PLAIN)
  RLT_PAGED_DH(float, RLT_KV_E4M3)
#undef RLT_PAGED_DH
#undef RLT_PAGED_CASE
}

int rows_call(bool write, const rlt_paged_kv *c, const rlt_paged_rows *w, void *k, void *v,
              int64_t ld, rlt_stream stream) {
  const int rc = paged_args_status(c, w);
  if (rc != RLT_OK) return rc;
  if (w->rows == 0) return RLT_OK;
  if (!dense_rows_ok(k, ld, c->n_kv_heads, c->head_dim, c->dtype) ||
      !dense_rows_ok(v, ld, c->n_kv_heads, c->head_dim, c->dtype))
    return RLT_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  return cuda_status_internal(
      write ? run_rows<true>(c, w, k, v, ld, st) : run_rows<false>(c, w, k, v, ld, st), __LINE__);
}

}  // namespace
}  // namespace rlt

extern "C" {

RLT_API int rlt_paged_append(const rlt_paged_kv *cache, const rlt_paged_rows *where, const void *k,
                             const void *v, int64_t ld, rlt_stream stream) {
  return rlt::rows_call(true, cache, where, const_cast<void *>(k), const_cast<void *>(v), ld,
                        stream);
}

RLT_API int rlt_paged_read(const rlt_paged_kv *cache, const rlt_paged_rows *where, void *k, void *v,
                           int64_t ld, rlt_stream stream) {
  return rlt::rows_call(false, cache, where, k, v, ld, stream);
}

}  // extern "C"
