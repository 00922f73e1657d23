// Rows of keys and values into a paged cache (rlt_paged_append) and out of it
// (rlt_paged_read), as they are or in 8 bits.
//
// One thread moves eight elements of a row's head: a 16-byte (bf16) or
// 32-byte (fp32) piece on the dense side, 8 bytes of e4m3 on the stored one,
// with the block's largest magnitude found by min(32, DH) / 8 neighbouring
// lanes. The least e with a <= 448 * 2^e comes from a's own bits: for
// a = f * 2^x, 1 <= f < 2, it is x - 8, plus one where f > 1.75 (448 = 1.75 *
// 2^8). x * 2^-e is exact, so the conversion to e4m3 is the only rounding.
// Bound by memory; a block takes a few neighbouring rows, finds their
// sequences once, and keeps four pieces a thread in flight.
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

// Eight dense elements <-> fp32.
__device__ __forceinline__ void load8(const float *p, float f[8]) {
  const float4 a = *reinterpret_cast<const float4 *>(p);
  const float4 b = *(reinterpret_cast<const float4 *>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void load8(const bf16 *p, float f[8]) { ld16_coherent(p, f); }
__device__ __forceinline__ void store8(float *p, const float f[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(bf16 *p, const float f[8]) {
  *reinterpret_cast<uint4 *>(p) =
      make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// Eight elements as e4m3 under a scale shared by LANES neighbouring lanes;
// returns the scale byte. The lanes of a block are all active.
template <int LANES>
__device__ __forceinline__ int quantise8(const float f[8], uint2 &out) {
  // magnitudes as bits: ordered like the values, infinities and NaN above all
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) a = max(a, __float_as_uint(f[i]) & 0x7fffffffu);
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(FULL_MASK, a, o));
  if (a >= 0x7f800000u) {
    out = make_uint2(0, 0);
    return 255;
  }
  // subnormals (exponent field 0) lie far below the least scale
  int e = (int)(a >> 23) - 127 - 8 + ((a & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, E4M3_EMIN);
  const float inv = pow2f(-e);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const float2 x = make_float2(f[4 * i] * inv, f[4 * i + 1] * inv);
    const float2 y = make_float2(f[4 * i + 2] * inv, f[4 * i + 3] * inv);
    w[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3) |
           ((uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3) << 16);
  }
  out = make_uint2(w[0], w[1]);
  return e + 127;
}

__device__ __forceinline__ void dequantise8(uint2 v, int sb, float f[8]) {
  const float s = __uint_as_float((uint32_t)sb << 23);  // byte 255: infinity, times zero NaN
  const uint32_t w[2] = {v.x, v.y};
#pragma unroll
  for (int i = 0; i < 2; i++) {
    // elements 1, 3 of the word, then 0, 2; raw bf16 bits widened to fp32
    const uint32_t odd = e4m3x2_raw(w[i]), even = e4m3x2_raw(w[i] << 8);
    const float p = __uint_as_float(0x7b800000u);  // 2^120
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

template <typename T, int KIND, int DH, bool WRITE>
__global__ void __launch_bounds__(PC_THREADS)
    k_paged_rows(PagedView C, RowsView R, T *k, T *v, int64_t ld, int rows_per_block) {
  __shared__ RowPlace place[PC_MAX_ROWS];
  pdl_wait();
  const int r0 = blockIdx.x * rows_per_block, nr = min(rows_per_block, R.rows - r0);
  find_rows(C, R, r0, nr, place);
  constexpr int PIECES = DH / 8;                       // of a row's head
  constexpr int BLOCK = DH < 32 ? DH : 32, LANES = BLOCK / 8;
  constexpr int SB = DH / BLOCK;                       // scale bytes of a row's head
  const int per_row = 2 * C.H * PIECES, total = nr * per_row;
  // every lane of a warp takes every trip: a block's lanes exchange their maxima
  for (int base = threadIdx.x & ~31; base < total; base += PC_THREADS) {
    const int i = base + (threadIdx.x & 31);
    const int row = i / per_row, j = i - row * per_row;
    const int kv = j / (C.H * PIECES), jj = j - kv * (C.H * PIECES);
    const int h = jj / PIECES, piece = jj - h * PIECES;
    const RowPlace p = i < total ? place[row] : RowPlace{-2, 0};
    T *dense = (kv ? v : k) + (int64_t)(r0 + row) * ld + h * DH + piece * 8;
    const size_t cell = (((size_t)max(p.page, 0) * C.H + h) * 2 + kv) * C.P + p.slot;
    if (KIND == RLT_KV_PLAIN) {
      T *held = reinterpret_cast<T *>(C.pages) + cell * DH + piece * 8;
      constexpr int N = 8 * sizeof(T) / 16;
      const uint4 *src = reinterpret_cast<const uint4 *>(WRITE ? dense : held);
      uint4 *dst = reinterpret_cast<uint4 *>(WRITE ? held : dense);
      if (p.page >= 0) {
#pragma unroll
        for (int x = 0; x < N; x++) dst[x] = src[x];
      } else if (!WRITE && p.page == -1) {
#pragma unroll
        for (int x = 0; x < N; x++) dst[x] = make_uint4(0, 0, 0, 0);
      }
    } else if (WRITE) {
      float f[8] = {};
      if (p.page >= 0) load8(dense, f);
      uint2 q;
      const int sb = quantise8<LANES>(f, q);
      if (p.page >= 0) {
        *reinterpret_cast<uint2 *>(C.pages + cell * DH + piece * 8) = q;
        if (piece % LANES == 0) C.scales[cell * SB + piece / LANES] = (uint8_t)sb;
      }
    } else {
      float f[8] = {};
      if (p.page >= 0)
        dequantise8(*reinterpret_cast<const uint2 *>(C.pages + cell * DH + piece * 8),
                    C.scales[cell * SB + piece / LANES], f);
      if (p.page >= -1) store8(dense, f);
    }
  }
}

template <bool WRITE>
cudaError_t run_rows(const rlt_paged_kv *c, const rlt_paged_rows *w, void *k, void *v, int64_t ld,
                     cudaStream_t st) {
  const PagedView C = paged_view(c);
  const RowsView R = rows_view(w);
  // about 2048 pieces a block, but blocks for every SM first
  const int per_row = 2 * c->n_kv_heads * c->head_dim / 8, sms = sm_count();
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
