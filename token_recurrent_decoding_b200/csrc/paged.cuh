// Device and host pieces shared by the paged serving kernels: the cache's
// view, which rows a call is about, and the 8-bit elements.
//
// An 8-bit element is an e4m3 float (sign, four exponent bits of bias 7, three
// of fraction) under a power of two shared by a block of B = min(32, DH)
// elements of a row. Its magnitude bits, shifted to a bf16's exponent and
// fraction, read as the value times 2^-120 (bf16's bias is 127; e4m3's
// subnormals become bf16 subnormals of the same scale), so two exact
// multiplications by powers of two give the value in bf16.
#pragma once

#include "../../include/rlt.h"
#include "common.cuh"
#include "internal.h"

namespace rlt {

constexpr float E4M3_MAX = 448.f;
constexpr int E4M3_EMIN = -110;  // keeps every stored value a normal bf16
constexpr int E4M3_EMAX = 120;   // of the largest finite numbers: 2^128 > 448 * 2^119

struct PagedView {
  uint8_t *pages;
  uint8_t *scales;
  int n_pages, P, H;  // pages, positions per page, kv heads
};

struct RowsView {
  const int *table, *cu, *len;
  int width, n, rows;
  int *status;
};

inline PagedView paged_view(const rlt_paged_kv *c) {
  return {static_cast<uint8_t *>(c->pages), c->scales, c->n_pages, c->page_size, c->n_kv_heads};
}
inline RowsView rows_view(const rlt_paged_rows *w) {
  return {w->page_table, w->cu_rows, w->kv_len, w->table_width, w->n, w->rows, w->status};
}

// Shape of a cache (host): INVALID_ARG, UNSUPPORTED or OK.
inline int paged_shape_status(const rlt_paged_kv *c) {
  if (!c) return RLT_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->page_size < 16 || c->page_size > 1024 || c->page_size % 16 ||
      c->n_kv_heads < 1 || c->n_kv_heads > 1024)
    return RLT_ERR_INVALID_ARG;
  if (c->dtype != RLT_F32 && c->dtype != RLT_BF16) return RLT_ERR_INVALID_ARG;
  if (c->kind != RLT_KV_PLAIN && c->kind != RLT_KV_E4M3) return RLT_ERR_INVALID_ARG;
  if (!(c->head_dim == 16 || c->head_dim == 32 || c->head_dim == 64 || c->head_dim == 128))
    return RLT_ERR_UNSUPPORTED;
  return RLT_OK;
}

inline int paged_args_status(const rlt_paged_kv *c, const rlt_paged_rows *w) {
  const int rc = paged_shape_status(c);
  if (rc != RLT_OK) return rc;
  if (!w || !c->pages || ((uintptr_t)c->pages & 15)) return RLT_ERR_INVALID_ARG;
  if (c->kind == RLT_KV_E4M3 && (!c->scales || ((uintptr_t)c->scales & 15)))
    return RLT_ERR_INVALID_ARG;
  // (2^30: block and row numbers stay in 32 bits)
  if (!w->page_table || !w->cu_rows || !w->kv_len || w->table_width < 1 || w->rows < 0 ||
      w->rows > 1 << 30 || w->n < 1 || w->n > RLT_PAGED_MAX_SEQS)
    return RLT_ERR_INVALID_ARG;
  return RLT_OK;
}

// Whether dense rows of `heads` heads can be walked in 16-byte steps.
inline bool dense_rows_ok(const void *p, int64_t ld, int heads, int dh, int dtype) {
  const int es = dtype == RLT_BF16 ? 2 : 4;
  return p && !((uintptr_t)p & 15) && ld >= (int64_t)heads * dh && ld * es % 16 == 0 &&
         ld <= (int64_t)1 << 40;
}

inline int sm_count() {
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return v;
}

// Launch with programmatic stream serialisation (see common.cuh): every paged
// kernel waits for its predecessors before it reads what they wrote.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), int grid, int block, size_t smem, cudaStream_t st,
                       Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = st == nullptr ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

__device__ __forceinline__ void flag_rows(const RowsView &R, int bit) {
  if (R.status) atomicOr(R.status, bit);
}

// Sequence b's rows [lo, hi); false (and flagged) where they are not rows of the call.
__device__ __forceinline__ bool seq_rows(const RowsView &R, int b, int &lo, int &hi) {
  lo = R.cu[b];
  hi = R.cu[b + 1];
  if (lo < 0 || hi < lo || hi > R.rows) {
    flag_rows(R, RLT_PAGED_BAD_ROWS);
    return false;
  }
  return true;
}

// ------------------------------------------------------------ 8-bit elements
// Two e4m3 codes in the upper bytes of w's halves -> their values * 2^-120 as bf16.
__device__ __forceinline__ uint32_t e4m3x2_raw(uint32_t w) {
  return (w & 0x80008000u) | ((w >> 4) & 0x07f007f0u);
}
__device__ __forceinline__ uint32_t bmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
constexpr uint32_t BF2_P120 = 0x7b807b80u;  // 2^120 twice
// scale bytes (biased by 127, as bf16's exponent) -> a pair of powers of two
__device__ __forceinline__ uint32_t scale_pair(uint32_t lo, uint32_t hi) {
  return (lo << 7) | (hi << 23);
}
__device__ __forceinline__ uint32_t e4m3x2_value(uint32_t w, uint32_t scale2) {
  return bmul2(bmul2(e4m3x2_raw(w), BF2_P120), scale2);
}
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }

}  // namespace rlt
