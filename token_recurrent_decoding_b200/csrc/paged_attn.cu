// rlt_attend_paged: checks, the choice of kernels, launches.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "paged_attn.cuh"
#include "paged_attn_tc.cuh"

namespace rlt {
namespace {

bool wide_kernel(const rlt_paged_kv *c) {
  return c->dtype == RLT_BF16 && (c->head_dim == 64 || c->head_dim == 128);
}
int64_t partial_rows_of(const rlt_paged_kv *c, int n, int n_heads, int rows, int max_rows,
                        int max_len) {
  return partial_rows(wide_kernel(c), c->n_kv_heads, n, n_heads, rows, max_rows, max_len);
}

bool attn_shape_ok(const rlt_paged_kv *c, int n, int n_heads, int rows, int max_rows, int max_len) {
  return paged_shape_status(c) == RLT_OK && n >= 1 && n <= RLT_PAGED_MAX_SEQS && n_heads >= 1 &&
         n_heads <= 1024 && n_heads % c->n_kv_heads == 0 && rows >= 0 && max_rows >= 0 &&
         max_len >= 0 && max_len <= (1 << 28) && (int64_t)rows * n_heads <= (1 << 28) &&
         (int64_t)max_rows * n_heads <= (1 << 28) &&
         partial_rows_of(c, n, n_heads, rows, max_rows, max_len) <= (1 << 30);
}

size_t workspace_bytes_of(int dh, int64_t part_rows) {
  const size_t b = (size_t)part_rows * (dh + 2) * sizeof(float);
  return (b + 255) / 256 * 256 + 256;
}

template <int KIND, int DH, int MT>
cudaError_t launch_warp_kernel(const AttnArgs &A, int sms, cudaStream_t st) {
  using Cfg = PaCfg<KIND, DH, MT>;
  const cudaError_t e = ensure_smem_limit(k_pattn<KIND, DH, MT>, Cfg::bytes(RLT_PAGED_MAX_SEQS));
  if (e != cudaSuccess) return e;
  const int smem = Cfg::bytes(A.R.n), per_sm = std::max(1, std::min(Cfg::CTAS, 227 * 1024 / (smem + 1024)));
  // items of the batch, at most: a grid no larger than its work
  const int64_t tiles = (int64_t)A.R.rows * A.group / Cfg::RT + A.R.n;
  int64_t items = tiles * A.C.H * PA_MAX_SPLITS;
  const int64_t most = (int64_t)sms * per_sm;
  return launch_pdl(k_pattn<KIND, DH, MT>, (int)(items < most ? items : most), PA_THREADS, smem,
                    st, A);
}

template <int KIND, int DH>
cudaError_t launch_warp(const AttnArgs &A, int sms, cudaStream_t st) {
  // one tile of 16 rows where no sequence has more; three-part operands leave
  // no registers for a second
  if (KIND == PA_F32 || KIND == PA_E4M3_F32 || (int64_t)A.max_rows * A.group <= 16)
    return launch_warp_kernel<KIND, DH, 1>(A, sms, st);
  if constexpr (KIND == PA_BF16 || KIND == PA_E4M3)
    return launch_warp_kernel<KIND, DH, 2>(A, sms, st);
  return cudaErrorUnknown;
}

template <int KIND> cudaError_t launch_attn(const AttnArgs &A, int dh, int sms, cudaStream_t st) {
  switch (dh) {
    case 16: return launch_warp<KIND, 16>(A, sms, st);
    case 32: return launch_warp<KIND, 32>(A, sms, st);
    case 64: return launch_warp<KIND, 64>(A, sms, st);
    default: return launch_warp<KIND, 128>(A, sms, st);
  }
}

template <bool E4, int DH>
cudaError_t launch_wide_kernel(const AttnArgs &A, int sms, cudaStream_t st) {
  using Cfg = PwCfg<DH>;
  const cudaError_t e = ensure_smem_limit(k_pattn_wide<E4, DH>, Cfg::bytes(RLT_PAGED_MAX_SEQS));
  if (e != cudaSuccess) return e;
  return launch_pdl(k_pattn_wide<E4, DH>, sms, PW_THREADS, Cfg::bytes(A.R.n), st, A);
}

cudaError_t launch_wide(const AttnArgs &A, bool e4, int dh, int sms, cudaStream_t st) {
  if (dh == 64)
    return e4 ? launch_wide_kernel<true, 64>(A, sms, st) : launch_wide_kernel<false, 64>(A, sms, st);
  return e4 ? launch_wide_kernel<true, 128>(A, sms, st) : launch_wide_kernel<false, 128>(A, sms, st);
}

template <typename T>
cudaError_t launch_merge(const AttnArgs &A, int dh, int sms, cudaStream_t st) {
  const int64_t warps = (int64_t)A.R.rows * A.heads;
  const int grid = (int)(warps / 8 + 1 < 4 * sms ? warps / 8 + 1 : 4 * sms);
  const size_t smem = Plan::bytes(A.R.n);
  switch (dh) {
    case 16: return launch_pdl(k_pattn_merge<T, 16>, grid, 256, smem, st, A);
    case 32: return launch_pdl(k_pattn_merge<T, 32>, grid, 256, smem, st, A);
    case 64: return launch_pdl(k_pattn_merge<T, 64>, grid, 256, smem, st, A);
    default: return launch_pdl(k_pattn_merge<T, 128>, grid, 256, smem, st, A);
  }
}

}  // namespace
}  // namespace rlt

using namespace rlt;

extern "C" {

RLT_API size_t rlt_attend_paged_workspace_bytes(const rlt_paged_kv *cache, int n, int n_heads,
                                                int rows, int max_rows, int max_len) {
  if (!attn_shape_ok(cache, n, n_heads, rows, max_rows, max_len)) return 0;
  return workspace_bytes_of(cache->head_dim,
                            partial_rows_of(cache, n, n_heads, rows, max_rows, max_len));
}

RLT_API int rlt_attend_paged(const rlt_paged_kv *c, const rlt_paged_rows *w, const void *q,
                             int64_t ldq, int n_heads, int max_rows, int max_len, int window,
                             void *out, int64_t ldo, float *lse, void *workspace,
                             size_t workspace_bytes, rlt_stream stream) {
  const int rc = paged_args_status(c, w);
  if (rc != RLT_OK) return rc;
  if (window < 0 || !attn_shape_ok(c, w->n, n_heads, w->rows, max_rows, max_len))
    return RLT_ERR_INVALID_ARG;
  if (w->rows == 0 || max_rows == 0) return RLT_OK;
  if (!dense_rows_ok(q, ldq, n_heads, c->head_dim, c->dtype) ||
      !dense_rows_ok(out, ldo, n_heads, c->head_dim, c->dtype) || !workspace ||
      ((uintptr_t)workspace & 255) || ((uintptr_t)lse & 3))
    return RLT_ERR_INVALID_ARG;
  const int64_t parts = partial_rows_of(c, w->n, n_heads, w->rows, max_rows, max_len);
  if (workspace_bytes < workspace_bytes_of(c->head_dim, parts)) return RLT_ERR_CAPACITY;
  AttnArgs A;
  A.C = paged_view(c);
  A.R = rows_view(w);
  A.q = q;
  A.out = out;
  A.lse = lse;
  A.ldq = ldq;
  A.ldo = ldo;
  A.heads = n_heads;
  A.group = n_heads / c->n_kv_heads;
  A.max_rows = max_rows;
  A.max_len = max_len;
  // positions are below max_len: a window of that or more hides nothing (and what
  // is left cannot overflow from rows before position 0)
  A.window = window < max_len ? window : 0;
  A.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)c->head_dim));
  A.part = static_cast<float *>(workspace);
  A.part_rows = (int)parts;
  A.wide = wide_kernel(c);
  A.es = c->kind == RLT_KV_E4M3 ? 1 : c->dtype == RLT_BF16 ? 2 : 4;
  cudaStream_t st = (cudaStream_t)stream;
  const int sms = sm_count(), dh = c->head_dim;
  const bool e4 = c->kind == RLT_KV_E4M3;
  if (sms < 1) return cuda_status_internal(cudaErrorInvalidDevice, __LINE__);
  cudaError_t e;
  if (c->dtype == RLT_BF16)
    e = e4 ? launch_attn<PA_E4M3>(A, dh, sms, st) : launch_attn<PA_BF16>(A, dh, sms, st);
  else
    e = e4 ? launch_attn<PA_E4M3_F32>(A, dh, sms, st) : launch_attn<PA_F32>(A, dh, sms, st);
  if (e == cudaSuccess && may_be_wide(A.wide, c->n_kv_heads, n_heads, max_rows))
    e = launch_wide(A, e4, dh, sms, st);
  if (e == cudaSuccess && parts > 0)
    e = c->dtype == RLT_BF16 ? launch_merge<bf16>(A, dh, sms, st)
                             : launch_merge<float>(A, dh, sms, st);
  return cuda_status_internal(e, __LINE__);
}

}  // extern "C"
