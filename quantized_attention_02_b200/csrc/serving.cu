// serving.cu -- C ABI of the serving operators declared in include/sage_attn.h: argument checks and
// launches of the query / key norm with rotation and of the append into a paged cache.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "rope_kernels.cuh"
#include "sage_attn.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool stride_ok(int64_t s, int64_t extent) { return extent <= 1 || (s > 0 && s % 8 == 0); }

// A view [B][H][N][d]: present, aligned, strides usable.
bool view_ok(const void* p, const sage_strides* s, int64_t B, int64_t H, int64_t N) {
  return p && s && aligned16(p) && stride_ok(s->b, B) && stride_ok(s->h, H) && stride_ok(s->n, N);
}

int check_common(int Hq, int Hk, int d, int dtype) {
  if (Hq <= 0 || Hk < 0 || d <= 0) return SAGE_ERR_INVALID;
  if (dtype != SAGE_F16 && dtype != SAGE_BF16) return SAGE_ERR_INVALID;
  if (d != 64 && d != 128) return SAGE_ERR_UNSUPPORTED;
  return SAGE_OK;
}

int check_rope(const float* cos, const float* sin, const void* qw, const void* kw, int d, int rot, int table_rows,
               bool by_token, int N, float eps) {
  if (!cos || !sin || !aligned16(cos) || !aligned16(sin) || !aligned16(qw) || !aligned16(kw)) return SAGE_ERR_INVALID;
  if (rot < 16 || rot > d || rot % 16 != 0 || table_rows <= 0) return SAGE_ERR_INVALID;
  if (by_token && table_rows < N) return SAGE_ERR_INVALID;
  return std::isfinite(eps) && eps >= 0.f ? SAGE_OK : SAGE_ERR_INVALID;
}

// log2 of a supported page size, -1 for the others
int page_shift(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

int check_pages(int num_pages, int page_size) {
  if (num_pages <= 0 || page_size <= 0) return SAGE_ERR_INVALID;
  if (page_shift(page_size) < 0 || static_cast<int64_t>(num_pages) * page_size >= (1ll << 31))
    return SAGE_ERR_UNSUPPORTED;
  return SAGE_OK;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? SAGE_OK : SAGE_ERR_CUDA; }

}  // namespace

extern "C" {

int sage_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const sage_strides* q_st,
                      const sage_strides* k_st, const sage_strides* q_out_st, const sage_strides* k_out_st,
                      const void* q_weight, const void* k_weight, const float* cos, const float* sin,
                      const int32_t* positions, int positions_per_batch, int B, int Hq, int Hk, int N, int d,
                      int rot_dim, int table_rows, int interleaved, float eps, int dtype, void* stream) {
  if (B < 0 || N < 0) return SAGE_ERR_INVALID;
  int rc = check_common(Hq, Hk, d, dtype);
  if (rc) return rc;
  if ((rc = check_rope(cos, sin, q_weight, k_weight, d, rot_dim, table_rows, !positions, N, eps))) return rc;
  if (B == 0 || N == 0) return SAGE_OK;
  if (!view_ok(q, q_st, B, Hq, N) || !view_ok(q_out, q_out_st, B, Hq, N)) return SAGE_ERR_INVALID;
  if (Hk > 0 && (!view_ok(k, k_st, B, Hk, N) || !view_ok(k_out, k_out_st, B, Hk, N))) return SAGE_ERR_INVALID;
  if (static_cast<int64_t>(B) * N * (Hq + static_cast<int64_t>(Hk)) >= (1ll << 31)) return SAGE_ERR_UNSUPPORTED;
  sage::RopeArgs a{};
  a.q = {q, q_out, q_weight, *q_st, *q_out_st};
  if (Hk > 0) a.k = {k, k_out, k_weight, *k_st, *k_out_st};
  a.cos = cos;
  a.sin = sin;
  a.positions = positions;
  a.positions_stride_b = positions_per_batch ? N : 0;
  a.B = B, a.N = N, a.Hq = Hq, a.Hk = Hk;
  a.d = d, a.rot = rot_dim, a.table_rows = table_rows;
  a.eps = eps;
  a.interleaved = interleaved != 0;
  a.bf16 = dtype == SAGE_BF16;
  return cuda_status(sage::launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream)));
}

int sage_qk_norm_rope_append(const void* q, const void* k, const void* v, void* q_out, void* k_cache, void* v_cache,
                             const sage_strides* q_st, const sage_strides* k_st, const sage_strides* v_st,
                             const sage_strides* q_out_st, const sage_strides* k_cache_st,
                             const sage_strides* v_cache_st, const void* q_weight, const void* k_weight,
                             const float* cos, const float* sin, const int32_t* positions, const int32_t* slots,
                             int T, int Hq, int Hk, int d, int rot_dim, int table_rows, int num_pages, int page_size,
                             int interleaved, float eps, int dtype, void* stream) {
  if (T < 0 || Hk <= 0) return SAGE_ERR_INVALID;
  int rc = check_common(Hq, Hk, d, dtype);
  if (rc) return rc;
  if ((rc = check_rope(cos, sin, q_weight, k_weight, d, rot_dim, table_rows, !positions, T, eps))) return rc;
  if ((rc = check_pages(num_pages, page_size))) return rc;
  if (T == 0) return SAGE_OK;
  if (!slots || !view_ok(q, q_st, 1, Hq, T) || !view_ok(q_out, q_out_st, 1, Hq, T) || !view_ok(k, k_st, 1, Hk, T) ||
      !view_ok(v, v_st, 1, Hk, T) || !view_ok(k_cache, k_cache_st, num_pages, Hk, page_size) ||
      !view_ok(v_cache, v_cache_st, num_pages, Hk, page_size))
    return SAGE_ERR_INVALID;
  if (static_cast<int64_t>(T) * (Hq + 2ll * Hk) >= (1ll << 31)) return SAGE_ERR_UNSUPPORTED;
  sage::RopeArgs a{};
  a.q = {q, q_out, q_weight, *q_st, *q_out_st};
  a.k = {k, k_cache, k_weight, *k_st, *k_cache_st};
  a.v = {v, v_cache, nullptr, *v_st, *v_cache_st};
  a.cos = cos;
  a.sin = sin;
  a.positions = positions;
  a.slots = slots;
  a.B = 1, a.N = T, a.Hq = Hq, a.Hk = Hk, a.Hv = Hk;
  a.d = d, a.rot = rot_dim, a.table_rows = table_rows;
  a.page_shift = page_shift(page_size);
  a.slot_count = num_pages * page_size;
  a.eps = eps;
  a.interleaved = interleaved != 0;
  a.bf16 = dtype == SAGE_BF16;
  return cuda_status(sage::launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
