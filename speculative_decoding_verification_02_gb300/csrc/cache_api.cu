// C ABI of the 8-bit cache: argument checks and parameter blocks.
#include <algorithm>
#include <cmath>
#include <cstdio>

#include "cache.cuh"
#include "launch.h"

namespace sv {
namespace {

constexpr int64_t kMaxGrid = 2147483647;

int cache_fail(cudaError_t e, const char *where) {
  char text[256];
  std::snprintf(text, sizeof text, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
  set_last_error(text);
  return SPEC_ECUDA;
}

bool on_grain(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// SPEC_OK when the pool's geometry is one that the kernels serve.
int check_cache(const spec_cache *c, CacheView *out) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return SPEC_EINVAL;
  if (c->num_pages < 1 || c->kv_heads < 1 || c->kv_heads > 65535 || c->table_stride < 0) return SPEC_EINVAL;
  if (c->table_stride > 0 && !c->table) return SPEC_EINVAL;
  if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16) return SPEC_EINVAL;
  int shift = 4;
  while (shift < 8 && (1 << shift) != c->page_size) ++shift;
  if ((1 << shift) != c->page_size) return SPEC_EINVAL;
  if ((static_cast<int64_t>(c->table_stride) << shift) > 2147483647LL - 256) return SPEC_EINVAL;  // positions are int32
  if (c->page_stride % 16 || c->page_stride < static_cast<int64_t>(c->kv_heads) * c->page_size * c->head_dim) return SPEC_EINVAL;
  if (c->scale_stride < c->kv_heads) return SPEC_EINVAL;
  if (!on_grain(c->k, 16) || !on_grain(c->v, 16) || !on_grain(c->k_scale, 4) || !on_grain(c->v_scale, 4)) return SPEC_EINVAL;
  *out = CacheView{static_cast<uint8_t *>(c->k), static_cast<uint8_t *>(c->v), c->k_scale, c->v_scale, c->page_stride,
                   c->scale_stride, c->num_pages, c->kv_heads, shift, c->head_dim, c->table, c->table_stride};
  return SPEC_OK;
}

int check_rows(int dtype, bool f32, const void *p) {
  if (dtype != SPEC_DTYPE_BF16 && dtype != SPEC_DTYPE_F16 && !(f32 && dtype == SPEC_DTYPE_F32)) return SPEC_EDTYPE;
  return on_grain(p, dtype == SPEC_DTYPE_F32 ? 4 : 2) ? SPEC_OK : SPEC_EINVAL;
}

bool strides_ok(const int64_t *s, int n) {
  if (!s) return false;
  for (int i = 0; i < n; ++i)
    if (s[i] < 0) return false;
  return true;
}

// SPEC_OK when a call that needs `need` bytes was given them.
int check_workspace(size_t need, const void *ws, size_t bytes) {
  return need == 0 || (ws && bytes >= need && on_grain(ws, 256)) ? SPEC_OK : SPEC_EWORKSPACE;
}

// (a smaller cap would overflow its reciprocal times a score)
bool cap_ok(float softcap) { return softcap == 0.0f || (std::isfinite(softcap) && softcap >= 1e-18f); }

cudaStream_t stream_of(void *s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

cudaError_t cache_k_map(const CacheView &c, int page_rows, CUtensorMap *map) {
  using Encode = decltype(&cuTensorMapEncodeTiled);
  static Encode encode = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<Encode>(f);
  }();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.kv_heads) << c.page_shift,
                              static_cast<cuuint64_t>(c.num_pages)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.page_stride)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(c.head_dim), static_cast<cuuint32_t>(page_rows), 1};
  const cuuint32_t ones[3] = {1, 1, 1};
  auto make = [&] {
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, c.k, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  c.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = make();
  if (r != CUDA_SUCCESS) {  // a driver's call wants a context, which a host thread has after its first call of the runtime that needs one
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaSetDevice(dev);
    if (e != cudaSuccess) return e;
    r = make();
  }
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_cache_workspace_size(int op, const spec_cache *cache, int B, int N, int Hq) {
  CacheView c;
  if (check_cache(cache, &c) != SPEC_OK || B < 0 || N < 0) return 0;
  if (op == SPEC_OP_CACHE_ATTEND && N > 0 && N <= SPEC_MAX_NODES && Hq > 0 && Hq % c.kv_heads == 0) {
    CacheAttendParams P{};
    P.c = c, P.B = B, P.N = N, P.Hq = Hq, P.group = Hq / c.kv_heads;
    return cache_attend_workspace(P);
  }
  return 0;
}

int spec_cache_append(const spec_cache *cache, const void *k, const int64_t *k_stride, const void *v,
                      const int64_t *v_stride, int dtype, int B, int n, const int32_t *index, int index_stride,
                      int n_rows, const int32_t *counts, const int32_t *cache_len, int32_t *new_len,
                      int32_t *status, void *stream) {
  CacheAppendParams P{};
  int rc = check_cache(cache, &P.c);
  if (rc != SPEC_OK) return rc;
  if (B < 0 || n < 0 || n_rows < 0 || !strides_ok(k_stride, 3) || !strides_ok(v_stride, 3)) return SPEC_EINVAL;
  if (index ? n_rows > index_stride : n_rows != n) return SPEC_EINVAL;
  if ((rc = check_rows(dtype, true, k)) != SPEC_OK || (rc = check_rows(dtype, true, v)) != SPEC_OK) return rc;
  if (B == 0) return SPEC_OK;
  if (!cache_len || !new_len || cache_len == new_len || (n > 0 && (!k || !v))) return SPEC_EINVAL;
  const int page = 1 << P.c.page_shift;
  P.touched = std::max<int64_t>(1, std::min<int64_t>((static_cast<int64_t>(n_rows) + page - 2) / page + 1, P.c.table_stride));
  if (2LL * B * P.touched * P.c.kv_heads > kMaxGrid) return SPEC_EINVAL;
  P.k = static_cast<const char *>(k);
  P.v = static_cast<const char *>(v);
  std::copy(k_stride, k_stride + 3, P.ks);
  std::copy(v_stride, v_stride + 3, P.vs);
  P.dtype = dtype, P.B = B, P.n = n, P.n_rows = n_rows, P.index_stride = index_stride;
  P.index = index, P.counts = counts, P.cache_len = cache_len, P.new_len = new_len, P.status = status;
  const cudaError_t e = launch_cache_append(P, stream_of(stream));
  return e == cudaSuccess ? SPEC_OK : cache_fail(e, "spec_cache_append");
}

int spec_cache_attend(const spec_cache *cache, const void *q, const int64_t *q_stride, int dtype, int B, int N,
                      int Hq, const int32_t *cache_len, const int32_t *n_query, const uint8_t *mask, float scale,
                      float softcap, void *out, const int64_t *out_stride, float *lse, int32_t *status,
                      void *workspace, size_t workspace_bytes, void *stream) {
  CacheAttendParams P{};
  int rc = check_cache(cache, &P.c);
  if (rc != SPEC_OK) return rc;
  if (B < 0 || N < 0 || N > SPEC_MAX_NODES || Hq < 1 || Hq % P.c.kv_heads || !strides_ok(q_stride, 3) || !strides_ok(out_stride, 3))
    return SPEC_EINVAL;
  if (!std::isfinite(scale) || !cap_ok(softcap)) return SPEC_EINVAL;
  if ((rc = check_rows(dtype, false, q)) != SPEC_OK || (rc = check_rows(dtype, false, out)) != SPEC_OK) return rc;
  if (B == 0 || (N == 0 && !status)) return SPEC_OK;
  if ((N > 0 && (!q || !out)) || !cache_len || static_cast<int64_t>(B) * std::max(N, 1) * Hq > kMaxGrid / 8) return SPEC_EINVAL;
  P.q = static_cast<const char *>(q);
  P.out = static_cast<char *>(out);
  std::copy(q_stride, q_stride + 3, P.qs);
  std::copy(out_stride, out_stride + 3, P.os);
  P.dtype = dtype, P.B = B, P.N = N, P.Hq = Hq, P.group = Hq / P.c.kv_heads;
  P.cache_len = cache_len, P.n_query = n_query, P.mask = mask, P.scale = scale, P.softcap = softcap;
  P.lse = lse, P.status = status;
  if ((rc = check_workspace(cache_attend_workspace(P), workspace, workspace_bytes)) != SPEC_OK) return rc;
  const cudaError_t e = launch_cache_attend(P, workspace, stream_of(stream));
  return e == cudaSuccess ? SPEC_OK : cache_fail(e, "spec_cache_attend");
}

int spec_cache_weights(const spec_cache *cache, const void *q, const int64_t *q_stride, int dtype, int B, int N,
                       int Hq, const float *lse, const int64_t *lse_stride, const int32_t *index, int index_stride,
                       int n_rows, const int32_t *counts, const int32_t *cache_len, float scale, float softcap,
                       const float *prev, const int64_t *prev_stride, float *out, const int64_t *out_stride,
                       int positions, int32_t *status, void *workspace, size_t workspace_bytes, void *stream) {
  CacheWeightsParams P{};
  int rc = check_cache(cache, &P.c);
  if (rc != SPEC_OK) return rc;
  if (B < 0 || N < 0 || N > SPEC_MAX_NODES || n_rows < 0 || n_rows > SPEC_MAX_NODES || Hq < 1 || Hq % P.c.kv_heads ||
      !strides_ok(q_stride, 3) || !strides_ok(lse_stride, 3) || !strides_ok(out_stride, 2) || (prev && !strides_ok(prev_stride, 2)))
    return SPEC_EINVAL;
  if ((index ? n_rows > index_stride : n_rows != N) || positions < 0) return SPEC_EINVAL;
  if (!std::isfinite(scale) || !cap_ok(softcap)) return SPEC_EINVAL;
  if ((rc = check_rows(dtype, false, q)) != SPEC_OK) return rc;
  if (B == 0) return SPEC_OK;
  if (!cache_len || (positions > 0 && !out) || (N > 0 && (!q || !lse))) return SPEC_EINVAL;
  // (tiles of a launch, and blocks of the general kernel, are numbered by an int)
  if (static_cast<int64_t>(B) * P.c.kv_heads * ((static_cast<int64_t>(P.c.table_stride) << P.c.page_shift) / 128 + 8) > kMaxGrid)
    return SPEC_EINVAL;
  P.q = static_cast<const char *>(q);
  std::copy(q_stride, q_stride + 3, P.qs);
  std::copy(lse_stride, lse_stride + 3, P.ls);
  std::copy(out_stride, out_stride + 2, P.out_s);
  if (prev) std::copy(prev_stride, prev_stride + 2, P.prev_s);
  P.dtype = dtype, P.B = B, P.N = N, P.Hq = Hq, P.group = Hq / P.c.kv_heads, P.n_rows = n_rows, P.index_stride = index_stride;
  P.lse = lse, P.index = index, P.counts = counts, P.cache_len = cache_len, P.scale = scale, P.softcap = softcap;
  P.prev = prev, P.out = out, P.positions = positions, P.status = status;
  (void)workspace, (void)workspace_bytes;
  const cudaError_t e = launch_cache_weights(P, stream_of(stream));
  return e == cudaSuccess ? SPEC_OK : cache_fail(e, "spec_cache_weights");
}

int spec_cache_evict(const spec_cache *cache, const spec_cache *dst, int B, const int32_t *cache_len,
                     const float *weights, const int64_t *weights_stride, int positions, int keep, int recent,
                     int32_t *kept,
                     float *kept_weights, int32_t *new_len, int32_t *status, void *workspace,
                     size_t workspace_bytes, void *stream) {
  CacheEvictParams P{};
  int rc = check_cache(cache, &P.c);
  if (rc == SPEC_OK) rc = check_cache(dst, &P.d);
  if (rc != SPEC_OK) return rc;
  if (P.c.kv_heads != P.d.kv_heads || P.c.page_shift != P.d.page_shift || P.c.head_dim != P.d.head_dim) return SPEC_EINVAL;
  if (B < 0 || positions < 0 || keep < 1 || keep > (1 << 30) || recent < 0 || recent > keep || !strides_ok(weights_stride, 2)) return SPEC_EINVAL;
  if (B == 0) return SPEC_OK;
  if (!cache_len || (positions > 0 && !weights) || !kept || !new_len || cache_len == new_len) return SPEC_EINVAL;
  const int64_t pages = (static_cast<int64_t>(keep) + (1 << P.c.page_shift) - 1) >> P.c.page_shift;
  if (2LL * B * P.c.kv_heads * std::max<int64_t>(pages, 16) > kMaxGrid) return SPEC_EINVAL;
  P.B = B, P.positions = positions, P.keep = keep, P.recent = recent, P.cache_len = cache_len, P.weights = weights;
  std::copy(weights_stride, weights_stride + 2, P.ws);
  P.kept = kept, P.kept_weights = kept_weights, P.new_len = new_len, P.status = status;
  (void)workspace, (void)workspace_bytes;
  const cudaError_t e = launch_cache_evict(P, stream_of(stream));
  return e == cudaSuccess ? SPEC_OK : cache_fail(e, "spec_cache_evict");
}

}  // extern "C"
