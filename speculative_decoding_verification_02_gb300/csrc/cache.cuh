// Shared parts of the 8-bit cache kernels: the pool's geometry, the page
// table, e4m3 conversions and block scales, and the parameter blocks.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "spec_verify.h"

namespace sv {

// A pool of pages and a page table, as the kernels use them.
struct CacheView {
  uint8_t *k, *v;
  float *k_scale, *v_scale;
  int64_t page_stride, scale_stride;
  int num_pages, kv_heads, page_shift, head_dim;  // page_size = 1 << page_shift
  const int32_t *table;
  int table_stride;
};

// Positions that a request's table can hold.
inline int64_t capacity_of(const CacheView &c) { return static_cast<int64_t>(c.table_stride) << c.page_shift; }

struct CacheAppendParams {
  CacheView c;
  const char *k, *v;
  int64_t ks[3], vs[3];  // element strides: request, token, head
  int dtype, B, n, n_rows, index_stride;
  int touched;  // pages that a request's rows can touch at most
  const int32_t *index, *counts, *cache_len;
  int32_t *new_len, *status;
};

struct CacheAttendParams {
  CacheView c;
  const char *q;
  char *out;
  int64_t qs[3], os[3];
  int dtype, B, N, Hq, group;  // group: query heads to a kv head
  const int32_t *cache_len, *n_query;
  const uint8_t *mask;
  float scale, softcap;
  float *lse;
  int32_t *status;
};

constexpr int kTilePositions = 128;  // positions to a tile of the tensor-core kernels
constexpr int kTileRequests = 256;   // requests to one of their launches
constexpr int kTileUnitCost = 8;     // (cache_attend_tile.cuh)

// A launch of spec_cache_attend's tensor-core path.
struct CacheTilePlan {
  CacheAttendParams p;
  int first, count;     // requests of this launch
  int page_rows;        // rows of a page that one copy brings: min(page size, 128)
  bool q_vec, out_vec;  // rows of q and out start on 8-byte boundaries
  uint32_t group_inverse;  // 2^32 / group, rounded up
  uint64_t ctas_inverse;   // 2^64 / CTAs, rounded up
  int *verdict;          // the requests' status
  int2 *range;           // [CTA] first tile; whether it gave up waiting
  int4 *begun;           // [CTA] the unit that it began and a later one ended
  float2 *ml;           // [CTA][2][rows of a unit]: reference and sum of partial rows
  float *part;          // [CTA][2][head_dim / 4][rows of a unit][4]
};

struct CacheWeightsParams {
  CacheView c;
  const char *q;
  int64_t qs[3];
  int dtype, B, N, Hq, group, n_rows, index_stride;
  const float *lse;
  int64_t ls[3];
  const int32_t *index, *counts, *cache_len;
  float scale, softcap;
  const float *prev;
  float *out;
  int64_t prev_s[2], out_s[2];
  int positions;
  int32_t *status;
};

struct CacheEvictParams {
  CacheView c, d;
  int B, positions, keep, recent;
  const int32_t *cache_len;
  const float *weights;
  int64_t ws[2];
  int32_t *kept;
  float *kept_weights;
  int32_t *new_len, *status;
};

cudaError_t launch_cache_append(const CacheAppendParams &P, cudaStream_t st);
// Heads of 64 and 128 take the tensor-core path and need a workspace.
bool cache_attend_on_tensor_cores(const CacheAttendParams &P);
size_t cache_attend_workspace(const CacheAttendParams &P);
cudaError_t launch_cache_attend(const CacheAttendParams &P, void *workspace, cudaStream_t st);
cudaError_t launch_cache_attend_bf16(const CacheTilePlan &A, const CUtensorMap &map, int copies, cudaStream_t st);
cudaError_t launch_cache_attend_f16(const CacheTilePlan &A, const CUtensorMap &map, int copies, cudaStream_t st);
// Tensor map of the keys for copies of page_rows rows of one page and head,
// in the shared-memory swizzle of a row's length (cache_api.cu).
cudaError_t cache_k_map(const CacheView &c, int page_rows, CUtensorMap *map);
cudaError_t launch_cache_weights(const CacheWeightsParams &P, cudaStream_t st);
cudaError_t launch_cache_evict(const CacheEvictParams &P, cudaStream_t st);

// f() the first time it is called for the current device, as `done` remembers.
template <class F>
inline cudaError_t once_per_device(F &&f, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit && done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = f();
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

#ifdef __CUDACC__

constexpr int kScaleLow = -60, kScaleHigh = 60;  // exponents that a block's scale can have
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The smallest power of two s with amax <= 448 s, within the exponents above.
// 448 = 1.75 * 2^8: the exponent of amax less 8, and one more when its
// significand is above 1.75.  Exact: it reads amax's bits.
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(kScaleLow, min(kScaleHigh, e));
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// |x| for the maximum of a block: infinities and NaN do not count.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.0f;
}

// Two values (already divided by the scale) to e4m3, a in the low byte:
// nearest even, saturated at 448; infinities become NaN, as NaN does.
__device__ __forceinline__ uint32_t finite_e4m3x2(float a, float b) {  // (neither is infinite)
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  if (fabsf(a) == INFINITY) a = NAN;
  if (fabsf(b) == INFINITY) b = NAN;
  return finite_e4m3x2(a, b);
}

// y with its last bit set where rounding to it left something out (`rest`: the
// exact value less y, of which the sign counts), and cut off instead of rounded.
// Rounding that to e4m3 gives what one rounding of the exact value does; of y
// itself, a value close to the middle of two would have become the middle.
__device__ __forceinline__ float round_to_odd(float y, float rest) {
  if (!(fabsf(rest) > 0.0f) || y == 0.0f) return y;
  return __uint_as_float((__float_as_uint(y) - ((rest > 0.0f) != (y > 0.0f) ? 1u : 0u)) | 1u);
}
__device__ __forceinline__ float product_to_odd(float a, float b) {
  const float y = a * b;
  return round_to_odd(y, fmaf(a, b, -y));
}

// Two e4m3 bytes (low byte first) to two halves: exact.
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return *reinterpret_cast<__half2 *>(&r);
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) { return __half22float2(e4m3x2_to_half2(two)); }

template <int DT>
__device__ __forceinline__ float row_value(const char *p, int64_t i) {
  if constexpr (DT == SPEC_DTYPE_F32) return reinterpret_cast<const float *>(p)[i];
  else if constexpr (DT == SPEC_DTYPE_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
  else return __half2float(reinterpret_cast<const __half *>(p)[i]);
}

// A lane's 2 or 4 consecutive values of a row, from one load.
template <int EACH>
__device__ __forceinline__ uint2 raw_each(const char *row, int lane) {
  if constexpr (EACH == 4) return reinterpret_cast<const uint2 *>(row)[lane];
  else return make_uint2(reinterpret_cast<const uint32_t *>(row)[lane], 0);
}
template <int DT, int EACH>
__device__ __forceinline__ void unpack_each(const uint2 &v, float *x) {
  const uint32_t w[2] = {v.x, v.y};
#pragma unroll
  for (int e = 0; e < EACH / 2; ++e) {
    if constexpr (DT == SPEC_DTYPE_BF16) {
      x[2 * e] = __uint_as_float(w[e] << 16), x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
      x[2 * e] = f.x, x[2 * e + 1] = f.y;
    }
  }
}

// Rounded once, to nearest even.
template <int DT>
__device__ __forceinline__ void put_value(char *p, int64_t i, float x) {
  if constexpr (DT == SPEC_DTYPE_BF16) reinterpret_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16(x);
  else reinterpret_cast<__half *>(p)[i] = __float2half(x);
}

// Page of a request's position block `i`, or -1 when the table names a page
// outside the pool.
__device__ __forceinline__ int page_at(const CacheView &c, int b, int64_t i) {
  const int p = c.table[static_cast<int64_t>(b) * c.table_stride + i];
  return p >= 0 && p < c.num_pages ? p : -1;
}

// Byte offset of (page, head, slot 0) in the pool.
__device__ __forceinline__ int64_t block_offset(const CacheView &c, int page, int head) {
  return page * c.page_stride + (static_cast<int64_t>(head) << c.page_shift) * c.head_dim;
}

// Positions that a request's table can hold.
__device__ __forceinline__ int64_t capacity(const CacheView &c) {
  return static_cast<int64_t>(c.table_stride) << c.page_shift;
}

// Capped score in units of log 2: x = scale q.k.
__device__ __forceinline__ float capped_log2(float x, float softcap) {
  return (softcap > 0.0f ? softcap * tanhf(x / softcap) : x) * kLog2e;
}

// Several scores in units of log 2 capped: cap tanh(x / cap), inv_cap = 1 / cap.  A formula of exponentials alone is off by a fixed
// part of the cap, 2^-22 and more, which at a cap of 30 is 1e-5 of a small score and of its weight.  So up to half the cap
// x P((x / cap)^2) is taken, P the polynomial through tanh(u) / u at the Chebyshev points of u^2 in [0, 1/4] (3e-8 off), and only a
// warp that holds a larger score goes on to 1 - 2 / (1 + exp(2 u)).  Every lane of the warp calls.
template <int N>
__device__ __forceinline__ void cap_scores(float *x, float inv_cap, float cap) {
  float most = 0.0f;
#pragma unroll
  for (int e = 0; e < N; ++e) most = fmaxf(most, fabsf(x[e]));
  const bool far = __any_sync(~0u, most * inv_cap > 0.5f);
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float u = x[e] * inv_cap, w = u * u;
    float y = x[e] * fmaf(fmaf(fmaf(fmaf(0.017131345f, w, -0.052984238f), w, 0.13324751f), w, -0.33333069f), w, 1.0f);
    if (far) [[unlikely]] {
      const float z = u * (2.0f * kLog2e);
      if (fabsf(u) > 0.5f) y = cap * (1.0f - __fdividef(2.0f, 1.0f + ex2(z > 120.0f ? 120.0f : z)));
    }
    x[e] = y;
  }
}

#endif

}  // namespace sv
