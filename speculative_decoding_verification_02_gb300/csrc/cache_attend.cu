// spec_cache_attend: attention of the drafted rows over the 8-bit cache.
//
//   x_j = cap tanh(scale q.k_j / cap) over the positions that the row sees
//   out = sum_j exp(x_j - m) v_j / sum_j exp(x_j - m),  lse = m + log sum_j exp(x_j - m)
//
// in one pass with the running maximum m and sum.  Heads of 64 and 128 run on
// the tensor cores (cache_attend_tile.cuh), other widths a warp to a row.
#include <algorithm>

#include "cache.cuh"
#include "common.cuh"
#include "launch.h"

namespace sv {
namespace {

constexpr int kRowWarps = 4;  // rows to a CTA of the general kernel

// One warp to a row: 32 positions at a time, a lane scoring one of them, then
// the lanes across the components for the values.
template <int DT>
__global__ void __launch_bounds__(32 * kRowWarps) cache_attend_rows_kernel(const CacheAttendParams P) {
  __shared__ float s_q[kRowWarps][256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t rows = static_cast<int64_t>(P.B) * P.N * P.Hq;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kRowWarps + warp;
  if (r >= rows) return;
  const int h = static_cast<int>(r % P.Hq), i = static_cast<int>(r / P.Hq % P.N), b = static_cast<int>(r / P.Hq / P.N);
  const int head = h / P.group, D = P.c.head_dim;
  const int64_t base = P.cache_len[b];
  const int n = P.n_query ? P.n_query[b] : P.N;
  int st = SPEC_STATUS_OK;
  if (base < 0 || n < 0 || n > P.N || base + n > capacity(P.c)) st = SPEC_STATUS_BAD_LENGTH;

  const char *q = P.q + (b * P.qs[0] + i * P.qs[1] + h * P.qs[2]) * 2;
  for (int d = lane; d < D; d += 32) s_q[warp][d] = row_value<DT>(q, d);
  __syncwarp();
  float m = -INFINITY, sum = 0.0f, acc[8] = {};
  const int64_t T = st == SPEC_STATUS_OK ? base + n : 0;
  const bool live = i < n;
  const uint8_t *mask = P.mask ? P.mask + (static_cast<int64_t>(b) * P.N + i) * P.N : nullptr;
  for (int64_t t0 = 0; t0 < T; t0 += 32) {
    const int64_t j = t0 + lane;
    const int page = j < T ? page_at(P.c, b, j >> P.c.page_shift) : 0;
    if (__any_sync(~0u, page < 0)) {
      st = SPEC_STATUS_BAD_PAGE;
      break;
    }
    if (!live) continue;  // (the pages of a request decide its status on every row)
    const bool sees = j < T && (j < base || (mask ? mask[j - base] != 0 : j - base <= i));
    const int64_t at = block_offset(P.c, page, head) + (j & ((1 << P.c.page_shift) - 1)) * D;
    float x = -INFINITY;
    if (sees) {
      const uint4 *k = reinterpret_cast<const uint4 *>(P.c.k + at);
      float dot = 0.0f;
      for (int g = 0; g < D / 16; ++g) {
        const uint4 w4 = k[g];
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 lo = e4m3x2_to_float2(w[e] & 0xffff), hi = e4m3x2_to_float2(w[e] >> 16);
          const float *qq = &s_q[warp][g * 16 + e * 4];
          dot = fmaf(qq[0], lo.x, fmaf(qq[1], lo.y, fmaf(qq[2], hi.x, fmaf(qq[3], hi.y, dot))));
        }
      }
      x = capped_log2(P.scale * dot * P.c.k_scale[page * P.c.scale_stride + head], P.softcap);
    }
    float top = x;
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    const float next = fmaxf(m, top);
    const float ref = next == -INFINITY ? 0.0f : next;
    const float keep = exp2f(m - ref);
    const float p = sees ? exp2f(x - ref) : 0.0f;
    m = next;
    sum = sum * keep + warp_sum(p);
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] *= keep;
    const float vs = sees ? P.c.v_scale[page * P.c.scale_stride + head] : 0.0f;
    for (unsigned left = __ballot_sync(~0u, sees); left; left &= left - 1) {
      const int o = __ffs(left) - 1;
      const float w = __shfl_sync(~0u, p * vs, o);
      const uint8_t *v = P.c.v + __shfl_sync(~0u, at, o);
      for (int c = 0; c < 8; ++c) {
        const int d = lane + 32 * c;
        if (d < D) acc[c] = fmaf(w, e4m3x2_to_float2(v[d]).x, acc[c]);
      }
    }
  }
  const bool empty = st != SPEC_STATUS_OK || !live || sum == 0.0f;
  const float inv = 1.0f / sum;
  char *out = P.out + (b * P.os[0] + i * P.os[1] + h * P.os[2]) * 2;
  for (int c = 0; c < 8; ++c) {
    const int d = lane + 32 * c;
    if (d < D) put_value<DT>(out, d, empty ? 0.0f : acc[c] * inv);
  }
  if (lane == 0) {
    if (P.lse) P.lse[r] = empty ? -INFINITY : (m + log2f(sum)) * kLn2;
    if (P.status && i == 0 && h == 0) P.status[b] = st;
  }
}

// ------------------------------------------------------------------- host

int copies_of(int N, int group) {
  const int64_t rows = static_cast<int64_t>(N) * group;
  return rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
}

// Whether every row starts on an 8-byte boundary.
bool rows_on_grain(const void *p, const int64_t *s) {
  return reinterpret_cast<uintptr_t>(p) % 8 == 0 && s[0] % 4 == 0 && s[1] % 4 == 0 && s[2] % 4 == 0;
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// Requests to a launch: at most kTileRequests, and tiles that an int can number.
int requests_at_once(const CacheAttendParams &P) {
  const int rt = 128 / copies_of(P.N, P.group);
  const int64_t row_tiles = (static_cast<int64_t>(P.N) * P.group + rt - 1) / rt;
  const int64_t tiles = ((static_cast<int64_t>(P.c.table_stride) << P.c.page_shift) / kTilePositions + 1 + kTileUnitCost) * row_tiles * P.c.kv_heads;
  return static_cast<int>(std::min<int64_t>(kTileRequests, 2000000000LL / std::max(tiles, row_tiles * rt * P.c.kv_heads)));
}

size_t lay_out(CacheTilePlan &A, char *ws, int D) {
  const int ctas = device_sm_count(), rt = 128 / copies_of(A.p.N, A.p.group);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char *p = ws ? ws + off : nullptr;
    off = round256(off + bytes);
    return p;
  };
  A.verdict = reinterpret_cast<int *>(take(sizeof(int) * kTileRequests));
  A.range = reinterpret_cast<int2 *>(take(sizeof(int2) * ctas));
  A.begun = reinterpret_cast<int4 *>(take(sizeof(int4) * ctas));
  A.ml = reinterpret_cast<float2 *>(take(sizeof(float2) * 2 * ctas * rt));
  A.part = reinterpret_cast<float *>(take(sizeof(float) * 2 * ctas * rt * D));
  return off;
}

}  // namespace

bool cache_attend_on_tensor_cores(const CacheAttendParams &P) {
  // (a row's number times the group stays below 2^32: the multiplication that divides by it is exact)
  return (P.c.head_dim == 64 || P.c.head_dim == 128) && static_cast<int64_t>(P.N) * P.group * P.group < (1LL << 32) &&
         requests_at_once(P) > 0;
}

size_t cache_attend_workspace(const CacheAttendParams &P) {
  if (!cache_attend_on_tensor_cores(P)) return 0;
  CacheTilePlan A{};
  A.p = P;
  return lay_out(A, nullptr, P.c.head_dim);
}

cudaError_t launch_cache_attend(const CacheAttendParams &P, void *workspace, cudaStream_t st) {
  if (cache_attend_on_tensor_cores(P)) {
    CacheTilePlan A{};
    A.p = P;
    A.page_rows = std::min(1 << P.c.page_shift, kTilePositions);
    A.q_vec = rows_on_grain(P.q, P.qs);
    A.out_vec = rows_on_grain(P.out, P.os);
    A.ctas_inverse = ~0ull / device_sm_count() + 1;
    A.group_inverse = static_cast<uint32_t>((0x100000000ull + P.group - 1) / P.group);
    lay_out(A, static_cast<char *>(workspace), P.c.head_dim);
    CUtensorMap map;
    const cudaError_t made = cache_k_map(P.c, A.page_rows, &map);
    if (made != cudaSuccess) return made;
    const int at_once = requests_at_once(P), copies = copies_of(P.N, P.group);
    for (A.first = 0; A.first < P.B; A.first += at_once) {
      A.count = std::min(at_once, P.B - A.first);
      const cudaError_t e = (P.dtype == SPEC_DTYPE_BF16 ? launch_cache_attend_bf16 : launch_cache_attend_f16)(A, map, copies, st);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
  const int64_t rows = static_cast<int64_t>(P.B) * P.N * P.Hq;
  const unsigned grid = static_cast<unsigned>((rows + kRowWarps - 1) / kRowWarps);
  return trace_launch("cache_attend_rows", st, [&] {
    if (P.dtype == SPEC_DTYPE_BF16) cache_attend_rows_kernel<SPEC_DTYPE_BF16><<<grid, 32 * kRowWarps, 0, st>>>(P);
    else cache_attend_rows_kernel<SPEC_DTYPE_F16><<<grid, 32 * kRowWarps, 0, st>>>(P);
  });
}

}  // namespace sv
