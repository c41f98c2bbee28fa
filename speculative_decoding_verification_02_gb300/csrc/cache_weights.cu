// spec_cache_weights: the attention weight that each cached token received.
//
//   out_j = prev_j + sum over rows of exp(x_rj - lse_r)
//
// A thread owns a position, so the sum is over a thread's own registers, in
// the rows' order: no atomics, the same bits on every run.
#include "cache.cuh"
#include "common.cuh"
#include "launch.h"

namespace sv {
namespace {

constexpr int kSpan = 128;     // positions (threads) to a CTA
constexpr int kRowsAtOnce = 8; // rows staged in shared memory

template <int DT>
__global__ void __launch_bounds__(kSpan) cache_weights_rows_kernel(const CacheWeightsParams P, int spans) {
  __shared__ float s_q[kRowsAtOnce][256];
  __shared__ float s_lse[kRowsAtOnce];
  __shared__ int s_row[kRowsAtOnce];
  int64_t x = blockIdx.x;
  const int span = static_cast<int>(x % spans);
  x /= spans;
  const int head = static_cast<int>(x % P.c.kv_heads), b = static_cast<int>(x / P.c.kv_heads);
  const int tid = threadIdx.x, D = P.c.head_dim;
  const int64_t base = P.cache_len[b];
  const int cnt = P.counts ? P.counts[b] : P.n_rows;
  const bool bad_len = base < 0 || cnt < 0 || cnt > P.n_rows || base + cnt > min(capacity(P.c), static_cast<int64_t>(P.positions));
  const int64_t T = bad_len ? 0 : base + cnt;
  int64_t j = static_cast<int64_t>(span) * kSpan;
  if (j >= T && !(span == 0 && head == 0)) return;

  int bad = 0;
  for (int64_t i = tid; i << P.c.page_shift < T; i += kSpan) bad |= page_at(P.c, b, i) < 0 ? 1 : 0;
  if (P.index && !bad_len)
    for (int i = tid; i < cnt; i += kSpan) {
      const int t = P.index[static_cast<int64_t>(b) * P.index_stride + i];
      bad |= t < 0 || t >= P.N ? 2 : 0;
    }
  const int bad_page = __syncthreads_or(bad & 1), bad_index = __syncthreads_or(bad & 2);
  if (span == 0 && head == 0 && tid == 0 && P.status)
    P.status[b] = bad_len     ? SPEC_STATUS_BAD_LENGTH
                  : bad_page  ? SPEC_STATUS_BAD_PAGE
                  : bad_index ? SPEC_STATUS_BAD_INDEX
                              : SPEC_STATUS_OK;
  if (bad_page || bad_index || j >= T) return;

  j += tid;
  const bool mine = j < T;
  const int page = mine ? page_at(P.c, b, j >> P.c.page_shift) : 0;
  const uint4 *k = reinterpret_cast<const uint4 *>(P.c.k + block_offset(P.c, page, head) +
                                                   (j & ((1 << P.c.page_shift) - 1)) * D);
  const float ks = mine ? P.scale * P.c.k_scale[page * P.c.scale_stride + head] : 0.0f;
  float total = 0.0f;
  const int rows = cnt * P.group;
  for (int r0 = 0; r0 < rows; r0 += kRowsAtOnce) {
    __syncthreads();
    const int here = min(kRowsAtOnce, rows - r0);
    for (int e = tid; e < here * D; e += kSpan) {
      const int r = r0 + e / D, i = r / P.group, h = head * P.group + r % P.group;
      const int t = P.index ? P.index[static_cast<int64_t>(b) * P.index_stride + i] : i;
      s_q[e / D][e % D] = row_value<DT>(P.q + (b * P.qs[0] + t * P.qs[1] + h * P.qs[2]) * 2, e % D);
      if (e % D == 0) {
        s_lse[e / D] = P.lse[(static_cast<int64_t>(b) * P.N + t) * P.Hq + h] * kLog2e;
        s_row[e / D] = i;
      }
    }
    __syncthreads();
    if (!mine) continue;
    for (int r = 0; r < here; ++r) {
      if (s_lse[r] == -INFINITY || j - base > s_row[r]) continue;
      float dot = 0.0f;
      for (int g = 0; g < D / 16; ++g) {
        const uint4 w4 = k[g];
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 lo = e4m3x2_to_float2(w[e] & 0xffff), hi = e4m3x2_to_float2(w[e] >> 16);
          const float *qq = &s_q[r][g * 16 + e * 4];
          dot = fmaf(qq[0], lo.x, fmaf(qq[1], lo.y, fmaf(qq[2], hi.x, fmaf(qq[3], hi.y, dot))));
        }
      }
      total += exp2f(capped_log2(dot * ks, P.softcap) - s_lse[r]);
    }
  }
  if (!mine) return;
  const float prev = P.prev ? P.prev[b * P.prev_s[0] + head * P.prev_s[1] + j] : 0.0f;
  P.out[b * P.out_s[0] + head * P.out_s[1] + j] = prev + total;
}

}  // namespace

cudaError_t launch_cache_weights(const CacheWeightsParams &P, cudaStream_t st) {
  const int64_t most = static_cast<int64_t>(P.c.table_stride) << P.c.page_shift;
  const int spans = most > 0 ? static_cast<int>((most + kSpan - 1) / kSpan) : 1;
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(spans) * P.c.kv_heads * P.B);
  return trace_launch("cache_weights_rows", st, [&] {
    if (P.dtype == SPEC_DTYPE_BF16) cache_weights_rows_kernel<SPEC_DTYPE_BF16><<<grid, kSpan, 0, st>>>(P, spans);
    else cache_weights_rows_kernel<SPEC_DTYPE_F16><<<grid, kSpan, 0, st>>>(P, spans);
  });
}

}  // namespace sv
