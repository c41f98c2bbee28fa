// spec_cache_evict: a smaller cache of the heaviest tokens.
//
// First kernel, a CTA to (request, head): the weight of the last token that
// is kept, by radix selection over the weights' order-preserving bits, then
// one pass that writes the kept positions in order.  Second kernel, a CTA to
// (request, head, new page, K or V): gathers the kept rows and gives the block
// the scale they need.
#include "cache.cuh"
#include "launch.h"

namespace sv {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kGatherThreads = 256;

// Bits that order as the weights do: NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (!(w == w)) return 0;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Sum over the CTA's threads of lower index, and over all of them.
__device__ __forceinline__ int block_rank(int v, int *s_warp, int &all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int y = lane < kSelectThreads / 32 ? s_warp[lane] : 0;
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(~0u, y, o);
    if (lane >= o) y += z;
  }
  all = __shfl_sync(~0u, y, 31);
  const int before = __shfl_sync(~0u, y, max(warp - 1, 0));
  return x - v + (warp > 0 ? before : 0);
}

__global__ void __launch_bounds__(kSelectThreads) cache_select_kernel(const CacheEvictParams P) {
  __shared__ int s_hist[256], s_warp[32], s_digit, s_above;
  const int head = blockIdx.x % P.c.kv_heads, b = blockIdx.x / P.c.kv_heads;
  const int tid = threadIdx.x;
  const int64_t len = P.cache_len[b];
  const int64_t cap_d = capacity(P.d);
  const bool bad_len = len < 0 || len > min(capacity(P.c), static_cast<int64_t>(P.positions)) ||
                       min(len, static_cast<int64_t>(P.keep)) > cap_d;
  const int T = bad_len ? 0 : static_cast<int>(len);
  const int kc = min(P.keep, T), late = min(P.recent, kc);
  int bad = 0;
  for (int64_t i = tid; i << P.c.page_shift < T; i += kSelectThreads) bad |= page_at(P.c, b, i) < 0;
  for (int64_t i = tid; i << P.d.page_shift < kc; i += kSelectThreads) bad |= page_at(P.d, b, i) < 0;
  const bool bad_page = __syncthreads_or(bad);
  const int total = bad_page ? 0 : kc;
  if (head == 0 && tid == 0) {
    if (P.status) P.status[b] = bad_len ? SPEC_STATUS_BAD_LENGTH : bad_page ? SPEC_STATUS_BAD_PAGE : SPEC_STATUS_OK;
    P.new_len[b] = total;
  }
  int32_t *kept = P.kept + (static_cast<int64_t>(b) * P.c.kv_heads + head) * P.keep;
  float *kw = P.kept_weights ? P.kept_weights + (static_cast<int64_t>(b) * P.c.kv_heads + head) * P.keep : nullptr;
  for (int i = total + tid; i < P.keep; i += kSelectThreads) {
    kept[i] = -1;
    if (kw) kw[i] = 0.0f;
  }
  if (total == 0) return;

  const float *w = P.weights + b * P.ws[0] + head * P.ws[1];
  const int M = T - late;  // positions that compete
  const int want = kc - late;
  // The want-th largest key, a byte at a time; `left` of those equal to it are kept.
  uint32_t key = 0;
  int left = want;
  for (int shift = 24; want > 0 && shift >= 0; shift -= 8) {
    if (tid < 256) s_hist[tid] = 0;
    __syncthreads();
    const uint32_t high = shift == 24 ? 0 : ~0u << (shift + 8);
    for (int i = tid; i < M; i += kSelectThreads) {
      const uint32_t u = weight_key(w[i]);
      if ((u & high) == (key & high)) atomicAdd(&s_hist[u >> shift & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int above = 0, d = 255;
      while (d > 0 && above + s_hist[d] < left) above += s_hist[d--];
      s_digit = d;
      s_above = above;
    }
    __syncthreads();
    key |= static_cast<uint32_t>(s_digit) << shift;
    left -= s_above;
    __syncthreads();
  }
  // Kept positions in order: above the key, or equal to it and among the first `left` of those.
  int out = 0, equal = 0;
  for (int i0 = 0; i0 < M && want > 0; i0 += kSelectThreads) {
    const int i = i0 + tid;
    const float x = i < M ? w[i] : 0.0f;
    const uint32_t u = weight_key(x);
    const bool tie = i < M && u == key;
    int ties, taken;
    const int before = block_rank(tie, s_warp, ties);
    const bool take = i < M && (u > key || (tie && equal + before < left));
    const int at = block_rank(take, s_warp, taken);
    if (take) {
      kept[out + at] = i;
      if (kw) kw[out + at] = x;
    }
    out += taken;
    equal += ties;
  }
  for (int i = tid; i < late; i += kSelectThreads) {
    kept[want + i] = M + i;
    if (kw) kw[want + i] = w[M + i];
  }
}

__global__ void __launch_bounds__(kGatherThreads) cache_gather_kernel(const CacheEvictParams P, int pages) {
  __shared__ float s_max[kGatherThreads / 32];
  int64_t x = blockIdx.x;
  const bool is_v = x & 1;
  x >>= 1;
  const int w = static_cast<int>(x % pages);
  x /= pages;
  const int head = static_cast<int>(x % P.c.kv_heads), b = static_cast<int>(x / P.c.kv_heads);
  const int tid = threadIdx.x, D = P.c.head_dim, shift = P.c.page_shift;
  const int rows = min(P.new_len[b] - (w << shift), 1 << shift);
  if (rows <= 0) return;
  const int32_t *kept = P.kept + (static_cast<int64_t>(b) * P.c.kv_heads + head) * P.keep + (w << shift);
  const uint8_t *pool = is_v ? P.c.v : P.c.k;
  const float *scales = is_v ? P.c.v_scale : P.c.k_scale;
  const int pairs = D / 2;
  auto value = [&](int i) {
    const int t = kept[i / pairs];
    const int page = page_at(P.c, b, t >> shift);
    const uint16_t two = *reinterpret_cast<const uint16_t *>(pool + block_offset(P.c, page, head) +
                                                             static_cast<int64_t>(t & ((1 << shift) - 1)) * D + i % pairs * 2);
    const float s = scales[page * P.c.scale_stride + head];
    float2 f = e4m3x2_to_float2(two);
    f.x *= s;
    f.y *= s;
    return f;
  };
  float amax = 0.0f;
  for (int i = tid; i < rows * pairs; i += kGatherThreads) {
    const float2 f = value(i);
    amax = fmaxf(amax, fmaxf(finite_abs(f.x), finite_abs(f.y)));
  }
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  if ((tid & 31) == 0) s_max[tid >> 5] = amax;
  __syncthreads();
  amax = s_max[0];
  for (int i = 1; i < kGatherThreads / 32; ++i) amax = fmaxf(amax, s_max[i]);
  const float scale = block_scale(amax);
  const int page = page_at(P.d, b, w);
  uint16_t *to = reinterpret_cast<uint16_t *>((is_v ? P.d.v : P.d.k) + block_offset(P.d, page, head));
  for (int i = tid; i < rows * pairs; i += kGatherThreads) {
    const float2 f = value(i);
    to[i] = static_cast<uint16_t>(to_e4m3x2(f.x / scale, f.y / scale));
  }
  if (tid == 0) (is_v ? P.d.v_scale : P.d.k_scale)[page * P.d.scale_stride + head] = scale;
}

}  // namespace

cudaError_t launch_cache_evict(const CacheEvictParams &P, cudaStream_t st) {
  const unsigned heads = static_cast<unsigned>(P.B * P.c.kv_heads);
  cudaError_t e = trace_launch("cache_select", st, [&] { cache_select_kernel<<<heads, kSelectThreads, 0, st>>>(P); });
  if (e != cudaSuccess) return e;
  const int pages = (P.keep + (1 << P.c.page_shift) - 1) >> P.c.page_shift;
  return trace_launch("cache_gather", st, [&] {
    cache_gather_kernel<<<2 * heads * pages, kGatherThreads, 0, st>>>(P, pages);
  });
}

}  // namespace sv
