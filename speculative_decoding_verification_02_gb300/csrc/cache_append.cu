// spec_cache_append: rows of 16 or 32 bits into blocks of e4m3.
//
//   s'   = max(s if the block held tokens, smallest 2^e with amax(new rows) <= 448 2^e)
//   byte = RN_e4m3(x / s')   for the new rows; old rows again when s' > s
//
// Bound by memory: 2 bytes read and 1 written a value.  A block's scale needs
// all of its new rows, so the unit of work is one block (request, page, head,
// K or V).
#include "cache.cuh"
#include "launch.h"

namespace sv {
namespace {

constexpr int kAppendThreads = 256;

// The pages and index entries that the whole request uses, looked over by one
// CTA of each request, which sets its status and new length.
__device__ void append_verdict(const CacheAppendParams &P, int b, int64_t base, int cnt, bool bad_len) {
  int bad = 0;
  if (!bad_len && cnt > 0) {
    const int64_t first = base >> P.c.page_shift, last = (base + cnt - 1) >> P.c.page_shift;
    for (int64_t i = first + threadIdx.x; i <= last; i += blockDim.x) bad |= page_at(P.c, b, i) < 0 ? 1 : 0;
    if (P.index)
      for (int i = threadIdx.x; i < cnt; i += blockDim.x) {
        const int t = P.index[static_cast<int64_t>(b) * P.index_stride + i];
        bad |= t < 0 || t >= P.n ? 2 : 0;
      }
  }
  const int page = __syncthreads_or(bad & 1), index = __syncthreads_or(bad & 2);
  if (threadIdx.x == 0) {
    const int st = bad_len ? SPEC_STATUS_BAD_LENGTH
                   : page  ? SPEC_STATUS_BAD_PAGE
                   : index ? SPEC_STATUS_BAD_INDEX
                           : SPEC_STATUS_OK;
    if (P.status) P.status[b] = st;
    P.new_len[b] = static_cast<int>(base) + (st == SPEC_STATUS_OK ? cnt : 0);
  }
}

template <int DT>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const CacheAppendParams P) {
  // block index: ((request, touched page), head, K or V)
  int64_t x = blockIdx.x;
  const bool is_v = x & 1;
  x >>= 1;
  const int head = static_cast<int>(x % P.c.kv_heads);
  x /= P.c.kv_heads;
  const int w = static_cast<int>(x % P.touched);
  const int b = static_cast<int>(x / P.touched);
  const int tid = threadIdx.x;

  const int64_t base = P.cache_len[b];
  const int cnt = P.counts ? P.counts[b] : P.n_rows;
  const bool bad_len = base < 0 || cnt < 0 || cnt > P.n_rows || base + cnt > capacity(P.c);
  if (w == 0 && head == 0 && !is_v) append_verdict(P, b, base, cnt, bad_len);
  if (bad_len) return;
  const int page_size = 1 << P.c.page_shift;
  const int64_t block = (base >> P.c.page_shift) + w;
  const int64_t start = block << P.c.page_shift;
  const int lo = static_cast<int>(max(base - start, static_cast<int64_t>(0)));
  const int hi = static_cast<int>(min(base + cnt - start, static_cast<int64_t>(page_size)));
  if (lo >= hi) return;
  const int page = page_at(P.c, b, block);
  if (page < 0) return;

  const int D = P.c.head_dim, rows = hi - lo;
  const char *src = is_v ? P.v : P.k;
  const int64_t es = DT == SPEC_DTYPE_F32 ? 4 : 2;
  const int64_t s0 = is_v ? P.vs[0] : P.ks[0], s1 = is_v ? P.vs[1] : P.ks[1], s2 = is_v ? P.vs[2] : P.ks[2];
  const int first = static_cast<int>(start + lo - base);  // the block's first new row
  const int32_t *index = P.index ? P.index + static_cast<int64_t>(b) * P.index_stride : nullptr;
  auto row_of = [&](int r) -> const char * {
    const int t = index ? index[first + r] : first + r;
    if (t < 0 || t >= P.n) return nullptr;
    return src + (b * s0 + t * s1 + head * s2) * es;
  };

  __shared__ float s_max[kAppendThreads / 32];
  float amax = 0.0f;
  const int pairs = D / 2;
  for (int i = tid; i < rows * pairs; i += kAppendThreads) {
    const char *row = row_of(i / pairs);
    if (!row) continue;
    const int d = i % pairs * 2;
    amax = fmaxf(amax, fmaxf(finite_abs(row_value<DT>(row, d)), finite_abs(row_value<DT>(row, d + 1))));
  }
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  if ((tid & 31) == 0) s_max[tid >> 5] = amax;
  float *scale = (is_v ? P.c.v_scale : P.c.k_scale) + page * P.c.scale_stride + head;
  const float was = *scale;
  __syncthreads();
  amax = s_max[0];
  for (int i = 1; i < kAppendThreads / 32; ++i) amax = fmaxf(amax, s_max[i]);
  const float need = block_scale(amax);
  const float now = lo > 0 ? fmaxf(was, need) : need;

  uint8_t *dst = (is_v ? P.c.v : P.c.k) + block_offset(P.c, page, head);
  if (lo > 0 && now > was) {  // tokens already there, rounded again
    uint16_t *old = reinterpret_cast<uint16_t *>(dst);
    for (int i = tid; i < lo * pairs; i += kAppendThreads) {
      const float2 x2 = e4m3x2_to_float2(old[i]);
      old[i] = static_cast<uint16_t>(to_e4m3x2(x2.x * was / now, x2.y * was / now));
    }
  }
  uint16_t *to = reinterpret_cast<uint16_t *>(dst + static_cast<int64_t>(lo) * D);
  for (int i = tid; i < rows * pairs; i += kAppendThreads) {
    const char *row = row_of(i / pairs);
    if (!row) continue;
    const int d = i % pairs * 2;
    to[i] = static_cast<uint16_t>(to_e4m3x2(row_value<DT>(row, d) / now, row_value<DT>(row, d + 1) / now));
  }
  if (tid == 0) *scale = now;
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendParams &P, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(2LL * P.B * P.touched * P.c.kv_heads);
  return trace_launch("cache_append", st, [&] {
    if (P.dtype == SPEC_DTYPE_F32) cache_append_kernel<SPEC_DTYPE_F32><<<grid, kAppendThreads, 0, st>>>(P);
    else if (P.dtype == SPEC_DTYPE_BF16) cache_append_kernel<SPEC_DTYPE_BF16><<<grid, kAppendThreads, 0, st>>>(P);
    else cache_append_kernel<SPEC_DTYPE_F16><<<grid, kAppendThreads, 0, st>>>(P);
  });
}

}  // namespace sv
