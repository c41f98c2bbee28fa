// spec_cache_append: rows of 16 or 32 bits into blocks of e4m3.
//
//   s'   = max(s if the block held tokens, smallest 2^e with amax(new rows) <= 448 2^e)
//   byte = RN_e4m3(x / s')   for the new rows; old rows again when s' > s
//
// 2 bytes are read and 1 written a value.  A block's scale needs all of its new
// rows, so the unit of work is one block (request, page, head, K or V), a CTA to
// each.  Four prompts of 3,000 to 8,001 tokens, 8 heads of 128 in bf16: 30 us,
// 5.1 TB/s, bound by instruction issue (74% of the slots); with a division for
// each 16 bytes' row it was 36 us, reading the rows twice 73 us.  A batch's nine
// rows a request: 8.7 us for 64 requests.  16 requests are one turn of CTAs, a
// block's chain of loads (4.3 us); 64 are 2,048 CTAs, four of them to an SM at
// 64 registers, so more than three turns, half of them for second pages that
// few requests' rows reach.
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

// 16 bytes of a row in registers: 8 values of 16 bits, or 4 of 32.
template <int DT>
struct Piece {
  static constexpr int kSize = DT == SPEC_DTYPE_F32 ? 4 : 2, kValues = 16 / kSize;
  // Sign-less bits order as magnitudes do, so the maximum is taken over them, two 16-bit values at a time.  kNext: what carries
  // the first infinity into the sign's place.
  static constexpr uint32_t kMagnitude = DT == SPEC_DTYPE_F32 ? 0x7fffffffu : 0x7fff7fffu;
  static constexpr uint32_t kNext = DT == SPEC_DTYPE_F32 ? 0x00800000u : DT == SPEC_DTYPE_BF16 ? 0x00800080u : 0x04000400u;
  static constexpr uint32_t kSign = ~kMagnitude;

  // The largest finite magnitudes' bits so far; the answer says whether the piece holds an infinity or NaN.
  __device__ static bool largest(const uint4 &w, uint32_t &most) {
    uint32_t u[4] = {w.x & kMagnitude, w.y & kMagnitude, w.z & kMagnitude, w.w & kMagnitude};
    const uint32_t odd = ((u[0] + kNext) | (u[1] + kNext) | (u[2] + kNext) | (u[3] + kNext)) & kSign;
    if (odd) [[unlikely]] {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t t = (u[e] + kNext) & kSign;
        u[e] &= kSize == 4 ? (t ? 0u : ~0u) : ~((t >> 15) * 0xffffu);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) most = kSize == 4 ? max(most, u[e]) : __vmaxu2(most, u[e]);
    return odd != 0;
  }
  __device__ static float magnitude(uint32_t most) {
    if constexpr (kSize == 4) return __uint_as_float(most);
    const uint32_t m = max(most & 0xffff, most >> 16);
    if constexpr (DT == SPEC_DTYPE_BF16) return __uint_as_float(m << 16);
    return __half2float(__ushort_as_half(static_cast<unsigned short>(m)));
  }
  __device__ static void unpack(const uint4 &w, float *x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (DT == SPEC_DTYPE_F32) {
        x[e] = __uint_as_float(u[e]);
      } else if constexpr (DT == SPEC_DTYPE_BF16) {
        x[2 * e] = __uint_as_float(u[e] << 16);
        x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[e]));
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
      }
    }
  }
};

// The rare cases are functions of their own: inlined, they took a tenth of the
// kernel's time for their instructions alone.

// A piece that holds an infinity or NaN, or goes into a block whose scale of a
// caller's own stays: the quotients rounded to odd, and so once, as the
// definition has it.
template <int DT>
__device__ __noinline__ uint2 odd_codes(uint4 v, float scale) {
  using W = Piece<DT>;
  float x[W::kValues];
  W::unpack(v, x);
#pragma unroll
  for (int e = 0; e < W::kValues; ++e) {
    const float y = x[e] / scale;
    x[e] = fabsf(x[e]) == INFINITY ? NAN : round_to_odd(y, fmaf(-y, scale, x[e]));
  }
  uint32_t code[2] = {};
#pragma unroll
  for (int e = 0; e < W::kValues; e += 2) code[e / 4] |= finite_e4m3x2(x[e], x[e + 1]) << (8 * (e & 2));
  return make_uint2(code[0], code[1]);
}

// Four stored values of a block whose scale grows from `was` to the power of two 1 / inv.
__device__ __noinline__ uint32_t rounded_again(uint32_t v, float was, float inv) {
  const float2 a = e4m3x2_to_float2(v & 0xffff), c = e4m3x2_to_float2(v >> 16);
  return to_e4m3x2(product_to_odd(a.x, was) * inv, product_to_odd(a.y, was) * inv) |
         to_e4m3x2(product_to_odd(c.x, was) * inv, product_to_odd(c.y, was) * inv) << 16;
}

// VEC: every row starts on a 16-byte boundary.  A thread keeps up to kHeld
// pieces of the block in registers between the maximum and the rounding, which
// at 128 tokens of 128 values is all of them: the rows are read once.
constexpr int kHeld = 8;

// PER_ROW: pieces of a row (a power of two), 0: any.
template <int DT, bool VEC, int PER_ROW>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const CacheAppendParams P) {
  using W = Piece<DT>;
  // block index: ((request, touched page), head, K or V)
  uint32_t x = blockIdx.x;
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

  const int D = P.c.head_dim, rows = hi - lo;
  const int64_t s0 = is_v ? P.vs[0] : P.ks[0], s1 = is_v ? P.vs[1] : P.ks[1], s2 = is_v ? P.vs[2] : P.ks[2];
  const int first = static_cast<int>(start + lo - base);  // the block's first new row
  const char *src = (is_v ? P.v : P.k) + (b * s0 + head * s2) * W::kSize;
  const int32_t *index = P.index ? P.index + static_cast<int64_t>(b) * P.index_stride + first : nullptr;
  const int per_row = PER_ROW ? PER_ROW : D / W::kValues, pieces = rows * per_row;
  // piece i of the block's new rows; false for a row whose index is out of range
  auto load = [&](int i, uint4 &v) {
    const int r = i / per_row, t = index ? index[r] : first + r;
    if (t < 0 || t >= P.n) return false;
    const char *p = src + t * s1 * W::kSize + (i - r * per_row) * 16;
    if constexpr (VEC) {
      v = *reinterpret_cast<const uint4 *>(p);
    } else if constexpr (W::kSize == 4) {
      const uint32_t *q = reinterpret_cast<const uint32_t *>(p);
      v = make_uint4(q[0], q[1], q[2], q[3]);
    } else {
      const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
      v = make_uint4(q[0] | q[1] << 16, q[2] | q[3] << 16, q[4] | q[5] << 16, q[6] | q[7] << 16);
    }
    return true;
  };
  __shared__ float s_max[kAppendThreads / 32];
  uint4 held[kHeld];
  bool real[kHeld];
  uint32_t most = 0;
  bool odd = false;  // an infinity or NaN among this thread's values
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int i = tid + k * kAppendThreads;
    held[k] = make_uint4(0, 0, 0, 0);
    real[k] = i < pieces && load(i, held[k]);
  }
  float *scale = (is_v ? P.c.v_scale : P.c.k_scale) + max(page, 0) * P.c.scale_stride + head;
  const float was = *scale;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) odd |= W::largest(held[k], most);
  for (int i = tid + kHeld * kAppendThreads; i < pieces; i += kAppendThreads) {
    uint4 v;
    if (load(i, v)) odd |= W::largest(v, most);
  }
  float amax = W::magnitude(most);
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  if ((tid & 31) == 0) s_max[tid >> 5] = amax;
  __syncthreads();
  if (page < 0) return;
#pragma unroll
  for (int i = 0; i < kAppendThreads / 32; ++i) amax = fmaxf(amax, s_max[i]);
  const float need = block_scale(amax);
  const float now = lo > 0 ? fmaxf(was, need) : need;
  // a power of two but where a caller's own scale stays
  const float inv = 1.0f / now;
  const bool exact = (__float_as_uint(now) & 0x7fffffu) == 0;

  uint8_t *dst = (is_v ? P.c.v : P.c.k) + block_offset(P.c, page, head);
  if (lo > 0 && now > was) {  // tokens already there, rounded again (now is a power of two)
    uint32_t *old = reinterpret_cast<uint32_t *>(dst);
    for (int i = tid; i < lo * D / 4; i += kAppendThreads) old[i] = rounded_again(old[i], was, inv);
  }
  uint8_t *to = dst + static_cast<int64_t>(lo) * D;
  auto put = [&](int i, const uint4 &v) {
    float x[W::kValues];
    W::unpack(v, x);
    uint32_t code[W::kValues / 4];
#pragma unroll
    for (int e = 0; e < W::kValues; ++e) x[e] *= inv;
#pragma unroll
    for (int e = 0; e < W::kValues / 4; ++e)
      code[e] = finite_e4m3x2(x[4 * e], x[4 * e + 1]) | finite_e4m3x2(x[4 * e + 2], x[4 * e + 3]) << 16;
    uint2 two = make_uint2(code[0], W::kValues == 8 ? code[W::kValues / 4 - 1] : 0);
    if (odd || !exact) [[unlikely]] two = odd_codes<DT>(v, now);
    if constexpr (W::kValues == 8) reinterpret_cast<uint2 *>(to)[i] = two;
    else reinterpret_cast<uint32_t *>(to)[i] = two.x;
  };
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (real[k]) put(tid + k * kAppendThreads, held[k]);
  for (int i = tid + kHeld * kAppendThreads; i < pieces; i += kAppendThreads) {
    uint4 v;
    if (load(i, v)) put(i, v);
  }
  if (tid == 0) *scale = now;
}

template <int DT>
void launch_append(const CacheAppendParams &P, unsigned grid, cudaStream_t st) {
  constexpr int kRow128 = 128 / Piece<DT>::kValues, kRow64 = 64 / Piece<DT>::kValues;
  constexpr int kSize = Piece<DT>::kSize;
  bool vec = reinterpret_cast<uintptr_t>(P.k) % 16 == 0 && reinterpret_cast<uintptr_t>(P.v) % 16 == 0;
  for (int i = 0; i < 3; ++i) vec = vec && P.ks[i] * kSize % 16 == 0 && P.vs[i] * kSize % 16 == 0;
  if (vec && P.c.head_dim == 128) cache_append_kernel<DT, true, kRow128><<<grid, kAppendThreads, 0, st>>>(P);
  else if (vec && P.c.head_dim == 64) cache_append_kernel<DT, true, kRow64><<<grid, kAppendThreads, 0, st>>>(P);
  else if (vec) cache_append_kernel<DT, true, 0><<<grid, kAppendThreads, 0, st>>>(P);
  else cache_append_kernel<DT, false, 0><<<grid, kAppendThreads, 0, st>>>(P);
}

}  // namespace

cudaError_t launch_cache_append(const CacheAppendParams &P, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(2LL * P.B * P.touched * P.c.kv_heads);
  return trace_launch("cache_append", st, [&] {
    if (P.dtype == SPEC_DTYPE_F32) launch_append<SPEC_DTYPE_F32>(P, grid, st);
    else if (P.dtype == SPEC_DTYPE_BF16) launch_append<SPEC_DTYPE_BF16>(P, grid, st);
    else launch_append<SPEC_DTYPE_F16>(P, grid, st);
  });
}

}  // namespace sv
