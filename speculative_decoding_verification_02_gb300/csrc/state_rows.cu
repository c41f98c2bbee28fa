// Linear attention over states for a few rows at a time, in fp32: single
// tokens and short chains, commits, and trees of any size; and every call that
// the tensor-core kernels (state_chunk.cuh) do not take.
//
// A CTA has one state head of one request and 16 columns (of value_dim) for
// each of its warps; the state's part stays in registers from its one load to
// its one store.  Lane 4 g + c of a warp holds rows [RPL g, RPL (g + 1)) of
// key_dim and columns 4 c .. 4 c + 3, two rows to a register pair.  Tokens are
// taken kBlock at a time.  With G the running sum of the decays within a block:
//   o_i = scale (e^{G_i} q_i S + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j)
//   S  <- e^{G_last} S + sum_j k_j (e^{G_last - G_j} v_j)^T
// so a row costs one packed multiply-add for two elements of S (the recurrence
// token by token: three).  Lane group g adds the terms of tokens g and g + 8 to
// its part of q_i S, so one reduction over the groups serves both.  The sums
// are exact (fixed point), so their differences are: forgetful tokens and long
// blocks lose nothing.  A tree's row takes its ancestors' terms instead, one
// after another along its path, with k and v from memory.
//
// The rows' copies to shared memory are under way before the state's loads
// wait for the request's slot.
//
// Bound by the state's bytes: 64 requests' single tokens, 48 heads of 128 x 128,
// 71 us in a graph of calls (5.7 TB/s; copying the states alone 60 us, as fast
// as a plain copy), their commits of up to 9 rows 76 us; as many read only 69 us
// (3.1 TB/s): the rows' arithmetic, some 60 instructions a row and warp, is not
// hidden.  One request's token 4.8 us, 5 rows 5.7 us: a chain of loads.  CTAs
// that stay and fetch the next unit's state ahead were slower (82, 90, 119 us):
// fewer warps.
#include <algorithm>
#include <type_traits>

#include "launch.h"
#include "state.cuh"

namespace sv {
namespace {

constexpr int kBlock = 16;  // tokens to a block
constexpr int kMaxWarps = 4;
constexpr int kMaxPath = SPEC_MAX_DEPTH + 1;

enum Mode { kCommit, kChain, kTree };

__device__ __forceinline__ float warp_add(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// Rows in shared memory, in their own type: RPL values to each of the 8 lane
// groups, and 16 bytes more, so that 8 rows' same pieces lie in different banks.
template <int RPL>
struct RowTile {
  static constexpr int kStride = 8 * RPL * 2 + 16;
};

__device__ __forceinline__ void copy_piece(void *to, const char *from, bool vec) {  // 8 values
  if (vec) {
    cp_async16(to, from);
  } else {
    const uint16_t *h = reinterpret_cast<const uint16_t *>(from);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = h[2 * e] | static_cast<uint32_t>(h[2 * e + 1]) << 16;
    *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Eight values of a row in 16 bytes to four register pairs.
template <int DT>
__device__ __forceinline__ void widen8(const uint4 &v, pair_t *x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = widen2<DT>(w[e]);
    x[e] = pack2(f.x, f.y);
  }
}

// q_i S for the four columns of a lane, summed over its group's rows of S.
template <int DT, int RPL>
__device__ __forceinline__ float4 row_product(const char *q, int g, const pair_t (&S)[RPL / 2][4]) {
  pair_t o[4] = {0, 0, 0, 0};
#pragma unroll
  for (int r = 0; r < RPL / 8; ++r) {
    pair_t x[4];
    widen8<DT>(*reinterpret_cast<const uint4 *>(q + (g * RPL + 8 * r) * 2), x);
#pragma unroll
    for (int y = 0; y < 4; ++y)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = fma2(x[y], S[4 * r + y][e], o[e]);
  }
  const float2 a = unpack2(o[0]), b = unpack2(o[1]), c = unpack2(o[2]), d = unpack2(o[3]);
  return make_float4(a.x + a.y, b.x + b.y, c.x + c.y, d.x + d.y);
}

// The sum over a warp's 8 lane groups: lane 4 g + c ends with column
// 4 c + 2 (g >> 2) + (g >> 1 & 1), as does the lane whose g differs by one.
__device__ __forceinline__ float group_sum(const float4 &f, int g) {
  const bool hi2 = g & 4, hi1 = g & 2;
  const float s0 = __shfl_xor_sync(~0u, hi2 ? f.x : f.z, 16), s1 = __shfl_xor_sync(~0u, hi2 ? f.y : f.w, 16);
  const float a0 = (hi2 ? f.z : f.x) + s0, a1 = (hi2 ? f.w : f.y) + s1;
  const float sum = (hi1 ? a1 : a0) + __shfl_xor_sync(~0u, hi1 ? a0 : a1, 8);
  return sum + __shfl_xor_sync(~0u, sum, 4);
}

template <int DT, int RPL, Mode MODE>
__global__ void __launch_bounds__(32 * kMaxWarps, RPL == 32 ? 2 : 4) state_rows_kernel(const StateParams P, const int blocks_x) {
  using Tile = RowTile<RPL>;
  __shared__ __align__(16) char qs[MODE == kCommit ? 1 : kBlock][MODE == kCommit ? 16 : Tile::kStride];
  __shared__ __align__(16) char ks[MODE == kTree ? 1 : kBlock][MODE == kTree ? 16 : Tile::kStride];
  __shared__ __align__(16) uint16_t vs[MODE == kTree ? 1 : kBlock][kMaxWarps * 16];
  __shared__ float gs[2][kBlock], left[kBlock], from_state[kBlock];
  __shared__ float total, total_more, from_more[kBlock];  // (more: a second factor, 1 unless the first alone would be no number)
  __shared__ float pair[MODE == kChain ? kBlock : 1][kBlock];
  __shared__ float path_w[MODE == kTree ? kBlock : 1][kMaxPath];
  __shared__ int path[MODE == kTree ? kBlock : 1][kMaxPath], path_len[kBlock];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  const int x = blockIdx.x % blocks_x, unit = blockIdx.x / blocks_x;
  const int b = unit / P.heads, h = unit - b * P.heads, hk = h / P.group;
  const int g = lane >> 2, c = lane & 3;
  const int first_col = x * warps * 16, col0 = first_col + warp * 16;
  const bool live = col0 < P.value_dim;

  // ---- the request
  bool ok = true;
  int status = SPEC_STATUS_OK;
  const int slot = state_slot(P.from, b, true, ok);
  const int to_slot = state_slot(P.to, b, false, ok);
  int count = P.counts ? P.counts[b] : P.n_rows;

  const char *qp = P.q + (b * P.qs[0] + hk * P.qs[2]) * 2;
  const char *kp = P.k + (b * P.ks[0] + hk * P.ks[2]) * 2;
  const char *vp = P.v + (b * P.vs[0] + h * P.vs[2]) * 2;
  const float *gp = P.decay + b * P.gs[0] + h * P.gs[2];
  const int dpieces = P.key_dim >> 3, vpieces = min(warps * 16, P.value_dim - first_col) >> 3;
  const int32_t *index = MODE == kCommit && P.index ? P.index + static_cast<int64_t>(b) * P.index_stride : nullptr;
  auto token = [&](int i) -> int64_t {
    if (!index) return i;
    const int r = index[i];  // (an entry that names no row is refused below, or lies past the count)
    return r < 0 || r >= P.n ? 0 : r;
  };
  // Rows [t0, t0 + m): on their way to shared memory.
  auto fetch = [&](int t0, int m, int side) {
    for (int i = tid; i < m * dpieces; i += blockDim.x) {
      const int r = i / dpieces, d = (i - r * dpieces) * 8;
      const int64_t t = token(t0 + r);
      if (MODE != kCommit) copy_piece(&qs[r][d * 2], qp + (t * P.qs[1] + d) * 2, P.vec);
      if (MODE != kTree) copy_piece(&ks[r][d * 2], kp + (t * P.ks[1] + d) * 2, P.vec);
    }
    if (MODE != kTree) {
      for (int i = tid; i < m * vpieces; i += blockDim.x) {
        const int r = i / vpieces, d = (i - r * vpieces) * 8;
        copy_piece(&vs[r][d], vp + (token(t0 + r) * P.vs[1] + first_col + d) * 2, P.vec);
      }
      if (tid < m) gs[side][tid] = gp[token(t0 + tid) * P.gs[1]];
    }
  };
  if (P.key_dim < 8 * RPL) {  // the rows' ends, which no copy fills
    const int pad = 8 * RPL - P.key_dim;
    for (int i = tid; i < kBlock * pad; i += blockDim.x) {
      const int r = i / pad, d = P.key_dim + i % pad;
      if (MODE != kCommit) *reinterpret_cast<uint16_t *>(&qs[r][d * 2]) = 0;
      if (MODE != kTree) *reinterpret_cast<uint16_t *>(&ks[r][d * 2]) = 0;
    }
  }
  fetch(0, P.n > 0 ? min(kBlock, P.n_rows) : 0, 0);  // (whatever the count: the rows exist)

  // its part of the state
  if (!ok) status = SPEC_STATUS_BAD_SLOT;
  pair_t S[RPL / 2][4];
  if (slot >= 0 && ok && live) {
    const float *p = P.from.state + slot * P.from.slot_stride + static_cast<int64_t>(h) * P.key_dim * P.value_dim + col0 + 4 * c;
#pragma unroll
    for (int r = 0; r < RPL; r += 2) {
      const int d = g * RPL + r;  // (key_dim is even)
      float4 u = {}, w = {};
      if (d < P.key_dim) {
        u = *reinterpret_cast<const float4 *>(p + static_cast<int64_t>(d) * P.value_dim);
        w = *reinterpret_cast<const float4 *>(p + static_cast<int64_t>(d + 1) * P.value_dim);
      }
      S[r / 2][0] = pack2(u.x, w.x), S[r / 2][1] = pack2(u.y, w.y), S[r / 2][2] = pack2(u.z, w.z), S[r / 2][3] = pack2(u.w, w.w);
    }
  } else {
#pragma unroll
    for (int r = 0; r < RPL / 2; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[r][e] = 0;
  }
  if (count < 0 || count > P.n_rows) status = SPEC_STATUS_BAD_LENGTH;

  // rows that a request names: all of them are looked at before anything is written
  if (status == SPEC_STATUS_OK && index) {
    bool bad = false;
    for (int i = tid; i < count; i += blockDim.x) bad |= index[i] < 0 || index[i] >= P.n;
    if (__syncthreads_or(bad)) status = SPEC_STATUS_BAD_INDEX;
  }
  const int32_t *parents = MODE == kTree ? P.parents + static_cast<int64_t>(b) * P.n : nullptr;
  if (status == SPEC_STATUS_OK && MODE == kTree) {
    bool bad = false;
    for (int i = tid; i < count; i += blockDim.x) {
      const int p = parents[i];
      bad |= i == 0 ? p != -1 : (p < 0 || p >= i);
    }
    bad = __syncthreads_or(bad);
    if (!bad) {  // every parent lies before its child, so each walk ends
      for (int i = tid; i < count; i += blockDim.x) {
        int depth = 0;
        for (int p = i; p > 0 && depth <= SPEC_MAX_DEPTH; ++depth) p = parents[p];
        bad |= depth > SPEC_MAX_DEPTH;
      }
      bad = __syncthreads_or(bad);
    }
    if (bad) status = SPEC_STATUS_BAD_TREE;
  }
  if (P.status && x == 0 && h == 0 && tid == 0) P.status[b] = status;
  if (status != SPEC_STATUS_OK) count = 0;

#pragma unroll 1
  for (int t0 = 0; t0 < count; t0 += kBlock) {
    const int m = min(kBlock, count - t0), side = t0 / kBlock & 1;
    if (t0 > 0) fetch(t0, m, side);
    cp_async_wait_all();
    __syncthreads();
    bool grows = false;  // some factor of the block's on the state takes two
    if (MODE != kTree) {
      // ---- decays: every warp the sums it needs, the first the factors
      const Log2Sum upto = running<kBlock>(lane < m ? log2_of(gs[side][lane]) : Log2Sum{0}, lane);
      const uint32_t nan = __ballot_sync(~0u, lane < m && gs[side][lane & 15] != gs[side][lane & 15]);
      grows = __any_sync(~0u, lane < m && upto.units > P.most_units);
      const Log2Sum all = of_lane(upto, m - 1);
      if (warp == 0 && lane < m) {
        const Log2Parts p = upto.parts(nan & ((2u << lane) - 1));
        float more;
        from_state[lane] = state_factor(p, MODE == kChain ? P.scale : 1.0f, P.scale_log2, more);
        from_more[lane] = more;
        left[lane] = (all - upto).parts(nan >> lane >> 1).power();
        if (lane == m - 1) total = state_factor(p, 1.0f, 0.0f, more), total_more = more;
      }
      if constexpr (MODE == kChain) {
        // ---- the pairs' weights: a row to a warp, a token before it to 2, 4 or 8 lanes, each of its share of key_dim's pieces
        const int shift = m <= 4 ? 2 : m <= 8 ? 3 : 4, j = lane & ((1 << shift) - 1);
        for (int i = warp; i < m; i += warps) {
          float s = 0.0f;
          if (j <= i) {
#pragma unroll 2
            for (int e = lane >> shift; e < RPL; e += 32 >> shift) {
              pair_t a[4], d[4];
              widen8<DT>(*reinterpret_cast<const uint4 *>(&qs[i][e * 16]), a);
              widen8<DT>(*reinterpret_cast<const uint4 *>(&ks[j][e * 16]), d);
              const float2 u = unpack2(fma2(a[0], d[0], fma2(a[1], d[1], fma2(a[2], d[2], mul2(a[3], d[3])))));
              s += u.x + u.y;
            }
          }
          for (int o = 1 << shift; o < 32; o <<= 1) s += __shfl_xor_sync(~0u, s, o);
          const Log2Sum after = of_lane(upto, i) - of_lane(upto, j);
          // (tokens j + 1 to i)
          const bool lost = nan & ((2u << i) - 1) & ~((2u << j) - 1);
          if (lane >> shift == 0) pair[i][j] = j <= i ? s * after.parts(lost).power() * P.scale : 0.0f;
        }
      }
      __syncthreads();
    } else {
      if (tid < m) {  // the row's path from itself up, and the decays that lie before each node of it
        int len = 0;
        Log2Sum sum{0};
        bool nan = false;
        for (int p = t0 + tid; p >= 0; p = parents[p]) {
          path[tid][len] = p;
          path_w[tid][len] = sum.parts(nan).power();
          ++len;
          const float x = gp[p * P.gs[1]];
          sum += log2_of(x), nan |= x != x;
        }
        path_len[tid] = len;
        from_state[tid] = state_factor(sum.parts(nan), P.scale, P.scale_log2, from_more[tid]);
      }
      __syncthreads();
      for (int i = 0; i < m; ++i) {
        for (int p = warp; p < path_len[i]; p += warps) {
          const char *row = kp + static_cast<int64_t>(path[i][p]) * P.ks[1] * 2;
          float s = 0.0f;
          for (int d = lane * 2; d < P.key_dim; d += 64) {
            const uint16_t *u = reinterpret_cast<const uint16_t *>(row) + d;
            const float2 f = widen2<DT>(*reinterpret_cast<const uint32_t *>(&qs[i][d * 2]));
            s = fmaf(f.x, widen<DT>(u[0]), fmaf(f.y, widen<DT>(u[1]), s));
          }
          s = warp_add(s);
          if (lane == 0) path_w[i][p] = s * path_w[i][p] * P.scale;
        }
      }
      __syncthreads();
    }

    // ---- outputs
    if (MODE != kCommit && live) {
      const int col = 4 * c + 2 * (g >> 2) + (g >> 1 & 1);
      uint16_t *o16 = reinterpret_cast<uint16_t *>(P.out) + b * P.os[0] + static_cast<int64_t>(t0) * P.os[1] + h * P.os[2] + col0 + col;
      if constexpr (MODE == kChain) {
        // the lane's columns of tokens g and g + 8 (zeros where there are none: their weights are, and no row sees them)
        float4 v0 = {}, v1 = {};
        auto load_v = [&](int j) -> float4 {
          const uint2 w = *reinterpret_cast<const uint2 *>(&vs[j][warp * 16 + 4 * c]);
          const float2 y = widen2<DT>(w.x), z = widen2<DT>(w.y);
          return make_float4(y.x, y.y, z.x, z.y);
        };
        if (g < m) v0 = load_v(g);
        if (g + 8 < m) v1 = load_v(g + 8);
        auto row = [&](int i, auto grown) -> float {
          float4 s = row_product<DT, RPL>(qs[i], g, S);
          if constexpr (decltype(grown)::value) s = make_float4(s.x * from_more[i], s.y * from_more[i], s.z * from_more[i], s.w * from_more[i]);
          const float e = from_state[i];
          float4 f = make_float4(s.x * e, s.y * e, s.z * e, s.w * e);
          if (g <= i) {
            const float w = pair[i][g];
            f = make_float4(fmaf(w, v0.x, f.x), fmaf(w, v0.y, f.y), fmaf(w, v0.z, f.z), fmaf(w, v0.w, f.w));
          }
          if (g + 8 <= i) {
            const float w = pair[i][g + 8];
            f = make_float4(fmaf(w, v1.x, f.x), fmaf(w, v1.y, f.y), fmaf(w, v1.z, f.z), fmaf(w, v1.w, f.w));
          }
          return group_sum(f, g);
        };
        int i = 0;
        if (grows) [[unlikely]] {
#pragma unroll 1
          for (; i < m; ++i, o16 += P.os[1]) {
            const float a = row(i, std::true_type{});
            if (!(g & 1)) *o16 = narrow<DT>(a);
          }
        }
#pragma unroll 1
        for (; i + 2 <= m; i += 2) {  // two rows side by side: the one's reduction behind the other's products
          const float a = row(i, std::false_type{}), d = row(i + 1, std::false_type{});
          o16[(g & 1) * P.os[1]] = narrow<DT>(g & 1 ? d : a);
          o16 += 2 * P.os[1];
        }
        if (i < m) {
          const float a = row(i, std::false_type{});
          if (!(g & 1)) *o16 = narrow<DT>(a);
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < m; ++i) {
          float sum = group_sum(row_product<DT, RPL>(qs[i], g, S), g) * from_more[i] * from_state[i], terms = 0.0f;
          for (int p = g & 1; p < path_len[i]; p += 2) {
            const uint16_t v = *reinterpret_cast<const uint16_t *>(vp + (static_cast<int64_t>(path[i][p]) * P.vs[1] + col0 + col) * 2);
            terms = fmaf(path_w[i][p], widen<DT>(v), terms);
          }
          sum += terms + __shfl_xor_sync(~0u, terms, 4);
          if (!(g & 1)) *o16 = narrow<DT>(sum);
          o16 += P.os[1];
        }
      }
    }

    // ---- the state behind the block
    if (MODE != kTree && live && (P.to.state || t0 + kBlock < count)) {
      if (grows) [[unlikely]] {
        const pair_t more = pack2(total_more, total_more);
#pragma unroll
        for (int r = 0; r < RPL / 2; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[r][e] = mul2(S[r][e], more);
      }
      const pair_t f2 = pack2(total, total);
#pragma unroll
      for (int r = 0; r < RPL / 2; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[r][e] = mul2(S[r][e], f2);
#pragma unroll 1
      for (int j = 0; j < m; ++j) {
        const uint2 v = *reinterpret_cast<const uint2 *>(&vs[j][warp * 16 + 4 * c]);
        const float2 y0 = widen2<DT>(v.x), y1 = widen2<DT>(v.y);
        const float w = left[j];
        const pair_t v2[4] = {pack2(y0.x * w, y0.x * w), pack2(y0.y * w, y0.y * w), pack2(y1.x * w, y1.x * w), pack2(y1.y * w, y1.y * w)};
#pragma unroll
        for (int r = 0; r < RPL / 8; ++r) {
          pair_t k[4];
          widen8<DT>(*reinterpret_cast<const uint4 *>(&ks[j][(g * RPL + 8 * r) * 2]), k);
#pragma unroll
          for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[4 * r + y][e] = fma2(k[y], v2[e], S[4 * r + y][e]);
        }
      }
    }
    if (t0 + kBlock < count) __syncthreads();  // before the next block's rows
  }
  cp_async_wait_all();

  if (MODE != kCommit) {  // rows past the count
    const int cols = min(warps * 16, P.value_dim - first_col);
    uint16_t *o = reinterpret_cast<uint16_t *>(P.out) + b * P.os[0] + h * P.os[2] + first_col;
    if (P.vec) {
      const int pieces = cols >> 3;
      for (int64_t i = tid; i < static_cast<int64_t>(P.n - count) * pieces; i += blockDim.x)
        *reinterpret_cast<uint4 *>(o + (count + i / pieces) * P.os[1] + i % pieces * 8) = make_uint4(0, 0, 0, 0);
    } else {
      for (int64_t i = tid; i < static_cast<int64_t>(P.n - count) * cols; i += blockDim.x) o[(count + i / cols) * P.os[1] + i % cols] = 0;
    }
  }
  if (MODE != kTree && P.to.state && status == SPEC_STATUS_OK && live) {
    float *p = P.to.state + to_slot * P.to.slot_stride + static_cast<int64_t>(h) * P.key_dim * P.value_dim + col0 + 4 * c;
#pragma unroll
    for (int r = 0; r < RPL; r += 2) {
      const int d = g * RPL + r;
      if (d < P.key_dim) {
        const float2 s0 = unpack2(S[r / 2][0]), s1 = unpack2(S[r / 2][1]), s2 = unpack2(S[r / 2][2]), s3 = unpack2(S[r / 2][3]);
        *reinterpret_cast<float4 *>(p + static_cast<int64_t>(d) * P.value_dim) = make_float4(s0.x, s1.x, s2.x, s3.x);
        *reinterpret_cast<float4 *>(p + static_cast<int64_t>(d + 1) * P.value_dim) = make_float4(s0.y, s1.y, s2.y, s3.y);
      }
    }
  }
}

template <int DT, int RPL>
cudaError_t launch_rows(const StateParams &P, cudaStream_t st) {
  const int groups = P.value_dim / 16;
  const int64_t units = static_cast<int64_t>(P.B) * P.heads;
  // four warps share a block's rows, fewer when that leaves SMs without a CTA (eight: 64 requests' single tokens 92 us, not 81)
  int warps = kMaxWarps;
  while (warps > 2 && units * ((groups + warps - 1) / warps) < device_sm_count()) warps /= 2;
  const int x = (groups + warps - 1) / warps;
  const dim3 grid(static_cast<unsigned>(units * x)), block(32 * warps);
  if (P.parents) return trace_launch("state_tree_rows", st, [&] { state_rows_kernel<DT, RPL, kTree><<<grid, block, 0, st>>>(P, x); });
  const bool again = !state_overlaps(P);
  if (P.q) return trace_launch("state_rows", st, [&] { state_rows_kernel<DT, RPL, kChain><<<grid, block, 0, st>>>(P, x); }, again);
  return trace_launch("state_commit", st, [&] { state_rows_kernel<DT, RPL, kCommit><<<grid, block, 0, st>>>(P, x); }, again);
}

template <int DT>
cudaError_t launch_dim(const StateParams &P, cudaStream_t st) {
  return P.key_dim <= 64 ? launch_rows<DT, 8>(P, st) : P.key_dim <= 128 ? launch_rows<DT, 16>(P, st) : launch_rows<DT, 32>(P, st);
}

}  // namespace

cudaError_t launch_state_rows(const StateParams &P, cudaStream_t st) {
  return P.dtype == SPEC_DTYPE_BF16 ? launch_dim<SPEC_DTYPE_BF16>(P, st) : launch_dim<SPEC_DTYPE_F16>(P, st);
}

}  // namespace sv
