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
// token by token: three), and decays are sums of the g's between two tokens,
// never a difference of running sums: -inf and long blocks lose nothing.
// A tree's row takes its ancestors' terms instead, one after another along its
// path, with k and v from memory.
#include <algorithm>

#include "launch.h"
#include "state.cuh"

namespace sv {
namespace {

constexpr int kBlock = 16;  // tokens to a block
constexpr int kMaxWarps = 8;
constexpr int kMaxPath = SPEC_MAX_DEPTH + 1;

enum Mode { kCommit, kChain, kTree };

__device__ __forceinline__ float warp_add(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// Rows of q or k in shared memory: RPL values of each of the 8 lane groups,
// padded by 4 (a warp's reads then meet no bank twice).
template <int RPL>
struct RowTile {
  static constexpr int kStride = 8 * (RPL + 4);
  static __device__ __forceinline__ int at(int d) { return d / RPL * (RPL + 4) + d % RPL; }
};

// Row `row` of a key head (or, COLS, columns of a state head's v) as fp32.
template <int DT>
__device__ __forceinline__ void load_piece(const char *p, bool vec, float *x) {  // 8 values
  uint32_t w[4];
  if (vec) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else {
    const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = h[2 * e] | static_cast<uint32_t>(h[2 * e + 1]) << 16;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = widen2<DT>(w[e]);
    x[2 * e] = f.x, x[2 * e + 1] = f.y;
  }
}

// q_i . k_j, a warp: both rows in shared memory.
template <int RPL>
__device__ __forceinline__ float dot_rows(const float *a, const float *b, int lane) {
  float sum = 0.0f;
#pragma unroll
  for (int e = 0; e < (RPL * 8 + 127) / 128; ++e) {
    const int d = (e * 32 + lane) * 4;
    if (RPL >= 16 || d < RPL * 8) {
      const float4 x = *reinterpret_cast<const float4 *>(a + RowTile<RPL>::at(d));
      const float4 y = *reinterpret_cast<const float4 *>(b + RowTile<RPL>::at(d));
      sum = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, sum))));
    }
  }
  return warp_add(sum);
}

template <int DT, int RPL, Mode MODE>
__global__ void __launch_bounds__(32 * kMaxWarps) state_rows_kernel(const StateParams P, const int blocks_x) {
  using Tile = RowTile<RPL>;
  __shared__ __align__(16) float qs[MODE == kCommit ? 1 : kBlock][Tile::kStride];
  __shared__ __align__(16) float ks[MODE == kTree ? 1 : kBlock][Tile::kStride];
  __shared__ __align__(16) float vs[MODE == kTree ? 1 : kBlock][kMaxWarps * 16];
  __shared__ float gs[kBlock], left[kBlock], from_state[kBlock];
  __shared__ float total;
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
  if (!ok) status = SPEC_STATUS_BAD_SLOT;
  int count = P.counts ? P.counts[b] : P.n_rows;
  if (count < 0 || count > P.n_rows) status = SPEC_STATUS_BAD_LENGTH;

  // its part of the state, on the way while the rows are fetched
  pair_t S[RPL / 2][4];
  if (slot >= 0 && status == SPEC_STATUS_OK && live) {
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

  // rows that a request names: all of them are looked at before anything is written
  if (status == SPEC_STATUS_OK && MODE == kCommit && P.index) {
    bool bad = false;
    for (int i = tid; i < count; i += blockDim.x) {
      const int r = P.index[static_cast<int64_t>(b) * P.index_stride + i];
      bad |= r < 0 || r >= P.n;
    }
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

  const char *qp = P.q + (b * P.qs[0] + hk * P.qs[2]) * 2;
  const char *kp = P.k + (b * P.ks[0] + hk * P.ks[2]) * 2;
  const char *vp = P.v + (b * P.vs[0] + h * P.vs[2]) * 2;
  const float *gp = P.decay + b * P.gs[0] + h * P.gs[2];
  if (P.key_dim < 8 * RPL) {  // the rows' ends, which no load fills
    const int pad = 8 * RPL - P.key_dim;
    for (int i = tid; i < kBlock * pad; i += blockDim.x) {
      const int r = i / pad, d = P.key_dim + i % pad;
      if (MODE != kCommit) qs[r][Tile::at(d)] = 0.0f;
      if (MODE != kTree) ks[r][Tile::at(d)] = 0.0f;
    }
  }

  const int dpieces = P.key_dim >> 3, vpieces = min(warps * 16, P.value_dim - first_col) >> 3;
#pragma unroll 1
  for (int t0 = 0; t0 < count; t0 += kBlock) {
    const int m = min(kBlock, count - t0);
    auto token = [&](int i) -> int64_t {
      return MODE == kCommit && P.index ? P.index[static_cast<int64_t>(b) * P.index_stride + t0 + i] : t0 + i;
    };
    // ---- the block's rows
    for (int i = tid; i < m * dpieces; i += blockDim.x) {
      const int r = i / dpieces, d = (i - r * dpieces) * 8;
      const int64_t t = token(r);
      float f[8];
      if (MODE != kCommit) {
        load_piece<DT>(qp + (t * P.qs[1] + d) * 2, P.vec, f);
        *reinterpret_cast<float4 *>(&qs[r][Tile::at(d)]) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4 *>(&qs[r][Tile::at(d + 4)]) = make_float4(f[4], f[5], f[6], f[7]);
      }
      if (MODE != kTree) {
        load_piece<DT>(kp + (t * P.ks[1] + d) * 2, P.vec, f);
        *reinterpret_cast<float4 *>(&ks[r][Tile::at(d)]) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4 *>(&ks[r][Tile::at(d + 4)]) = make_float4(f[4], f[5], f[6], f[7]);
      }
    }
    if (MODE != kTree) {
      for (int i = tid; i < m * vpieces; i += blockDim.x) {
        const int r = i / vpieces, d = (i - r * vpieces) * 8;
        float f[8];
        load_piece<DT>(vp + (token(r) * P.vs[1] + first_col + d) * 2, P.vec, f);
        *reinterpret_cast<float4 *>(&vs[r][d]) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4 *>(&vs[r][d + 4]) = make_float4(f[4], f[5], f[6], f[7]);
      }
      if (tid < m) gs[tid] = gp[token(tid) * P.gs[1]];
      __syncthreads();
      if (tid < m) {  // e^ of the sums up to and from a token on
        float to = 0.0f, past = 0.0f;
        for (int j = 0; j <= tid; ++j) to += gs[j];
        for (int j = tid + 1; j < m; ++j) past += gs[j];
        from_state[tid] = expf(to) * (MODE == kChain ? P.scale : 1.0f);
        left[tid] = expf(past);
        if (tid == m - 1) total = expf(to);
      }
      if constexpr (MODE == kChain) {
        int i = 0, at = 0;  // pair number `at` is (i, 0)
        for (int p = warp; p < m * (m + 1) / 2; p += warps) {
          while (p > at + i) at += i + 1, ++i;
          const int j = p - at;
          const float s = dot_rows<RPL>(qs[i], ks[j], lane);
          const float between = warp_add(lane > j && lane <= i ? gs[lane] : 0.0f);
          if (lane == 0) pair[i][j] = s * expf(between) * P.scale;
        }
      }
      __syncthreads();
    } else {
      if (tid < m) {  // the row's path from itself up, and the decays that lie before each node of it
        int len = 0;
        float sum = 0.0f;
        for (int p = t0 + tid; p >= 0; p = parents[p]) {
          path[tid][len] = p;
          path_w[tid][len] = sum;
          ++len;
          sum += gp[p * P.gs[1]];
        }
        path_len[tid] = len;
        from_state[tid] = expf(sum) * P.scale;
      }
      __syncthreads();
      for (int i = 0; i < m; ++i) {
        for (int p = warp; p < path_len[i]; p += warps) {
          const char *row = kp + static_cast<int64_t>(path[i][p]) * P.ks[1] * 2;
          float s = 0.0f;
          for (int d = lane * 2; d < P.key_dim; d += 64) {
            const uint16_t *u = reinterpret_cast<const uint16_t *>(row) + d;
            const int at = Tile::at(d);
            s = fmaf(qs[i][at], widen<DT>(u[0]), fmaf(qs[i][at + 1], widen<DT>(u[1]), s));
          }
          s = warp_add(s);
          if (lane == 0) path_w[i][p] = s * expf(path_w[i][p]) * P.scale;
        }
      }
      __syncthreads();
    }

    // ---- outputs
    if (MODE != kCommit && live) {
      const int col = 4 * c + 2 * (g >> 2) + (g >> 1 & 1);  // the column that this lane ends up with, and the lane whose g differs by one
#pragma unroll 1
      for (int i = 0; i < m; ++i) {
        pair_t o[4] = {0, 0, 0, 0};
        const ulonglong2 *q = reinterpret_cast<const ulonglong2 *>(&qs[i][g * (RPL + 4)]);
#pragma unroll
        for (int r = 0; r < RPL / 4; ++r) {
          const ulonglong2 u = q[r];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = fma2(u.y, S[2 * r + 1][e], fma2(u.x, S[2 * r][e], o[e]));
        }
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 w = unpack2(o[e]);
          f[e] = w.x + w.y;
        }
        const bool hi2 = g & 4, hi1 = g & 2;
        const float s0 = __shfl_xor_sync(~0u, hi2 ? f[0] : f[2], 16), s1 = __shfl_xor_sync(~0u, hi2 ? f[1] : f[3], 16);
        const float a0 = (hi2 ? f[2] : f[0]) + s0, a1 = (hi2 ? f[3] : f[1]) + s1;
        float sum = (hi1 ? a1 : a0) + __shfl_xor_sync(~0u, hi1 ? a0 : a1, 8);
        sum *= from_state[i];
        if constexpr (MODE == kChain) {
          for (int j = g & 1; j <= i; j += 2) sum = fmaf(pair[i][j], vs[j][warp * 16 + col], sum);
        } else {
          for (int p = g & 1; p < path_len[i]; p += 2) {
            const uint16_t v = *reinterpret_cast<const uint16_t *>(vp + (static_cast<int64_t>(path[i][p]) * P.vs[1] + col0 + col) * 2);
            sum = fmaf(path_w[i][p], widen<DT>(v), sum);
          }
        }
        sum += __shfl_xor_sync(~0u, sum, 4);
        if (!(g & 1)) {
          uint16_t *o16 = reinterpret_cast<uint16_t *>(P.out) + b * P.os[0] + static_cast<int64_t>(t0 + i) * P.os[1] + h * P.os[2] + col0 + col;
          *o16 = narrow<DT>(sum);
        }
      }
    }

    // ---- the state behind the block
    if (MODE != kTree && live && (P.to.state || t0 + kBlock < count)) {
      const pair_t f2 = pack2(total, total);
#pragma unroll
      for (int r = 0; r < RPL / 2; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[r][e] = mul2(S[r][e], f2);
#pragma unroll 1
      for (int j = 0; j < m; ++j) {
        const float4 v = *reinterpret_cast<const float4 *>(&vs[j][warp * 16 + 4 * c]);
        const float w = left[j];
        const float f[4] = {v.x * w, v.y * w, v.z * w, v.w * w};
        const ulonglong2 *k = reinterpret_cast<const ulonglong2 *>(&ks[j][g * (RPL + 4)]);
        pair_t v2[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v2[e] = pack2(f[e], f[e]);
#pragma unroll
        for (int r = 0; r < RPL / 4; ++r) {
          const ulonglong2 u = k[r];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            S[2 * r][e] = fma2(u.x, v2[e], S[2 * r][e]);
            S[2 * r + 1][e] = fma2(u.y, v2[e], S[2 * r + 1][e]);
          }
        }
      }
    }
    __syncthreads();  // before the next block's rows
  }

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
  // eight warps share a block's rows; fewer when that leaves SMs without a CTA
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
