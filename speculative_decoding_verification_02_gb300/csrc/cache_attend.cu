// spec_cache_attend: attention of the drafted rows over the 8-bit cache.
//
//   x_j = cap tanh(scale q.k_j / cap) over the positions that the row sees
//   out = sum_j exp(x_j - m) v_j / sum_j exp(x_j - m),  lse = m + log sum_j exp(x_j - m)
//
// in one pass with the running maximum m and sum.  Heads of 64 and 128 run on
// the tensor cores (cache_attend_tile.cuh); other widths, and a few rows over
// many heads or a short context, on the scalar units.
#include <algorithm>
#include <cooperative_groups.h>

#include "cache.cuh"
#include "common.cuh"
#include "launch.h"
#include "ring.h"

namespace sv {
namespace {

constexpr int kRowThreads = 128;  // (512 units of 1,500 positions: 25.2 us, all resident at once; 256 threads 27.1 us)
constexpr int kSpanPages = 256;  // pages whose places are held in shared memory at a time
constexpr int kAtOnce = 4;       // positions that a group of lanes has in flight

// Up to ROWS rows of a kv head to a cluster of CTAs, each with a share of the
// positions.  LANES lanes score a position, 16 bytes of its key each, and add
// 16 bytes of its value; every such group of lanes keeps its own running
// maximum, sum and result, joined in the warp, the CTA and the cluster at the
// end.  Keys and values are read once and never staged, and one launch does
// all, without a workspace; the arithmetic is scalar, so its time goes with the
// rows.  32 requests of one row, 16 heads of 64, 375 to 1,501 positions, capped:
// 24 us, 2.5 TB/s (the tensor-core kernel: 50 us); one request of four rows,
// 8 heads of 128, 2,000 positions: 13.3 us (16 us).
template <int DT, int LANES, int ROWS, bool CAP>
__global__ void __launch_bounds__(kRowThreads) cache_attend_rows_kernel(const CacheAttendParams P, int chunks) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ int64_t s_at[kSpanPages];
  __shared__ float2 s_scale[kSpanPages];
  __shared__ float s_acc[kRowThreads / 32][ROWS][LANES * 16];
  __shared__ float2 s_ml[kRowThreads / 32][ROWS];
  __shared__ float s_all[ROWS][LANES * 16];
  __shared__ float2 s_all_ml[ROWS];
  constexpr int kGroups = 32 / LANES, kAll = kRowThreads / LANES;
  const int splits = static_cast<int>(cluster.num_blocks()), split = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, part = lane % LANES, group = tid / LANES;
  int x = blockIdx.x / splits;
  const int chunk = x % chunks;
  x /= chunks;
  const int head = x % P.c.kv_heads, b = x / P.c.kv_heads, D = P.c.head_dim, shift = P.c.page_shift;
  const bool used = part * 16 < D;

  int base = P.cache_len[b], n = P.n_query ? P.n_query[b] : P.N;
  int st = SPEC_STATUS_OK;
  if (base < 0 || n < 0 || n > P.N || base + static_cast<int64_t>(n) > capacity(P.c)) st = SPEC_STATUS_BAD_LENGTH, base = n = 0;
  // a bad page anywhere takes the request out, for every row alike
  int bad = 0;
  for (int i = tid; static_cast<int64_t>(i) << shift < base + n; i += kRowThreads) bad |= page_at(P.c, b, i) < 0;
  if (__syncthreads_or(bad)) st = SPEC_STATUS_BAD_PAGE;
  if (P.status && head == 0 && chunk == 0 && split == 0 && tid == 0) P.status[b] = st;
  if (st != SPEC_STATUS_OK) base = n = 0;

  const int row0 = chunk * ROWS, rows = min(ROWS, n * P.group - row0);
  int token[ROWS];
  float q[ROWS][16];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    const int row = row0 + k;
    token[k] = row / P.group;
#pragma unroll
    for (int e = 0; e < 16; ++e) q[k][e] = 0.0f;
    if (k < rows && used) {
      const char *src = P.q + (b * P.qs[0] + token[k] * P.qs[1] + (head * P.group + row % P.group) * P.qs[2]) * 2;
#pragma unroll
      for (int e = 0; e < 16; ++e) q[k][e] = row_value<DT>(src, part * 16 + e) * (P.scale * kLog2e);
    }
  }
  // positions of this CTA: whole steps of all its groups
  const int T = rows > 0 ? (P.mask ? base + n : base + token[0] + 1 + (rows - 1 + row0 % P.group) / P.group) : 0;
  const int share = ((T + splits - 1) / splits + kAll - 1) / kAll * kAll;
  const int from = min(T, split * share), to = min(T, from + share);
  const uint8_t *mask = P.mask ? P.mask + static_cast<int64_t>(b) * P.N * P.N : nullptr;

  const float cap2 = P.softcap * kLog2e, in_cap = CAP ? 1.0f / cap2 : 0.0f;
  float m[ROWS], sum[ROWS], acc[ROWS][16];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    m[k] = -INFINITY, sum[k] = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[k][e] = 0.0f;
  }
  for (int s0 = from >> shift << shift, s1; s0 < to; s0 = s1) {
    s1 = next_span(s0, to, kSpanPages << shift);
    __syncthreads();
    for (int i = tid; i << shift < s1 - s0; i += kRowThreads) {
      const int page = page_at(P.c, b, (s0 >> shift) + i);
      const int64_t at = page * P.c.scale_stride + head;
      s_at[i] = block_offset(P.c, page, head);
      s_scale[i] = make_float2(P.c.k_scale[at], P.c.v_scale[at]);
    }
    __syncthreads();
    // (every lane of a warp takes as many steps: the shuffles below need them all)
    for (int t0 = max(from, s0); t0 < s1; t0 += kAll * kAtOnce) {
      uint4 kk[kAtOnce], vv[kAtOnce];
      float2 sc[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int t = t0 + u * kAll + group;
        kk[u] = vv[u] = make_uint4(0, 0, 0, 0);
        sc[u] = make_float2(0.0f, 0.0f);
        if (t < s1) {
          const int i = (t - s0) >> shift;
          const int64_t at = s_at[i] + (t & ((1 << shift) - 1)) * D + part * 16;
          sc[u] = s_scale[i];
          if (used) {
            kk[u] = ld_stream16(P.c.k + at);
            vv[u] = ld_stream16(P.c.v + at);
          }
        }
      }
      float score[kAtOnce][ROWS];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        float dot[ROWS] = {};
        const uint32_t w[4] = {kk[u].x, kk[u].y, kk[u].z, kk[u].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 a = e4m3x2_to_float2(w[e] & 0xffff), c = e4m3x2_to_float2(w[e] >> 16);
#pragma unroll
          for (int k = 0; k < ROWS; ++k)
            dot[k] = fmaf(q[k][4 * e], a.x, fmaf(q[k][4 * e + 1], a.y, fmaf(q[k][4 * e + 2], c.x, fmaf(q[k][4 * e + 3], c.y, dot[k]))));
        }
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1)
#pragma unroll
          for (int k = 0; k < ROWS; ++k) dot[k] += __shfl_xor_sync(~0u, dot[k], o);
        const int t = t0 + u * kAll + group, j = t - base;
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
          const float y = dot[k] * sc[u].x;
          if (CAP) {  // capped, and masked, when all are there
            score[u][k] = y;
            continue;
          }
          const bool sees = t < s1 && k < rows && (j < 0 || (mask ? mask[static_cast<int64_t>(token[k]) * P.N + j] != 0 : j <= token[k]));
          score[u][k] = sees ? y : -INFINITY;
        }
        if (!CAP && j >= 0) [[unlikely]] {  // a value that no row may look at, or that is no number, has no part in the others
          bool any = false;
#pragma unroll
          for (int k = 0; k < ROWS; ++k) any |= score[u][k] != -INFINITY;
          if (!any) vv[u] = make_uint4(0, 0, 0, 0);
        }
      }
      if (CAP) {
        cap_scores<kAtOnce * ROWS>(&score[0][0], in_cap, cap2);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const int t = t0 + u * kAll + group, j = t - base;
          bool any = false;
#pragma unroll
          for (int k = 0; k < ROWS; ++k) {
            const bool sees = t < s1 && k < rows && (j < 0 || (mask ? mask[static_cast<int64_t>(token[k]) * P.N + j] != 0 : j <= token[k]));
            if (!sees) score[u][k] = -INFINITY;
            any |= sees;
          }
          if (j >= 0 && !any) vv[u] = make_uint4(0, 0, 0, 0);
        }
      }
      bool moves = false;
      float next[ROWS];
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        next[k] = m[k];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) next[k] = fmaxf(next[k], score[u][k]);
        moves |= next[k] > m[k];
      }
      if (__any_sync(~0u, moves)) {
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
          const float keep = next[k] == -INFINITY ? 0.0f : ex2(m[k] - next[k]);
          m[k] = next[k];
          sum[k] *= keep;
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[k][e] *= keep;
        }
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        float p[ROWS];
        bool part_of[ROWS];
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
          part_of[k] = score[u][k] != -INFINITY;
          p[k] = part_of[k] ? ex2(score[u][k] - m[k]) : 0.0f;
          sum[k] += p[k];
          p[k] *= sc[u].y;
        }
        const bool plain = t0 + u * kAll + group < base;  // every row sees it
        const uint32_t w[4] = {vv[u].x, vv[u].y, vv[u].z, vv[u].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 a = e4m3x2_to_float2(w[e] & 0xffff), c = e4m3x2_to_float2(w[e] >> 16);
#pragma unroll
          for (int k = 0; k < ROWS; ++k) {
            if (ROWS > 1 && !plain && !part_of[k]) continue;
            acc[k][4 * e] = fmaf(p[k], a.x, acc[k][4 * e]);
            acc[k][4 * e + 1] = fmaf(p[k], a.y, acc[k][4 * e + 1]);
            acc[k][4 * e + 2] = fmaf(p[k], c.x, acc[k][4 * e + 2]);
            acc[k][4 * e + 3] = fmaf(p[k], c.y, acc[k][4 * e + 3]);
          }
        }
      }
    }
  }
  // the groups of a warp, then its sums to shared memory
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
#pragma unroll
    for (int o = LANES; o < 32; o <<= 1) {
      const float other = __shfl_xor_sync(~0u, m[k], o), both = fmaxf(m[k], other), ref = both == -INFINITY ? 0.0f : both;
      const float keep = ex2(m[k] - ref);
      m[k] = both;
      sum[k] *= keep;
      sum[k] += __shfl_xor_sync(~0u, sum[k], o);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        acc[k][e] *= keep;
        acc[k][e] += __shfl_xor_sync(~0u, acc[k][e], o);
      }
    }
    if (lane < LANES) {
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<float4 *>(&s_acc[warp][k][part * 16 + e]) = make_float4(acc[k][e], acc[k][e + 1], acc[k][e + 2], acc[k][e + 3]);
      if (lane == 0) s_ml[warp][k] = make_float2(m[k], sum[k]);
    }
  }
  __syncthreads();
  // the CTA's warps, a column to a thread
  const int all = ROWS * D;
  auto put = [&](int k, int d, float top, float l, float o) {
    const int row = row0 + k, i_tok = row / P.group, h = head * P.group + row % P.group;
    if (row >= P.N * P.group) return;
    put_value<DT>(P.out + (b * P.os[0] + i_tok * P.os[1] + h * P.os[2]) * 2, d, l == 0.0f ? 0.0f : __fdividef(o, l));
    if (d == 0 && P.lse) P.lse[(static_cast<int64_t>(b) * P.N + i_tok) * P.Hq + h] = l == 0.0f ? -INFINITY : (top + __log2f(l)) * kLn2;
  };
  for (int i = tid; i < all; i += kRowThreads) {
    const int k = i / D, d = i - k * D;
    float top = -INFINITY, l = 0.0f, o = 0.0f;
#pragma unroll
    for (int w = 0; w < kRowThreads / 32; ++w) top = fmaxf(top, s_ml[w][k].x);
    const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int w = 0; w < kRowThreads / 32; ++w) {
      const float weight = ex2(s_ml[w][k].x - ref);
      l = fmaf(s_ml[w][k].y, weight, l);
      o = fmaf(s_acc[w][k][d], weight, o);
    }
    if (splits == 1) {
      put(k, d, top, l, o);
    } else {
      s_all[k][d] = o;
      if (d == 0) s_all_ml[k] = make_float2(top, l);
    }
  }
  if (splits == 1) return;
  // the cluster's CTAs, each joining a share of the columns
  cluster.sync();
  for (int i = split * kRowThreads + tid; i < all; i += splits * kRowThreads) {
    const int k = i / D, d = i - k * D;
    float2 ml[8];
    float o[8], top = -INFINITY, l = 0.0f, sum_o = 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      ml[c] = make_float2(-INFINITY, 0.0f), o[c] = 0.0f;
      if (c < splits) {
        ml[c] = *cluster.map_shared_rank(&s_all_ml[k], c);
        o[c] = *cluster.map_shared_rank(&s_all[k][d], c);
      }
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) top = fmaxf(top, ml[c].x);
    const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float weight = ex2(ml[c].x - ref);
      l = fmaf(ml[c].y, weight, l);
      sum_o = fmaf(o[c], weight, sum_o);
    }
    put(k, d, top, l, sum_o);
  }
  cluster.sync();  // no CTA leaves while its sums are read
}

// ------------------------------------------------------------------- host

// Chunks of rows of a kv head: one at least, which sets the status.
int64_t row_chunks(const CacheAttendParams &P, int rows_to_a_chunk) {
  return std::max<int64_t>(1, (static_cast<int64_t>(P.N) * P.group + rows_to_a_chunk - 1) / rows_to_a_chunk);
}

int64_t row_units(const CacheAttendParams &P, int rows_to_a_unit) {
  return static_cast<int64_t>(P.B) * P.c.kv_heads * row_chunks(P, rows_to_a_unit);
}

int rows_of(const CacheAttendParams &P) {
  const int64_t rows = static_cast<int64_t>(P.N) * P.group;
  return rows <= 1 ? 1 : rows <= 2 ? 2 : 4;
}

// CTAs that are on the GPU at once: their registers allow 2 of four rows to an
// SM, 3 of two, 4 of one.
int row_ctas(const CacheAttendParams &P) {
  const int rows = rows_of(P);
  return device_sm_count() * (rows == 4 ? 2 : rows == 2 ? 3 : 4);
}

// CTAs to a unit: as many as are on the GPU at once, eight at most, and no share
// of the positions below 64.  (64 units of four rows, 64 wide, 600 positions:
// 11.5 us with 256 CTAs, 17.8 with 512, which take two turns.)
int row_splits(const CacheAttendParams &P) {
  const int64_t units = row_units(P, rows_of(P)), most = capacity_of(P.c);
  int n = 1;
  while (n < 8 && units * 2 * n <= row_ctas(P) && most / (2 * n) >= 64) n *= 2;
  return n;
}

template <int DT, int LANES, int ROWS>
cudaError_t launch_rows(const CacheAttendParams &P, cudaStream_t st) {
  const int splits = row_splits(P);
  const int chunks = static_cast<int>(row_chunks(P, ROWS));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(row_units(P, ROWS) * splits));
  cfg.blockDim = dim3(kRowThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = splits;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kern = P.softcap > 0.0f ? cache_attend_rows_kernel<DT, LANES, ROWS, true> : cache_attend_rows_kernel<DT, LANES, ROWS, false>;
  return trace_launch_ex("cache_attend_rows", st, [&] { return cudaLaunchKernelEx(&cfg, kern, P, chunks); });
}

template <int DT, int LANES>
cudaError_t launch_rows(const CacheAttendParams &P, cudaStream_t st) {
  const int rows = rows_of(P);
  return rows == 1 ? launch_rows<DT, LANES, 1>(P, st) : rows == 2 ? launch_rows<DT, LANES, 2>(P, st) : launch_rows<DT, LANES, 4>(P, st);
}

template <int DT>
cudaError_t launch_rows(const CacheAttendParams &P, cudaStream_t st) {
  const int D = P.c.head_dim;
  return D <= 64 ? launch_rows<DT, 4>(P, st) : D <= 128 ? launch_rows<DT, 8>(P, st) : launch_rows<DT, 16>(P, st);
}

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
  const int64_t tiles = (capacity_of(P.c) / kTilePositions + 1 + kTileUnitCost) * row_tiles * P.c.kv_heads;
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
  if (P.N == 0 || (P.c.head_dim != 64 && P.c.head_dim != 128) || static_cast<int64_t>(P.N) * P.group * P.group >= (1LL << 32) ||
      requests_at_once(P) <= 0)
    return false;
  // The tensor cores work on 128 rows whatever there are, and their kernel starts and joins its units slowly; the scalar kernel's
  // time goes with the rows and the components.  Measured (scalar against tensor cores, us): one row, 64 wide, 32 requests of 16
  // heads and 1,500 positions 26 and 38, 64 of 8 and 4,000 54 and 58; 128 wide, 1,500: 42 and 45, 4,000: 97 and 72; four rows,
  // 128 wide, 8 heads: 300 positions 10 and 11, 2,000: 12 and 13, 16,000: 33 and 19.  More rows are chunks of four, each reading
  // the positions again: worth it while all chunks are on the GPU at once and a CTA's share is short.  8 heads, 8 rows, 64 wide,
  // 40 positions: 7.4 and 8.8, 600: 9.1 and 10.9, 6,000: 20 and 15; 36 rows, 128 wide, 40: 8.0 and 10.4, 2,000: 31 and 19; 64
  // units of 16 rows, 64 wide, 150 positions: 10.1 and 12.0, of 36 rows (two turns): 19 and 13.
  // The bound on one row does not fit few units over long contexts, since a unit has eight CTAs at most: 64 wide, 131,067 positions,
  // 1 unit 134 and 68, 8 units 182 and 51, 32 units 195 and 136; 128 wide, 1 unit 324 and 86; 16,000 positions, 8 units, 64 wide 20
  // and 20, 128 wide 48 and 24.  It goes by the room in the table, as all of these do: the lengths are on the GPU.
  const int64_t rows = static_cast<int64_t>(P.N) * P.group, D = P.c.head_dim;
  if (rows == 1 && D == 64) return false;
  const int64_t work = static_cast<int64_t>(P.B) * P.c.kv_heads * capacity_of(P.c) * D * rows;
  if (rows > 4) {
    const int splits = row_splits(P);
    return row_units(P, 4) * splits > row_ctas(P) || capacity_of(P.c) * D > 24000LL * splits;
  }
  return work > (rows == 1 ? 100000000 : 16000000);
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
  return P.dtype == SPEC_DTYPE_BF16 ? launch_rows<SPEC_DTYPE_BF16>(P, st) : launch_rows<SPEC_DTYPE_F16>(P, st);
}

}  // namespace sv
