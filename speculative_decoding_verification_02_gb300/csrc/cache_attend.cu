// spec_cache_attend: attention of the drafted rows over the 8-bit cache.
//
//   x_j = cap tanh(scale q.k_j / cap) over the positions that the row sees
//   out = sum_j exp(x_j - m) v_j / sum_j exp(x_j - m),  lse = m + log sum_j exp(x_j - m)
//
// in one pass with the running maximum m and sum.  Heads of 64 and 128 run on
// the tensor cores (cache_attend_tile_kernel and the merge after it), other
// widths a warp to a row (cache_attend_rows_kernel).
#include <algorithm>

#include "cache.cuh"
#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"

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


// ---------------------------------------------------------------- tensor cores
//
// The rows of a kv head (token i, query head g of its group: row i * group + g)
// are taken RT at a time, the positions 128 at a time.  The tiles of all
// (request, head, row tile) units are laid end to end and cut into equal
// ranges, one to a CTA, so a batch of any lengths fills every SM; a unit that
// crosses a cut leaves partial sums that cache_attend_merge_kernel joins.
//
//   scores  S = Q K^T   kind::f8f6f4.  K goes from the pool to the tensor core
//           as it is.  A row of q, scaled by a power of two to at most 256, is
//           the sum of PIECES e4m3 numbers: two hold a bf16's 8 bits and
//           three an fp16's 11; what is left is at most 2^-10 (half a
//           subnormal step) against a largest element of at least 128.
//   values  O += P V    kind::f16, P from tensor memory.  V's bytes become
//           halves in shared memory, exactly; P is rounded to 11 bits.
//
// P carries the V block's scale: with lv = log2(v_scale), e = 2^(x + lv - m + 7)
// and the sum takes e / v_scale.  The reference m follows the running
// maximum of x + lv only when that has grown by more than 8, so O in tensor
// memory is rarely rescaled; e stays within 2^15 and keeps 11 bits down to
// 2^-29 of the largest.
//
// A unit of few rows leaves lanes of the 128-row operand free.  They hold
// REPL copies of the rows (RT = 128 / REPL); copy w, on its own warps, takes
// the w-th part of each tile's positions, its P zero elsewhere, and the copies
// are summed at the unit's end.  So four warps share the exponentials of 32
// rows or fewer.

constexpr int kTile = 128;         // positions to a tile
constexpr int kMaxRequests = 1024;  // requests to a launch
constexpr int kTileThreads = 320;  // 4 softmax warps, 1 loading, 1 issuing, 4 widening V
constexpr int kRing = 8;           // tiles whose scales are held

template <int DT, int D>
struct TileShape {
  static constexpr int kPieces = DT == SPEC_DTYPE_BF16 ? 2 : 3;
  static constexpr int kStage = kTile * D;
  static constexpr int kStagesK = D == 128 ? 3 : 6;
  static constexpr int kStagesV = D == 128 ? (kPieces == 2 ? 4 : 3) : 6;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + kPieces * kTile * D;
  static constexpr int kV8 = kK + kStagesK * kStage;
  static constexpr int kV16 = kV8 + kStagesV * kStage;
  static constexpr int kFold = kV16 + 2 * 2 * kStage;       // 128 x 17 floats: the copies' sums, 16 columns at a time
  static constexpr int kSmall = kFold + 128 * 17 * 4;
  static constexpr int kBytes = kSmall + 8192 + 1024;       // (1024: alignment of the base)
};

// Small arrays, after the operands.
struct TileSmall {
  int start[kMaxRequests + 1];
  float4 ring[kRing][8];  // a 16-position group's k_scale, log2(v_scale), 1 / v_scale
  float row_factor[128];
  float2 ml[128];
  uint32_t poison[2][4];
  uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6], w_full[2], s_full[2], s_empty[2], p_full[2], pv_done[2];
  uint64_t q_full, o_free, meet, ring_full[kRing], ring_empty[kRing];
  uint32_t tmem;
  int dead;
};
static_assert(sizeof(TileSmall) <= 8192);

struct TilePlan {
  CacheAttendParams p;
  int first, count;  // requests of this launch
  int page_rows;     // rows of a page that one copy brings: min(page size, 128)
  int *start, *verdict, *dead;
  float2 *ml;  // [CTA][2][RT]
  float *part; // [CTA][2][RT][D]
};

struct Unit {
  int b, head, row0, rows;  // request, kv head, first row, rows
  int base, n, T;           // context, query tokens, positions that its rows can see
  int tile0, tiles;         // its tiles in the launch's order
};

__device__ __forceinline__ int unit_positions(int base, int n, int group, int row_tile, int rt, bool masked) {
  return masked ? base + n : base + (min((rt + 1) * row_tile, n * group) - 1) / group + 1;
}

// The request's lengths, SPEC_STATUS_OK or _BAD_LENGTH.
__device__ __forceinline__ int request_lengths(const CacheAttendParams &P, int b, int &base, int &n) {
  base = P.cache_len[b];
  n = P.n_query ? P.n_query[b] : P.N;
  if (base < 0 || n < 0 || n > P.N || base + static_cast<int64_t>(n) > capacity(P.c)) return SPEC_STATUS_BAD_LENGTH;
  return SPEC_STATUS_OK;
}

__device__ __forceinline__ int request_tiles(const CacheAttendParams &P, int row_tile, int base, int n) {
  int tiles = 0;
  for (int rt = 0; rt * row_tile < n * P.group; ++rt)
    tiles += (unit_positions(base, n, P.group, row_tile, rt, P.mask != nullptr) + kTile - 1) / kTile;
  return tiles;
}

// The unit of request b (its tiles begin at `start`, span of them) that holds tile t.
__device__ Unit unit_of(const TilePlan &A, int row_tile, int b, int start, int span, int t) {
  const CacheAttendParams &P = A.p;
  Unit u;
  u.b = A.first + b;
  request_lengths(P, u.b, u.base, u.n);
  const int per_head = span / P.c.kv_heads;
  u.head = (t - start) / per_head;
  u.tile0 = start + u.head * per_head;
  for (int rt = 0;; ++rt) {
    u.T = unit_positions(u.base, u.n, P.group, row_tile, rt, P.mask != nullptr);
    u.tiles = (u.T + kTile - 1) / kTile;
    if (t < u.tile0 + u.tiles || (rt + 1) * row_tile >= u.n * P.group) {
      u.row0 = rt * row_tile;
      u.rows = min(row_tile, u.n * P.group - u.row0);
      return u;
    }
    u.tile0 += u.tiles;
  }
}

__device__ Unit find_unit(const TilePlan &A, const int *start, int row_tile, int t) {
  int lo = 0, hi = A.count - 1;  // the last request whose start is <= t has tiles after it: equal starts are empty requests
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (start[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return unit_of(A, row_tile, lo, start[lo], start[lo + 1] - start[lo], t);
}

__device__ __forceinline__ int cut(int total, int parts, int i) {
  return static_cast<int>(static_cast<int64_t>(total) * i / parts);
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 16-byte chunk index of a row in the K-major swizzle of its row length.
template <int D>
__device__ __forceinline__ int swizzled(int row, int chunk) {
  return D == 128 ? chunk ^ (row & 7) : chunk ^ (row >> 1 & 3);
}

template <int DT, int D, int REPL>
__global__ void __launch_bounds__(kTileThreads, 1)
    cache_attend_tile_kernel(const TilePlan A, const __grid_constant__ CUtensorMap k_map) {
  using S = TileShape<DT, D>;
  constexpr int RT = 128 / REPL;        // rows to a unit
  constexpr int OWN = kTile / REPL;     // positions that a copy takes of each tile
  constexpr uint32_t kCols = 512, kO = 256, kP = 384;  // tensor memory: S at 0 and 128, O, P at 384 and 448
  extern __shared__ char raw[];
  char *const smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  TileSmall &sm = *reinterpret_cast<TileSmall *>(smem + S::kSmall);
  const CacheAttendParams &P = A.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;

  if (tid == 0) {
    for (int i = 0; i < S::kStagesK; ++i) bar_init(&sm.k_full[i], 1), bar_init(&sm.k_empty[i], 1);
    for (int i = 0; i < S::kStagesV; ++i) bar_init(&sm.v_full[i], 1), bar_init(&sm.v_empty[i], 128);
    for (int i = 0; i < 2; ++i) {
      bar_init(&sm.w_full[i], 128);
      bar_init(&sm.s_full[i], 1);
      bar_init(&sm.s_empty[i], 128);
      bar_init(&sm.p_full[i], 128);
      bar_init(&sm.pv_done[i], 1);
    }
    bar_init(&sm.q_full, 128);
    bar_init(&sm.o_free, 128);
    bar_init(&sm.meet, 128);
    for (int i = 0; i < kRing; ++i) bar_init(&sm.ring_full[i], 32), bar_init(&sm.ring_empty[i], 128);
    bar_init_fence();
    sm.dead = 0;
  }
  if (warp == 5) tmem_alloc(&sm.tmem, kCols);
  // Every request's tiles, then their running sum.
  for (int b = tid; b < A.count; b += kTileThreads) {
    int base, n;
    const bool ok = request_lengths(P, A.first + b, base, n) == SPEC_STATUS_OK;
    sm.start[b + 1] = ok ? request_tiles(P, RT, base, n) * P.c.kv_heads : 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    int carry = 0;
    for (int b0 = 0; b0 < A.count; b0 += 32) {
      int x = b0 + lane < A.count ? sm.start[b0 + lane + 1] : 0;
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
      }
      x += carry;
      if (b0 + lane < A.count) {
        sm.start[b0 + lane + 1] = x;
        if (cta == 0) A.start[b0 + lane + 1] = x;
      }
      carry = __shfl_sync(~0u, x, 31);
    }
    if (lane == 0) {
      sm.start[0] = 0;
      if (cta == 0) A.start[0] = 0;
    }
  }
  __syncthreads();
  const int total = sm.start[A.count];
  const int lo = cut(total, ctas, cta), hi = cut(total, ctas, cta + 1);
  const uint32_t tmem = sm.tmem;
  volatile int *dead = &sm.dead;

  if (warp == 4) {
    // ---- loading: a lane to a group of 16 positions (the first 8 lanes), two tiles ahead with the page table
    const int shift = P.c.page_shift;
    const int page_rows = A.page_rows;
    int ahead_t = lo, ahead_end = lo;
    Unit au{};
    // the next tile's position of this lane's group, its request and head; -1 past the range or the unit's positions
    int g_pos[2], g_b[2], g_head[2], g_page[2];
    auto advance = [&](int slot) {
      g_page[slot] = -1;
      g_pos[slot] = -1;
      if (ahead_t >= hi) return;
      if (ahead_t >= ahead_end) {
        au = find_unit(A, sm.start, RT, ahead_t);
        ahead_end = au.tile0 + au.tiles;
      }
      const int pos = (ahead_t - au.tile0) * kTile + lane * 16;
      g_b[slot] = au.b;
      g_head[slot] = au.head;
      if (lane < 8 && pos < au.T) {
        g_pos[slot] = pos;
        g_page[slot] = page_at(P.c, au.b, pos >> shift);
      }
      ++ahead_t;
    };
    float ks = 0.0f, vs = 1.0f, ks1 = 0.0f, vs1 = 1.0f;
    auto scales = [&](int slot, float &k, float &v) {
      k = 0.0f, v = 1.0f;
      if (g_page[slot] >= 0) {
        const int64_t at = g_page[slot] * P.c.scale_stride + g_head[slot];
        k = P.c.k_scale[at];
        v = P.c.v_scale[at];
      }
    };
    advance(0);
    advance(1);
    scales(0, ks, vs);
    for (int t = lo; t < hi; ++t) {
      const int i = t - lo, cur = 0;
      // this tile's data, and the loads of the next ones'
      const int pos = g_pos[cur], page = g_page[cur], head = g_head[cur];
      scales(1, ks1, vs1);
      g_pos[0] = g_pos[1], g_b[0] = g_b[1], g_head[0] = g_head[1], g_page[0] = g_page[1];
      advance(1);
      const int r = i % kRing;
      if (i >= kRing && !warp_wait(&sm.ring_empty[r], (i / kRing - 1) & 1, dead)) break;
      if (lane < 8) sm.ring[r][lane] = make_float4(ks, log2f(vs), 1.0f / vs, 0.0f);
      bar_arrive(&sm.ring_full[r]);
      const bool load = pos >= 0 && page >= 0 && (pos & (page_rows - 1)) == 0;
      const uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(~0u, load)) * page_rows * D);
      const int sk = i % S::kStagesK, sv = i % S::kStagesV;
      if (i >= S::kStagesK && !warp_wait(&sm.k_empty[sk], (i / S::kStagesK - 1) & 1, dead)) break;
      if (lane == 0) bar_expect(&sm.k_full[sk], bytes);
      __syncwarp();
      const int in_page = pos & ((1 << shift) - 1), in_tile = lane * 16;
      if (load) tensor_load_3d(smem + S::kK + sk * S::kStage + in_tile * D, &k_map, 0, (head << shift) + in_page, page, &sm.k_full[sk]);
      if (i >= S::kStagesV && !warp_wait(&sm.v_empty[sv], (i / S::kStagesV - 1) & 1, dead)) break;
      if (lane == 0) bar_expect(&sm.v_full[sv], bytes);
      __syncwarp();
      if (load)
        bulk_load(smem + S::kV8 + sv * S::kStage + in_tile * D, P.c.v + block_offset(P.c, page, head) + static_cast<int64_t>(in_page) * D,
                  page_rows * D, &sm.v_full[sv]);
      ks = ks1, vs = vs1;
    }
    __syncwarp();
    if (*dead) {  // the copies in flight land before the CTA leaves
      for (int s = 0; s < S::kStagesK; ++s)
        for (int k = 0; k < 4096 && !bar_try(&sm.k_full[s], 0) && !bar_try(&sm.k_full[s], 1); ++k) {}
      for (int s = 0; s < S::kStagesV; ++s)
        for (int k = 0; k < 4096 && !bar_try(&sm.v_full[s], 0) && !bar_try(&sm.v_full[s], 1); ++k) {}
    }
  } else if (warp == 5) {
    // ---- issuing: S of tile i, then O += P V of tile i - 1
    if (lane == 0) {
      constexpr uint32_t kIdS = mma_desc(kTile, false), kIdO = mma_desc(D, true);
      constexpr uint64_t kSw = D == 128 ? kSwizzle128 : kSwizzle64;
      const uint64_t q_desc = matrix_desc(smem_u32(smem + S::kQ), 16, 8 * D, kSw);
      const uint64_t k_desc = matrix_desc(smem_u32(smem + S::kK), 16, 8 * D, kSw);
      const uint64_t v_desc = matrix_desc(smem_u32(smem + S::kV16), kTile * 128, 1024, kSwizzle128);
      int unit_end = lo, units = 0;
      bool first = false, was_first = false, ok = true;
      auto values = [&](int i, bool fresh, int unit) {  // O += P V of tile i
        const int w = i & 1;
        if (!bar_wait(&sm.w_full[w], (i >> 1) & 1, dead) || !bar_wait(&sm.p_full[w], (i >> 1) & 1, dead)) return false;
        if (fresh && unit > 1 && !bar_wait(&sm.o_free, unit & 1, dead)) return false;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_f16_ta(tmem + kO, tmem + kP + w * 64 + k * 8, v_desc + ((w * 2 * S::kStage + k * 2048) >> 4), kIdO, !(fresh && k == 0));
        tc_commit(&sm.pv_done[w]);
        return true;
      };
      for (int t = lo; t < hi && ok; ++t) {
        const int i = t - lo, sk = i % S::kStagesK;
        was_first = first;
        first = t >= unit_end;
        if (first) {
          // (the tile before closes its unit: its values first, while q's rows are being written)
          if (i > 0 && !(ok = values(i - 1, was_first, units))) break;
          const Unit u = find_unit(A, sm.start, RT, t);
          unit_end = u.tile0 + u.tiles;
          if (!bar_wait(&sm.q_full, units & 1, dead)) break;
          ++units;
        }
        if (!bar_wait(&sm.k_full[sk], (i / S::kStagesK) & 1, dead)) break;
        if (i >= 2 && !bar_wait(&sm.s_empty[i & 1], (i / 2 - 1) & 1, dead)) break;
        tc_fence_after();
#pragma unroll
        for (int piece = 0; piece < S::kPieces; ++piece)
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            mma_f8(tmem + (i & 1) * 128, q_desc + ((piece * kTile * D + k * 32) >> 4), k_desc + ((sk * S::kStage + k * 32) >> 4), kIdS,
                   piece + k > 0);
        tc_commit(&sm.k_empty[sk]);
        tc_commit(&sm.s_full[i & 1]);
        if (i > 0 && !first) ok = values(i - 1, was_first, units);
      }
      if (ok && hi > lo && !*dead) values(hi - lo - 1, first, units);
    }
    __syncwarp();
  } else if (warp >= 6) {
    // ---- widening V: 16 bytes of a position to 16 halves, in the MN-major layout of the operand
    const int w4 = warp - 6;
    for (int b = cta; b < A.count; b += ctas) {  // and, on the way, the page tables: a request with a bad page gives nothing
      int base, n;
      int st = request_lengths(P, A.first + b, base, n);
      int bad = 0;
      if (st == SPEC_STATUS_OK)
        for (int j = tid - 192; static_cast<int64_t>(j) << P.c.page_shift < base + n; j += 128) bad |= page_at(P.c, A.first + b, j) < 0;
      if (tid == 192) A.verdict[b] = st;
      asm volatile("bar.sync 2, 128;" ::: "memory");
      if (bad) A.verdict[b] = SPEC_STATUS_BAD_PAGE;
    }
    int unit_end = lo;
    Unit u{};
    constexpr int kLanes = D / 16;        // lanes to a position
    constexpr int kPer = 32 / kLanes;     // positions to a step
    const int piece = lane % kLanes, sub = lane / kLanes;
    for (int t = lo; t < hi; ++t) {
      const int i = t - lo, sv = i % S::kStagesV, w = i & 1;
      if (t >= unit_end) {
        u = find_unit(A, sm.start, RT, t);
        unit_end = u.tile0 + u.tiles;
      }
      const int pos0 = (t - u.tile0) * kTile;
      const bool edge = pos0 + kTile > u.base;
      if (!warp_wait(&sm.v_full[sv], (i / S::kStagesV) & 1, dead)) break;
      if (i >= 2 && !warp_wait(&sm.pv_done[w], (i / 2 - 1) & 1, dead)) break;
      const char *src = smem + S::kV8 + sv * S::kStage;
      char *dst = smem + S::kV16 + w * 2 * S::kStage;
      uint32_t poison = 0;
#pragma unroll
      for (int step = 0; step < 32 / kPer; ++step) {
        const int at = step * kPer + sub, row = w4 * 32 + at;
        uint4 x = *reinterpret_cast<const uint4 *>(src + row * D + piece * 16);
        if (edge) {  // nothing past the last position, and no NaN where a row may not look
          const int pos = pos0 + row;
          bool nan = false;
          if (pos >= u.T) x = make_uint4(0, 0, 0, 0);
          else if (pos >= u.base) {
            uint32_t *e = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              // bytes of 0x7f under the sign: 0x80 after adding one
              const uint32_t hit = ((e[c] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
              if (hit) {
                nan = true;
                e[c] &= ~(hit | (hit - (hit >> 7)));
              }
            }
          }
          const uint32_t vote = __ballot_sync(~0u, nan);
#pragma unroll
          for (int c = 0; c < kPer; ++c)
            if (vote >> (c * kLanes) & ((1u << kLanes) - 1)) poison |= 1u << (step * kPer + c);
        }
        uint4 h[2];
        uint32_t *o = reinterpret_cast<uint32_t *>(h);
        const uint32_t in[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const __half2 a = e4m3x2_to_half2(in[c] & 0xffff), b = e4m3x2_to_half2(in[c] >> 16);
          o[2 * c] = *reinterpret_cast<const uint32_t *>(&a);
          o[2 * c + 1] = *reinterpret_cast<const uint32_t *>(&b);
        }
        // columns of 64: 16 KB apart; eight positions: 1024 bytes; chunks of 16 bytes swizzled by the position
        char *to = dst + (piece >> 2) * (kTile * 128) + (row >> 3) * 1024 + (row & 7) * 128;
        const int c0 = (piece & 3) * 2;
        const int flip = piece >> 2 & 1;  // (the two column groups store their chunks in opposite order: no bank conflict)
        *reinterpret_cast<uint4 *>(to + (((c0 + flip) ^ (row & 7)) << 4)) = h[flip];
        *reinterpret_cast<uint4 *>(to + (((c0 + 1 - flip) ^ (row & 7)) << 4)) = h[1 - flip];
      }
      if (edge && lane == 0) sm.poison[w][w4] = poison;
      fence_async_shared();
      bar_arrive(&sm.v_empty[sv]);
      bar_arrive(&sm.w_full[w]);
    }
  } else {
    // ---- softmax: a thread to a row (of its copy), OWN positions of each tile
    const int copy = warp * 32 / RT;                       // which copy of the rows
    const int r = (warp * 32 + lane) % RT;                 // the row
    const int col0 = copy * OWN;                           // its positions in the tile
    const uint32_t lanes = static_cast<uint32_t>(warp) << 21;  // this warp's lanes of tensor memory
    if (REPL > 1) {
      uint32_t zero[16] = {};
      for (int c = 0; c < 128; c += 16) tmem_st16(tmem + lanes + kP + c, zero);
      tc_wait_st();
    }
    const bool negative = P.scale < 0.0f;
    bool ok = true;
    uint32_t meetings = 0;
    auto together = [&] {  // a barrier of the four warps, bounded like every wait
      bar_arrive(&sm.meet);
      return warp_wait(&sm.meet, meetings++ & 1, dead);
    };
    // A unit's rows of q as e4m3 pieces; every earlier score product that reads them has completed.
    auto write_q = [&](const Unit &u) {
      constexpr int kEach = D / 32;  // elements to a lane
      for (int r0 = warp; r0 < u.rows; r0 += 4) {
        const int row = u.row0 + r0;
        const char *q = P.q + (u.b * P.qs[0] + row / P.group * P.qs[1] + (u.head * P.group + row % P.group) * P.qs[2]) * 2;
        float x[kEach], top = 0.0f;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          x[e] = row_value<DT>(q, lane * kEach + e);
          if (negative) x[e] = -x[e];
          top = fmaxf(top, finite_abs(x[e]));
        }
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        // 2^ex with top / 2^ex in [128, 256)
        const int ex = top > 0.0f ? max(static_cast<int>(__float_as_uint(top) >> 23) - 127 - 7, -110) : 0;
        const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
#pragma unroll
        for (int e = 0; e < kEach; ++e) x[e] *= down;
#pragma unroll
        for (int piece = 0; piece < S::kPieces; ++piece) {
          uint32_t code = 0;
#pragma unroll
          for (int e = 0; e < kEach; e += 2) {
            const uint32_t two = to_e4m3x2(x[e], x[e + 1]);
            const float2 back = e4m3x2_to_float2(two);
            x[e] -= back.x;
            x[e + 1] -= back.y;
            code |= two << (8 * e);
          }
#pragma unroll
          for (int c = 0; c < REPL; ++c) {
            const int a = c * RT + r0;
            char *to = smem + S::kQ + piece * kTile * D + a * D + (swizzled<D>(a, lane * kEach >> 4) << 4) + (lane * kEach & 15);
            if (kEach == 4) *reinterpret_cast<uint32_t *>(to) = code;
            else *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(code);
          }
        }
        if (lane == 0) sm.row_factor[r0] = fabsf(P.scale) * kLog2e * __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
      }
      fence_async_shared();
      bar_arrive(&sm.q_full);
      return together();
    };
    Unit next{};
    if (lo < hi) {
      next = find_unit(A, sm.start, RT, lo);
      ok = write_q(next);
    }
    for (int t = lo; t < hi && ok;) {
      const Unit u = next;
      const int t_end = min(hi, u.tile0 + u.tiles);
      const bool live = r < u.rows;
      const float factor = live ? sm.row_factor[r] : 0.0f;
      const int token = live ? (u.row0 + r) / P.group : 0;
      const uint8_t *mask = P.mask ? P.mask + (static_cast<int64_t>(u.b) * P.N + token) * P.N : nullptr;
      const float cap2 = P.softcap * kLog2e;                            // the cap in units of log 2
      const float in_cap = P.softcap > 0.0f ? 2.0f / P.softcap : 0.0f;  // (of x in units of log 2) to 2 x / cap in units of log 2
      float m = -INFINITY, sum = 0.0f;
      bool spoiled = false;

      for (; t < t_end; ++t) {
        const int i = t - lo, sb = i & 1, ring = i % kRing;
        if (!(ok = warp_wait(&sm.ring_full[ring], (i / kRing) & 1, dead))) break;
        if (!(ok = warp_wait(&sm.s_full[sb], (i >> 1) & 1, dead))) break;
        tc_fence_after();
        float s[OWN];
#pragma unroll
        for (int c = 0; c < OWN; c += 32) tmem_ld32(tmem + lanes + sb * 128 + col0 + c, s + c);
        tc_wait_ld();
        tc_fence_before();
        bar_arrive(&sm.s_empty[sb]);

        const int pos0 = (t - u.tile0) * kTile + col0;
        const bool edge = pos0 + OWN > u.base;
        uint32_t sees[OWN / 32];
        if (edge) {
#pragma unroll
          for (int c = 0; c < OWN / 32; ++c) {
            uint32_t bits = 0;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int j = pos0 + c * 32 + e - u.base;
              const bool yes = j < 0 || (j < u.n && (mask ? mask[j] != 0 : j <= token));
              bits |= yes ? 1u << e : 0u;
            }
            sees[c] = live ? bits : 0;
          }
        }
        // x = score + log2(v_scale), in units of log 2
        float top = -INFINITY;
#pragma unroll
        for (int g = 0; g < OWN / 16; ++g) {
          const float4 sc = sm.ring[ring][col0 / 16 + g];
          const float f = factor * sc.x;
          if (P.softcap > 0.0f) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              // cap tanh(x / cap) = cap (1 - 2 / (1 + exp(2 x / cap)))
              const float y = s[g * 16 + e] * f * in_cap;
              s[g * 16 + e] = cap2 * (1.0f - __fdividef(2.0f, 1.0f + ex2(y > 120.0f ? 120.0f : y)));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) s[g * 16 + e] *= f;
          }
          float high = -INFINITY;
          if (edge) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (sees[g / 2] >> (g % 2 * 16 + e) & 1) high = fmaxf(high, s[g * 16 + e]);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) high = fmaxf(high, s[g * 16 + e]);
          }
          top = fmaxf(top, high + sc.y);
        }
        // the reference, and O with it when it moves
        const bool moves = live && top > m + 8.0f;
        if (__any_sync(~0u, moves)) {
          const float next = moves ? top : m;
          const float keep = m == -INFINITY ? 0.0f : ex2(m - next);
          m = next;
          sum *= keep;
          const int done = i - 1;
          if (t > max(lo, u.tile0)) {
            if (!(ok = warp_wait(&sm.pv_done[done & 1], (done >> 1) & 1, dead))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float o[16];
              tmem_ld16(tmem + lanes + kO + c, o);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= keep;
              tmem_st16(tmem + lanes + kO + c, reinterpret_cast<uint32_t *>(o));
            }
            tc_wait_st();
          }
        }
        if (i >= 2 && !(ok = warp_wait(&sm.pv_done[sb], (i / 2 - 1) & 1, dead))) break;  // P's columns are free
        tc_fence_after();
        const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int c = 0; c < OWN / 32; ++c) {
          uint32_t p[16];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float4 sc = sm.ring[ring][col0 / 16 + c * 2 + g];
            const float shift = sc.y - ref + 7.0f;
            float part = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const int at = c * 32 + g * 16 + e;
              float a = ex2(s[at] + shift), b = ex2(s[at + 1] + shift);
              if (edge) {
                if (!(sees[c] >> (g * 16 + e) & 1)) a = 0.0f;
                if (!(sees[c] >> (g * 16 + e + 1) & 1)) b = 0.0f;
              }
              part += a + b;
              p[g * 8 + e / 2] = half2_bits(a, b);
            }
            sum = fmaf(part, sc.z, sum);
          }
          tmem_st16(tmem + lanes + kP + sb * 64 + (col0 + c * 32) / 2, p);
        }
        if (edge) {  // a row that sees a position whose V was NaN
          if (!(ok = warp_wait(&sm.w_full[sb], (i >> 1) & 1, dead))) break;
#pragma unroll
          for (int c = 0; c < OWN / 32; ++c) spoiled |= (sees[c] & sm.poison[sb][col0 / 32 + c]) != 0;
        }
        bar_arrive(&sm.ring_empty[ring]);
        tc_wait_st();
        tc_fence_before();
        bar_arrive(&sm.p_full[sb]);
      }
      if (!ok) break;

      if (t < hi) {  // the next unit's q, while this one's last values are being summed
        next = find_unit(A, sm.start, RT, t);
        if (!(ok = write_q(next))) break;
      }
      // The unit's end in this CTA: sum the copies, and write the rows or leave them as partial sums.
      const int last = t - 1 - lo;
      if (!(ok = warp_wait(&sm.pv_done[last & 1], (last >> 1) & 1, dead))) break;
      tc_fence_after();
      const bool whole = lo <= u.tile0 && t == u.tile0 + u.tiles;
      const int slot = cta * 2 + (u.tile0 >= lo && t == hi && max(lo, u.tile0) != lo ? 1 : 0);
      float *fold = reinterpret_cast<float *>(smem + S::kFold);
      float w_own = 1.0f, m_all = m, l_all = sum;
      if (REPL > 1) {
        sm.ml[warp * 32 + lane] = make_float2(m, sum);
        if (!(ok = together())) break;
        for (int c = 0; c < REPL; ++c) m_all = fmaxf(m_all, sm.ml[c * RT + r].x);
        const float ref = m_all == -INFINITY ? 0.0f : m_all;
        l_all = 0.0f;
        for (int c = 0; c < REPL; ++c) l_all += sm.ml[c * RT + r].y * ex2(sm.ml[c * RT + r].x - ref);
        w_own = ex2(m - ref);
      }
      const float norm = whole ? (l_all == 0.0f ? 0.0f : 1.0f / l_all) : 1.0f;
      if (live && (REPL == 1 || copy == 0)) {
        const int row = u.row0 + r;
        if (whole) {
          if (P.lse)
            P.lse[(static_cast<int64_t>(u.b) * P.N + token) * P.Hq + u.head * P.group + row % P.group] =
                l_all == 0.0f ? -INFINITY : (m_all - 7.0f + log2f(l_all)) * kLn2;
        } else {
          A.ml[static_cast<int64_t>(slot) * RT + r] = make_float2(m_all, l_all);
        }
      }
      // O of a row with no visible position at all is zero: P was.  (0 * scale: w_own is 1 or 0 there.)
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        float o[16];
        tmem_ld16(tmem + lanes + kO + c, o);
        tc_wait_ld();
        if (spoiled) o[0] = o[1] = o[2] = o[3] = o[4] = o[5] = o[6] = o[7] = o[8] = o[9] = o[10] = o[11] = o[12] = o[13] = o[14] = o[15] = NAN;
        if (REPL == 1) {
          if (live) {
            if (whole) {
              const int row = u.row0 + r;
              char *out = P.out + (u.b * P.os[0] + token * P.os[1] + (u.head * P.group + row % P.group) * P.os[2]) * 2;
#pragma unroll
              for (int e = 0; e < 16; ++e) put_value<DT>(out, c + e, o[e] * norm);
            } else {
              float4 *to = reinterpret_cast<float4 *>(A.part + (static_cast<int64_t>(slot) * RT + r) * D + c);
#pragma unroll
              for (int e = 0; e < 4; ++e) to[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
          }
        } else {
          if (!(ok = together())) break;  // the columns before have been read
#pragma unroll
          for (int e = 0; e < 16; ++e) fold[(warp * 32 + lane) * 17 + e] = o[e] * w_own;
          if (!(ok = together())) break;
          for (int x = tid; x < RT * 16; x += 128) {
            const int rr = x >> 4, e = x & 15;
            if (rr >= u.rows) break;
            float y = 0.0f;
#pragma unroll
            for (int k = 0; k < REPL; ++k) y += fold[(k * RT + rr) * 17 + e];
            if (whole) {
              const int row = u.row0 + rr;
              float l = 0.0f, mm = -INFINITY;
              for (int k = 0; k < REPL; ++k) mm = fmaxf(mm, sm.ml[k * RT + rr].x);
              const float ref = mm == -INFINITY ? 0.0f : mm;
              for (int k = 0; k < REPL; ++k) l += sm.ml[k * RT + rr].y * ex2(sm.ml[k * RT + rr].x - ref);
              char *out = P.out + (u.b * P.os[0] + row / P.group * P.os[1] + (u.head * P.group + row % P.group) * P.os[2]) * 2;
              put_value<DT>(out, c + e, l == 0.0f ? 0.0f : y / l);
            } else {
              A.part[(static_cast<int64_t>(slot) * RT + rr) * D + c + e] = y;
            }
          }
        }
      }
      tc_fence_before();
      bar_arrive(&sm.o_free);
      if (REPL > 1) ok = ok && together();  // ml has been read
    }
  }
  tc_fence_before();
  __syncthreads();
  pdl_launch_dependents();
  if (tid == 0) A.dead[cta] = sm.dead;
  if (warp == 5) {
    tc_fence_after();
    tmem_free(tmem, kCols);
  }
}

// Joins the partial sums of the units that more than one CTA worked on, a warp
// to a row, and writes what no unit covers: rows past n_query, bad requests.
template <int DT, int D>
__global__ void __launch_bounds__(256) cache_attend_merge_kernel(const TilePlan A, int row_tile, int ctas) {
  const CacheAttendParams &P = A.p;
  const int lane = threadIdx.x & 31;
  const int64_t x = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  pdl_wait();
  if (x >= static_cast<int64_t>(A.count) * P.N * P.Hq) return;
  const int h = static_cast<int>(x % P.Hq), i = static_cast<int>(x / P.Hq % P.N), bl = static_cast<int>(x / P.Hq / P.N);
  const int b = A.first + bl;
  int st = A.verdict[bl];
  int gone = 0;
  for (int c = lane; c < ctas; c += 32) gone |= A.dead[c];
  if (__any_sync(~0u, gone)) st = SPEC_STATUS_TIMEOUT;
  if (P.status && i == 0 && h == 0 && lane == 0) P.status[b] = st;
  constexpr int kEach = D / 32;
  char *out = P.out + (b * P.os[0] + i * P.os[1] + h * P.os[2]) * 2;
  const int64_t at_lse = (static_cast<int64_t>(b) * P.N + i) * P.Hq + h;
  int base, n;
  request_lengths(P, b, base, n);
  if (st != SPEC_STATUS_OK || i >= n) {
    for (int e = 0; e < kEach; ++e) put_value<DT>(out, lane * kEach + e, 0.0f);
    if (lane == 0 && P.lse) P.lse[at_lse] = -INFINITY;
    return;
  }
  // the row's unit, and the CTAs whose ranges it meets
  const int total = A.start[A.count], start = A.start[bl], span = A.start[bl + 1] - start;
  const int head = h / P.group, row = i * P.group + h % P.group, rt = row / row_tile, r = row % row_tile;
  int tile0 = start + head * (span / P.c.kv_heads);
  for (int k = 0; k < rt; ++k) tile0 += (unit_positions(base, n, P.group, row_tile, k, P.mask != nullptr) + kTile - 1) / kTile;
  const int tiles = (unit_positions(base, n, P.group, row_tile, rt, P.mask != nullptr) + kTile - 1) / kTile;
  int c0 = static_cast<int>(static_cast<int64_t>(tile0) * ctas / total);
  while (cut(total, ctas, c0 + 1) <= tile0) ++c0;
  int c1 = c0;
  while (cut(total, ctas, c1 + 1) < tile0 + tiles) ++c1;
  if (c0 == c1) return;
  auto slot_of = [&](int c) {
    const int s = c * 2 + (c == c0 && cut(total, ctas, c) < tile0 ? 1 : 0);
    return static_cast<int64_t>(s) * row_tile + r;
  };
  auto has = [&](int c) { return cut(total, ctas, c + 1) > cut(total, ctas, c); };
  float m = -INFINITY;
  for (int c = c0 + lane; c <= c1; c += 32)
    if (has(c)) m = fmaxf(m, A.ml[slot_of(c)].x);
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  const float ref = m == -INFINITY ? 0.0f : m;
  float acc[kEach] = {}, sum = 0.0f;
  for (int cc = c0; cc <= c1; cc += 32) {
    const int c = cc + lane;
    float w = 0.0f, l = 0.0f;
    int64_t s = 0;
    if (c <= c1 && has(c)) {
      s = slot_of(c);
      const float2 ml = A.ml[s];
      w = ex2(ml.x - ref);
      l = ml.y * w;
    }
    sum += warp_sum(l);
    const int here = min(32, c1 - cc + 1);
    for (int k = 0; k < here; ++k) {
      const float wk = __shfl_sync(~0u, w, k);
      const float *o = A.part + __shfl_sync(~0u, s, k) * D + lane * kEach;
      if (!has(cc + k)) continue;
#pragma unroll
      for (int e = 0; e < kEach; ++e) acc[e] = fmaf(o[e], wk, acc[e]);
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int e = 0; e < kEach; ++e) put_value<DT>(out, lane * kEach + e, acc[e] * inv);
  if (lane == 0 && P.lse) P.lse[at_lse] = sum == 0.0f ? -INFINITY : (m - 7.0f + log2f(sum)) * kLn2;
}

// ------------------------------------------------------------------- host

int copies_of(int N, int group) {
  const int64_t rows = static_cast<int64_t>(N) * group;
  return rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// Requests to a launch: at most kMaxRequests, and tiles that an int can number.
int requests_at_once(const CacheAttendParams &P) {
  const int rt = 128 / copies_of(P.N, P.group);
  const int64_t row_tiles = (static_cast<int64_t>(P.N) * P.group + rt - 1) / rt;
  const int64_t tiles = ((static_cast<int64_t>(P.c.table_stride) << P.c.page_shift) / kTile + 1) * row_tiles * P.c.kv_heads;
  return static_cast<int>(std::min<int64_t>(kMaxRequests, 2000000000LL / tiles));
}

size_t lay_out(TilePlan &A, char *ws, int D) {
  const int ctas = device_sm_count(), rt = 128 / copies_of(A.p.N, A.p.group);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char *p = ws ? ws + off : nullptr;
    off = round256(off + bytes);
    return p;
  };
  A.start = reinterpret_cast<int *>(take(sizeof(int) * (kMaxRequests + 1)));
  A.verdict = reinterpret_cast<int *>(take(sizeof(int) * kMaxRequests));
  A.dead = reinterpret_cast<int *>(take(sizeof(int) * ctas));
  A.ml = reinterpret_cast<float2 *>(take(sizeof(float2) * 2 * ctas * rt));
  A.part = reinterpret_cast<float *>(take(sizeof(float) * 2 * ctas * rt * D));
  return off;
}

template <int DT, int D, int REPL>
cudaError_t launch_tiles(TilePlan A, const CUtensorMap &map, cudaStream_t st) {
  using S = TileShape<DT, D>;
  auto kern = cache_attend_tile_kernel<DT, D, REPL>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
  if (e != cudaSuccess) return e;
  const int ctas = device_sm_count();
  e = trace_launch("cache_attend_tile", st, [&] { kern<<<ctas, kTileThreads, S::kBytes, st>>>(A, map); });
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(A.count) * A.p.N * A.p.Hq;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = trace_enabled() ? 0 : 1;
  return trace_launch_ex("cache_attend_merge", st,
                         [&] { return cudaLaunchKernelEx(&cfg, cache_attend_merge_kernel<DT, D>, A, 128 / REPL, ctas); });
}

template <int DT, int D>
cudaError_t launch_tiles(const TilePlan &A, const CUtensorMap &map, cudaStream_t st) {
  const int copies = copies_of(A.p.N, A.p.group);
  if (copies == 4) return launch_tiles<DT, D, 4>(A, map, st);
  if (copies == 2) return launch_tiles<DT, D, 2>(A, map, st);
  return launch_tiles<DT, D, 1>(A, map, st);
}

}  // namespace

bool cache_attend_on_tensor_cores(const CacheAttendParams &P) {
  return (P.c.head_dim == 64 || P.c.head_dim == 128) && requests_at_once(P) > 0;
}

size_t cache_attend_workspace(const CacheAttendParams &P) {
  if (!cache_attend_on_tensor_cores(P)) return 0;
  TilePlan A{};
  A.p = P;
  return lay_out(A, nullptr, P.c.head_dim);
}

cudaError_t launch_cache_attend(const CacheAttendParams &P, void *workspace, cudaStream_t st) {
  if (cache_attend_on_tensor_cores(P)) {
    TilePlan A{};
    A.p = P;
    A.page_rows = std::min(1 << P.c.page_shift, kTile);
    lay_out(A, static_cast<char *>(workspace), P.c.head_dim);
    CUtensorMap map;
    const cudaError_t made = cache_k_map(P.c, A.page_rows, &map);
    if (made != cudaSuccess) return made;
    const int at_once = requests_at_once(P);
    for (A.first = 0; A.first < P.B; A.first += at_once) {
      A.count = std::min(at_once, P.B - A.first);
      cudaError_t e;
      if (P.dtype == SPEC_DTYPE_BF16)
        e = P.c.head_dim == 128 ? launch_tiles<SPEC_DTYPE_BF16, 128>(A, map, st) : launch_tiles<SPEC_DTYPE_BF16, 64>(A, map, st);
      else
        e = P.c.head_dim == 128 ? launch_tiles<SPEC_DTYPE_F16, 128>(A, map, st) : launch_tiles<SPEC_DTYPE_F16, 64>(A, map, st);
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
