// The tensor-core path of spec_cache_attend (heads of 64 and 128).
#pragma once

#include <algorithm>
#include <atomic>

#include "cache.cuh"
#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"

namespace sv {
namespace {

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
// REPL copies of the rows (RT = 128 / REPL); copy w takes the w-th part of each
// tile's positions, its P zero elsewhere, and the copies are summed at the
// unit's end.  With four copies four warps do the exponentials, 32 positions
// to a thread.  With two or one, each 32 lanes are served by two warps, each of
// half of the positions, which agree on their rows' reference: that costs a
// barrier, and halves what a thread does between the two products.

// Heads of 128, 8 of them, in a graph of calls.  One request, 131,072 positions,
// 20 rows (four copies): 57 us, 4.7 TB/s, bound by the tensor pipe: a tile takes
// 1,220 cycles, its 16 instructions of about 77.  64 requests of up to 12,000
// positions, 36 rows (two copies): 175 us, 5.4 TB/s, a tile takes as long as its
// softmax (1,350 cycles) and 13% goes to units' starts and ends.  16 trees of 60
// nodes, 240 rows, up to 6,000 positions: 106 us, 600 TFLOP/s, bound by the
// exponentials and the chain around them (2,290 cycles a tile; 27% starts and
// ends).

constexpr int kTile = 128;         // positions to a tile
// What a unit costs a CTA besides its tiles (its q, its end), in tiles: the cuts
// count it, so that a CTA of many short units gets fewer tiles.
constexpr int kUnitCost = kTileUnitCost;
constexpr int kMaxRequests = kTileRequests;
// 8 softmax warps (4 of them idle with four copies), 4 widening V, 2 loading, 2
// issuing.  A warp's scheduler is its number modulo 4: the widening warps share
// two of them and the others the other two, so a scheduler runs few different
// loops (their instructions compete for its cache).
constexpr int kTileThreads = 512;
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
  static constexpr int kSmall = kV16 + 2 * 2 * kStage;
  static constexpr int kBytes = kSmall + 13312 + 1024;  // (1024: alignment of the base)
};

// What a CTA keeps of the launch's requests.
struct Requests {
  int start[kMaxRequests + 1];  // running sum of their tiles
  int2 lens[kMaxRequests];      // context, query tokens
  int per_head[kMaxRequests];   // tiles of a kv head
};

// Small arrays, after the operands.
struct TileSmall {
  Requests q;
  float4 ring[kRing][8];  // a 16-position group's k_scale, log2(v_scale), 1 / v_scale
  float tops[2][2][128];  // the two threads' maxima of a row, for two tiles
  float2 ml[2][128];      // reference and sum of a thread's positions
  int4 begun;  // the unit that begins here and ends in a later CTA
  float row_factor[2][128];  // by the unit's number: a warp may write the next unit's before another has read this one's
  float weight[128];   // of a copy's row when the copies are summed
  int64_t out_at[128];  // element offset of a row in out
  uint32_t poison[2][4];
  int spoiled[128];    // rows that saw a NaN value
  uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6], w_full[2], s_full[2], s_empty[2], p_full[2], pv_done[2];
  uint64_t q_full, o_free[2], meet, ring_full[kRing], ring_empty[kRing];
  uint32_t tmem;
  int dead;
  int copies_k, copies_v, products_s, products_o;  // how many were begun
};
static_assert(sizeof(TileSmall) <= 13312);

struct Unit {
  int b, head, row0, rows;  // request, kv head, first row, rows
  int base, n, T;           // context, query tokens, positions that its rows can see
  int start, tile0, tiles;  // its place in the launch's order: kUnitCost from start on, then its tiles
};

// x / group for the rows of a unit: a multiplication (x * group < 2^32), a few
// instructions where a division is forty.
__device__ __forceinline__ int by_group(const CacheTilePlan &A, int x) {
  return A.p.group == 1 ? x : static_cast<int>(__umulhi(static_cast<uint32_t>(x), A.group_inverse));
}

__device__ __forceinline__ int unit_positions(const CacheTilePlan &A, int base, int n, int row_tile, int rt) {
  return A.p.mask ? base + n : base + by_group(A, min((rt + 1) * row_tile, n * A.p.group) - 1) + 1;
}

// The request's lengths, SPEC_STATUS_OK or _BAD_LENGTH.
__device__ __forceinline__ int request_lengths(const CacheAttendParams &P, int b, int &base, int &n) {
  base = P.cache_len[b];
  n = P.n_query ? P.n_query[b] : P.N;
  if (base < 0 || n < 0 || n > P.N || base + static_cast<int64_t>(n) > capacity(P.c)) return SPEC_STATUS_BAD_LENGTH;
  return SPEC_STATUS_OK;
}

__device__ __forceinline__ int request_tiles(const CacheTilePlan &A, int row_tile, int base, int n) {
  int tiles = 0;
  for (int rt = 0; rt * row_tile < n * A.p.group; ++rt)
    tiles += kUnitCost + (unit_positions(A, base, n, row_tile, rt) + kTile - 1) / kTile;
  return tiles;
}

// The unit of request b that holds place t.
__device__ __forceinline__ Unit unit_of(const CacheTilePlan &A, const Requests &q, int row_tile, int b, int t) {
  const CacheAttendParams &P = A.p;
  Unit u;
  u.b = A.first + b;
  u.base = q.lens[b].x;
  u.n = q.lens[b].y;
  const int start = q.start[b], per_head = q.per_head[b];
  // the quotient from floats: off by one at most below 2^24, and put right
  u.head = static_cast<int>(__fdividef(static_cast<float>(t - start), static_cast<float>(per_head)));
  while (u.head > 0 && u.head * per_head > t - start) --u.head;
  while ((u.head + 1) * per_head <= t - start) ++u.head;
  u.start = start + u.head * per_head;
  for (int rt = 0;; ++rt) {
    u.T = unit_positions(A, u.base, u.n, row_tile, rt);
    u.tiles = (u.T + kTile - 1) / kTile;
    if (t < u.start + kUnitCost + u.tiles || (rt + 1) * row_tile >= u.n * P.group) {
      u.tile0 = u.start + kUnitCost;
      u.row0 = rt * row_tile;
      u.rows = min(row_tile, u.n * P.group - u.row0);
      return u;
    }
    u.start += kUnitCost + u.tiles;
  }
}

__device__ __noinline__ Unit find_unit(const CacheTilePlan &A, const Requests &q, int row_tile, int t) {
  int lo = 0, hi = A.count - 1;  // the last request whose start is <= t has tiles after it: equal starts are empty requests
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (q.start[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return unit_of(A, q, row_tile, lo, t);
}

// Where CTA i's range begins: floor(total * i / CTAs) (by a multiplication, exact
// below 2^64 / CTAs), or i itself when there is less to do than CTAs, so that no
// CTA has an empty range before one that has not.
__device__ __forceinline__ int cut(const CacheTilePlan &A, int total, int ctas, int i) {
  return total < ctas ? min(i, total) : static_cast<int>(__umul64hi(static_cast<uint64_t>(total) * i, A.ctas_inverse));
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Which of 32 drafted positions from j0 (negative: context) a row's token sees.
__device__ __noinline__ uint32_t row_sees(const uint8_t *mask, int token, int n, int j0) {
  if (!mask) {  // all up to itself
    const int most = min(token, n - 1) - j0 + 1;
    return most >= 32 ? ~0u : most <= 0 ? 0u : (1u << most) - 1;
  }
  uint32_t bits = 0;
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    const int j = j0 + e;
    const uint8_t x = j >= 0 && j < n ? __ldg(mask + j) : 0;
    bits |= j < 0 || x ? 1u << e : 0u;
  }
  return bits;
}

// 16-byte chunk index of a row in the K-major swizzle of its row length.
template <int D>
__device__ __forceinline__ int swizzled(int row, int chunk) {
  return D == 128 ? chunk ^ (row & 7) : chunk ^ (row >> 1 & 3);
}

// Two values in the rows' type, the first in the low half.
template <int DT>
__device__ __forceinline__ uint32_t pair_bits(float lo, float hi) {
  if constexpr (DT == SPEC_DTYPE_F16) return half2_bits(lo, hi);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A loading warp's way through its CTA's tiles: lane l < 8 has positions
// [16 l, 16 l + 16) of each; this tile's and the next one's.
struct TileWalk {
  const CacheTilePlan &A;
  const Requests &q;
  int row_tile, t, hi, lane, end;
  Unit u;
  bool more[2];                  // whether there is a tile
  int pos[2], page[2], head[2];  // pos -1: past the unit's positions; page -1: none, or outside the pool

  __device__ TileWalk(const CacheTilePlan &a, const Requests &r, int rt, int lo, int h, int l)
      : A(a), q(r), row_tile(rt), t(lo), hi(h), lane(l), end(lo), u{} {}
  __device__ __forceinline__ bool advance(int slot) {  // whether a new unit begins

    pos[slot] = page[slot] = -1;
    head[slot] = 0;
    more[slot] = t < hi;
    if (t >= hi) return false;
    const bool fresh = t >= end;
    if (fresh) {
      u = find_unit(A, q, row_tile, t);
      end = u.tile0 + u.tiles;
      t = max(t, u.tile0);
    }
    const int at = (t - u.tile0) * kTile + (lane & 7) * 16;  // (of all lanes it could pass an int at the longest contexts)
    head[slot] = u.head;
    if (lane < 8 && at < u.T) {
      pos[slot] = at;
      page[slot] = page_at(A.p.c, u.b, at >> A.p.c.page_shift);
    }
    ++t;
    return fresh;
  }
  __device__ __forceinline__ bool shift() {
    more[0] = more[1], pos[0] = pos[1], page[0] = page[1], head[0] = head[1];
    return advance(1);
  }
  // the blocks' scales; 1 where there is no block
  __device__ __forceinline__ void scales(int slot, float &k, float &v) const {
    k = v = 1.0f;
    if (page[slot] >= 0) {
      const int64_t at = page[slot] * A.p.c.scale_stride + head[slot];
      k = A.p.c.k_scale[at];
      v = A.p.c.v_scale[at];
    }
  }
};

// Row x = token * Hq + head of request b as one that sees nothing, by one thread.
template <int DT, int D>
__device__ void zero_row(const CacheAttendParams &P, int b, int x) {
  char *out = P.out + (b * P.os[0] + x / P.Hq * P.os[1] + x % P.Hq * P.os[2]) * 2;
  for (int d = 0; d < D; ++d) put_value<DT>(out, d, 0.0f);
  if (P.lse) P.lse[static_cast<int64_t>(b) * P.N * P.Hq + x] = -INFINITY;
}

// Waits for every copy and product that the CTA began.
__device__ __noinline__ void land_all(TileSmall &sm, int stages_k, int stages_v) {
  ring_land(sm.k_full, stages_k, sm.copies_k);
  ring_land(sm.v_full, stages_v, sm.copies_v);
  ring_land(sm.k_empty, stages_k, sm.products_s);
  ring_land(sm.s_full, 2, sm.products_s);
  ring_land(sm.pv_done, 2, sm.products_o);
}

template <int DT, int D, int REPL, bool CAP>
__global__ void __launch_bounds__(kTileThreads, 1)
    cache_attend_tile_kernel(const CacheTilePlan A, const __grid_constant__ CUtensorMap k_map) {
  using S = TileShape<DT, D>;
  constexpr int RT = 128 / REPL;        // rows to a unit
  constexpr int HALVES = REPL == 4 ? 1 : 2;  // warps to 32 lanes
  constexpr int OWN = kTile / REPL / HALVES;  // positions that a thread takes of each tile
  constexpr int kSoft = 128 * HALVES;         // softmax threads
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
      bar_init(&sm.s_full[i], 2);
      bar_init(&sm.s_empty[i], kSoft);
      bar_init(&sm.p_full[i], kSoft);
      bar_init(&sm.pv_done[i], 1);
      bar_init(&sm.o_free[i], kSoft);
    }
    bar_init(&sm.q_full, kSoft);
    bar_init(&sm.meet, kSoft);
    for (int i = 0; i < kRing; ++i) bar_init(&sm.ring_full[i], 32), bar_init(&sm.ring_empty[i], kSoft);
    bar_init_fence();
    sm.dead = 0;
    sm.begun = make_int4(-1, 0, 0, 0);
  }
  if (tid < 128) sm.spoiled[tid] = 0;
  if (warp == 14) tmem_alloc(&sm.tmem, kCols);
  // Every request's tiles, then their running sum.
  for (int b = tid; b < A.count; b += kTileThreads) {
    int base, n;
    const bool ok = request_lengths(P, A.first + b, base, n) == SPEC_STATUS_OK;
    sm.q.lens[b] = make_int2(base, n);
    const int tiles = ok ? request_tiles(A, RT, base, n) : 0;
    sm.q.per_head[b] = max(tiles, 1);
    sm.q.start[b + 1] = tiles * P.c.kv_heads;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    int carry = 0;
    for (int b0 = 0; b0 < A.count; b0 += 32) {
      int x = b0 + lane < A.count ? sm.q.start[b0 + lane + 1] : 0;
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
      }
      x += carry;
      if (b0 + lane < A.count) sm.q.start[b0 + lane + 1] = x;
      carry = __shfl_sync(~0u, x, 31);
    }
    if (lane == 0) sm.q.start[0] = 0;
  }
  __syncthreads();
  const int total = sm.q.start[A.count];
  const int lo = cut(A, total, ctas, cta);
  int hi = cut(A, total, ctas, cta + 1);
  if (hi < total) {  // a cut at or before a unit's first tile ends with the unit before
    const Unit u = find_unit(A, sm.q, RT, hi);
    if (hi <= u.tile0) hi = u.start;
  }
  const uint32_t tmem = sm.tmem;
  volatile int *dead = &sm.dead;

  if (warp == 10) {
    // ---- loading K: a lane to a group of 16 positions (the first 8 lanes), the page table two tiles ahead
    TileWalk walk(A, sm.q, RT, lo, hi, lane);
    walk.advance(0);
    walk.advance(1);
    int sk = 0, lap = 0;
    while (walk.more[0]) {
      const int pos = walk.pos[0], page = walk.page[0], head = walk.head[0];
      if (walk.shift()) [[unlikely]] {  // a unit some tiles ahead: its rows of q into L2, which the stream of keys keeps emptying
#pragma unroll 1
        for (int r = lane; r < walk.u.rows; r += 32) {
          const int row = walk.u.row0 + r, tok = by_group(A, row);
          const char *q = P.q + (walk.u.b * P.qs[0] + tok * P.qs[1] + (walk.u.head * P.group + row - tok * P.group) * P.qs[2]) * 2;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
          if (D == 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 128));
        }
      }
      const bool load = pos >= 0 && page >= 0 && (pos & (A.page_rows - 1)) == 0;
      const uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(~0u, load)) * A.page_rows * D);
      if (lap > 0 && !warp_wait(&sm.k_empty[sk], (lap - 1) & 1, dead)) break;
      if (lane == 0) bar_expect(&sm.k_full[sk], bytes);
      __syncwarp();
      if (load)
        tensor_load_3d(smem + S::kK + sk * S::kStage + lane * 16 * D, &k_map, 0,
                       (head << P.c.page_shift) + (pos & ((1 << P.c.page_shift) - 1)), page, &sm.k_full[sk]);
      if (++sk == S::kStagesK) sk = 0, ++lap;
    }
    sm.copies_k = lap * S::kStagesK + sk;
  } else if (warp == 11) {
    // ---- loading V and the blocks' scales, likewise; the scales one tile ahead
    TileWalk walk(A, sm.q, RT, lo, hi, lane);
    walk.advance(0);
    walk.advance(1);
    float ks, vs, ks1, vs1;
    walk.scales(0, ks, vs);
    int sv = 0, lap = 0;
    for (int i = 0; walk.more[0]; ++i) {
      const int r = i % kRing;
      const int pos = walk.pos[0], page = walk.page[0], head = walk.head[0];
      walk.scales(1, ks1, vs1);
      walk.shift();
      if (i >= kRing && !warp_wait(&sm.ring_empty[r], (i / kRing - 1) & 1, dead)) break;
      if (lane < 8) sm.ring[r][lane] = make_float4(ks, __log2f(vs), __fdividef(1.0f, vs), 0.0f);
      bar_arrive(&sm.ring_full[r]);
      const bool load = pos >= 0 && page >= 0 && (pos & (A.page_rows - 1)) == 0;
      const uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(~0u, load)) * A.page_rows * D);
      if (lap > 0 && !warp_wait(&sm.v_empty[sv], (lap - 1) & 1, dead)) break;
      if (lane == 0) bar_expect(&sm.v_full[sv], bytes);
      __syncwarp();
      if (load)
        bulk_load(smem + S::kV8 + sv * S::kStage + lane * 16 * D,
                  P.c.v + block_offset(P.c, page, head) + static_cast<int64_t>(pos & ((1 << P.c.page_shift) - 1)) * D, A.page_rows * D,
                  &sm.v_full[sv]);
      ks = ks1, vs = vs1;
      if (++sv == S::kStagesV) sv = 0, ++lap;
    }
    sm.copies_v = lap * S::kStagesV + sv;
  } else if (warp == 14) {
    // ---- issuing S = Q K^T
    constexpr uint32_t kId = mma_desc(kTile, false);
    constexpr uint64_t kSw = D == 128 ? kSwizzle128 : kSwizzle64;
    const uint64_t q_desc = matrix_desc(smem_u32(smem + S::kQ), 16, 8 * D, kSw);
    const uint64_t k_desc = matrix_desc(smem_u32(smem + S::kK), 16, 8 * D, kSw);
    int unit_end = lo, units = 0, i = 0, sk = 0, lap = 0;
    for (int t = lo; t < hi; ++t, ++i) {
      if (t >= unit_end) {
        const Unit u = find_unit(A, sm.q, RT, t);
        unit_end = u.tile0 + u.tiles;
        t = max(t, u.tile0);
        if (!warp_wait(&sm.q_full, units & 1, dead)) break;
        ++units;
      }
      if (i >= 2 && !warp_wait(&sm.s_empty[i & 1], (i / 2 - 1) & 1, dead)) break;
      if (!warp_wait(&sm.ring_full[i % kRing], (i / kRing) & 1, dead)) break;
      if (lane == 0) bar_arrive(&sm.s_full[i & 1]);  // (with this arrival S full says that the tile's scales are there too)
      if (!warp_wait(&sm.k_full[sk], lap & 1, dead)) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int piece = 0; piece < S::kPieces; ++piece)
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            mma_f8(tmem + (i & 1) * 128, q_desc + ((piece * kTile * D + k * 32) >> 4), k_desc + ((sk * S::kStage + k * 32) >> 4), kId,
                   piece + k > 0);
        tc_commit(&sm.k_empty[sk]);
        tc_commit(&sm.s_full[i & 1]);
      }
      __syncwarp();
      if (++sk == S::kStagesK) sk = 0, ++lap;
    }
    sm.products_s = i;
  } else if (warp == 15) {
    // ---- issuing O += P V
    constexpr uint32_t kId = mma_desc(D, true);
    const uint64_t v_desc = matrix_desc(smem_u32(smem + S::kV16), kTile * 128, 1024, kSwizzle128);
    int unit_end = lo, units = 0, i = 0;
    for (int t = lo; t < hi; ++t, ++i) {
      const int w = i & 1;
      const bool fresh = t >= unit_end;
      if (fresh) {
        const Unit u = find_unit(A, sm.q, RT, t);
        unit_end = u.tile0 + u.tiles;
        t = max(t, u.tile0);
        if (units > 0 && !warp_wait(&sm.o_free[(units - 1) & 1], (units - 1) >> 1 & 1, dead)) break;
        ++units;
      }
      if (!warp_wait(&sm.w_full[w], (i >> 1) & 1, dead)) break;
      if (!warp_wait(&sm.p_full[w], (i >> 1) & 1, dead)) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_f16_ta(tmem + kO, tmem + kP + w * 64 + k * 8, v_desc + ((w * 2 * S::kStage + k * 2048) >> 4), kId, !(fresh && k == 0));
        tc_commit(&sm.pv_done[w]);
      }
      __syncwarp();
    }
    sm.products_o = i;
  } else if (warp >= 8) {
    // ---- widening V: 16 bytes of a position to 16 halves, in the MN-major layout of the operand
    const int w4 = (warp >> 1 & 2) | (warp & 1), wide = w4 * 32 + lane;  // warps 8, 9, 12, 13
    for (int b = cta; b < A.count; b += ctas) {  // and, on the way, the page tables: a request with a bad page gives nothing
      int base, n;
      int st = request_lengths(P, A.first + b, base, n);
      int bad = 0;
      if (st == SPEC_STATUS_OK)
        for (int j = wide; static_cast<int64_t>(j) << P.c.page_shift < base + n; j += 128) bad |= page_at(P.c, A.first + b, j) < 0;
      if (wide == 0) A.verdict[b] = st;
      asm volatile("bar.sync 2, 128;" ::: "memory");
      if (bad) A.verdict[b] = SPEC_STATUS_BAD_PAGE;
      // rows that no unit covers
      for (int x = wide + (st == SPEC_STATUS_OK ? n : 0) * P.Hq; x < P.N * P.Hq; x += 128) zero_row<DT, D>(P, A.first + b, x);
    }
    int unit_end = lo;
    Unit u{};
    // 16 bytes of a position to a lane, 4 or 8 positions to a step.  Eight lanes in a row take 64 bytes of each of two positions
    // (of different halves of them when a position has 128), so neither their loads nor their swizzled stores share a bank;
    // every step's addresses are a lane's own plus a constant.
    constexpr int kPer = 512 / D;
    const int part = lane & 3, sub = D == 128 ? (lane >> 4) * 2 + (lane >> 2 & 1) : lane >> 2;
    const int group = D == 128 ? (lane >> 3 & 1) ^ (lane >> 2 & 1) : 0;  // 64 columns
    const int from = (w4 * 32 + sub) * D + group * 64 + part * 16;
    const int to = group * (kTile * 128) + w4 * 4096 + sub * 128 + ((part * 2 ^ sub) << 4);
    int unit = -1, ended1 = -1, ended2 = -1;  // this unit's number; the unit that tile i - 1, i - 2 closed, or -1
    for (int t = lo, i = 0, sv = 0, lap = 0; t < hi; ++t, ++i) {
      const int w = i & 1;
      if (t >= unit_end) {
        u = find_unit(A, sm.q, RT, t);
        unit_end = u.tile0 + u.tiles;
        t = max(t, u.tile0);
        ++unit;
      }
      const int pos0 = (t - u.tile0) * kTile;
      const bool edge = pos0 + kTile > u.base;
      if (i >= 2 && !warp_wait(&sm.pv_done[w], (i / 2 - 1) & 1, dead)) break;
      // (a unit's end goes through the halves of its last tile, two tiles before the ones to replace them)
      if (ended2 >= 0 && !warp_wait(&sm.o_free[ended2 & 1], ended2 >> 1 & 1, dead)) break;
      ended2 = ended1;
      ended1 = t + 1 == unit_end ? unit : -1;
      if (!warp_wait(&sm.v_full[sv], lap & 1, dead)) break;
      const char *src = smem + S::kV8 + sv * S::kStage;
      char *dst = smem + S::kV16 + w * 2 * S::kStage;
      uint32_t poison = 0;
      auto widen = [&](uint4 x, int step) {
        uint4 h[2];
        uint32_t *o = reinterpret_cast<uint32_t *>(h);
        const uint32_t in[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const __half2 a = e4m3x2_to_half2(in[c] & 0xffff), b = e4m3x2_to_half2(in[c] >> 16);
          o[2 * c] = *reinterpret_cast<const uint32_t *>(&a);
          o[2 * c + 1] = *reinterpret_cast<const uint32_t *>(&b);
        }
        // eight positions: 1024 bytes; 16-byte chunks swizzled by the position in them (in the upper four: 4 more)
        const int at = D == 128 ? (to ^ (step & 1) << 6) + (step >> 1) * 1024 + (step & 1) * 512 : to + step * 1024;
        *reinterpret_cast<uint4 *>(dst + at) = h[0];
        *reinterpret_cast<uint4 *>(dst + (at ^ 16)) = h[1];
      };
      constexpr int kSteps = 32 / kPer;
      if (!edge) [[likely]] {
#pragma unroll
        for (int step = 0; step < kSteps; step += 4) {
          uint4 x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = *reinterpret_cast<const uint4 *>(src + from + (step + k) * kPer * D);
#pragma unroll
          for (int k = 0; k < 4; ++k) widen(x[k], step + k);
        }
      } else {  // nothing past the last position, and no NaN where a row may not look
#pragma unroll 1
        for (int step = 0; step < kSteps; ++step) {
          const int pos = pos0 + w4 * 32 + step * kPer + sub;
          uint4 x = *reinterpret_cast<const uint4 *>(src + from + step * kPer * D);
          bool nan = false;
          if (pos >= u.T) x = make_uint4(0, 0, 0, 0);
          else if (pos >= u.base) {
            uint32_t *e = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              // bytes of 0x7f under the sign: 0x80 after adding one
              const uint32_t hit = ((e[c] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
              nan |= hit != 0;
              e[c] &= ~(hit | (hit - (hit >> 7)));
            }
          }
          const uint32_t vote = __ballot_sync(~0u, nan);
#pragma unroll
          for (int c = 0; c < kPer; ++c) {
            const uint32_t lanes_of = D == 128 ? (c & 1 ? 0xf0f0u : 0x0f0fu) << (c >> 1) * 16 : 0xfu << c * 4;
            if (vote & lanes_of) poison |= 1u << (step * kPer + c);
          }
          widen(x, step);
        }
      }
      if (edge && lane == 0) sm.poison[w][w4] = poison;
      fence_async_shared();
      bar_arrive(&sm.v_empty[sv]);
      bar_arrive(&sm.w_full[w]);
      if (++sv == S::kStagesV) sv = 0, ++lap;
    }
  } else if (warp < 4 * HALVES) {
    // ---- softmax: one or two threads to a row (of its copy), each with OWN positions of each tile
    const int half = warp >> 2, quarter = warp & 3;
    const int spot = quarter * 32 + lane;                  // lane of tensor memory
    const int copy = spot / RT, r = spot % RT;             // which copy of the rows, and the row
    const int col0 = (copy * HALVES + half) * OWN;          // its positions in the tile
    const uint32_t lanes = static_cast<uint32_t>(quarter) << 21;
    if (REPL > 1) {
      const uint32_t zero[16] = {};
      for (int c = half * 64; c < 64 * (HALVES == 1 ? 2 : half + 1); c += 16) tmem_st16(tmem + lanes + kP + c, zero);
      tc_wait_st();
      tc_fence_before();
    }
    const bool negative = P.scale < 0.0f;
    bool ok = true;
    uint32_t meetings = 0;
    auto together = [&] {  // a barrier of the eight warps, bounded like every wait
      bar_arrive(&sm.meet);
      return warp_wait(&sm.meet, meetings++ & 1, dead);
    };
    // The number-th unit's rows of q as e4m3 pieces; every earlier score product that reads them has completed.
    auto write_q = [&](const Unit &u, int number) {
      constexpr int kEach = D / 32, kWarpsQ = 4 * HALVES;  // elements to a lane
      // Four rows side by side in a loop that is not unrolled: its instructions are fetched once, and fetching is what a unit's
      // start and end spend most on.  (Rows past the last one repeat it.)
#pragma unroll 1
      for (int first = warp; first < u.rows; first += 4 * kWarpsQ) {
        float x[4][kEach], top[4];
        int ex[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = u.row0 + min(first + k * kWarpsQ, u.rows - 1), tok = by_group(A, row);
          const char *q = P.q + (u.b * P.qs[0] + tok * P.qs[1] + (u.head * P.group + row - tok * P.group) * P.qs[2]) * 2;
          if (A.q_vec) [[likely]] {
            unpack_each<DT, kEach>(raw_each<kEach>(q, lane), x[k]);
          } else {
#pragma unroll
            for (int e = 0; e < kEach; ++e) x[k][e] = row_value<DT>(q, lane * kEach + e);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          top[k] = 0.0f;
#pragma unroll
          for (int e = 0; e < kEach; ++e) {
            if (negative) x[k][e] = -x[k][e];
            top[k] = fmaxf(top[k], finite_abs(x[k][e]));
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
          for (int k = 0; k < 4; ++k) top[k] = fmaxf(top[k], __shfl_xor_sync(~0u, top[k], o));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // 2^ex with top / 2^ex in [128, 256)
          ex[k] = top[k] > 0.0f ? max(static_cast<int>(__float_as_uint(top[k]) >> 23) - 127 - 7, -110) : 0;
          const float down = __uint_as_float(static_cast<uint32_t>(127 - ex[k]) << 23);
#pragma unroll
          for (int e = 0; e < kEach; ++e) x[k][e] *= down;
        }
#pragma unroll
        for (int piece = 0; piece < S::kPieces; ++piece) {
          uint32_t code[4] = {};
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < kEach; e += 2) {
              const uint32_t two = to_e4m3x2(x[k][e], x[k][e + 1]);
              const float2 back = e4m3x2_to_float2(two);
              x[k][e] -= back.x;
              x[k][e + 1] -= back.y;
              code[k] |= two << (8 * e);
            }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int r0 = first + kWarpsQ * k;
            if (r0 >= u.rows) continue;
#pragma unroll
            for (int c = 0; c < REPL; ++c) {
              const int a = c * RT + r0;
              char *to = smem + S::kQ + piece * kTile * D + a * D + (swizzled<D>(a, lane * kEach >> 4) << 4) + (lane * kEach & 15);
              if (kEach == 4) *reinterpret_cast<uint32_t *>(to) = code[k];
              else *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(code[k]);
            }
          }
        }
        const int mine = first + kWarpsQ * lane;
        if (lane < 4 && mine < u.rows) {
          const int e = lane == 0 ? ex[0] : lane == 1 ? ex[1] : lane == 2 ? ex[2] : ex[3];
          sm.row_factor[number & 1][mine] = fmaxf(fabsf(P.scale) * kLog2e * __uint_as_float(static_cast<uint32_t>(e + 127) << 23), 1e-30f);
        }
      }
      fence_async_shared();
      bar_arrive(&sm.q_full);
      return together();
    };
    int unit = 0;
    Unit next{};
    if (lo < hi) {
      next = find_unit(A, sm.q, RT, lo);
      ok = write_q(next, 0);
    }
    for (int t = lo, i = 0; t < hi && ok;) {
      const Unit u = next;
      t = max(t, u.tile0);
      const int t_begin = t, t_end = min(hi, u.tile0 + u.tiles);
      const bool live = r < u.rows;
      const float factor = live ? sm.row_factor[unit & 1][r] : 0.0f;
      const int token = live ? by_group(A, u.row0 + r) : 0;
      const uint8_t *mask = P.mask ? P.mask + (static_cast<int64_t>(u.b) * P.N + token) * P.N : nullptr;
      const float cap2 = P.softcap * kLog2e;                // the cap in units of log 2
      const float in_cap = CAP ? 1.0f / cap2 : 0.0f;
      float m = -INFINITY, sum = 0.0f;

      for (; t < t_end; ++t, ++i) {
        const int sb = i & 1, ring = i % kRing;
        const int pos0 = (t - u.tile0) * kTile + col0;
        const bool edge = pos0 + OWN > u.base;
        if (!(ok = warp_wait(&sm.s_full[sb], (i >> 1) & 1, dead))) break;
        tc_fence_after();
        float x[OWN];
        if (OWN == 16) {
          tmem_ld16(tmem + lanes + sb * 128 + col0, x);
        } else {
#pragma unroll
          for (int c = 0; c < OWN; c += 32) tmem_ld32(tmem + lanes + sb * 128 + col0 + c, x + c);
        }
        float4 sc[(OWN + 15) / 16];
#pragma unroll
        for (int g = 0; g < (OWN + 15) / 16; ++g) sc[g] = sm.ring[ring][col0 / 16 + g];
        tc_wait_ld();
        tc_fence_before();
        bar_arrive(&sm.s_empty[sb]);
        bar_arrive(&sm.ring_empty[ring]);

        // x f is the score in units of log 2; with a cap it is formed here
        if (CAP) {
#pragma unroll
          for (int g = 0; g < OWN / 16; ++g) {
            const float f = factor * sc[g].x;
#pragma unroll
            for (int e = 0; e < 16; ++e) x[g * 16 + e] *= f;
            cap_scores<16>(x + g * 16, in_cap, cap2);
          }
        }
        uint32_t sees[(OWN + 31) / 32];
        if (edge) [[unlikely]] {  // (the factor below is never 0, so -inf stays -inf)
#pragma unroll
          for (int c = 0; c < (OWN + 31) / 32; ++c) {
            sees[c] = live ? row_sees(mask, token, u.n, pos0 + c * 32 - u.base) : 0;
#pragma unroll
            for (int e = 0; e < (OWN < 32 ? OWN : 32); ++e)
              if (!(sees[c] >> e & 1)) x[c * 32 + e] = -INFINITY;
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int g = 0; g < OWN / 16; ++g) {
          float high = fmaxf(x[g * 16], x[g * 16 + 1]);
#pragma unroll
          for (int e = 2; e < 16; e += 2) high = fmaxf(high, fmaxf(x[g * 16 + e], x[g * 16 + e + 1]));
          top = fmaxf(top, fmaf(high, CAP ? 1.0f : fmaxf(factor * sc[g].x, 1.2e-38f), sc[g].y));
        }
        // the two threads of a row agree on its maximum
        if (HALVES == 2) {
          sm.tops[sb][half][spot] = top;
          asm volatile("bar.sync %0, 64;" ::"r"(3 + quarter) : "memory");
          top = fmaxf(top, sm.tops[sb][1 - half][spot]);
        }
        // the reference, and O with it when it moves
        const bool moves = live && top > m + 8.0f;
        if (__any_sync(~0u, moves)) [[unlikely]] {
          const float next_m = moves ? top : m;
          const float keep = m == -INFINITY ? 0.0f : ex2(m - next_m);
          m = next_m;
          sum *= keep;
          const int done = i - 1;
          if (t > t_begin) {
            if (!(ok = warp_wait(&sm.pv_done[done & 1], (done >> 1) & 1, dead))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = half * (D / HALVES); c < (half + 1) * (D / HALVES); c += 16) {
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
        const float ref = m == -INFINITY ? 0.0f : m;
        uint32_t p[OWN / 2];
#pragma unroll
        for (int g = 0; g < OWN / 16; ++g) {
          const float shift = sc[g].y - ref + 7.0f, f = CAP ? 1.0f : fmaxf(factor * sc[g].x, 1.2e-38f);
          // two positions to an instruction, except the exponentials and their rounding
          const float2 f2 = make_float2(f, f), shift2 = make_float2(shift, shift);
          float2 part[2] = {};
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float2 y = __ffma2_rn(make_float2(x[g * 16 + e], x[g * 16 + e + 1]), f2, shift2);
            const float2 z = make_float2(ex2(y.x), ex2(y.y));
            part[e >> 1 & 1] = __fadd2_rn(part[e >> 1 & 1], z);
            p[g * 8 + e / 2] = half2_bits(z.x, z.y);
          }
          const float2 both = __fadd2_rn(part[0], part[1]);
          sum = fmaf(both.x + both.y, sc[g].z, sum);
        }
        if (i >= 2 && !(ok = warp_wait(&sm.pv_done[sb], (i / 2 - 1) & 1, dead))) break;  // P's columns are free
        tc_fence_after();
        if (OWN == 16) tmem_st8(tmem + lanes + kP + sb * 64 + col0 / 2, p);
#pragma unroll
        for (int c = 0; c + 16 <= OWN / 2; c += 16) tmem_st16(tmem + lanes + kP + sb * 64 + col0 / 2 + c, p + c);
        if (edge) [[unlikely]] {  // a row that sees a position whose V was NaN
          if (!(ok = warp_wait(&sm.w_full[sb], (i >> 1) & 1, dead))) break;
          uint32_t bad = 0;
#pragma unroll
          for (int c = 0; c < (OWN + 31) / 32; ++c) {
            const uint32_t at = sm.poison[sb][col0 / 32 + c] >> (OWN < 32 ? col0 & 31 : 0);
            bad |= sees[c] & (OWN < 32 ? at & ((1u << OWN) - 1) : at);
          }
          if (bad) sm.spoiled[r] = 1;
        }
        tc_wait_st();
        tc_fence_before();
        bar_arrive(&sm.p_full[sb]);
      }
      if (!ok) break;

      // the next unit's q, while this one's last values are being summed
      if (t < hi) {
        next = find_unit(A, sm.q, RT, t);
        if (!(ok = write_q(next, unit + 1))) break;
      }
      // The unit's end in this CTA: the rows' sums over copies and halves, and what each copy's O is multiplied by.
      const bool whole = t_begin == u.tile0 && t == u.tile0 + u.tiles;
      const int slot = cta * 2 + (unit > 0 ? 1 : 0);  // (only a CTA's first unit and its last can be cut)
      sm.ml[half][spot] = make_float2(m, sum);
      if (!(ok = together())) break;
      if (tid < u.rows) {
        float m_all = -INFINITY, l_all = 0.0f;
#pragma unroll
        for (int c = 0; c < REPL; ++c) m_all = fmaxf(m_all, sm.ml[0][c * RT + tid].x);
        const float ref = m_all == -INFINITY ? 0.0f : m_all;
#pragma unroll
        for (int c = 0; c < REPL; ++c)
          l_all += (sm.ml[0][c * RT + tid].y + (HALVES == 2 ? sm.ml[1][c * RT + tid].y : 0.0f)) * ex2(sm.ml[0][c * RT + tid].x - ref);
        float norm = 1.0f;
        const int row = u.row0 + tid, tok = by_group(A, row), h = u.head * P.group + row - tok * P.group;
        if (whole) {
          norm = l_all == 0.0f ? 0.0f : __fdividef(1.0f, l_all);
          if (P.lse)
            P.lse[(static_cast<int64_t>(u.b) * P.N + tok) * P.Hq + h] = l_all == 0.0f ? -INFINITY : (m_all - 7.0f + __log2f(l_all)) * kLn2;
          sm.out_at[tid] = u.b * P.os[0] + tok * P.os[1] + h * P.os[2];
        } else {
          A.ml[static_cast<int64_t>(slot) * RT + tid] = make_float2(m_all, l_all);
          if (tid == 0 && t_begin == u.tile0) sm.begun = make_int4(u.b - A.first, u.head << 8 | u.rows, u.row0 * 2 + (slot & 1), u.tile0 + u.tiles);
        }
        if (sm.spoiled[tid]) norm = NAN;
        sm.spoiled[tid] = 0;
#pragma unroll
        for (int c = 0; c < REPL; ++c) sm.weight[c * RT + tid] = norm * ex2(sm.ml[0][c * RT + tid].x - ref);
      }
      const int last = i - 1;
      if (!(ok = warp_wait(&sm.pv_done[last & 1], (last >> 1) & 1, dead))) break;
      tc_fence_after();
      if (!(ok = together())) break;
      const float w_own = live ? sm.weight[spot] : 0.0f;
      // Partial rows lie column by column, four at a time, so that a warp's rows are side by side: [D / 4][RT].
      float4 *part = reinterpret_cast<float4 *>(A.part) + static_cast<int64_t>(slot) * RT * (D / 4);
      if (REPL == 1 && !whole) {
#pragma unroll 1
        for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
          float o[16];
          tmem_ld16(tmem + lanes + kO + c, o);
          tc_wait_ld();
          if (live)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              part[(c / 4 + e) * RT + r] = make_float4(o[4 * e] * w_own, o[4 * e + 1] * w_own, o[4 * e + 2] * w_own, o[4 * e + 3] * w_own);
        }
      } else {
        // 64 columns at a time, over the halves of the last tile (its product is done): [128][16 chunks of 4], swizzled by the row
        float4 *fold = reinterpret_cast<float4 *>(smem + S::kV16 + (last & 1) * 2 * S::kStage);
        constexpr int kFoldCols = D == 128 ? 64 : 32;
        constexpr int kChunks = kFoldCols / 4;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += kFoldCols) {
          if (c0 > 0 && !(ok = together())) break;  // the columns before have been read
#pragma unroll 1
          for (int c = half * (kFoldCols / HALVES); c < (half + 1) * (kFoldCols / HALVES); c += 16) {
            float o[16];
            tmem_ld16(tmem + lanes + kO + c0 + c, o);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 4; ++e)
              fold[spot * kChunks + ((c / 4 + e) ^ (spot & (kChunks - 1)))] =
                  make_float4(o[4 * e] * w_own, o[4 * e + 1] * w_own, o[4 * e + 2] * w_own, o[4 * e + 3] * w_own);
          }
          if (!(ok = together())) break;
          auto folded = [&](int rr, int chunk) {
            float4 y = fold[rr * kChunks + (chunk ^ (rr & (kChunks - 1)))];
#pragma unroll
            for (int k = 1; k < REPL; ++k) {
              const int row = k * RT + rr;
              const float4 z = fold[row * kChunks + (chunk ^ (row & (kChunks - 1)))];
              y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
            }
            return y;
          };
          if (whole) {
            for (int x = tid; x < u.rows * kChunks; x += kSoft) {
              const int rr = x / kChunks, c = c0 + x % kChunks * 4;
              const float4 y = folded(rr, x % kChunks);
              char *out = P.out + sm.out_at[rr] * 2;
              if (A.out_vec) {
                *reinterpret_cast<uint2 *>(out + c * 2) = make_uint2(pair_bits<DT>(y.x, y.y), pair_bits<DT>(y.z, y.w));
              } else {
                put_value<DT>(out, c, y.x), put_value<DT>(out, c + 1, y.y), put_value<DT>(out, c + 2, y.z), put_value<DT>(out, c + 3, y.w);
              }
            }
          } else {
            for (int x = tid; x < RT * kChunks; x += kSoft)
              if (x % RT < u.rows) part[(c0 / 4 + x / RT) * RT + x % RT] = folded(x % RT, x / RT);
          }
        }
      }
      if (!ok) break;
      tc_fence_before();
      bar_arrive(&sm.o_free[unit & 1]);
      ++unit;
      ok = together();  // the shared arrays have been read
    }
    if (!ok) tc_wait_st();  // (a warp that gave up may have stores to tensor memory in flight)
    // a warp that gave up lets its partner, which may be waiting for its maxima, go on to give up too
    if (HALVES == 2 && !ok) asm volatile("bar.arrive %0, 64;" ::"r"(3 + quarter) : "memory");
  }
  tc_fence_before();
  __syncthreads();
  if (*dead) [[unlikely]] {  // nothing that was begun may reach shared or tensor memory that the CTA has left (else all was waited for)
    if (warp == 0) land_all(sm, S::kStagesK, S::kStagesV);
    __syncthreads();
  }
  pdl_launch_dependents();  // (not earlier: the merge's blocks would crowd onto the SMs that finish first)
  if (tid == 0) {
    A.range[cta] = make_int2(lo, sm.dead);
    A.begun[cta] = sm.begun;
  }
  if (warp == 14) {
    tc_fence_after();
    tmem_free(tmem, kCols);
  }
}

// Joins the partial sums of the units that more than one CTA worked on: block
// (c, j) takes 32 rows, a lane each, of the unit that CTA c began and a later
// one ended, each warp an eighth of the columns.  The last blocks set the
// requests' status, and clear the outputs of those with a bad page.  It lasts
// about as long as its instructions take to arrive, so there are few, and few
// loads wait for one another.
template <int DT, int D>
__global__ void __launch_bounds__(256) cache_attend_merge_kernel(const CacheTilePlan A, int row_tile, int ctas) {
  const CacheAttendParams &P = A.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kOwn = D / 32;  // float4s of a row to a warp
  pdl_wait();
  const int chunks = row_tile >> 5, shift = chunks >> 1;  // (1, 2 or 4)
  if (static_cast<int>(blockIdx.x) >= ctas * chunks) {
    const int bl = (blockIdx.x - ctas * chunks) * 8 + warp, b = A.first + bl;
    if (bl >= A.count) return;
    int st = A.verdict[bl];
    bool gone = false;
    for (int c = lane; c < ctas; c += 32) gone |= A.range[c].y != 0;
    if (__any_sync(~0u, gone)) st = SPEC_STATUS_TIMEOUT;
    if (lane == 0 && P.status) P.status[b] = st;
    if (st == SPEC_STATUS_BAD_PAGE || st == SPEC_STATUS_TIMEOUT)
      for (int x = lane; x < P.N * P.Hq; x += 32) zero_row<DT, D>(P, b, x);
    return;
  }
  const int c0 = blockIdx.x >> shift, r = (blockIdx.x & (chunks - 1)) * 32 + lane;
  const int4 unit = A.begun[c0];  // request, head << 8 | rows, 2 * first row + c0's slot, end of its tiles
  if (unit.x < 0) return;
  const int verdict = A.verdict[unit.x];
  // the last CTA that begins before the unit's end
  int later = 0;
  for (int c = c0 + 1; c < ctas; c += 160) {
#pragma unroll
    for (int k = 0; k < 5; ++k) later += c + k * 32 + lane < ctas && A.range[c + k * 32 + lane].x < unit.w ? 1 : 0;
  }
  later = __reduce_add_sync(~0u, later);
  const int rows = unit.y & 255, from = min(r, rows - 1);  // (rows that are not there would be read from DRAM: nothing wrote them)
  const bool live = r < rows;
  if ((r & ~31) >= rows) return;
  float m = -INFINITY, sum = 0.0f;
  float4 acc[kOwn];
#pragma unroll
  for (int e = 0; e < kOwn; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  // four CTAs' parts at a time (past the last one: that one again, without weight)
#pragma unroll 1
  for (int k = 0; k <= later; k += 4) {
    float2 ml[4];
    float4 o[4][kOwn];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = c0 + min(k + q, later), slot = c * 2 + (c == c0 ? unit.z & 1 : 0);
      ml[q] = A.ml[slot * row_tile + from];
      const float4 *part = reinterpret_cast<const float4 *>(A.part) + (static_cast<int64_t>(slot) * (D / 4) + warp * kOwn) * row_tile + from;
#pragma unroll
      for (int e = 0; e < kOwn; ++e) o[q][e] = part[e * row_tile];
    }
    const float top = fmaxf(fmaxf(fmaxf(m, ml[0].x), ml[1].x), fmaxf(ml[2].x, ml[3].x)), ref = top == -INFINITY ? 0.0f : top;
    const float keep = ex2(m - ref);
    m = top;
    sum *= keep;
#pragma unroll
    for (int e = 0; e < kOwn; ++e) acc[e].x *= keep, acc[e].y *= keep, acc[e].z *= keep, acc[e].w *= keep;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (k + q > later) break;
      const float w = ex2(ml[q].x - ref);
      sum = fmaf(ml[q].y, w, sum);
#pragma unroll
      for (int e = 0; e < kOwn; ++e) {
        acc[e].x = fmaf(o[q][e].x, w, acc[e].x);
        acc[e].y = fmaf(o[q][e].y, w, acc[e].y);
        acc[e].z = fmaf(o[q][e].z, w, acc[e].z);
        acc[e].w = fmaf(o[q][e].w, w, acc[e].w);
      }
    }
  }
  if (!live || verdict != SPEC_STATUS_OK) return;
  const int b = A.first + unit.x, row = (unit.z >> 1) + r, i = by_group(A, row), h = (unit.y >> 8) * P.group + row - i * P.group;
  char *out = P.out + (b * P.os[0] + i * P.os[1] + h * P.os[2]) * 2;
  const float inv = sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
#pragma unroll
  for (int e = 0; e < kOwn; ++e) {
    const int d = (warp * kOwn + e) * 4;
    if (A.out_vec) [[likely]] {
      *reinterpret_cast<uint2 *>(out + d * 2) =
          make_uint2(pair_bits<DT>(acc[e].x * inv, acc[e].y * inv), pair_bits<DT>(acc[e].z * inv, acc[e].w * inv));
    } else {
      put_value<DT>(out, d, acc[e].x * inv), put_value<DT>(out, d + 1, acc[e].y * inv);
      put_value<DT>(out, d + 2, acc[e].z * inv), put_value<DT>(out, d + 3, acc[e].w * inv);
    }
  }
  if (warp == 0 && P.lse)
    P.lse[(static_cast<int64_t>(b) * P.N + i) * P.Hq + h] = sum == 0.0f ? -INFINITY : (m - 7.0f + __log2f(sum)) * kLn2;
}

// Devices on which a kernel may already use its shared memory.
template <int DT, int D, int REPL, bool CAP>
std::atomic<uint64_t> big_smem{0};

template <int DT, int D, int REPL>
cudaError_t launch_tiles(const CacheTilePlan &A, const CUtensorMap &map, cudaStream_t st) {
  using S = TileShape<DT, D>;
  auto kern = A.p.softcap > 0.0f ? cache_attend_tile_kernel<DT, D, REPL, true> : cache_attend_tile_kernel<DT, D, REPL, false>;
  cudaError_t e = once_per_device([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes); },
                                  A.p.softcap > 0.0f ? big_smem<DT, D, REPL, true> : big_smem<DT, D, REPL, false>);
  if (e != cudaSuccess) return e;
  const int ctas = device_sm_count();
  e = trace_launch("cache_attend_tile", st, [&] { kern<<<ctas, kTileThreads, S::kBytes, st>>>(A, map); });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas * (128 / REPL / 32) + (A.count + 7) / 8));
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
cudaError_t launch_tiles(const CacheTilePlan &A, const CUtensorMap &map, int copies, cudaStream_t st) {
  if (copies == 4) return launch_tiles<DT, D, 4>(A, map, st);
  if (copies == 2) return launch_tiles<DT, D, 2>(A, map, st);
  return launch_tiles<DT, D, 1>(A, map, st);
}

}  // namespace
}  // namespace sv
