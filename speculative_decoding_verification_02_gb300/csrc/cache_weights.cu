// spec_cache_weights: the attention weight that each cached token received.
//
//   out_j = prev_j + sum over rows of exp(x_rj - lse_r)
//
// A thread owns a position, so the sum is over a thread's own registers, in
// the rows' order: no atomics, the same bits on every run.  Heads of 64 and 128
// take the scores from the tensor cores (cache_weights_tile_kernel), other
// widths a dot product to a thread.
#include <algorithm>
#include <atomic>

#include "cache.cuh"
#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"

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
        s_lse[e / D] = P.lse[b * P.ls[0] + t * P.ls[1] + h * P.ls[2]] * kLog2e;
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

// ---------------------------------------------------------------- tensor cores
//
// S^T = K Q^T by kind::f8f6f4: 128 positions are the operand's rows, straight
// from the pool, and the query rows its columns, so that a position's scores
// are all in one lane of tensor memory.  A row of q, scaled by a power of two
// to at most 256, is the sum of e4m3 numbers x0 + x1 / 16 + x2 / 256 (the last
// for fp16 alone), each a column of its own: nothing is lost of a bf16, and
// what is left of small elements is 2^-14 against a largest of 128 or more.
//
// The tiles of all (request, head) units are laid end to end and cut evenly
// over the CTAs, a unit's start counting as some tiles.  Rows are taken 64 at a
// time (the operand holds as many as there are, in sixteens); further rows of a
// unit go over its tiles again, adding to what is there.  A tile is 256
// positions, two operands of 128, a side of four warps to each: with 128 to a
// tile the loading and the issuing warp took longer over one (about 900 cycles,
// most of them waits that were over already) than its bytes take to arrive.
// Bound by reading K (head_dim bytes a position and kv head) for few rows, by
// the exponentials for many.  One row over 131,068 positions, 8 heads of 128:
// 30 us, 4.7 TB/s; 64 requests of up to 5,000 positions, 20 rows on average:
// 67 us, a third of it the units' starts.  1 us of each is the status's own
// kernel, which a call without a status does not launch.

constexpr int kTile = 256;      // positions to a tile
constexpr int kThreads = 320;  // two sides of 4 summing warps, 1 loading, 1 issuing
constexpr int kRing = 8;
constexpr int kMaxRows = 64;   // rows at a time
constexpr int kUnitCost = 4;   // what a unit costs besides its tiles, in tiles
constexpr int kNoRow = -2147483647 - 1;  // the place of a row that sees no position

template <int DT, int D>
struct WeightShape {
  static constexpr int kPieces = DT == SPEC_DTYPE_BF16 ? 2 : 3;
  static constexpr int kStage = kTile * D;
  static constexpr int kStages = D == 128 ? 4 : 6;
  static constexpr int kQ = 0;
  static constexpr int kK = kPieces * kMaxRows * D;
  static constexpr int kSmall = kK + kStages * kStage;
  static constexpr int kBytes = kSmall + 8192 + 1024;
};

struct WeightSmall {
  int start[kTileRequests + 1];  // running sum of the requests' tiles
  int2 lens[kTileRequests];      // context, rows
  alignas(16) float2 row[kMaxRows];          // factor of a row's scores, its lse negated; both in units of log 2
  int token[kMaxRows];           // its place behind the context; kNoRow: adds nothing
  float ring[kRing][16];         // k_scale of 16 positions
  uint64_t k_full[6], k_empty[6], s_full[2], s_empty[2], q_full, meet, ring_full[kRing], ring_empty[kRing];
  uint32_t tmem;
  int bad[2], dead;
  int copies, products;  // how many were begun
};
static_assert(sizeof(WeightSmall) <= 8192);

struct WeightUnit {
  int b, head, base, cnt, T, start, tile0, tiles;  // b: within the launch; start: its place, kUnitCost before its tiles
};

__device__ __noinline__ WeightUnit weight_unit(const WeightSmall &sm, int count, int heads, int t) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (sm.start[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  WeightUnit u;
  u.b = lo;
  u.base = sm.lens[lo].x;
  u.cnt = sm.lens[lo].y;
  u.T = u.base + u.cnt;
  u.tiles = (u.T + kTile - 1) / kTile;
  const int span = u.tiles + kUnitCost, at = t - sm.start[lo];
  u.head = static_cast<int>(__fdividef(static_cast<float>(at), static_cast<float>(span)));  // off by one at most, and put right
  while (u.head > 0 && u.head * span > at) --u.head;
  while ((u.head + 1) * span <= at) ++u.head;
  u.start = sm.start[lo] + u.head * span;
  u.tile0 = u.start + kUnitCost;
  return u;
}

__device__ __forceinline__ bool weight_lengths(const CacheWeightsParams &P, int b, int &base, int &cnt) {
  base = P.cache_len[b];
  cnt = P.counts ? P.counts[b] : P.n_rows;
  return base >= 0 && cnt >= 0 && cnt <= P.n_rows &&
         base + static_cast<int64_t>(cnt) <= min(capacity(P.c), static_cast<int64_t>(P.positions));
}

// A position's sum where the kernel's came out as NaN.  exp2(x - inf) is the 0 that a row of lse -inf, or none, has to add, unless
// x is NaN or infinite (of what such a row's q holds, or of 0 times a NaN key); here only rows that see the position count.
// at: the warp's lanes of the tile's scores.  The whole warp calls.
template <int PIECES, bool CAP>
__device__ __noinline__ float sum_of_seers(const WeightSmall &sm, uint32_t at, int padded, int place, float ks, float in_cap, float cap2) {
  float sum = 0.0f;
#pragma unroll 1
  for (int r = 0; r < padded; r += 16, at += 16) {
    float x[16], y[16], z[16];
    tmem_ld16(at, x);
    tmem_ld16(at + padded, y);
    if (PIECES == 3) tmem_ld16(at + 2 * padded, z);
    tc_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      if (PIECES == 3) y[e] = fmaf(z[e], 1.0f / 16, y[e]);
      x[e] = fmaf(y[e], 1.0f / 16, x[e]) * (sm.row[r + e].x * ks);
    }
    if (CAP) cap_scores<16>(x, in_cap, cap2);
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (place <= sm.token[r + e]) sum += ex2(x[e] + sm.row[r + e].y);
  }
  return sum;
}

// The requests' status before the kernel below, whose CTAs then raise it, in any
// order and several to a request: SPEC_STATUS_TIMEOUT is the largest and stays.
__global__ void cache_weights_status_kernel(int32_t *status, int count) {
  pdl_launch_dependents();
  for (int b = threadIdx.x; b < count; b += blockDim.x) status[b] = SPEC_STATUS_OK;
}
static_assert(SPEC_STATUS_TIMEOUT > SPEC_STATUS_BAD_INDEX && SPEC_STATUS_TIMEOUT > SPEC_STATUS_BAD_PAGE &&
              SPEC_STATUS_TIMEOUT > SPEC_STATUS_BAD_LENGTH && SPEC_STATUS_OK == 0);

template <int DT, int D, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
    cache_weights_tile_kernel(const CacheWeightsParams P, int first, int count, uint32_t group_inverse, int page_rows, bool q_vec,
                              const __grid_constant__ CUtensorMap k_map) {
  using S = WeightShape<DT, D>;
  extern __shared__ char raw[];
  char *const smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  WeightSmall &sm = *reinterpret_cast<WeightSmall *>(smem + S::kSmall);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, ctas = gridDim.x, heads = P.c.kv_heads;

  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) bar_init(&sm.k_full[i], 1), bar_init(&sm.k_empty[i], 1);
    for (int i = 0; i < 2; ++i) bar_init(&sm.s_full[i], 2), bar_init(&sm.s_empty[i], 256);
    bar_init(&sm.q_full, 256);
    bar_init(&sm.meet, 256);
    for (int i = 0; i < kRing; ++i) bar_init(&sm.ring_full[i], 32), bar_init(&sm.ring_empty[i], 256);
    bar_init_fence();
    sm.dead = sm.bad[0] = sm.bad[1] = 0;
  }
  if (warp == 9) tmem_alloc(&sm.tmem, 512);
  pdl_wait();
  for (int b = tid; b < count; b += kThreads) {
    int base, cnt;
    const bool ok = weight_lengths(P, first + b, base, cnt);
    sm.lens[b] = make_int2(base, cnt);
    sm.start[b + 1] = ok && base + cnt > 0 ? ((base + cnt + kTile - 1) / kTile + kUnitCost) * heads : 0;
    if (cta == 0 && P.status && !ok) atomicMax(&P.status[first + b], SPEC_STATUS_BAD_LENGTH);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    int carry = 0;
    for (int b0 = 0; b0 < count; b0 += 32) {
      int x = b0 + lane < count ? sm.start[b0 + lane + 1] : 0;
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
      }
      x += carry;
      if (b0 + lane < count) sm.start[b0 + lane + 1] = x;
      carry = __shfl_sync(~0u, x, 31);
    }
    if (lane == 0) sm.start[0] = 0;
  }
  __syncthreads();
  const int total = sm.start[count];
  const int lo = static_cast<int>(static_cast<int64_t>(total) * cta / ctas);
  int hi = static_cast<int>(static_cast<int64_t>(total) * (cta + 1) / ctas);
  if (hi < total) {  // a cut at or before a unit's first tile ends with the unit before
    const WeightUnit u = weight_unit(sm, count, heads, hi);
    if (hi <= u.tile0) hi = u.start;
  }
  const uint32_t tmem = sm.tmem;
  volatile int *dead = &sm.dead;
  constexpr int kBuffers = S::kPieces == 2 ? 2 : 1, kSideCols = 256 / kBuffers;  // tensor memory: scores of a tile's sides
  auto chunks_of = [&](const WeightUnit &u) { return max(1, (u.cnt * P.group + kMaxRows - 1) / kMaxRows); };  // (no rows: prev is copied)
  auto padded_of = [&](const WeightUnit &u, int c) { return max(16, (min(kMaxRows, u.cnt * P.group - c * kMaxRows) + 15) / 16 * 16); };

  if (warp == 8) {
    // ---- loading K and its scales: a lane to 16 positions (the first 16 lanes); the next tile's page is looked up meanwhile
    const int shift = P.c.page_shift;
    int stage = 0, lap = 0, i = 0;
    bool ok = true;
    for (int t = lo; t < hi && ok;) {
      const WeightUnit u = weight_unit(sm, count, heads, t);
      const int end = min(hi, u.tile0 + u.tiles), chunks = chunks_of(u);
      t = max(t, u.tile0);
      for (int c = 0; c < chunks && ok; ++c) {
        auto page_of = [&](int k) {
          if (k >= end || lane >= 16) return -1;  // (past the last tile a position could pass an int)
          const int pos = (k - u.tile0) * kTile + lane * 16;
          return pos < u.T ? page_at(P.c, first + u.b, pos >> shift) : -1;
        };
        auto scale_of = [&](int page) { return page >= 0 ? P.c.k_scale[page * P.c.scale_stride + u.head] : 1.0f; };
        int page = page_of(t), page1 = page_of(t + 1);
        float scale = scale_of(page);
        for (int k = t; k < end; ++k, ++i) {
          const float scale1 = scale_of(page1);
          const int page2 = page_of(k + 2), pos = (k - u.tile0) * kTile + lane * 16, r = i % kRing;
          if (i >= kRing && !(ok = warp_wait(&sm.ring_empty[r], (i / kRing - 1) & 1, dead))) break;
          if (lane < 16) sm.ring[r][lane] = scale;
          bar_arrive(&sm.ring_full[r]);
          const bool load = page >= 0 && (pos & (page_rows - 1)) == 0;
          const uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(~0u, load)) * page_rows * D);
          if (lap > 0 && !(ok = warp_wait(&sm.k_empty[stage], (lap - 1) & 1, dead))) break;
          if (lane == 0) bar_expect(&sm.k_full[stage], bytes);
          __syncwarp();
          if (load)
            tensor_load_3d(smem + S::kK + stage * S::kStage + lane * 16 * D, &k_map, 0, (u.head << shift) + (pos & ((1 << shift) - 1)), page,
                           &sm.k_full[stage]);
          if (++stage == S::kStages) stage = 0, ++lap;
          page = page1, page1 = page2, scale = scale1;
        }
      }
      t = end;
    }
    sm.copies = lap * S::kStages + stage;
  } else if (warp == 9) {
    // ---- issuing S^T = K Q^T
    constexpr uint64_t kSw = D == 128 ? kSwizzle128 : kSwizzle64;
    const uint64_t q_desc = matrix_desc(smem_u32(smem + S::kQ), 16, 8 * D, kSw);
    const uint64_t k_desc = matrix_desc(smem_u32(smem + S::kK), 16, 8 * D, kSw);
    int stage = 0, lap = 0, i = 0, writes = 0;
    bool ok = true;
    for (int t = lo; t < hi && ok;) {
      const WeightUnit u = weight_unit(sm, count, heads, t);
      const int end = min(hi, u.tile0 + u.tiles), chunks = chunks_of(u);
      t = max(t, u.tile0);
      for (int c = 0; c < chunks && ok; ++c) {
        if (!(ok = warp_wait(&sm.q_full, writes++ & 1, dead))) break;
        const uint32_t idesc = mma_desc(S::kPieces * padded_of(u, c), false);
        for (int k = t; k < end; ++k, ++i) {
          const int buffer = i % kBuffers;
          if (i >= kBuffers && !(ok = warp_wait(&sm.s_empty[buffer], (i / kBuffers - 1) & 1, dead))) break;
          if (!(ok = warp_wait(&sm.ring_full[i % kRing], (i / kRing) & 1, dead))) break;
          if (lane == 0) bar_arrive(&sm.s_full[buffer]);  // (with this arrival S full says that the tile's scales are there too)
          if (!(ok = warp_wait(&sm.k_full[stage], lap & 1, dead))) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int e = 0; e < D / 32; ++e)
#pragma unroll
              for (int half = 0; half < 2; ++half)  // (in turn: a product waits for the one before on its own accumulator)
                mma_f8(tmem + (buffer * 2 + half) * kSideCols, k_desc + ((stage * S::kStage + half * 128 * D + e * 32) >> 4),
                       q_desc + ((e * 32) >> 4), idesc, e > 0);
            tc_commit(&sm.k_empty[stage]);
            tc_commit(&sm.s_full[buffer]);
          }
          __syncwarp();
          if (++stage == S::kStages) stage = 0, ++lap;
        }
      }
      t = end;
    }
    sm.products = i;
  } else {
    // ---- summing
    const int side = warp >> 2, quarter = warp & 3, spot = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter) << 21;
    const bool negative = P.scale < 0.0f;
    const float cap2 = P.softcap * kLog2e, in_cap = CAP ? 1.0f / cap2 : 0.0f;
    uint32_t meetings = 0;
    auto together = [&] {
      bar_arrive(&sm.meet);
      return warp_wait(&sm.meet, meetings++ & 1, dead);
    };
    int i = 0, segment = 0;
    bool ok = true;
    for (int t = lo; t < hi && ok; ++segment) {
      const WeightUnit u = weight_unit(sm, count, heads, t);
      const int end = min(hi, u.tile0 + u.tiles), chunks = chunks_of(u), b = first + u.b, rows = u.cnt * P.group;
      t = max(t, u.tile0);
      const int t0 = t;
      const int32_t *index = P.index ? P.index + static_cast<int64_t>(b) * P.index_stride : nullptr;
      // the request's pages and indexes: a bad one takes the request out
      int bad = 0;
      for (int k = tid; static_cast<int64_t>(k) << P.c.page_shift < u.T; k += 256) bad |= page_at(P.c, b, k) < 0 ? 1 : 0;
      if (index)
        for (int k = tid; k < u.cnt; k += 256) bad |= index[k] < 0 || index[k] >= P.N ? 2 : 0;
      bad = __reduce_or_sync(~0u, bad);
      if (lane == 0 && bad) atomicOr(&sm.bad[segment & 1], bad);
      for (int c = 0; c < chunks && ok; ++c) {
        const int row0 = c * kMaxRows, here = min(kMaxRows, rows - row0), padded = padded_of(u, c);
        // every product that reads the rows before has completed for both sides
        if (!(ok = together())) break;
        if (c == 0) {
          bad = sm.bad[segment & 1];
          if (tid == 0) sm.bad[(segment + 1) & 1] = 0;  // (the segment before's; the next one's is set after the next meeting)
          if (bad && tid == 0 && u.head == 0 && t0 == u.tile0 && P.status)
            atomicMax(&P.status[b], bad & 1 ? SPEC_STATUS_BAD_PAGE : SPEC_STATUS_BAD_INDEX);
        }
        constexpr int kEach = D / 32;
#pragma unroll 1
        for (int r0 = warp; r0 < padded; r0 += 16) {  // two rows side by side
          float x[2][kEach], top[2];
          int ex[2], tok[2], at[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int r = r0 + 8 * k, row = row0 + r;
            tok[k] = P.group == 1 ? row : static_cast<int>(__umulhi(static_cast<uint32_t>(row), group_inverse));
            const bool real = r < here;
            at[k] = real ? (index ? index[tok[k]] : tok[k]) : -1;
            if (at[k] < 0 || at[k] >= P.N) at[k] = -1;
            const int h = u.head * P.group + row - tok[k] * P.group;
            const char *q = P.q + (b * P.qs[0] + max(at[k], 0) * P.qs[1] + h * P.qs[2]) * 2;
            top[k] = 0.0f;
#pragma unroll
            for (int e = 0; e < kEach; ++e) x[k][e] = 0.0f;
            if (at[k] >= 0) {
              if (q_vec) unpack_each<DT, kEach>(raw_each<kEach>(q, lane), x[k]);
              else
#pragma unroll
                for (int e = 0; e < kEach; ++e) x[k][e] = row_value<DT>(q, lane * kEach + e);
            }
          }
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
              if (negative) x[k][e] = -x[k][e];
              top[k] = fmaxf(top[k], finite_abs(x[k][e]));
            }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < 2; ++k) top[k] = fmaxf(top[k], __shfl_xor_sync(~0u, top[k], o));
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int r = r0 + 8 * k;
            if (r >= padded) break;
            // 2^ex with top / 2^ex in [128, 256)
            ex[k] = top[k] > 0.0f ? max(static_cast<int>(__float_as_uint(top[k]) >> 23) - 127 - 7, -110) : 0;
            const float down = __uint_as_float(static_cast<uint32_t>(127 - ex[k]) << 23);
#pragma unroll
            for (int e = 0; e < kEach; ++e) x[k][e] *= down;
#pragma unroll
            for (int piece = 0; piece < S::kPieces; ++piece) {
              uint32_t code = 0;
#pragma unroll
              for (int e = 0; e < kEach; e += 2) {
                const uint32_t two = to_e4m3x2(x[k][e], x[k][e + 1]);
                const float2 back = e4m3x2_to_float2(two);
                x[k][e] = (x[k][e] - back.x) * 16.0f;
                x[k][e + 1] = (x[k][e + 1] - back.y) * 16.0f;
                code |= two << (8 * e);
              }
              const int a = piece * padded + r, chunk = lane * kEach >> 4;
              char *to = smem + S::kQ + a * D + ((D == 128 ? chunk ^ (a & 7) : chunk ^ (a >> 1 & 3)) << 4) + (lane * kEach & 15);
              if (kEach == 4) *reinterpret_cast<uint32_t *>(to) = code;
              else *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(code);
            }
            if (lane == 0) {
              const int h = u.head * P.group + row0 + r - tok[k] * P.group;
              const float z = at[k] >= 0 ? P.lse[b * P.ls[0] + at[k] * P.ls[1] + h * P.ls[2]] : -INFINITY;
              sm.row[r] = make_float2(fabsf(P.scale) * kLog2e * __uint_as_float(static_cast<uint32_t>(ex[k] + 127) << 23),
                                      z == -INFINITY ? -INFINITY : -z * kLog2e);
              sm.token[r] = z == -INFINITY ? kNoRow : tok[k];
            }
          }
        }
        fence_async_shared();
        bar_arrive(&sm.q_full);
        if (!(ok = together())) break;

        for (int k = t; k < end; ++k, ++i) {
          const int buffer = i % kBuffers, ring = i % kRing, j = (k - u.tile0) * kTile + side * 128 + spot;
          const bool mine = j < u.T && !bad;
          const bool edge = (k - u.tile0) * kTile + kTile > u.base;
          float *out = P.out + b * P.out_s[0] + u.head * P.out_s[1] + j;
          float sum = 0.0f, held = 0.0f;
          if (mine) held = c > 0 ? *out : P.prev ? P.prev[b * P.prev_s[0] + u.head * P.prev_s[1] + j] : 0.0f;
          if (!(ok = warp_wait(&sm.s_full[buffer], (i / kBuffers) & 1, dead))) break;
          tc_fence_after();
          const float ks = sm.ring[ring][side * 8 + (spot >> 4)];
          bar_arrive(&sm.ring_empty[ring]);
#pragma unroll 1
          for (int r = 0; r < padded; r += 16) {
            float x[16], y[16];
            const uint32_t at = tmem + lanes + (buffer * 2 + side) * kSideCols + r;
            tmem_ld16(at, x);
            tmem_ld16(at + padded, y);
            if (S::kPieces == 3) {
              float z[16];
              tmem_ld16(at + 2 * padded, z);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = fmaf(z[e], 1.0f / 16, y[e]);
            } else {
              tc_wait_ld();
            }
            if (CAP) {
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = fmaf(y[e], 1.0f / 16, x[e]) * (sm.row[r + e].x * ks);
              cap_scores<16>(x, in_cap, cap2);
            }
            float part[2] = {};
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float4 f = *reinterpret_cast<const float4 *>(&sm.row[r + e]);  // two rows'
              float s0, s1;
              if (CAP) {
                s0 = x[e] + f.y;
                s1 = x[e + 1] + f.w;
              } else {
                s0 = fmaf(fmaf(y[e], 1.0f / 16, x[e]), f.x * ks, f.y);
                s1 = fmaf(fmaf(y[e + 1], 1.0f / 16, x[e + 1]), f.z * ks, f.w);
              }
              float p0 = ex2(s0), p1 = ex2(s1);
              if (edge) [[unlikely]] {
                if (j - u.base > sm.token[r + e]) p0 = 0.0f;
                if (j - u.base > sm.token[r + e + 1]) p1 = 0.0f;
              }
              part[0] += p0;
              part[1] += p1;
            }
            sum += part[0] + part[1];
          }
          if (__any_sync(~0u, mine && sum != sum)) [[unlikely]] {
            const float seen = sum_of_seers<S::kPieces, CAP>(sm, tmem + lanes + (buffer * 2 + side) * kSideCols, padded, j - u.base, ks, in_cap, cap2);
            if (sum != sum) sum = seen;
          }
          tc_fence_before();
          bar_arrive(&sm.s_empty[buffer]);
          if (mine) *out = held + sum;
        }
      }
      t = end;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*dead) [[unlikely]] {  // nothing that was begun may reach shared or tensor memory that the CTA has left (else all was waited for)
    if (warp == 0) {
      ring_land(sm.k_full, S::kStages, sm.copies);
      ring_land(sm.k_empty, S::kStages, sm.products);
      ring_land(sm.s_full, kBuffers, sm.products);
    }
    __syncthreads();
  }
  if (*dead && P.status)  // a wait ran out: what the CTA worked on is void
    for (int b = tid; b < count; b += kThreads) atomicMax(&P.status[first + b], SPEC_STATUS_TIMEOUT);
  if (warp == 9) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// The sums go where they were: a second launch would add the rows once more.
bool in_place(const CacheWeightsParams &P) { return P.prev == P.out; }

std::atomic<uint64_t> weights_ready[8];

template <int DT, int D, bool CAP>
cudaError_t launch_weight_tiles(const CacheWeightsParams &P, cudaStream_t st) {
  using S = WeightShape<DT, D>;
  auto kern = cache_weights_tile_kernel<DT, D, CAP>;
  cudaError_t e = once_per_device([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes); },
                                  weights_ready[CAP * 4 + (DT == SPEC_DTYPE_BF16) * 2 + (D == 128)]);
  if (e != cudaSuccess) return e;
  const int page_rows = std::min(1 << P.c.page_shift, kTilePositions);
  CUtensorMap map;
  if ((e = cache_k_map(P.c, page_rows, &map)) != cudaSuccess) return e;
  const uint32_t group_inverse = static_cast<uint32_t>((0x100000000ull + P.group - 1) / P.group);
  const bool q_vec = reinterpret_cast<uintptr_t>(P.q) % 8 == 0 && P.qs[0] % 4 == 0 && P.qs[1] % 4 == 0 && P.qs[2] % 4 == 0;
  for (int first = 0; first < P.B; first += kTileRequests) {
    const int count = std::min(kTileRequests, P.B - first);
    if (P.status) {
      e = trace_launch("cache_weights_status", st, [&] { cache_weights_status_kernel<<<1, kTileRequests, 0, st>>>(P.status + first, count); });
      if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(device_sm_count()));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = P.status && !trace_enabled() ? 1 : 0;
    e = trace_launch_ex("cache_weights_tile", st,
                        [&] { return cudaLaunchKernelEx(&cfg, kern, P, first, count, group_inverse, page_rows, q_vec, map); }, !in_place(P));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int DT>
cudaError_t launch_weight_tiles(const CacheWeightsParams &P, cudaStream_t st) {
  if (P.c.head_dim == 128) return P.softcap > 0.0f ? launch_weight_tiles<DT, 128, true>(P, st) : launch_weight_tiles<DT, 128, false>(P, st);
  return P.softcap > 0.0f ? launch_weight_tiles<DT, 64, true>(P, st) : launch_weight_tiles<DT, 64, false>(P, st);
}

}  // namespace

cudaError_t launch_cache_weights(const CacheWeightsParams &P, cudaStream_t st) {
  // (a row's number times the group stays below 2^32: the multiplication that divides by it is exact)
  const bool tiles = static_cast<int64_t>(P.n_rows) * P.group * P.group < (1LL << 32);
  if (tiles && (P.c.head_dim == 64 || P.c.head_dim == 128))
    return P.dtype == SPEC_DTYPE_BF16 ? launch_weight_tiles<SPEC_DTYPE_BF16>(P, st) : launch_weight_tiles<SPEC_DTYPE_F16>(P, st);
  const int64_t most = static_cast<int64_t>(P.c.table_stride) << P.c.page_shift;
  const int spans = most > 0 ? static_cast<int>((most + kSpan - 1) / kSpan) : 1;
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(spans) * P.c.kv_heads * P.B);
  return trace_launch("cache_weights_rows", st, [&] {
    if (P.dtype == SPEC_DTYPE_BF16) cache_weights_rows_kernel<SPEC_DTYPE_BF16><<<grid, kSpan, 0, st>>>(P, spans);
    else cache_weights_rows_kernel<SPEC_DTYPE_F16><<<grid, kSpan, 0, st>>>(P, spans);
  }, !in_place(P));
}

}  // namespace sv
