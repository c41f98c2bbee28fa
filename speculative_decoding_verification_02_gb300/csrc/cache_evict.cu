// spec_cache_evict: a smaller cache of the heaviest tokens.
//
// First kernel, a cluster of CTAs to (request, head), each with a slice of the
// positions: the weight of the last token that is kept, by radix selection
// over the weights' order-preserving bits (11, 11 and 10 of them, the CTAs'
// histograms added through distributed shared memory), then one ordered pass
// that writes the kept positions.  The keys stay in shared memory between the
// passes, so the weights are read once.  Second kernel, a CTA to (request,
// head, new page, K or V): gathers the kept rows, 16 bytes to a thread, and
// gives the block the scale they need.
//
// 131,071 positions of 8 heads to 4,096: 35 us, of them about 24 the selection
// (eight CTAs to a head, bound by its barriers).  32 requests of up to 7,001 to
// 1,000, 8 heads of 64: 47 us, about half of it the gathering of 64-byte rows.
#include <algorithm>
#include <cooperative_groups.h>

#include "cache.cuh"
#include "common.cuh"
#include "launch.h"

namespace sv {
namespace {

constexpr int kGatherThreads = 256;
constexpr int kBins = 2048;
constexpr int kSliceKeys = 40960;  // keys of a CTA's slice that fit its shared memory
constexpr int kMaxCluster = 16;    // for slices that would not fit otherwise; else
constexpr int kFastCluster = 8;    // (131,072 positions, 8 heads: 33 us with 8 CTAs to a head, 46 with 16, 45 with 4)
std::atomic<uint64_t> select_ready[2];

// Bits that order as the weights do: NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (!(w == w)) return 0;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The weight that a key was made of; NaN has to be read again.
__device__ __forceinline__ float key_weight(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u); }

// Sum over the CTA's threads of lower index.
template <int THREADS>
__device__ __forceinline__ int block_rank(int v, int *s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int y = lane < THREADS / 32 ? s_warp[lane] : 0;
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(~0u, y, o);
    if (lane >= o) y += z;
  }
  const int before = __shfl_sync(~0u, y, max(warp - 1, 0));
  return x - v + (warp > 0 ? before : 0);
}

// What the CTAs of a cluster read of one another.
struct SelectShared {
  int hist[kBins];   // this slice's
  int sum[kBins];    // the bins that this CTA adds up for the cluster
  int total[kBins];  // the cluster's
  int warp[32];
  int2 count;        // this slice's positions above the key, and equal to it
  int2 counts[32];   // a warp's
  int digit, above;
  int2 before;       // kept positions, and ties, of the slices before
};

// THREADS: 512 where a CTA has a head to itself, so that an SM holds two heads;
// 1,024 in a cluster.
template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) cache_select_kernel(const CacheEvictParams P, int slice_room) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ uint32_t s_key[];
  __shared__ SelectShared sh;
  const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int unit = blockIdx.x / ranks, head = unit % P.c.kv_heads, b = unit / P.c.kv_heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto meet = [&] {
    if (ranks > 1) cluster.sync();
    else __syncthreads();
  };
  const int64_t len = P.cache_len[b];
  const bool bad_len = len < 0 || len > min(capacity(P.c), static_cast<int64_t>(P.positions)) ||
                       min(len, static_cast<int64_t>(P.keep)) > capacity(P.d);
  const int T = bad_len ? 0 : static_cast<int>(len);
  const int kc = min(P.keep, T), late = min(P.recent, kc);
  int bad = 0;
  for (int64_t i = tid; i << P.c.page_shift < T; i += THREADS) bad |= page_at(P.c, b, i) < 0;
  for (int64_t i = tid; i << P.d.page_shift < kc; i += THREADS) bad |= page_at(P.d, b, i) < 0;
  const bool bad_page = __syncthreads_or(bad);  // (every CTA of the cluster finds the same)
  const int total = bad_page ? 0 : kc;
  if (head == 0 && rank == 0 && tid == 0) {
    if (P.status) P.status[b] = bad_len ? SPEC_STATUS_BAD_LENGTH : bad_page ? SPEC_STATUS_BAD_PAGE : SPEC_STATUS_OK;
    P.new_len[b] = total;
  }
  int32_t *kept = P.kept + (static_cast<int64_t>(b) * P.c.kv_heads + head) * P.keep;
  float *kw = P.kept_weights ? P.kept_weights + (static_cast<int64_t>(b) * P.c.kv_heads + head) * P.keep : nullptr;
  for (int i = total + rank * THREADS + tid; i < P.keep; i += ranks * THREADS) {
    kept[i] = -1;
    if (kw) kw[i] = 0.0f;
  }
  const float *w = P.weights + b * P.ws[0] + head * P.ws[1];
  const int M = total ? T - late : 0;       // positions that compete
  const int want = total ? kc - late : 0;
  for (int i = rank * THREADS + tid; i < (total ? late : 0); i += ranks * THREADS) {
    kept[want + i] = M + i;
    if (kw) kw[want + i] = w[M + i];
  }
  if (want == 0) return;  // (the whole cluster)

  // this CTA's slice of the positions, whole warps of them
  const int slice = ((M + ranks - 1) / ranks + 31) / 32 * 32;
  const int from = min(rank * slice, M), mine = min(slice, M - from);
  const bool in_shared = slice <= slice_room;
  if (in_shared) {
#pragma unroll 16
    for (int i = tid; i < mine; i += THREADS) s_key[i] = weight_key(w[from + i]);
  }
  auto key_at = [&](int i) { return in_shared ? s_key[i] : weight_key(w[from + i]); };

  // The want-th largest key, digit by digit; `left` of those equal to it are kept.  All keys when all are kept.
  uint32_t key = 0;
  int left = want;
  if (want < M) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
      const uint32_t high = pass == 0 ? 0 : ~0u << (pass == 1 ? 21 : 10);
      for (int i = tid; i < bins; i += THREADS) sh.hist[i] = 0;
      __syncthreads();
      for (int i0 = 0; i0 < mine; i0 += THREADS) {
        const int i = i0 + tid;
        const uint32_t u = i < mine ? key_at(i) : 0;
        const bool in = i < mine && (u & high) == key;
        const int bin = in ? static_cast<int>(u >> shift & (bins - 1)) : -1;
        int same;
        __match_all_sync(~0u, bin, &same);  // (a warp of equal keys adds once)
        if (same) {
          if (lane == 0 && in) atomicAdd(&sh.hist[bin], 32);
        } else if (in) {
          atomicAdd(&sh.hist[bin], 1);
        }
      }
      meet();
      const int *totals = sh.hist;
      if (ranks > 1) {  // each CTA adds up its share of the bins and gives the sums to all
        totals = sh.total;
        const int share = bins / ranks, first = rank * share;
        for (int i = tid; i < share; i += THREADS) sh.sum[i] = 0;
        __syncthreads();
        for (int i = tid; i < bins; i += THREADS)
          atomicAdd(&sh.sum[i % share], cluster.map_shared_rank(sh.hist, i / share)[first + i % share]);
        __syncthreads();
        for (int i = tid; i < bins; i += THREADS)
          cluster.map_shared_rank(sh.total, i / share)[first + i % share] = sh.sum[i % share];
        cluster.sync();
      }
      // thread t: a few bins from the top; the digit is where their running sum reaches `left`
      constexpr int kOwn = kBins / THREADS;
      int here[kOwn], sum = 0;
#pragma unroll
      for (int k = 0; k < kOwn; ++k) {
        const int bin = bins - 1 - (kOwn * tid + k);
        here[k] = bin >= 0 ? totals[bin] : 0;
        sum += here[k];
      }
      int before = block_rank<THREADS>(sum, sh.warp);
      if (before < left && before + sum >= left) {
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
          if (before < left && before + here[k] >= left) {
            sh.digit = bins - 1 - (kOwn * tid + k);
            sh.above = before;
          }
          before += here[k];
        }
      }
      __syncthreads();
      key |= static_cast<uint32_t>(sh.digit) << shift;
      left -= sh.above;
    }
  }
  // A warp to a run of the slice: how many each keeps, then the kept positions in order -- those above the key, and of those
  // equal to it the first `left`.
  const int run = (slice + THREADS - 1) / THREADS * 32;
  const int run0 = min(warp * run, mine), run1 = min(run0 + run, mine);
  int2 seen = make_int2(0, 0);
  if (want < M) {
    for (int i0 = run0; i0 < run1; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t u = i < run1 ? key_at(i) : 0;
      seen.x += __popc(__ballot_sync(~0u, i < run1 && u > key));
      seen.y += __popc(__ballot_sync(~0u, i < run1 && u == key));
    }
  } else {
    seen.x = run1 - run0;
  }
  if (lane == 0) sh.counts[warp] = seen;
  __syncthreads();
  // running sums over the warps
  int2 c = lane < THREADS / 32 ? sh.counts[lane] : make_int2(0, 0);
  const int2 own = c;
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(~0u, c.x, o), y = __shfl_up_sync(~0u, c.y, o);
    if (lane >= o) c.x += x, c.y += y;
  }
  int out = __shfl_sync(~0u, c.x - own.x, warp), ties = __shfl_sync(~0u, c.y - own.y, warp);
  if (ranks > 1) {
    if (tid == 31) sh.count = c;
    cluster.sync();
    if (warp == 0) {
      int2 other = lane < rank ? *cluster.map_shared_rank(&sh.count, lane) : make_int2(0, 0);
      for (int o = 16; o > 0; o >>= 1) {
        other.x += __shfl_xor_sync(~0u, other.x, o);
        other.y += __shfl_xor_sync(~0u, other.y, o);
      }
      if (lane == 0) sh.before = other;
    }
    cluster.sync();  // (and no CTA leaves while its counts are read)
    out += sh.before.x;
    ties += sh.before.y;
  }
  out += min(ties, left);  // of the ties before, the kept ones (left is 0 where all are kept: no ties were counted)
  for (int i0 = run0; i0 < run1; i0 += 32) {
    const int i = i0 + lane;
    bool take = i < run1;
    const uint32_t u = i < run1 ? key_at(i) : 0;
    if (want < M) {
      const bool tie = i < run1 && u == key;
      const uint32_t votes = __ballot_sync(~0u, tie);
      take = i < run1 && (u > key || (tie && ties + __popc(votes & ((1u << lane) - 1)) < left));
      ties += __popc(votes);
    }
    const uint32_t votes = __ballot_sync(~0u, take);
    if (take) {
      const int at = out + __popc(votes & ((1u << lane) - 1));
      kept[at] = from + i;
      if (kw) kw[at] = u ? key_weight(u) : w[from + i];
    }
    out += __popc(votes);
  }
}

// The largest of 16 stored magnitudes, NaN aside (they order as their bits do).
__device__ __forceinline__ uint32_t most_of(const uint4 &v) {
  const uint32_t u[4] = {v.x & 0x7f7f7f7fu, v.y & 0x7f7f7f7fu, v.z & 0x7f7f7f7fu, v.w & 0x7f7f7f7fu};
  uint32_t most = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t nan = ((u[e] + 0x01010101u) & 0x80808080u) >> 7;  // 1 in a byte of 0x7f
    most = __vmaxu4(most, u[e] & ~(nan * 0xffu));
  }
  most = __vmaxu4(most, most >> 16);
  return max(most & 0xff, most >> 8 & 0xff);
}

// 16 stored values times a ratio of scales, rounded again: for any ratio (a
// function of its own, which few caches need).
__device__ __noinline__ uint4 rescaled_by_any(uint4 v, float ratio) {
  const uint32_t in[4] = {v.x, v.y, v.z, v.w};
  uint32_t out[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 a = e4m3x2_to_float2(in[e] & 0xffff), b = e4m3x2_to_float2(in[e] >> 16);
    out[e] = to_e4m3x2(product_to_odd(a.x, ratio), product_to_odd(a.y, ratio)) |
             to_e4m3x2(product_to_odd(b.x, ratio), product_to_odd(b.y, ratio)) << 16;
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// A power of two goes through halves: the product of four bits and a power of
// two is exact in them, or so far below e4m3's smallest step that it rounds to
// zero either way.
__device__ __forceinline__ uint4 rescaled(const uint4 &v, float ratio) {
  if (!(ratio <= 32768.0f && (__float_as_uint(ratio) & 0x7fffffu) == 0)) [[unlikely]] return rescaled_by_any(v, ratio);
  uint4 r;
  const uint32_t in[4] = {v.x, v.y, v.z, v.w};
  uint32_t *out = reinterpret_cast<uint32_t *>(&r);
  const __half2 k = __float2half2_rn(ratio);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint16_t c[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __half2 x = __hmul2(e4m3x2_to_half2(h ? in[e] >> 16 : in[e] & 0xffff), k);
      asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c[h]) : "r"(*reinterpret_cast<const uint32_t *>(&x)));
    }
    out[e] = c[0] | static_cast<uint32_t>(c[1]) << 16;
  }
  return r;
}

constexpr int kGatherHeld = 2;  // 16-byte pieces that a thread holds

// TEAM threads to a block, so that each has about two pieces of it; PER_ROW:
// pieces of a row, 0: any.
template <int TEAM, int PER_ROW>
__global__ void __launch_bounds__(kGatherThreads, 5) cache_gather_kernel(const CacheEvictParams P, int pages, uint32_t blocks) {
  __shared__ float s_max[kGatherThreads / 32];
  const int tid = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  uint32_t x = blockIdx.x * (kGatherThreads / TEAM) + team;
  const bool real = x < blocks;
  x = min(x, blocks - 1);
  const bool is_v = x & 1;
  x >>= 1;
  const int w = static_cast<int>(x % pages);
  x /= pages;
  const int head = static_cast<int>(x % P.c.kv_heads), b = static_cast<int>(x / P.c.kv_heads);
  const int D = P.c.head_dim, shift = P.c.page_shift;
  const int per_row = PER_ROW ? PER_ROW : D / 16;
  const int32_t *kept = P.kept + (static_cast<int64_t>(b) * P.c.kv_heads + head) * P.keep + (w << shift);
  const int32_t *table = P.c.table + static_cast<int64_t>(b) * P.c.table_stride;
  const uint8_t *pool = (is_v ? P.c.v : P.c.k) + (static_cast<int64_t>(head) << shift) * D;
  const float *scales = (is_v ? P.c.v_scale : P.c.k_scale) + head;
  pdl_wait();
  const int rows = real ? min(P.new_len[b] - (w << shift), 1 << shift) : 0;
  const int pieces = max(rows, 0) * per_row;
  // a piece and its scale (the pages have been looked over by the selection: a request with a bad one has no rows)
  auto load = [&](int t, int part, uint4 &v, float &s) {
    const int page = table[t >> shift];
    v = reinterpret_cast<const uint4 *>(pool + page * P.c.page_stride + (t & ((1 << shift) - 1)) * D)[part];
    s = scales[page * P.c.scale_stride];
  };
  uint4 held[kGatherHeld];
  float from[kGatherHeld], amax = 0.0f;  // (of products rounded up: one just above what a scale holds asks for the next)
  int token[kGatherHeld];
#pragma unroll
  for (int k = 0; k < kGatherHeld; ++k) {
    const int i = tid + k * TEAM;
    token[k] = i < pieces ? kept[i / per_row] : -1;
  }
#pragma unroll
  for (int k = 0; k < kGatherHeld; ++k)
    if (token[k] >= 0) load(token[k], (tid + k * TEAM) % per_row, held[k], from[k]);
#pragma unroll
  for (int k = 0; k < kGatherHeld; ++k)
    if (token[k] >= 0) amax = fmaxf(amax, __fmul_ru(e4m3x2_to_float2(most_of(held[k])).x, from[k]));
  for (int i = tid + kGatherHeld * TEAM; i < pieces; i += TEAM) {
    uint4 v;
    float s;
    load(kept[i / per_row], i % per_row, v, s);
    amax = fmaxf(amax, __fmul_ru(e4m3x2_to_float2(most_of(v)).x, s));
  }
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  if (TEAM > 32) {
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TEAM / 32; ++i) amax = fmaxf(amax, s_max[team * (TEAM / 32) + i]);
  }
  if (rows <= 0) return;
  const float scale = block_scale(amax), inv = 1.0f / scale;  // (a power of two: exact)
  const int page = page_at(P.d, b, w);
  uint4 *to = reinterpret_cast<uint4 *>((is_v ? P.d.v : P.d.k) + block_offset(P.d, page, head));
#pragma unroll
  for (int k = 0; k < kGatherHeld; ++k)
    if (token[k] >= 0) to[tid + k * TEAM] = from[k] == scale ? held[k] : rescaled(held[k], from[k] * inv);
  for (int i = tid + kGatherHeld * TEAM; i < pieces; i += TEAM) {
    uint4 v;
    float s;
    load(kept[i / per_row], i % per_row, v, s);
    to[i] = s == scale ? v : rescaled(v, s * inv);
  }
  if (tid == 0) (is_v ? P.d.v_scale : P.d.k_scale)[page * P.d.scale_stride + head] = scale;
}

template <int TEAM>
cudaError_t launch_gather(const CacheEvictParams &P, cudaStream_t st) {
  const int pages = (P.keep + (1 << P.c.page_shift) - 1) >> P.c.page_shift;
  const uint32_t blocks = 2u * P.B * P.c.kv_heads * pages;
  auto kern = P.c.head_dim == 128 ? cache_gather_kernel<TEAM, 8> : P.c.head_dim == 64 ? cache_gather_kernel<TEAM, 4> : cache_gather_kernel<TEAM, 0>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((blocks + kGatherThreads / TEAM - 1) / (kGatherThreads / TEAM));
  cfg.blockDim = dim3(kGatherThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = trace_enabled() ? 0 : 1;
  return trace_launch_ex("cache_gather", st, [&] { return cudaLaunchKernelEx(&cfg, kern, P, pages, blocks); });
}

// CTAs to a (request, head): enough for a slice of a few thousand positions,
// as many as the GPU holds at once (one of a cluster's CTAs to an SM), and a
// slice that fits shared memory where sixteen of them can make it so.
int select_cluster(int64_t positions, int64_t heads) {
  int n = 1;
  while (n < kFastCluster && positions / n > 4096 && heads * n * 2 <= device_sm_count()) n *= 2;
  while (n < kMaxCluster && positions / n > kSliceKeys) n *= 2;
  return n;
}

}  // namespace

cudaError_t launch_cache_evict(const CacheEvictParams &P, cudaStream_t st) {
  const unsigned heads = static_cast<unsigned>(P.B * P.c.kv_heads);
  const int64_t positions =
      std::min<int64_t>(static_cast<int64_t>(P.c.table_stride) << P.c.page_shift, P.positions);
  const int ranks = select_cluster(positions, heads);
  const int room = static_cast<int>(std::min<int64_t>((positions + ranks - 1) / ranks + 64, kSliceKeys));
  auto kern = ranks > 1 ? cache_select_kernel<1024> : cache_select_kernel<512>;
  cudaError_t e = once_per_device(
      [&] {
        cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSliceKeys * 4);
        if (r == cudaSuccess) r = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        return r;
      },
      select_ready[ranks > 1]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(heads * ranks);
  cfg.blockDim = dim3(ranks > 1 ? 1024 : 512);
  cfg.dynamicSmemBytes = room * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = trace_launch_ex("cache_select", st, [&] { return cudaLaunchKernelEx(&cfg, kern, P, room); });
  if (e != cudaSuccess) return e;
  // two pieces to a thread
  const int pieces = (P.c.head_dim << P.c.page_shift) / 16;
  if (pieces <= 64) return launch_gather<32>(P, st);
  if (pieces <= 128) return launch_gather<64>(P, st);
  if (pieces <= 256) return launch_gather<128>(P, st);
  return launch_gather<256>(P, st);
}

}  // namespace sv
