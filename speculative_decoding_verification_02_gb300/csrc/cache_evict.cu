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
#include <algorithm>
#include <cooperative_groups.h>

#include "cache.cuh"
#include "launch.h"

namespace sv {
namespace {

constexpr int kSelectThreads = 1024;
constexpr int kGatherThreads = 256;
constexpr int kBins = 2048;
constexpr int kSliceKeys = 40960;  // keys of a CTA's slice that fit its shared memory
constexpr int kMaxCluster = 16;
std::atomic<uint64_t> select_ready{0};

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

// What the CTAs of a cluster read of one another.
struct SelectShared {
  int hist[kBins];
  int warp[32];
  int count[2];  // this slice's positions above the key, and equal to it
  int digit, above;
};

__global__ void __launch_bounds__(kSelectThreads) cache_select_kernel(const CacheEvictParams P, int slice_room) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ uint32_t s_key[];
  __shared__ SelectShared sh;
  const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int unit = blockIdx.x / ranks, head = unit % P.c.kv_heads, b = unit / P.c.kv_heads;
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t len = P.cache_len[b];
  const bool bad_len = len < 0 || len > min(capacity(P.c), static_cast<int64_t>(P.positions)) ||
                       min(len, static_cast<int64_t>(P.keep)) > capacity(P.d);
  const int T = bad_len ? 0 : static_cast<int>(len);
  const int kc = min(P.keep, T), late = min(P.recent, kc);
  int bad = 0;
  for (int64_t i = tid; i << P.c.page_shift < T; i += kSelectThreads) bad |= page_at(P.c, b, i) < 0;
  for (int64_t i = tid; i << P.d.page_shift < kc; i += kSelectThreads) bad |= page_at(P.d, b, i) < 0;
  const bool bad_page = __syncthreads_or(bad);  // (every CTA of the cluster finds the same)
  const int total = bad_page ? 0 : kc;
  if (head == 0 && rank == 0 && tid == 0) {
    if (P.status) P.status[b] = bad_len ? SPEC_STATUS_BAD_LENGTH : bad_page ? SPEC_STATUS_BAD_PAGE : SPEC_STATUS_OK;
    P.new_len[b] = total;
  }
  int32_t *kept = P.kept + (static_cast<int64_t>(b) * P.c.kv_heads + head) * P.keep;
  float *kw = P.kept_weights ? P.kept_weights + (static_cast<int64_t>(b) * P.c.kv_heads + head) * P.keep : nullptr;
  for (int i = total + rank * kSelectThreads + tid; i < P.keep; i += ranks * kSelectThreads) {
    kept[i] = -1;
    if (kw) kw[i] = 0.0f;
  }
  const float *w = P.weights + b * P.ws[0] + head * P.ws[1];
  const int M = total ? T - late : 0;       // positions that compete
  const int want = total ? kc - late : 0;
  for (int i = rank * kSelectThreads + tid; i < (total ? late : 0); i += ranks * kSelectThreads) {
    kept[want + i] = M + i;
    if (kw) kw[want + i] = w[M + i];
  }
  if (want == 0) return;  // (the whole cluster)

  // this CTA's slice of the positions, whole warps of them
  const int slice = ((M + ranks - 1) / ranks + 31) / 32 * 32;
  const int from = min(rank * slice, M), mine = min(slice, M - from);
  const bool in_shared = slice <= slice_room;
  if (in_shared)
    for (int i = tid; i < mine; i += kSelectThreads) s_key[i] = weight_key(w[from + i]);
  auto key_at = [&](int i) { return in_shared ? s_key[i] : weight_key(w[from + i]); };

  // The want-th largest key, digit by digit; `left` of those equal to it are kept.  All keys when all are kept.
  uint32_t key = 0;
  int left = want;
  if (want < M) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
      const uint32_t high = pass == 0 ? 0 : ~0u << (pass == 1 ? 21 : 10);
      for (int i = tid; i < bins; i += kSelectThreads) sh.hist[i] = 0;
      __syncthreads();
      for (int i0 = 0; i0 < mine; i0 += kSelectThreads) {
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
      cluster.sync();
      // thread t: bins from the top, two at a time; the digit is where their running sum reaches `left`
      int here[2] = {0, 0};
      const int top = bins - 1 - 2 * tid;
      if (top > 0) {
        for (int r = 0; r < ranks; ++r) {
          const int *other = cluster.map_shared_rank(sh.hist, r);
          here[0] += other[top];
          here[1] += other[top - 1];
        }
      }
      int all;
      const int before = block_rank(here[0] + here[1], sh.warp, all);
      if (top > 0 && before < left && before + here[0] + here[1] >= left) {
        const bool second = before + here[0] < left;
        sh.digit = top - second;
        sh.above = before + (second ? here[0] : 0);
      }
      __syncthreads();
      key |= static_cast<uint32_t>(sh.digit) << shift;
      left -= sh.above;
      cluster.sync();  // every histogram has been read
    }
  }
  // How many each slice keeps, then its kept positions in order: those above the key, and of those equal to it the first.
  int above = 0, equal = 0;
  if (want < M) {
    for (int i = tid; i < mine; i += kSelectThreads) {
      const uint32_t u = key_at(i);
      above += u > key;
      equal += u == key;
    }
    int all_above, all_equal;
    block_rank(above, sh.warp, all_above);
    block_rank(equal, sh.warp, all_equal);
    if (tid == 0) sh.count[0] = all_above, sh.count[1] = all_equal;
  }
  cluster.sync();
  int out = from;  // (all kept: in place)
  int ties_before = 0;
  if (want < M) {
    out = 0;
    for (int r = 0; r < rank; ++r) {
      const int *other = cluster.map_shared_rank(sh.count, r);
      const int ties = min(other[1], max(left - ties_before, 0));
      out += other[0] + ties;
      ties_before += other[1];
    }
  }
  cluster.sync();  // no CTA leaves while its counts are read
  for (int i0 = 0; i0 < mine; i0 += kSelectThreads) {
    const int i = i0 + tid;
    const uint32_t u = i < mine ? key_at(i) : 0;
    bool take = i < mine;
    if (want < M) {
      const bool tie = i < mine && u == key;
      int ties;
      const int before = block_rank(tie, sh.warp, ties);
      take = i < mine && (u > key || (tie && ties_before + before < left));
      ties_before += ties;
    }
    int taken;
    const int at = block_rank(take, sh.warp, taken);
    if (take) {
      kept[out + at] = from + i;
      if (kw) kw[out + at] = w[from + i];
    }
    out += taken;
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

constexpr int kGatherHeld = 4;  // 16-byte pieces that a thread holds: 128 rows of 128 bytes to a CTA

__global__ void __launch_bounds__(kGatherThreads) cache_gather_kernel(const CacheEvictParams P, int pages) {
  __shared__ float s_max[kGatherThreads / 32];
  __shared__ const uint8_t *s_row[256];
  __shared__ float s_scale[256];
  uint32_t x = blockIdx.x;
  const bool is_v = x & 1;
  x >>= 1;
  const int w = static_cast<int>(x % pages);
  x /= pages;
  const int head = static_cast<int>(x % P.c.kv_heads), b = static_cast<int>(x / P.c.kv_heads);
  const int tid = threadIdx.x, D = P.c.head_dim, shift = P.c.page_shift;
  const int rows = min(P.new_len[b] - (w << shift), 1 << shift);
  if (rows <= 0) return;
  const int32_t *kept = P.kept + (static_cast<int64_t>(b) * P.c.kv_heads + head) * P.keep + (w << shift);
  if (tid < rows) {
    const int t = kept[tid], page = page_at(P.c, b, t >> shift);
    s_row[tid] = (is_v ? P.c.v : P.c.k) + block_offset(P.c, page, head) + static_cast<int64_t>(t & ((1 << shift) - 1)) * D;
    s_scale[tid] = (is_v ? P.c.v_scale : P.c.k_scale)[page * P.c.scale_stride + head];
  }
  __syncthreads();
  const int per_row = D / 16, pieces = rows * per_row;
  uint4 held[kGatherHeld];
  float amax = 0.0f;
#pragma unroll
  for (int k = 0; k < kGatherHeld; ++k) {
    const int i = tid + k * kGatherThreads;
    if (i < pieces) held[k] = reinterpret_cast<const uint4 *>(s_row[i / per_row])[i % per_row];
  }
  auto piece_max = [&](int i, const uint4 &v) { amax = fmaxf(amax, e4m3x2_to_float2(most_of(v)).x * s_scale[i / per_row]); };
#pragma unroll
  for (int k = 0; k < kGatherHeld; ++k) {
    const int i = tid + k * kGatherThreads;
    if (i < pieces) piece_max(i, held[k]);
  }
  for (int i = tid + kGatherHeld * kGatherThreads; i < pieces; i += kGatherThreads)
    piece_max(i, reinterpret_cast<const uint4 *>(s_row[i / per_row])[i % per_row]);
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  if ((tid & 31) == 0) s_max[tid >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kGatherThreads / 32; ++i) amax = fmaxf(amax, s_max[i]);
  const float scale = block_scale(amax), inv = 1.0f / scale;  // (a power of two: exact)
  const int page = page_at(P.d, b, w);
  uint4 *to = reinterpret_cast<uint4 *>((is_v ? P.d.v : P.d.k) + block_offset(P.d, page, head));
  auto put = [&](int i, uint4 v) {
    const float s = s_scale[i / per_row];
    if (s != scale) {
      uint32_t *u = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = e4m3x2_to_float2(u[e] & 0xffff), c = e4m3x2_to_float2(u[e] >> 16);
        u[e] = to_e4m3x2(a.x * s * inv, a.y * s * inv) | to_e4m3x2(c.x * s * inv, c.y * s * inv) << 16;
      }
    }
    to[i] = v;
  };
#pragma unroll
  for (int k = 0; k < kGatherHeld; ++k) {
    const int i = tid + k * kGatherThreads;
    if (i < pieces) put(i, held[k]);
  }
  for (int i = tid + kGatherHeld * kGatherThreads; i < pieces; i += kGatherThreads)
    put(i, reinterpret_cast<const uint4 *>(s_row[i / per_row])[i % per_row]);
  if (tid == 0) (is_v ? P.d.v_scale : P.d.k_scale)[page * P.d.scale_stride + head] = scale;
}

// CTAs to a (request, head): enough for a slice of a few thousand positions,
// as many as the GPU holds at once (one CTA of 1,024 threads to an SM), and a
// slice that fits shared memory where sixteen of them can make it so.
int select_cluster(int64_t positions, int64_t heads) {
  int n = 1;
  while (n < kMaxCluster && positions / n > 4096 && heads * n * 2 <= device_sm_count()) n *= 2;
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
  cudaError_t e = once_per_device(
      [&] {
        cudaError_t r = cudaFuncSetAttribute(cache_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSliceKeys * 4);
        if (r == cudaSuccess) r = cudaFuncSetAttribute(cache_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        return r;
      },
      select_ready);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(heads * ranks);
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = room * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = trace_launch_ex("cache_select", st, [&] { return cudaLaunchKernelEx(&cfg, cache_select_kernel, P, room); });
  if (e != cudaSuccess) return e;
  const int pages = (P.keep + (1 << P.c.page_shift) - 1) >> P.c.page_shift;
  return trace_launch("cache_gather", st, [&] {
    cache_gather_kernel<<<2 * heads * pages, kGatherThreads, 0, st>>>(P, pages);
  });
}

}  // namespace sv
