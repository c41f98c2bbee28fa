// Linear attention over states on the tensor cores: prompts, and drafted rows
// and trees of up to 64 nodes.
#pragma once

#include <algorithm>
#include <atomic>

#include "cache.cuh"
#include "launch.h"
#include "state.cuh"
#include "tcgen05.cuh"

namespace sv {
namespace {

// A CTA has one state head of one request, 128 columns of value_dim (lanes of
// tensor memory) and a run of chunks of 64 tokens.  With G the running sum of
// the decays within a chunk, everything is held transposed, a lane to a column
// of value_dim:
//   O1 = S^T Q^T            [dv x i]   S in pieces of 16 bits in tensor memory, Q as it came
//   P  = Q K^T              [i x j]
//   A  = P e^{G_i - G_j}, 0 where row i does not follow row j, in pieces in shared memory
//   O2 = V^T A^T            [dv x i]   V as it came
//   dS = V^T K'             [dv x dk]  K' = e^{G_last - G_j} k_j in pieces in shared memory
//   out_i = scale (e^{G_i} O1_i + O2_i),   S <- e^{G_last} S + dS
// S itself stays in fp32 registers; what a product takes of it, of A and of
// K' is the sum of pieces of the rows' type, each what those before it left
// out: three in bf16, which hold all 24 digits, two in fp16, scaled by a power
// of two (one for a lane of S, a row of A, a chunk's K') that brings the
// largest of them to 2^14: they leave out 2^-23 of a value, or 2^-39 of that
// largest where a value is less than 2^-16 of it.  The smallest pieces are added
// first, since the accumulator cuts off: after 500 chunks a state is 2.3e-7
// off on the whole (two pieces of K' in bf16: 2.4e-6; 32-bit sums: 1.8e-7),
// and bf16 outputs are as near to the plain form's as those of 32-bit sums
// (4e-5 in the root of squares; with two pieces of S and A 1e-4).
//
// e^{G_i - G_j} is taken from differences of running sums in fixed point,
// handed on as whole units of log 2 and a rest, so that a difference of large
// sums is as exact as one of small ones.
//
// Warps (their number modulo 4 is the quarter of the lanes that they can reach,
// and their scheduler): 2 loads, 3 decays, 10 issues O1 and O2, 11 issues P and dS;
// 4, 5, 8, 9 make A; 0, 1, 6, 7 write the outputs; 12 to 27 hold S, and make K'
// kAhead chunks ahead: with outputs, those of the two schedulers that have no
// warps with A (a document 671 us with all of them, 623 so).  The code of the
// roles is kept short, one site to each and loops rolled where registers allow:
// unrolled further, warps waited for their instructions.
//
// One request of 32,003 tokens, 48 heads of 128 x 128 (three to a key head), in
// a graph of calls: 640 us, of which this kernel takes 455 on 144 SMs (2.7 us a
// chunk) and the launch before it 178; the bytes are 156 us at the copy rate.
// A chunk's products take 2,600 cycles of the tensor pipe when nothing waits,
// and some 2,100 cycles of shared memory's reads, which the other warps' loads
// and stores queue behind; issue slots are used at 54%.
// 256 prompts' heads of up to 8,001 tokens: 544 us, 2.8 TB/s.
//
// A long prompt of few heads is cut into segments: a first launch (OUT false)
// computes what each but the last adds to a state of zeros, state_join_kernel
// turns that into the state before each, and the main launch has a CTA for
// every segment.
constexpr int kChunk = 64;
constexpr int kChunkThreads = 896;
constexpr int kStateWarps = 16;
template <bool OUT>
constexpr int kKeyWarps = OUT ? 8 : 16;  // those of them that make K'
constexpr int kDecayRing = 4;

// Pieces of a value that a product takes.
template <int DT>
constexpr int kPieces = DT == SPEC_DTYPE_BF16 ? 3 : 2;

template <int DT, int DK, bool OUT>
struct ChunkShape {
  static constexpr int kKeyPieces = kPieces<DT>;  // of K'
  static constexpr int kHalf = kChunk * 128;  // bytes of 64 columns of a tile
  static constexpr int kTileK = DK / 64 * kHalf, kTileV = 2 * kHalf;
  // Chunks that K' is made ahead of its use, and buffers of it: two of three pieces would leave room for two stages of values (a
  // document 761 us, one with three stages 595; in the launch before the main one, 196 of these with one buffer, 179 with two)
  static constexpr int kAhead = DK == 128 && OUT && kKeyPieces == 3 ? 1 : 2;
  static constexpr int kStagesK = DK == 64 ? 4 : OUT ? 2 : 3;
  static constexpr int kStagesV = DK == 128 && OUT ? 3 : 4;
  static constexpr int kStagesQ = OUT ? kStagesV : 0;
  static constexpr int kK = 0;
  static constexpr int kQ = kK + kStagesK * kTileK;
  static constexpr int kV = kQ + kStagesQ * kTileK;  // (P's product reads 64 rows past a half of Q: of Q, or of V)
  static constexpr int kKt = kV + kStagesV * kTileV;
  static constexpr int kA = kKt + kAhead * kKeyPieces * kTileK;
  static constexpr int kSmall = kA + (OUT ? kPieces<DT> * kHalf : 0);
  static constexpr int kBytes = kSmall + 17920 + 1024;  // (1024: alignment of the base)
  // Tensor memory: dS, P in its place while K' is made; S's pieces; O1, two in turn; O2.  (One O1 and a place for P alone: a document
  // 701 us, since the outputs then stand between two chunks' O1.)
  static constexpr uint32_t kDS = 0, kP = 0, kS = 128, kPieceS = DK / 2, kO1 = 320, kO2 = 448;
  static_assert(kS + kPieces<DT> * kPieceS <= kO1);
};

struct alignas(16) Decays {
  float nhi[kChunk], nlo[kChunk];  // minus the running sum in units of log 2: whole ones, rest
  float ei[kChunk], more[kChunk];  // scale e^{G_i}: the product of both; more is written where grows is true, else all are 1
  float left[kChunk];              // e^{G_last - G_j}, 0 past the request's rows
  float afac[kChunk];              // fp16: what row i of A was divided by
  float sfac[128];                 // fp16: what a lane of S was divided by
  float lam, lam_more;             // e^{G_last}: the product of both
  int grows;
  float kfac;                      // fp16: what K' was divided by
};

struct ChunkSmall {
  Decays d[kDecayRing];
  alignas(16) uint16_t stage[4][16][32];  // outputs on their way
  uint32_t smax[2][4][128], amax[2][2][kChunk];  // (by the chunk's number: the next one's may be written before these are read)
  // One barrier for each product, counted by chunk (four of them in turn, so that whoever waits for a chunk's phase is never a
  // lap behind): that P, O1, O2, dS are there, and so that their operands are free.
  uint64_t p_full[4], o1_full[4], o2_full[4], ds_full[4];
  uint64_t full[4], k_read[4];  // a chunk's rows loaded; its keys read by those who make K'
  uint64_t kt_full[2], p_empty, a_full, ds_empty, s_full, o_empty;
  uint64_t dec_full[kDecayRing], dec_empty[kDecayRing], meet_s, meet_a;
  uint32_t tmem;
  int dead;
  int copies, products_p, products_o1, products_o2, products_s;  // how many were begun
};
static_assert(sizeof(ChunkSmall) <= 17920);
template <int DT>
constexpr bool chunks_fit() {
  return ChunkShape<DT, 128, true>::kBytes <= 232448 && ChunkShape<DT, 128, false>::kBytes <= 232448 && ChunkShape<DT, 64, true>::kBytes <= 232448 &&
         ChunkShape<DT, 64, false>::kBytes <= 232448;
}
static_assert(chunks_fit<SPEC_DTYPE_BF16>() && chunks_fit<SPEC_DTYPE_F16>());

// Arrival of a warp whose lanes have all done what the barrier stands for.
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
  __syncwarp();
  if (lane == 0) bar_arrive(bar);
}

// The rows' type: code in an instruction descriptor (fp16 0, bf16 1).
template <int DT>
__device__ __forceinline__ constexpr uint32_t rows_desc(int n, bool a_mn, bool b_mn) {
  return mma_desc(n, b_mn) | (DT == SPEC_DTYPE_BF16 ? 1u << 7 | 1u << 10 : 0u) | (a_mn ? 1u << 15 : 0u);
}

__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
      : "memory");
}

__device__ __forceinline__ void tensor_load_4d(void *dst, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// What a value of the rows' type leaves out of an fp32 one: an instruction that takes both.
template <int DT>
__device__ __forceinline__ float left_out(uint16_t piece, float x) {
  float r;
  if constexpr (DT == SPEC_DTYPE_BF16) asm("fma.rn.f32.bf16 %0, %1, %2, %3;" : "=f"(r) : "h"(piece), "h"(static_cast<uint16_t>(0xbf80)), "f"(x));
  else asm("fma.rn.f32.f16 %0, %1, %2, %3;" : "=f"(r) : "h"(piece), "h"(static_cast<uint16_t>(0xbc00)), "f"(x));
  return r;
}

// Two values in pieces of the rows' type.  fp16: each rounds what the ones before it left out.  bf16: each cuts off what follows its 8
// digits, so that no finite value becomes an infinity.
template <int DT>
__device__ __forceinline__ void split(pair_t v, uint32_t *piece, int stride) {
  float2 x = unpack2(v);
#pragma unroll
  for (int p = 0; p < kPieces<DT>; ++p) {
    const uint32_t w = DT == SPEC_DTYPE_BF16 ? __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632) : narrow2<DT>(x);
    piece[p * stride] = w;
    if (p + 1 < kPieces<DT>) x = make_float2(left_out<DT>(static_cast<uint16_t>(w), x.x), left_out<DT>(static_cast<uint16_t>(w >> 16), x.y));
  }
}

// The power of two that brings a largest magnitude (as bits) to [2^14, 2^15), and its inverse; 1 for zero, infinities and NaN.
__device__ __forceinline__ float fit_half(uint32_t amax, float &back) {
  const int e = static_cast<int>(amax >> 23) - 127;
  const int s = amax == 0 || e == 128 ? 0 : max(-112, min(112, 14 - e));
  back = __uint_as_float(static_cast<uint32_t>(127 - s) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + s) << 23);
}

// The largest finite magnitude of a key in fp16 (its 16-byte pieces from another one on in each lane: other banks).
template <int DK>
__device__ __forceinline__ float largest_key(const char *keys, int row) {
  const char *at = keys + row * 128;
  __half2 most = __half2half2(__ushort_as_half(0));
#pragma unroll 4
  for (int e = 0; e < DK / 8; ++e) {
    const uint4 v = *reinterpret_cast<const uint4 *>(at + (e >> 3) * kChunk * 128 + ((e ^ threadIdx.x) & 7) * 16);
    const __half2 *x = reinterpret_cast<const __half2 *>(&v);
    most = __hmax2(most, __hmax2(__hmax2(__habs2(x[0]), __habs2(x[1])), __hmax2(__habs2(x[2]), __habs2(x[3]))));
  }
  const float2 two = __half22float2(most);
  float top = fmaxf(two.x, two.y);
  if (!(top < INFINITY)) [[unlikely]] {
    top = 0.0f;
#pragma unroll 1
    for (int e = 0; e < DK; ++e) {
      const float x = fabsf(__half2float(*reinterpret_cast<const __half *>(at + (e >> 6) * kChunk * 128 + (e & 63) * 2)));
      top = x < INFINITY ? fmaxf(top, x) : top;
    }
  }
  return top;
}

// Row i's weight for row j without what P held: e^{G_i - G_j} from the handed-on parts.
__device__ __forceinline__ float between(const Decays &d, int i, int j) {
  return ex2((d.nhi[j] - d.nhi[i]) + (d.nlo[j] - d.nlo[i]));
}

// The decays of a chunk: two tokens next to one another to a lane.  Sums up to each of them, the whole's, and where a NaN has a part.
struct ChunkSums {
  Log2Sum g0, g1, total;
  bool bad0, bad1, spoilt;
};

__device__ __forceinline__ ChunkSums chunk_sums(float x0, float x1, int lane) {
  ChunkSums s{log2_of(x0), log2_of(x1)};
  const uint32_t nan0 = __ballot_sync(~0u, x0 != x0), nan1 = __ballot_sync(~0u, x1 != x1);
  s.g1 += s.g0;  // the lane's two, then the lanes before it
  const Log2Sum before = running<32>(s.g1, lane) - s.g1;
  s.g0 += before, s.g1 += before;
  s.total = of_lane(s.g1, 31);
  const uint32_t to = (2u << lane) - 1, under = to >> 1;
  s.bad0 = nan0 & to || nan1 & under, s.bad1 = nan0 & to || nan1 & to;
  s.spoilt = nan0 || nan1;
  return s;
}

__device__ __forceinline__ void put_sums(Decays &d, const ChunkSums &s, float scale, float scale_log2, int lane) {
  const Log2Parts p0 = s.g0.parts(s.bad0), p1 = s.g1.parts(s.bad1);
  *reinterpret_cast<float2 *>(&d.nhi[2 * lane]) = make_float2(-p0.hi, -p1.hi);
  *reinterpret_cast<float2 *>(&d.nlo[2 * lane]) = make_float2(-p0.lo, -p1.lo);
  float2 more;
  *reinterpret_cast<float2 *>(&d.ei[2 * lane]) = make_float2(state_factor(p0, scale, scale_log2, more.x), state_factor(p1, scale, scale_log2, more.y));
  const bool grows = __any_sync(~0u, more.x != 1.0f || more.y != 1.0f);
  if (grows) [[unlikely]] *reinterpret_cast<float2 *>(&d.more[2 * lane]) = more;
  if (lane == 0) d.grows = grows;
}

// 32 weights of a row of A from what P's product left in tensor memory: scale P e^{G_i - G_j}, 0 for rows that it does not follow
// (bits of sees), in pairs; the largest magnitude's bits.  A whole warp.
template <int DT>
__device__ __forceinline__ uint32_t pair_weights(uint32_t p, const Decays &d, int i, int j0, uint32_t sees, float log2_scale, pair_t *y) {
  float x[32];
  tmem_ld32(p + j0, x);
  const float mh = -d.nhi[i], ml = log2_scale - d.nlo[i];
  const pair_t h2 = pack2(mh, mh), l2 = pack2(ml, ml);
  const bool every = __all_sync(~0u, sees == ~0u);
  tc_wait_ld();
  uint32_t most = 0;
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    const ulonglong2 nh = *reinterpret_cast<const ulonglong2 *>(&d.nhi[j0 + 2 * e]);
    const ulonglong2 nl = *reinterpret_cast<const ulonglong2 *>(&d.nlo[j0 + 2 * e]);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const float2 g = unpack2(add2(add2(h2, w ? nh.y : nh.x), add2(l2, w ? nl.y : nl.x)));
      float2 z = unpack2(mul2(pack2(x[2 * (e + w)], x[2 * (e + w) + 1]), pack2(ex2(g.x), ex2(g.y))));
      if (!every) {
        z.x = sees >> (2 * (e + w)) & 1 ? z.x : 0.0f;
        z.y = sees >> (2 * (e + w) + 1) & 1 ? z.y : 0.0f;
      }
      if constexpr (DT == SPEC_DTYPE_F16) most = max(most, max(__float_as_uint(z.x) & 0x7fffffffu, __float_as_uint(z.y) & 0x7fffffffu));
      y[e + w] = pack2(z.x, z.y);
    }
  }
  return most;
}

// Half of a row of A, scaled by fit, to shared memory: its pieces lie kHalf bytes apart.  Zeros where any is false (one for a warp).
template <int DT>
__device__ __forceinline__ void put_weights(char *a, int i, int half, const pair_t *y, float fit, bool any) {
  char *row = a + i * 128;
  const pair_t f = pack2(fit, fit);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t w[kPieces<DT>][4] = {};
    if (any) {
#pragma unroll
      for (int x = 0; x < 4; ++x) split<DT>(DT == SPEC_DTYPE_F16 ? mul2(y[4 * e + x], f) : y[4 * e + x], &w[0][x], 4);
    }
    const int to = ((half * 4 + e) ^ (i & 7)) << 4;
#pragma unroll
    for (int p = 0; p < kPieces<DT>; ++p)
      *reinterpret_cast<uint4 *>(row + p * kChunk * 128 + to) = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
  }
}

// 16 tokens' outputs from k on, from a column of value_dim to a lane through shared memory to 16 bytes of a token's row to a lane
// (of the token that out points at and the eighth after it; out goes on to the sixteenth).  bad: no number where a sum of O2 is none.
template <int DT>
__device__ __forceinline__ void put_outputs(uint32_t o1, uint32_t o2, const Decays &d, int k, int m, float sf, uint16_t *stage, char *&out,
                                            int64_t stride, bool store, pair_t &bad) {
  const int lane = threadIdx.x & 31, token = lane >> 2;
  const pair_t sf2 = pack2(sf, sf), none = 0;
  float x[16], y[16];
  tmem_ld16(o1 + k, x);
  tmem_ld16(o2 + k, y);
  tc_wait_ld();
  if (k + 16 > m) [[unlikely]] {
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e] = k + e < m ? y[e] : 0.0f;
  }
  __syncwarp();
#pragma unroll
  for (int e = 0; e < 16; e += 4) {
    const ulonglong2 ei = *reinterpret_cast<const ulonglong2 *>(&d.ei[k + e]);
    ulonglong2 af;
    if constexpr (DT == SPEC_DTYPE_F16) af = *reinterpret_cast<const ulonglong2 *>(&d.afac[k + e]);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int z = e + 2 * w;
      pair_t f = w ? ei.y : ei.x, v = pack2(y[z], y[z + 1]);
      bad = fma2(v, none, bad);
      if constexpr (DT == SPEC_DTYPE_F16) f = mul2(f, sf2), v = mul2(v, w ? af.y : af.x);
      const uint32_t u2 = narrow2<DT>(unpack2(fma2(pack2(x[z], x[z + 1]), f, v)));
      stage[z * 32 + lane] = static_cast<uint16_t>(u2);
      stage[(z + 1) * 32 + lane] = static_cast<uint16_t>(u2 >> 16);
    }
  }
  __syncwarp();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (store && k + token + 8 * e < m) *reinterpret_cast<uint4 *>(out) = *reinterpret_cast<const uint4 *>(stage + e * 256 + lane * 8);
    out += stride * 16;
  }
}

// A row's sum over the rows that it follows, taken again from memory without
// those that it does not: where a value of theirs is infinite or NaN, the
// product of a weight of 0 is not 0.  A warp: lane = column of value_dim.
template <int DT>
__device__ __noinline__ float row_again(const StateParams &P, const Decays &d, uint64_t sees, int b, int h, int t0, int i, int col) {
  const int hk = h / P.group, lane = threadIdx.x & 31;
  const uint16_t *q = reinterpret_cast<const uint16_t *>(P.q) + b * P.qs[0] + (t0 + i) * P.qs[1] + hk * P.qs[2];
  float sum = 0.0f;
  for (int j = 0; j <= i; ++j) {
    if (!(sees >> j & 1)) continue;
    const uint16_t *k = reinterpret_cast<const uint16_t *>(P.k) + b * P.ks[0] + (t0 + j) * P.ks[1] + hk * P.ks[2];
    float s = 0.0f;
    for (int e = lane; e < P.key_dim; e += 32) s = fmaf(widen<DT>(q[e]), widen<DT>(k[e]), s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    if (col < P.value_dim) {
      const uint16_t *v = reinterpret_cast<const uint16_t *>(P.v) + b * P.vs[0] + (t0 + j) * P.vs[1] + h * P.vs[2];
      sum = fmaf(s * between(d, i, j), widen<DT>(v[col]), sum);
    }
  }
  return sum;
}

// Waits for every copy and product that the CTA began.
static __device__ __noinline__ void land_chunks(ChunkSmall &sm) {
  ring_land(sm.full, 4, sm.copies);
  ring_land(sm.p_full, 4, sm.products_p);
  ring_land(sm.o1_full, 4, sm.products_o1);
  ring_land(sm.o2_full, 4, sm.products_o2);
  ring_land(sm.ds_full, 4, sm.products_s);
}

template <int DT, int DK, bool OUT>
__global__ void __launch_bounds__(kChunkThreads, 1)
    state_chunk_kernel(const StateChunkPlan A, const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map) {
  using S = ChunkShape<DT, DK, OUT>;
  constexpr bool F16 = DT == SPEC_DTYPE_F16;
  constexpr uint32_t kDS = S::kDS, kO2 = S::kO2, kP = S::kP;
  extern __shared__ char raw[];
  char *const smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  ChunkSmall &sm = *reinterpret_cast<ChunkSmall *>(smem + S::kSmall);
  const StateParams &P = A.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  pdl_wait();
  // ---- the unit: heads next to one another share keys, so they run side by side
  const int blocks = (P.value_dim + 127) >> 7;
  int u = blockIdx.x;
  const int h = u % P.heads;
  u /= P.heads;
  const int dv0 = u % blocks * 128;
  u /= blocks;
  // (the longest requests first)
  const int piece = u % A.pieces, b = A.order[u / A.pieces], seg = OUT ? piece : piece / A.parts;
  const int hk = h / P.group;
  const bool ok = A.verdict[b] == SPEC_STATUS_OK;
  const int len = ok ? (P.counts ? P.counts[b] : P.n) : 0;
  const int all = (len + kChunk - 1) / kChunk;
  int c0 = static_cast<int>(static_cast<int64_t>(all) * seg / A.segs);
  int chunks = static_cast<int>(static_cast<int64_t>(all) * (seg + 1) / A.segs) - c0;
  if (!OUT) {  // a part of the segment
    const int part = piece - seg * A.parts, of = chunks;
    c0 += static_cast<int>(static_cast<int64_t>(of) * part / A.parts);
    chunks = static_cast<int>(static_cast<int64_t>(of) * (part + 1) / A.parts) - static_cast<int>(static_cast<int64_t>(of) * part / A.parts);
  }
  const bool last_seg = seg + 1 == A.segs;
  // (a chunk's state is needed by the next, and by whoever reads the state written)
  const bool writes = OUT ? last_seg && P.to.state && ok : true;
  const int updates = writes ? chunks : max(chunks - 1, 0);

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      bar_init(&sm.full[i], 1), bar_init(&sm.k_read[i], kKeyWarps<OUT> + (F16 ? 1 : 0));
      bar_init(&sm.p_full[i], 1), bar_init(&sm.o1_full[i], 1), bar_init(&sm.o2_full[i], 1), bar_init(&sm.ds_full[i], 1);
    }
    for (int i = 0; i < 2; ++i) bar_init(&sm.kt_full[i], kKeyWarps<OUT>);
    bar_init(&sm.p_empty, 4), bar_init(&sm.a_full, 4), bar_init(&sm.ds_empty, kStateWarps), bar_init(&sm.s_full, kStateWarps), bar_init(&sm.o_empty, 4);
    for (int i = 0; i < kDecayRing; ++i) bar_init(&sm.dec_full[i], 1), bar_init(&sm.dec_empty[i], OUT ? kStateWarps + 8 : kStateWarps);
    bar_init(&sm.meet_s, kStateWarps), bar_init(&sm.meet_a, 4);
    bar_init_fence();
    sm.dead = 0;
    sm.copies = sm.products_p = sm.products_o1 = sm.products_o2 = sm.products_s = 0;
  }
  if (warp == 10) tmem_alloc(&sm.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  volatile int *dead = &sm.dead;
  auto o1_of = [&](int c) -> uint32_t { return tmem + S::kO1 + (c & 1) * 64; };
  // of the barriers counted by chunk
  auto wait4 = [&](uint64_t *bars, int c) -> bool { return warp_wait(&bars[c & 3], c >> 2 & 1, dead); };

  if (warp == 2) {
    // ---- loading
    int n = 0;
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
      const int t0 = (c0 + c) * kChunk;
      const int sk = c % S::kStagesK, sv = c % S::kStagesV;
      // the stages' last products: P and K' of the keys, O1 of the queries, O2 and dS of the values
      const int k = c - S::kStagesK, v = c - S::kStagesV;
      if (k >= 0 && !(wait4(sm.k_read, k) && (!OUT || wait4(sm.p_full, k)))) break;
      if (v >= 0 && !((v >= updates || wait4(sm.ds_full, v)) && (!OUT || (wait4(sm.o1_full, v) && wait4(sm.o2_full, v))))) break;
      if (lane == 0) {
        uint64_t *full = &sm.full[c & 3];
        bar_expect(full, (OUT ? 2 : 1) * S::kTileK + S::kTileV);
        for (int e = 0; e < DK / 64; ++e) {
          tensor_load_4d(smem + S::kK + sk * S::kTileK + e * S::kHalf, &k_map, e * 64, hk, t0, b, full);
          if (OUT) tensor_load_4d(smem + S::kQ + sv * S::kTileK + e * S::kHalf, &q_map, e * 64, hk, t0, b, full);
        }
        for (int e = 0; e < 2; ++e) tensor_load_4d(smem + S::kV + sv * S::kTileV + e * S::kHalf, &v_map, dv0 + e * 64, h, t0, b, full);
      }
      ++n;
      __syncwarp();
    }
    if (lane == 0) sm.copies = n;
  } else if (warp == 3) {
    // ---- decays: two tokens next to one another to a lane
    const float *gp = P.decay + b * P.gs[0] + h * P.gs[2];
    long long whole = 0, rest = 0;  // of the segment's sum: units of log 2, 2^-40ths
    auto fetch = [&](int c, float &x0, float &x1) {
      const int t = (c0 + c) * kChunk + 2 * lane;
      x0 = c < chunks && t < len ? gp[t * P.gs[1]] : 0.0f;
      x1 = c < chunks && t + 1 < len ? gp[(t + 1) * P.gs[1]] : 0.0f;
    };
    float x0, x1;
    bool lost = false, forgot = false;
    fetch(0, x0, x1);
    for (int c = 0; c < chunks; ++c) {
      const int r = c % kDecayRing, t0 = (c0 + c) * kChunk;
      const int m = min(kChunk, len - t0);
      const ChunkSums sums = chunk_sums(x0, x1, lane);
      fetch(c + 1, x0, x1);
      rest += sums.total.units;
      whole += rest >> kLog2Bits, rest &= (1ll << kLog2Bits) - 1;
      lost |= sums.spoilt, forgot |= sums.total.units < kForgets / 2;
      if (c >= kDecayRing && !warp_wait(&sm.dec_empty[r], (c / kDecayRing - 1) & 1, dead)) break;
      Decays &d = sm.d[r];
      put_sums(d, sums, P.scale, P.scale_log2, lane);
      const Log2Parts q0 = (sums.total - sums.g0).parts(sums.spoilt), q1 = (sums.total - sums.g1).parts(sums.spoilt);
      *reinterpret_cast<float2 *>(&d.left[2 * lane]) = make_float2(2 * lane < m ? q0.power() : 0.0f, 2 * lane + 1 < m ? q1.power() : 0.0f);
      if (lane == 0) d.lam = state_factor(sums.total.parts(sums.spoilt), 1.0f, 0.0f, d.lam_more);
      if constexpr (F16) {  // K' divided by the power of two that its largest finite value asks for, as these factors go into it
        if (!wait4(sm.full, c)) break;
        const char *keys = smem + S::kK + c % S::kStagesK * S::kTileK;
        const float2 left = *reinterpret_cast<const float2 *>(&d.left[2 * lane]);
        const float most = fmaxf(largest_key<DK>(keys, 2 * lane) * left.x, largest_key<DK>(keys, 2 * lane + 1) * left.y);
        warp_arrive(&sm.k_read[c & 3], lane);
        float back;
        const float fit = fit_half(__reduce_max_sync(~0u, __float_as_uint(fmaxf(most, 0.0f))), back);
        // (no infinity for a key of zeros: the others' stay below 2^39; NaN stays)
        auto kept = [](float x) { return x > 0x1p126f ? 0x1p126f : x; };
        *reinterpret_cast<float2 *>(&d.left[2 * lane]) = make_float2(kept(left.x * fit), kept(left.y * fit));
        if (lane == 0) d.kfac = back;
      }
      warp_arrive(&sm.dec_full[r], lane);
    }
    if (!OUT && lane == 0 && dv0 == 0) {  // (the whole part no further than fp32's exponents)
      const Log2Sum all_of{((forgot ? -4096ll : max(-4096ll, min(4096ll, whole))) << kLog2Bits) + rest};
      const Log2Parts p = all_of.parts(lost);
      A.total[(static_cast<int64_t>(b) * P.heads + h) * A.slots() + piece] = make_float2(p.hi, p.lo);
    }
  } else if (warp == 10) {
    // ---- issuing O1 and O2
    if constexpr (OUT) {
      constexpr uint32_t kId1 = rows_desc<DT>(kChunk, false, false), kId2 = rows_desc<DT>(kChunk, true, false);
      const uint64_t q_desc = matrix_desc(smem_u32(smem + S::kQ), 16, 1024, kSwizzle128);
      const uint64_t v_desc = matrix_desc(smem_u32(smem + S::kV), S::kHalf, 1024, kSwizzle128);
      const uint64_t a_desc = matrix_desc(smem_u32(smem + S::kA), 16, 1024, kSwizzle128);
      int n1 = 0, n2 = 0;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        const int sv = c % S::kStagesV;
        if (!wait4(sm.full, c)) break;
        if (!warp_wait(&sm.s_full, c & 1, dead)) break;
        tc_fence_after();
        if (elect_one()) {  // (into the one that chunk c - 2 left: its outputs were waited for before the last O2)
#pragma unroll 1
          for (int x = 0; x < kPieces<DT> * DK / 64; ++x) {  // a piece's 64 columns of a half of Q, the smallest piece first
            const int half = x % (DK / 64), p = kPieces<DT> - 1 - x / (DK / 64);
            const uint32_t piece = tmem + S::kS + p * S::kPieceS + half * 32;
            const uint64_t q = q_desc + ((sv * S::kTileK + half * S::kHalf) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f16_ta(o1_of(c), piece + k * 8, q + 2 * k, kId1, x + k > 0);
          }
          tc_commit(&sm.o1_full[c & 3]);
        }
        __syncwarp();
        ++n1;
        if (!warp_wait(&sm.a_full, c & 1, dead)) break;
        if (c > 0 && !warp_wait(&sm.o_empty, (c - 1) & 1, dead)) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll 1
          for (int p = kPieces<DT> - 1; p >= 0; --p) {
            const uint64_t v = v_desc + ((sv * S::kTileV) >> 4), a = a_desc + ((p * S::kHalf) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f16_ss(tmem + kO2, v + 128 * k, a + 2 * k, kId2, p + 1 < kPieces<DT> || k > 0);
          }
          tc_commit(&sm.o2_full[c & 3]);
        }
        __syncwarp();
        ++n2;
      }
      if (lane == 0) sm.products_o1 = n1, sm.products_o2 = n2;
    }
  } else if (warp == 11) {
    // ---- issuing P and dS
    constexpr uint32_t kIdP = rows_desc<DT>(kChunk, false, false), kIdS = rows_desc<DT>(DK, true, true);
    const uint64_t q_desc = matrix_desc(smem_u32(smem + S::kQ), 16, 1024, kSwizzle128);
    const uint64_t k_desc = matrix_desc(smem_u32(smem + S::kK), 16, 1024, kSwizzle128);
    const uint64_t v_desc = matrix_desc(smem_u32(smem + S::kV), S::kHalf, 1024, kSwizzle128);
    const uint64_t kt_desc = matrix_desc(smem_u32(smem + S::kKt), S::kHalf, 1024, kSwizzle128);
    int np = 0, ns = 0;
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
      if (!wait4(sm.full, c)) break;
      if (c > 0 && !warp_wait(&sm.ds_empty, (c - 1) & 1, dead)) break;  // (every chunk but the last has a dS)
      if (OUT) {
        const int sk = c % S::kStagesK, sq = c % S::kStagesV;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll 1
          for (int x = 0; x < DK / 64; ++x) {
            const uint64_t q = q_desc + ((sq * S::kTileK + x * S::kHalf) >> 4), k0 = k_desc + ((sk * S::kTileK + x * S::kHalf) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f16_ss(tmem + kP, q + 2 * k, k0 + 2 * k, kIdP, x + k > 0);
          }
          tc_commit(&sm.p_full[c & 3]);
        }
        __syncwarp();
        ++np;
      }
      if (c < updates) {
        if (OUT && !warp_wait(&sm.p_empty, c & 1, dead)) break;
        if (!warp_wait(&sm.kt_full[c % S::kAhead], c / S::kAhead & 1, dead)) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll 1
          for (int piece = S::kKeyPieces - 1; piece >= 0; --piece) {  // (the smallest first: the accumulator cuts off)
            const uint64_t v = v_desc + ((c % S::kStagesV * S::kTileV) >> 4);
            const uint64_t kt = kt_desc + (((c % S::kAhead * S::kKeyPieces + piece) * S::kTileK) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f16_ss(tmem + kDS, v + 128 * k, kt + 128 * k, kIdS, piece + 1 < S::kKeyPieces || k > 0);
          }
          tc_commit(&sm.ds_full[c & 3]);
        }
        __syncwarp();
        ++ns;
      }
    }
    if (lane == 0) sm.products_p = np, sm.products_s = ns;
  } else if (warp >= 12) {
    // ---- the state: a quarter of a lane's row to a thread, in pairs of columns
    constexpr int OWN = DK / 4;
    const int four = (warp - 12) >> 2, at = (warp & 3) * 32 + lane, dv = dv0 + at;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const int64_t size = static_cast<int64_t>(P.key_dim) * P.value_dim;
    pair_t s[OWN / 2];
#pragma unroll
    for (int e = 0; e < OWN / 2; ++e) s[e] = 0;
    const float *from = nullptr;
    if (OUT && A.segs > 1) {
      from = A.local + ((static_cast<int64_t>(b) * P.heads + h) * A.slots() + seg * A.parts) * size;
    } else if (OUT && ok && P.from.state) {
      const int slot = P.from.slots ? P.from.slots[b] : b;
      if (slot >= 0) from = P.from.state + slot * P.from.slot_stride + h * size;
    }
    if (from && ok && dv < P.value_dim) {
#pragma unroll
      for (int e = 0; e < OWN / 2; ++e) {
        const int d = four * OWN + 2 * e;
        if (d < P.key_dim) s[e] = pack2(from[static_cast<int64_t>(d) * P.value_dim + dv], from[static_cast<int64_t>(d + 1) * P.value_dim + dv]);
      }
    }
    // fp16: a thread's part of what the scale of chunk c's pieces is taken from
    auto show_most = [&](int c) {
      uint32_t most = 0;
#pragma unroll
      for (int e = 0; e < OWN / 2; ++e) {
        const float2 x = unpack2(s[e]);
        most = max(most, max(__float_as_uint(x.x) & 0x7fffffffu, __float_as_uint(x.y) & 0x7fffffffu));
      }
      sm.smax[c & 1][four][at] = most;
      warp_arrive(&sm.meet_s, lane);
    };
    // the pieces of S that chunk c's product takes
    auto hand_on = [&](int c) -> bool {
      pair_t f = 0;
      if constexpr (F16) {
        if (!warp_wait(&sm.meet_s, c & 1, dead)) return false;
        float back;
        const auto &tops = sm.smax[c & 1];
        const float fit = fit_half(max(max(tops[0][at], tops[1][at]), max(tops[2][at], tops[3][at])), back);
        f = pack2(fit, fit);
        if (four == 0) sm.d[c % kDecayRing].sfac[at] = back;
      }
      if (c > 0 && !wait4(sm.o1_full, c - 1)) return false;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < OWN / 16; ++k) {
        uint32_t w[kPieces<DT>][8];
#pragma unroll
        for (int e = 0; e < 8; ++e) split<DT>(F16 ? mul2(s[8 * k + e], f) : s[8 * k + e], &w[0][e], 8);
#pragma unroll
        for (int p = 0; p < kPieces<DT>; ++p) tmem_st8(tmem + lanes + S::kS + p * S::kPieceS + four * (OWN / 2) + k * 8, w[p]);
      }
      tc_wait_st();
      tc_fence_before();
      warp_arrive(&sm.s_full, lane);
      return true;
    };
    // K' of chunk c
    constexpr int kParts = DK / 4 / kKeyWarps<OUT>;  // 16 bytes each, of a row to a thread
    const bool makes = !OUT || (warp & 2);
    const int own = (OUT ? four * 2 + (warp & 1) : warp - 12) * 32 + lane, row = own & 63, part = (own >> 6) * kParts;
    auto keys = [&](int c) -> bool {
      const int r = c % kDecayRing, sk = c % S::kStagesK, m = min(kChunk, len - (c0 + c) * kChunk);
      if (!warp_wait(&sm.dec_full[r], (c / kDecayRing) & 1, dead)) return false;
      if (!wait4(sm.full, c)) return false;
      if (c < updates) {
        if (c >= S::kAhead && !wait4(sm.ds_full, c - S::kAhead)) return false;
        const float left = sm.d[r].left[row];
        const bool past = row >= m;
        const int base = (part >> 3) * S::kHalf + row * 128, first = part & 7;
        const char *from = smem + S::kK + sk * S::kTileK + base;
        char *to = smem + S::kKt + c % S::kAhead * S::kKeyPieces * S::kTileK + base;
        const pair_t f = pack2(left, left);
#pragma unroll 2
        for (int e = 0; e < kParts; ++e) {
          const int o = ((first + e) ^ (row & 7)) << 4;
          const uint4 x = *reinterpret_cast<const uint4 *>(from + o);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
          uint32_t pieces[S::kKeyPieces][4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float2 k = widen2<DT>(w[y]);
            split<DT>(mul2(pack2(k.x, k.y), f), &pieces[0][y], 4);
          }
          if (past) [[unlikely]] {
#pragma unroll
            for (int y = 0; y < 4 * S::kKeyPieces; ++y) pieces[0][y] = 0;
          }
#pragma unroll
          for (int y = 0; y < S::kKeyPieces; ++y)
            *reinterpret_cast<uint4 *>(to + y * S::kTileK + o) = make_uint4(pieces[y][0], pieces[y][1], pieces[y][2], pieces[y][3]);
        }
        if (m < kChunk) {
          const int sv = c % S::kStagesV;
          for (int e = own; e < (kChunk - m) * 16; e += 32 * kKeyWarps<OUT>)
            *reinterpret_cast<uint4 *>(smem + S::kV + sv * S::kTileV + (e & 1) * S::kHalf + (m + (e >> 4)) * 128 + (e >> 1 & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_async_shared();
        warp_arrive(&sm.kt_full[c % S::kAhead], lane);
      }
      warp_arrive(&sm.k_read[c & 3], lane);
      return true;
    };
    bool going = true;
    if (OUT && F16 && chunks > 0) show_most(0);
#pragma unroll 1
    for (int c = -S::kAhead; c < chunks; ++c) {
      const int r = c & (kDecayRing - 1);
      if (OUT && c >= 0 && !(going = hand_on(c))) break;
      // K' before the update where it is two chunks ahead; fp16's maxima have its time to meet
      constexpr bool kKeysFirst = S::kAhead == 2 && !F16;
      if (kKeysFirst && makes && c + S::kAhead < chunks && !(going = keys(c + S::kAhead))) break;
      if (c >= 0) {
        if (!(going = warp_wait(&sm.dec_full[r], (c / kDecayRing) & 1, dead))) break;
        if (c < updates) {
          if (!(going = wait4(sm.ds_full, c))) break;
          tc_fence_after();
          const float lam = sm.d[r].lam, kf = F16 ? sm.d[r].kfac : 1.0f;
          const pair_t l2 = pack2(lam, lam), k2 = pack2(kf, kf);
          if (sm.d[r].grows) [[unlikely]] {
            const pair_t more = pack2(sm.d[r].lam_more, sm.d[r].lam_more);
#pragma unroll
            for (int e = 0; e < OWN / 2; ++e) s[e] = mul2(s[e], more);
          }
#pragma unroll
          for (int k = 0; k < OWN / 16; ++k) {
            float x[16];
            tmem_ld16(tmem + lanes + kDS + four * OWN + k * 16, x);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              pair_t &y = s[8 * k + e];
              if constexpr (F16) y = fma2(pack2(x[2 * e], x[2 * e + 1]), k2, mul2(y, l2));
              else y = fma2(y, l2, pack2(x[2 * e], x[2 * e + 1]));
            }
          }
          tc_fence_before();
          warp_arrive(&sm.ds_empty, lane);
        }
        warp_arrive(&sm.dec_empty[r], lane);
        if (OUT && F16 && c + 1 < chunks) show_most(c + 1);
      }
      if (!kKeysFirst && makes && c + S::kAhead < chunks && !(going = keys(c + S::kAhead))) break;
    }
    float *to = nullptr;
    if (!OUT) {
      to = A.local + ((static_cast<int64_t>(b) * P.heads + h) * A.slots() + piece) * size;
    } else if (writes && going) {
      to = P.to.state + (P.to.slots ? P.to.slots[b] : b) * P.to.slot_stride + h * size;
    }
    if (to && dv < P.value_dim) {
#pragma unroll
      for (int e = 0; e < OWN / 2; ++e) {
        const int d = four * OWN + 2 * e;
        const float2 x = unpack2(s[e]);
        if (d < P.key_dim) to[static_cast<int64_t>(d) * P.value_dim + dv] = x.x, to[static_cast<int64_t>(d + 1) * P.value_dim + dv] = x.y;
      }
    }
  } else if (warp == 4 || warp == 5 || warp == 8 || warp == 9) {
    // ---- A: half of a row to a thread
    if constexpr (OUT) {
      const int i = (warp & 1) * 32 + lane, half = warp >> 3, j0 = half * 32;
      const int group = (warp >> 3) * 64 + i;  // the thread among the 128
      const float log2_scale = log2f(P.scale);
      int met = 0;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        const int r = c % kDecayRing, m = min(kChunk, len - (c0 + c) * kChunk);
        if (!warp_wait(&sm.dec_full[r], (c / kDecayRing) & 1, dead)) break;
        if (!wait4(sm.p_full, c)) break;
        tc_fence_after();
        const Decays &d = sm.d[r];
        // which of the half's rows this one follows
        const uint32_t sees = i >= j0 + 31 ? ~0u : i < j0 ? 0u : (2u << (i - j0)) - 1;
        pair_t y[16];
        float fit = 1.0f, back = 1.0f;
        const bool any = __any_sync(~0u, sees != 0);
        if (any) {
          const uint32_t most = pair_weights<DT>(tmem + (static_cast<uint32_t>(warp & 3) << 21) + kP, d, i, j0, sees, log2_scale, y);
          if constexpr (F16) sm.amax[c & 1][half][i] = most;
          tc_fence_before();
          warp_arrive(&sm.p_empty, lane);
          if constexpr (F16) {
            warp_arrive(&sm.meet_a, lane);
            if (!warp_wait(&sm.meet_a, met++ & 1, dead)) break;
            fit = fit_half(max(most, sm.amax[c & 1][half ^ 1][i]), back);
          }
        } else {
          warp_arrive(&sm.p_empty, lane);
          if constexpr (F16) {
            sm.amax[c & 1][half][i] = 0;
            warp_arrive(&sm.meet_a, lane);
            if (!warp_wait(&sm.meet_a, met++ & 1, dead)) break;
            fit_half(sm.amax[c & 1][half ^ 1][i], back);
          }
        }
        if (F16 && half == 0) sm.d[r].afac[i] = back;
        if (c > 0 && !wait4(sm.o2_full, c - 1)) break;
        put_weights<DT>(smem + S::kA, i, half, y, fit, any);
        if (m < kChunk) {  // values past the request's rows take no part, whatever they are
          const int sv = c % S::kStagesV;
          if (!wait4(sm.full, c)) break;
          for (int e = group; e < (kChunk - m) * 16; e += 128)
            *reinterpret_cast<uint4 *>(smem + S::kV + sv * S::kTileV + (e & 1) * S::kHalf + (m + (e >> 4)) * 128 + (e >> 1 & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_async_shared();
        warp_arrive(&sm.a_full, lane);
        warp_arrive(&sm.dec_empty[r], lane);
      }
    }
  } else {
    // ---- the outputs
    const int quarter = warp & 3, at = quarter * 32 + lane;
    if constexpr (OUT) {
      const uint32_t lanes = static_cast<uint32_t>(quarter) << 21;
      const int dv = dv0 + at;
      uint16_t *out = reinterpret_cast<uint16_t *>(P.out) + b * P.os[0] + h * P.os[2] + dv;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        const int r = c % kDecayRing, t0 = (c0 + c) * kChunk, m = min(kChunk, len - t0);
        if (!wait4(sm.o2_full, c)) break;
        tc_fence_after();
        const Decays &d = sm.d[r];
        const float sf = F16 ? d.sfac[at] : 1.0f;
        pair_t bad = 0;
        const int col = quarter * 32 + (lane & 3) * 8;
        char *o = reinterpret_cast<char *>(P.out) + (b * P.os[0] + h * P.os[2] + (t0 + (lane >> 2)) * P.os[1] + dv0 + col) * 2;
#pragma unroll 1
        for (int k = 0; k < kChunk; k += 16)
          put_outputs<DT>(o1_of(c) + lanes, tmem + lanes + kO2, d, k, m, sf, sm.stage[quarter][0], o, P.os[1],
                          dv0 + col < P.value_dim, bad);
        const float2 b2 = unpack2(bad);
        if (__any_sync(~0u, !(b2.x == 0.0f && b2.y == 0.0f)) || d.grows) [[unlikely]] {  // a row's sum that is no number: without the rows that it
          // does not follow; or growth beyond one factor
          __syncwarp();  // (other lanes' stores of the same rows)
#pragma unroll 1
          for (int i = 0; i < m; ++i) {
            const uint64_t sees = (2ull << i) - 1;
            float x[8];
            tmem_ld8(o1_of(c) + lanes + (i & ~7), x);
            tc_wait_ld();
            float v = x[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) v = (i & 7) == e ? x[e] : v;
            v = fmaf(d.grows ? v * d.more[i] : v, d.ei[i] * sf, row_again<DT>(P, d, sees, b, h, t0, i, dv) * P.scale);
            if (dv < P.value_dim) out[(t0 + i) * P.os[1]] = narrow<DT>(v);
          }
        }
        tc_fence_before();
        warp_arrive(&sm.o_empty, lane);
        warp_arrive(&sm.dec_empty[r], lane);
      }
      // rows past the count: each segment's share of them
      const int pieces = min(128, P.value_dim - dv0) >> 3;
      const int64_t gap = P.n - len, z0 = gap * seg / A.segs, z1 = gap * (seg + 1) / A.segs;
      uint16_t *o = reinterpret_cast<uint16_t *>(P.out) + b * P.os[0] + h * P.os[2] + dv0;
      for (int64_t e = at; e < (z1 - z0) * pieces; e += 128)
        *reinterpret_cast<uint4 *>(o + (len + z0 + e / pieces) * P.os[1] + e % pieces * 8) = make_uint4(0, 0, 0, 0);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*dead) [[unlikely]] {  // nothing that was begun may reach shared or tensor memory that the CTA has left (else all was waited for)
    if (warp == 0) land_chunks(sm);
    __syncthreads();
    if (tid == 0 && P.status) atomicMax(&P.status[b], SPEC_STATUS_TIMEOUT);
  }
  tc_fence_after();
  if (warp == 10) tmem_free(tmem, 512);
}

// A launch whose blocks may start before the kernel in front of it has ended (they wait for it before they read anything it wrote).
template <class Kernel>
cudaError_t launch_behind(Kernel kern, unsigned grid, int threads, int bytes, cudaStream_t st, const StateChunkPlan &A, const CUtensorMap *maps) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = trace_enabled() ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, kern, A, maps[0], maps[1], maps[2]);
}

template <int DT, int DK, bool OUT>
std::atomic<uint64_t> chunk_smem{0};

template <int DT, int DK, bool OUT>
cudaError_t launch_chunks(const StateChunkPlan &A, const CUtensorMap *maps, cudaStream_t st) {
  using S = ChunkShape<DT, DK, OUT>;
  auto kern = state_chunk_kernel<DT, DK, OUT>;
  const cudaError_t e =
      once_per_device([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes); }, chunk_smem<DT, DK, OUT>);
  if (e != cudaSuccess) return e;
  StateChunkPlan B = A;
  B.pieces = OUT ? A.segs : (A.segs - 1) * A.parts;
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(A.p.B) * B.pieces * ((A.p.value_dim + 127) / 128) * A.p.heads);
  const bool again = !state_overlaps(A.p);
  return trace_launch_ex(OUT ? "state_chunk" : "state_chunk_local", st, [&] { return launch_behind(kern, grid, kChunkThreads, S::kBytes, st, B, maps); },
                         again || !OUT);
}

// ------------------------------------------------------------------ up to 64 rows over states that stay
//
// A chain or a tree of one chunk, nothing written but outputs: a CTA for each
// (request, head, 128 columns) goes through the steps above once, P's columns
// of tensor memory becoming O2's, so that two CTAs share an SM and one loads
// its state while the other computes.  16 trees of 60 nodes, 48 heads: 64 us
// as a chunk of the kernel above (one CTA to an SM), 34 us so.  Half of tensor
// memory holds two of S's pieces at a time: in bf16 the largest waits in
// registers until O1 has taken the others.
constexpr int kShortThreads = 256;

template <int DT, int DK>
struct ShortShape {
  static constexpr int kHalf = kChunk * 128;
  static constexpr int kTileK = DK / 64 * kHalf, kTileV = 2 * kHalf;
  static constexpr int kQ = 0, kK = kQ + kTileK, kV = kK + kTileK, kA = kV + kTileV, kSmall = kA + kPieces<DT> * kHalf;
  static constexpr int kBytes = kSmall + 14336 + 1024;
};

struct ShortSmall {
  Decays d;
  alignas(16) uint16_t stage[8][16][32];
  uint32_t follows[kChunk][2];  // the rows that a row follows, itself among them
  uint32_t smax[2][128], amax[2][kChunk];
  int parent[kChunk];
  long long units[kChunk];  // the nodes' decays
  uint64_t full, p_full, o1_full, o2_full;
  uint32_t tmem;
  int dead;
};
static_assert(sizeof(ShortSmall) <= 14336 && ShortShape<SPEC_DTYPE_BF16, 128>::kBytes <= 113 * 1024);

template <int DT, int DK>
__global__ void __launch_bounds__(kShortThreads, 2)
    state_short_kernel(const StateChunkPlan A, const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                       const __grid_constant__ CUtensorMap v_map) {
  using S = ShortShape<DT, DK>;
  constexpr bool F16 = DT == SPEC_DTYPE_F16;
  constexpr uint32_t kS = 0, kO1 = 128, kP = 192;  // tensor memory: two of S's pieces, the smaller first; O2 in P's place
  extern __shared__ char raw[];
  char *const smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  ShortSmall &sm = *reinterpret_cast<ShortSmall *>(smem + S::kSmall);
  const StateParams &P = A.p;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quarter = warp & 3, half = warp >> 2, at = quarter * 32 + lane;
  const uint32_t lanes = static_cast<uint32_t>(quarter) << 21;
  if (tid == 0) {
    bar_init(&sm.full, 1), bar_init(&sm.p_full, 1), bar_init(&sm.o1_full, 1), bar_init(&sm.o2_full, 1);
    bar_init_fence();
    sm.dead = 0;
  }
  if (warp == 0) tmem_alloc(&sm.tmem, 256);
  pdl_wait();
  const int blocks = (P.value_dim + 127) >> 7;
  int u = blockIdx.x;
  const int h = u % P.heads;
  u /= P.heads;
  const int dv0 = u % blocks * 128, b = u / blocks, hk = h / P.group, dv = dv0 + at;
  const bool ok = A.verdict[b] == SPEC_STATUS_OK;
  const int m = ok ? (P.counts ? P.counts[b] : P.n) : 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  volatile int *dead = &sm.dead;

  if (m > 0) {
    if (tid == 0) {
      bar_expect(&sm.full, 2 * S::kTileK + S::kTileV);
      for (int e = 0; e < DK / 64; ++e) {
        tensor_load_4d(smem + S::kQ + e * S::kHalf, &q_map, e * 64, hk, 0, b, &sm.full);
        tensor_load_4d(smem + S::kK + e * S::kHalf, &k_map, e * 64, hk, 0, b, &sm.full);
      }
      for (int e = 0; e < 2; ++e) tensor_load_4d(smem + S::kV + e * S::kHalf, &v_map, dv0 + e * 64, h, 0, b, &sm.full);
    }
    __syncwarp();
    // ---- the state: half of a lane's row to a thread, its pieces to tensor memory
    constexpr int OWN = DK / 2;
    float s[OWN];
    const float *from = nullptr;
    const int64_t size = static_cast<int64_t>(P.key_dim) * P.value_dim;
    if (P.from.state) {
      const int slot = P.from.slots ? P.from.slots[b] : b;
      if (slot >= 0) from = P.from.state + slot * P.from.slot_stride + h * size;
    }
    const bool mine = from && dv < P.value_dim;
#pragma unroll
    for (int e = 0; e < OWN; ++e) {
      const int d = half * OWN + e;
      s[e] = mine && d < P.key_dim ? from[static_cast<int64_t>(d) * P.value_dim + dv] : 0.0f;
    }
    // ---- the decays, while the state is on its way
    if (warp == 1) {
      const float *gp = P.decay + b * P.gs[0] + h * P.gs[2];
      ChunkSums sums;
      if (P.parents) {  // over each row's path, and which rows lie on it
        uint32_t nan[2];
        for (int e = 0; e < 2; ++e) {
          const int i = lane + 32 * e;
          const float x = i < m ? gp[i * P.gs[1]] : 0.0f;
          if (i < m) sm.parent[i] = P.parents[static_cast<int64_t>(b) * P.n + i], sm.units[i] = log2_of(x).units;
          nan[e] = __ballot_sync(~0u, x != x);
        }
        __syncwarp();
        for (int e = 0; e < 2; ++e) {
          const int i = 2 * lane + e;
          uint32_t bits[2] = {0, 0};
          Log2Sum path{0};
          if (i < m) {
            for (int p = i; p >= 0; p = sm.parent[p]) {
              path += Log2Sum{sm.units[p]};
              bits[p >> 5] |= 1u << (p & 31);
            }
          }
          sm.follows[i][0] = bits[0], sm.follows[i][1] = bits[1];
          (e ? sums.g1 : sums.g0) = path, (e ? sums.bad1 : sums.bad0) = bits[0] & nan[0] || bits[1] & nan[1];
        }
      } else {
        sums = chunk_sums(2 * lane < m ? gp[2 * lane * P.gs[1]] : 0.0f, 2 * lane + 1 < m ? gp[(2 * lane + 1) * P.gs[1]] : 0.0f, lane);
        for (int e = 0; e < 2; ++e) {
          const uint64_t bits = (2ull << (2 * lane + e)) - 1;
          sm.follows[2 * lane + e][0] = static_cast<uint32_t>(bits), sm.follows[2 * lane + e][1] = static_cast<uint32_t>(bits >> 32);
        }
      }
      put_sums(sm.d, sums, P.scale, P.scale_log2, lane);
    }
    float sf = 1.0f;
    if constexpr (F16) {
      uint32_t most = 0;
#pragma unroll
      for (int e = 0; e < OWN; ++e) most = max(most, __float_as_uint(s[e]) & 0x7fffffffu);
      sm.smax[half][at] = most;
      __syncthreads();
      const float fit = fit_half(max(most, sm.smax[half ^ 1][at]), sf);
#pragma unroll
      for (int e = 0; e < OWN; ++e) s[e] *= fit;
    }
    constexpr int kLast = kPieces<DT> - 1;
    uint32_t largest[kLast == 2 ? OWN / 2 : 1];
#pragma unroll
    for (int k = 0; k < OWN / 16; ++k) {
      uint32_t w[kPieces<DT>][8];
#pragma unroll
      for (int e = 0; e < 8; ++e) split<DT>(pack2(s[16 * k + 2 * e], s[16 * k + 2 * e + 1]), &w[0][e], 8);
      tmem_st8(tmem + lanes + kS + half * (OWN / 2) + k * 8, w[kLast]);
      tmem_st8(tmem + lanes + kS + 64 + half * (OWN / 2) + k * 8, w[kLast - 1]);
      if constexpr (kLast == 2) {
#pragma unroll
        for (int e = 0; e < 8; ++e) largest[8 * k + e] = w[0][e];
      }
    }
    tc_wait_st();
    tc_fence_before();
    __syncthreads();
    // ---- O1 of two pieces, P
    int begun = 0;  // products (warp 0)
    constexpr uint32_t kId = rows_desc<DT>(kChunk, false, false);
    const uint64_t q_desc = matrix_desc(smem_u32(smem + S::kQ), 16, 1024, kSwizzle128);
    auto piece_product = [&](int place, bool more) {  // (one lane)
#pragma unroll 1
      for (int x = 0; x < DK / 64; ++x)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f16_ta(tmem + kO1, tmem + kS + place * 64 + x * 32 + k * 8, q_desc + ((x * S::kHalf) >> 4) + 2 * k, kId, more || x + k > 0);
    };
    if (warp == 0 && warp_wait(&sm.full, 0, dead)) {
      tc_fence_after();
      if (elect_one()) {
        const uint64_t k_desc = matrix_desc(smem_u32(smem + S::kK), 16, 1024, kSwizzle128);
#pragma unroll 1
        for (int place = 0; place < 2; ++place) piece_product(place, place > 0);
        tc_commit(&sm.o1_full);
#pragma unroll 1
        for (int x = 0; x < DK / 64; ++x)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16_ss(tmem + kP, q_desc + ((x * S::kHalf) >> 4) + 2 * k, k_desc + ((x * S::kHalf) >> 4) + 2 * k, kId, x + k > 0);
        tc_commit(&sm.p_full);
      }
      begun = 2;
    }
    __syncwarp();
    if constexpr (kLast == 2) {  // the largest piece in the smallest's place
      if (warp_wait(&sm.o1_full, 0, dead)) {
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < OWN / 16; ++k) tmem_st8(tmem + lanes + kS + half * (OWN / 2) + k * 8, largest + 8 * k);
        tc_wait_st();
        tc_fence_before();
      }
    }
    // ---- A: half of a row to a thread of the lower lanes
    const int i = at;
    uint32_t most = 0;
    pair_t y[16];
    bool any = false;
    if (quarter < 2 && warp_wait(&sm.p_full, 0, dead)) {
      tc_fence_after();
      const uint32_t sees = sm.follows[i][half];
      any = __any_sync(~0u, sees != 0);
      if (any) most = pair_weights<DT>(tmem + lanes + kP, sm.d, i, half * 32, sees, log2f(P.scale), y);
    }
    float fit = 1.0f;
    if constexpr (F16) {
      if (quarter < 2) sm.amax[half][i] = most;
      __syncthreads();
      if (quarter < 2) {
        float back;
        fit = fit_half(max(most, sm.amax[half ^ 1][i]), back);
        if (half == 0) sm.d.afac[i] = back;
      }
    }
    if (quarter < 2) {
      put_weights<DT>(smem + S::kA, i, half, y, fit, any);
    } else {  // values past the request's rows take no part, whatever they are (their copy has landed when P has)
      if (warp_wait(&sm.full, 0, dead))
        for (int e = (half * 2 + quarter - 2) * 32 + lane; e < (kChunk - m) * 16; e += 128)
          *reinterpret_cast<uint4 *>(smem + S::kV + (e & 1) * S::kHalf + (m + (e >> 4)) * 128 + (e >> 1 & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_async_shared();
    tc_fence_before();
    __syncthreads();
    // ---- O1 of the largest piece, O2
    const bool off = __any_sync(~0u, *dead);
    if (warp == 0 && !off) {
      tc_fence_after();
      if (elect_one()) {
        if (kLast == 2) piece_product(0, true);
        constexpr uint32_t kIdO = rows_desc<DT>(kChunk, true, false);
        const uint64_t v_desc = matrix_desc(smem_u32(smem + S::kV), S::kHalf, 1024, kSwizzle128);
        const uint64_t a_desc = matrix_desc(smem_u32(smem + S::kA), 16, 1024, kSwizzle128);
#pragma unroll 1
        for (int p = kLast; p >= 0; --p)
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_f16_ss(tmem + kP, v_desc + 128 * k, a_desc + ((p * S::kHalf) >> 4) + 2 * k, kIdO, p < kLast || k > 0);
        tc_commit(&sm.o2_full);
      }
      begun = 3;
    }
    __syncwarp();
    // ---- the outputs: half of the tokens to a warp
    if (!off && warp_wait(&sm.o1_full, 0, dead) && warp_wait(&sm.o2_full, 0, dead)) {
      tc_fence_after();
      pair_t bad = 0;
      const int col = quarter * 32 + (lane & 3) * 8;
      char *o = reinterpret_cast<char *>(P.out) + (b * P.os[0] + h * P.os[2] + (half * 32 + (lane >> 2)) * P.os[1] + dv0 + col) * 2;
#pragma unroll 1
      for (int k = half * 32; k < half * 32 + 32 && k < m; k += 16)
        put_outputs<DT>(tmem + lanes + kO1, tmem + lanes + kP, sm.d, k, m, sf, sm.stage[warp][0], o, P.os[1], dv0 + col < P.value_dim, bad);
      const float2 b2 = unpack2(bad);
      if (__any_sync(~0u, !(b2.x == 0.0f && b2.y == 0.0f)) || sm.d.grows) [[unlikely]] {  // as in the kernel above
        __syncwarp();
#pragma unroll 1
        for (int r = half * 32; r < min(m, half * 32 + 32); ++r) {
          float x[8];
          tmem_ld8(tmem + lanes + kO1 + (r & ~7), x);
          tc_wait_ld();
          float v = x[0];
#pragma unroll
          for (int e = 1; e < 8; ++e) v = (r & 7) == e ? x[e] : v;
          const uint64_t sees = static_cast<uint64_t>(sm.follows[r][1]) << 32 | sm.follows[r][0];
          v = fmaf(sm.d.grows ? v * sm.d.more[r] : v, sm.d.ei[r] * sf, row_again<DT>(P, sm.d, sees, b, h, 0, r, dv) * P.scale);
          if (dv < P.value_dim) reinterpret_cast<uint16_t *>(P.out)[b * P.os[0] + r * P.os[1] + h * P.os[2] + dv] = narrow<DT>(v);
        }
      }
    }
    if (warp == 0 && __any_sync(~0u, *dead)) [[unlikely]] {  // (nothing that was begun may reach memory that the CTA has left)
      ring_land(&sm.full, 1, 1);
      if (begun >= 1) ring_land(&sm.p_full, 1, 1), ring_land(&sm.o1_full, 1, 1);
      if (begun == 3) ring_land(&sm.o2_full, 1, 1);
    }
  }
  // rows past the count
  const int pieces = min(128, P.value_dim - dv0) >> 3;
  uint16_t *o = reinterpret_cast<uint16_t *>(P.out) + b * P.os[0] + h * P.os[2] + dv0;
  for (int e = tid; e < (P.n - m) * pieces; e += kShortThreads)
    *reinterpret_cast<uint4 *>(o + (m + e / pieces) * P.os[1] + e % pieces * 8) = make_uint4(0, 0, 0, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && *dead && P.status) atomicMax(&P.status[b], SPEC_STATUS_TIMEOUT);
  if (warp == 0) tmem_free(tmem, 256);
}

template <int DT, int DK>
std::atomic<uint64_t> short_smem{0};

template <int DT, int DK>
cudaError_t launch_short(const StateChunkPlan &A, const CUtensorMap *maps, cudaStream_t st) {
  auto kern = state_short_kernel<DT, DK>;
  const int bytes = ShortShape<DT, DK>::kBytes;
  const cudaError_t e = once_per_device([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); }, short_smem<DT, DK>);
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(A.p.B) * ((A.p.value_dim + 127) / 128) * A.p.heads);
  return trace_launch_ex("state_short", st, [&] { return launch_behind(kern, grid, kShortThreads, bytes, st, A, maps); });
}

}  // namespace
}  // namespace sv
