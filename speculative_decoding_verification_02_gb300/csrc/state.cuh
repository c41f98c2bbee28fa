// Shared parts of the linear-attention kernels: the pool of states, the
// parameter blocks, packed arithmetic.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "spec_verify.h"

namespace sv {

// Bits of a decay's fraction in fixed point (units of log 2).
constexpr int kLog2Bits = 40;

struct StatePool {
  float *state;  // null: states of zeros (read), or none to write
  int64_t slot_stride;
  int num_slots;
  const int32_t *slots;
};

struct StateParams {
  StatePool from, to;
  int heads, key_heads, group, key_dim, value_dim;  // group: state heads to a key head
  const char *q, *k, *v;
  char *out;
  int64_t qs[3], ks[3], vs[3], os[3], gs[3];  // element strides: request, token, head
  int dtype, B, n, n_rows, index_stride;
  const float *decay;
  const int32_t *counts, *parents, *index;
  float scale, scale_log2;  // |scale| < 2^scale_log2, which is not below 0
  int64_t most_units;       // of a decay of the state's that one factor holds beside the scale: 2^-40ths of log 2
  int32_t *status;
  bool vec;  // rows of q, k, v and out start on 16-byte boundaries
};

// A call of the tensor-core kernels: each request's chunks cut into segs runs, the states before all but the first of them from
// a launch of their own, which has parts CTAs for each run but the last.
struct StateChunkPlan {
  StateParams p;
  int segs, parts, pieces;  // pieces: of a request, a launch's
  int *verdict;   // [B] the requests' status
  int *order;     // [B] the requests, longest first
  float2 *total;  // [B][heads][slots] the decay over a part: whole units of log 2, rest
  float *local;   // [B][heads][slots][key_dim][value_dim] what a part adds to zeros; then, where a run begins, the state before it
  __host__ __device__ int slots() const { return (segs - 1) * parts + 1; }
};

// Whether the states written lie where some are read: such a call is not the same call when it is made again.
inline bool state_overlaps(const StateParams &P) {
  if (!P.from.state || !P.to.state) return false;
  const float *a = P.from.state, *b = P.to.state;
  return a < b + P.to.num_slots * P.to.slot_stride && b < a + P.from.num_slots * P.from.slot_stride;
}

// Whether the tensor-core kernels take a call, from its sizes and layout; the workspace that they need (for any layout).
bool state_on_tensor_cores(const StateParams &P);
size_t state_chunk_workspace(const StateParams &P);
cudaError_t launch_state_chunks(const StateParams &P, void *workspace, cudaStream_t st);
cudaError_t launch_state_chunk_bf16(const StateChunkPlan &A, bool outputs, const CUtensorMap *maps, cudaStream_t st);
cudaError_t launch_state_chunk_f16(const StateChunkPlan &A, bool outputs, const CUtensorMap *maps, cudaStream_t st);
cudaError_t launch_state_short_bf16(const StateChunkPlan &A, const CUtensorMap *maps, cudaStream_t st);
cudaError_t launch_state_short_f16(const StateChunkPlan &A, const CUtensorMap *maps, cudaStream_t st);

// A launch of the kernels for a few rows: chains (q given: with outputs), commits (q null), trees (parents given).
cudaError_t launch_state_rows(const StateParams &P, cudaStream_t st);

#ifdef __CUDACC__

// Slot of request b, -1 for a state of zeros; ok is false when there is none.
__device__ __forceinline__ int state_slot(const StatePool &p, int b, bool may_lack, bool &ok) {
  if (!p.state) return -1;
  const int s = p.slots ? p.slots[b] : b;
  if (s >= p.num_slots || s < (may_lack ? -1 : 0)) ok = false;
  return s;
}

// Two fp32 values to a register pair, and arithmetic on both at once.
using pair_t = unsigned long long;
__device__ __forceinline__ pair_t pack2(float a, float b) {
  pair_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(pair_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ pair_t fma2(pair_t a, pair_t b, pair_t c) {
  pair_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ pair_t mul2(pair_t a, pair_t b) {
  pair_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ pair_t add2(pair_t a, pair_t b) {
  pair_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Two values of a row in one word to fp32, exactly.
template <int DT>
__device__ __forceinline__ float2 widen2(uint32_t w) {
  if constexpr (DT == SPEC_DTYPE_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <int DT>
__device__ __forceinline__ float widen(uint16_t w) {
  if constexpr (DT == SPEC_DTYPE_BF16) return __uint_as_float(static_cast<uint32_t>(w) << 16);
  else return __half2float(__ushort_as_half(w));
}
// Rounded once, to nearest even.
template <int DT>
__device__ __forceinline__ uint32_t narrow2(float2 x) {
  uint32_t r;
  if constexpr (DT == SPEC_DTYPE_BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x.y), "f"(x.x));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x.y), "f"(x.x));
  return r;
}
template <int DT>
__device__ __forceinline__ uint16_t narrow(float x) {
  if constexpr (DT == SPEC_DTYPE_BF16) return __bfloat16_as_ushort(__float2bfloat16(x));
  else return __half_as_ushort(__float2half(x));
}

// A sum of decays in units of log 2, in fixed point of 64 bits: 2^-40ths.  A
// token's is off by one of them (1e-12, which a decay that is the same for a
// million tokens adds up to 1e-6), sums and differences not at all, however
// large: what 64-bit floats would do at many times the cost.
struct Log2Parts {
  float hi, lo;  // a whole number and a rest in [-1/2, 1/2]
  __device__ __forceinline__ float power() const {  // 2^(hi + lo), subnormal or infinite where fp32 is; NaN stays
    const int h = static_cast<int>(fminf(fmaxf(hi, -252.0f), 254.0f)), most = min(max(h, -126), 127);
    const float f = exp2f(lo) * __uint_as_float(static_cast<uint32_t>(most + 127) << 23) * __uint_as_float(static_cast<uint32_t>(h - most + 127) << 23);
    return hi == hi ? f : hi;
  }
};
// scale 2^(hi + lo), by which sums over the state are multiplied, in two finite
// factors, so that a state of zeros stays one and a small one grows to what it
// should: the second is 1 unless the first alone would be no number.
// scale_log2: 0 or above, scale is below its power of two.
__device__ __forceinline__ float state_factor(const Log2Parts &p, float scale, float scale_log2, float &second) {
  second = 1.0f;
  if (!(p.hi + scale_log2 > 126.0f)) [[likely]] return p.power() * scale;
  const int half = min(127, (static_cast<int>(p.hi + scale_log2) + 1) >> 1);
  const float hi = p.hi - static_cast<float>(half);
  second = __uint_as_float(static_cast<uint32_t>(half + 127) << 23);
  return Log2Parts{fminf(hi, 127.0f), p.lo}.power() * scale;
}
struct Log2Sum {
  long long units;
  __device__ __forceinline__ Log2Sum &operator+=(const Log2Sum &x) {
    units += x.units;
    return *this;
  }
  __device__ __forceinline__ Log2Sum operator-(const Log2Sum &x) const { return Log2Sum{units - x.units}; }
  __device__ __forceinline__ Log2Parts parts(bool nan) const {
    const int whole = static_cast<int>((units + (1ll << (kLog2Bits - 1))) >> kLog2Bits);
    const int rest = static_cast<int>((units - (static_cast<long long>(whole) << kLog2Bits)) >> (kLog2Bits - 32));  // 2^-32ths
    return Log2Parts{nan ? NAN : static_cast<float>(whole), static_cast<float>(rest) * 0x1p-32f};
  }
};
__device__ __forceinline__ Log2Sum of_lane(const Log2Sum &x, int lane) { return Log2Sum{__shfl_sync(~0u, x.units, lane)}; }
// The sum over a lane's own and those of the lanes below it.
template <int LANES>
__device__ __forceinline__ Log2Sum running(Log2Sum x, int lane) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    const Log2Sum y{__shfl_up_sync(~0u, x.units, o)};
    if (lane >= o) x += y;
  }
  return x;
}
// A natural logarithm.  Below -120 the factor is 0, and so is every product with it, whatever grows behind it: 64 tokens' growth, of
// 174 units at most each (beyond 120 an infinite factor in fp32 whatever it is), stays far below kForgets.  NaN gives 0.
constexpr long long kForgets = -(1ll << (kLog2Bits + 15));
__device__ __forceinline__ Log2Sum log2_of(float g) {
  if (g < -120.0f) return Log2Sum{kForgets};
  const float x = fminf(g, 120.0f);
  const float y = x * 1.44269502f, e = fmaf(x, 1.44269502f, -y) + x * 1.92596303e-8f;  // log2(e) in two parts
  const float w = rintf(y);
  const long long units = (static_cast<long long>(static_cast<int>(w)) << kLog2Bits) + __float2ll_rn((y - w) * 0x1p40f) + __float2int_rn(e * 0x1p40f);
  return Log2Sum{g == g ? units : 0};
}

#endif

}  // namespace sv
