// Linear attention on the tensor cores: which calls, the launches around the
// main one (state_chunk.cuh).
#include <algorithm>

#include "launch.h"
#include "state.cuh"

namespace sv {
namespace {

constexpr int kChunkRows = 64;

// Each request's status, before any of its units runs: several CTAs share a
// request, and one that gave up a wait must not be overwritten by another's OK.
__global__ void __launch_bounds__(64) state_verdict_kernel(const StateParams P, int *verdict) {
  const int b = blockIdx.x, tid = threadIdx.x;
  bool ok = true;
  state_slot(P.from, b, true, ok);
  state_slot(P.to, b, false, ok);
  int status = ok ? SPEC_STATUS_OK : SPEC_STATUS_BAD_SLOT;
  const int count = P.counts ? P.counts[b] : P.n;
  if (count < 0 || count > P.n) status = SPEC_STATUS_BAD_LENGTH;
  if (P.parents && status == SPEC_STATUS_OK) {  // (at most 64 nodes: no path is longer than SPEC_MAX_DEPTH)
    const int p = tid < count ? P.parents[static_cast<int64_t>(b) * P.n + tid] : -1;
    if (__syncthreads_or(tid < count && (tid == 0 ? p != -1 : p < 0 || p >= tid))) status = SPEC_STATUS_BAD_TREE;
  }
  if (tid == 0) {
    verdict[b] = status;
    if (P.status) P.status[b] = status;
  }
}

// From what each segment adds to zeros, the state before each: a thread to four elements of a head.
__global__ void __launch_bounds__(256) state_join_kernel(const StateChunkPlan A) {
  const StateParams &P = A.p;
  const int size = P.key_dim * P.value_dim;
  const int per = (size / 4 + 255) / 256;
  const int unit = blockIdx.x / per, e = ((blockIdx.x % per) * 256 + threadIdx.x) * 4;
  const int b = unit / P.heads, h = unit - b * P.heads;
  if (e >= size || A.verdict[b] != SPEC_STATUS_OK) return;
  float4 s = {};
  if (P.from.state) {
    const int slot = P.from.slots ? P.from.slots[b] : b;
    if (slot >= 0) s = *reinterpret_cast<const float4 *>(P.from.state + slot * P.from.slot_stride + static_cast<int64_t>(h) * size + e);
  }
  float *p = A.local + static_cast<int64_t>(unit) * A.segs * size + e;
  for (int g = 0; g < A.segs; ++g, p += size) {
    float4 x = {};
    float f = 0.0f;
    if (g + 1 < A.segs) {
      x = *reinterpret_cast<const float4 *>(p);
      f = A.total[static_cast<int64_t>(unit) * A.segs + g];
    }
    *reinterpret_cast<float4 *>(p) = s;
    s = make_float4(fmaf(s.x, f, x.x), fmaf(s.y, f, x.y), fmaf(s.z, f, x.z), fmaf(s.w, f, x.w));
  }
}

int value_blocks(const StateParams &P) { return (P.value_dim + 127) / 128; }

// Segments to a request: as many as leave no SM with a second CTA, of four chunks each at least.
int segments(const StateParams &P) {
  const int64_t units = static_cast<int64_t>(P.B) * P.heads * value_blocks(P);
  const int64_t chunks = (static_cast<int64_t>(P.n) + kChunkRows - 1) / kChunkRows;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(device_sm_count() / std::max<int64_t>(units, 1), chunks / 4)));
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

bool taken_sizes(const StateParams &P) {
  return P.key_dim <= 128 && P.n > 16 && (!P.parents || P.n <= kChunkRows) && static_cast<int64_t>(P.B) * P.heads * 2 < (1 << 26);
}

// A copy reads 64 columns of 64 tokens of one head.
cudaError_t rows_map(const void *p, const int64_t *s, int D, int heads, int n, int B, CUtensorMap *map) {
  using Encode = decltype(&cuTensorMapEncodeTiled);
  static Encode encode = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<Encode>(f);
  }();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(B)};
  const cuuint64_t one = static_cast<cuuint64_t>(D) * 2;  // (of an axis of one entry: any)
  const cuuint64_t strides[3] = {heads > 1 ? static_cast<cuuint64_t>(s[2]) * 2 : one, n > 1 ? static_cast<cuuint64_t>(s[1]) * 2 : one,
                                 B > 1 ? static_cast<cuuint64_t>(s[0]) * 2 : one};
  const cuuint32_t box[4] = {64, 1, kChunkRows, 1}, ones[4] = {1, 1, 1, 1};
  auto make = [&] {
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void *>(p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = make();
  if (r != CUDA_SUCCESS) {  // a driver's call wants a context, which a host thread has after its first call of the runtime that needs one
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaSetDevice(dev);
    if (e != cudaSuccess) return e;
    r = make();
  }
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Strides that a tensor map can hold.
bool map_strides(const int64_t *s, int heads, int n, int B) {
  const int64_t most = int64_t{1} << 38;
  auto fits = [&](int64_t x, int extent) { return extent <= 1 || (x > 0 && x < most); };
  return fits(s[0], B) && fits(s[1], n) && fits(s[2], heads);
}

}  // namespace

bool state_on_tensor_cores(const StateParams &P) {
  return P.vec && taken_sizes(P) && map_strides(P.qs, P.key_heads, P.n, P.B) && map_strides(P.ks, P.key_heads, P.n, P.B) &&
         map_strides(P.vs, P.heads, P.n, P.B);
}

size_t state_chunk_workspace(const StateParams &P) {
  if (!taken_sizes(P)) return 0;
  const size_t units = static_cast<size_t>(P.B) * P.heads;
  const int segs = segments(P);
  return round256(P.B * sizeof(int)) +
         (segs > 1 ? round256(units * segs * sizeof(float)) + units * segs * P.key_dim * P.value_dim * sizeof(float) : 0);
}

cudaError_t launch_state_chunks(const StateParams &P, void *workspace, cudaStream_t st) {
  StateChunkPlan A{};
  A.p = P;
  A.segs = segments(P);
  char *ws = static_cast<char *>(workspace);
  A.verdict = reinterpret_cast<int *>(ws);
  ws += round256(P.B * sizeof(int));
  const size_t units = static_cast<size_t>(P.B) * P.heads;
  A.total = reinterpret_cast<float *>(ws);
  A.local = reinterpret_cast<float *>(ws + round256(units * A.segs * sizeof(float)));
  CUtensorMap maps[3];
  cudaError_t e = rows_map(P.q, P.qs, P.key_dim, P.key_heads, P.n, P.B, &maps[0]);
  if (e == cudaSuccess) e = rows_map(P.k, P.ks, P.key_dim, P.key_heads, P.n, P.B, &maps[1]);
  if (e == cudaSuccess) e = rows_map(P.v, P.vs, P.value_dim, P.heads, P.n, P.B, &maps[2]);
  if (e != cudaSuccess) return e;
  e = trace_launch("state_verdict", st, [&] { state_verdict_kernel<<<P.B, 64, 0, st>>>(P, A.verdict); });
  auto chunks = P.dtype == SPEC_DTYPE_BF16 ? launch_state_chunk_bf16 : launch_state_chunk_f16;
  if (e == cudaSuccess && A.segs > 1) {
    e = chunks(A, false, maps, st);
    const int per = (P.key_dim * P.value_dim / 4 + 255) / 256;
    if (e == cudaSuccess)
      e = trace_launch("state_join", st, [&] { state_join_kernel<<<static_cast<unsigned>(units * per), 256, 0, st>>>(A); }, false);
  }
  return e == cudaSuccess ? chunks(A, true, maps, st) : e;
}

}  // namespace sv
