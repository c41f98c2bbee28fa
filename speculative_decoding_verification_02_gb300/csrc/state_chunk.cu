// Linear attention on the tensor cores: which calls, the launches around the
// main one (state_chunk.cuh).
#include <algorithm>
#include <utility>

#include "launch.h"
#include "state.cuh"

namespace sv {
namespace {

constexpr int kChunkRows = 64;
constexpr int64_t kMostUnits = 1 << 26;  // (CTAs are numbered by an int, segments and halves of value_dim among them)
constexpr int kSortedRequests = 4096;  // (each counts those before it)

__device__ __forceinline__ int block_sum64(int x) {
  __shared__ int part[2];
  x = __reduce_add_sync(~0u, x);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  return part[0] + part[1];
}

// Each request's status, before any of its units runs: several CTAs share a
// request, and one that gave up a wait must not be overwritten by another's OK.
// And the requests' order, longest first, so that the launch's last CTAs are short.
__global__ void __launch_bounds__(64) state_verdict_kernel(const StateParams P, int *verdict, int *order) {
  pdl_launch_dependents();
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
  int before = 0;
  const bool sorted = P.counts && P.B <= kSortedRequests;
  if (sorted)
    for (int i = tid; i < P.B; i += 64) before += P.counts[i] > count || (P.counts[i] == count && i < b);
  before = sorted ? block_sum64(before) : b;
  if (tid == 0) {
    order[before] = b;
    verdict[b] = status;
    if (P.status) P.status[b] = status;
  }
}

// From what each segment adds to zeros, the state before each: a thread to four elements of a head.
__global__ void __launch_bounds__(256) state_join_kernel(const StateChunkPlan A) {
  pdl_launch_dependents();
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
  float *p = A.local + static_cast<int64_t>(unit) * A.slots() * size + e;
  const float2 *f = A.total + static_cast<int64_t>(unit) * A.slots();
  float4 ahead = *reinterpret_cast<const float4 *>(p);
  for (int g = 0; g + 1 < A.slots(); ++g, p += size) {
    const float4 x = ahead;
    if (g + 2 < A.slots()) ahead = *reinterpret_cast<const float4 *>(p + size);
    if (g % A.parts == 0) *reinterpret_cast<float4 *>(p) = s;
    float more;
    const float w = state_factor(Log2Parts{f[g].x, f[g].y}, 1.0f, 0.0f, more);
    s = make_float4(fmaf(s.x * more, w, x.x), fmaf(s.y * more, w, x.y), fmaf(s.z * more, w, x.z), fmaf(s.w * more, w, x.w));
  }
  *reinterpret_cast<float4 *>(p) = s;
}

int value_blocks(const StateParams &P) { return (P.value_dim + 127) / 128; }

// One chunk's rows over states that are only read.
bool is_short(const StateParams &P) { return P.n <= kChunkRows && !P.to.state; }

// Segments to a request: as many as leave no SM with a second CTA, of four chunks each at least.
int segments(const StateParams &P) {
  const int64_t units = static_cast<int64_t>(P.B) * P.heads * value_blocks(P);
  const int64_t chunks = (static_cast<int64_t>(P.n) + kChunkRows - 1) / kChunkRows;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(device_sm_count() / std::max<int64_t>(units, 1), chunks / 4)));
}

// CTAs to a segment in the launch before: the finer, the fewer SMs stay without one in its last turn.
int segment_parts(const StateParams &P, int segs) {
  if (segs < 2) return 1;
  const int64_t units = static_cast<int64_t>(P.B) * P.heads * value_blocks(P) * (segs - 1), sms = device_sm_count();
  const int64_t chunks = (static_cast<int64_t>(P.n) + kChunkRows - 1) / kChunkRows / segs;
  int best = 1;
  double least = 1e30;
  for (int p = 1; p <= 4 && p * 4 <= std::max<int64_t>(chunks, 4); ++p) {
    const double turns = static_cast<double>((units * p + sms - 1) / sms) / p;
    if (turns < least * 0.95) best = p, least = turns;
  }
  return best;
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// A call's plan over a workspace, and the workspace's size.
std::pair<StateChunkPlan, size_t> chunk_plan(const StateParams &P, void *workspace) {
  StateChunkPlan A{};
  A.p = P;
  A.segs = segments(P);
  A.parts = segment_parts(P, A.segs);
  const size_t per_head = A.segs > 1 ? static_cast<size_t>(P.B) * P.heads * A.slots() : 0;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char *p = static_cast<char *>(workspace) + at;
    at += round256(bytes);
    return workspace ? p : nullptr;
  };
  A.verdict = reinterpret_cast<int *>(take(P.B * sizeof(int)));
  A.order = reinterpret_cast<int *>(take(P.B * sizeof(int)));
  A.total = reinterpret_cast<float2 *>(take(per_head * sizeof(float2)));
  A.local = reinterpret_cast<float *>(take(per_head * P.key_dim * P.value_dim * sizeof(float)));
  return {A, at};
}

// Fewest tokens of a call.  48 heads of 128 x 128, bf16, in a graph of calls, the kernel for few rows against these, us (1, 8 and 64
// requests):
//   chains, states only read  8 rows 6.6 / 8.2, 13 / 15, 72 / 82; 9 rows 7.7 / 8.3, 15 / 15, 86 / 83; 12 rows 8.7 / 8.2, 17 / 15, 98 / 83.
//                             Of drafts of different lengths the one for few rows does those that there are: 9 rows at most
//                             6.3 / 8.7, 13 / 16, 70 / 84; 12 rows 8.3 / 8.6, 15 / 16, 80 / 85; 16 rows 7.2 / 8.6, 18 / 16, 94 / 85
//   trees (a path of rows)    4 rows 8.7 / 8.3, 16 / 16, 113 / 84; 8 rows 16 / 8.7, 28 / 16, 202 / 88
//   states written            16 tokens 12 / 12, 29 / 32, 173 / 256; 24: 17 / 12, 40 / 32, 244 / 257; 32: 21 / 12, 50 / 32, 317 / 257
//                             (a CTA of the main kernel has an SM to itself, and its start is not hidden: the more units, the later
//                             it pays)
// A state of 16 heads of 64 x 64, fp16, is a twelfth of that, and the kernels meet later where there are many:
//   chains                    12 rows 6.8 / 7.2, 6.9 / 7.4, 14 / 24; 16 rows 8.0 / 7.2, 8.1 / 7.5, 17 / 24; 24 rows 12 / 7.4, 12 / 7.7, 29 / 26
//   states written            24 tokens 13 / 10, 13 / 10, 33 / 55; 64: 29 / 10, 30 / 10, 78 / 55
// n is the padded length: of a batch whose requests have few of it, the one for few rows does those that there are.
int fewest_tokens(const StateParams &P) {
  if (P.parents) return 4;
  if (is_short(P)) return P.counts ? 12 : 9;
  return static_cast<int64_t>(P.B) * P.heads * value_blocks(P) > 4 * device_sm_count() ? 25 : 17;
}

bool taken_sizes(const StateParams &P) {
  return P.key_dim <= 128 && P.n >= fewest_tokens(P) && (!P.parents || P.n <= kChunkRows) && static_cast<int64_t>(P.B) * P.heads * 2 < kMostUnits;
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
  return P.vec && taken_sizes(P) && P.scale > 1e-30f && P.scale < 1e30f && map_strides(P.qs, P.key_heads, P.n, P.B) && map_strides(P.ks, P.key_heads, P.n, P.B) &&
         map_strides(P.vs, P.heads, P.n, P.B);
}

// (whatever the call: with or without parents, counts and states to write)
size_t state_chunk_workspace(const StateParams &P) {
  return P.key_dim <= 128 && P.n >= 4 && static_cast<int64_t>(P.B) * P.heads * 2 < kMostUnits ? chunk_plan(P, nullptr).second : 0;
}

cudaError_t launch_state_chunks(const StateParams &P, void *workspace, cudaStream_t st) {
  const StateChunkPlan A = chunk_plan(P, workspace).first;
  const size_t units = static_cast<size_t>(P.B) * P.heads;
  CUtensorMap maps[3];
  cudaError_t e = rows_map(P.q, P.qs, P.key_dim, P.key_heads, P.n, P.B, &maps[0]);
  if (e == cudaSuccess) e = rows_map(P.k, P.ks, P.key_dim, P.key_heads, P.n, P.B, &maps[1]);
  if (e == cudaSuccess) e = rows_map(P.v, P.vs, P.value_dim, P.heads, P.n, P.B, &maps[2]);
  if (e != cudaSuccess) return e;
  e = trace_launch("state_verdict", st, [&] { state_verdict_kernel<<<P.B, 64, 0, st>>>(P, A.verdict, A.order); });
  if (e == cudaSuccess && is_short(P)) return (P.dtype == SPEC_DTYPE_BF16 ? launch_state_short_bf16 : launch_state_short_f16)(A, maps, st);
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
