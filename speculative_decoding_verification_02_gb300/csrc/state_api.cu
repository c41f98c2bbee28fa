// C ABI of the linear-attention states: argument checks and parameter blocks.
#include <algorithm>
#include <cmath>
#include <cstdio>

#include "launch.h"
#include "state.cuh"

namespace sv {
namespace {

constexpr int64_t kMaxGrid = 2147483647;
constexpr int kMaxTokens = 1 << 30;  // (tokens are numbered by an int, a chunk past the last among them)

int state_fail(cudaError_t e, const char *where) {
  char text[256];
  std::snprintf(text, sizeof text, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
  set_last_error(text);
  return SPEC_ECUDA;
}

bool on_grain(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_geometry(const spec_state *s) {
  if (!s || s->heads < 1 || s->heads > 65535) return SPEC_EINVAL;
  if (s->key_dim < 16 || s->key_dim > 256 || s->key_dim % 16 || s->value_dim < 16 || s->value_dim > 256 || s->value_dim % 16)
    return SPEC_EINVAL;
  return SPEC_OK;
}

int check_pool(const spec_state *s, StatePool *out) {
  const int rc = check_geometry(s);
  if (rc != SPEC_OK) return rc;
  *out = StatePool{s->state, s->slot_stride, s->num_slots, s->slots};
  if (!s->state) return SPEC_OK;
  const int64_t size = static_cast<int64_t>(s->heads) * s->key_dim * s->value_dim;
  if (s->num_slots < 1 || s->slot_stride % 4 || s->slot_stride < size || !on_grain(s->state, 16)) return SPEC_EINVAL;
  return SPEC_OK;
}

bool strides_ok(const int64_t *s) { return s && s[0] >= 0 && s[1] >= 0 && s[2] >= 0; }

bool rows_vec(const void *p, const int64_t *s) { return on_grain(p, 16) && s[0] % 8 == 0 && s[1] % 8 == 0 && s[2] % 8 == 0; }

cudaStream_t stream_of(void *s) { return reinterpret_cast<cudaStream_t>(s); }

// What the three calls share: states, k, v, decay.  q and out are null in a commit.
int check_call(StateParams &P, const spec_state *from, const spec_state *to, const void *q, const int64_t *q_stride, const void *k,
               const int64_t *k_stride, const void *v, const int64_t *v_stride, int dtype, int B, int n, int key_heads,
               const float *decay, const int64_t *decay_stride, void *out, const int64_t *out_stride, bool outputs) {
  int rc = check_pool(from, &P.from);
  if (rc != SPEC_OK) return rc;
  if (to) {
    if ((rc = check_pool(to, &P.to)) != SPEC_OK) return rc;
    if (to->heads != from->heads || to->key_dim != from->key_dim || to->value_dim != from->value_dim) return SPEC_EINVAL;
  }
  if (dtype != SPEC_DTYPE_BF16 && dtype != SPEC_DTYPE_F16) return SPEC_EDTYPE;
  if (B < 0 || n < 0 || n > kMaxTokens || key_heads < 1 || from->heads % key_heads || !strides_ok(k_stride) || !strides_ok(v_stride) ||
      !strides_ok(decay_stride) || (outputs && (!strides_ok(q_stride) || !strides_ok(out_stride))))
    return SPEC_EINVAL;
  if (!on_grain(k, 2) || !on_grain(v, 2) || !on_grain(decay, 4) || !on_grain(q, 2) || !on_grain(out, 2)) return SPEC_EINVAL;
  if (n > 0 && B > 0 && (!k || !v || !decay || (outputs && (!q || !out)))) return SPEC_EINVAL;
  if (static_cast<int64_t>(B) * from->heads > kMaxGrid / 16) return SPEC_EINVAL;
  P.heads = from->heads, P.key_heads = key_heads, P.group = from->heads / key_heads, P.key_dim = from->key_dim, P.value_dim = from->value_dim;
  P.q = static_cast<const char *>(q), P.k = static_cast<const char *>(k), P.v = static_cast<const char *>(v), P.out = static_cast<char *>(out);
  std::copy(k_stride, k_stride + 3, P.ks);
  std::copy(v_stride, v_stride + 3, P.vs);
  std::copy(decay_stride, decay_stride + 3, P.gs);
  P.vec = rows_vec(k, k_stride) && rows_vec(v, v_stride);
  if (outputs) {
    std::copy(q_stride, q_stride + 3, P.qs);
    std::copy(out_stride, out_stride + 3, P.os);
    P.vec = P.vec && rows_vec(q, q_stride) && rows_vec(out, out_stride);
  }
  P.dtype = dtype, P.B = B, P.n = n, P.n_rows = n, P.decay = decay;
  return SPEC_OK;
}

void set_scale(StateParams &P, float scale) {
  int e = 0;
  std::frexp(scale, &e);
  P.scale = scale, P.scale_log2 = static_cast<float>(std::max(e, 0));
  P.most_units = static_cast<int64_t>(126 - std::max(e, 0)) * (int64_t{1} << kLog2Bits);
}

int run(const StateParams &P, void *workspace, size_t workspace_bytes, void *stream, const char *what) {
  const bool chunks = state_on_tensor_cores(P);
  if (chunks && (!workspace || workspace_bytes < state_chunk_workspace(P) || !on_grain(workspace, 256))) return SPEC_EWORKSPACE;
  const cudaError_t e = chunks ? launch_state_chunks(P, workspace, stream_of(stream)) : launch_state_rows(P, stream_of(stream));
  return e == cudaSuccess ? SPEC_OK : state_fail(e, what);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

size_t spec_state_workspace_size(int op, const spec_state *state, int B, int n) {
  if (check_geometry(state) != SPEC_OK || B < 0 || n < 0 || n > kMaxTokens) return 0;
  if (op != SPEC_OP_STATE_FORWARD && (op != SPEC_OP_STATE_ATTEND || n > SPEC_MAX_NODES)) return 0;
  StateParams P{};
  P.B = B, P.n = n, P.heads = state->heads, P.key_dim = state->key_dim, P.value_dim = state->value_dim;
  return state_chunk_workspace(P);
}

int spec_state_forward(const spec_state *from, const spec_state *to, const void *q, const int64_t *q_stride,
                       const void *k, const int64_t *k_stride, const void *v, const int64_t *v_stride, int dtype,
                       int B, int n, int key_heads, const float *decay, const int64_t *decay_stride,
                       const int32_t *counts, float scale, void *out, const int64_t *out_stride, int32_t *status,
                       void *workspace, size_t workspace_bytes, void *stream) {
  StateParams P{};
  const int rc = check_call(P, from, to, q, q_stride, k, k_stride, v, v_stride, dtype, B, n, key_heads, decay, decay_stride, out,
                            out_stride, true);
  if (rc != SPEC_OK) return rc;
  if (!std::isfinite(scale)) return SPEC_EINVAL;
  if (B == 0) return SPEC_OK;
  P.counts = counts, P.status = status;
  set_scale(P, scale);
  return run(P, workspace, workspace_bytes, stream, "spec_state_forward");
}

int spec_state_attend(const spec_state *from, const void *q, const int64_t *q_stride, const void *k,
                      const int64_t *k_stride, const void *v, const int64_t *v_stride, int dtype, int B, int N,
                      int key_heads, const float *decay, const int64_t *decay_stride, const int32_t *parents,
                      const int32_t *n_query, float scale, void *out, const int64_t *out_stride, int32_t *status,
                      void *workspace, size_t workspace_bytes, void *stream) {
  StateParams P{};
  const int rc = check_call(P, from, nullptr, q, q_stride, k, k_stride, v, v_stride, dtype, B, N, key_heads, decay, decay_stride, out,
                            out_stride, true);
  if (rc != SPEC_OK) return rc;
  if (!std::isfinite(scale) || N > SPEC_MAX_NODES) return SPEC_EINVAL;
  if (B == 0) return SPEC_OK;
  P.counts = n_query, P.parents = parents, P.status = status;
  set_scale(P, scale);
  return run(P, workspace, workspace_bytes, stream, "spec_state_attend");
}

int spec_state_commit(const spec_state *from, const spec_state *to, const void *k, const int64_t *k_stride,
                      const void *v, const int64_t *v_stride, int dtype, int B, int n, int key_heads,
                      const float *decay, const int64_t *decay_stride, const int32_t *index, int index_stride,
                      int n_rows, const int32_t *counts, int32_t *status, void *stream) {
  StateParams P{};
  const int rc = check_call(P, from, to, nullptr, nullptr, k, k_stride, v, v_stride, dtype, B, n, key_heads, decay, decay_stride,
                            nullptr, nullptr, false);
  if (rc != SPEC_OK) return rc;
  if (!P.to.state || n_rows < 0 || (index ? n_rows > index_stride : n_rows != n)) return SPEC_EINVAL;
  if (B == 0) return SPEC_OK;
  P.index = index, P.index_stride = index_stride, P.n_rows = n_rows, P.counts = counts, P.status = status;
  set_scale(P, 1.0f);
  const cudaError_t e = launch_state_rows(P, stream_of(stream));
  return e == cudaSuccess ? SPEC_OK : state_fail(e, "spec_state_commit");
}

}  // extern "C"
