"""ctypes binding over libspecverify.so.

The functions carry the C entry points' names and do argument marshalling
only: shapes and dtypes are read off torch tensors, pointers and strides are
passed through, outputs are allocated on the inputs' device, and the call is
enqueued on the current torch stream.  Every step of verification runs in the
library's CUDA kernels; there is no fallback.  Loading fails loudly when the
library has not been built (``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")

SPEC_OK, SPEC_EINVAL, SPEC_EDTYPE, SPEC_EWORKSPACE, SPEC_ECUDA = 0, -1, -2, -3, -4
STATUS_OK, STATUS_TOKEN_RANGE, STATUS_BAD_TREE, STATUS_BAD_LENGTH = 0, 1, 2, 3
STATUS_BAD_PAGE, STATUS_BAD_INDEX, STATUS_TIMEOUT, STATUS_BAD_SLOT = 5, 6, 7, 8
DTYPE_F32, DTYPE_BF16, DTYPE_F16 = 0, 1, 2
OP_NGRAM, OP_GREEDY, OP_SAMPLE, OP_TREE, OP_DRAW, OP_FILTER = 0, 1, 2, 3, 4, 5
OP_CACHE_ATTEND, OP_CACHE_WEIGHTS, OP_CACHE_EVICT = 6, 7, 8
OP_STATE_FORWARD, OP_STATE_ATTEND = 9, 10
CHAIN_AUTO, CHAIN_TWO_PASS, CHAIN_FUSED, CHAIN_CHUNKED = 0, 1, 2, 3
TREE_SIBLINGS_WITHOUT_REPLACEMENT = 1

_lock = threading.Lock()
_lib = None
_workspaces: dict = {}
_stream_locks: dict = {}


class SpecError(RuntimeError):
    """A libspecverify call returned a non-zero status."""


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(the CUDA library is required; there is no fallback)")
        L = ctypes.CDLL(LIB_PATH)
        P, I, I64, F, Z = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                           ctypes.c_size_t)
        L.spec_ngram_draft.argtypes = [P, P, I, I, I, I, P, P, P, P]
        L.spec_verify_greedy.argtypes = [P, I64, I64, I, I, I, I, P, P, P, P, P, P, P, P, Z, P]
        L.spec_verify_sample.argtypes = [P, I64, P, I64, I64, I, I, I, I, F, P, P, P, P, P, P, P,
                                         P, P, P, P, P, Z, P]
        L.spec_verify_tree.argtypes = [P, I64, P, I64, I64, I, I, I, I, F, P, P, P, I, P, P, P, P,
                                       P, P, Z, P]
        L.spec_verify_tree_ex.argtypes = [P, I64, P, I64, I64, I, I, I, I, F, P, P, P, I, I, P, P, P, P,
                                          P, P, Z, P]
        L.spec_workspace_size.argtypes = [I, I, I, I, I]
        L.spec_workspace_size.restype = Z
        L.spec_status_string.argtypes = [I]
        L.spec_status_string.restype = ctypes.c_char_p
        L.spec_last_error.argtypes = []
        L.spec_last_error.restype = ctypes.c_char_p
        L.spec_trace_enable.argtypes = [I]
        L.spec_trace_repeat.argtypes = [I]
        L.spec_trace_collect.argtypes = [P, P, P, I]
        L.spec_launch_count.argtypes = []
        L.spec_launch_count.restype = ctypes.c_int64
        L.spec_set_chain_path.argtypes = [I]
        L.spec_tree_rerank.argtypes = [P, P, P, I, I, I, I, P, P, P, P, P, P, P, P, P]
        L.spec_sample.argtypes = [P, I64, I, I, I, F, P, P, P, P, P, Z, P]
        L.spec_verify_sample_topkp.argtypes = [P, I64, P, I64, I64, I, I, I, I, F, I, F, P, P, P, P, P, P, P, P,
                                               P, P, P, P, Z, P]
        L.spec_sample_topkp.argtypes = [P, I64, I, I, I, F, I, F, P, P, P, P, P, Z, P]
        L.spec_filter_rows.argtypes = [P, I64, I, I, I, F, I, F, P, P, P, Z, P]
        D = ctypes.c_double
        L.spec_expected_tokens.argtypes = [D, I, P]
        L.spec_speedup.argtypes = [D, I, D, P]
        L.spec_best_k.argtypes = [D, D, I, P, P]
        L.spec_alpha_estimate.argtypes = [P, P, I, I, P, P]
        L.spec_cache_append.argtypes = [P, P, P, P, P, I, I, I, P, I, I, P, P, P, P, P]
        L.spec_cache_attend.argtypes = [P, P, P, I, I, I, I, P, P, P, F, F, P, P, P, P, P, Z, P]
        L.spec_cache_weights.argtypes = [P, P, P, I, I, I, I, P, P, P, I, I, P, P, F, F, P, P, P, P, I, P, P, Z, P]
        L.spec_cache_evict.argtypes = [P, P, I, P, P, P, I, I, I, P, P, P, P, P, Z, P]
        L.spec_cache_workspace_size.argtypes = [I, P, I, I, I]
        L.spec_cache_workspace_size.restype = Z
        L.spec_state_forward.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, P, P, P, F, P, P, P, P, Z, P]
        L.spec_state_attend.argtypes = [P, P, P, P, P, P, P, I, I, I, I, P, P, P, P, F, P, P, P, P, Z, P]
        L.spec_state_commit.argtypes = [P, P, P, P, P, P, I, I, I, I, P, P, P, I, I, P, P, P]
        L.spec_state_workspace_size.argtypes = [I, P, I, I]
        L.spec_state_workspace_size.restype = Z
        _lib = L
        return L


# ------------------------------------------------------------------ helpers

def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return DTYPE_F32
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _stream(stream, device):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _check(rc: int, what: str):
    if rc != SPEC_OK:
        L = lib()
        msg = L.spec_status_string(rc).decode()
        err = L.spec_last_error().decode()
        detail = err and rc in (SPEC_ECUDA, SPEC_EWORKSPACE)
        raise SpecError(f"{what}: {msg}" + (f" [{err}]" if detail else ""))


def _call(dev, fn, *args):
    """fn(*args), a stream last, with the tensors' device current: the library
    sizes its launches for the current device, and the no-allocation entry
    point looks up its scratch array there."""
    with torch.cuda.device(dev), _stream_lock(dev.index, args[-1].value or 0):
        return fn(*args)


def _stream_lock(device: int, stream: int):
    """Held while a call launches: several kernels of it use the stream's
    workspace, and another host thread's on the same stream must not come
    between them."""
    lock = _stream_locks.get((device, stream))
    return lock if lock is not None else _stream_locks.setdefault((device, stream), threading.RLock())


def _i32(t, shape, name, device):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != device:
        raise TypeError(f"{name} must be an int32 tensor on {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.contiguous()


def _f32(t, shape, name, device):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.device != device:
        raise TypeError(f"{name} must be a float32 tensor on {device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.contiguous()


def _logits3(t, name):
    if t.dim() != 3 or (t.stride(2) != 1 and t.numel() > 0 and t.shape[2] > 1):
        raise ValueError(f"{name} must be [B, rows, V] with contiguous rows")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    return t


def spec_workspace_size(op: int, B: int, rows_per_req: int, V: int, dtype: int) -> int:
    return int(lib().spec_workspace_size(op, B, rows_per_req, V, dtype))


def workspace(nbytes: int, device, stream=None) -> torch.Tensor:
    """A 256-byte aligned workspace of at least nbytes.

    One buffer is cached per (device, stream): calls on one stream are
    ordered (those of several host threads by a lock), so they may share it,
    while calls on different streams could overlap and must not."""
    device = torch.device(device)
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return _workspace(nbytes, device, s.cuda_stream)


def _workspace(nbytes: int, device, stream: int) -> torch.Tensor:
    key = (device.index, stream)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < max(nbytes, 1):
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)  # needs no initialisation
        if ws.data_ptr() % 256:
            raise RuntimeError("workspace allocation is not 256-byte aligned")
        _workspaces[key] = ws
    return ws


def set_chain_path(path: int):
    """Chain verification path for later calls, process-wide: CHAIN_AUTO,
    CHAIN_TWO_PASS, CHAIN_FUSED or CHAIN_CHUNKED (same results, different
    speed)."""
    _check(lib().spec_set_chain_path(int(path)), "spec_set_chain_path")


def trace_enable(on: bool = True):
    lib().spec_trace_enable(1 if on else 0)


def trace_repeat(reps: int = 1):
    """While tracing, launch each kernel reps times inside its event pair."""
    _check(lib().spec_trace_repeat(int(reps)), "spec_trace_repeat")


def trace_collect(cap: int = 16) -> dict:
    """{kernel name: (total ms, launches)} since the last collect."""
    names = (ctypes.c_char_p * cap)()
    ms = (ctypes.c_double * cap)()
    cnt = (ctypes.c_int64 * cap)()
    n = lib().spec_trace_collect(ctypes.cast(names, ctypes.c_void_p), ctypes.cast(ms, ctypes.c_void_p),
                                 ctypes.cast(cnt, ctypes.c_void_p), cap)
    if n < 0:
        _check(n, "spec_trace_collect")
    return {names[i].decode(): (ms[i], cnt[i]) for i in range(min(n, cap))}


def launch_count() -> int:
    return int(lib().spec_launch_count())


# --------------------------------------------------------------- entry points

def spec_ngram_draft(history: torch.Tensor, hist_len: torch.Tensor, window: int, k: int, *,
                     out=None, stream=None) -> dict:
    """history int32 [B, H], hist_len int32 [B] -> draft [B, k], draft_len [B], status [B]."""
    dev = history.device
    B, H = history.shape
    history = _i32(history, (B, H), "history", dev)
    hist_len = _i32(hist_len, (B,), "hist_len", dev)
    o = out or dict(draft=torch.empty((B, k), dtype=torch.int32, device=dev),
                    draft_len=torch.empty(B, dtype=torch.int32, device=dev),
                    status=torch.empty(B, dtype=torch.int32, device=dev))
    rc = _call(dev, lib().spec_ngram_draft, _p(history), _p(hist_len), B, H, int(window), int(k), _p(o["draft"]),
                                _p(o["draft_len"]), _p(o["status"]), _stream(stream, dev))
    _check(rc, "spec_ngram_draft")
    return o


def spec_verify_greedy(target: torch.Tensor, draft: torch.Tensor, draft_len=None, max_emit=None, *,
                       out=None, ws=None, stream=None) -> dict:
    """target [B, k+1, V] fp32/bf16, draft int32 [B, k] -> accepted, out_tokens, n_emit, status."""
    target = _logits3(target, "target")
    dev = target.device
    B, R, V = target.shape
    k = R - 1
    draft = _i32(draft, (B, k), "draft", dev)
    draft_len = _i32(draft_len, (B,), "draft_len", dev)
    max_emit = _i32(max_emit, (B,), "max_emit", dev)
    dt = _dtype_code(target)
    need = spec_workspace_size(OP_GREEDY, B, k, V, dt)
    ws = ws if ws is not None else workspace(need, dev, stream)
    o = out or dict(accepted=torch.empty(B, dtype=torch.int32, device=dev),
                    out_tokens=torch.empty((B, k + 1), dtype=torch.int32, device=dev),
                    n_emit=torch.empty(B, dtype=torch.int32, device=dev),
                    status=torch.empty(B, dtype=torch.int32, device=dev))
    rc = _call(dev, lib().spec_verify_greedy, _p(target), target.stride(0), target.stride(1), dt, B, k, V,
                                  _p(draft), _p(draft_len), _p(max_emit), _p(o["accepted"]),
                                  _p(o["out_tokens"]), _p(o["n_emit"]), _p(o["status"]), _p(ws),
                                  ws.numel(), _stream(stream, dev))
    _check(rc, "spec_verify_greedy")
    return o


def spec_verify_sample(target: torch.Tensor, draft_logits: torch.Tensor, draft: torch.Tensor,
                       uniforms: torch.Tensor, temperature: float = 1.0, draft_len=None,
                       max_emit=None, *, probs: bool = True, top_k: int = 0, top_p: float = 1.0, out=None,
                       ws=None, stream=None) -> dict:
    """target [B, k+1, V], draft_logits [B, k, V] (same dtype), draft int32 [B, k],
    uniforms fp32 [B, k+1] -> accepted, out_tokens, n_emit, p_tok, q_tok, resid_mass, status.
    top_k / top_p (0 / 1.0: off) filter p and q alike (spec_verify_sample_topkp)."""
    target = _logits3(target, "target")
    draft_logits = _logits3(draft_logits, "draft_logits")
    dev = target.device
    B, R, V = target.shape
    k = R - 1
    if tuple(draft_logits.shape) != (B, k, V) or draft_logits.dtype != target.dtype:
        raise ValueError("draft_logits must be [B, k, V] with the target's dtype")
    if k > 1 and draft_logits.stride(1) != target.stride(1):
        raise ValueError("target and draft rows must share a row stride")
    draft = _i32(draft, (B, k), "draft", dev)
    uniforms = _f32(uniforms, (B, k + 1), "uniforms", dev)
    draft_len = _i32(draft_len, (B,), "draft_len", dev)
    max_emit = _i32(max_emit, (B,), "max_emit", dev)
    dt = _dtype_code(target)
    need = spec_workspace_size(OP_SAMPLE, B, k, V, dt)
    ws = ws if ws is not None else workspace(need, dev, stream)
    o = out
    if o is None:
        o = dict(accepted=torch.empty(B, dtype=torch.int32, device=dev),
                 out_tokens=torch.empty((B, k + 1), dtype=torch.int32, device=dev),
                 n_emit=torch.empty(B, dtype=torch.int32, device=dev),
                 status=torch.empty(B, dtype=torch.int32, device=dev))
        if probs:
            o.update(p_tok=torch.empty((B, k), dtype=torch.float32, device=dev),
                     q_tok=torch.empty((B, k), dtype=torch.float32, device=dev),
                     resid_mass=torch.empty(B, dtype=torch.float32, device=dev))
    head = (_p(target), target.stride(0), _p(draft_logits), draft_logits.stride(0), target.stride(1), dt, B, k, V,
            float(temperature))
    tail = (_p(draft), _p(draft_len), _p(max_emit), _p(uniforms), _p(o["accepted"]), _p(o["out_tokens"]),
            _p(o["n_emit"]), _p(o.get("p_tok")), _p(o.get("q_tok")), _p(o.get("resid_mass")), _p(o["status"]),
            _p(ws), ws.numel(), _stream(stream, dev))
    if top_k or top_p != 1.0:
        _check(_call(dev, lib().spec_verify_sample_topkp, *head, int(top_k), float(top_p), *tail), "spec_verify_sample_topkp")
    else:
        _check(_call(dev, lib().spec_verify_sample, *head, *tail), "spec_verify_sample")
    return o


def spec_verify_tree(target: torch.Tensor, draft_logits, parents: torch.Tensor, node_tok: torch.Tensor,
                     uniforms: torch.Tensor, temperature: float, max_depth: int, *, flags: int = 0, out=None,
                     stream=None) -> dict:
    """target/draft_logits [B, N, V], parents/node_tok int32 [B, N], uniforms fp32 [B, N+1]
    -> accepted_len, path_nodes, out_tokens, n_emit, status.  temperature <= 0: greedy.
    flags != 0 (TREE_SIBLINGS_WITHOUT_REPLACEMENT) goes through spec_verify_tree_ex."""
    target = _logits3(target, "target")
    dev = target.device
    B, N, V = target.shape
    greedy = not temperature > 0
    if draft_logits is not None:
        draft_logits = _logits3(draft_logits, "draft_logits")
        if tuple(draft_logits.shape) != (B, N, V) or draft_logits.dtype != target.dtype:
            raise ValueError("draft_logits must be [B, N, V] with the target's dtype")
        if N > 1 and draft_logits.stride(1) != target.stride(1):
            raise ValueError("target and draft rows must share a row stride")
    elif not greedy:
        raise ValueError("sampling tree verification needs draft_logits")
    parents = _i32(parents, (B, N), "parents", dev)
    node_tok = _i32(node_tok, (B, N), "node_tok", dev)
    uniforms = _f32(uniforms, (B, N + 1), "uniforms", dev)
    W = max_depth + 1
    o = out or dict(accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
                    path_nodes=torch.empty((B, W), dtype=torch.int32, device=dev),
                    out_tokens=torch.empty((B, W), dtype=torch.int32, device=dev),
                    n_emit=torch.empty(B, dtype=torch.int32, device=dev),
                    status=torch.empty(B, dtype=torch.int32, device=dev))
    d_req = draft_logits.stride(0) if draft_logits is not None else 0
    head = (_p(target), target.stride(0), _p(draft_logits), d_req, target.stride(1), _dtype_code(target), B, N,
            V, float(temperature), _p(parents), _p(node_tok), _p(uniforms), int(max_depth))
    tail = (_p(o["accepted_len"]), _p(o["path_nodes"]), _p(o["out_tokens"]), _p(o["n_emit"]), _p(o["status"]),
            None, 0, _stream(stream, dev))
    if flags:
        rc = _call(dev, lib().spec_verify_tree_ex, *head, int(flags), *tail)
        _check(rc, "spec_verify_tree_ex")
    else:
        rc = _call(dev, lib().spec_verify_tree, *head, *tail)
        _check(rc, "spec_verify_tree")
    return o


def spec_sample(logits: torch.Tensor, uniforms: torch.Tensor, temperature: float = 1.0, *, probs: bool = True,
                top_k: int = 0, top_p: float = 1.0, out=None, ws=None, stream=None) -> dict:
    """logits [B, V] (fp32 or bf16, each row contiguous), uniforms fp32 [B]
    -> tokens int32 [B] drawn from softmax(logits / T), probs fp32 [B] (the
    drawn tokens' probabilities), status.  top_k / top_p (0 / 1.0: off):
    draw from the filtered rows (spec_sample_topkp)."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be a [B, V] tensor")
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("logits must be float32 or bfloat16")
    if logits.stride(1) != 1:
        logits = logits.contiguous()
    dev = logits.device
    B, V = logits.shape
    uniforms = _f32(uniforms, (B,), "uniforms", dev)
    dt = _dtype_code(logits)
    need = spec_workspace_size(OP_DRAW, B, 0, V, dt)
    ws = ws if ws is not None else workspace(need, dev, stream)
    o = out or dict(tokens=torch.empty(B, dtype=torch.int32, device=dev),
                    probs=torch.empty(B, dtype=torch.float32, device=dev) if probs else None,
                    status=torch.empty(B, dtype=torch.int32, device=dev))
    tail = (_p(uniforms), _p(o["tokens"]), _p(o.get("probs")), _p(o["status"]), _p(ws), ws.numel(),
            _stream(stream, dev))
    if top_k or top_p != 1.0:
        rc = _call(dev, lib().spec_sample_topkp, _p(logits), logits.stride(0), dt, B, V, float(temperature), int(top_k),
                                     float(top_p), *tail)
        _check(rc, "spec_sample_topkp")
    else:
        _check(_call(dev, lib().spec_sample, _p(logits), logits.stride(0), dt, B, V, float(temperature), *tail), "spec_sample")
    return o


def spec_filter_rows(logits: torch.Tensor, temperature: float = 1.0, top_k: int = 0, top_p: float = 1.0, *,
                     out=None, stream=None) -> dict:
    """logits [R, V] (fp32 or bf16, each row contiguous) -> theta fp32 [R]
    (the smallest logit the top-k / top-p filter keeps) and kept int32 [R]."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be a [R, V] tensor")
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("logits must be float32 or bfloat16")
    if logits.stride(1) != 1:
        logits = logits.contiguous()
    dev = logits.device
    R, V = logits.shape
    dt = _dtype_code(logits)
    ws = workspace(spec_workspace_size(OP_FILTER, R, 0, V, dt), dev, stream)
    o = out or dict(theta=torch.empty(R, dtype=torch.float32, device=dev),
                    kept=torch.empty(R, dtype=torch.int32, device=dev))
    _check(_call(dev, lib().spec_filter_rows, _p(logits), logits.stride(0), dt, R, V, float(temperature), int(top_k),
                                  float(top_p), _p(o["theta"]), _p(o.get("kept")), _p(ws), ws.numel(),
                                  _stream(stream, dev)), "spec_filter_rows")
    return o


def spec_tree_rerank(parents: torch.Tensor, conf: torch.Tensor, m: int, max_depth: int = 64, node_tok=None, *,
                     mask: bool = True, out=None, stream=None) -> dict:
    """parents int32 [B, N], conf fp32 [B, N] (node_tok int32 [B, N] or None)
    -> sel_nodes, sel_parents, sel_depth, sel_value, sel_tok (with node_tok),
    mask uint8 [B, m, m] (unless mask=False), n_sel, status."""
    dev = parents.device
    if parents.dim() != 2:
        raise ValueError("parents must be [B, N]")
    B, N = parents.shape
    parents = _i32(parents, (B, N), "parents", dev)
    conf = _f32(conf, (B, N), "conf", dev)
    node_tok = _i32(node_tok, (B, N), "node_tok", dev) if node_tok is not None else None
    i32 = dict(dtype=torch.int32, device=dev)
    o = out or dict(sel_nodes=torch.empty((B, m), **i32), sel_parents=torch.empty((B, m), **i32),
                    sel_depth=torch.empty((B, m), **i32),
                    sel_value=torch.empty((B, m), dtype=torch.float32, device=dev),
                    sel_tok=torch.empty((B, m), **i32) if node_tok is not None else None,
                    mask=torch.empty((B, m, m), dtype=torch.uint8, device=dev) if mask else None,
                    n_sel=torch.empty(B, **i32), status=torch.empty(B, **i32))
    rc = _call(dev, lib().spec_tree_rerank, _p(parents), _p(conf), _p(node_tok), B, N, int(m), int(max_depth),
                                _p(o["sel_nodes"]), _p(o["sel_parents"]), _p(o["sel_depth"]),
                                _p(o.get("sel_value")), _p(o.get("sel_tok")), _p(o.get("mask")),
                                _p(o["n_sel"]), _p(o.get("status")), _stream(stream, dev))
    _check(rc, "spec_tree_rerank")
    return o


def spec_verify_sample_noalloc(target: torch.Tensor, draft_logits: torch.Tensor, draft: torch.Tensor,
                               uniforms: torch.Tensor, temperature: float = 1.0, draft_len=None,
                               max_emit=None, *, out=None, stream=None) -> dict:
    """spec_verify_sample without a workspace, for callers that cannot allocate
    device memory while they run: the library's fixed scratch array is used
    instead (SPEC_NOALLOC_SCRATCH_BYTES; larger problems raise SpecError).
    Outputs are allocated here unless `out` is given."""
    L = lib()
    fn = L.spec_verify_sample_noalloc
    P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    fn.argtypes = [P, I64, P, I64, I64, I, I, I, I, F, P, P, P, P, P, P, P, P, P, P, P, P]
    target = _logits3(target, "target")
    draft_logits = _logits3(draft_logits, "draft_logits")
    dev = target.device
    B, R, V = target.shape
    k = R - 1
    if tuple(draft_logits.shape) != (B, k, V) or draft_logits.dtype != target.dtype:
        raise ValueError("draft_logits must be [B, k, V] with the target's dtype")
    if k > 1 and draft_logits.stride(1) != target.stride(1):
        raise ValueError("target and draft rows must share a row stride")
    draft = _i32(draft, (B, k), "draft", dev)
    uniforms = _f32(uniforms, (B, k + 1), "uniforms", dev)
    draft_len = _i32(draft_len, (B,), "draft_len", dev)
    max_emit = _i32(max_emit, (B,), "max_emit", dev)
    o = out or dict(accepted=torch.empty(B, dtype=torch.int32, device=dev),
                    out_tokens=torch.empty((B, k + 1), dtype=torch.int32, device=dev),
                    n_emit=torch.empty(B, dtype=torch.int32, device=dev),
                    status=torch.empty(B, dtype=torch.int32, device=dev),
                    p_tok=torch.empty((B, k), dtype=torch.float32, device=dev),
                    q_tok=torch.empty((B, k), dtype=torch.float32, device=dev),
                    resid_mass=torch.empty(B, dtype=torch.float32, device=dev))
    rc = _call(dev, fn, _p(target), target.stride(0), _p(draft_logits), draft_logits.stride(0), target.stride(1),
            _dtype_code(target), B, k, V, float(temperature), _p(draft), _p(draft_len), _p(max_emit),
            _p(uniforms), _p(o["accepted"]), _p(o["out_tokens"]), _p(o["n_emit"]), _p(o.get("p_tok")),
            _p(o.get("q_tok")), _p(o.get("resid_mass")), _p(o["status"]), _stream(stream, dev))
    _check(rc, "spec_verify_sample_noalloc")
    return o


# ------------------------------------------------------- host analysis helpers
# Host-side (no GPU): the choice of the draft length from measured acceptance.

def expected_tokens(alpha: float, k: int) -> float:
    """Expected tokens per round, 1 + alpha + ... + alpha^k."""
    out = ctypes.c_double()
    _check(lib().spec_expected_tokens(float(alpha), int(k), ctypes.byref(out)), "spec_expected_tokens")
    return out.value


def speedup(alpha: float, k: int, draft_cost: float) -> float:
    """Expected tokens per round over the round's cost k c + 1 (in target forwards)."""
    out = ctypes.c_double()
    _check(lib().spec_speedup(float(alpha), int(k), float(draft_cost), ctypes.byref(out)), "spec_speedup")
    return out.value


def best_k(alpha: float, draft_cost: float, k_max: int) -> tuple:
    """(k in [0, k_max] with the largest speedup, that speedup)."""
    k = ctypes.c_int()
    s = ctypes.c_double()
    _check(lib().spec_best_k(float(alpha), float(draft_cost), int(k_max), ctypes.byref(k), ctypes.byref(s)),
           "spec_best_k")
    return k.value, s.value


def alpha_estimate(accepted, draft_len=None, k: int = 0) -> tuple:
    """(alpha, positions tested) from rounds' accepted counts (host arrays or
    tensors, copied to the host) and draft lengths (None: all k)."""
    import numpy as np
    acc = np.ascontiguousarray(torch.as_tensor(accepted).cpu().numpy(), dtype=np.int32).reshape(-1)
    dl = None if draft_len is None else np.ascontiguousarray(torch.as_tensor(draft_len).cpu().numpy(),
                                                             dtype=np.int32).reshape(-1)
    if dl is not None and dl.size != acc.size:
        raise ValueError("draft_len must match accepted")
    a = ctypes.c_double()
    t = ctypes.c_int64()
    _check(lib().spec_alpha_estimate(acc.ctypes.data, None if dl is None else dl.ctypes.data, acc.size, int(k),
                                     ctypes.byref(a), ctypes.byref(t)), "spec_alpha_estimate")
    return a.value, t.value


# ------------------------------------------------------- the cache in 8 bits

class KVCache(NamedTuple):
    """A pool of pages: k, v e4m3 [pages, kv_heads, page_size, head_dim] (pages may lie further apart than their size), and
    the blocks' scales, fp32 [pages, kv_heads].  Any four such tensors in this order are a cache to the functions below."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


class _CacheStruct(ctypes.Structure):  # struct spec_cache
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("scale_stride", ctypes.c_int64), ("num_pages", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int32)]


# The same struct, and strides, as packed bytes: a third of the time of a ctypes object, which counts in calls of a few
# microseconds on the GPU.
_pack_cache = struct.Struct("@PPPPqqiiiiPi4x").pack
_pack3 = struct.Struct("@qqq").pack
_pack2 = struct.Struct("@qq").pack
_F8, _F32, _I32 = torch.float8_e4m3fn, torch.float32, torch.int32
_ROW_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16, torch.float32: DTYPE_F32}


def spec_cache_new(pages: int, kv_heads: int, page_size: int, head_dim: int, device="cuda") -> KVCache:
    """A pool of zeros (every scale 1)."""
    shape = (pages, kv_heads, page_size, head_dim)
    k, v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2))
    return KVCache(k, v, torch.ones(shape[:2], device=device), torch.ones(shape[:2], device=device))


def _cache_struct(cache, table, B, dev, name="cache"):
    """(packed struct spec_cache, kv_heads, page_size, head_dim)"""
    k, v, ks, vs = cache
    if not (k.dtype is v.dtype is _F8 and ks.dtype is vs.dtype is _F32):
        raise TypeError(f"{name}: k and v must be float8_e4m3fn and their scales float32")
    shape, st, of, ss = k.shape, k.stride(), ks.shape, ks.stride()
    if len(shape) != 4 or v.shape != shape or v.stride() != st or of != shape[:2] or vs.shape != of:
        raise ValueError(f"{name}: k and v must be [pages, kv_heads, page_size, head_dim] alike, their scales [pages, kv_heads]")
    n, H, P, D = shape
    if st[3] != 1 or st[2] != D or (H > 1 and st[1] != P * D) or vs.stride() != ss or (H > 1 and ss[1] != 1):
        raise ValueError(f"{name}: the heads of a page must lie side by side")
    i = dev.index  # (None for tensors of the host, whose get_device() is -1)
    if not k.get_device() == v.get_device() == ks.get_device() == vs.get_device() == i:
        raise ValueError(f"{name} must live on the rows' CUDA device")
    ts = table.shape
    if table.dtype is not _I32 or table.get_device() != i or len(ts) != 2 or ts[0] != B or not table.is_contiguous():
        raise TypeError(f"the page table must be a contiguous int32 [{B}, pages of a request] tensor on {dev}")
    return _pack_cache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), st[0] if n > 1 else H * P * D,
                       ss[0] if n > 1 else H, n, H, P, D, table.data_ptr(), ts[1]), H, P, D


def _rows(t, name, dev, dtypes):
    """dtype code and strides of rows [B, tokens, heads, head_dim]."""
    st = t.stride()
    if len(st) != 4 or (st[3] != 1 and t.shape[3] > 1):
        raise ValueError(f"{name} must be [B, tokens, heads, head_dim] with contiguous heads")
    if t.get_device() != dev.index:
        raise ValueError(f"{name} must live on {dev}")
    code = _ROW_DTYPES.get(t.dtype)
    if code is None or code not in dtypes:
        raise TypeError(f"{name} cannot be {t.dtype}")
    return code, _pack3(st[0], st[1], st[2])


def _index_rows(index, counts, B, n, dev):
    """(index, its stride, rows a request at most)"""
    if counts is not None:
        _lengths(counts, B, "counts", dev)
    if index is None:
        return None, 0, n
    shape, st = index.shape, index.stride()
    if index.dtype is not _I32 or index.get_device() != dev.index or len(shape) != 2 or shape[0] != B or (st[1] != 1 and shape[1] > 1):
        raise TypeError(f"index must be an int32 [{B}, rows] tensor on {dev}")
    return index.data_ptr(), st[0] if B > 1 else shape[1], shape[1]


def _on(dev, fn, *args):
    """fn(*args) with dev current."""
    if torch._C._cuda_getDevice() == dev.index:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def _lengths(t, B, name, dev):
    if t.dtype is not _I32 or t.get_device() != dev.index or t.shape != (B,) or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 [{B}] tensor on {dev}")
    return t.data_ptr()


def _status(o, B, dev):
    t = o.get("status")
    return None if t is None else _lengths(t, B, "status", dev)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _with_workspace(fn, what, op, cs, B, N, Hq, dev, ws, stream, *args):
    """fn(*args, workspace, its size, stream) with the stream's workspace as it is; the size that the call needs is asked for only
    when that is too small (the library looks at it before it does anything)."""
    with _stream_lock(dev.index, stream):
        have = ws if ws is not None else _workspaces.get((dev.index, stream))
        p, n = (None, 0) if have is None else (have.data_ptr(), have.numel())
        rc = _on(dev, fn, *args, p, n, stream)
        if rc == SPEC_EWORKSPACE and ws is None:
            have = _workspace(_on(dev, lib().spec_cache_workspace_size, op, cs, B, N, Hq), dev, stream)
            rc = _on(dev, fn, *args, have.data_ptr(), have.numel(), stream)
    _check(rc, what)


def _raw_stream(dev) -> int:
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _on_stream(stream, fn, *args, **kw):
    """fn with stream current: the tensors that it makes and the copies that it takes belong to that stream, as its kernels do."""
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def spec_cache_append(cache, table: torch.Tensor, cache_len: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, counts=None,
                      index=None, out=None, stream=None) -> dict:
    """Writes rows of k, v [B, n, kv_heads, head_dim] (bf16, fp16 or fp32) behind each request's cache_len tokens: all n of
    them, or counts int32 [B]; with index int32 [B, rows], row i is token index[b, i] (the accepted path: index = path_nodes,
    counts = n_emit of a verify call) -> new_len [B], status [B]."""
    dev = k.device
    if stream is not None:
        return _on_stream(stream, spec_cache_append, cache, table, cache_len, k, v, counts=counts, index=index, out=out)
    st = _raw_stream(dev)
    code, kst = _rows(k, "k", dev, (DTYPE_BF16, DTYPE_F16, DTYPE_F32))
    vcode, vst = _rows(v, "v", dev, (DTYPE_BF16, DTYPE_F16, DTYPE_F32))
    shape = k.shape
    B, n, heads, D = shape
    cs, H, P, hd = _cache_struct(cache, table, B, dev)
    if v.shape != shape or vcode != code or heads != H or D != hd:
        raise ValueError(f"k and v must both be [B, n, {H}, {hd}] of one dtype")
    lp = _lengths(cache_len, B, "cache_len", dev)
    ip, ist, rows = _index_rows(index, counts, B, n, dev)
    o = out or dict(new_len=torch.empty(B, dtype=torch.int32, device=dev), status=torch.empty(B, dtype=torch.int32, device=dev))
    rc = _on(dev, (_lib or lib()).spec_cache_append, cs, k.data_ptr(), kst, v.data_ptr(), vst, code, B, n, ip, ist, rows,
             _ptr(counts), lp, _lengths(o["new_len"], B, "new_len", dev), _status(o, B, dev), st)
    _check(rc, "spec_cache_append")
    return o


def spec_cache_attend(q: torch.Tensor, cache, table: torch.Tensor, cache_len: torch.Tensor, *, n_query=None, mask=None,
                      scale=None, softcap: float = 0.0, lse: bool = True, out=None, ws=None, stream=None) -> dict:
    """Attention of q [B, N, Hq, head_dim] (bf16 or fp16), the N rows whose keys and values lie behind each request's
    cache_len tokens: row i sees the context and the rows up to itself, or with mask uint8 [B, N, N] (spec_tree_rerank's) the
    rows j with mask[b, i, j].  n_query int32 [B]: rows of a request (default N).  scale: head_dim ** -0.5 by default.
    -> out (as q), lse fp32 [B, N, Hq], status.  ws: the caller's own workspace, for a call captured into a graph that outlives
    larger calls on its stream (they replace the stream's)."""
    dev = q.device
    if stream is not None:
        return _on_stream(stream, spec_cache_attend, q, cache, table, cache_len, n_query=n_query, mask=mask, scale=scale,
                          softcap=softcap, lse=lse, out=out, ws=ws)
    st = _raw_stream(dev)
    B, N, Hq, D = q.shape
    cs, H, P, hd = _cache_struct(cache, table, B, dev)
    if D != hd:
        raise ValueError(f"q must be [B, N, heads, {hd}]")
    code, qst = _rows(q, "q", dev, (DTYPE_BF16, DTYPE_F16))
    lp = _lengths(cache_len, B, "cache_len", dev)
    np_ = None if n_query is None else _lengths(n_query, B, "n_query", dev)
    if mask is not None:
        if mask.dtype not in (torch.uint8, torch.bool) or mask.device != dev or tuple(mask.shape) != (B, N, N):
            raise TypeError(f"mask must be a uint8 [{B}, {N}, {N}] tensor on {dev}")
        mask = mask.contiguous()
    o = out or dict(out=torch.empty((B, N, Hq, D), dtype=q.dtype, device=dev),
                    lse=torch.empty((B, N, Hq), dtype=torch.float32, device=dev) if lse else None,
                    status=torch.empty(B, dtype=torch.int32, device=dev))
    _, ost = _rows(o["out"], "out", dev, (code,))
    if o["out"].shape != q.shape:
        raise ValueError("out must have q's shape")
    if o.get("lse") is not None:
        _f32_like(o["lse"], (B, N, Hq), "lse", dev)
    _with_workspace((_lib or lib()).spec_cache_attend, "spec_cache_attend", OP_CACHE_ATTEND, cs, B, N, Hq, dev, ws, st,
                    cs, q.data_ptr(), qst, code, B, N, Hq, lp, np_, _ptr(mask), D ** -0.5 if scale is None else float(scale),
                    float(softcap), o["out"].data_ptr(), ost, _ptr(o.get("lse")), _status(o, B, dev))
    return o


def _f32_like(t, shape, name, dev):
    if t.dtype is not torch.float32 or t.get_device() != dev.index or t.shape != shape or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 {list(shape)} tensor on {dev}")
    return t.data_ptr()


def _positions(t, name, B, H, dev):
    """Strides of fp32 [B, kv_heads, positions]."""
    if t.dtype != torch.float32 or t.device != dev or t.dim() != 3 or tuple(t.shape[:2]) != (B, H) or (t.shape[2] > 1 and t.stride(2) != 1):
        raise TypeError(f"{name} must be a float32 [{B}, {H}, positions] tensor on {dev} with contiguous positions")
    st = t.stride()
    return _pack2(st[0], st[1])


def spec_cache_weights(q: torch.Tensor, lse: torch.Tensor, cache, table: torch.Tensor, cache_len: torch.Tensor, *, prev=None,
                       counts=None, index=None, scale=None, softcap: float = 0.0, out=None, ws=None, stream=None) -> dict:
    """The attention weight each cached token received from rows of q [B, N, Hq, head_dim] with their lse (spec_cache_attend's),
    added to prev fp32 [B, kv_heads, positions] (zeros when None): rows and counts as in spec_cache_append, row i at position
    cache_len + i and seeing every position up to its own -> weights (prev's shape; positions past the rows' are not written:
    zeros in a new tensor), status.  out["weights"] may be prev."""
    dev = q.device
    if stream is not None:
        return _on_stream(stream, spec_cache_weights, q, lse, cache, table, cache_len, prev=prev, counts=counts, index=index,
                          scale=scale, softcap=softcap, out=out, ws=ws)
    st = _raw_stream(dev)
    B, N, Hq, D = q.shape
    cs, H, P, hd = _cache_struct(cache, table, B, dev)
    if D != hd:
        raise ValueError(f"q must be [B, N, heads, {hd}]")
    code, qst = _rows(q, "q", dev, (DTYPE_BF16, DTYPE_F16))
    lp = _lengths(cache_len, B, "cache_len", dev)
    if lse.dtype is not torch.float32 or lse.device != dev or lse.shape != (B, N, Hq):
        raise TypeError(f"lse must be a float32 {[B, N, Hq]} tensor on {dev}")
    ip, ist, rows = _index_rows(index, counts, B, N, dev)
    pst = None if prev is None else _positions(prev, "prev", B, H, dev)
    o = out
    if o is None:
        w = torch.zeros((B, H, table.shape[1] * P), device=dev) if prev is None else prev.clone()
        o = dict(weights=w, status=torch.empty(B, dtype=torch.int32, device=dev))
    ost = _positions(o["weights"], "weights", B, H, dev)
    room = o["weights"].shape[2] if prev is None else min(prev.shape[2], o["weights"].shape[2])
    _with_workspace((_lib or lib()).spec_cache_weights, "spec_cache_weights", OP_CACHE_WEIGHTS, cs, B, rows, Hq, dev, ws, st,
                    cs, q.data_ptr(), qst, code, B, N, Hq, lse.data_ptr(), _pack3(*lse.stride()), ip, ist, rows, _ptr(counts),
                    lp, D ** -0.5 if scale is None else float(scale), float(softcap), _ptr(prev), pst,
                    o["weights"].data_ptr(), ost, room, _status(o, B, dev))
    return o


def spec_cache_evict(cache, table: torch.Tensor, cache_len: torch.Tensor, weights: torch.Tensor, keep: int, recent: int,
                     dst_table: torch.Tensor, *, dst_cache=None, out=None, ws=None, stream=None) -> dict:
    """Copies to the pages of dst_table (of dst_cache, or of the same pool: other pages than any that are read), per kv head, the
    `recent` last tokens and the others of largest weight (weights fp32 [B, kv_heads, positions]), min(keep, cache_len) in all and
    in their order -> kept int32 [B, kv_heads, keep] (positions, then -1), weights [B, kv_heads, keep] (then 0), new_len, status."""
    dev = weights.device
    if stream is not None:
        return _on_stream(stream, spec_cache_evict, cache, table, cache_len, weights, keep, recent, dst_table,
                          dst_cache=dst_cache, out=out, ws=ws)
    st = _raw_stream(dev)
    B = weights.shape[0]
    cs, H, P, hd = _cache_struct(cache, table, B, dev)
    ds = _cache_struct(cache if dst_cache is None else dst_cache, dst_table, B, dev, "dst_cache")[0]
    lp = _lengths(cache_len, B, "cache_len", dev)
    wst = _positions(weights, "weights", B, H, dev)
    keep = int(keep)
    o = out or dict(kept=torch.empty((B, H, max(keep, 0)), dtype=torch.int32, device=dev),
                    weights=torch.empty((B, H, max(keep, 0)), device=dev),
                    new_len=torch.empty(B, dtype=torch.int32, device=dev), status=torch.empty(B, dtype=torch.int32, device=dev))
    kept, of = o["kept"], (B, H, max(keep, 0))
    if kept.dtype is not _I32 or kept.get_device() != dev.index or kept.shape != of or not kept.is_contiguous():
        raise TypeError(f"kept must be a contiguous int32 {list(of)} tensor on {dev}")
    if o.get("weights") is not None:
        _f32_like(o["weights"], of, "the kept weights", dev)
    _with_workspace((_lib or lib()).spec_cache_evict, "spec_cache_evict", OP_CACHE_EVICT, cs, B, keep, 0, dev, ws, st,
                    cs, ds, B, lp, weights.data_ptr(), wst, weights.shape[2], keep, int(recent), kept.data_ptr(),
                    _ptr(o.get("weights")), _lengths(o["new_len"], B, "new_len", dev), _status(o, B, dev))
    return o


# ------------------------------------------------------- linear attention

class _StateStruct(ctypes.Structure):  # struct spec_state
    _fields_ = [("state", ctypes.c_void_p), ("slot_stride", ctypes.c_int64), ("num_slots", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("key_dim", ctypes.c_int32), ("value_dim", ctypes.c_int32), ("slots", ctypes.c_void_p)]


_pack_state = struct.Struct("@PqiiiiP").pack


def spec_state_new(slots: int, heads: int, key_dim: int, value_dim: int, device="cuda") -> torch.Tensor:
    """A pool of states of zeros: fp32 [slots, heads, key_dim, value_dim]."""
    return torch.zeros((slots, heads, key_dim, value_dim), device=device)


def _state_struct(state, slots, B, dims, dev, name):
    """packed struct spec_state"""
    H, Dk, Dv = dims
    if state is None:
        return _pack_state(0, 0, 0, H, Dk, Dv, 0)
    if state.dtype is not _F32 or state.get_device() != dev.index:
        raise TypeError(f"{name} must be a float32 tensor on {dev}")
    shape, st = state.shape, state.stride()
    if len(shape) != 4 or shape[1:] != dims or st[3] != 1 or st[2] != Dv or (H > 1 and st[1] != Dk * Dv):
        raise ValueError(f"{name} must be [slots, {H}, {Dk}, {Dv}], the heads of a slot side by side")
    return _pack_state(state.data_ptr(), st[0] if shape[0] > 1 else H * Dk * Dv, shape[0], H, Dk, Dv,
                       0 if slots is None else _lengths(slots, B, "slots", dev))


def _state_rows(k, v, decay, dev):
    """Checks of the rows that every call has -> (dtype code, k's strides, v's strides, decay's strides)"""
    code, kst = _rows(k, "k", dev, (DTYPE_BF16, DTYPE_F16))
    vcode, vst = _rows(v, "v", dev, (DTYPE_BF16, DTYPE_F16))
    B, n, H, _ = v.shape
    if vcode != code or k.shape[:2] != (B, n):
        raise ValueError("k and v must be rows of the same tokens, of one dtype")
    if decay.dtype is not _F32 or decay.get_device() != dev.index or decay.shape != (B, n, H):
        raise TypeError(f"decay must be a float32 {[B, n, H]} tensor on {dev}")
    return code, kst, vst, _pack3(*decay.stride())


def _state_out(o, q, v, code, dev):
    """Strides of the outputs [B, n, heads, value_dim]."""
    if o["out"].shape != v.shape:
        raise ValueError("out must have v's shape")
    return _rows(o["out"], "out", dev, (code,))[1]


def _state_pools(state, slots, dst, dst_slots, B, dims, dev):
    """The states before and after: in place unless dst is given."""
    if dst is None and dst_slots is not None:
        if state is None:
            raise ValueError("dst_slots without a state to write")
        dst = state
    elif dst is None:
        dst, dst_slots = state, slots
    return _state_struct(state, slots, B, dims, dev, "state"), None if dst is None else _state_struct(dst, dst_slots, B, dims, dev, "dst")


def spec_state_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, decay: torch.Tensor, state, *, slots=None, dst=None,
                       dst_slots=None, counts=None, scale=None, write: bool = True, out=None, ws=None, stream=None) -> dict:
    """Linear attention S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale q_t^T S_t over the tokens of q, k [B, n, key_heads, key_dim]
    and v [B, n, heads, value_dim] (bf16 or fp16) with decay g, fp32 [B, n, heads]: n of them, or counts int32 [B].
    state: fp32 [slots, heads, key_dim, value_dim] (spec_state_new), of which request b has slot b, or slots int32 [B] (-1: a
    state of zeros); None: zeros, whatever slots says.  The states after go to dst (its slots: dst_slots), by default to the same slots of state; with
    write=False nowhere.  scale: key_dim ** -0.5 by default.
    -> out (as v; rows past a count are 0), status.  ws: as in spec_cache_attend."""
    dev = q.device
    if stream is not None:
        return _on_stream(stream, spec_state_forward, q, k, v, decay, state, slots=slots, dst=dst, dst_slots=dst_slots, counts=counts,
                          scale=scale, write=write, out=out, ws=ws)
    st = _raw_stream(dev)
    code, kst, vst, gst = _state_rows(k, v, decay, dev)
    qcode, qst = _rows(q, "q", dev, (code,))
    B, n, Hk, Dk = q.shape
    if k.shape != q.shape:
        raise ValueError("q and k must have one shape")
    before, after = _state_pools(state, slots, dst, dst_slots, B, (v.shape[2], Dk, v.shape[3]), dev)
    if write and after is None:
        raise ValueError("no state to write: give dst, or write=False")
    cp = None if counts is None else _lengths(counts, B, "counts", dev)
    o = out or dict(out=torch.empty(v.shape, dtype=v.dtype, device=dev), status=torch.empty(B, dtype=torch.int32, device=dev))
    ost = _state_out(o, q, v, code, dev)
    _state_call((_lib or lib()).spec_state_forward, "spec_state_forward", OP_STATE_FORWARD, before, B, n, dev, ws, st,
                before, after if write else None, q.data_ptr(), qst, k.data_ptr(), kst, v.data_ptr(), vst, code, B, n, Hk,
                decay.data_ptr(), gst, cp, Dk ** -0.5 if scale is None else float(scale), o["out"].data_ptr(), ost, _status(o, B, dev))
    return o


def spec_state_attend(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, decay: torch.Tensor, state, *, slots=None, parents=None,
                      n_query=None, scale=None, out=None, ws=None, stream=None) -> dict:
    """The outputs of N drafted rows behind each request's state, which stays as it is: a chain, or with parents int32 [B, N]
    (spec_tree_rerank's sel_parents, spec_verify_tree's parents) a tree, whose row i follows row parents[b, i].  n_query int32
    [B]: rows of a request (default N).  The rest as in spec_state_forward -> out, status."""
    dev = q.device
    if stream is not None:
        return _on_stream(stream, spec_state_attend, q, k, v, decay, state, slots=slots, parents=parents, n_query=n_query,
                          scale=scale, out=out, ws=ws)
    st = _raw_stream(dev)
    code, kst, vst, gst = _state_rows(k, v, decay, dev)
    qcode, qst = _rows(q, "q", dev, (code,))
    B, n, Hk, Dk = q.shape
    if k.shape != q.shape:
        raise ValueError("q and k must have one shape")
    before = _state_pools(state, slots, None, None, B, (v.shape[2], Dk, v.shape[3]), dev)[0]
    if parents is not None and (parents.dtype is not _I32 or parents.get_device() != dev.index or parents.shape != (B, n) or
                                not parents.is_contiguous()):
        raise TypeError(f"parents must be a contiguous int32 {[B, n]} tensor on {dev}")
    np_ = None if n_query is None else _lengths(n_query, B, "n_query", dev)
    o = out or dict(out=torch.empty(v.shape, dtype=v.dtype, device=dev), status=torch.empty(B, dtype=torch.int32, device=dev))
    ost = _state_out(o, q, v, code, dev)
    _state_call((_lib or lib()).spec_state_attend, "spec_state_attend", OP_STATE_ATTEND, before, B, n, dev, ws, st,
                before, q.data_ptr(), qst, k.data_ptr(), kst, v.data_ptr(), vst, code, B, n, Hk, decay.data_ptr(), gst,
                _ptr(parents), np_, Dk ** -0.5 if scale is None else float(scale), o["out"].data_ptr(), ost, _status(o, B, dev))
    return o


def _state_call(fn, what, op, before, B, n, dev, ws, stream, *args):
    """As _with_workspace."""
    with _stream_lock(dev.index, stream):
        have = ws if ws is not None else _workspaces.get((dev.index, stream))
        p, size = (None, 0) if have is None else (have.data_ptr(), have.numel())
        rc = _on(dev, fn, *args, p, size, stream)
        if rc == SPEC_EWORKSPACE and ws is None:
            have = _workspace(_on(dev, lib().spec_state_workspace_size, op, before, B, n), dev, stream)
            rc = _on(dev, fn, *args, have.data_ptr(), have.numel(), stream)
    _check(rc, what)


def spec_state_commit(k: torch.Tensor, v: torch.Tensor, decay: torch.Tensor, state, *, slots=None, dst=None, dst_slots=None,
                      counts=None, index=None, out=None, stream=None) -> dict:
    """Advances each request's state by rows of k, v and decay: all of them, or counts int32 [B]; with index int32 [B, rows], row
    i is token index[b, i] (the accepted path: index = path_nodes, counts = n_emit of a verify call).  The states as in
    spec_state_forward -> status."""
    dev = k.device
    if stream is not None:
        return _on_stream(stream, spec_state_commit, k, v, decay, state, slots=slots, dst=dst, dst_slots=dst_slots, counts=counts,
                          index=index, out=out)
    st = _raw_stream(dev)
    code, kst, vst, gst = _state_rows(k, v, decay, dev)
    B, n, Hk, Dk = k.shape
    before, after = _state_pools(state, slots, dst, dst_slots, B, (v.shape[2], Dk, v.shape[3]), dev)
    ip, ist, rows = _index_rows(index, counts, B, n, dev)
    o = out or dict(status=torch.empty(B, dtype=torch.int32, device=dev))
    rc = _on(dev, (_lib or lib()).spec_state_commit, before, after, k.data_ptr(), kst, v.data_ptr(), vst, code, B, n, Hk,
             decay.data_ptr(), gst, ip, ist, rows, _ptr(counts), _status(o, B, dev), st)
    _check(rc, "spec_state_commit")
    return o
