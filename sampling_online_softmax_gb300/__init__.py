"""Speculative-decoding verify-and-sample step for NVIDIA GB300 (sm_103a).

Python binding of ``libspecverify.so`` (C ABI in ``include/spec_verify.h``).
This module only marshals arguments: it allocates outputs and the workspace
with PyTorch, passes raw device pointers and the current CUDA stream, and
raises ``SpecError`` on a non-OK status.  Every step of the computation runs in
the library's CUDA kernels; there is no fallback, and importing the functions
fails loudly when the library has not been built.

Entry points (same names as the C ABI):
  spec_verify_linear   accept/reject K draft tokens per sequence and draw the
                       extra token ("Beschleunigung von Sonar durch Spekulation",
                       sections "Spekulatives Decoding" and "Ziel-Entwurf")
  spec_sample_bonus    the extra token alone, given accept_len
  spec_verify_tree     greedy walk of a Medusa candidate tree
                       ("Speculative-Decoding / Medusa", section 三)
  spec_verify_tree_sample  the same walk with the target's choice drawn at
                       every node (the section's sampled variant)
  spec_sample_rows     one token per row (the draft side's next token)
  spec_tree_mask       the tree attention mask (ancestor bits) and depths
  spec_build_sparse_tree  the greedy sparse candidate tree from per-head top-i
                       accuracies (the blog's section 四; host code)
  spec_mtp_plug        the MTP draft layer's next input tokens from a verify's
                       outputs, and the advanced lengths, on the device
                       ("Beschleunigung von Sonar durch Spekulation", sections
                       "MTP" and "MTP-Zeitplan für ein einzelnes Token")
  spec_sample_filtered, spec_top_logits, spec_distill, spec_distill_backward
                       operators on rows of logits
  spec_adjust_logits   penalties, biases and grammar masks on a verify's rows
  spec_tree_attention, spec_cache_append, spec_cache_read
                       attention of drafted tokens over a paged cache, which is
                       written and read back in 8 bits or as it is
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libspecverify.so")

SPEC_OK = 0
SPEC_ERR_INVALID_ARG = 1
SPEC_ERR_UNSUPPORTED = 2
SPEC_ERR_CUDA = 3
SPEC_ERR_WORKSPACE = 4

SPEC_F32 = 0
SPEC_BF16 = 1
SPEC_F16 = 2
SPEC_E4M3 = 3

DEV_BAD_TOKEN = 1
DEV_NONFINITE = 2
DEV_TIMEOUT = 4
DEV_ZERO_RESIDUAL = 8
DEV_BAD_TREE = 16
DEV_BAD_LENGTH = 32
DEV_BAD_PARAM = 64
DEV_BAD_PAGE = 128

MAX_ROW_BYTES = 1 << 20  # SPEC_MAX_ROW_BYTES
MAX_TOP = 1024           # SPEC_MAX_TOP
MAX_NODES = 1024         # SPEC_MAX_NODES
MAX_BIASES = 1024        # SPEC_MAX_BIASES


class SpecError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__("%s (%s)" % (detail, _status_name(status)))
        self.status = status


class _Cache(ctypes.Structure):
    """spec_cache of the C ABI."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("dtype", ctypes.c_int), ("pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("table_width", ctypes.c_int)]


_lock = threading.Lock()
_lib = None


def load_library():
    """Load libspecverify.so; raises ImportError if it was not built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ImportError("libspecverify.so is not built (run __graft_entry__.build() or "
                              "python -m sampling_online_softmax_gb300.build)")
        lib = ctypes.CDLL(LIB_PATH)
        P, i32, u64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
        lib.spec_workspace_bytes_linear.argtypes = [i32, i32, i32, i32]
        lib.spec_workspace_bytes_linear.restype = u64
        lib.spec_workspace_bytes_bonus.argtypes = [i32, i32, i32]
        lib.spec_workspace_bytes_bonus.restype = u64
        lib.spec_workspace_bytes_tree.argtypes = [i32, i32, i32, i32]
        lib.spec_workspace_bytes_tree.restype = u64
        lib.spec_workspace_bytes_tree_sample.argtypes = [i32, i32, i32, i32]
        lib.spec_workspace_bytes_rows.argtypes = [i32, i32, i32]
        lib.spec_workspace_bytes_rows.restype = u64
        lib.spec_sample_rows.argtypes = [P, i32, i32, i32, P, f32, P, P, P, u64, P]
        lib.spec_sample_rows.restype = i32
        lib.spec_tree_mask.argtypes = [P, i32, P, P, P, P]
        lib.spec_tree_mask.restype = i32
        lib.spec_build_sparse_tree.argtypes = [P, i32, i32, i32, P, P, P, P, P]
        lib.spec_build_sparse_tree.restype = i32
        lib.spec_mtp_plug.argtypes = [P, i32, i32, P, P, ctypes.c_int32, P, P, P, P]
        lib.spec_mtp_plug.restype = i32
        lib.spec_workspace_bytes_tree_sample.restype = u64
        lib.spec_verify_linear.argtypes = [P, P, i32, i32, i32, i32, P, P, P, f32, P, P, P, P, P, P, u64, P]
        lib.spec_verify_linear.restype = i32
        lib.spec_verify_linear_static.argtypes = [P, P, i32, i32, i32, i32, P, P, P, f32, P, P, P, P, P, P]
        lib.spec_verify_linear_static.restype = i32
        lib.spec_sample_bonus.argtypes = [P, P, i32, i32, i32, i32, P, P, f32, P, P, P, u64, P]
        lib.spec_sample_bonus.restype = i32
        lib.spec_verify_tree.argtypes = [P, i32, i32, i32, i32, P, P, i32, P, P, P, P, P, u64, P]
        lib.spec_verify_tree.restype = i32
        lib.spec_verify_tree_sample.argtypes = [P, i32, i32, i32, i32, P, P, P, f32, i32, P, P, P, P, P, u64, P]
        lib.spec_verify_tree_sample.restype = i32
        lib.spec_sample_filtered.argtypes = [P, i32, i32, i32, P, P, P, P, P, P, P, P]
        lib.spec_sample_filtered.restype = i32
        lib.spec_top_logits.argtypes = [P, i32, i32, i32, i32, f32, P, P, P, P, P]
        lib.spec_top_logits.restype = i32
        lib.spec_distill.argtypes = [P, i32, i32, i32, P, P, i32, P, f32, P, P, P, P, P, P]
        lib.spec_distill.restype = i32
        lib.spec_distill_backward.argtypes = [P, i32, i32, i32, P, P, i32, P, f32, P, P, P, P, P, P]
        lib.spec_distill_backward.restype = i32
        lib.spec_adjust_logits.argtypes = [P, i32, i32, i32, i32, P, i32, P, P, P, P, P, P, P, P, P, i32, P, P, P, P]
        lib.spec_adjust_logits.restype = i32
        lib.spec_cache_append.argtypes = [P, P, i32, i32, i32, P, P, i32, P, P, P, P, P]
        lib.spec_cache_append.restype = i32
        lib.spec_cache_read.argtypes = [P, i32, i32, P, P, P, P, i32, P, P]
        lib.spec_cache_read.restype = i32
        lib.spec_workspace_bytes_attention.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.spec_workspace_bytes_attention.restype = u64
        lib.spec_tree_attention.argtypes = [P, P, P, i32, i32, i32, i32, P, P, P, i32, P, f32, P, P, P, P, u64, P]
        lib.spec_tree_attention.restype = i32
        lib.spec_status_string.argtypes = [i32]
        lib.spec_status_string.restype = ctypes.c_char_p
        lib.spec_last_error.argtypes = []
        lib.spec_last_error.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _status_name(status: int) -> str:
    try:
        return load_library().spec_status_string(int(status)).decode()
    except ImportError:
        return "status %d" % status


def _check(status: int):
    if status != SPEC_OK:
        raise SpecError(status, load_library().spec_last_error().decode() or "call failed")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SPEC_F32
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    raise TypeError("logits must be float32 or bfloat16, got %s" % t.dtype)


def _cuda(t, name, dtype=None, device=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, the logits on %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return t


def _outputs(out, shapes, device):
    """Check caller-provided output tensors: every name present, int32/float32 as
    given, on `device`, contiguous, with exactly the shape the kernel writes."""
    for name, (shape, dtype) in shapes.items():
        t = out.get(name)
        if t is None:
            raise ValueError("out[%r] is missing" % name)
        _cuda(t, "out[%r]" % name, dtype, device)
        if tuple(t.shape) != tuple(shape):
            raise ValueError("out[%r] must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return out


def _status(status, device, stream):
    if status is None:
        with torch.cuda.stream(stream):
            return torch.zeros(1, dtype=torch.int32, device=device)
    _cuda(status, "status", torch.int32, device)
    if status.numel() < 1:
        raise ValueError("status must hold at least one int32")
    return status


def _ws(workspace, nbytes, device, stream):
    if workspace is None:
        return _workspace(device, stream, nbytes)
    _cuda(workspace, "workspace", None, device)
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError("workspace needs %d bytes" % nbytes)
    return workspace


def _tree_shapes(parents, node_tokens, B, N):
    if parents.numel() != N:
        raise ValueError("parents must hold N = %d entries" % N)
    if tuple(node_tokens.shape) != (B, N):
        raise ValueError("node_tokens must be [B, N]")


def _tree_inputs(target, parents, node_tokens):
    """Check the inputs of a tree verify; returns (B, N, V, device)."""
    _cuda(target, "target")
    if target.dim() != 3:
        raise ValueError("target must be [B, N, V]")
    B, N, V = target.shape
    dev = target.device
    if parents is None or node_tokens is None:
        raise ValueError("parents and node_tokens are required")
    _cuda(parents, "parents", torch.int32, dev)
    _cuda(node_tokens, "node_tokens", torch.int32, dev)
    _tree_shapes(parents, node_tokens, B, N)
    return B, N, V, dev


def _tree_outputs(out, B, D, dev):
    if D < 0:
        raise ValueError("max_depth must be >= 0")
    if out is None:
        out = dict(path_nodes=torch.empty((B, D + 1), dtype=torch.int32, device=dev),
                   path_len=torch.empty(B, dtype=torch.int32, device=dev),
                   out_tokens=torch.empty((B, D + 1), dtype=torch.int32, device=dev))
    return _outputs(out, {"path_nodes": ((B, D + 1), torch.int32), "path_len": ((B,), torch.int32),
                          "out_tokens": ((B, D + 1), torch.int32)}, dev)


def _stream_handle(device, stream):
    s = torch.cuda.current_stream(device) if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream), s


# one zero-filled workspace per (device, stream), grown on demand; every call
# leaves it zero-filled again, so it is cleared only when allocated
_ws_cache = {}
_ws_lock = threading.Lock()


def _workspace(device, stream, nbytes):
    key = (device.index, stream.cuda_stream)
    with _ws_lock:
        ws = _ws_cache.get(key)
        if ws is None or ws.numel() < nbytes:
            with torch.cuda.stream(stream):
                ws = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
            _ws_cache[key] = ws
        return ws


def _dtype_arg(dtype) -> int:
    if isinstance(dtype, torch.dtype):
        return SPEC_F32 if dtype == torch.float32 else SPEC_BF16
    return int(dtype)


def spec_workspace_bytes_linear(B: int, K: int, V: int, dtype) -> int:
    return int(load_library().spec_workspace_bytes_linear(int(B), int(K), int(V), _dtype_arg(dtype)))


def spec_workspace_bytes_bonus(B: int, V: int, dtype) -> int:
    return int(load_library().spec_workspace_bytes_bonus(int(B), int(V), _dtype_arg(dtype)))


def spec_workspace_bytes_tree(B: int, N: int, V: int, dtype) -> int:
    return int(load_library().spec_workspace_bytes_tree(int(B), int(N), int(V), _dtype_arg(dtype)))


def spec_workspace_bytes_rows(B: int, V: int, dtype) -> int:
    return int(load_library().spec_workspace_bytes_rows(int(B), int(V), _dtype_arg(dtype)))


def spec_workspace_bytes_tree_sample(B: int, N: int, V: int, dtype) -> int:
    return int(load_library().spec_workspace_bytes_tree_sample(int(B), int(N), int(V), _dtype_arg(dtype)))


def _linear_inputs(target, draft, draft_tokens, u_accept, u_bonus):
    """Check the inputs of a linear verify; returns (B, K, V, device)."""
    _cuda(target, "target")
    if target.dim() != 3:
        raise ValueError("target must be [B, K+1, V]")
    B, K1, V = target.shape
    K = K1 - 1
    dev = target.device
    _cuda(draft, "draft", None, dev)
    _cuda(draft_tokens, "draft_tokens", torch.int32, dev)
    _cuda(u_accept, "u_accept", torch.float32, dev)
    _cuda(u_bonus, "u_bonus", torch.float32, dev)
    if draft is not None and (draft.dtype != target.dtype or tuple(draft.shape) != (B, K, V)):
        raise ValueError("draft must match target's dtype with shape [B, K, V]")
    if draft_tokens is not None and tuple(draft_tokens.shape) != (B, K):
        raise ValueError("draft_tokens must be [B, K]")
    if u_accept is not None and tuple(u_accept.shape) != (B, K):
        raise ValueError("u_accept must be [B, K]")
    if u_bonus is not None and tuple(u_bonus.shape) != (B,):
        raise ValueError("u_bonus must be [B]")
    return B, K, V, dev


def _linear_outputs(out, B, K, dev):
    shapes = {"accept_len": ((B,), torch.int32), "out_tokens": ((B, K + 1), torch.int32),
              "num_emitted": ((B,), torch.int32)}
    if out.get("probs") is not None:
        shapes["probs"] = ((B, K, 3), torch.float32)
    return _outputs(out, shapes, dev)


def spec_verify_linear(target, draft, draft_tokens, u_accept, u_bonus, temperature, *,
                       probs: bool = False, status=None, out=None, workspace=None, stream=None):
    """Verify K draft tokens per sequence; returns a dict of device tensors.

    target [B, K+1, V] and draft [B, K, V] (float32 or bfloat16; draft may be
    None in greedy mode), draft_tokens [B, K] int32, u_accept [B, K] float32,
    u_bonus [B] float32 or None (no extra token), temperature >= 0 (0: greedy).
    Result: accept_len [B], out_tokens [B, K+1], num_emitted [B], status [1]
    (SPEC_DEV_* bits, int32), and probs [B, K, 3] when requested.
    """
    lib = load_library()
    B, K, V, dev = _linear_inputs(target, draft, draft_tokens, u_accept, u_bonus)
    h, s = _stream_handle(dev, stream)
    if out is None:
        out = dict(accept_len=torch.empty(B, dtype=torch.int32, device=dev),
                   out_tokens=torch.empty((B, K + 1), dtype=torch.int32, device=dev),
                   num_emitted=torch.empty(B, dtype=torch.int32, device=dev))
        if probs:
            out["probs"] = torch.empty((B, K, 3), dtype=torch.float32, device=dev)
    _linear_outputs(out, B, K, dev)
    status = _status(status, dev, s)
    out["status"] = status
    nbytes = spec_workspace_bytes_linear(B, K, V, target.dtype)
    ws = _ws(workspace, nbytes, dev, s)
    with torch.cuda.device(dev):
        st = lib.spec_verify_linear(
            _ptr(target), _ptr(draft), _dtype_code(target), B, K, V, _ptr(draft_tokens), _ptr(u_accept),
            _ptr(u_bonus), float(temperature), _ptr(out["accept_len"]), _ptr(out["out_tokens"]),
            _ptr(out["num_emitted"]), _ptr(out.get("probs")), _ptr(status), _ptr(ws), ws.numel(), h)
    _check(st)
    return out


def spec_verify_linear_static(target, draft, draft_tokens, u_accept, u_bonus, temperature, *, out, status,
                              stream=None):
    """spec_verify_linear on the library's built-in per-device workspace.

    For callers that must not allocate device memory during the step: nothing
    is allocated here either, so `out` (accept_len, out_tokens, num_emitted and
    optionally probs, as returned by spec_verify_linear) and `status` (int32 [1],
    zeroed by the caller) must be passed in.  Calls that may overlap in time
    share the one workspace and race; keep them on one stream.
    """
    lib = load_library()
    B, K, V, dev = _linear_inputs(target, draft, draft_tokens, u_accept, u_bonus)
    _linear_outputs(out, B, K, dev)
    if status is None:
        raise ValueError("status must be passed in (nothing is allocated here)")
    _cuda(status, "status", torch.int32, dev)
    if status.numel() < 1:
        raise ValueError("status must hold at least one int32")
    h, _ = _stream_handle(dev, stream)
    with torch.cuda.device(dev):
        st = lib.spec_verify_linear_static(
            _ptr(target), _ptr(draft), _dtype_code(target), B, K, V, _ptr(draft_tokens), _ptr(u_accept),
            _ptr(u_bonus), float(temperature), _ptr(out["accept_len"]), _ptr(out["out_tokens"]),
            _ptr(out["num_emitted"]), _ptr(out.get("probs")), _ptr(status), h)
    _check(st)
    out["status"] = status
    return out


def spec_sample_bonus(target, draft, accept_len, u_bonus, temperature, *, status=None, out=None, workspace=None,
                      stream=None):
    """The extra token alone at row accept_len[b]; returns dict(bonus_token [B], status [1])."""
    lib = load_library()
    _cuda(target, "target")
    if target.dim() != 3:
        raise ValueError("target must be [B, K+1, V]")
    B, K1, V = target.shape
    K = K1 - 1
    dev = target.device
    _cuda(draft, "draft", None, dev)
    _cuda(accept_len, "accept_len", torch.int32, dev)
    _cuda(u_bonus, "u_bonus", torch.float32, dev)
    if draft is not None and (draft.dtype != target.dtype or tuple(draft.shape) != (B, K, V)):
        raise ValueError("draft must match target's dtype with shape [B, K, V]")
    if accept_len is not None and tuple(accept_len.shape) != (B,):
        raise ValueError("accept_len must be [B]")
    if u_bonus is not None and tuple(u_bonus.shape) != (B,):
        raise ValueError("u_bonus must be [B]")
    h, s = _stream_handle(dev, stream)
    if out is None:
        out = torch.empty(B, dtype=torch.int32, device=dev)
    _outputs(dict(bonus_token=out), {"bonus_token": ((B,), torch.int32)}, dev)
    status = _status(status, dev, s)
    nbytes = spec_workspace_bytes_bonus(B, V, target.dtype)
    ws = _ws(workspace, nbytes, dev, s)
    with torch.cuda.device(dev):
        st = lib.spec_sample_bonus(_ptr(target), _ptr(draft), _dtype_code(target), B, K, V, _ptr(accept_len),
                                   _ptr(u_bonus), float(temperature), _ptr(out), _ptr(status), _ptr(ws),
                                   ws.numel(), h)
    _check(st)
    return dict(bonus_token=out, status=status)


def spec_verify_tree(target, parents, node_tokens, max_depth, *, status=None, out=None, workspace=None,
                     stream=None):
    """Greedy tree walk; returns dict(path_nodes, path_len, out_tokens, status)."""
    lib = load_library()
    B, N, V, dev = _tree_inputs(target, parents, node_tokens)
    h, s = _stream_handle(dev, stream)
    D = int(max_depth)
    out = _tree_outputs(out, B, D, dev)
    status = _status(status, dev, s)
    out["status"] = status
    nbytes = spec_workspace_bytes_tree(B, N, V, target.dtype)
    ws = _ws(workspace, nbytes, dev, s)
    with torch.cuda.device(dev):
        st = lib.spec_verify_tree(_ptr(target), _dtype_code(target), B, N, V, _ptr(parents), _ptr(node_tokens), D,
                                  _ptr(out["path_nodes"]), _ptr(out["path_len"]), _ptr(out["out_tokens"]),
                                  _ptr(status), _ptr(ws), ws.numel(), h)
    _check(st)
    return out


def spec_verify_tree_sample(target, parents, node_tokens, u_nodes, temperature, max_depth, *, status=None,
                            out=None, workspace=None, stream=None):
    """Tree walk with the target's choice drawn at every node (u_nodes [B, N] fp32);
    returns dict(path_nodes, path_len, out_tokens, status)."""
    lib = load_library()
    B, N, V, dev = _tree_inputs(target, parents, node_tokens)
    if u_nodes is None:
        raise ValueError("u_nodes is required")
    _cuda(u_nodes, "u_nodes", torch.float32, dev)
    if tuple(u_nodes.shape) != (B, N):
        raise ValueError("u_nodes must be [B, N]")
    h, s = _stream_handle(dev, stream)
    D = int(max_depth)
    out = _tree_outputs(out, B, D, dev)
    status = _status(status, dev, s)
    out["status"] = status
    nbytes = spec_workspace_bytes_tree_sample(B, N, V, target.dtype)
    ws = _ws(workspace, nbytes, dev, s)
    with torch.cuda.device(dev):
        st = lib.spec_verify_tree_sample(_ptr(target), _dtype_code(target), B, N, V, _ptr(parents),
                                         _ptr(node_tokens), _ptr(u_nodes), float(temperature), D,
                                         _ptr(out["path_nodes"]), _ptr(out["path_len"]), _ptr(out["out_tokens"]),
                                         _ptr(status), _ptr(ws), ws.numel(), h)
    _check(st)
    return out


def spec_sample_rows(logits, u, temperature, *, status=None, out=None, workspace=None, stream=None):
    """One token per row of logits [B, V]: a draw from softmax(l / T) at u [B] (float32), or the
    argmax when temperature == 0 (u may be None); returns dict(tokens [B], status)."""
    lib = load_library()
    _cuda(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [B, V]")
    B, V = logits.shape
    dev = logits.device
    _cuda(u, "u", torch.float32, dev)
    if u is not None and tuple(u.shape) != (B,):
        raise ValueError("u must be [B]")
    h, s = _stream_handle(dev, stream)
    if out is None:
        out = dict(tokens=torch.empty(B, dtype=torch.int32, device=dev))
    _outputs(out, {"tokens": ((B,), torch.int32)}, dev)
    status = _status(status, dev, s)
    out["status"] = status
    nbytes = spec_workspace_bytes_rows(B, V, logits.dtype)
    ws = _ws(workspace, nbytes, dev, s)
    with torch.cuda.device(dev):
        st = lib.spec_sample_rows(_ptr(logits), _dtype_code(logits), B, V, _ptr(u), float(temperature),
                                  _ptr(out["tokens"]), _ptr(status), _ptr(ws), ws.numel(), h)
    _check(st)
    return out


# The operators on rows of logits are short calls (a few microseconds on the device), so their checks
# take the quick way first: one look at each tensor, and the named refusal only where it fails.
def _need(t, name, dtype, shape, dev, index):
    """`t` is on the device, contiguous, and of this type and shape; returns its address."""
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous()):  # (a CPU tensor's: -1)
        _cuda(t, name, dtype, dev)
        if tuple(t.shape) != tuple(shape):
            raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return t.data_ptr()


def _may(t, name, dtype, shape, dev, index):
    return None if t is None else _need(t, name, dtype, shape, dev, index)


def _logits_2d(t, name):
    """Checks a matrix of logits; returns (rows, V, device, its index, dtype code)."""
    if not (t.is_cuda and t.is_contiguous()):
        _cuda(t, name)
    if t.dim() != 2:
        raise ValueError("%s must be [rows, V]" % name)
    rows, V = t.shape
    dev = t.device
    return rows, V, dev, dev.index, _dtype_code(t)


_ON_CURRENT = contextlib.nullcontext()


def _results(out, shapes, status, dev, index, stream):
    """The outputs (new ones, from the memory of the stream that the kernel runs on, where `out` is
    None) and the status word: returns (out, the addresses by shapes' order, status' address)."""
    if out is None or status is None:
        with _ON_CURRENT if stream is None else torch.cuda.stream(stream):
            if out is None:
                out = {n: torch.empty(shape, dtype=dtype, device=dev) for n, (shape, dtype) in shapes.items()}
            if status is None:
                status = torch.zeros(1, dtype=torch.int32, device=dev)
    at = []
    for name, (shape, dtype) in shapes.items():
        t = out.get(name)
        if t is None:
            raise ValueError("out[%r] is missing" % name)
        at.append(_need(t, "out[%r]" % name, dtype, shape, dev, index))
    if not (status.is_cuda and status.dtype is torch.int32 and status.get_device() == index and status.is_contiguous()):
        _cuda(status, "status", torch.int32, dev)
    if status.numel() < 1:
        raise ValueError("status must hold at least one int32")
    out["status"] = status
    return out, at, status.data_ptr()


def _raw_stream(index):
    """The handle of the device's current stream (torch.cuda.current_stream, without the object: 2 us)."""
    return torch._C._cuda_getCurrentRawStream(index)


def _alloc(nbytes, stream):
    """Memory of the caching allocator for a stream (its handle) of the current device: the address.  (torch.empty takes 5 us
    more beside a launch.)"""
    return torch._C._cuda_cudaCachingAllocator_raw_alloc(nbytes, stream)


def _free(at):
    """Gives memory of _alloc back: what the stream has enqueued keeps it, as it does a freed tensor's."""
    torch._C._cuda_cudaCachingAllocator_raw_delete(at)


def _capturing(stream):
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _launch(fn, args, tensors, dev, stream):
    """Calls the library on `stream` (the device's current one where it is None), with the tensors'
    device current.  A stream that is not the current one first waits for it, where the tensors were
    made (not into or out of a graph capture: there the caller orders), and keeps their memory until
    it is done."""
    current = None
    if stream is None:
        h = _raw_stream(dev.index)
    else:
        h = stream.cuda_stream
        current = torch.cuda.current_stream(dev)
        if stream == current:
            current = None
        elif not (_capturing(stream) or _capturing(current)):
            stream.wait_stream(current)
    if dev.index == torch.cuda.current_device():
        st = fn(*args, h)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, h)
    if st != SPEC_OK:
        _check(st)
    if current is not None:
        for t in tensors:
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)


def spec_sample_filtered(logits, u, temperature, *, top_k=None, top_p=None, min_p=None, status=None, out=None,
                         stream=None):
    """One token per row of logits [B, V] under temperature [B] (float32; 0: the argmax), top_k [B]
    (int32; <= 0: no limit), top_p [B] and min_p [B] (float32), at u [B] (float32, in [0, 1)); a
    filter left None does not limit.  Returns dict(tokens [B], status).

    Draft tokens for spec_verify_linear come from spec_sample_rows, or from this without filters at
    the verify's temperature: it tests them against the whole draft row's softmax."""
    lib = load_library()
    B, V, dev, i, code = _logits_2d(logits, "logits")
    if u is None or temperature is None:
        raise ValueError("u and temperature are required")
    f32, row = torch.float32, (B,)
    args = [_need(temperature, "temperature", f32, row, dev, i), _may(top_k, "top_k", torch.int32, row, dev, i),
            _may(top_p, "top_p", f32, row, dev, i), _may(min_p, "min_p", f32, row, dev, i), _need(u, "u", f32, row, dev, i)]
    out, (tokens,), st = _results(out, {"tokens": (row, torch.int32)}, status, dev, i, stream)
    _launch(lib.spec_sample_filtered, (logits.data_ptr(), code, B, V, *args, tokens, st),
            (logits, u, temperature, top_k, top_p, min_p, *out.values()), dev, stream)
    return out


def spec_top_logits(logits, k, *, temperature=1.0, lse=False, status=None, out=None, stream=None):
    """The k largest logits of each row of logits [B, V], falling, the lower index first among equal
    ones: returns dict(values [B, k] float32, ids [B, k] int32, status), and with lse=True also
    lse [B] float32, the log-normaliser log sum exp(l / temperature).  Entries past a row's last
    unmasked token are (-inf, -1)."""
    lib = load_library()
    B, V, dev, i, code = _logits_2d(logits, "logits")
    k = int(k)
    if k < 1:
        raise ValueError("k must be >= 1")
    shapes = {"values": ((B, k), torch.float32), "ids": ((B, k), torch.int32)}
    if lse:
        shapes["lse"] = ((B,), torch.float32)
    out, at, st = _results(out, shapes, status, dev, i, stream)
    _launch(lib.spec_top_logits, (logits.data_ptr(), code, B, V, k, float(temperature), at[0], at[1], at[2] if lse else None, st),
            (logits, *out.values()), dev, stream)
    return out


def _overwritten(grad):
    """A gradient written into the caller's tensor, the logits' own perhaps: autograd, which sees only the
    address change hands, refuses a graph that saved what was there."""
    torch.autograd.graph.increment_version(grad)


def _distill_inputs(student, top_ids, top_logits, top_lse, row_weight, temperature):
    """Checks the inputs of a distillation; returns (N, V, device, its index, the call's first arguments)."""
    N, V, dev, i, code = _logits_2d(student, "student")
    if top_ids is None or top_logits is None:
        raise ValueError("top_ids and top_logits are required")
    if top_ids.dim() != 2 or top_ids.shape[1] < 1:
        raise ValueError("top_ids must be [N, K]")
    K = top_ids.shape[1]
    f32 = torch.float32
    return N, V, dev, i, (student.data_ptr(), code, N, V, _need(top_ids, "top_ids", torch.int32, (N, K), dev, i),
                          _need(top_logits, "top_logits", f32, (N, K), dev, i), K, _may(top_lse, "top_lse", f32, (N,), dev, i),
                          float(temperature), _may(row_weight, "row_weight", f32, (N,), dev, i))


def spec_distill(student, top_ids, top_logits, temperature=1.0, *, top_lse=None, row_weight=None, grad=False,
                 status=None, out=None, stream=None):
    """Distillation loss of student logits [N, V] against a teacher's largest logits (top_ids [N, K]
    int32, top_logits [N, K] float32, and with top_lse [N] float32 its log-normaliser, which weighs
    a row by the mass P of its entries, the rest of the teacher entering nothing; as
    spec_top_logits returns them): returns dict(loss [N], stats [N, 2], status), and with grad=True
    also grad [N, V], the gradient of the summed losses in student's dtype (out["grad"] may be
    student itself: autograd then refuses a graph that saved the logits).  row_weight [N] scales
    each row; a row of weight 0 is not read.

    No autograd graph is recorded: pass the gradient on with student.backward(r["grad"]), or keep
    stats for spec_distill_backward."""
    lib = load_library()
    N, V, dev, i, args = _distill_inputs(student, top_ids, top_logits, top_lse, row_weight, temperature)
    shapes = {"loss": ((N,), torch.float32), "stats": ((N, 2), torch.float32)}
    if grad:
        shapes["grad"] = ((N, V), student.dtype)
    given = grad and out is not None
    out, at, st = _results(out, shapes, status, dev, i, stream)
    _launch(lib.spec_distill, (*args, at[0], at[1], at[2] if grad else None, st),
            (student, top_ids, top_logits, top_lse, row_weight, *out.values()), dev, stream)
    if given:
        _overwritten(out["grad"])
    return out


def spec_distill_backward(student, top_ids, top_logits, stats, grad_loss, temperature=1.0, *, top_lse=None,
                          row_weight=None, status=None, out=None, stream=None):
    """The gradient of sum(grad_loss * loss) with respect to student, from spec_distill's stats of
    the same inputs: returns dict(grad [N, V] in student's dtype, status).  out may be student."""
    lib = load_library()
    N, V, dev, i, args = _distill_inputs(student, top_ids, top_logits, top_lse, row_weight, temperature)
    if stats is None or grad_loss is None:
        raise ValueError("stats and grad_loss are required")
    f32 = torch.float32
    more = (_need(stats, "stats", f32, (N, 2), dev, i), _need(grad_loss, "grad_loss", f32, (N,), dev, i))
    r, (g,), st = _results(None if out is None else dict(grad=out), {"grad": ((N, V), student.dtype)}, status, dev, i, stream)
    _launch(lib.spec_distill_backward, (*args, *more, g, st),
            (student, top_ids, top_logits, top_lse, row_weight, stats, grad_loss, *r.values()), dev, stream)
    if out is not None:
        _overwritten(out)
    return r


def spec_adjust_logits(logits, *, tokens=None, prompt_len=None, total_len=None, node_tokens=None, mask=None, repetition=None,
                       frequency=None, presence=None, bias_ids=None, bias=None, allowed=None, out=None, status=None, stream=None):
    """Penalties for repeated tokens, biases and grammar masks on logits [B, N, V] (a verify's target rows: N = K + 1 for a
    linear draft, the tree's nodes, or 1 without a draft): returns dict(logits [B, N, V], status).

    tokens [B, L] int32 is the history (prompt_len [B], total_len [B]: where the prompt and the history end; -1 is no token),
    node_tokens [B, N] int32 the drafted tokens (column 0, the root, ignored), mask [N, ceil(N/32)] their paths as
    spec_tree_mask gives them (None: a chain).  A row counts the history and its own path: repetition (divides or
    multiplies), frequency (a count) and presence [B] float32.  bias_ids, bias [B, M] add to tokens; allowed
    [B, N, ceil(V/32)] int32 holds a bit a token, 0 for -inf.  out=dict(logits=logits) works in place (autograd then
    refuses a graph that saved the logits).  No autograd graph is recorded."""
    lib = load_library()
    if not (logits.is_cuda and logits.is_contiguous()):
        _cuda(logits, "logits")
    if logits.dim() != 3:
        raise ValueError("logits must be [B, N, V]")
    B, N, V = logits.shape
    dev = logits.device
    i, code, i32, f32 = dev.index, _dtype_code(logits), torch.int32, torch.float32
    if N < 1 or V < 1:
        raise ValueError("logits must have at least one row and one token")
    L = M = 0
    if tokens is not None:
        if tokens.dim() != 2:
            raise ValueError("tokens must be [B, L]")
        L = tokens.shape[1]
    if (bias_ids is None) != (bias is None):
        raise ValueError("bias_ids and bias go together")
    if bias_ids is not None:
        if bias_ids.dim() != 2:
            raise ValueError("bias_ids must be [B, M]")
        M = bias_ids.shape[1]
    row = (B,)
    args = (_may(tokens, "tokens", i32, (B, L), dev, i), L, _may(prompt_len, "prompt_len", i32, row, dev, i),
            _may(total_len, "total_len", i32, row, dev, i), _may(node_tokens, "node_tokens", i32, (B, N), dev, i),
            _may(mask, "mask", i32, (N, (N + 31) // 32), dev, i), _may(repetition, "repetition", f32, row, dev, i),
            _may(frequency, "frequency", f32, row, dev, i), _may(presence, "presence", f32, row, dev, i),
            _may(bias_ids, "bias_ids", i32, (B, M), dev, i), _may(bias, "bias", f32, (B, M), dev, i), M,
            _may(allowed, "allowed", i32, (B, N, (V + 31) // 32), dev, i))
    given = out is not None
    out, (at,), st = _results(out, {"logits": ((B, N, V), logits.dtype)}, status, dev, i, stream)
    _launch(lib.spec_adjust_logits, (logits.data_ptr(), code, B, N, V, *args, at, st),
            (logits, tokens, prompt_len, total_len, node_tokens, mask, repetition, frequency, presence, bias_ids, bias, allowed,
             *out.values()), dev, stream)
    if given:
        _overwritten(out["logits"])
    return out


_CODES = {torch.bfloat16: SPEC_BF16, torch.float16: SPEC_F16}


def _cache_arg(k_cache, v_cache, page_table, k_scale, v_scale, B, heads, dim, dtype, dev, i):
    """Checks a paged cache for keys and values of `heads` heads of `dim`; returns the C struct."""
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, kv_heads, page_size, head_dim]")
    pages, kv, page, d = k_cache.shape
    if (kv, d) != (heads, dim):
        raise ValueError("k_cache must have %d heads of %d, got %d of %d" % (heads, dim, kv, d))
    q8 = k_cache.dtype is torch.float8_e4m3fn
    if not q8 and k_cache.dtype is not dtype:
        raise TypeError("k_cache must be %s or torch.float8_e4m3fn, got %s" % (dtype, k_cache.dtype))
    if q8 != (k_scale is not None) or q8 != (v_scale is not None):
        raise ValueError("k_scale and v_scale belong to a float8_e4m3fn cache, and it needs both")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, width]")
    shape, width = (pages, kv, page), page_table.shape[1]
    return _Cache(_need(k_cache, "k_cache", k_cache.dtype, (pages, kv, page, d), dev, i), _need(v_cache, "v_cache", k_cache.dtype, (pages, kv, page, d), dev, i),
                  _may(k_scale, "k_scale", torch.uint8, shape, dev, i), _may(v_scale, "v_scale", torch.uint8, shape, dev, i),
                  _need(page_table, "page_table", torch.int32, (B, width), dev, i), SPEC_E4M3 if q8 else _CODES[dtype], pages, page, kv, d, width)


def _on_gpu(t, name):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)


def _token_rows(t, name, shape, dtype, dev):
    """Checks [B, N, heads, dim], whose heads lie together while its tokens may be strided; returns (address, batch
    and token strides, None where it is contiguous)."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev.index and t.is_contiguous():  # (a CPU tensor's: -1)
        p = t.data_ptr()
        if p % 16 == 0:
            return p, None
    _on_gpu(t, name)
    if t.device != dev:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, dev))
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    B, N, heads, dim = shape
    sb, sn, sh, sd = t.stride()
    if t.numel() and ((dim > 1 and sd != 1) or (heads > 1 and sh != dim)):
        raise ValueError("%s must have its heads next to each other (strides %s)" % (name, t.stride()))
    sn = sn if N > 1 else heads * dim  # (an axis of one entry has any stride)
    sb = sb if B > 1 else N * heads * dim
    if sb % 8 or sn % 8 or sb < 0 or sn < 0 or t.data_ptr() % 16:
        raise ValueError("%s must start on a 16-byte boundary with strides of whole 16 bytes (strides %s)" % (name, t.stride()))
    return t.data_ptr(), (sb, sn)


def _new_tokens(t, name):
    _on_gpu(t, name)
    if t.dim() != 4:
        raise ValueError("%s must be [B, N, heads, head_dim]" % name)
    if t.dtype not in _CODES:
        raise TypeError("%s must be bfloat16 or float16, got %s" % (name, t.dtype))
    return t.shape, t.dtype, t.device, t.device.index


def _strides(shapes, rows):
    """Batch and token strides of what _token_rows returned, as the C ABI takes them (NULL: all contiguous; the array takes 1.3 us)."""
    for r in rows:
        if r[1] is not None:
            break
    else:
        return None
    each = [r[1] or (n * heads * dim, heads * dim) for (_, n, heads, dim), r in zip(shapes, rows)]
    return (ctypes.c_longlong * (2 * len(rows)))(*(x for e in each for x in e))


def spec_cache_append(k, v, k_cache, v_cache, page_table, start, *, count=None, select=None, k_scale=None, v_scale=None, status=None,
                      stream=None):
    """Writes k, v [B, N, kv_heads, head_dim] (bfloat16 or float16; tokens may be strided) into a paged cache
    [pages, kv_heads, page_size, head_dim] of their type, or of float8_e4m3fn with k_scale, v_scale
    [pages, kv_heads, page_size] uint8 (a power of two a row): row i of sequence b goes to position start[b] + i, which
    page_table [B, width] int32 places.  select [B, S] int32 picks the rows (spec_verify_tree's path_nodes; -1: none);
    count [B] int32 limits them; a negative start leaves a sequence out.  Two different rows must not go to one slot.
    Returns dict(status)."""
    lib = load_library()
    shape, dtype, dev, i = _new_tokens(k, "k")
    B, N, heads, dim = shape
    at, sk = _token_rows(k, "k", shape, dtype, dev), _token_rows(v, "v", shape, dtype, dev)
    cache = _cache_arg(k_cache, v_cache, page_table, k_scale, v_scale, B, heads, dim, dtype, dev, i)
    if select is not None and select.dim() != 2:
        raise ValueError("select must be [B, S]")
    S = N if select is None else select.shape[1]
    i32 = torch.int32
    args = (_may(select, "select", i32, (B, S), dev, i), S, _need(start, "start", i32, (B,), dev, i), _may(count, "count", i32, (B,), dev, i))
    out, _, st = _results({}, {}, status, dev, i, stream)
    _launch(lib.spec_cache_append, (at[0], sk[0], _CODES[dtype], B, N, _strides((shape, shape), (at, sk)), *args, ctypes.byref(cache), st),
            (k, v, k_cache, v_cache, page_table, start, count, select, k_scale, v_scale, *out.values()), dev, stream)
    _overwritten((k_cache, v_cache) if k_scale is None else (k_cache, v_cache, k_scale, v_scale))
    return out


def spec_cache_read(k_cache, v_cache, page_table, start, n, *, count=None, k_scale=None, v_scale=None, dtype=None, status=None,
                    out=None, stream=None):
    """Reads n positions of every sequence, from start[b] on, out of a paged cache as spec_cache_append writes it: returns
    dict(k, v [B, n, kv_heads, head_dim], status), of the cache's type, or of `dtype` (bfloat16, float16; None: out's,
    or bfloat16) where the cache is float8_e4m3fn.  Rows from count[b] on are left as they were (new ones: 0)."""
    lib = load_library()
    _on_gpu(k_cache, "k_cache")
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [pages, kv_heads, page_size, head_dim]")
    _, heads, _, dim = k_cache.shape
    dev, n = k_cache.device, int(n)
    i = dev.index
    if k_cache.dtype in _CODES:
        dtype = k_cache.dtype
    elif dtype is None:
        dtype = torch.bfloat16 if out is None or out.get("k") is None else out["k"].dtype
    if dtype not in _CODES:
        raise TypeError("dtype must be bfloat16 or float16, got %s" % dtype)
    if n < 0:
        raise ValueError("n must be >= 0")
    if start is None or start.dim() != 1:
        raise ValueError("start must be [B]")
    B = start.shape[0]
    cache = _cache_arg(k_cache, v_cache, page_table, k_scale, v_scale, B, heads, dim, dtype, dev, i)
    args = (_need(start, "start", torch.int32, (B,), dev, i), _may(count, "count", torch.int32, (B,), dev, i))
    shape, given = (B, n, heads, dim), out is not None
    if not given:
        with _ON_CURRENT if stream is None else torch.cuda.stream(stream):
            out = {x: torch.zeros(shape, dtype=dtype, device=dev) for x in ("k", "v")}
    out, at, st = _results(out, {"k": (shape, dtype), "v": (shape, dtype)}, status, dev, i, stream)
    _launch(lib.spec_cache_read, (ctypes.byref(cache), B, n, *args, *at, _CODES[dtype], st),
            (k_cache, v_cache, page_table, start, count, k_scale, v_scale, *out.values()), dev, stream)
    if given:
        _overwritten((out["k"], out["v"]))
    return out


def spec_workspace_bytes_attention(B: int, N: int, heads: int, kv_heads: int, head_dim: int, shared_len: int = 0) -> int:
    return int(load_library().spec_workspace_bytes_attention(int(B), int(N), int(heads), int(kv_heads), int(head_dim), int(shared_len)))


@functools.lru_cache(maxsize=256)
def _attention_room(lib, *sizes):  # (of the sizes alone)
    return lib.spec_workspace_bytes_attention(*sizes)


def spec_tree_attention(q, k, v, k_cache, v_cache, page_table, context_lens, *, mask=None, shared_len=0, scale=None, k_scale=None,
                        v_scale=None, lse=False, status=None, out=None, workspace=None, stream=None):
    """Attention of the N drafted nodes of each sequence over its cached context and their own paths: q [B, N, heads,
    head_dim], k, v [B, N, kv_heads, head_dim] (bfloat16 or float16; tokens may be strided; not in the cache yet) and a paged
    cache as spec_cache_append writes it, of which sequence b holds context_lens[b] positions (int32; negative: left out).
    mask [N, ceil(N/32)] int32 as spec_tree_mask gives it (None: a chain, nodes 0 .. n; N = 1 is plain decoding).  The
    first shared_len positions are the same in every sequence and are read once, through page_table[0].  scale
    is 1 / sqrt(head_dim) where it is None.  Returns dict(out [B, N, heads, head_dim], status), with lse=True also
    lse [B, N, heads] float32, the log of the softmax's sum.  No autograd graph is recorded."""
    lib = load_library()
    qs, dtype, dev, i = _new_tokens(q, "q")
    B, N, heads, dim = qs
    if k.dim() != 4:
        raise ValueError("k must be [B, N, kv_heads, head_dim]")
    kv = k.shape[2]
    if N < 1 or kv < 1 or heads < 1 or heads % kv:
        raise ValueError("need N >= 1 and heads a multiple of kv_heads, got %d and %d of %d" % (N, heads, kv))
    ks = (B, N, kv, dim)
    at = [_token_rows(q, "q", qs, dtype, dev), _token_rows(k, "k", ks, dtype, dev), _token_rows(v, "v", ks, dtype, dev)]
    cache = _cache_arg(k_cache, v_cache, page_table, k_scale, v_scale, B, kv, dim, dtype, dev, i)
    shared_len = int(shared_len)
    args = (_need(context_lens, "context_lens", torch.int32, (B,), dev, i), shared_len, _may(mask, "mask", torch.int32, (N, (N + 31) // 32), dev, i),
            float(scale) if scale is not None else dim ** -0.5)
    shapes = {"out": (qs, dtype)}
    if lse:
        shapes["lse"] = ((B, N, heads), torch.float32)
    given = out is not None
    out, to, st = _results(out, shapes, status, dev, i, stream)
    own = None
    if workspace is None:  # the stream's own memory, or of the graph that is being captured, given back once the call is enqueued
        room = max(_attention_room(lib, B, N, heads, kv, dim, shared_len), 16)
        with _ON_CURRENT if i == torch.cuda.current_device() else torch.cuda.device(dev):
            at_ws = own = _alloc(room, _raw_stream(i) if stream is None else stream.cuda_stream)
    else:
        _cuda(workspace, "workspace", None, dev)
        at_ws, room = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    try:
        _launch(lib.spec_tree_attention, (at[0][0], at[1][0], at[2][0], _CODES[dtype], B, N, heads, _strides((qs, ks, ks), at), ctypes.byref(cache), *args,
                                          to[0], to[1] if lse else None, st, at_ws, room),
                (q, k, v, k_cache, v_cache, page_table, context_lens, mask, k_scale, v_scale, workspace, *out.values()), dev, stream)
    finally:
        if own is not None:
            _free(own)
    if given:
        _overwritten([out[x] for x in shapes])
    return out


def spec_tree_mask(parents, *, status=None, out=None, stream=None):
    """Tree attention mask of a parent array [N] (int32, CUDA): returns dict(mask [N, ceil(N/32)]
    (int32 words holding uint32 bits: bit j % 32 of word j // 32 of row i is set iff node j is node
    i or an ancestor), depth [N], status)."""
    lib = load_library()
    _cuda(parents, "parents", torch.int32)
    N = parents.numel()
    dev = parents.device
    h, s = _stream_handle(dev, stream)
    W = (N + 31) // 32
    if out is None:
        out = dict(mask=torch.empty((N, W), dtype=torch.int32, device=dev),
                   depth=torch.empty(N, dtype=torch.int32, device=dev))
    _outputs(out, {"mask": ((N, W), torch.int32), "depth": ((N,), torch.int32)}, dev)
    status = _status(status, dev, s)
    out["status"] = status
    with torch.cuda.device(dev):
        st = lib.spec_tree_mask(_ptr(parents), N, _ptr(out["mask"]), _ptr(out["depth"]), _ptr(status), h)
    _check(st)
    return out


def spec_mtp_plug(in_tokens, out_tokens, num_emitted, pad=0, seq_lens=None, *, in_place=False, out=None,
                  status=None, stream=None):
    """The MTP draft layer's next input tokens [B, K+1]: in_tokens shifted left by one, with
    the verify's emitted tokens (out_tokens [B, K+1], num_emitted [B]) in their places and
    `pad` at the end; seq_lens [B] (int32, optional) grows by num_emitted in place.
    in_place=True writes into in_tokens.  Returns dict(next_tokens, seq_lens, status)."""
    lib = load_library()
    _cuda(in_tokens, "in_tokens", torch.int32)
    if in_tokens.dim() != 2:
        raise ValueError("in_tokens must be [B, K+1]")
    B, W = in_tokens.shape
    dev = in_tokens.device
    _cuda(out_tokens, "out_tokens", torch.int32, dev)
    _cuda(num_emitted, "num_emitted", torch.int32, dev)
    _cuda(seq_lens, "seq_lens", torch.int32, dev)
    if out_tokens is None or tuple(out_tokens.shape) != (B, W):
        raise ValueError("out_tokens must be [B, K+1]")
    if num_emitted is None or tuple(num_emitted.shape) != (B,):
        raise ValueError("num_emitted must be [B]")
    if seq_lens is not None and tuple(seq_lens.shape) != (B,):
        raise ValueError("seq_lens must be [B]")
    h, s = _stream_handle(dev, stream)
    if in_place:
        nxt = in_tokens
    else:
        nxt = out if out is not None else torch.empty((B, W), dtype=torch.int32, device=dev)
        _outputs(dict(next_tokens=nxt), {"next_tokens": ((B, W), torch.int32)}, dev)
    status = _status(status, dev, s)
    with torch.cuda.device(dev):
        st = lib.spec_mtp_plug(_ptr(in_tokens), B, W - 1, _ptr(out_tokens), _ptr(num_emitted), int(pad), _ptr(nxt),
                               _ptr(seq_lens), _ptr(status), h)
    _check(st)
    return dict(next_tokens=nxt, seq_lens=seq_lens, status=status)


def spec_build_sparse_tree(accuracy, n_nodes):
    """Greedy sparse candidate tree (host): accuracy [K, S] (a_k^(i) at [k-1, i-1], numpy or
    a CPU tensor, values in [0, 1]) and the node count wanted (root included).  Returns
    dict(parents, depth, rank) as int32 numpy arrays of the nodes built, and expected_len."""
    import numpy as np
    lib = load_library()
    acc = np.ascontiguousarray(np.asarray(accuracy, dtype=np.float64))
    if acc.ndim != 2:
        raise ValueError("accuracy must be [K, S]")
    K, S = acc.shape
    n = int(n_nodes)
    par, dep, rk = (np.zeros(max(n, 1), np.int32) for _ in range(3))
    nb, el = ctypes.c_int(0), ctypes.c_double(0.0)
    st = lib.spec_build_sparse_tree(acc.ctypes.data_as(ctypes.c_void_p), K, S, n,
                                    par.ctypes.data_as(ctypes.c_void_p), dep.ctypes.data_as(ctypes.c_void_p),
                                    rk.ctypes.data_as(ctypes.c_void_p), ctypes.byref(nb), ctypes.byref(el))
    _check(st)
    m = nb.value
    return dict(parents=par[:m].copy(), depth=dep[:m].copy(), rank=rk[:m].copy(), expected_len=el.value)
