"""Thin Python binding of ``include/gdn_tree.h`` and ``include/gdn_layer.h``:
argument marshalling only.

Every function has the name of the C entry point it calls.  Tensors are torch
tensors on the current CUDA device (torch provides memory and streams; every step of
the computation runs in the library's kernels).  The library is loaded on
first use from ``_build/libgdn_tree.so``; if it is missing the call raises,
there is no other implementation to fall back to.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

import torch

from . import build as _build

GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED = 0, 1, 2
GDN_ERR_INVALID_TREE, GDN_ERR_INVALID_PATH, GDN_ERR_CUDA, GDN_ERR_DEVICE = 3, 4, 5, 6
GDN_F32, GDN_BF16 = 0, 1
DEV_BITS = {1: "BAD_TREE", 2: "BAD_PATH", 4: "TOO_MANY", 8: "TOO_DEEP", 16: "TIMEOUT", 64: "INTERNAL",
            32: "BAD_DESC", 128: "BAD_SLOT"}
GDN_ACTS = {"silu": 0, "sigmoid": 1}

_P = ctypes.c_void_p
_I = ctypes.c_int32
_L = ctypes.c_int64
_F = ctypes.c_float


class VerifyArgs(ctypes.Structure):
    _fields_ = [("batch", _I), ("n_k_heads", _I), ("n_v_heads", _I), ("d_k", _I), ("d_v", _I),
                ("total_nodes", _I), ("max_nodes", _I), ("max_depth", _I), ("scale", ctypes.c_float),
                ("qkv_dtype", _I), ("out_dtype", _I), ("node_offsets", _P), ("q", _P), ("k", _P),
                ("v", _P), ("g", _P), ("beta", _P), ("S0", _P), ("parent", _P), ("anc_mask", _P),
                ("mask_words", _I), ("depth", _P), ("o", _P), ("dev_status", _P)]


class CommitArgs(ctypes.Structure):
    _fields_ = [("batch", _I), ("n_k_heads", _I), ("n_v_heads", _I), ("d_k", _I), ("d_v", _I),
                ("total_nodes", _I), ("max_nodes", _I), ("max_path", _I), ("qkv_dtype", _I),
                ("node_offsets", _P),
                ("k", _P), ("v", _P),
                ("g", _P), ("beta", _P), ("S0", _P), ("parent", _P), ("path_offsets", _P),
                ("path_idx", _P), ("S_new", _P), ("dev_status", _P)]


class StatesArgs(ctypes.Structure):
    _fields_ = [("batch", _I), ("n_k_heads", _I), ("n_v_heads", _I), ("d_k", _I), ("d_v", _I),
                ("total_nodes", _I), ("max_nodes", _I), ("qkv_dtype", _I),
                ("node_offsets", _P), ("k", _P), ("v", _P), ("g", _P), ("beta", _P), ("S0", _P),
                ("parent", _P), ("anc_mask", _P), ("mask_words", _I), ("n_sel", _I),
                ("sel_request", _P), ("sel_node", _P), ("S_sel", _P), ("dev_status", _P)]


class PrefillArgs(ctypes.Structure):
    _fields_ = [("batch", _I), ("n_k_heads", _I), ("n_v_heads", _I), ("d_k", _I), ("d_v", _I),
                ("total_tokens", _I), ("max_tokens", _I), ("n_states", _I), ("scale", _F), ("qkv_dtype", _I),
                ("out_dtype", _I), ("q_stride", _L), ("k_stride", _L), ("v_stride", _L), ("token_offsets", _P),
                ("q", _P), ("k", _P), ("v", _P), ("g", _P), ("beta", _P), ("S0", _P), ("slots", _P),
                ("fresh", _P), ("o", _P), ("S_new", _P), ("workspace", _P), ("workspace_bytes", _L),
                ("dev_status", _P)]


class DecodeArgs(ctypes.Structure):
    _fields_ = [("batch", _I), ("n_k_heads", _I), ("n_v_heads", _I), ("d_k", _I), ("d_v", _I), ("n_states", _I),
                ("scale", _F), ("qkv_dtype", _I), ("out_dtype", _I), ("q_stride", _L), ("k_stride", _L),
                ("v_stride", _L), ("q", _P), ("k", _P), ("v", _P), ("g", _P), ("beta", _P), ("S", _P),
                ("slots", _P), ("o", _P), ("dev_status", _P)]


class QkGatesArgs(ctypes.Structure):
    _fields_ = [("total_tokens", _I), ("n_k_heads", _I), ("n_v_heads", _I), ("d_k", _I), ("eps", _F),
                ("dtype", _I), ("q_stride", _L), ("k_stride", _L), ("a_stride", _L), ("b_stride", _L), ("q", _P),
                ("k", _P), ("a", _P), ("b", _P), ("A_log", _P), ("dt_bias", _P), ("q_out", _P), ("k_out", _P),
                ("g", _P), ("beta", _P)]


class NormGateArgs(ctypes.Structure):
    _fields_ = [("total_tokens", _I), ("n_v_heads", _I), ("d_v", _I), ("eps", _F), ("act", _I), ("dtype", _I),
                ("weight_dtype", _I), ("o_stride", _L), ("z_stride", _L), ("o", _P), ("z", _P), ("weight", _P),
                ("y", _P)]


class ResidualNormArgs(ctypes.Structure):
    _fields_ = [("total_tokens", _I), ("width", _I), ("scale", _F), ("eps", _F), ("dtype", _I),
                ("weight_dtype", _I), ("x_stride", _L), ("y_stride", _L), ("x", _P), ("y", _P), ("weight", _P),
                ("post_weight", _P), ("h", _P), ("n", _P)]


class GdnError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"gdn status {code}: {msg}")
        self.code = code


class GdnDeviceError(RuntimeError):
    def __init__(self, bits: int):
        names = [n for b, n in DEV_BITS.items() if bits & b]
        super().__init__(f"device status {bits} ({', '.join(names)})")
        self.bits = bits


_lib = None


def lib_path() -> str:
    return _build.LIB


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with gated_delta_net_gb300.build.build()")
        L = ctypes.CDLL(path)
        L.gdn_tree_build_desc.argtypes = [_P, _P, _I, _I, _P, _I, _P, _P, _P]
        L.gdn_tree_build_desc.restype = ctypes.c_int
        for fn in (L.gdn_tree_verify, L.gdn_tree_verify_branches):
            fn.argtypes = [ctypes.POINTER(VerifyArgs), _P]
            fn.restype = ctypes.c_int
        L.gdn_tree_commit.argtypes = [ctypes.POINTER(CommitArgs), _P]
        L.gdn_tree_commit.restype = ctypes.c_int
        L.gdn_tree_commit_verify.argtypes = [ctypes.POINTER(CommitArgs), ctypes.POINTER(VerifyArgs), _P]
        L.gdn_tree_commit_verify.restype = ctypes.c_int
        L.gdn_tree_states.argtypes = [ctypes.POINTER(StatesArgs), _P]
        L.gdn_tree_states.restype = ctypes.c_int
        L.gdn_tree_grow.argtypes = [_P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P]
        L.gdn_tree_grow.restype = ctypes.c_int
        L.gdn_tree_relabel.argtypes = [_P, _P, _I, _I, _I, _P, _P, _P, _P, _P]
        L.gdn_tree_relabel.restype = ctypes.c_int
        L.gdn_gather_rows.argtypes = [_P, _P, _P, _P, _I, _I, ctypes.c_int64, _P, _P]
        L.gdn_gather_rows.restype = ctypes.c_int
        for fn in (L.gdn_prefill, L.gdn_decode, L.gdn_qk_gates, L.gdn_norm_gate, L.gdn_residual_norm):
            fn.argtypes = [_P, _P]
            fn.restype = ctypes.c_int
        L.gdn_prefill_workspace.argtypes = [_P]
        L.gdn_prefill_workspace.restype = _L
        L.gdn_last_error.restype = ctypes.c_char_p
        L.gdn_tree_version.restype = ctypes.c_int
        L.gdn_test_set_wait_probe.argtypes = [_I]
        L.gdn_test_set_wait_probe.restype = None
        _lib = L
    return _lib


def _check(code: int):
    if code != GDN_OK:
        raise GdnError(code, lib().gdn_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:  # the handle without its object
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()))
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _here() -> int:
    """The current device, where kernels are launched (-1: there is none)."""
    try:
        return torch._C._cuda_getDevice()
    except RuntimeError:
        return -1


def _dev(t: torch.Tensor, name: str, here: int, dtype=None) -> torch.Tensor:
    at = t.get_device() if isinstance(t, torch.Tensor) else -1
    if at < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    if at != here:
        raise ValueError(f"{name} is on cuda:{at}, which is not the current device")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _status_ptr(t: Optional[torch.Tensor], here: int):
    return None if t is None else _ptr(_dev(t, "dev_status", here))


def _code(dtype: torch.dtype) -> int:
    if dtype == torch.float32:
        return GDN_F32
    if dtype == torch.bfloat16:
        return GDN_BF16
    raise TypeError(f"unsupported dtype {dtype}")


def _on(stream, device):
    """``stream`` (torch's, or a handle) as one that torch can allocate for.  The handles 0 to 2 are the default
    stream's names; the one for each thread (2) is ordered with it."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return torch.cuda.default_stream(device) if handle <= 2 else torch.cuda.ExternalStream(handle, device=device)


def _scratch(shape, dtype, device, stream, zero: bool = False) -> torch.Tensor:
    """Memory that only a launch on ``stream`` (None: the current one) uses.  It is allocated for that stream:
    a block of another one's may still be in use there by what that stream has yet to do."""
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_on(stream, device)):
        return make(shape, dtype=dtype, device=device)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """Memory for a result of a launch on ``stream``: as above, and recorded on the current stream, where the
    caller may use it after a wait of its own."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    t = _scratch(shape, dtype, device, stream)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def gdn_test_set_wait_probe(polls: int) -> None:
    """Test hook: later tensor-core verify/commit launches make one bounded wait of
    ``polls`` polls that runs out (GDN_DEV_TIMEOUT); 0 turns it off."""
    lib().gdn_test_set_wait_probe(int(polls))


def new_status(device=None) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def check_status(dev_status: torch.Tensor):
    """Synchronise on the status word and raise GdnDeviceError if any bit is set."""
    bits = int(dev_status.item())
    if bits:
        raise GdnDeviceError(bits)


def gdn_tree_build_desc(parent: torch.Tensor, node_offsets: torch.Tensor, max_nodes: int,
                        anc_mask: Optional[torch.Tensor] = None,
                        depth: Optional[torch.Tensor] = None, mask_words: Optional[int] = None,
                        dev_status: Optional[torch.Tensor] = None, stream=None):
    """Ancestor bitmask [T, mask_words] (int32 storage of uint32 words) and depth [T]."""
    here = _here()
    _dev(parent, "parent", here, torch.int32)
    _dev(node_offsets, "node_offsets", here, torch.int32)
    T = parent.numel()
    words = mask_words or max(1, (max_nodes + 31) // 32)
    if anc_mask is None:
        anc_mask = _empty((T, words), torch.int32, parent.device, stream)
    if depth is None:
        depth = _empty(T, torch.int32, parent.device, stream)
    _dev(anc_mask, "anc_mask", here, torch.int32)
    _dev(depth, "depth", here, torch.int32)
    if anc_mask.shape != (T, words) or depth.numel() != T:
        raise ValueError("anc_mask must be [T, mask_words] and depth [T]")
    _check(lib().gdn_tree_build_desc(_ptr(parent), _ptr(node_offsets), node_offsets.numel() - 1,
                                     int(max_nodes), _ptr(anc_mask), words, _ptr(depth),
                                     _status_ptr(dev_status, here), _stream(stream)))
    return anc_mask, depth


def gdn_tree_states(k, v, g, beta, S0, node_offsets, parent, anc_mask, sel_request, sel_node,
                    max_nodes: int, out=None, dev_status=None, stream=None) -> torch.Tensor:
    """The state at each selected node [n_sel, Hv, d_v, d_k] (fp32)."""
    here = _here()
    for name, t in (("k", k), ("v", v)):
        _dev(t, name, here)
    for name, t in (("g", g), ("beta", beta), ("S0", S0)):
        _dev(t, name, here, torch.float32)
    for name, t in (("node_offsets", node_offsets), ("parent", parent), ("anc_mask", anc_mask),
                    ("sel_request", sel_request), ("sel_node", sel_node)):
        _dev(t, name, here, torch.int32)
    T, Hk, dk = k.shape
    Hv, dv = v.shape[1], v.shape[2]
    B = node_offsets.numel() - 1
    n_sel = sel_request.numel()
    if sel_node.numel() != n_sel or S0.shape != (B, Hv, dv, dk):
        raise ValueError("inconsistent selection / S0 shapes")
    if out is None:
        out = _empty((n_sel, Hv, dv, dk), torch.float32, S0.device, stream)
    _dev(out, "out", here, torch.float32)
    if out.shape != (n_sel, Hv, dv, dk):
        raise ValueError("out must be [n_sel, Hv, d_v, d_k]")
    a = StatesArgs(B, Hk, Hv, dk, dv, T, int(max_nodes), _code(k.dtype), _ptr(node_offsets), _ptr(k),
                   _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(parent), _ptr(anc_mask),
                   anc_mask.shape[1] if anc_mask.dim() == 2 else 1, n_sel, _ptr(sel_request),
                   _ptr(sel_node), _ptr(out), _status_ptr(dev_status, here))
    _check(lib().gdn_tree_states(ctypes.byref(a), _stream(stream)))
    return out


def gdn_tree_grow(node_offsets: torch.Tensor, n_children: torch.Tensor, draws: torch.Tensor,
                  width: int, max_depth: int = 16, dev_status=None, stream=None):
    """Top-w best-first trees: (parent [T] int32, score [T] float32, n_nodes [B] int32)."""
    here = _here()
    _dev(node_offsets, "node_offsets", here, torch.int32)
    _dev(n_children, "n_children", here, torch.int32)
    _dev(draws, "draws", here, torch.float32)
    T = n_children.numel()
    if draws.dim() != 2 or draws.shape[0] != T or not draws.is_contiguous():
        raise ValueError("draws must be a contiguous [T, max_children] tensor")
    B = node_offsets.numel() - 1
    parent = _empty(T, torch.int32, draws.device, stream)
    score = _empty(T, torch.float32, draws.device, stream)
    n_nodes = _empty(B, torch.int32, draws.device, stream)
    _check(lib().gdn_tree_grow(_ptr(node_offsets), B, T, int(width), int(max_depth), draws.shape[1],
                               _ptr(n_children), _ptr(draws), _ptr(parent), _ptr(score), _ptr(n_nodes),
                               _status_ptr(dev_status, here), _stream(stream)))
    return parent, score, n_nodes


def gdn_tree_relabel(parent: torch.Tensor, node_offsets: torch.Tensor, max_nodes: int,
                     dev_status: Optional[torch.Tensor] = None, stream=None):
    """Topological relabelling by (depth, old id): (order, rank, parent_out), each [T] int32
    with request-local ids."""
    here = _here()
    _dev(parent, "parent", here, torch.int32)
    _dev(node_offsets, "node_offsets", here, torch.int32)
    T = parent.numel()
    order = _empty(T, torch.int32, parent.device, stream)
    rank = _empty(T, torch.int32, parent.device, stream)
    parent_out = _empty(T, torch.int32, parent.device, stream)
    _check(lib().gdn_tree_relabel(_ptr(parent), _ptr(node_offsets), node_offsets.numel() - 1, T,
                                  int(max_nodes), _ptr(order), _ptr(rank), _ptr(parent_out),
                                  _status_ptr(dev_status, here), _stream(stream)))
    return order, rank, parent_out


def gdn_gather_rows(src: torch.Tensor, index: torch.Tensor, node_offsets: torch.Tensor,
                    out: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """Rows permuted within each request: out[lo + j] = src[lo + index[lo + j]]."""
    here = _here()
    _dev(src, "src", here)
    _dev(index, "index", here, torch.int32)
    _dev(node_offsets, "node_offsets", here, torch.int32)
    if not src.is_contiguous():
        raise ValueError("src must be contiguous")
    T = src.shape[0]
    if index.numel() != T:
        raise ValueError("index must have one entry per row")
    if out is None:
        out = _empty(src.shape, src.dtype, src.device, stream)
    _dev(out, "out", here, src.dtype)
    if out.shape != src.shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor shaped like src")
    row_bytes = src[0].numel() * src.element_size() if T else 16
    _check(lib().gdn_gather_rows(_ptr(src), _ptr(out), _ptr(index), _ptr(node_offsets),
                                 node_offsets.numel() - 1, T, row_bytes, _status_ptr(dev_status, here),
                                 _stream(stream)))
    return out


def _verify_args(q, k, v, g, beta, S0, node_offsets, parent, anc_mask, depth, max_nodes,
                 max_depth, scale, out, out_dtype, dev_status, stream):
    here = _here()
    for name, t in (("q", q), ("k", k), ("v", v)):
        _dev(t, name, here)
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share a dtype")
    for name, t in (("g", g), ("beta", beta), ("S0", S0)):
        _dev(t, name, here, torch.float32)
    for name, t in (("node_offsets", node_offsets), ("parent", parent), ("anc_mask", anc_mask),
                    ("depth", depth)):
        _dev(t, name, here, torch.int32)
    T, Hk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    B = node_offsets.numel() - 1
    if k.shape != q.shape or v.shape[0] != T or g.shape != (T, Hv) or beta.shape != (T, Hv):
        raise ValueError("inconsistent token shapes")
    if S0.shape != (B, Hv, dv, dk) or parent.numel() != T or depth.numel() != T:
        raise ValueError("inconsistent S0 / tree shapes")
    od = out_dtype or q.dtype
    if out is None:
        out = _empty((T, Hv, dv), od, q.device, stream)
    _dev(out, "out", here, od)
    if out.shape != (T, Hv, dv):
        raise ValueError("out must be [T, Hv, d_v]")
    a = VerifyArgs(B, Hk, Hv, dk, dv, T, int(max_nodes), int(max_depth), float(scale), _code(q.dtype),
                   _code(od), _ptr(node_offsets), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                   _ptr(S0), _ptr(parent), _ptr(anc_mask), anc_mask.shape[1] if anc_mask.dim() == 2 else 1,
                   _ptr(depth), _ptr(out), _status_ptr(dev_status, here))
    return a, out


def gdn_tree_verify(q, k, v, g, beta, S0, node_offsets, parent, anc_mask, depth, max_nodes: int,
                    max_depth: int = 0, scale: float = 1.0, out=None, out_dtype=None,
                    dev_status=None, stream=None) -> torch.Tensor:
    """Every node's output o [T, Hv, d_v]; S0 is only read."""
    a, out = _verify_args(q, k, v, g, beta, S0, node_offsets, parent, anc_mask, depth, max_nodes,
                          max_depth, scale, out, out_dtype, dev_status, stream)
    _check(lib().gdn_tree_verify(ctypes.byref(a), _stream(stream)))
    return out


def gdn_tree_verify_branches(q, k, v, g, beta, S0, node_offsets, parent, anc_mask, depth,
                             max_nodes: int, max_depth: int = 0, scale: float = 1.0, out=None,
                             out_dtype=None, dev_status=None, stream=None) -> torch.Tensor:
    """Per-branch recurrent baseline; same results as gdn_tree_verify up to rounding."""
    a, out = _verify_args(q, k, v, g, beta, S0, node_offsets, parent, anc_mask, depth, max_nodes,
                          max_depth, scale, out, out_dtype, dev_status, stream)
    _check(lib().gdn_tree_verify_branches(ctypes.byref(a), _stream(stream)))
    return out


def _commit_args(k, v, g, beta, S0, node_offsets, parent, path_offsets, path_idx, max_nodes,
                 max_path, out, dev_status, stream):
    here = _here()
    for name, t in (("k", k), ("v", v)):
        _dev(t, name, here)
    for name, t in (("g", g), ("beta", beta), ("S0", S0)):
        _dev(t, name, here, torch.float32)
    for name, t in (("node_offsets", node_offsets), ("parent", parent),
                    ("path_offsets", path_offsets), ("path_idx", path_idx)):
        _dev(t, name, here, torch.int32)
    T, Hk, dk = k.shape
    Hv, dv = v.shape[1], v.shape[2]
    B = node_offsets.numel() - 1
    if S0.shape != (B, Hv, dv, dk) or path_offsets.numel() != B + 1:
        raise ValueError("inconsistent S0 / path shapes")
    if out is None:
        out = _empty(S0.shape, torch.float32, S0.device, stream)
    _dev(out, "out", here, torch.float32)
    if out.shape != S0.shape:
        raise ValueError("out must match S0")
    pidx = path_idx if path_idx.numel() else _scratch(1, torch.int32, k.device, stream, zero=True)
    a = CommitArgs(B, Hk, Hv, dk, dv, T, int(max_nodes), int(max_path), _code(k.dtype),
                   _ptr(node_offsets), _ptr(k),
                   _ptr(v), _ptr(g), _ptr(beta), _ptr(S0), _ptr(parent), _ptr(path_offsets),
                   _ptr(pidx), _ptr(out), _status_ptr(dev_status, here))
    return a, out, pidx


def gdn_tree_commit(k, v, g, beta, S0, node_offsets, parent, path_offsets, path_idx,
                    max_nodes: int, max_path: int = 0, out=None, dev_status=None,
                    stream=None) -> torch.Tensor:
    """State after each request's accepted path [B, Hv, d_v, d_k]; ``out`` may be ``S0``."""
    a, out, _keep = _commit_args(k, v, g, beta, S0, node_offsets, parent, path_offsets, path_idx,
                                 max_nodes, max_path, out, dev_status, stream)
    _check(lib().gdn_tree_commit(ctypes.byref(a), _stream(stream)))
    return out


def gdn_tree_commit_verify(prev: dict, S0, max_nodes_prev: int, max_path: int,
                           q, k, v, g, beta, node_offsets, parent, anc_mask, depth, max_nodes: int,
                           max_depth: int = 16, scale: float = 1.0, S_new=None, out=None,
                           out_dtype=None, dev_status=None, stream=None):
    """Commit S0 along the previous tree's accepted path (``prev``: k, v, g, beta,
    node_offsets, parent, path_offsets, path_idx), write it to ``S_new`` (may be
    ``S0``), and verify the new tree from it.  Returns (o, S_new)."""
    c, S_new, _keep = _commit_args(prev["k"], prev["v"], prev["g"], prev["beta"], S0,
                                   prev["node_offsets"], prev["parent"], prev["path_offsets"],
                                   prev["path_idx"], max_nodes_prev, max_path, S_new, dev_status, stream)
    a, out = _verify_args(q, k, v, g, beta, S_new, node_offsets, parent, anc_mask, depth, max_nodes,
                          max_depth, scale, out, out_dtype, dev_status, stream)
    _check(lib().gdn_tree_commit_verify(ctypes.byref(c), ctypes.byref(a), _stream(stream)))
    return out, S_new


# ----------------------------------------------------------------------------
# the layer around the tree (gdn_layer.h)
# ----------------------------------------------------------------------------

# These calls serve single tokens, where the host's time counts: one pass over each tensor's
# attributes and none over the outputs made here, pointers as plain integers, the current stream's
# handle without its object, the arguments packed in one go (0.3 us against the Structure's 0.8).

_FORMATS = {_I: "i", _F: "f", _L: "q", _P: "P"}


def _packer(args):
    """What lays the values of a Structure's fields out as the Structure does."""
    return struct.Struct("@" + "".join(_FORMATS[kind] for _, kind in args._fields_)).pack


_prefill_args, _decode_args, _qk_gates_args, _norm_gate_args, _residual_norm_args = map(
    _packer, (PrefillArgs, DecodeArgs, QkGatesArgs, NormGateArgs, ResidualNormArgs))


def _device(t, name: str) -> int:
    """The device of a call's first tensor.  It has to be the current one, where kernels are launched, and all
    other tensors have to be there as well."""
    dev = t.get_device()
    if dev < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on cuda:{dev}, which is not the current device")
    return dev


def _rows(t: torch.Tensor, name: str, dtype, shape, dev: int) -> int:
    """The distance between the tokens of ``t`` in elements (0: contiguous), after a check of its
    type, shape and device; its other dimensions are contiguous."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
            if t.is_contiguous():
                return 0
            stride = t.stride()
            if len(shape) == 3:
                if stride[2] == 1 and stride[1] == shape[2] and stride[0] >= shape[1] * shape[2]:
                    return stride[0]
            elif stride[1] == 1 and stride[0] >= shape[1]:
                return stride[0]
            row = 1  # sizes of one, whose strides do not count, or a mistake
            for n, st in zip(reversed(shape[1:]), reversed(stride[1:])):
                if st != row and n != 1:
                    raise ValueError(f"{name} must be contiguous inside a token")
                row *= n
            if stride[0] < row:
                raise ValueError(f"the tokens of {name} overlap")
            return stride[0]
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, dev)


def _flat(t: torch.Tensor, name: str, dtype, shape, dev: int) -> int:
    """The address of ``t`` after a check of its type, shape and device; contiguous."""
    try:
        if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev:
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, dev)


def _refuse(t, name: str, dtype, shape, dev: int):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the first tensor on cuda:{dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be a contiguous {list(shape)} tensor, got {list(t.shape)}")


def _handle(stream, dev: int) -> int:
    """The handle of ``stream``, or of the current stream of device ``dev``."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _status(t: Optional[torch.Tensor], dev: int) -> int:
    return 0 if t is None else _flat(t, "dev_status", torch.int32, t.shape, dev)


_CODES = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}


def _dtype_code(dtype) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def gdn_prefill(q, k, v, g, beta, token_offsets, max_tokens: int, S0=None, slots=None, fresh=None,
                scale: float = 1.0, S_new=None, out=None, out_dtype=None, workspace=None, dev_status=None,
                stream=None):
    """Prompts, packed: (o [T, Hv, d_v], S_new).  Prompt b is rows token_offsets[b] to
    token_offsets[b + 1] of q, k [T, Hk, d_k], v [T, Hv, d_v] (tokens may be strided) and of
    g, beta [T, Hv]; max_tokens bounds its length.  Its state is row slots[b] (or b) of the pools
    S0 (None: zero; a prompt with fresh[b] != 0 starts from zero too) and S_new (may be S0).
    bf16 in and out with heads of 128 take the chunked kernel; other types and widths, out_dtype=float32
    among them, the recurrent one: fp32 arithmetic, about ten times as long."""
    T, Hk, dk = q.shape
    _, Hv, dv = v.shape
    dt, dev = q.dtype, _device(q, "q")
    od = out_dtype or dt
    code, out_code = _dtype_code(dt), _dtype_code(od)
    qs, ks, vs = _rows(q, "q", dt, (T, Hk, dk), dev), _rows(k, "k", dt, (T, Hk, dk), dev), _rows(v, "v", dt, (T, Hv, dv), dev)
    gp, bp = _flat(g, "g", torch.float32, (T, Hv), dev), _flat(beta, "beta", torch.float32, (T, Hv), dev)
    B = token_offsets.numel() - 1
    op = _flat(token_offsets, "token_offsets", torch.int32, (B + 1,), dev)
    sp = 0 if slots is None else _flat(slots, "slots", torch.int32, (B,), dev)
    fp = 0 if fresh is None else _flat(fresh, "fresh", torch.int32, (B,), dev)
    if S_new is None:
        if slots is not None:
            raise ValueError("slots need S_new: the pool that they point into")
        S_new = _empty((B, Hv, dv, dk), torch.float32, q.device, stream)
    n_states = S_new.shape[0]
    if slots is None and n_states < B:
        raise ValueError("the pool has fewer states than there are prompts")
    np_ = _flat(S_new, "S_new", torch.float32, (n_states, Hv, dv, dk), dev)
    s0 = 0 if S0 is None else _flat(S0, "S0", torch.float32, (n_states, Hv, dv, dk), dev)
    if out is None:
        out = _empty((T, Hv, dv), od, q.device, stream)
        outp = out.data_ptr()
    else:
        outp = _flat(out, "out", od, (T, Hv, dv), dev)
    a = (B, Hk, Hv, dk, dv, T, max_tokens, n_states, scale, code, out_code, qs, ks, vs, op, q.data_ptr(), k.data_ptr(),
         v.data_ptr(), gp, bp, s0, sp, fp, outp, np_)
    st, stream_handle, L = _status(dev_status, dev), _handle(stream, dev), lib()
    packed = None
    if workspace is None:
        packed = _prefill_args(*a, 0, 0, st)
        need = L.gdn_prefill_workspace(packed)
        if need > 0:
            workspace = _scratch(need, torch.uint8, q.device, stream)
    if workspace is not None:
        packed = _prefill_args(*a, _flat(workspace, "workspace", torch.uint8, workspace.shape, dev), workspace.numel(), st)
    _check(L.gdn_prefill(packed, stream_handle))
    return out, S_new


def gdn_prefill_workspace(batch: int, n_k_heads: int, n_v_heads: int, d_k: int, d_v: int, total_tokens: int,
                          max_tokens: int, dtype=torch.bfloat16, out_dtype=None) -> int:
    """Bytes of ``workspace`` with which gdn_prefill takes these sizes (it allocates its own otherwise)."""
    a = PrefillArgs(batch, n_k_heads, n_v_heads, d_k, d_v, total_tokens, max_tokens, batch, 1.0, _dtype_code(dtype),
                    _dtype_code(out_dtype or dtype))
    need = lib().gdn_prefill_workspace(ctypes.byref(a))
    if need < 0:
        _check(GDN_ERR_INVALID_ARG)
    return need


def gdn_decode(q, k, v, g, beta, S, slots=None, scale: float = 1.0, out=None, out_dtype=None, dev_status=None,
               stream=None) -> torch.Tensor:
    """One token a request: o [B, Hv, d_v]; state slots[b] (or b) of the pool S is updated in place.
    A row whose slot is -1 is not in use: its outputs are zero."""
    B, Hk, dk = q.shape
    _, Hv, dv = v.shape
    dt, dev = q.dtype, _device(q, "q")
    od = out_dtype or dt
    code, out_code = _dtype_code(dt), _dtype_code(od)
    qs, ks, vs = _rows(q, "q", dt, (B, Hk, dk), dev), _rows(k, "k", dt, (B, Hk, dk), dev), _rows(v, "v", dt, (B, Hv, dv), dev)
    gp, bp = _flat(g, "g", torch.float32, (B, Hv), dev), _flat(beta, "beta", torch.float32, (B, Hv), dev)
    n_states = S.shape[0]
    Sp = _flat(S, "S", torch.float32, (n_states, Hv, dv, dk), dev)
    sp = 0 if slots is None else _flat(slots, "slots", torch.int32, (B,), dev)
    if slots is None and n_states < B:
        raise ValueError("the pool has fewer states than there are requests")
    if out is None:
        out = _empty((B, Hv, dv), od, q.device, stream)
        outp = out.data_ptr()
    else:
        outp = _flat(out, "out", od, (B, Hv, dv), dev)
    _check(lib().gdn_decode(
        _decode_args(B, Hk, Hv, dk, dv, n_states, scale, code, out_code, qs, ks, vs, q.data_ptr(), k.data_ptr(),
                     v.data_ptr(), gp, bp, Sp, sp, outp, _status(dev_status, dev)), _handle(stream, dev)))
    return out


def gdn_qk_gates(q, k, a, b, A_log, dt_bias, eps: float = 1e-6, q_out=None, k_out=None, stream=None):
    """Before the rule: (q, k of unit length per head, g [T, Hv], beta [T, Hv]) from a layer's
    projections q, k [T, Hk, d_k] and a, b [T, Hv] (tokens may be strided) and its A_log, dt_bias [Hv]."""
    T, Hk, dk = q.shape
    _, Hv = a.shape
    dt, dev = q.dtype, _device(q, "q")
    code = _dtype_code(dt)
    qs, ks = _rows(q, "q", dt, (T, Hk, dk), dev), _rows(k, "k", dt, (T, Hk, dk), dev)
    as_, bs = _rows(a, "a", dt, (T, Hv), dev), _rows(b, "b", dt, (T, Hv), dev)
    Ap, dp = _flat(A_log, "A_log", torch.float32, (Hv,), dev), _flat(dt_bias, "dt_bias", torch.float32, (Hv,), dev)
    if q_out is None:
        q_out = _empty((T, Hk, dk), dt, q.device, stream)
        qp = q_out.data_ptr()
    else:
        qp = _flat(q_out, "q_out", dt, (T, Hk, dk), dev)
    if k_out is None:
        k_out = _empty((T, Hk, dk), dt, q.device, stream)
        kp = k_out.data_ptr()
    else:
        kp = _flat(k_out, "k_out", dt, (T, Hk, dk), dev)
    g = _empty((T, Hv), torch.float32, q.device, stream)
    beta = _empty((T, Hv), torch.float32, q.device, stream)
    _check(lib().gdn_qk_gates(
        _qk_gates_args(T, Hk, Hv, dk, eps, code, qs, ks, as_, bs, q.data_ptr(), k.data_ptr(), a.data_ptr(),
                       b.data_ptr(), Ap, dp, qp, kp, g.data_ptr(), beta.data_ptr()), _handle(stream, dev)))
    return q_out, k_out, g, beta


def gdn_norm_gate(o, z, weight, eps: float = 1e-6, act: str = "silu", out=None, stream=None) -> torch.Tensor:
    """After the rule: o [T, Hv, d_v] normed per head, times weight [d_v] and act(z) (silu or sigmoid)."""
    T, Hv, dv = o.shape
    dt, dev = o.dtype, _device(o, "o")
    os_, zs = _rows(o, "o", dt, (T, Hv, dv), dev), _rows(z, "z", dt, (T, Hv, dv), dev)
    kind = GDN_ACTS.get(act)
    if kind is None:
        raise ValueError(f"act must be one of {sorted(GDN_ACTS)}, got {act!r}")
    if out is None:
        out = _empty((T, Hv, dv), dt, o.device, stream)
        outp = out.data_ptr()
    else:
        outp = _flat(out, "out", dt, (T, Hv, dv), dev)
    _check(lib().gdn_norm_gate(
        _norm_gate_args(T, Hv, dv, eps, kind, _dtype_code(dt), _dtype_code(weight.dtype), os_, zs, o.data_ptr(),
                        z.data_ptr(), _flat(weight, "weight", weight.dtype, (dv,), dev), outp), _handle(stream, dev)))
    return out


def gdn_residual_norm(x, y, weight, scale: float = 1.0, post_weight=None, eps: float = 1e-6, h=None, out=None,
                      stream=None):
    """Between two blocks: (h, n) with h = x + scale * y (y normed first where post_weight is given)
    and n = h normed, times weight; x, y [T, width] (tokens may be strided)."""
    T, D = x.shape
    dt, dev = x.dtype, _device(x, "x")
    xs, ys = _rows(x, "x", dt, (T, D), dev), _rows(y, "y", dt, (T, D), dev)
    wp = _flat(weight, "weight", weight.dtype, (D,), dev)
    pp = 0 if post_weight is None else _flat(post_weight, "post_weight", weight.dtype, (D,), dev)
    if h is None:
        h = _empty((T, D), dt, x.device, stream)
        hp = h.data_ptr()
    else:
        hp = _flat(h, "h", dt, (T, D), dev)
    if out is None:
        out = _empty((T, D), dt, x.device, stream)
        outp = out.data_ptr()
    else:
        outp = _flat(out, "out", dt, (T, D), dev)
    _check(lib().gdn_residual_norm(
        _residual_norm_args(T, D, scale, eps, _dtype_code(dt), _dtype_code(weight.dtype), xs, ys, x.data_ptr(),
                            y.data_ptr(), wp, pp, hp, outp), _handle(stream, dev)))
    return h, out


# ----------------------------------------------------------------------------
# upload of a seeded workload (marshalling only)
# ----------------------------------------------------------------------------

def upload(tb, device="cuda", pin: bool = False) -> dict:
    """Copy a ``workloads.TreeBatch`` into tensors (device, or pinned host if ``pin``)."""
    qdt = torch.bfloat16 if tb.qkv_dtype == "bf16" else torch.float32

    def put(x, dtype):
        t = torch.from_numpy(x).to(dtype)
        if pin:
            return t.pin_memory()
        return t.to(device)

    return {
        "q": put(tb.q, qdt), "k": put(tb.k, qdt), "v": put(tb.v, qdt),
        "g": put(tb.g, torch.float32), "beta": put(tb.beta, torch.float32),
        "S0": put(tb.S0, torch.float32),
        "node_offsets": put(tb.node_offsets, torch.int32), "parent": put(tb.parent, torch.int32),
        "path_offsets": put(tb.path_offsets, torch.int32),
        "path_idx": put(tb.path_idx if len(tb.path_idx) else tb.path_idx.reshape(0), torch.int32),
    }
