"""Thin ctypes binding over libvsa.so (the C ABI declared in include/vsa.h).

Argument marshalling only: torch allocates device memory for outputs and
workspaces and supplies the current CUDA stream; every step of the VSA
forward runs in the library's CUDA kernels.  There is no CPU fallback: if the
shared library is missing or a call fails, these functions raise.
"""

from __future__ import annotations

import array
import ctypes
import math
import os
import struct

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libvsa.so")

VSA_OK = 0
VSA_MAX_BLOCKS = 2048
STATUS_NAMES = {
    0: "VSA_OK", 1: "VSA_ERR_INVALID_ARG", 2: "VSA_ERR_SHAPE", 3: "VSA_ERR_UNSUPPORTED",
    4: "VSA_ERR_CUDA", 5: "VSA_ERR_DEVICE_TIMEOUT", 6: "VSA_ERR_INDEX_RANGE",
    7: "VSA_ERR_WORKSPACE", 8: "VSA_ERR_BLOCK_SIZE",
}

_c_void_p = ctypes.c_void_p
_c_int = ctypes.c_int
_c_int64 = ctypes.c_int64
_c_size_t = ctypes.c_size_t
_c_float = ctypes.c_float
_P32 = ctypes.POINTER(ctypes.c_int32)
_P64 = ctypes.POINTER(ctypes.c_int64)


class VsaStrides(ctypes.Structure):
    """vsa_strides: element strides over (batch, head, sequence slot)."""
    _fields_ = [("batch", ctypes.c_int64), ("head", ctypes.c_int64), ("seq", ctypes.c_int64)]


class VsaLayout(ctypes.Structure):
    """vsa_layout: the strides of q, k, v, out and the gate of one call."""
    _fields_ = [("q", VsaStrides), ("k", VsaStrides), ("v", VsaStrides), ("out", VsaStrides),
                ("gate", VsaStrides)]


class VsaDenseLayout(ctypes.Structure):
    """vsa_dense_layout: the strides of the [H, rows, D] views of one dense call."""
    _fields_ = [(n, VsaStrides) for n in ("q", "k", "v", "out", "dout", "dq", "dk", "dv")]


class VsaPrefixLayout(ctypes.Structure):
    """vsa_prefix_layout: the strides of one shared_prefix_attn call."""
    _fields_ = [(n, VsaStrides) for n in ("q", "out", "k_prefix", "v_prefix", "k_suffix", "v_suffix")]


_PL = ctypes.POINTER(VsaLayout)
VSA_LAYOUT_BHSD, VSA_LAYOUT_BSHD = 0, 1

# name -> (restype, argtypes); mirrors include/vsa.h
SIGNATURES = {
    "vsa_status_string": (ctypes.c_char_p, [_c_int]),
    "vsa_abi_version": (_c_int, []),
    "vsa_get_device_status": (_c_int, [_c_void_p]),
    "vsa_forward_workspace_size": (_c_size_t, [_c_int] * 5),
    "vsa_forward": (_c_int, [_c_void_p] * 4 + [_c_void_p, _c_void_p] + [_c_int] * 6 +
                    [_c_float, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_void_p,
                     _c_size_t, _c_void_p]),
    "vsa_make_layout": (_c_int, [_c_int] * 6 + [_PL]),
    "vsa_forward_strided": (_c_int, [_c_void_p] * 4 + [_PL, _c_void_p, _c_void_p] + [_c_int] * 7 +
                            [_c_float, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_void_p,
                             _c_void_p, _c_size_t, _c_void_p]),
    "vsa_forward_bshd": (_c_int, [_c_void_p] * 4 + [_c_void_p, _c_void_p] + [_c_int] * 6 +
                         [_c_float, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_void_p,
                          _c_size_t, _c_void_p]),
    "vsa_forward_noalloc": (_c_int, [_c_void_p] * 4 + [_c_void_p, _c_void_p] + [_c_int] * 6 +
                            [_c_float, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_void_p,
                             _c_void_p]),
    "vsa_forward_host_workspace_size": (_c_size_t, [_c_int] * 8),
    "vsa_forward_host": (_c_int, [_c_void_p] * 4 + [_c_void_p, _c_void_p] + [_c_int] * 6 +
                         [_c_float, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_void_p, _c_int,
                          _c_void_p, _c_size_t, _c_void_p]),
    "block_sparse_attn_from_indices_workspace_size": (_c_size_t, [_c_int] * 4),
    "block_sparse_attn_from_indices": (_c_int, [_c_void_p] * 7 + [_c_int] * 7 +
                                       [_c_float, _c_void_p, _c_void_p, _PL, _c_void_p, _c_size_t,
                                        _c_void_p]),
    "block_sparse_attn": (_c_int, [_c_void_p] * 6 + [_c_int] * 6 +
                          [_c_float, _c_void_p, _c_void_p, _c_void_p, _PL, _c_void_p, _c_size_t,
                           _c_void_p]),
    "block_sparse_attn_varlen_workspace_size": (_c_size_t, [_c_int] * 4),
    "block_sparse_attn_backward_workspace_size": (_c_size_t, [_c_int] * 4),
    "block_sparse_attn_backward": (_c_int, [_c_void_p] * 10 + [_c_int] * 6 +
                                   [_c_float, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                    _c_size_t, _c_void_p]),
    "block_sparse_attn_backward_ex_workspace_size": (_c_size_t, [_c_int] * 6),
    "block_sparse_attn_backward_ex": (_c_int, [_c_void_p] * 10 + [_c_int] * 7 +
                                      [_c_float, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                       _c_size_t, _c_void_p]),
    "block_sparse_attn_varlen_backward_workspace_size": (_c_size_t, [_c_int] * 5),
    "block_sparse_attn_varlen_backward": (_c_int, [_c_void_p] * 6 + [_P32] * 6 + [_c_int] * 3 +
                                          [_c_void_p, _c_void_p, _c_int, _c_float, _c_void_p,
                                           _c_void_p, _c_void_p, _c_void_p, _c_size_t,
                                           _c_void_p]),
    "block_sparse_attn_varlen": (_c_int, [_c_void_p] * 3 + [_P32, _P32, _P32, _P32, _P32, _P32] +
                                 [_c_int] * 3 + [_c_void_p, _c_void_p, _c_int, _c_float,
                                                 _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                                 _c_void_p, _c_size_t, _c_void_p]),
    "dense_attn_varlen": (_c_int, [_c_void_p] * 6 + [_c_int] * 4 +
                          [_c_int64, _c_int64, _c_int, _c_float, _c_void_p, _c_void_p, _c_void_p]),
    "dense_attn_varlen_backward_workspace_size": (_c_size_t, [_c_void_p] * 2 + [_c_int] * 4 + [_c_int64] * 2 +
                                                  [_c_int]),
    "dense_attn_varlen_backward": (_c_int, [_c_void_p] * 9 + [_c_int] * 4 +
                                   [_c_int64, _c_int64, _c_int, _c_float, _c_void_p, _c_void_p, _c_void_p,
                                    _c_void_p, _c_size_t, _c_void_p]),
    "shared_prefix_attn_workspace_size": (_c_size_t, [_c_int] * 5 + [_c_int64] * 2),
    "shared_prefix_attn": (_c_int, [_c_void_p] * 7 + [_c_int] * 5 +
                           [_c_int64, _c_int64, _c_float, _c_void_p, _c_void_p, _c_void_p, _c_size_t,
                            _c_void_p]),
    "build_vsa_metadata": (_c_int, [_c_int] * 6 + [_P64, _P64, _P32, _P64, _P64, _P32]),
    "vsa_gather_tokens": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int64, _c_int64, _c_int64,
                                   _c_int, _c_void_p]),
    "vsa_scatter_tokens": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int64, _c_int64,
                                    _c_int64, _c_int, _c_void_p]),
    "vsa_selftest_umma": (_c_int, [_c_int, _c_int, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "vsa_selftest_exp2": (_c_int, [_c_void_p, _c_void_p, _c_int64, _c_void_p, _c_void_p]),
    "vsa_permute_rows": (_c_int, [_c_void_p, _c_void_p, _P64, _P64, _c_int, _c_void_p]),
    "vsa_set_profile_events": (_c_int, [ctypes.POINTER(_c_void_p)]),
}

_LIB = None


class VSAError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(code, code)}")
        self.code = code


def lib() -> ctypes.CDLL:
    """Load libvsa.so (built in-tree); raise if it is missing."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run `python -m block_sparse_attention_15_b200.build`")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = h
    return _LIB


def _check(fn: str, code: int):
    if code != VSA_OK:
        raise VSAError(fn, code)


def _ptr(t):
    return None if t is None else _c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return _c_void_p(s.cuda_stream)


def _require(t, dtype, name, device=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _require_view(t, name):
    """A bf16 CUDA tensor whose last (head-dim) axis is contiguous and whose
    other strides are multiples of 8 elements (any layout: BHSD, BSHD, a
    slice of a fused tensor, a transposed view)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 4 or t.stride(3) != 1:
        raise ValueError(f"{name} must be a 4-D view with a contiguous last axis")
    for ax in range(3):
        if t.shape[ax] > 1 and (t.stride(ax) <= 0 or t.stride(ax) % 8):
            raise ValueError(f"{name}: stride {t.stride(ax)} of axis {ax} is not a positive "
                             "multiple of 8 elements")
    if t.data_ptr() % 16:
        raise ValueError(f"{name} must start on a 16-byte boundary")


def _strides_bhsd(t):
    """vsa_strides of a [B, H, S, D] view."""
    return VsaStrides(t.stride(0), t.stride(1), t.stride(2))


def _layout(q, k, v, out, gate_bshd=None):
    """vsa_layout of [B, H, S, D] views q, k, v, out and a [B, S, H, D] gate."""
    g = (VsaStrides(gate_bshd.stride(0), gate_bshd.stride(2), gate_bshd.stride(1))
         if gate_bshd is not None else VsaStrides(0, 0, 0))
    return VsaLayout(_strides_bhsd(q), _strides_bhsd(k), _strides_bhsd(v), _strides_bhsd(out), g)


def _block_sizes_tensor(bs, n, device):
    if bs is None:
        return None
    if not isinstance(bs, torch.Tensor):
        bs = torch.tensor(list(bs), dtype=torch.int32)
    bs = bs.to(device=device, dtype=torch.int32).contiguous()
    if bs.numel() != n:
        raise ValueError(f"expected {n} block sizes, got {bs.numel()}")
    return bs


def get_device_status(stream=None) -> int:
    """Synchronise the stream, then read and clear the device status word."""
    return lib().vsa_get_device_status(_stream(stream))


def check_device_status(stream=None):
    code = get_device_status(stream)
    if code != VSA_OK:
        raise VSAError("device status", code)


def vsa_forward(q, k, v, gate=None, q_block_sizes=None, kv_block_sizes=None, *, topk: int,
                scale: float | None = None, idx_stride: int | None = None, out=None,
                return_out_c: bool = False, return_pooled: bool = False, workspace=None,
                block: int = 64, stream=None):
    """Full VSA forward through ``vsa_forward_strided`` (see include/vsa.h).

    q: [B, H, Sq_pad, D] bf16; k, v: [B, H, Skv_pad, D]; gate: [B, Sq_pad, H, D]
    or None.  Any of them may be a strided view (head dim contiguous, other
    strides multiples of 8): a BSHD tensor transposed to [B, H, S, D], a
    slice of a fused QKV tensor.  ``out`` (allocated like q if None) may be a
    view too.  ``block``: slots per block, 64, 128 or 256 (VSA-128 / VSA-256
    tiles; S is then padded to multiples of the block).  Returns ``(out, q2k_idx, q2k_num)`` plus
    ``out_c`` and the pooled (qc, kc, vc) when asked.
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require_view(t, n)
    B, H, Sq, D = q.shape
    Skv = k.shape[2]
    if k.shape != (B, H, Skv, D) or v.shape != k.shape:
        raise ValueError("k and v must be [B, H, Skv_pad, D] matching q")
    if gate is not None:
        _require_view(gate, "gate")
        if gate.shape != (B, Sq, H, D):
            raise ValueError(f"gate must be [B, Sq_pad, H, D] = {(B, Sq, H, D)}, got {tuple(gate.shape)}")
    nq, nkv = Sq // block, Skv // block
    k_eff = min(int(topk), nkv)
    stride = k_eff if idx_stride is None else int(idx_stride)
    dev = q.device
    qbs = _block_sizes_tensor(q_block_sizes, nq, dev)
    kbs = _block_sizes_tensor(kv_block_sizes, nkv, dev)
    if out is None:
        out = torch.empty_like(q)
    _require_view(out, "out")
    if out.shape != q.shape:
        raise ValueError("out must be shaped like q")
    q2k_idx = torch.empty((B, H, nq, stride), dtype=torch.int32, device=dev)
    q2k_num = torch.empty((B, H, nq), dtype=torch.int32, device=dev)
    out_c = torch.empty((B, H, nq, D), dtype=torch.float32, device=dev) if return_out_c else None
    L = lib()
    ws_bytes = L.vsa_forward_workspace_size(B, H, nq, nkv, D)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
    lay = _layout(q, k, v, out, gate)
    _check("vsa_forward_strided", L.vsa_forward_strided(
        _ptr(q), _ptr(k), _ptr(v), _ptr(gate), ctypes.byref(lay), _ptr(qbs), _ptr(kbs), B, H, Sq,
        Skv, D, int(block), int(topk), float(scale) if scale is not None else 0.0, _ptr(out), _ptr(q2k_idx),
        _ptr(q2k_num), stride, _ptr(out_c), _ptr(workspace), workspace.numel(), _stream(stream)))
    res = [out, q2k_idx, q2k_num]
    if return_out_c:
        res.append(out_c)
    if return_pooled:
        res.append(pooled_views(workspace, B, H, nq, nkv, D))
    return tuple(res)


def vsa_forward_host(q, k, v, gate=None, q_block_sizes=None, kv_block_sizes=None, *, topk: int,
                     scale: float | None = None, idx_stride: int | None = None, out=None,
                     return_indices: bool = False, return_out_c: bool = False,
                     heads_per_chunk: int = 0, workspace=None, device=None, stream=None):
    """Full VSA forward on HOST tensors through ``vsa_forward_host`` (see
    include/vsa.h): the library stages chunks of heads onto the GPU, runs the
    forward and copies the results back, overlapping the three.

    q, k, v, gate: CPU bf16 tensors, shapes as in :func:`vsa_forward` (page-locked
    for the copies to overlap).  Returns ``out`` (a page-locked CPU tensor unless
    ``out`` is given) and, when asked, the host ``q2k_idx``, ``q2k_num`` and
    ``out_c``.  The call is asynchronous on ``stream``; synchronise it before
    reading the results.
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, torch.bfloat16, n, device=False)
        if t.is_cuda:
            raise ValueError(f"{n} must be a CPU tensor")
    B, H, Sq, D = q.shape
    Skv = k.shape[2]
    if k.shape != (B, H, Skv, D) or v.shape != k.shape:
        raise ValueError("k and v must be [B, H, Skv_pad, D] matching q")
    if gate is not None:
        _require(gate, torch.bfloat16, "gate", device=False)
        if gate.is_cuda or gate.shape != (B, Sq, H, D):
            raise ValueError(f"gate must be a CPU [B, Sq_pad, H, D] = {(B, Sq, H, D)} tensor")
    nq, nkv = Sq // 64, Skv // 64
    k_eff = min(int(topk), nkv)
    stride = k_eff if idx_stride is None else int(idx_stride)
    qbs = None if q_block_sizes is None else torch.tensor(list(q_block_sizes), dtype=torch.int32)
    kbs = None if kv_block_sizes is None else torch.tensor(list(kv_block_sizes), dtype=torch.int32)
    for bs, n, name in ((qbs, nq, "q_block_sizes"), (kbs, nkv, "kv_block_sizes")):
        if bs is not None and bs.numel() != n:
            raise ValueError(f"expected {n} {name}, got {bs.numel()}")
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, pin_memory=True)
    elif out.is_cuda or out.dtype != torch.bfloat16 or out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous CPU bf16 tensor shaped like q")
    q2k_idx = torch.empty((B, H, nq, stride), dtype=torch.int32, pin_memory=True) if return_indices else None
    q2k_num = torch.empty((B, H, nq), dtype=torch.int32, pin_memory=True) if return_indices else None
    out_c = torch.empty((B, H, nq, D), dtype=torch.float32, pin_memory=True) if return_out_c else None
    L = lib()
    ws_bytes = L.vsa_forward_host_workspace_size(B, H, nq, nkv, D, stride, 1 if gate is not None else 0,
                                                 int(heads_per_chunk))
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        _check("vsa_forward_host", L.vsa_forward_host(
            _ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(qbs), _ptr(kbs), B, H, Sq, Skv, D, int(topk),
            float(scale) if scale is not None else 0.0, _ptr(out), _ptr(q2k_idx), _ptr(q2k_num), stride,
            _ptr(out_c), int(heads_per_chunk), _ptr(workspace), workspace.numel(), _stream(stream)))
    res = [out]
    if return_indices:
        res += [q2k_idx, q2k_num]
    if return_out_c:
        res.append(out_c)
    return res[0] if len(res) == 1 else tuple(res)


def pooled_views(workspace, B, H, nq, nkv, D):
    """(qc, kc, vc) fp32 views of a vsa_forward workspace (its documented order)."""
    g = B * H * D * 4

    def a256(x):
        return (x + 255) // 256 * 256

    offs = [0, a256(g * nq), a256(g * nq) + a256(g * nkv)]
    shapes = [(B, H, nq, D), (B, H, nkv, D), (B, H, nkv, D)]
    views = []
    for off, shp in zip(offs, shapes):
        n = int(np.prod(shp))
        views.append(workspace[off:off + 4 * n].view(torch.float32).view(shp))
    return tuple(views)


def _sparse_common(q, k, v, out):
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require_view(t, n)
    B, H, Sq, D = q.shape
    Skv = k.shape[2]
    if k.shape != (B, H, Skv, D) or v.shape != k.shape:
        raise ValueError("k and v must be [B, H, Skv_pad, D] matching q")
    if out is None:
        out = torch.empty_like(q)
    _require_view(out, "out")
    if out.shape != q.shape:
        raise ValueError("out must be shaped like q")
    return B, H, Sq, Skv, D, out


def block_sparse_attn_from_indices(q, k, v, q2k_idx, q2k_num, q_block_sizes=None,
                                   kv_block_sizes=None, *, scale: float | None = None, out=None,
                                   logit_bound: bool = True, block: int = 64,
                                   return_lse: bool = False, stream=None):
    """Block-sparse attention over the listed tiles (``block_sparse_attn_from_indices``).

    q, k, v, out: [B, H, S, D] views (see :func:`vsa_forward`).  With
    ``logit_bound`` (default) a workspace is passed, so the library bounds
    each query block's logits first and the kernel skips its running-max
    check where the bound allows (same results).  With ``return_lse`` also
    returns the fp32 [B, H, Sq] natural-log log-sum-exp per query row (the
    normaliser :func:`block_sparse_attn_backward` takes)."""
    B, H, Sq, Skv, D, out = _sparse_common(q, k, v, out)
    _require(q2k_idx, torch.int32, "q2k_idx")
    _require(q2k_num, torch.int32, "q2k_num")
    nq, nkv = Sq // block, Skv // block
    if q2k_idx.dim() != 4 or q2k_idx.shape[:3] != (B, H, nq) or q2k_num.shape != (B, H, nq):
        raise ValueError("q2k_idx must be [B, H, n_q_blocks, stride], q2k_num [B, H, n_q_blocks]")
    dev = q.device
    qbs = _block_sizes_tensor(q_block_sizes, nq, dev)
    kbs = _block_sizes_tensor(kv_block_sizes, nkv, dev)
    L = lib()
    ws = None
    if logit_bound:
        ws = torch.empty(max(L.block_sparse_attn_from_indices_workspace_size(B, H, nq, nkv), 256),
                         dtype=torch.uint8, device=dev)
    lay = _layout(q, k, v, out)
    lse = torch.empty((B, H, Sq), dtype=torch.float32, device=dev) if return_lse else None
    _check("block_sparse_attn_from_indices", L.block_sparse_attn_from_indices(
        _ptr(q), _ptr(k), _ptr(v), _ptr(q2k_idx), _ptr(q2k_num), _ptr(qbs), _ptr(kbs), B, H, Sq,
        Skv, D, int(block), q2k_idx.shape[3], float(scale) if scale is not None else 0.0, _ptr(out),
        _ptr(lse), ctypes.byref(lay), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))
    return (out, lse) if return_lse else out


def block_sparse_attn(q, k, v, block_map, q_block_sizes=None, kv_block_sizes=None, *,
                      scale: float | None = None, out=None, return_indices: bool = False,
                      block: int = 64, stream=None):
    """Block-sparse attention from a bool block map [B, H, n_q_blocks,
    n_kv_blocks] (``block_sparse_attn``): converted on the device to index
    rows, then the index-native kernel.  With ``return_indices`` also
    returns the (q2k_idx, q2k_num) it produced."""
    B, H, Sq, Skv, D, out = _sparse_common(q, k, v, out)
    nq, nkv = Sq // block, Skv // block
    if not isinstance(block_map, torch.Tensor) or block_map.dtype != torch.bool:
        raise TypeError("block_map must be a torch.bool tensor")
    if tuple(block_map.shape) != (B, H, nq, nkv) or not block_map.is_cuda or not block_map.is_contiguous():
        raise ValueError(f"block_map must be a contiguous CUDA [B, H, n_q_blocks, n_kv_blocks] = "
                         f"{(B, H, nq, nkv)} tensor")
    dev = q.device
    qbs = _block_sizes_tensor(q_block_sizes, nq, dev)
    kbs = _block_sizes_tensor(kv_block_sizes, nkv, dev)
    q2k_idx = torch.empty((B, H, nq, nkv), dtype=torch.int32, device=dev)
    q2k_num = torch.empty((B, H, nq), dtype=torch.int32, device=dev)
    L = lib()
    ws = torch.empty(max(L.block_sparse_attn_from_indices_workspace_size(B, H, nq, nkv), 256),
                     dtype=torch.uint8, device=dev)
    lay = _layout(q, k, v, out)
    _check("block_sparse_attn", L.block_sparse_attn(
        _ptr(q), _ptr(k), _ptr(v), _ptr(block_map), _ptr(qbs), _ptr(kbs), B, H, Sq, Skv, D,
        int(block), float(scale) if scale is not None else 0.0, _ptr(out), _ptr(q2k_idx), _ptr(q2k_num),
        ctypes.byref(lay), _ptr(ws), ws.numel(), _stream(stream)))
    return (out, q2k_idx, q2k_num) if return_indices else out


def video_sparse_attn_bshd(q, k, v, gate=None, q_block_sizes=None, kv_block_sizes=None, *,
                           topk: int, scale: float | None = None, idx_stride: int | None = None,
                           out=None, return_out_c: bool = False, workspace=None, block: int = 64,
                           stream=None):
    """The whole VSA forward on BSHD tensors: q [B, Sq_pad, H, D], k and v
    [B, Skv_pad, H, D], gate [B, Sq_pad, H, D]; the output is BSHD too.  The
    library reads and writes the BSHD memory in place (strided views, no
    transposed copies).  Returns ``(out, q2k_idx, q2k_num)`` (+ ``out_c``)."""
    if out is None and isinstance(q, torch.Tensor):
        out = torch.empty_like(q)
    res = vsa_forward(q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2), gate,
                      q_block_sizes, kv_block_sizes, topk=topk, scale=scale, idx_stride=idx_stride,
                      out=None if out is None else out.transpose(1, 2), return_out_c=return_out_c,
                      workspace=workspace, block=block, stream=stream)
    return (out,) + tuple(res[1:])


def block_sparse_attn_backward(q, k, v, out, dout, lse, q2k_idx, q2k_num, q_block_sizes=None,
                               kv_block_sizes=None, *, scale: float | None = None, block: int = 64,
                               stream=None):
    """dq, dk, dv of :func:`block_sparse_attn_from_indices` (contiguous BHSD)
    for the output gradient ``dout``; ``out`` and ``lse`` come from that
    forward call (``return_lse=True``), ``block`` is its block size.  Block
    64 calls ``block_sparse_attn_backward``; 128 and 256 call
    ``block_sparse_attn_backward_ex``, which rewrites the selection over
    64-slot sub-blocks on the device first."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _require(t, torch.bfloat16, n)
    _require(lse, torch.float32, "lse")
    _require(q2k_idx, torch.int32, "q2k_idx")
    _require(q2k_num, torch.int32, "q2k_num")
    B, H, Sq, D = q.shape
    Skv = k.shape[2]
    nq, nkv = Sq // block, Skv // block
    if out.shape != q.shape or dout.shape != q.shape or lse.shape != (B, H, Sq):
        raise ValueError("out and dout must be shaped like q, lse [B, H, Sq_pad]")
    if q2k_idx.dim() != 4 or q2k_idx.shape[:3] != (B, H, nq) or q2k_num.shape != (B, H, nq):
        raise ValueError("q2k_idx must be [B, H, n_q_blocks, stride], q2k_num [B, H, n_q_blocks]")
    dev = q.device
    qbs = _block_sizes_tensor(q_block_sizes, nq, dev)
    kbs = _block_sizes_tensor(kv_block_sizes, nkv, dev)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    L = lib()
    sc = float(scale) if scale is not None else 0.0
    width = q2k_idx.shape[3]
    if block == 64:
        ws = torch.empty(max(L.block_sparse_attn_backward_workspace_size(B, H, Sq, nkv), 256),
                         dtype=torch.uint8, device=dev)
        _check("block_sparse_attn_backward", L.block_sparse_attn_backward(
            _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(q2k_idx),
            _ptr(q2k_num), _ptr(qbs), _ptr(kbs), B, H, Sq, Skv, D, width, sc, _ptr(dq), _ptr(dk),
            _ptr(dv), _ptr(ws), ws.numel(), _stream(stream)))
        return dq, dk, dv
    need = L.block_sparse_attn_backward_ex_workspace_size(B, H, Sq, Skv, int(block), width)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _check("block_sparse_attn_backward_ex", L.block_sparse_attn_backward_ex(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(q2k_idx), _ptr(q2k_num),
        _ptr(qbs), _ptr(kbs), B, H, Sq, Skv, D, int(block), width, sc, _ptr(dq), _ptr(dk), _ptr(dv),
        _ptr(ws), ws.numel(), _stream(stream)))
    return dq, dk, dv


def _host_i32(xs):
    arr = np.ascontiguousarray(np.asarray(xs, dtype=np.int32))
    return arr, arr.ctypes.data_as(_P32)


def block_sparse_attn_varlen(q, k, v, cu_seqlens_q, cu_seqlens_kv, q2k_idx, q2k_num, *,
                             scale: float | None = None, q_block_sizes_list=None,
                             kv_block_sizes_list=None, return_aux: bool = False, out=None,
                             lse=None, stream=None):
    """Varlen block-sparse attention (``block_sparse_attn_varlen``).

    q: [H, total_q, D]; k, v: [H, total_kv, D]; cu_seqlens_*: host sequences
    of n+1 ints; q2k_idx: [H, total_q_blocks, stride] with per-sequence local
    indices.  With ``return_aux`` also returns (pack_index_q, pack_index_kv,
    q2k_idx_rebased).
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, torch.bfloat16, n)
    _require(q2k_idx, torch.int32, "q2k_idx")
    _require(q2k_num, torch.int32, "q2k_num")
    H, total_q, D = q.shape
    cq, cq_p = _host_i32(cu_seqlens_q)
    ck, ck_p = _host_i32(cu_seqlens_kv)
    n = len(cq) - 1
    keep = [cq, ck]

    def sizes(lst):
        if lst is None:
            return None, None, None
        flat = [int(s) for seq in lst for s in seq]
        cub = [0]
        for seq in lst:
            cub.append(cub[-1] + len(seq))
        a, ap = _host_i32(flat)
        b, bp = _host_i32(cub)
        keep.extend([a, b])
        return ap, bp, len(flat)

    qs_p, qcb_p, nqb = sizes(q_block_sizes_list)
    ks_p, kcb_p, nkb = sizes(kv_block_sizes_list)
    if nqb is None:
        nqb = sum(-(-(int(cq[i + 1]) - int(cq[i])) // 64) for i in range(n))
    if nkb is None:
        nkb = sum(-(-(int(ck[i + 1]) - int(ck[i])) // 64) for i in range(n))
    dev = q.device
    if out is None:
        out = torch.zeros_like(q)
    L = lib()
    ws_bytes = L.block_sparse_attn_varlen_workspace_size(max(n, 1), max(nqb, 1), max(nkb, 1), max(H, 1))
    ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
    aux = None
    if return_aux:
        aux = (torch.empty(64 * nqb, dtype=torch.int64, device=dev),
               torch.empty(64 * nkb, dtype=torch.int64, device=dev),
               torch.empty_like(q2k_idx))
    stride = q2k_idx.shape[-1]
    _check("block_sparse_attn_varlen", L.block_sparse_attn_varlen(
        _ptr(q), _ptr(k), _ptr(v), cq_p, ck_p, qs_p, qcb_p, ks_p, kcb_p, n, H, D, _ptr(q2k_idx),
        _ptr(q2k_num), stride, float(scale) if scale is not None else 0.0, _ptr(out), _ptr(lse),
        _ptr(aux[0]) if aux else None, _ptr(aux[1]) if aux else None,
        _ptr(aux[2]) if aux else None, _ptr(ws), ws.numel(), _stream(stream)))
    del keep
    return (out, *aux) if return_aux else out


def block_sparse_attn_varlen_backward(q, k, v, out, dout, lse, cu_seqlens_q, cu_seqlens_kv,
                                      q2k_idx, q2k_num, *, scale: float | None = None,
                                      stream=None):
    """dq, dk, dv of :func:`block_sparse_attn_varlen` (64-token blocks with a
    partial last block per sequence); ``out`` and ``lse`` [H, total_q] come
    from that forward call."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _require(t, torch.bfloat16, n)
    _require(lse, torch.float32, "lse")
    _require(q2k_idx, torch.int32, "q2k_idx")
    _require(q2k_num, torch.int32, "q2k_num")
    H, total_q, D = q.shape
    cq, cq_p = _host_i32(cu_seqlens_q)
    ck, ck_p = _host_i32(cu_seqlens_kv)
    n = len(cq) - 1
    nqb = sum(-(-(int(cq[i + 1]) - int(cq[i])) // 64) for i in range(n))
    nkb = sum(-(-(int(ck[i + 1]) - int(ck[i])) // 64) for i in range(n))
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    L = lib()
    ws = torch.empty(max(L.block_sparse_attn_varlen_backward_workspace_size(n, nqb, nkb, H, total_q), 256),
                     dtype=torch.uint8, device=q.device)
    _check("block_sparse_attn_varlen_backward", L.block_sparse_attn_varlen_backward(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), cq_p, ck_p, None, None, None,
        None, n, H, D, _ptr(q2k_idx), _ptr(q2k_num), q2k_idx.shape[-1],
        float(scale) if scale is not None else 0.0, _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws),
        ws.numel(), _stream(stream)))
    del cq, ck
    return dq, dk, dv


# The dense entries are called once per layer and token, and their kernels may
# take less time than Python's part of a call: each tensor is looked at once,
# and the structures the library takes are packed as bytes.
_LAYOUT8 = struct.Struct("24q")   # vsa_dense_layout
_LAYOUT6 = struct.Struct("18q")   # vsa_prefix_layout
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_Tensor, _BF16, _F32, _U8 = torch.Tensor, torch.bfloat16, torch.float32, torch.uint8


def _rows(t, name):
    """(H, rows, D, head stride, row stride, address) of a bf16 CUDA [H, rows, D]
    view: head dim contiguous, other strides multiples of 8 elements
    (token-major memory transposed, a slice of a fused tensor)."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != _BF16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be a 3-D [H, rows, D] view")
    h, r, d = shape
    if not (h and r and d):
        return h, r, d, 0, 0, t.data_ptr()
    s0, s1, s2 = t.stride()
    if s2 != 1 or (h > 1 and (s0 <= 0 or s0 & 7)) or (r > 1 and (s1 <= 0 or s1 & 7)):
        raise ValueError(f"{name}: strides {(s0, s1, s2)} must be positive multiples of 8 elements, "
                         "the last 1")
    ptr = t.data_ptr()
    if ptr & 15:
        raise ValueError(f"{name} must start on a 16-byte boundary")
    return h, r, d, s0, s1, ptr


def _heads(t, name):
    """(shape, strides, address) of a bf16 CUDA [B, H, S, D] view, likewise."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != _BF16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape = t.shape
    if len(shape) != 4:
        raise ValueError(f"{name} must be a 4-D [B, H, S, D] view")
    b, h, n, d = shape
    if not (b and h and n and d):
        return shape, (0, 0, 0), t.data_ptr()
    st = s0, s1, s2, s3 = t.stride()
    if (s3 != 1 or (b > 1 and (s0 <= 0 or s0 & 7)) or (h > 1 and (s1 <= 0 or s1 & 7)) or
            (n > 1 and (s2 <= 0 or s2 & 7))):
        raise ValueError(f"{name}: strides {st} must be positive multiples of 8 elements, the last 1")
    ptr = t.data_ptr()
    if ptr & 15:
        raise ValueError(f"{name} must start on a 16-byte boundary")
    return shape, (s0, s1, s2), ptr


def _same_device(index, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"a tensor is on {t.device}, q on cuda:{index}")


def _on(index, stream, call):
    """call(handle of the stream the kernels run on), with the tensors' device
    current and memory allocated on that stream."""
    if stream is None and torch.cuda.current_device() == index:
        return call(_raw_stream(index))
    if stream is not None and stream.device.index != index:
        # (kernels there would reach for this device's memory)
        raise ValueError(f"stream is on {stream.device}, q on cuda:{index}")
    with torch.cuda.device(index):
        if stream is None:
            return call(_raw_stream(index))
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)


def _cumulative(xs, name):
    """Host int32 copy of cumulative lengths, an array."""
    if isinstance(xs, (list, tuple)):
        try:
            return array.array("i", xs)
        except (TypeError, OverflowError):
            pass  # arrays' or tensors' elements, or what is refused below
    a = np.asarray(xs)
    if a.ndim != 1:
        raise ValueError(f"{name} must be a 1-D sequence")
    if a.dtype.kind not in "iu":
        raise TypeError(f"{name} must hold integers, got {a.dtype}")
    if a.size and (a.min() < -2 ** 31 or a.max() >= 2 ** 31):
        raise ValueError(f"{name} holds a value outside the 32-bit range")
    return array.array("i", a.tolist())


def _dense_common(q, k, v, cu_seqlens_q, cu_seqlens_kv):
    qi, ki, vi = _rows(q, "q"), _rows(k, "k"), _rows(v, "v")
    if vi[:3] != ki[:3] or ki[2] != qi[2]:
        raise ValueError("k and v must be [Hkv, kv_rows, D] with q's D")
    cq, ck = _cumulative(cu_seqlens_q, "cu_seqlens_q"), _cumulative(cu_seqlens_kv, "cu_seqlens_kv")
    if len(cq) != len(ck) or not cq:
        raise ValueError("cu_seqlens_q and cu_seqlens_kv must have n_seqs + 1 entries each")
    return qi, ki, vi, cq, ck


def _output(t, like, info, cu, name):
    """(tensor, head stride, row stride, address) of an output like the packed
    tensor `like` (its _rows `info`): `t` if given, else a new one whose rows past
    the last sequence are 0."""
    if t is None:
        t = torch.empty_like(like)
        if 0 <= cu[-1] < info[1]:
            t[:, cu[-1]:].zero_()
        s0, s1, _ = t.stride()
        return t, s0, s1, t.data_ptr()
    if t.shape != like.shape:
        raise ValueError(f"{name} must be shaped like its input, {tuple(like.shape)}")
    i = _rows(t, name)
    return t, i[3], i[4], i[5]


def _workspace(t, need, like):
    """(tensor, address, bytes)."""
    if t is None:
        t = torch.empty(max(need, 256), dtype=_U8, device=like.device)
    elif not t.is_contiguous():
        # an expanded view has fewer bytes behind it than elements
        raise ValueError("workspace must be contiguous")
    return t, t.data_ptr(), t.numel() * t.element_size()


def dense_attn_varlen(q, k, v, cu_seqlens_q, cu_seqlens_kv, *, causal: bool = True,
                      scale: float | None = None, out=None, return_lse: bool = False, stream=None):
    """Dense attention of packed sequences with grouped heads
    (``dense_attn_varlen``): causal (a sequence's last row sees all its keys,
    the row before it one fewer, ...) or full.

    q: [Hq, q_rows, D]; k, v: [Hkv, kv_rows, D]; any of them a strided view
    (token-major [rows, H, D] memory transposed, a slice of a fused QKV
    tensor).  cu_seqlens_*: host sequences of n + 1 ints from 0, as in
    :func:`block_sparse_attn_varlen`; lengths may be 0.  Rows of a given
    ``out`` past the last sequence are left as they were (0 when it is
    allocated here).  With ``return_lse`` also returns the fp32 [Hq, q_rows]
    natural-log log-sum-exp (-inf where a row sees no key), which
    :func:`dense_attn_varlen_backward` takes.  ``scale``: None, or a value <= 0,
    is 1/sqrt(D).  Probabilities are rounded to bf16 for the product with v.

    The result carries no autograd history, even where q, k or v require
    gradients: those come from :func:`dense_attn_varlen_backward`, called by a
    training step itself or in the backward of a ``torch.autograd.Function``."""
    qi, ki, vi, cq, ck = _dense_common(q, k, v, cu_seqlens_q, cu_seqlens_kv)
    index = q.get_device()
    _same_device(index, k, v, out)

    def call(st):
        o, o0, o1, op = _output(out, q, qi, cq, "out")
        lse = None
        if return_lse:
            lse = torch.empty((qi[0], qi[1]), dtype=_F32, device=q.device)
            if 0 <= cq[-1] < qi[1]:
                lse[:, cq[-1]:].zero_()
        lay = _LAYOUT8.pack(0, qi[3], qi[4], 0, ki[3], ki[4], 0, vi[3], vi[4], 0, o0, o1,
                            0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
        _check("dense_attn_varlen", lib().dense_attn_varlen(
            qi[5], ki[5], vi[5], lay, cq.buffer_info()[0], ck.buffer_info()[0], len(cq) - 1, qi[0], ki[0], qi[2],
            qi[1], ki[1], 1 if causal else 0, 0.0 if scale is None else float(scale), op,
            None if lse is None else lse.data_ptr(), st))
        return (o, lse) if return_lse else o

    return _on(index, stream, call)


def dense_attn_varlen_backward(q, k, v, out, dout, lse, cu_seqlens_q, cu_seqlens_kv, *, causal: bool = True,
                               scale: float | None = None, dq=None, dk=None, dv=None, workspace=None,
                               stream=None):
    """(dq, dk, dv) of :func:`dense_attn_varlen` (``dense_attn_varlen_backward``);
    ``out`` and ``lse`` come from that call, the other arguments are its own.
    ``dout`` and the gradients may be strided views like q and k.  dk and dv sum
    over the query heads of a key head.  Rows of given gradients past the last
    sequence are left as they were (0 where they are allocated here).
    Probabilities and ds are rounded to bf16 for the products that sum them."""
    qi, ki, vi, cq, ck = _dense_common(q, k, v, cu_seqlens_q, cu_seqlens_kv)
    oi, gi = _rows(out, "out"), _rows(dout, "dout")
    if oi[:3] != qi[:3] or gi[:3] != qi[:3]:
        raise ValueError("out and dout must be shaped like q")
    _require(lse, torch.float32, "lse")
    if lse.shape != (qi[0], qi[1]):
        raise ValueError(f"lse must be [Hq, q_rows] = {(qi[0], qi[1])}")
    index = q.get_device()
    _same_device(index, k, v, out, dout, lse, workspace, dq, dk, dv)
    L = lib()

    def call(st):
        a, a0, a1, ap = _output(dq, q, qi, cq, "dq")
        b, b0, b1, bp = _output(dk, k, ki, ck, "dk")
        c, c0, c1, cp = _output(dv, v, vi, ck, "dv")
        cqp, ckp, n = cq.buffer_info()[0], ck.buffer_info()[0], len(cq) - 1
        need = 0 if workspace is not None else L.dense_attn_varlen_backward_workspace_size(
            cqp, ckp, n, qi[0], ki[0], qi[2], qi[1], ki[1], 1 if causal else 0)
        ws, wp, nbytes = _workspace(workspace, need, q)
        lay = _LAYOUT8.pack(0, qi[3], qi[4], 0, ki[3], ki[4], 0, vi[3], vi[4], 0, oi[3], oi[4],
                            0, gi[3], gi[4], 0, a0, a1, 0, b0, b1, 0, c0, c1)
        _check("dense_attn_varlen_backward", L.dense_attn_varlen_backward(
            qi[5], ki[5], vi[5], oi[5], gi[5], lse.data_ptr(), lay, cqp, ckp, n, qi[0], ki[0], qi[2], qi[1], ki[1],
            1 if causal else 0, 0.0 if scale is None else float(scale), ap, bp, cp, wp, nbytes, st))
        return a, b, c

    return _on(index, stream, call)


def shared_prefix_attn(q, k_prefix, v_prefix, k_suffix, v_suffix, suffix_lens, *,
                       scale: float | None = None, out=None, return_lse: bool = False, workspace=None,
                       stream=None):
    """Attention of the newest tokens of many requests over a prefix they share
    and over their own keys behind it (``shared_prefix_attn``): one decoding
    step, or the check of a few drafted tokens.

    q: [B, Hq, T, D]; k_prefix, v_prefix: [Hkv, P, D], kept once for all
    requests (P may be 0; both None: no prefix); k_suffix, v_suffix: [B, Hkv,
    capacity, D], the last T of a request's ``suffix_lens[b]`` keys being its new
    tokens'; all may be strided views (token-major caches transposed).  suffix_lens: CUDA int32
    [B], read on the device.  Token t sees the prefix and its first
    ``suffix_lens[b] - T + 1 + t`` suffix keys.  Returns [B, Hq, T, D], with
    ``return_lse`` also the fp32 [B, Hq, T] natural-log log-sum-exp.  ``scale``:
    None, or a value <= 0, is 1/sqrt(D).  Probabilities are rounded to bf16 for
    the product with v.  A NaN or infinity in a new token's v may reach the
    request's earlier new tokens, although they do not see it."""
    (B, Hq, T, D), qs, qp = _heads(q, "q")
    ks_shape, kss, ksp = _heads(k_suffix, "k_suffix")
    vs_shape, vss, vsp = _heads(v_suffix, "v_suffix")
    if k_prefix is None and v_prefix is None:
        kp = vp = (ks_shape[1], 0, D, 0, 0, None)
    else:
        kp, vp = _rows(k_prefix, "k_prefix"), _rows(v_prefix, "v_prefix")
    _require(suffix_lens, torch.int32, "suffix_lens")
    Hkv, P, cap = kp[0], kp[1], ks_shape[2]
    if vp[:3] != kp[:3] or kp[2] != D:
        raise ValueError("k_prefix and v_prefix must be [Hkv, P, D] with q's D")
    if ks_shape != (B, Hkv, cap, D) or vs_shape != ks_shape:
        raise ValueError(f"k_suffix and v_suffix must be [B, Hkv, capacity, D] = {(B, Hkv, cap, D)}")
    if suffix_lens.shape != (B,):
        raise ValueError(f"suffix_lens must be [B] = [{B}]")
    index = q.get_device()
    _same_device(index, k_prefix, v_prefix, k_suffix, v_suffix, suffix_lens, out, workspace)
    L = lib()

    def call(st):
        o = torch.empty_like(q) if out is None else out
        shape, os_, op = _heads(o, "out")
        if shape != (B, Hq, T, D):
            raise ValueError("out must be shaped like q")
        lse = torch.empty((B, Hq, T), dtype=_F32, device=q.device) if return_lse else None
        need = 0 if workspace is not None else L.shared_prefix_attn_workspace_size(B, Hq, Hkv, T, D, P, cap)
        ws, wp, nbytes = _workspace(workspace, need, q)
        lay = _LAYOUT6.pack(*qs, *os_, 0, kp[3], kp[4], 0, vp[3], vp[4], *kss, *vss)
        _check("shared_prefix_attn", L.shared_prefix_attn(
            qp, kp[5], vp[5], ksp, vsp, suffix_lens.data_ptr(), lay, B, Hq, Hkv, T, D, P, cap,
            0.0 if scale is None else float(scale), op, None if lse is None else lse.data_ptr(), wp, nbytes, st))
        return (o, lse) if return_lse else o

    return _on(index, stream, call)


def build_vsa_metadata(T: int, Hh: int, W: int, tile=(4, 4, 4)) -> dict:
    """Tile metadata from the library's host routine (numpy arrays)."""
    L = lib()
    n_tiles = ctypes.c_int32(0)
    _check("build_vsa_metadata", L.build_vsa_metadata(T, Hh, W, *tile, None, None, None, None, None,
                                                      ctypes.byref(n_tiles)))
    N = T * Hh * W
    vol = int(np.prod(tile))
    nt = n_tiles.value
    perm = np.empty(N, dtype=np.int64)
    rev = np.empty(N, dtype=np.int64)
    vbs = np.empty(nt, dtype=np.int32)
    npi = np.empty(N, dtype=np.int64)
    slot = np.empty(nt * vol, dtype=np.int64)
    _check("build_vsa_metadata", L.build_vsa_metadata(
        T, Hh, W, *tile, perm.ctypes.data_as(_P64), rev.ctypes.data_as(_P64),
        vbs.ctypes.data_as(_P32), npi.ctypes.data_as(_P64), slot.ctypes.data_as(_P64),
        ctypes.byref(n_tiles)))
    return dict(tile_partition_indices=perm, reverse_tile_partition_indices=rev,
                variable_block_sizes=vbs, non_pad_index=npi, slot_token=slot, n_tiles=nt,
                max_block_size=vol)


def gather_tokens(x, slot_token, *, stream=None):
    """[G, N, D] tokens -> [G, n_slots, D] padded block layout (zeros in pads)."""
    _require(x, torch.bfloat16, "x")
    _require(slot_token, torch.int64, "slot_token")
    G, N, D = x.shape
    ns = slot_token.numel()
    dst = torch.empty((G, ns, D), dtype=x.dtype, device=x.device)
    _check("vsa_gather_tokens", lib().vsa_gather_tokens(_ptr(x), _ptr(dst), _ptr(slot_token), N, ns,
                                                        G, D, _stream(stream)))
    return dst


def scatter_tokens(x_pad, slot_token, n_tokens: int, *, stream=None):
    """Inverse of :func:`gather_tokens` on the real tokens."""
    _require(x_pad, torch.bfloat16, "x_pad")
    _require(slot_token, torch.int64, "slot_token")
    G, ns, D = x_pad.shape
    dst = torch.empty((G, n_tokens, D), dtype=x_pad.dtype, device=x_pad.device)
    _check("vsa_scatter_tokens", lib().vsa_scatter_tokens(_ptr(x_pad), _ptr(dst), _ptr(slot_token),
                                                          n_tokens, ns, G, D, _stream(stream)))
    return dst


def selftest_umma(mode: int, a, b, *, stream=None):
    """Run one tensor-core product of the sparse kernel on global operands."""
    _require(a, torch.bfloat16, "a")
    _require(b, torch.bfloat16, "b")
    D = b.shape[1] if mode >= 2 else a.shape[1]
    shape = {0: (128, 64), 1: (D, 64), 2: (128, 128), 3: (128, D)}[mode]
    c = torch.empty(shape, dtype=torch.float32, device=a.device)
    _check("vsa_selftest_umma", lib().vsa_selftest_umma(mode, D, _ptr(a), _ptr(b), _ptr(c),
                                                        _stream(stream)))
    return c


def permute_rows(src, extents, src_strides, *, out=None, stream=None):
    """``vsa_permute_rows``: rows of the last axis of ``src`` (a contiguous
    bf16 CUDA tensor, D = src.shape[-1]) gathered into a new tensor of shape
    (*extents, D): out[a0, a1, a2, a3] = src row a0*S0 + a1*S1 + a2*S2 + a3*S3."""
    _require(src, torch.bfloat16, "src")
    D = src.shape[-1]
    ext = [int(e) for e in extents]
    st = [int(x) for x in src_strides]
    if len(ext) != 4 or len(st) != 4:
        raise ValueError("extents and src_strides take four entries")
    rows = src.numel() // D
    if any(e > 0 for e in ext) and sum((e - 1) * s_ for e, s_ in zip(ext, st) if e > 0) >= rows:
        raise ValueError("the strides reach past the end of src")
    if out is None:
        out = torch.empty((*ext, D), dtype=src.dtype, device=src.device)
    _require(out, torch.bfloat16, "out")
    e64 = (ctypes.c_int64 * 4)(*ext)
    s64 = (ctypes.c_int64 * 4)(*st)
    _check("vsa_permute_rows", lib().vsa_permute_rows(_ptr(src), _ptr(out), e64, s64, D,
                                                      _stream(stream)))
    return out


def selftest_exp2(x, *, stream=None):
    """The sparse kernel's FMA-pipe 2^x on a device fp32 tensor; returns
    (y, number of elements whose packed halves disagree)."""
    _require(x, torch.float32, "x")
    y = torch.empty_like(x)
    mism = torch.zeros(1, dtype=torch.int32, device=x.device)
    _check("vsa_selftest_exp2", lib().vsa_selftest_exp2(_ptr(x), _ptr(y), x.numel(), _ptr(mism),
                                                        _stream(stream)))
    return y, int(mism.item())


def set_profile_events(events):
    """Record four torch.cuda.Event objects around vsa_forward's kernels
    (before pool, after pool, after coarse/top-k, after block-sparse), or
    switch the hook off with None."""
    if events is None:
        _check("vsa_set_profile_events", lib().vsa_set_profile_events(None))
        return
    for e in events:
        if not e.cuda_event:  # torch creates the handle on first record
            e.record()
    arr = (_c_void_p * 4)(*[e.cuda_event for e in events])
    _check("vsa_set_profile_events", lib().vsa_set_profile_events(arr))


def default_scale(D: int) -> float:
    return 1.0 / math.sqrt(D)
