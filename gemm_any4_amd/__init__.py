"""Python binding of libany4.so, the MI355X any4 dequantize-GEMM.

Argument marshalling only: every step runs in the HIP kernels behind the C ABI
in ``include/any4.h``.  PyTorch provides device memory and the current HIP
stream.  There is no CPU fallback: if the library is missing or a call fails,
a ``RuntimeError`` is raised.

Tensors
  idx     uint8  [N, K]     values 0..15, K a multiple of 128
  packed  uint8  [packed_bytes(N, K)]  the indices in the library's tile layout
                            (16 rows x 128 k per 1 KB tile; include/any4.h)
  lut     bf16   [N, 16]    per-row table
  alpha   bf16   [N, K/g]   per-group scale
  beta    bf16   [N, K/g]   per-group offset
  x       bf16   [M, K]     M = 1..16 (decode); larger M also accepted
  y       bf16   [M, N]
  w       bf16   [N, K]
(bf16 tensors may also be given as int16/uint16 bit patterns.)

Calls: pack, dequant, gemm (any4); gemm_int4 (plain int4, no table);
any2_pack / any2_dequant / any2_gemm and any3_pack / any3_dequant / any3_gemm
(2- and 3-bit codes in their own tile layouts); quantize (the weighted
k-means quantiser at 4, 3 or 2 bits); each also as a ``*_raw`` function on
device pointers that returns the C status.

For fine-tunes of such a layer: lora, gemm_lora, lora_backward and lora_plan
(low-rank adapters of many requests at once, and their gradients); act8_save,
act8_load and act8_empty (an activation kept in 8 bits); gemm_dx,
gemm_int4_dx, any2_gemm_dx and any3_gemm_dx (the gradient of a layer's input).
These take tensors of any GPU, run on that GPU's current stream (or `stream`,
on which their outputs and workspaces are then allocated too) and can be
captured into a graph.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libany4.so")

ANY4_OK = 0
_STATUS_NAMES = {0: "ANY4_OK", 1: "ANY4_E_NULL", 2: "ANY4_E_SHAPE", 3: "ANY4_E_ALIGN",
                 4: "ANY4_E_WORKSPACE", 5: "ANY4_E_HIP"}

# every symbol include/any4.h declares
EXPORTS = ("any4_packed_bytes", "any4_pack", "any4_dequant", "any4_gemm_workspace_size",
           "any4_gemm", "any4_gemm_noalloc", "any4_gemv_dot", "any4_gemm_int4", "any4_quantize", "any4_status_string",
           "any2_packed_bytes", "any2_pack", "any2_dequant", "any2_gemm",
           "any3_packed_bytes", "any3_pack", "any3_dequant", "any3_gemm", "any4_read_probe",
           "any4_lora_plan_bytes", "any4_lora_plan", "any4_lora_workspace_size", "any4_lora",
           "any4_lora_backward_workspace_size", "any4_lora_backward", "any4_act8_save",
           "any4_act8_load", "any4_gemm_dx_workspace_size", "any4_gemm_dx", "any4_gemm_int4_dx",
           "any2_gemm_dx", "any3_gemm_dx")

_lib = None


class Any4Error(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libany4.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "or python -m gemm_any4_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
        L.any4_packed_bytes.restype = SZ
        L.any4_packed_bytes.argtypes = [I64, I64]
        L.any4_pack.restype = ctypes.c_int
        L.any4_pack.argtypes = [P, P, I64, I64, P]
        L.any4_dequant.restype = ctypes.c_int
        L.any4_dequant.argtypes = [P, P, P, P, P, I64, I64, I64, P]
        L.any4_gemm_workspace_size.restype = SZ
        L.any4_gemm_workspace_size.argtypes = [I64, I64, I64, I64]
        L.any4_gemm.restype = ctypes.c_int
        L.any4_gemm.argtypes = [P, P, P, P, P, P, I64, I64, I64, I64, P, SZ, P]
        L.any4_gemm_noalloc.restype = ctypes.c_int
        L.any4_gemm_noalloc.argtypes = [P, P, P, P, P, P, I64, I64, I64, I64, P]
        L.any4_gemv_dot.restype = ctypes.c_int
        L.any4_gemv_dot.argtypes = [P, P, P, P, P, P, I64, I64, I64, P]
        L.any4_gemm_int4.restype = ctypes.c_int
        L.any4_gemm_int4.argtypes = [P, P, P, P, P, I64, I64, I64, I64, P, SZ, P]
        L.any4_quantize.restype = ctypes.c_int
        L.any4_quantize.argtypes = [P, P, P, P, P, P, I64, I64, I64, ctypes.c_int, ctypes.c_int, P]
        for v in ("any2", "any3"):
            getattr(L, v + "_packed_bytes").restype = SZ
            getattr(L, v + "_packed_bytes").argtypes = [I64, I64]
            getattr(L, v + "_pack").restype = ctypes.c_int
            getattr(L, v + "_pack").argtypes = [P, P, I64, I64, P]
            getattr(L, v + "_dequant").restype = ctypes.c_int
            getattr(L, v + "_dequant").argtypes = [P, P, P, P, P, I64, I64, I64, P]
            getattr(L, v + "_gemm").restype = ctypes.c_int
            getattr(L, v + "_gemm").argtypes = [P, P, P, P, P, P, I64, I64, I64, I64, P, SZ, P]
        for name, restype, argtypes in (
                ("any4_lora_plan_bytes", SZ, [I64] * 2),
                ("any4_lora_plan", ctypes.c_int, [P, P, SZ, I64, I64, P]),
                ("any4_lora_workspace_size", SZ, [I64] * 5),
                ("any4_lora", ctypes.c_int, [P] * 11 + [I64] * 5 + [P, SZ, P]),
                ("any4_lora_backward_workspace_size", SZ, [I64] * 5),
                ("any4_lora_backward", ctypes.c_int, [P] * 14 + [I64] * 5 + [P, SZ, P]),
                ("any4_act8_save", ctypes.c_int, [P] * 3 + [I64] * 2 + [P]),
                ("any4_act8_load", ctypes.c_int, [P] * 3 + [I64] * 2 + [P]),
                ("any4_gemm_dx_workspace_size", SZ, [I64] * 4),
                ("any4_gemm_dx", ctypes.c_int, [P] * 6 + [I64] * 4 + [P, SZ, P]),
                ("any4_gemm_int4_dx", ctypes.c_int, [P] * 5 + [I64] * 4 + [P, SZ, P]),
                ("any2_gemm_dx", ctypes.c_int, [P] * 6 + [I64] * 4 + [P, SZ, P]),
                ("any3_gemm_dx", ctypes.c_int, [P] * 6 + [I64] * 4 + [P, SZ, P])):
            getattr(L, name).restype = restype
            getattr(L, name).argtypes = argtypes
        L.any4_read_probe.restype = ctypes.c_int
        L.any4_read_probe.argtypes = [P, SZ, P, P]
        L.any4_status_string.restype = ctypes.c_char_p
        L.any4_status_string.argtypes = [ctypes.c_int]
        _lib = L
    return _lib


def status_string(s: int) -> str:
    return lib().any4_status_string(s).decode()


def check(s: int) -> None:
    if s != ANY4_OK:
        raise Any4Error(s, status_string(s))


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None or t.numel() == 0:
        return None
    return t.data_ptr()


def _u8(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype != torch.uint8:
        raise TypeError(f"{name} must be uint8, got {t.dtype}")
    return _dev(t, name)


def _b16(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"{name} must be bfloat16 (or 16-bit bit patterns), got {t.dtype}")
    return _dev(t, name)


def _dev(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


# --------------------------------------------------------------------------
# raw C-ABI calls (device pointers as ints)
# --------------------------------------------------------------------------
def pack_raw(idx_ptr, packed_ptr, N, K, stream=None) -> int:
    return lib().any4_pack(idx_ptr, packed_ptr, N, K, _stream(stream))


def dequant_raw(packed_ptr, lut_ptr, alpha_ptr, beta_ptr, w_ptr, N, K, g, stream=None) -> int:
    return lib().any4_dequant(packed_ptr, lut_ptr, alpha_ptr, beta_ptr, w_ptr, N, K, g,
                              _stream(stream))


def workspace_size(M: int, N: int, K: int, g: int) -> int:
    return int(lib().any4_gemm_workspace_size(M, N, K, g))


def packed_bytes(N: int, K: int) -> int:
    return int(lib().any4_packed_bytes(N, K))


def gemm_raw(x_ptr, packed_ptr, lut_ptr, alpha_ptr, beta_ptr, y_ptr, M, N, K, g,
             ws_ptr=None, ws_bytes=0, stream=None) -> int:
    return lib().any4_gemm(x_ptr, packed_ptr, lut_ptr, alpha_ptr, beta_ptr, y_ptr, M, N, K, g,
                           ws_ptr, ws_bytes, _stream(stream))


def gemm_noalloc_raw(x_ptr, packed_ptr, lut_ptr, alpha_ptr, beta_ptr, y_ptr, M, N, K, g,
                     stream=None) -> int:
    return lib().any4_gemm_noalloc(x_ptr, packed_ptr, lut_ptr, alpha_ptr, beta_ptr, y_ptr, M,
                                   N, K, g, _stream(stream))


def gemv_dot_raw(x_ptr, packed_ptr, lut_ptr, alpha_ptr, beta_ptr, y_ptr, N, K, g,
                 stream=None) -> int:
    return lib().any4_gemv_dot(x_ptr, packed_ptr, lut_ptr, alpha_ptr, beta_ptr, y_ptr, N, K, g,
                               _stream(stream))


def gemv_dot(x: torch.Tensor, packed: torch.Tensor, lut: torch.Tensor, alpha: torch.Tensor,
             beta: torch.Tensor, g: int, out: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
    """y [1, N] = x [1, K] * W^T on the vector ALUs (v_dot2) instead of the
    matrix cores: the same product as gemm at M = 1, for comparison."""
    _b16(x, "x"), _b16(lut, "lut"), _b16(alpha, "alpha"), _b16(beta, "beta")
    if x.dim() != 2 or x.shape[0] != 1:
        raise ValueError("x must be [1, K]")
    K = x.shape[1]
    N = lut.shape[0]
    if g <= 0 or K % g or alpha.shape != (N, K // g) or beta.shape != (N, K // g):
        raise ValueError("alpha/beta must be [N, K/g]")
    _check_packed(packed, N, K)
    if out is None:
        out = torch.empty((1, N), dtype=torch.bfloat16, device=x.device)
    _b16(out, "y")
    check(gemv_dot_raw(_ptr(x), _ptr(packed), _ptr(lut), _ptr(alpha), _ptr(beta), _ptr(out),
                       N, K, g, stream))
    return out


def gemm_int4_raw(x_ptr, packed_ptr, alpha_ptr, beta_ptr, y_ptr, M, N, K, g,
                  ws_ptr=None, ws_bytes=0, stream=None) -> int:
    return lib().any4_gemm_int4(x_ptr, packed_ptr, alpha_ptr, beta_ptr, y_ptr, M, N, K, g,
                                ws_ptr, ws_bytes, _stream(stream))


def quantize_raw(w_ptr, ex_ptr, idx_ptr, lut_ptr, alpha_ptr, beta_ptr, N, K, g, iters,
                 bits=4, stream=None) -> int:
    return lib().any4_quantize(w_ptr, ex_ptr, idx_ptr, lut_ptr, alpha_ptr, beta_ptr, N, K, g,
                               iters, bits, _stream(stream))


# --------------------------------------------------------------------------
# tensor API
# --------------------------------------------------------------------------
def pack(idx: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """idx uint8 [N, K] -> packed uint8 [packed_bytes(N, K)] (tile layout)."""
    _u8(idx, "idx")
    N, K = idx.shape
    nbytes = packed_bytes(N, K)
    if K % 128:
        raise ValueError("K must be a multiple of 128")
    if out is None:
        out = torch.empty((nbytes,), dtype=torch.uint8, device=idx.device)
    _u8(out, "packed")
    if out.numel() != nbytes:
        raise ValueError(f"packed must hold {nbytes} bytes")
    check(pack_raw(_ptr(idx), _ptr(out), N, K, stream))
    return out


def _check_packed(packed: torch.Tensor, N: int, K: int) -> None:
    _u8(packed, "packed")
    if packed.numel() != packed_bytes(N, K):
        raise ValueError(f"packed must hold packed_bytes({N}, {K}) = {packed_bytes(N, K)} bytes")


def dequant(packed: torch.Tensor, lut: torch.Tensor, alpha: torch.Tensor, beta: torch.Tensor,
            g: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Materialise the bf16 weights w [N, K] (N from lut, K = alpha.shape[1] * g)."""
    _b16(lut, "lut"), _b16(alpha, "alpha"), _b16(beta, "beta")
    if lut.dim() != 2 or lut.shape[1] != 16:
        raise ValueError("lut must be [N, 16]")
    N = lut.shape[0]
    if g <= 0 or alpha.dim() != 2 or alpha.shape[0] != N or beta.shape != alpha.shape:
        raise ValueError("alpha/beta must be [N, K/g]")
    K = alpha.shape[1] * g
    _check_packed(packed, N, K)
    if out is None:
        out = torch.empty((N, K), dtype=torch.bfloat16, device=lut.device)
    _b16(out, "w")
    if out.shape != (N, K):
        raise ValueError("w must be [N, K]")
    check(dequant_raw(_ptr(packed), _ptr(lut), _ptr(alpha), _ptr(beta), _ptr(out), N, K, g,
                      stream))
    return out


# One workspace per (device, stream), grown on demand: calls on one stream run
# one after another, so they can share it.  The kernels write every partial
# sum before they read it, so it needs no initialisation.
_workspaces: dict = {}


def _workspace(need: int, device: torch.device, stream_handle: int) -> torch.Tensor:
    key = (device.index, stream_handle)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.empty(max(need, 1 << 16), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def gemm(x: torch.Tensor, packed: torch.Tensor, lut: torch.Tensor, alpha: torch.Tensor,
         beta: torch.Tensor, g: int, out: torch.Tensor | None = None,
         workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [M, N] = x [M, K] * W^T with W the any4 weights (N from lut).

    workspace: optional uint8 device tensor of at least workspace_size(M, N, K, g)
    bytes (contents need not be initialised); with it, K may be split over
    workgroups, their fp32 partial sums kept there, or (M >= 128) the layer is
    dequantised into it for one library bf16 GEMM.  An empty tensor runs the
    kernels that need no workspace.  By default a workspace kept per device
    and stream is used."""
    _b16(x, "x"), _b16(lut, "lut"), _b16(alpha, "alpha"), _b16(beta, "beta")
    M, K = x.shape
    if lut.dim() != 2 or lut.shape[1] != 16:
        raise ValueError("lut must be [N, 16]")
    N = lut.shape[0]
    if g <= 0 or K % g or alpha.shape != (N, K // g) or beta.shape != (N, K // g):
        raise ValueError("alpha/beta must be [N, K/g]")
    _check_packed(packed, N, K)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _b16(out, "y")
    if out.shape != (M, N):
        raise ValueError("y must be [M, N]")
    sh = _stream(stream)
    ws_ptr, ws_bytes = _workspace_args(workspace, M, N, K, g, x.device, sh)
    check(gemm_raw(_ptr(x), _ptr(packed), _ptr(lut), _ptr(alpha), _ptr(beta), _ptr(out), M, N, K,
                   g, ws_ptr, ws_bytes, sh))
    return out


def _workspace_args(workspace, M: int, N: int, K: int, g: int, device, sh):
    """(pointer, bytes) of the workspace for a GEMM call (split-K partial sums,
    or the dequantised layer for prefill batches): the caller's
    tensor (an empty one: none), else the cached one of this device and
    stream, or (None, 0) where the shape needs none."""
    need = workspace_size(M, N, K, g)
    if not need:
        return None, 0
    if workspace is None:
        workspace = _workspace(need, device, sh)
    if not workspace.numel():
        return None, 0
    _dev(workspace, "workspace")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def gemm_int4(x: torch.Tensor, packed: torch.Tensor, alpha: torch.Tensor, beta: torch.Tensor,
              g: int, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """y [M, N] = x [M, K] * W^T with plain int4 weights w = alpha * q + beta
    (q the 4-bit code, 0..15; N from alpha).  workspace as for gemm()."""
    _b16(x, "x"), _b16(alpha, "alpha"), _b16(beta, "beta")
    M, K = x.shape
    if g <= 0 or K % g or alpha.dim() != 2 or alpha.shape[1] != K // g or beta.shape != alpha.shape:
        raise ValueError("alpha/beta must be [N, K/g]")
    N = alpha.shape[0]
    _check_packed(packed, N, K)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _b16(out, "y")
    if out.shape != (M, N):
        raise ValueError("y must be [M, N]")
    sh = _stream(stream)
    ws_ptr, ws_bytes = _workspace_args(workspace, M, N, K, g, x.device, sh)
    check(gemm_int4_raw(_ptr(x), _ptr(packed), _ptr(alpha), _ptr(beta), _ptr(out), M, N, K, g,
                        ws_ptr, ws_bytes, sh))
    return out


def quantize(W: torch.Tensor, ex: torch.Tensor, g: int, iters: int = 10, bits: int = 4,
             stream=None):
    """any4-quantise W fp32 [N, K] with channel importance ex fp32 [K] (E|x|);
    bits = 3 or 2 for any3 / any2 (8 or 4 table values, indices below them).

    Returns (idx uint8 [N, K], lut bf16 [N, 16], alpha bf16 [N, K/g],
    beta bf16 [N, K/g]); pack idx with pack() before gemm()."""
    for t, name in ((W, "W"), (ex, "ex")):
        if t.dtype != torch.float32:
            raise TypeError(f"{name} must be float32, got {t.dtype}")
        _dev(t, name)
    N, K = W.shape
    if ex.shape != (K,):
        raise ValueError("ex must be [K]")
    if g <= 0 or K % g:
        raise ValueError("g must divide K")
    dev = W.device
    idx = torch.empty((N, K), dtype=torch.uint8, device=dev)
    lut = torch.empty((N, 16), dtype=torch.bfloat16, device=dev)
    alpha = torch.empty((N, K // g), dtype=torch.bfloat16, device=dev)
    beta = torch.empty((N, K // g), dtype=torch.bfloat16, device=dev)
    check(quantize_raw(_ptr(W), _ptr(ex), _ptr(idx), _ptr(lut), _ptr(alpha), _ptr(beta), N, K, g,
                       iters, bits, stream))
    return idx, lut, alpha, beta


# --------------------------------------------------------------------------
# any2 (2-bit codes, four per byte) and any3 (3-bit codes, 12 bytes per 32):
# tile layouts in include/any4.h
# --------------------------------------------------------------------------
def any2_packed_bytes(N: int, K: int) -> int:
    return int(lib().any2_packed_bytes(N, K))


def any3_packed_bytes(N: int, K: int) -> int:
    return int(lib().any3_packed_bytes(N, K))


def any2_pack_raw(idx_ptr, packed_ptr, N, K, stream=None) -> int:
    return lib().any2_pack(idx_ptr, packed_ptr, N, K, _stream(stream))


def any3_pack_raw(idx_ptr, packed_ptr, N, K, stream=None) -> int:
    return lib().any3_pack(idx_ptr, packed_ptr, N, K, _stream(stream))


def any2_dequant_raw(packed_ptr, lut_ptr, alpha_ptr, beta_ptr, w_ptr, N, K, g,
                     stream=None) -> int:
    return lib().any2_dequant(packed_ptr, lut_ptr, alpha_ptr, beta_ptr, w_ptr, N, K, g,
                              _stream(stream))


def any3_dequant_raw(packed_ptr, lut_ptr, alpha_ptr, beta_ptr, w_ptr, N, K, g,
                     stream=None) -> int:
    return lib().any3_dequant(packed_ptr, lut_ptr, alpha_ptr, beta_ptr, w_ptr, N, K, g,
                              _stream(stream))


def any2_gemm_raw(x_ptr, packed_ptr, lut_ptr, alpha_ptr, beta_ptr, y_ptr, M, N, K, g,
                  ws_ptr=None, ws_bytes=0, stream=None) -> int:
    return lib().any2_gemm(x_ptr, packed_ptr, lut_ptr, alpha_ptr, beta_ptr, y_ptr, M, N, K, g,
                           ws_ptr, ws_bytes, _stream(stream))


def any3_gemm_raw(x_ptr, packed_ptr, lut_ptr, alpha_ptr, beta_ptr, y_ptr, M, N, K, g,
                  ws_ptr=None, ws_bytes=0, stream=None) -> int:
    return lib().any3_gemm(x_ptr, packed_ptr, lut_ptr, alpha_ptr, beta_ptr, y_ptr, M, N, K, g,
                           ws_ptr, ws_bytes, _stream(stream))


_LOWBIT = {2: (any2_packed_bytes, any2_pack_raw, any2_dequant_raw, any2_gemm_raw),
           3: (any3_packed_bytes, any3_pack_raw, any3_dequant_raw, any3_gemm_raw)}


def _lowbit_pack(bits: int, idx: torch.Tensor, out, stream) -> torch.Tensor:
    nbytes_of, pack_raw_, _, _ = _LOWBIT[bits]
    _u8(idx, "idx")
    N, K = idx.shape
    if K % 128:
        raise ValueError("K must be a multiple of 128")
    nbytes = nbytes_of(N, K)
    if out is None:
        out = torch.empty((nbytes,), dtype=torch.uint8, device=idx.device)
    _u8(out, "packed")
    if out.numel() != nbytes:
        raise ValueError(f"packed must hold {nbytes} bytes")
    check(pack_raw_(_ptr(idx), _ptr(out), N, K, stream))
    return out


def _check_lowbit_packed(bits: int, packed: torch.Tensor, N: int, K: int) -> None:
    _u8(packed, "packed")
    if packed.numel() != _LOWBIT[bits][0](N, K):
        raise ValueError(f"packed must hold any{bits}_packed_bytes({N}, {K}) bytes")


def _lowbit_dequant(bits: int, packed, lut, alpha, beta, g: int, out, stream) -> torch.Tensor:
    _b16(lut, "lut"), _b16(alpha, "alpha"), _b16(beta, "beta")
    if lut.dim() != 2 or lut.shape[1] != 16:
        raise ValueError("lut must be [N, 16]")
    N = lut.shape[0]
    if g <= 0 or alpha.dim() != 2 or alpha.shape[0] != N or beta.shape != alpha.shape:
        raise ValueError("alpha/beta must be [N, K/g]")
    K = alpha.shape[1] * g
    _check_lowbit_packed(bits, packed, N, K)
    if out is None:
        out = torch.empty((N, K), dtype=torch.bfloat16, device=lut.device)
    _b16(out, "w")
    if out.shape != (N, K):
        raise ValueError("w must be [N, K]")
    check(_LOWBIT[bits][2](_ptr(packed), _ptr(lut), _ptr(alpha), _ptr(beta), _ptr(out), N, K, g,
                           stream))
    return out


def _lowbit_gemm(bits: int, x, packed, lut, alpha, beta, g: int, out, workspace,
                 stream) -> torch.Tensor:
    _b16(x, "x"), _b16(lut, "lut"), _b16(alpha, "alpha"), _b16(beta, "beta")
    M, K = x.shape
    if lut.dim() != 2 or lut.shape[1] != 16:
        raise ValueError("lut must be [N, 16]")
    N = lut.shape[0]
    if g <= 0 or K % g or alpha.shape != (N, K // g) or beta.shape != (N, K // g):
        raise ValueError("alpha/beta must be [N, K/g]")
    _check_lowbit_packed(bits, packed, N, K)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _b16(out, "y")
    if out.shape != (M, N):
        raise ValueError("y must be [M, N]")
    sh = _stream(stream)
    ws_ptr, ws_bytes = _workspace_args(workspace, M, N, K, g, x.device, sh)
    check(_LOWBIT[bits][3](_ptr(x), _ptr(packed), _ptr(lut), _ptr(alpha), _ptr(beta), _ptr(out),
                           M, N, K, g, ws_ptr, ws_bytes, sh))
    return out


def any2_pack(idx: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """idx uint8 [N, K] (codes 0..3) -> packed uint8 [any2_packed_bytes(N, K)]."""
    return _lowbit_pack(2, idx, out, stream)


def any3_pack(idx: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """idx uint8 [N, K] (codes 0..7) -> packed uint8 [any3_packed_bytes(N, K)]."""
    return _lowbit_pack(3, idx, out, stream)


def any2_dequant(packed: torch.Tensor, lut: torch.Tensor, alpha: torch.Tensor,
                 beta: torch.Tensor, g: int, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """bf16 weights [N, K] of an any2 layer (N from lut, K = alpha.shape[1] * g)."""
    return _lowbit_dequant(2, packed, lut, alpha, beta, g, out, stream)


def any3_dequant(packed: torch.Tensor, lut: torch.Tensor, alpha: torch.Tensor,
                 beta: torch.Tensor, g: int, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """bf16 weights [N, K] of an any3 layer (N from lut, K = alpha.shape[1] * g)."""
    return _lowbit_dequant(3, packed, lut, alpha, beta, g, out, stream)


def any2_gemm(x: torch.Tensor, packed: torch.Tensor, lut: torch.Tensor, alpha: torch.Tensor,
              beta: torch.Tensor, g: int, out: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [M, N] = x [M, K] * W^T with W an any2 layer (N from lut); workspace
    as for gemm()."""
    return _lowbit_gemm(2, x, packed, lut, alpha, beta, g, out, workspace, stream)


def any3_gemm(x: torch.Tensor, packed: torch.Tensor, lut: torch.Tensor, alpha: torch.Tensor,
              beta: torch.Tensor, g: int, out: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [M, N] = x [M, K] * W^T with W an any3 layer (N from lut); workspace
    as for gemm()."""
    return _lowbit_gemm(3, x, packed, lut, alpha, beta, g, out, workspace, stream)


# --------------------------------------------------------------------------
# fine-tunes of a layer: adapters, activations in 8 bits, the input's gradient
# --------------------------------------------------------------------------
def lora_plan_raw(ids_ptr, plan_ptr, nbytes, M, L, stream=None) -> int:
    return lib().any4_lora_plan(ids_ptr, plan_ptr, nbytes, M, L, _stream(stream))


def lora_raw(x_ptr, A_ptr, B_ptr, scale_ptr, ids_ptr, plan_ptr, y_ptr, out_ptr, h_ptr, q_ptr,
             qs_ptr, M, N, K, r, L, ws_ptr, ws_bytes, stream=None) -> int:
    return lib().any4_lora(x_ptr, A_ptr, B_ptr, scale_ptr, ids_ptr, plan_ptr, y_ptr, out_ptr,
                           h_ptr, q_ptr, qs_ptr, M, N, K, r, L, ws_ptr, ws_bytes, _stream(stream))


def lora_backward_raw(dy_ptr, x_ptr, q_ptr, qs_ptr, h_ptr, A_ptr, B_ptr, scale_ptr, ids_ptr,
                      plan_ptr, dx_ptr, dx_out_ptr, dA_ptr, dB_ptr, M, N, K, r, L, ws_ptr,
                      ws_bytes, stream=None) -> int:
    return lib().any4_lora_backward(dy_ptr, x_ptr, q_ptr, qs_ptr, h_ptr, A_ptr, B_ptr, scale_ptr,
                                    ids_ptr, plan_ptr, dx_ptr, dx_out_ptr, dA_ptr, dB_ptr, M, N,
                                    K, r, L, ws_ptr, ws_bytes, _stream(stream))


def act8_save_raw(x_ptr, q_ptr, qs_ptr, M, K, stream=None) -> int:
    return lib().any4_act8_save(x_ptr, q_ptr, qs_ptr, M, K, _stream(stream))


def act8_load_raw(q_ptr, qs_ptr, x_ptr, M, K, stream=None) -> int:
    return lib().any4_act8_load(q_ptr, qs_ptr, x_ptr, M, K, _stream(stream))


def gemm_dx_raw(dy_ptr, packed_ptr, lut_ptr, alpha_ptr, beta_ptr, dx_ptr, M, N, K, g, ws_ptr,
                ws_bytes, stream=None, call="any4_gemm_dx") -> int:
    """call: "any4_gemm_dx", "any2_gemm_dx" or "any3_gemm_dx"."""
    return getattr(lib(), call)(dy_ptr, packed_ptr, lut_ptr, alpha_ptr, beta_ptr, dx_ptr, M, N, K,
                                g, ws_ptr, ws_bytes, _stream(stream))


def gemm_int4_dx_raw(dy_ptr, packed_ptr, alpha_ptr, beta_ptr, dx_ptr, M, N, K, g, ws_ptr, ws_bytes,
                     stream=None) -> int:
    return lib().any4_gemm_int4_dx(dy_ptr, packed_ptr, alpha_ptr, beta_ptr, dx_ptr, M, N, K, g,
                                   ws_ptr, ws_bytes, _stream(stream))


@functools.lru_cache(maxsize=4096)      # constant for its sizes
def lora_plan_bytes(M: int, L: int) -> int:
    return int(lib().any4_lora_plan_bytes(M, L))


@functools.lru_cache(maxsize=4096)      # constant for its sizes
def lora_workspace_size(M: int, N: int, K: int, r: int, L: int) -> int:
    return int(lib().any4_lora_workspace_size(M, N, K, r, L))


@functools.lru_cache(maxsize=4096)      # constant for its sizes
def lora_backward_workspace_size(M: int, N: int, K: int, r: int, L: int) -> int:
    return int(lib().any4_lora_backward_workspace_size(M, N, K, r, L))


@functools.lru_cache(maxsize=4096)      # constant for its sizes
def gemm_dx_workspace_size(M: int, N: int, K: int, g: int) -> int:
    return int(lib().any4_gemm_dx_workspace_size(M, N, K, g))


_HERE_AND_NOW = contextlib.nullcontext()

# the handle of a device's current stream; without the Stream object that
# torch.cuda.current_stream makes of it where torch has the shorter way (1.9 us
# of a call's 15)
_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(device: torch.device, stream):
    """A context in which `device` is current and `stream` (None: the device's
    current one) its current stream: what is allocated within belongs to the
    stream that the kernels run on."""
    if stream is None:
        if device.index == torch.cuda.current_device():
            return _HERE_AND_NOW
        return torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device) if handle else \
            torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"stream is of {stream.device}, the tensors are on {device}")
    return torch.cuda.stream(stream)


def _tensor(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device) -> int | None:
    """Checks one argument; its address."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr() or None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be a GPU tensor on {device}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _gpu(t: torch.Tensor, name: str, dims: int) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions")
    return t.device


def _scratch(workspace, need: int, device) -> tuple:
    """(tensor, address, bytes) of a workspace: the caller's, or one of this
    call (the allocator hands its memory on in stream order, and a graph under
    capture keeps it to itself)."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous GPU tensor on {device}")
    return workspace, workspace.data_ptr() or None, workspace.numel() * workspace.element_size()


class LoraPlan(NamedTuple):
    """Rows of a batch sorted by adapter (lora_plan): for M rows and L adapters."""
    words: torch.Tensor
    M: int
    L: int


def lora_plan(ids: torch.Tensor, L: int, stream=None) -> LoraPlan:
    """The rows of a batch by adapter, for the lora calls of every layer that
    the batch goes through: ids int32 [M], the adapter of each row (outside
    0..L-1: none).  The plan holds for these ids; calls that get none make it
    themselves, each time."""
    dev = _gpu(ids, "ids", 1)
    M = ids.shape[0]
    p_ids = _tensor(ids, "ids", torch.int32, (M,), dev)
    nbytes = lora_plan_bytes(M, L)
    with _on(dev, stream):
        words = torch.empty(nbytes // 4, dtype=torch.int32, device=dev)
        check(lora_plan_raw(p_ids, _ptr(words), nbytes, M, L))
    return LoraPlan(words, M, L)


def _plan_ptr(plan, M: int, L: int, device):
    if plan is None:
        return None
    if not isinstance(plan, LoraPlan):
        raise TypeError("plan must come from lora_plan()")
    if plan.M != M or plan.L != L or plan.words.device != device:
        raise ValueError(f"plan is for M = {plan.M}, L = {plan.L} on {plan.words.device}, "
                         f"the call for M = {M}, L = {L} on {device}")
    return _ptr(plan.words)


def _adapters(A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor, dev, K: int, N: int) -> tuple:
    if A.dim() != 3:
        raise ValueError("A must be [L, r, K]")
    L, r = A.shape[0], A.shape[1]
    return (L, r, _tensor(A, "A", torch.bfloat16, (L, r, K), dev),
            _tensor(B, "B", torch.bfloat16, (L, r, N), dev),
            _tensor(scale, "scale", torch.float32, (L,), dev))


def lora(x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor,
         ids: torch.Tensor, y: torch.Tensor, out: torch.Tensor | None = None,
         h: torch.Tensor | None = None, act: tuple | None = None, plan: LoraPlan | None = None,
         workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out [M, N] = y + scale[a] * (x A_a^T) B_a with a = ids[m], the adapters
    of many requests beside the projection y of x (from gemm, any2_gemm, ...).

    x bf16 [M, K]; A bf16 [L, r, K]; B bf16 [L, r, N] (the transpose of the
    usual [N, r]); scale fp32 [L]; ids int32 [M], outside 0..L-1: no adapter.
    out may be y.  For the backward pass: h fp32 [M, r] gets x A_a^T, and
    act = (q, qs) of act8_empty(x) gets x in 8 bits.
    plan: of lora_plan(ids, L), kept over the layers of a batch."""
    dev = _gpu(x, "x", 2)
    M, K = x.shape
    if y.dim() != 2:
        raise ValueError("y must be [M, N]")
    N = y.shape[1]
    bf16 = torch.bfloat16
    L, r, p_A, p_B, p_scale = _adapters(A, B, scale, dev, K, N)
    p_x, p_y = _tensor(x, "x", bf16, (M, K), dev), _tensor(y, "y", bf16, (M, N), dev)
    p_ids = _tensor(ids, "ids", torch.int32, (M,), dev)
    p_h = None if h is None else _tensor(h, "h", torch.float32, (M, r), dev)
    p_q = p_qs = None
    if act is not None:
        p_q = _tensor(act[0], "q", torch.int8, (M, K), dev)
        p_qs = _tensor(act[1], "qs", torch.float32, (M, K // 128), dev)
    p_plan = _plan_ptr(plan, M, L, dev)
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(y)
            p_out = _ptr(out)
        else:
            p_out = _tensor(out, "out", bf16, (M, N), dev)
        ws, p_ws, nbytes = _scratch(workspace, lora_workspace_size(M, N, K, r, L), dev)
        check(lib().any4_lora(p_x, p_A, p_B, p_scale, p_ids, p_plan, p_y, p_out, p_h, p_q, p_qs, M, N,
                              K, r, L, p_ws, nbytes, _current_handle(dev.index)))
    return out


def gemm_lora(x: torch.Tensor, packed: torch.Tensor, lut: torch.Tensor, alpha: torch.Tensor,
              beta: torch.Tensor, g: int, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor,
              ids: torch.Tensor, out: torch.Tensor | None = None, h: torch.Tensor | None = None,
              act: tuple | None = None, plan: LoraPlan | None = None,
              stream=None) -> torch.Tensor:
    """An any4 layer with the adapters of its requests: gemm, then lora in
    place on its output (so the projection is rounded to bf16 once more)."""
    dev = _gpu(x, "x", 2)
    with _on(dev, stream):
        ws = None
        if torch.cuda.is_current_stream_capturing():     # a graph keeps its workspace to itself
            need = workspace_size(x.shape[0], lut.shape[0], x.shape[1], g)
            ws = torch.empty(need, dtype=torch.uint8, device=dev)
        y = gemm(x, packed, lut, alpha, beta, g, out=out, workspace=ws)
        return lora(x, A, B, scale, ids, y, out=y, h=h, act=act, plan=plan)


def lora_backward(dy: torch.Tensor, x: torch.Tensor, h: torch.Tensor, A: torch.Tensor,
                  B: torch.Tensor, scale: torch.Tensor, ids: torch.Tensor,
                  dx: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  x_scale: torch.Tensor | None = None, dA: torch.Tensor | None = None,
                  dB: torch.Tensor | None = None, need_dx: bool = True,
                  plan: LoraPlan | None = None, workspace: torch.Tensor | None = None,
                  stream=None) -> tuple:
    """(dx', dA, dB) of lora() for dy bf16 [M, N]: the gradients with respect
    to x (dx' bf16 [M, K] = dx + the adapters' part, dx the projection's own
    from gemm_dx or None for zero), A (fp32 [L, r, K]) and B (fp32 [L, r, N]).
    The gradient of y is dy itself.

    x: the bf16 input, or its q int8 with x_scale = qs (act8_save, or lora's
    act); h as lora() wrote it.  out (may be dx), dA, dB: where the results go;
    need_dx = False leaves dx' out (None)."""
    dev = _gpu(dy, "dy", 2)
    M, N = dy.shape
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    K = x.shape[1]
    bf16, f32 = torch.bfloat16, torch.float32
    L, r, p_A, p_B, p_scale = _adapters(A, B, scale, dev, K, N)
    p_dy = _tensor(dy, "dy", bf16, (M, N), dev)
    p_x = p_q = p_qs = None
    if x_scale is None:
        p_x = _tensor(x, "x", bf16, (M, K), dev)
    else:
        p_q = _tensor(x, "x", torch.int8, (M, K), dev)
        p_qs = _tensor(x_scale, "x_scale", f32, (M, K // 128), dev)
    p_h, p_ids = _tensor(h, "h", f32, (M, r), dev), _tensor(ids, "ids", torch.int32, (M,), dev)
    p_dx = None if dx is None else _tensor(dx, "dx", bf16, (M, K), dev)
    p_plan = _plan_ptr(plan, M, L, dev)
    with _on(dev, stream):
        if not need_dx:
            out = None
        elif out is None:
            out = torch.empty((M, K), dtype=bf16, device=dev)
        dA = torch.empty((L, r, K), dtype=f32, device=dev) if dA is None else dA
        dB = torch.empty((L, r, N), dtype=f32, device=dev) if dB is None else dB
        p_out = None if out is None else _tensor(out, "out", bf16, (M, K), dev)
        p_dA, p_dB = _tensor(dA, "dA", f32, (L, r, K), dev), _tensor(dB, "dB", f32, (L, r, N), dev)
        ws, p_ws, nbytes = _scratch(workspace, lora_backward_workspace_size(M, N, K, r, L), dev)
        check(lib().any4_lora_backward(p_dy, p_x, p_q, p_qs, p_h, p_A, p_B, p_scale, p_ids, p_plan,
                                       p_dx, p_out, p_dA, p_dB, M, N, K, r, L, p_ws, nbytes,
                                       _current_handle(dev.index)))
    return out, dA, dB


def act8_empty(x: torch.Tensor) -> tuple:
    """(q int8 [M, K], qs fp32 [M, K/128]): room for x in 8 bits."""
    M, K = x.shape
    if K % 128:
        raise ValueError("K must be a multiple of 128")
    return (torch.empty((M, K), dtype=torch.int8, device=x.device),
            torch.empty((M, K // 128), dtype=torch.float32, device=x.device))


def act8_save(x: torch.Tensor, act: tuple | None = None, stream=None) -> tuple:
    """x bf16 [M, K] in 8 bits: (q int8 [M, K], qs fp32 [M, K/128]), one scale
    per 128 channels of a row (include/any4.h has the exact definition)."""
    dev = _gpu(x, "x", 2)
    M, K = x.shape
    p_x = _tensor(x, "x", torch.bfloat16, (M, K), dev)
    with _on(dev, stream):
        if act is None:
            q, qs = act8_empty(x)
            p_q, p_qs = q.data_ptr() or None, qs.data_ptr() or None
        else:
            q, qs = act
            p_q = _tensor(q, "q", torch.int8, (M, K), dev)
            p_qs = _tensor(qs, "qs", torch.float32, (M, K // 128), dev)
        check(lib().any4_act8_save(p_x, p_q, p_qs, M, K, _current_handle(dev.index)))
    return q, qs


def act8_load(q: torch.Tensor, qs: torch.Tensor, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """The bf16 [M, K] values of an activation in 8 bits."""
    dev = _gpu(q, "q", 2)
    M, K = q.shape
    if K % 128:
        raise ValueError("K must be a multiple of 128")
    p_q = _tensor(q, "q", torch.int8, (M, K), dev)
    p_qs = _tensor(qs, "qs", torch.float32, (M, K // 128), dev)
    with _on(dev, stream):
        if out is None:
            out = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
            p_x = out.data_ptr() or None
        else:
            p_x = _tensor(out, "out", torch.bfloat16, (M, K), dev)
        check(lib().any4_act8_load(p_q, p_qs, p_x, M, K, _current_handle(dev.index)))
    return out


def _gemm_dx(call: str, nbytes_of, dy, packed, lut, alpha, beta, g: int, out, workspace,
             stream) -> torch.Tensor:
    dev = _gpu(dy, "dy", 2)
    M, N = dy.shape
    bf16 = torch.bfloat16
    if g <= 0 or alpha.dim() != 2:
        raise ValueError("alpha/beta must be [N, K/g]")
    G = alpha.shape[1]
    K = G * g
    p_dy = _tensor(dy, "dy", bf16, (M, N), dev)
    p_packed = _tensor(packed, "packed", torch.uint8, (nbytes_of(N, K),), dev)
    tables = [] if lut is None else [_tensor(lut, "lut", bf16, (N, 16), dev)]
    p_alpha = _tensor(alpha, "alpha", bf16, (N, G), dev)
    p_beta = _tensor(beta, "beta", bf16, (N, G), dev)
    with _on(dev, stream):
        if out is None:
            out = torch.empty((M, K), dtype=bf16, device=dev)
        p_out = _tensor(out, "out", bf16, (M, K), dev)
        ws, p_ws, nbytes = _scratch(workspace, gemm_dx_workspace_size(M, N, K, g), dev)
        check(getattr(lib(), call)(p_dy, p_packed, *tables, p_alpha, p_beta, p_out, M, N, K, g,
                                   p_ws, nbytes, _current_handle(dev.index)))
    return out


def gemm_dx(dy: torch.Tensor, packed: torch.Tensor, lut: torch.Tensor, alpha: torch.Tensor,
            beta: torch.Tensor, g: int, out: torch.Tensor | None = None,
            workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dx [M, K] = dy [M, N] * W, the gradient of gemm()'s x (K = alpha.shape[1] * g)."""
    return _gemm_dx("any4_gemm_dx", packed_bytes, dy, packed, lut, alpha, beta, g, out, workspace,
                    stream)


def gemm_int4_dx(dy: torch.Tensor, packed: torch.Tensor, alpha: torch.Tensor, beta: torch.Tensor,
                 g: int, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """dx [M, K] = dy [M, N] * W, the gradient of gemm_int4()'s x."""
    return _gemm_dx("any4_gemm_int4_dx", packed_bytes, dy, packed, None, alpha, beta, g, out,
                    workspace, stream)


def any2_gemm_dx(dy: torch.Tensor, packed: torch.Tensor, lut: torch.Tensor, alpha: torch.Tensor,
                 beta: torch.Tensor, g: int, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dx [M, K] = dy [M, N] * W, the gradient of any2_gemm()'s x."""
    return _gemm_dx("any2_gemm_dx", any2_packed_bytes, dy, packed, lut, alpha, beta, g, out,
                    workspace, stream)


def any3_gemm_dx(dy: torch.Tensor, packed: torch.Tensor, lut: torch.Tensor, alpha: torch.Tensor,
                 beta: torch.Tensor, g: int, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """dx [M, K] = dy [M, N] * W, the gradient of any3_gemm()'s x."""
    return _gemm_dx("any3_gemm_dx", any3_packed_bytes, dy, packed, lut, alpha, beta, g, out,
                    workspace, stream)


def read_probe_raw(buf_ptr, nbytes: int, out_ptr, stream=None) -> int:
    """The streaming-read probe (a measurement aid; see include/any4.h)."""
    return lib().any4_read_probe(buf_ptr, nbytes, out_ptr, _stream(stream))
