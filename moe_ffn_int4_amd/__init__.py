"""MI355X (gfx950) int4 Mixture-of-Experts feed-forward layer.

Thin ctypes binding over ``libmoe_int4.so`` (C ABI in ``include/moe_int4.h``).
This module only checks and marshals arguments: torch provides device memory
and the current HIP stream, and every step of the layer runs in the library's
HIP kernels. There is no fallback: if the library is missing, importing the
functions below raises.

    q, s = quantize_int4(w_fp32_cuda)                 # int4 group quantizer
    experts = Int4Experts.empty(E, d, h, dev)         # routed experts, tiled int4
    experts.quantize_expert(e, w1, w3, w2)            #   (fp32 weights on the GPU)
    shared = pack_shared(s1, s3, s2)                  # shared expert, tiled bf16
    y = forward(x, router_w, router_b, experts, shared, top_k)
    r = route(x, router_w, router_b, top_k)           # routing/dispatch only

The layer's steps are also there one by one with their gradients, on row-major bf16 weights:
``permute_rows``, ``grouped_matmul`` (``_dx``, ``_dw``), ``swiglu`` (``_backward``), ``combine``
(``_backward``), and dense layers, ``linear`` (``linear_dz``, ``linear_dx``, ``linear_dw``). Gated blocks
are one pass each way, ``grouped_gated`` and ``gated_linear`` (``_dz``), ``adamw`` steps many tensors at once, and
``grouped_matmul_int4`` and ``linear_int4`` multiply by int4 weights outside the layer.
They take no part in torch's autograd: results carry no graph, also where an argument requires
gradients, and a program calls the gradients' functions itself (or in its own
``torch.autograd.Function``).

Weights of ``forward`` live in the tiled layouts the kernels read (see include/moe_int4.h);
untile_int4 / untile_scales / untile_bf16 convert them back to row-major.
"""
from __future__ import annotations

import array
import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_int4.so")
GROUP = 128                 # default int4 quantization group
GROUPS = (128, 64, 32)      # supported int4 groups (weights per scale)
TILE = 128                  # columns of a weight tile
PATHS = {"auto": 0, "prefill": 1, "decode": 2, "hybrid": 3, "prefill_wide": 4}

MOE_OK = 0


class MoEError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{_status_string(status)} [{status}]: {detail}")


class _Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int64), ("E", ctypes.c_int64),
                ("h", ctypes.c_int64), ("top_k", ctypes.c_int32), ("group_size", ctypes.c_int32)]


class _Experts(ctypes.Structure):
    _fields_ = [("w1q", ctypes.c_void_p), ("w3q", ctypes.c_void_p), ("w2q", ctypes.c_void_p),
                ("w1s", ctypes.c_void_p), ("w3s", ctypes.c_void_p), ("w2s", ctypes.c_void_p)]


class _Shared(ctypes.Structure):
    _fields_ = [("s1", ctypes.c_void_p), ("s3", ctypes.c_void_p), ("s2", ctypes.c_void_p)]


class _ExpertsBf16(ctypes.Structure):
    _fields_ = [("w1", ctypes.c_void_p), ("w3", ctypes.c_void_p), ("w2", ctypes.c_void_p)]


class _ExpertsFp8(ctypes.Structure):
    _fields_ = [("w1q", ctypes.c_void_p), ("w3q", ctypes.c_void_p), ("w2q", ctypes.c_void_p),
                ("w1s", ctypes.c_void_p), ("w3s", ctypes.c_void_p), ("w2s", ctypes.c_void_p),
                ("act_ub", ctypes.c_float)]


class _AdamWHyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64),
                ("step_device", ctypes.c_void_p), ("lr_device", ctypes.c_void_p),
                ("grad_scale", ctypes.c_void_p), ("fine", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m moe_ffn_int4_amd.build` (hipcc, gfx950)")
        L = ctypes.CDLL(LIB_PATH)
        P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_last_error.argtypes = []
        L.moe_last_error.restype = ctypes.c_char_p
        L.moe_abi_version.restype = ctypes.c_int
        L.moe_device_check.restype = ctypes.c_int
        L.moe_hbm_read.argtypes = [P, i64, P, P]
        L.moe_hbm_read.restype = ctypes.c_int
        L.moe_hbm_read_sink_words.restype = ctypes.c_int
        L.moe_hbm_copy.argtypes = [P, P, i64, P]
        L.moe_hbm_copy.restype = ctypes.c_int
        L.moe_quantize_int4.argtypes = [P, i64, i64, i32, P, P, P]
        L.moe_quantize_int4.restype = ctypes.c_int
        L.moe_quantize_int4_tiled.argtypes = [P, i64, i64, i32, P, P, P]
        L.moe_quantize_int4_tiled.restype = ctypes.c_int
        L.moe_tile_int4.argtypes = [P, P, i64, i64, i32, P, P, P]
        L.moe_tile_int4.restype = ctypes.c_int
        L.moe_pack_bf16_tiled.argtypes = [P, i64, i64, P, P]
        L.moe_pack_bf16_tiled.restype = ctypes.c_int
        L.moe_forward_workspace_bytes.argtypes = [ctypes.POINTER(_Dims)]
        L.moe_forward_workspace_bytes.restype = sz
        fwd = [ctypes.POINTER(_Dims), P, P, P, ctypes.POINTER(_Experts), ctypes.POINTER(_Shared),
               P, P, P]
        L.moe_forward.argtypes = fwd + [P, sz, P]
        L.moe_forward.restype = ctypes.c_int
        L.moe_forward_path.argtypes = fwd + [i32, P, sz, P]
        L.moe_forward_path.restype = ctypes.c_int
        L.moe_forward_noalloc.argtypes = fwd + [i32, P]
        L.moe_forward_noalloc.restype = ctypes.c_int
        fwd_bf16 = list(fwd)
        fwd_bf16[4] = ctypes.POINTER(_ExpertsBf16)
        L.moe_forward_bf16.argtypes = fwd_bf16 + [i32, P, sz, P]
        fwd_fp8 = list(fwd)
        fwd_fp8[4] = ctypes.POINTER(_ExpertsFp8)
        L.moe_forward_fp8.argtypes = fwd_fp8 + [i32, P, sz, P]
        L.moe_forward_fp8.restype = ctypes.c_int
        L.moe_forward_fp8_workspace_bytes.argtypes = [ctypes.POINTER(_Dims)]
        L.moe_forward_fp8_workspace_bytes.restype = sz
        L.moe_quantize_fp8_tiled.argtypes = [P, i64, i64, P, P, P]
        L.moe_quantize_fp8_tiled.restype = ctypes.c_int
        L.moe_quantize_fp8_rows.argtypes = [P, i64, i64, ctypes.c_float, P, P, P]
        L.moe_quantize_fp8_rows.restype = ctypes.c_int
        L.moe_forward_bf16.restype = ctypes.c_int
        L.moe_route_workspace_bytes.argtypes = [ctypes.POINTER(_Dims)]
        L.moe_route_workspace_bytes.restype = sz
        L.moe_route.argtypes = [ctypes.POINTER(_Dims), P, P, P, P, P, P, P, P, P, P, P, sz, P]
        L.moe_route.restype = ctypes.c_int
        products = [P, P, P, i64, i64, i64, i64, P, i32]
        L.moe_grouped_matmul.argtypes = products + [P]
        L.moe_grouped_matmul.restype = ctypes.c_int
        L.moe_grouped_matmul_dx.argtypes = products + [P]
        L.moe_grouped_matmul_dx.restype = ctypes.c_int
        L.moe_grouped_matmul_dw.argtypes = products + [i32, P]
        L.moe_grouped_matmul_dw.restype = ctypes.c_int
        L.moe_linear.argtypes = [P, P, P, i32, P, i64, i64, i64, P, i32, P, P]
        L.moe_linear.restype = ctypes.c_int
        L.moe_linear_dz_workspace_bytes.argtypes = [i64, i64]
        L.moe_linear_dz_workspace_bytes.restype = sz
        L.moe_linear_dz.argtypes = [P, P, i32, i64, i64, P, P, P, sz, P]
        L.moe_linear_dz.restype = ctypes.c_int
        L.moe_grouped_matmul_int4.argtypes = [P, P, P, P, i64, i64, i64, i64, i32, P, i32, P]
        L.moe_grouped_matmul_int4.restype = ctypes.c_int
        L.moe_linear_int4.argtypes = [P, P, P, P, i32, P, i64, i64, i64, i32, P, i32, P]
        L.moe_linear_int4.restype = ctypes.c_int
        L.moe_gated.argtypes = [P, P, P, P, i32, i64, i64, i64, i64, P, P, P]
        L.moe_gated.restype = ctypes.c_int
        L.moe_gated_dz.argtypes = [P, P, P, P, i32, i64, i64, i64, i64, P, P, P]
        L.moe_gated_dz.restype = ctypes.c_int
        L.moe_swiglu.argtypes = [P, i64, i64, P, P]
        L.moe_swiglu.restype = ctypes.c_int
        L.moe_swiglu_backward.argtypes = [P, P, i64, i64, P, P]
        L.moe_swiglu_backward.restype = ctypes.c_int
        L.moe_permute_rows.argtypes = [P, P, i64, i32, i64, P, P]
        L.moe_permute_rows.restype = ctypes.c_int
        L.moe_combine.argtypes = [P, i32, P, P, P, i64, i32, i64, P, P]
        L.moe_combine.restype = ctypes.c_int
        L.moe_combine_backward.argtypes = [P, P, i32, P, P, i64, i32, i64, P, P, P]
        L.moe_combine_backward.restype = ctypes.c_int
        L.moe_adamw.argtypes = [P, i32, ctypes.POINTER(_AdamWHyper), i32, P]
        L.moe_adamw.restype = ctypes.c_int
        L.moe_profile_enable.argtypes = [ctypes.c_int]
        L.moe_profile_enable.restype = ctypes.c_int
        L.moe_profile_read.argtypes = [P, P, ctypes.c_int]
        L.moe_profile_read.restype = ctypes.c_int
        L.moe_stage_name.argtypes = [ctypes.c_int]
        L.moe_stage_name.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def _check(status: int) -> None:
    if status != MOE_OK:
        raise MoEError(status, lib().moe_last_error().decode())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _need(t: torch.Tensor, name: str, dtype, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _dims(T, d, E, h, top_k, group: int = GROUP) -> _Dims:
    return _Dims(int(T), int(d), int(E), int(h), int(top_k), int(group))


# --------------------------------------------------------------- quantizer

def quantize_int4(w: torch.Tensor, q: Optional[torch.Tensor] = None,
                  scales: Optional[torch.Tensor] = None, tiled: bool = False,
                  group: int = GROUP):
    """Int4 group quantizer: fp32 [rows, K] -> (uint8 [rows, K/2], fp32 [rows, K/group]).

    ``w`` may have leading batch dims; they are flattened into rows. With
    ``tiled`` the outputs hold the same codes and scales in the 16-row tile
    order the forward pass reads (rows must be a multiple of 16). ``group``:
    128, 64 or 32 weights per scale (K a multiple of 128).
    """
    _need(w, "w", torch.float32)
    K = w.shape[-1]
    rows = w.numel() // K if K else 0
    if q is None:
        q = torch.empty(w.shape[:-1] + (K // 2,), dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty(w.shape[:-1] + (K // group,), dtype=torch.float32, device=w.device)
    _need(q, "q", torch.uint8)
    _need(scales, "scales", torch.float32)
    if q.numel() != rows * (K // 2) or scales.numel() != rows * (K // group):
        raise ValueError("q / scales have the wrong number of elements")
    fn = lib().moe_quantize_int4_tiled if tiled else lib().moe_quantize_int4
    _check(fn(_ptr(w), rows, K, int(group), _ptr(q), _ptr(scales), _stream(w.device)))
    return q, scales


def tile_int4(q: torch.Tensor, scales: torch.Tensor, group: int = GROUP,
              q_tiled: Optional[torch.Tensor] = None,
              scales_tiled: Optional[torch.Tensor] = None):
    """Row-major int4 (``quantize_int4`` output: uint8 [rows, K/2] and fp32
    [rows, K/group]) -> the tiled order the forward pass reads (same shapes)."""
    _need(q, "q", torch.uint8)
    _need(scales, "scales", torch.float32)
    if q.dim() != 2 or scales.dim() != 2:
        raise ValueError("q and scales must be 2-D")
    rows, K = q.shape[0], q.shape[1] * 2
    if tuple(scales.shape) != (rows, K // group):
        raise ValueError(f"scales has shape {tuple(scales.shape)}, expected {(rows, K // group)}")
    if q_tiled is None:
        q_tiled = torch.empty_like(q)
    if scales_tiled is None:
        scales_tiled = torch.empty_like(scales)
    _need(q_tiled, "q_tiled", torch.uint8)
    _need(scales_tiled, "scales_tiled", torch.float32)
    if q_tiled.numel() != q.numel() or scales_tiled.numel() != scales.numel():
        raise ValueError("q_tiled / scales_tiled have the wrong number of elements")
    _check(lib().moe_tile_int4(_ptr(q), _ptr(scales), rows, K, int(group), _ptr(q_tiled),
                               _ptr(scales_tiled), _stream(q.device)))
    return q_tiled, scales_tiled


def pack_bf16_tiled(src: torch.Tensor, dst: Optional[torch.Tensor] = None) -> torch.Tensor:
    """bf16 [rows, K] -> the tiled order the forward pass reads (same shape)."""
    _need(src, "src", torch.bfloat16)
    if src.dim() != 2:
        raise ValueError("src must be 2-D")
    rows, K = src.shape
    if dst is None:
        dst = torch.empty_like(src)
    _need(dst, "dst", torch.bfloat16, (rows, K))
    _check(lib().moe_pack_bf16_tiled(_ptr(src), rows, K, _ptr(dst), _stream(src.device)))
    return dst


def quantize_fp8(w: torch.Tensor, q: Optional[torch.Tensor] = None,
                 scales: Optional[torch.Tensor] = None):
    """fp32 weights [rows, K] -> fp8 E4M3 codes (uint8, tiled order) and fp32 row scales."""
    _need(w, "w", torch.float32)
    rows, K = w.shape
    if q is None:
        q = torch.empty(rows, K, dtype=torch.uint8, device=w.device)
    if scales is None:
        scales = torch.empty(rows, dtype=torch.float32, device=w.device)
    _need(q, "q", torch.uint8, (rows, K))
    _need(scales, "scales", torch.float32, (rows,))
    _check(lib().moe_quantize_fp8_tiled(_ptr(w), rows, K, _ptr(q), _ptr(scales), _stream(w.device)))
    return q, scales


def quantize_fp8_rows(x: torch.Tensor, ub: float):
    """bf16 activations [rows, K] -> row-major fp8 codes and fp32 row scales
    (the row maximum bounded by ``ub``; ``ub <= 0``: no bound)."""
    _need(x, "x", torch.bfloat16)
    rows, K = x.shape
    q = torch.empty(rows, K, dtype=torch.uint8, device=x.device)
    scales = torch.empty(rows, dtype=torch.float32, device=x.device)
    _check(lib().moe_quantize_fp8_rows(_ptr(x), rows, K, float(ub), _ptr(q), _ptr(scales),
                                       _stream(x.device)))
    return q, scales


def untile_fp8(q: torch.Tensor, rows: int, K: int) -> torch.Tensor:
    """Tiled fp8 codes back to row-major [rows, K] (CPU or GPU tensor)."""
    t = q.reshape(rows // 16, K // 128, 4, 16, 32)  # row tile, k tile, step, row, column
    return t.permute(0, 3, 1, 2, 4).reshape(rows, K)


def pack_shared(s1: torch.Tensor, s3: torch.Tensor, s2: torch.Tensor):
    """The shared expert's bf16 weights (S1, S3 [h, d], S2 [d, h]) in tiled order."""
    return tuple(pack_bf16_tiled(s) for s in (s1, s3, s2))


@dataclass
class Int4Experts:
    """Stacked routed experts in the library's int4 layout."""

    w1q: torch.Tensor  # uint8 [E, h, d/2]
    w3q: torch.Tensor  # uint8 [E, h, d/2]
    w2q: torch.Tensor  # uint8 [E, d, h/2]
    w1s: torch.Tensor  # fp32  [E, h, d/group]
    w3s: torch.Tensor  # fp32  [E, h, d/group]
    w2s: torch.Tensor  # fp32  [E, d, h/group]

    @property
    def E(self) -> int:
        return self.w1q.shape[0]

    @property
    def h(self) -> int:
        return self.w1q.shape[1]

    @property
    def d(self) -> int:
        return self.w2q.shape[1]

    @property
    def group(self) -> int:
        """Weights per scale (128, 64 or 32)."""
        return self.d // self.w1s.shape[2]

    @staticmethod
    def empty(E: int, d: int, h: int, device, group: int = GROUP) -> "Int4Experts":
        if group not in GROUPS:
            raise ValueError(f"group {group} unsupported {GROUPS}")
        u8, f32 = torch.uint8, torch.float32
        return Int4Experts(
            torch.empty(E, h, d // 2, dtype=u8, device=device),
            torch.empty(E, h, d // 2, dtype=u8, device=device),
            torch.empty(E, d, h // 2, dtype=u8, device=device),
            torch.empty(E, h, d // group, dtype=f32, device=device),
            torch.empty(E, h, d // group, dtype=f32, device=device),
            torch.empty(E, d, h // group, dtype=f32, device=device))

    def quantize_expert(self, e: int, w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor):
        """Quantize one expert's fp32 weights (on the GPU) into slot ``e`` (tiled)."""
        g = self.group
        quantize_int4(w1, self.w1q[e], self.w1s[e], tiled=True, group=g)
        quantize_int4(w3, self.w3q[e], self.w3s[e], tiled=True, group=g)
        quantize_int4(w2, self.w2q[e], self.w2s[e], tiled=True, group=g)

    def set_expert_rowmajor(self, e: int, q1, s1, q3, s3, q2, s2):
        """Slot ``e`` from row-major int4 (``quantize_int4`` without ``tiled``):
        W1, W3 codes [h, d/2] and scales [h, d/group], W2 [d, h/2] and [d, h/group],
        repacked into the tiled order by ``tile_int4``."""
        g = self.group
        tile_int4(q1, s1, g, self.w1q[e], self.w1s[e])
        tile_int4(q3, s3, g, self.w3q[e], self.w3s[e])
        tile_int4(q2, s2, g, self.w2q[e], self.w2s[e])

    def _struct(self) -> _Experts:
        for name in ("w1q", "w3q", "w2q"):
            _need(getattr(self, name), name, torch.uint8)
        for name in ("w1s", "w3s", "w2s"):
            _need(getattr(self, name), name, torch.float32)
        g = self.group
        if (g not in GROUPS or self.w1s.shape[2] * g != self.d or self.w3s.shape != self.w1s.shape
                or self.w2s.shape[2] * g != self.h):
            raise ValueError("int4 scales do not match one of the supported groups")
        return _Experts(*(getattr(self, n).data_ptr() for n in
                          ("w1q", "w3q", "w2q", "w1s", "w3s", "w2s")))


# ----------------------------------------------------------------- forward

def workspace_bytes(T: int, d: int, E: int, h: int, top_k: int, fp8: bool = False) -> int:
    """Workspace bytes of the forward (``fp8``: with fp8 routed experts)."""
    dims = _dims(T, d, E, h, top_k)
    fn = lib().moe_forward_fp8_workspace_bytes if fp8 else lib().moe_forward_workspace_bytes
    n = fn(ctypes.byref(dims))
    if n == 0:
        raise ValueError(f"invalid layer dims T={T} d={d} E={E} h={h} top_k={top_k}")
    return n


def alloc_workspace(T: int, d: int, E: int, h: int, top_k: int, device,
                    fp8: bool = False) -> torch.Tensor:
    return torch.empty(workspace_bytes(T, d, E, h, top_k, fp8), dtype=torch.uint8, device=device)


@dataclass
class Bf16Experts:
    """Stacked routed experts in bf16 (the pure-bf16 baseline path), each matrix in
    the tiled order of ``pack_bf16_tiled``."""

    w1: torch.Tensor  # bf16 [E, h, d]
    w3: torch.Tensor  # bf16 [E, h, d]
    w2: torch.Tensor  # bf16 [E, d, h]

    @property
    def E(self) -> int:
        return self.w1.shape[0]

    @property
    def h(self) -> int:
        return self.w1.shape[1]

    @property
    def d(self) -> int:
        return self.w2.shape[1]

    @staticmethod
    def empty(E: int, d: int, h: int, device) -> "Bf16Experts":
        b = torch.bfloat16
        return Bf16Experts(torch.empty(E, h, d, dtype=b, device=device),
                           torch.empty(E, h, d, dtype=b, device=device),
                           torch.empty(E, d, h, dtype=b, device=device))

    def set_expert(self, e: int, w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor):
        """Pack one expert's bf16 weights (W1, W3 [h, d], W2 [d, h]) into slot ``e``."""
        pack_bf16_tiled(w1, self.w1[e])
        pack_bf16_tiled(w3, self.w3[e])
        pack_bf16_tiled(w2, self.w2[e])

    def _struct(self) -> _ExpertsBf16:
        for name in ("w1", "w3", "w2"):
            _need(getattr(self, name), name, torch.bfloat16)
        return _ExpertsBf16(self.w1.data_ptr(), self.w3.data_ptr(), self.w2.data_ptr())


@dataclass
class Fp8Experts:
    """Stacked routed experts in fp8 E4M3 with one fp32 scale per weight row (the
    fp8_mixed path), codes in the tiled order of ``quantize_fp8``; ``act_ub`` bounds
    the activation row scales."""

    w1q: torch.Tensor  # uint8 [E, h, d]
    w3q: torch.Tensor  # uint8 [E, h, d]
    w2q: torch.Tensor  # uint8 [E, d, h]
    w1s: torch.Tensor  # fp32  [E, h]
    w3s: torch.Tensor  # fp32  [E, h]
    w2s: torch.Tensor  # fp32  [E, d]
    act_ub: float

    @property
    def E(self) -> int:
        return self.w1q.shape[0]

    @property
    def h(self) -> int:
        return self.w1q.shape[1]

    @property
    def d(self) -> int:
        return self.w2q.shape[1]

    @staticmethod
    def empty(E: int, d: int, h: int, device, act_ub: float) -> "Fp8Experts":
        u8, f32 = torch.uint8, torch.float32
        return Fp8Experts(
            torch.empty(E, h, d, dtype=u8, device=device),
            torch.empty(E, h, d, dtype=u8, device=device),
            torch.empty(E, d, h, dtype=u8, device=device),
            torch.empty(E, h, dtype=f32, device=device),
            torch.empty(E, h, dtype=f32, device=device),
            torch.empty(E, d, dtype=f32, device=device),
            float(act_ub))

    def quantize_expert(self, e: int, w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor):
        """Quantize one expert's fp32 weights (on the GPU) into slot ``e`` (tiled)."""
        quantize_fp8(w1, self.w1q[e], self.w1s[e])
        quantize_fp8(w3, self.w3q[e], self.w3s[e])
        quantize_fp8(w2, self.w2q[e], self.w2s[e])

    def _struct(self) -> _ExpertsFp8:
        for name in ("w1q", "w3q", "w2q"):
            _need(getattr(self, name), name, torch.uint8)
        for name in ("w1s", "w3s", "w2s"):
            _need(getattr(self, name), name, torch.float32)
        return _ExpertsFp8(*(getattr(self, n).data_ptr() for n in
                             ("w1q", "w3q", "w2q", "w1s", "w3s", "w2s")), float(self.act_ub))


def forward(x: torch.Tensor, router_w: torch.Tensor, router_b: Optional[torch.Tensor],
            experts, shared, top_k: int, path: str = "auto",
            y: Optional[torch.Tensor] = None, topk_ids: Optional[torch.Tensor] = None,
            topk_gates: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The MoE layer: y bf16 [T, d]. ``experts``: ``Int4Experts``, ``Bf16Experts`` or
    ``Fp8Experts``;
    ``shared`` = (S1 [h, d], S3 [h, d], S2 [d, h]) bf16, packed by ``pack_shared``."""
    _need(x, "x", torch.bfloat16)
    T, d = x.shape
    E, h = router_w.shape[0], experts.h
    _need(router_w, "router_w", torch.float32, (E, d))
    if router_b is not None:
        _need(router_b, "router_b", torch.float32, (E,))
    s1, s3, s2 = shared
    _need(s1, "S1", torch.bfloat16, (h, d))
    _need(s3, "S3", torch.bfloat16, (h, d))
    _need(s2, "S2", torch.bfloat16, (d, h))
    if experts.E != E or experts.d != d:
        raise ValueError("experts do not match the router / x")
    if y is None:
        y = torch.empty(T, d, dtype=torch.bfloat16, device=x.device)
    _need(y, "y", torch.bfloat16, (T, d))
    if topk_ids is not None:
        _need(topk_ids, "topk_ids", torch.int32, (T, top_k))
    if topk_gates is not None:
        _need(topk_gates, "topk_gates", torch.float32, (T, top_k))
    fp8 = isinstance(experts, Fp8Experts)
    if workspace is None:
        workspace = alloc_workspace(T, d, E, h, top_k, x.device, fp8)
    dims = _dims(T, d, E, h, top_k, experts.group if isinstance(experts, Int4Experts) else GROUP)
    ex = experts._struct()
    sh = _Shared(s1.data_ptr(), s3.data_ptr(), s2.data_ptr())
    if fp8:
        entry = lib().moe_forward_fp8
    elif isinstance(experts, Bf16Experts):
        entry = lib().moe_forward_bf16
    else:
        entry = lib().moe_forward_path
    _check(entry(
        ctypes.byref(dims), _ptr(x), _ptr(router_w), _ptr(router_b), ctypes.byref(ex),
        ctypes.byref(sh), _ptr(y), _ptr(topk_ids), _ptr(topk_gates), PATHS[path],
        _ptr(workspace), workspace.numel(), _stream(x.device)))
    return y


def forward_noalloc(x: torch.Tensor, router_w: torch.Tensor, router_b: Optional[torch.Tensor],
                    experts: "Int4Experts", shared, top_k: int, path: str = "auto",
                    y: Optional[torch.Tensor] = None, topk_ids: Optional[torch.Tensor] = None,
                    topk_gates: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``forward`` for int4 experts through the allocation-free entry point: its
    workspace is the library's static device scratch (NOALLOC_SCRATCH_BYTES),
    shared by every such call on the GPU, so overlapping calls race."""
    _need(x, "x", torch.bfloat16)
    T, d = x.shape
    E, h = router_w.shape[0], experts.h
    _need(router_w, "router_w", torch.float32, (E, d))
    if router_b is not None:
        _need(router_b, "router_b", torch.float32, (E,))
    s1, s3, s2 = shared
    _need(s1, "S1", torch.bfloat16, (h, d))
    _need(s3, "S3", torch.bfloat16, (h, d))
    _need(s2, "S2", torch.bfloat16, (d, h))
    if not isinstance(experts, Int4Experts) or experts.E != E or experts.d != d:
        raise ValueError("experts must be Int4Experts matching the router / x")
    if y is None:
        y = torch.empty(T, d, dtype=torch.bfloat16, device=x.device)
    _need(y, "y", torch.bfloat16, (T, d))
    if topk_ids is not None:
        _need(topk_ids, "topk_ids", torch.int32, (T, top_k))
    if topk_gates is not None:
        _need(topk_gates, "topk_gates", torch.float32, (T, top_k))
    dims = _dims(T, d, E, h, top_k, experts.group)
    ex = experts._struct()
    sh = _Shared(s1.data_ptr(), s3.data_ptr(), s2.data_ptr())
    _check(lib().moe_forward_noalloc(
        ctypes.byref(dims), _ptr(x), _ptr(router_w), _ptr(router_b), ctypes.byref(ex),
        ctypes.byref(sh), _ptr(y), _ptr(topk_ids), _ptr(topk_gates), PATHS[path],
        _stream(x.device)))
    return y


NOALLOC_SCRATCH_BYTES = 64 << 20


def route(x: torch.Tensor, router_w: torch.Tensor, router_b: Optional[torch.Tensor],
          top_k: int, workspace: Optional[torch.Tensor] = None) -> dict:
    """Routing and dispatch alone: ids, gates, logits, counts, offsets, perm, inv."""
    _need(x, "x", torch.bfloat16)
    T, d = x.shape
    E = router_w.shape[0]
    _need(router_w, "router_w", torch.float32, (E, d))
    if router_b is not None:
        _need(router_b, "router_b", torch.float32, (E,))
    dev = x.device
    P = T * top_k
    out = {
        "ids": torch.empty(T, top_k, dtype=torch.int32, device=dev),
        "gates": torch.empty(T, top_k, dtype=torch.float32, device=dev),
        "logits": torch.empty(T, E, dtype=torch.float32, device=dev),
        "counts": torch.empty(E, dtype=torch.int32, device=dev),
        "offsets": torch.empty(E + 1, dtype=torch.int32, device=dev),
        "perm": torch.empty(P, dtype=torch.int32, device=dev),
        "inv": torch.empty(P, dtype=torch.int32, device=dev),
    }
    dims = _dims(T, d, E, 128, top_k)
    if workspace is None:
        n = lib().moe_route_workspace_bytes(ctypes.byref(dims))
        if n == 0:
            raise ValueError(f"invalid routing dims T={T} d={d} E={E} top_k={top_k}")
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    _check(lib().moe_route(
        ctypes.byref(dims), _ptr(x), _ptr(router_w), _ptr(router_b), _ptr(out["ids"]),
        _ptr(out["gates"]), _ptr(out["logits"]), _ptr(out["counts"]), _ptr(out["offsets"]),
        _ptr(out["perm"]), _ptr(out["inv"]), _ptr(workspace), workspace.numel(), _stream(dev)))
    return out


# ------------------------------------- operators for training and dense layers
#
# The layer's products one by one, with their gradients. They run on the current
# stream of their first argument's device, which need not be the current device; all
# tensors must be on it. None is differentiated by torch's autograd.

ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
_OUT = (torch.bfloat16, torch.float32)


# the current stream's handle without a Stream object: the object costs 1.8 us of the
# 7 us that a small call takes on the host
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _run(fn, first: torch.Tensor, *args) -> None:
    """fn(*args, stream) with `first`'s device current."""
    index = first.get_device()
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status != MOE_OK:
        _check(status)


def _same_device(first: torch.Tensor, *rest: Optional[torch.Tensor]) -> None:
    index = first.get_device()
    for t in rest:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on {first.device} and {t.device}: one device is wanted")


def _output(out: Optional[torch.Tensor], name: str, shape, dtype, first: torch.Tensor) -> torch.Tensor:
    if dtype not in _OUT:
        raise TypeError(f"out_dtype must be torch.bfloat16 or torch.float32, got {dtype}")
    if out is None:
        return torch.empty(shape, dtype=dtype, device=first.device)
    _need(out, name, dtype, shape)
    _same_device(first, out)
    return out


def _two_dim(t: torch.Tensor, name: str) -> None:
    _need(t, name, torch.bfloat16)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")


def _act(act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"act {act!r} unknown: one of {', '.join(ACTS)}")
    return ACTS[act]


def _groups(w: torch.Tensor, offsets: torch.Tensor, first: torch.Tensor):
    _need(w, "w", torch.bfloat16)
    if w.dim() != 3:
        raise ValueError("w must be [E, N, K]")
    _need(offsets, "offsets", torch.int32, (w.shape[0] + 1,))
    _same_device(first, w, offsets)
    return w.shape


def grouped_matmul(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                   out: Optional[torch.Tensor] = None,
                   out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Products of the rows of each expert with its weights: y[s] = x[s] w[e]^T for
    rows s in [offsets[e], offsets[e+1]).

    x bf16 [P, K] (rows in expert order, ``permute_rows``), w bf16 [E, N, K] row-major,
    offsets int32 [E+1] (``route``), y [P, N] bf16 or fp32. N and K multiples of 8.
    Experts may have no rows; rows of ``out`` outside every expert stay as they were."""
    _two_dim(x, "x")
    E, N, K = _groups(w, offsets, x)
    P = x.shape[0]
    if x.shape[1] != K:
        raise ValueError(f"x has {x.shape[1]} columns, w {K}")
    y = _output(out, "out", (P, N), out.dtype if out is not None else out_dtype, x)
    _run(lib().moe_grouped_matmul, x, x.data_ptr(), w.data_ptr(), offsets.data_ptr(), P, E, N, K,
         y.data_ptr(), y.dtype == torch.float32)
    return y


def grouped_matmul_dx(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                      out: Optional[torch.Tensor] = None,
                      out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Gradient of ``grouped_matmul`` for its rows: dx[s] = dy[s] w[e]; dy bf16 [P, N],
    dx [P, K] bf16 or fp32."""
    _two_dim(dy, "dy")
    E, N, K = _groups(w, offsets, dy)
    P = dy.shape[0]
    if dy.shape[1] != N:
        raise ValueError(f"dy has {dy.shape[1]} columns, w {N} rows")
    dx = _output(out, "out", (P, K), out.dtype if out is not None else out_dtype, dy)
    _run(lib().moe_grouped_matmul_dx, dy, dy.data_ptr(), w.data_ptr(), offsets.data_ptr(), P, E, N, K,
         dx.data_ptr(), dx.dtype == torch.float32)
    return dx


def grouped_matmul_dw(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor,
                      out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                      accumulate: bool = False) -> torch.Tensor:
    """Gradient of ``grouped_matmul`` for its weights: dw[e] = sum over the expert's
    rows of dy[s]^T x[s], [E, N, K] bf16 or fp32; zero for an expert without rows.
    ``accumulate`` adds it to ``out``."""
    _two_dim(dy, "dy")
    _two_dim(x, "x")
    _need(offsets, "offsets", torch.int32)
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets must be [E + 1]")
    _same_device(dy, x, offsets)
    P, N, K, E = dy.shape[0], dy.shape[1], x.shape[1], offsets.shape[0] - 1
    if x.shape[0] != P:
        raise ValueError(f"dy has {P} rows, x {x.shape[0]}")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    dw = _output(out, "out", (E, N, K), out.dtype if out is not None else out_dtype, dy)
    _run(lib().moe_grouped_matmul_dw, dy, dy.data_ptr(), x.data_ptr(), offsets.data_ptr(), P, E, N, K,
         dw.data_ptr(), dw.dtype == torch.float32, bool(accumulate))
    return dw


def linear(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "none",
           residual: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
           out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Dense layer act(x w^T + bias) + residual in one pass.

    x bf16 [T, K], w bf16 [N, K] row-major, bias fp32 [N], residual bf16 [T, N], act
    one of ``ACTS``. ``z`` (bf16 [T, N]), if given, receives x w^T + bias for
    ``linear_dz``. A bf16 ``out`` may be ``residual`` itself. N and K multiples of 8."""
    _two_dim(x, "x")
    _two_dim(w, "w")
    (T, K), N = x.shape, w.shape[0]
    if w.shape[1] != K:
        raise ValueError(f"x has {K} columns, w {w.shape[1]}")
    if bias is not None:
        _need(bias, "bias", torch.float32, (N,))
    if residual is not None:
        _need(residual, "residual", torch.bfloat16, (T, N))
    if z is not None:
        _need(z, "z", torch.bfloat16, (T, N))
    _same_device(x, w, bias, residual, z)
    y = _output(out, "out", (T, N), out.dtype if out is not None else out_dtype, x)
    _run(lib().moe_linear, x, x.data_ptr(), w.data_ptr(), _ptr(bias), _act(act), _ptr(residual), T, N, K,
         y.data_ptr(), y.dtype == torch.float32, _ptr(z))
    return y


def linear_dz_workspace_bytes(T: int, N: int) -> int:
    """Workspace bytes of ``linear_dz`` for dz [T, N]."""
    n = lib().moe_linear_dz_workspace_bytes(int(T), int(N))
    if n == 0:
        raise ValueError(f"invalid dims T={T} N={N}")
    return n


def linear_dz(dy: torch.Tensor, z: Optional[torch.Tensor], act: str = "none",
              out: Optional[torch.Tensor] = None, db: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None):
    """Gradient of ``linear`` through its activation: (dz, db) with dz = dy * act'(z)
    bf16 [T, N] and db fp32 [N] the column sums of dz, the bias's gradient. With act
    "none" dz is dy itself and z is not read. ``out`` may be dy or z."""
    _two_dim(dy, "dy")
    T, N = dy.shape
    code = _act(act)
    if code:
        if z is None:
            raise ValueError(f"act {act!r} needs z")
        _need(z, "z", torch.bfloat16, (T, N))
        dz = _output(out, "out", (T, N), torch.bfloat16, dy)
    else:
        if out is not None:
            raise ValueError("act 'none' writes no dz: it is dy")
        z, dz = None, None
    if db is None:
        db = torch.empty(N, dtype=torch.float32, device=dy.device)
    _need(db, "db", torch.float32, (N,))
    if workspace is None:
        workspace = torch.empty(linear_dz_workspace_bytes(T, N), dtype=torch.uint8, device=dy.device)
    _need(workspace, "workspace", torch.uint8)
    _same_device(dy, z, db, workspace)
    _run(lib().moe_linear_dz, dy, dy.data_ptr(), _ptr(z), code, T, N, _ptr(dz), db.data_ptr(),
         workspace.data_ptr(), workspace.numel())
    return (dy if dz is None else dz), db


def linear_dx(dz: torch.Tensor, w: torch.Tensor, out: Optional[torch.Tensor] = None,
              out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Gradient of ``linear`` for x: dz w, dz bf16 [T, N], w bf16 [N, K]."""
    _two_dim(dz, "dz")
    _two_dim(w, "w")
    (T, N), K = dz.shape, w.shape[1]
    if w.shape[0] != N:
        raise ValueError(f"dz has {N} columns, w {w.shape[0]} rows")
    _same_device(dz, w)
    dx = _output(out, "out", (T, K), out.dtype if out is not None else out_dtype, dz)
    _run(lib().moe_grouped_matmul_dx, dz, dz.data_ptr(), w.data_ptr(), None, T, 1, N, K,
         dx.data_ptr(), dx.dtype == torch.float32)
    return dx


def linear_dw(dz: torch.Tensor, x: torch.Tensor, out: Optional[torch.Tensor] = None,
              out_dtype: torch.dtype = torch.bfloat16, accumulate: bool = False) -> torch.Tensor:
    """Gradient of ``linear`` for w: dz^T x, [N, K]; ``accumulate`` adds it to ``out``."""
    _two_dim(dz, "dz")
    _two_dim(x, "x")
    (T, N), K = dz.shape, x.shape[1]
    if x.shape[0] != T:
        raise ValueError(f"dz has {T} rows, x {x.shape[0]}")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    _same_device(dz, x)
    dw = _output(out, "out", (N, K), out.dtype if out is not None else out_dtype, dz)
    _run(lib().moe_grouped_matmul_dw, dz, dz.data_ptr(), x.data_ptr(), None, T, 1, N, K,
         dw.data_ptr(), dw.dtype == torch.float32, bool(accumulate))
    return dw


def _int4_weights(q: torch.Tensor, scales: torch.Tensor, dims: int):
    """(shape of the weights, group) of tiled codes [.., N, K/2] and scales [.., N, K/group]."""
    _need(q, "q", torch.uint8)
    _need(scales, "scales", torch.float32)
    if q.dim() != dims or scales.dim() != dims or scales.shape[:-1] != q.shape[:-1]:
        raise ValueError(f"q {tuple(q.shape)} and scales {tuple(scales.shape)} must be "
                         f"{'[E, N, K/2] and [E, N, K/group]' if dims == 3 else '[N, K/2] and [N, K/group]'}")
    K, per = q.shape[-1] * 2, scales.shape[-1]
    if per == 0 or K % per or K // per not in GROUPS:
        raise ValueError(f"{K} columns with {per} scales a row: not a supported group {GROUPS}")
    return (*q.shape[:-1], K), K // per


def grouped_matmul_int4(x: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, offsets: torch.Tensor,
                        out: Optional[torch.Tensor] = None,
                        out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """``grouped_matmul`` with int4 weights: y[s] = x[s] (scale * code)[e]^T.

    q uint8 [E, N, K/2] and scales fp32 [E, N, K/group] in the tiled order of ``quantize_int4(tiled=True)`` or
    ``tile_int4`` (``Int4Experts`` holds its matrices so); N a multiple of 16, K of 128. The weights are
    not rounded to bf16."""
    _two_dim(x, "x")
    (E, N, K), group = _int4_weights(q, scales, 3)
    _need(offsets, "offsets", torch.int32, (E + 1,))
    _same_device(x, q, scales, offsets)
    P = x.shape[0]
    if x.shape[1] != K:
        raise ValueError(f"x has {x.shape[1]} columns, q {K}")
    y = _output(out, "out", (P, N), out.dtype if out is not None else out_dtype, x)
    _run(lib().moe_grouped_matmul_int4, x, x.data_ptr(), q.data_ptr(), scales.data_ptr(), offsets.data_ptr(), P, E,
         N, K, group, y.data_ptr(), y.dtype == torch.float32)
    return y


def linear_int4(x: torch.Tensor, q: torch.Tensor, scales: torch.Tensor, bias: Optional[torch.Tensor] = None,
                act: str = "none", residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """``linear`` with int4 weights: act(x (scale * code)^T + bias) + residual, from one token on.

    q uint8 [N, K/2] and scales fp32 [N, K/group], tiled as for ``grouped_matmul_int4``; bias fp32 [N],
    residual bf16 [T, N], which a bf16 ``out`` may be itself. Errors go by sum |x scale|, also under codes of 0 (up to 2^-17 of it):
    below a bf16 result's rounding but for rows of a few very large x."""
    _two_dim(x, "x")
    (N, K), group = _int4_weights(q, scales, 2)
    T = x.shape[0]
    if x.shape[1] != K:
        raise ValueError(f"x has {x.shape[1]} columns, q {K}")
    if bias is not None:
        _need(bias, "bias", torch.float32, (N,))
    if residual is not None:
        _need(residual, "residual", torch.bfloat16, (T, N))
    _same_device(x, q, scales, bias, residual)
    y = _output(out, "out", (T, N), out.dtype if out is not None else out_dtype, x)
    _run(lib().moe_linear_int4, x, x.data_ptr(), q.data_ptr(), scales.data_ptr(), _ptr(bias), _act(act), _ptr(residual),
         T, N, K, group, y.data_ptr(), y.dtype == torch.float32)
    return y


def _gated(x, w, bias, offsets, act, z, out, E, h2, d):
    P = x.shape[0]
    if x.shape[1] != d:
        raise ValueError(f"x has {x.shape[1]} columns, w {d}")
    if h2 % 2:
        raise ValueError("w must have as many gate rows as up rows")
    h = h2 // 2
    if z is not None:
        _need(z, "z", torch.bfloat16, (P, h2))
    _same_device(x, w, bias, offsets, z)
    y = _output(out, "out", (P, h), torch.bfloat16, x)
    _run(lib().moe_gated, x, x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(offsets), _act(act), P, E, h, d,
         y.data_ptr(), _ptr(z))
    return y


def grouped_gated(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, act: str = "silu",
                  z: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Both up-projections of each expert's rows, the activation and the product in one pass: y[s] =
    act(g) * u with [g | u] = x[s] w[e]^T.

    x bf16 [P, d] (rows in expert order), w bf16 [E, 2h, d], the gate's h rows first, offsets int32
    [E+1] (``route``), act one of ``ACTS``, y bf16 [P, h]. ``z`` (bf16 [P, 2h]), if given, receives [g | u]
    for ``grouped_gated_dz``. What ``grouped_matmul`` and ``swiglu`` do in two passes, with z."""
    _two_dim(x, "x")
    E, h2, d = _groups(w, offsets, x)
    return _gated(x, w, None, offsets, act, z, out, E, h2, d)


def gated_linear(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "silu",
                 z: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``grouped_gated`` of one dense block: w bf16 [2h, d], bias fp32 [2h] (its gradient: ``linear_dz`` of dz
    with act "none")."""
    _two_dim(x, "x")
    _two_dim(w, "w")
    if bias is not None:
        _need(bias, "bias", torch.float32, (w.shape[0],))
    return _gated(x, w, bias, None, act, z, out, 1, w.shape[0], w.shape[1])


def _gated_dz(dy, w2, z, offsets, act, y, out, E, d, h):
    P = dy.shape[0]
    if dy.shape[1] != d:
        raise ValueError(f"dy has {dy.shape[1]} columns, w2 {d} rows")
    _need(z, "z", torch.bfloat16, (P, 2 * h))
    if y is not None:
        _need(y, "y", torch.bfloat16, (P, h))
    _same_device(dy, w2, z, offsets, y)
    dz = _output(out, "out", (P, 2 * h), torch.bfloat16, dy)
    _run(lib().moe_gated_dz, dy, dy.data_ptr(), w2.data_ptr(), z.data_ptr(), _ptr(offsets), _act(act), P, E, h, d,
         dz.data_ptr(), _ptr(y))
    return dz


def grouped_gated_dz(dy: torch.Tensor, w2: torch.Tensor, z: torch.Tensor, offsets: torch.Tensor, act: str = "silu",
                     y: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of a gated block's projections, from that of the down-projection's output: dz[s] =
    [dh u act'(g) | dh act(g)], bf16 [P, 2h], with dh = dy[s] w2[e].

    dy bf16 [P, d], w2 bf16 [E, d, h] (the weights of ``grouped_matmul`` behind the block), z = [g | u] bf16
    [P, 2h]. ``y`` (bf16 [P, h]), if given, receives act(g) * u, of which w2's gradient is made, so that the
    forward need not keep it. ``out`` may be z. Then ``grouped_matmul_dx`` and ``_dw`` of dz."""
    _two_dim(dy, "dy")
    E, d, h = _groups(w2, offsets, dy)
    return _gated_dz(dy, w2, z, offsets, act, y, out, E, d, h)


def gated_linear_dz(dy: torch.Tensor, w2: torch.Tensor, z: torch.Tensor, act: str = "silu",
                    y: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``grouped_gated_dz`` of one dense block: w2 bf16 [d, h]."""
    _two_dim(dy, "dy")
    _two_dim(w2, "w2")
    return _gated_dz(dy, w2, z, None, act, y, out, 1, w2.shape[0], w2.shape[1])


def swiglu(z: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """silu(g) * u of rows z = [g | u], bf16 [rows, 2h] -> [rows, h] (h a multiple of 8)."""
    _two_dim(z, "z")
    rows, h = z.shape[0], z.shape[1] // 2
    if z.shape[1] != 2 * h:
        raise ValueError("z must have an even number of columns")
    y = _output(out, "out", (rows, h), torch.bfloat16, z)
    _run(lib().moe_swiglu, z, z.data_ptr(), rows, h, y.data_ptr())
    return y


def swiglu_backward(dy: torch.Tensor, z: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of ``swiglu``: dz = [dy u silu'(g) | dy silu(g)], bf16 [rows, 2h].
    ``out`` may be z."""
    _two_dim(dy, "dy")
    rows, h = dy.shape
    _need(z, "z", torch.bfloat16, (rows, 2 * h))
    _same_device(dy, z)
    dz = _output(out, "out", (rows, 2 * h), torch.bfloat16, dy)
    _run(lib().moe_swiglu_backward, dy, dy.data_ptr(), z.data_ptr(), rows, h, dz.data_ptr())
    return dz


def permute_rows(x: torch.Tensor, perm: torch.Tensor, top_k: int,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Tokens copied to their expert rows: xp[s] = x[perm[s] // top_k]; x bf16 [T, d],
    perm int32 [T*top_k] (``route``). Its gradient is ``combine`` without gates."""
    _two_dim(x, "x")
    T, d = x.shape
    _need(perm, "perm", torch.int32)
    if perm.numel() != T * top_k:
        raise ValueError(f"perm has {perm.numel()} entries, expected {T * top_k}")
    _same_device(x, perm)
    xp = _output(out, "out", (T * top_k, d), torch.bfloat16, x)
    _run(lib().moe_permute_rows, x, x.data_ptr(), perm.data_ptr(), T, top_k, d, xp.data_ptr())
    return xp


def _pairs(T: int, inv: torch.Tensor, gates: Optional[torch.Tensor], top_k: int) -> None:
    _need(inv, "inv", torch.int32)
    if inv.numel() != T * top_k:
        raise ValueError(f"inv has {inv.numel()} entries, expected {T * top_k}")
    if gates is not None:
        _need(gates, "gates", torch.float32, (T, top_k))


def combine(o: torch.Tensor, inv: torch.Tensor, gates: Optional[torch.Tensor] = None,
            residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
            top_k: Optional[int] = None) -> torch.Tensor:
    """Expert rows summed back to their tokens: y[t] = sum_j gates[t, j] o[inv[t, j]] +
    residual[t], bf16 [T, d].

    o bf16 or fp32 [T*top_k, d], inv int32 [T, top_k] or flat (``route``), gates fp32
    [T, top_k] (none: 1). top_k comes from gates or a 2-D inv, or is given. ``out`` may
    be ``residual`` itself."""
    if not isinstance(o, torch.Tensor) or o.dtype not in _OUT:
        raise TypeError("o must be a bf16 or fp32 tensor")
    _need(o, "o", o.dtype)
    if o.dim() != 2:
        raise ValueError("o must be 2-D")
    if top_k is None:
        if gates is not None:
            top_k = gates.shape[-1]
        elif inv.dim() == 2:
            top_k = inv.shape[1]
        else:
            raise ValueError("a flat inv without gates needs top_k")
    P, d = o.shape
    if top_k < 1 or P % top_k:
        raise ValueError(f"o has {P} rows: not a multiple of top_k = {top_k}")
    T = P // top_k
    _pairs(T, inv, gates, top_k)
    if residual is not None:
        _need(residual, "residual", torch.bfloat16, (T, d))
    _same_device(o, inv, gates, residual)
    y = _output(out, "out", (T, d), torch.bfloat16, o)
    _run(lib().moe_combine, o, o.data_ptr(), o.dtype == torch.float32, inv.data_ptr(), _ptr(gates),
         _ptr(residual), T, top_k, d, y.data_ptr())
    return y


def combine_backward(dy: torch.Tensor, o: torch.Tensor, inv: torch.Tensor, gates: torch.Tensor,
                     out: Optional[torch.Tensor] = None):
    """Gradient of ``combine``: (d_o, d_gates) with d_o[inv[t, j]] = gates[t, j] dy[t], bf16
    [T*top_k, d], and d_gates[t, j] = <dy[t], o[inv[t, j]]>, fp32 [T, top_k]."""
    _two_dim(dy, "dy")
    T, d = dy.shape
    _need(gates, "gates", torch.float32)
    if gates.dim() != 2 or gates.shape[0] != T:
        raise ValueError(f"gates must be [{T}, top_k]")
    top_k = gates.shape[1]
    _pairs(T, inv, gates, top_k)
    if not isinstance(o, torch.Tensor) or o.dtype not in _OUT:
        raise TypeError("o must be a bf16 or fp32 tensor")
    _need(o, "o", o.dtype, (T * top_k, d))
    _same_device(dy, o, inv, gates)
    d_o = _output(out, "out", (T * top_k, d), torch.bfloat16, dy)
    d_gates = torch.empty(T, top_k, dtype=torch.float32, device=dy.device)
    _run(lib().moe_combine_backward, dy, dy.data_ptr(), o.data_ptr(), o.dtype == torch.float32,
         inv.data_ptr(), gates.data_ptr(), T, top_k, d, d_o.data_ptr(), d_gates.data_ptr())
    return d_o, d_gates


# ---------------------------------------------------------------- optimizer step

ADAMW_BLOCK = 128  # elements that share a scale of an 8-bit moment
_ADAMW_WORDS = 9   # of 8 bytes: a moe_adamw_tensor


@dataclass
class AdamWState:
    """What ``adamw`` keeps between steps for a list of parameters.

    The moments of all parameters stand in one tensor each, parameter i's from ``starts()[i]``,
    a multiple of 128; what lies between them is zero and stays so. In 32 bits ``m`` and ``v`` are
    fp32 [total]. In 8 bits they are uint8, E4M3 codes of m and of sqrt(v), with fp32 scales
    [total / 128]; ``m`` is [total], and ``v`` [2 total]: behind its codes stands a byte for each element with what both
    moments' codes leave, four bits each (``fine``). A state may be made of codes alone, v [total], for betas up to 0.9 and
    0.95: changes of less than half a code's step (3 to 6 %) are then lost, and slower moments would stand still
    (``torch.cat([v, torch.zeros_like(v)])`` makes of it one that keeps them). ``master``, if
    there, holds the fp32 copies of bf16 parameters in the same places as m, which a step updates and rounds to the
    parameters (what stands at an fp32 parameter's place is not used)."""

    params: list  # bf16 or fp32 tensors of any shape, contiguous, updated in place
    m: torch.Tensor
    v: torch.Tensor
    m_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None
    master: Optional[torch.Tensor] = None

    @property
    def fine(self) -> Optional[torch.Tensor]:
        """uint8 [total] behind the codes of an 8-bit v: what both moments' codes leave, m's in the low four bits, sqrt(v)'s in the
        high four, in fourteenths of a code's step. None for codes alone and in 32 bits."""
        total = self.m.numel()
        return self.v[total:] if self.m.dtype == torch.uint8 and self.v.numel() == 2 * total else None

    @staticmethod
    def zeros(params, bits: int = 32, master: bool = True) -> "AdamWState":
        """State before the first step. ``bits``: of a moment, 32 or 8 (of its code; 12 with the fine bits). ``master``: keep fp32
        copies of bf16 parameters (without, a step smaller than half a bf16 step is lost)."""
        if bits not in (8, 32):
            raise ValueError(f"bits = {bits}: 8 or 32")
        params = list(params)
        if not params:
            raise ValueError("no parameters")
        total, dev = _adamw_starts(params)[-1], params[0].device
        moment = torch.uint8 if bits == 8 else torch.float32
        m, v = (torch.zeros(n, dtype=moment, device=dev) for n in (total, 2 * total if bits == 8 else total))
        scales = [torch.zeros(total // ADAMW_BLOCK, dtype=torch.float32, device=dev) if bits == 8 else None
                  for _ in range(2)]
        state = AdamWState(params, m, v, *scales)
        if master and any(p.dtype == torch.bfloat16 for p in params):
            state.master = torch.zeros(total, dtype=torch.float32, device=dev)
            for p, at in zip(params, state.starts()):
                state.master[at:at + p.numel()].copy_(p.detach().reshape(-1))
        return state

    def starts(self) -> list:
        """Where each parameter's elements begin in the moments, and the total."""
        return _adamw_starts(self.params)

    def moments(self, i: int):
        """(m, v) of parameter i, fp32 in its shape."""
        p, at = self.params[i], self.starts()[i]
        n = p.numel()
        if self.m.dtype != torch.uint8:
            return tuple(t[at:at + n].reshape(p.shape).clone() for t in (self.m, self.v))
        end = self.starts()[i + 1]
        out, fine = [], self.fine
        for codes, scale, shift in ((self.m, self.m_scale, 0), (self.v, self.v_scale, 4)):
            x = codes[at:end].view(torch.float8_e4m3fn).float()
            if fine is not None:
                # 2^e of the code, its step times eight
                power = (x.view(torch.int32) & 0x7F800000).clamp(min=0x3C800000).view(torch.float32)
                k = ((fine[at:end] >> shift) & 15).float()
                x = x + torch.where(k > 7, k - 16.0, k) * (power * torch.tensor(1.0 / 112.0, device=x.device))
            x = x.reshape(-1, ADAMW_BLOCK)
            x = x * scale[at // ADAMW_BLOCK:end // ADAMW_BLOCK].unsqueeze(1)
            out.append(x.reshape(-1)[:n].reshape(p.shape))
        return out[0], out[1] * out[1]


def _adamw_starts(params) -> list:
    at = [0]
    for p in params:
        at.append(at[-1] + (p.numel() + ADAMW_BLOCK - 1) // ADAMW_BLOCK * ADAMW_BLOCK)
    return at


def _device_scalar(t: torch.Tensor, name: str, dtype) -> int:
    _need(t, name, dtype)
    if t.numel() != 1:
        raise ValueError(f"{name} must have one element")
    return t.data_ptr()


def adamw(state: AdamWState, grads, step, lr, betas=(0.9, 0.999), eps: float = 1e-8,
          weight_decay: float = 0.01, grad_scale: Optional[torch.Tensor] = None) -> None:
    """One AdamW step of all of ``state.params``, in place, in a launch for each 52 of them.

    ``grads``: a bf16 or fp32 tensor for each parameter, or None for one that is left alone.
    ``step``: this step's number, 1 for the first, and ``lr``: numbers, or tensors of one element
    on the GPU (int32, fp32), which a captured graph reads anew at each replay. ``grad_scale``
    (fp32, one element on the GPU) multiplies the gradients: a clipping factor. As with torch's own
    in-place operations a stepped parameter's version moves, so that a backward pass through a graph that still needs
    its old values raises (a replayed graph of steps moves none)."""
    params, grads = state.params, list(grads)
    if len(grads) != len(params):
        raise ValueError(f"{len(grads)} gradients for {len(params)} parameters")
    if not params:
        return
    m, v, bits = state.m, state.v, 8 if state.m.dtype == torch.uint8 else 32
    moment = torch.uint8 if bits == 8 else torch.float32
    first = params[0]
    index = first.get_device()
    words, at, stepped = [], 0, []
    base_m, base_v, base_p = m.data_ptr(), v.data_ptr(), _ptr(state.master)
    width = 1 if bits == 8 else 4
    scale_m, scale_v = (_ptr(state.m_scale) or 0, _ptr(state.v_scale) or 0) if bits == 8 else (0, 0)
    half, full, block = torch.bfloat16, torch.float32, ADAMW_BLOCK
    add = words.extend
    for p, g in zip(params, grads):
        dtype, n, start = p.dtype, p.numel(), at
        if (dtype is not half and dtype is not full) or not p.is_contiguous() or p.get_device() != index or index < 0:
            raise ValueError("parameters must be bf16 or fp32, contiguous, and on one GPU")
        at += -(-n // block) * block
        if g is None:
            continue
        gtype = g.dtype
        if ((gtype is not half and gtype is not full) or not g.is_contiguous() or g.get_device() != index
                or g.shape != p.shape):
            raise ValueError("gradients must be bf16 or fp32, contiguous, of their parameter's shape and on its GPU")
        stepped.append(p)
        add((p.data_ptr(), g.data_ptr(), base_p + 4 * start if base_p and dtype is half else 0,
             base_m + width * start, base_v + width * start,
             scale_m and scale_m + start // block * 4, scale_v and scale_v + start // block * 4,
             n, (dtype is full) | (gtype is full) << 32))
    _need(m, "m", moment, (at,))
    fine = state.fine if bits == 8 else None
    _need(v, "v", moment, (at,) if fine is None else (2 * at,))
    scales = (at // ADAMW_BLOCK,)
    for t, name in ((state.m_scale, "m_scale"), (state.v_scale, "v_scale")):
        if bits == 8:
            _need(t, name, torch.float32, scales)
        elif t is not None:
            raise ValueError(f"{name} with moments of 32 bits")
    if state.master is not None:
        _need(state.master, "master", torch.float32, (at,))
    h = _AdamWHyper(0.0, float(betas[0]), float(betas[1]), float(eps), float(weight_decay), 0)
    if isinstance(step, torch.Tensor):
        h.step_device = _device_scalar(step, "step", torch.int32)
    else:
        h.step = int(step)
    if isinstance(lr, torch.Tensor):
        h.lr_device = _device_scalar(lr, "lr", torch.float32)
    else:
        h.lr = float(lr)
    if grad_scale is not None:
        h.grad_scale = _device_scalar(grad_scale, "grad_scale", torch.float32)
    if fine is not None:
        h.fine = fine.data_ptr() - base_v
    _same_device(first, m, v, state.m_scale, state.v_scale, state.master, grad_scale,
                 step if isinstance(step, torch.Tensor) else None, lr if isinstance(lr, torch.Tensor) else None)
    table = array.array("Q", words)
    _run(lib().moe_adamw, first, table.buffer_info()[0], len(words) // _ADAMW_WORDS, ctypes.byref(h), bits)
    torch.autograd.graph.increment_version(stepped)


def untile_int4(q: torch.Tensor, rows: int, K: int) -> torch.Tensor:
    """Tiled int4 bytes of one [rows, K] matrix -> row-major bytes [rows, K/2]."""
    t = q.reshape(rows // 16, K // TILE, 4, 16, 16)  # row tile, k tile, step, row, byte
    return t.permute(0, 3, 1, 2, 4).reshape(rows, K // 2)


def untile_scales(s: torch.Tensor, rows: int, K: int, group: int = GROUP) -> torch.Tensor:
    """Tiled scales of one [rows, K] matrix -> row-major [rows, K/group]."""
    S = TILE // group
    return s.reshape(rows // 16, K // TILE, 16, S).permute(0, 2, 1, 3).reshape(rows, K // group)


def untile_bf16(t: torch.Tensor, rows: int, K: int) -> torch.Tensor:
    """Tiled bf16 [rows, K] (pack_bf16_tiled order) -> row-major [rows, K]."""
    return t.reshape(rows // 16, K // TILE, 4, 16, 32).permute(0, 3, 1, 2, 4).reshape(rows, K)


def unpack_int4(q: torch.Tensor) -> torch.Tensor:
    """Packed bytes [..., K/2] -> int8 codes [..., K] (low nibble = even index)."""
    lo = (q.to(torch.int16) & 0xF)
    hi = (q.to(torch.int16) >> 4) & 0xF
    codes = torch.stack([lo, hi], dim=-1).reshape(*q.shape[:-1], q.shape[-1] * 2)
    return torch.where(codes >= 8, codes - 16, codes).to(torch.int8)


# ------------------------------------------------------------------ timing

STAGE_COUNT = 10


def hbm_read(buf: torch.Tensor, sink: torch.Tensor) -> None:
    """Stream every 16-byte word of `buf` once (measurement helper); each block
    writes the XOR of the words it read into `sink` (uint32/int32,
    ``hbm_read_sink_words()`` entries)."""
    if not buf.is_cuda or not sink.is_cuda or sink.numel() < hbm_read_sink_words():
        raise ValueError("buf and sink must be device tensors, sink of hbm_read_sink_words() words")
    _check(lib().moe_hbm_read(buf.data_ptr(), buf.numel() * buf.element_size(), sink.data_ptr(),
                              _stream(buf.device)))


def hbm_read_sink_words() -> int:
    return int(lib().moe_hbm_read_sink_words())


def hbm_copy(dst: torch.Tensor, src: torch.Tensor) -> None:
    """Copy `src` into `dst` with the library's plain copy kernel (measurement helper)."""
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes or not dst.is_cuda or not src.is_cuda:
        raise ValueError("dst and src must be device tensors of the same size")
    _check(lib().moe_hbm_copy(dst.data_ptr(), src.data_ptr(), nbytes, _stream(src.device)))


def profile_enable(on: bool = True) -> None:
    """Time each stage of later calls with events that its kernels record at
    their own start and end."""
    _check(lib().moe_profile_enable(1 if on else 0))


def profile_read() -> dict:
    """{stage name: (summed ms, launches)} since the last read; resets the sums."""
    ms = (ctypes.c_double * STAGE_COUNT)()
    n = (ctypes.c_int64 * STAGE_COUNT)()
    _check(lib().moe_profile_read(ms, n, STAGE_COUNT))
    return {lib().moe_stage_name(i).decode(): (ms[i], n[i]) for i in range(STAGE_COUNT)}
