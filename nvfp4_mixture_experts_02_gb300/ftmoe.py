"""Thin ctypes binding of libftmoe.so (include/ft_moe.h): argument checks and marshalling.

Every step of the layer runs in the library's CUDA kernels. torch supplies device
memory and streams; there is no CPU fallback, and importing this module without the
built library raises. Tensors are checked before their pointers are handed over (device,
element type, contiguity, shape): the expert objects once when built, the per-call tensors
on every call.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from dataclasses import dataclass
from typing import NamedTuple

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libftmoe.so")

FT_OK = 0
STATUS_NAMES = {0: "FT_OK", 1: "FT_ERR_INVALID_ARG", 2: "FT_ERR_UNSUPPORTED_SHAPE",
                3: "FT_ERR_MISALIGNED", 4: "FT_ERR_WORKSPACE_TOO_SMALL", 5: "FT_ERR_CUDA",
                6: "FT_ERR_DEVICE_FLAG", 7: "FT_ERR_TIMEOUT"}

EXPORTED = ["ft_moe_abi_version", "ft_status_string", "ft_moe_route", "ft_moe_workspace_bytes",
            "ft_moe_workspace_init", "ft_moe_nvfp4_decode", "ft_moe_nvfp4_prefill",
            "ft_moe_get_error", "ft_moe_last_cuda_error", "ft_moe_nvfp4_decode_noalloc",
            "ft_moe_nvfp4_decode_routed", "ft_moe_decode_smem_bytes",
            "ft_moe_debug_set_wait_limit", "ft_moe_layer_from_host",
            "ft_moe_fp8block_workspace_bytes", "ft_moe_fp8block_decode",
            "ft_moe_router_logits", "ft_moe_router_route",
            "ft_nvfp4_linear_workspace_bytes", "ft_nvfp4_linear", "ft_kv_append", "ft_paged_attention_workspace_bytes",
            "ft_paged_decode_attention", "ft_residual_norm",
            "ft_residual_norm_backward_workspace_bytes", "ft_residual_norm_backward"]

# Leading bytes of a workspace that must be zero before a call (FT_MOE_WORKSPACE_HEAD_BYTES);
# the rest is scratch whose contents never reach an output.
WORKSPACE_HEAD_BYTES = 1024


class FtError(RuntimeError):
    def __init__(self, status: int, what: str, detail: str = ""):
        msg = f"{what}: {STATUS_NAMES.get(status, status)}"
        super().__init__(msg + (f" ({detail})" if detail else ""))
        self.status = status


class _Experts(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("w13", ctypes.c_void_p), ("w13_scale", ctypes.c_void_p),
                ("w13_gscale", ctypes.c_void_p), ("w2", ctypes.c_void_p),
                ("w2_scale", ctypes.c_void_p), ("w2_gscale", ctypes.c_void_p)]


class _Shared(ctypes.Structure):
    _fields_ = [("w13", ctypes.c_void_p), ("w13_scale", ctypes.c_void_p),
                ("w13_gscale", ctypes.c_void_p), ("w2", ctypes.c_void_p),
                ("w2_scale", ctypes.c_void_p), ("w2_gscale", ctypes.c_void_p),
                ("gate", ctypes.c_void_p)]


class _F8Experts(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("w13", ctypes.c_void_p), ("w13_scale", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("w2_scale", ctypes.c_void_p)]


class _F8Shared(ctypes.Structure):
    _fields_ = [("w13", ctypes.c_void_p), ("w13_scale", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("w2_scale", ctypes.c_void_p),
                ("gate", ctypes.c_void_p)]


class _Matrix(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("K", ctypes.c_int32), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("gscale", ctypes.c_void_p)]


class _PagedKV(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32),
                ("k_page_stride", ctypes.c_int64), ("k_slot_stride", ctypes.c_int64),
                ("k_head_stride", ctypes.c_int64), ("v_page_stride", ctypes.c_int64),
                ("v_slot_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with __graft_entry__.build() "
                          "(nvcc, sm_103a); there is no fallback implementation")
    lib = ctypes.CDLL(path)
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    lib.ft_moe_abi_version.restype = i32
    lib.ft_status_string.restype = ctypes.c_char_p
    lib.ft_status_string.argtypes = [ctypes.c_int]
    lib.ft_moe_route.restype = ctypes.c_int
    lib.ft_moe_route.argtypes = [vp, i32, i32, i32, vp, vp, vp]
    lib.ft_moe_workspace_bytes.restype = sz
    lib.ft_moe_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32, i32]
    lib.ft_moe_decode_smem_bytes.restype = sz
    lib.ft_moe_decode_smem_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.ft_moe_workspace_init.restype = ctypes.c_int
    lib.ft_moe_workspace_init.argtypes = [vp, sz, vp]
    layer = [vp, i32, vp, vp, i32, ctypes.POINTER(_Experts), ctypes.POINTER(_Shared), f32,
             vp, vp, sz, vp]
    for name in ("ft_moe_nvfp4_decode", "ft_moe_nvfp4_prefill"):
        getattr(lib, name).restype = ctypes.c_int
        getattr(lib, name).argtypes = layer
    lib.ft_moe_nvfp4_decode_noalloc.restype = ctypes.c_int
    lib.ft_moe_nvfp4_decode_noalloc.argtypes = layer[:9] + [vp]
    lib.ft_moe_nvfp4_decode_routed.restype = ctypes.c_int
    lib.ft_moe_nvfp4_decode_routed.argtypes = [vp, i32, vp, i32, ctypes.POINTER(_Experts),
                                               ctypes.POINTER(_Shared), f32, vp, vp, vp, vp, sz,
                                               vp]
    lib.ft_moe_last_cuda_error.restype = ctypes.c_char_p
    lib.ft_moe_get_error.restype = ctypes.c_int
    lib.ft_moe_get_error.argtypes = [vp, vp]
    lib.ft_moe_layer_from_host.restype = ctypes.c_int
    lib.ft_moe_layer_from_host.argtypes = [vp, vp, i32, i32, ctypes.POINTER(_Experts),
                                           ctypes.POINTER(_Shared), f32, vp, vp, vp, vp, vp, vp,
                                           vp, sz, vp]
    lib.ft_moe_router_logits.restype = ctypes.c_int
    lib.ft_moe_router_logits.argtypes = [vp, i32, i32, vp, i32, vp, vp, vp, vp]
    lib.ft_moe_router_route.restype = ctypes.c_int
    lib.ft_moe_router_route.argtypes = [vp, i32, i32, vp, i32, vp, i32, vp, vp, vp, vp, vp]
    lib.ft_moe_fp8block_workspace_bytes.restype = sz
    lib.ft_moe_fp8block_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.ft_moe_fp8block_decode.restype = ctypes.c_int
    lib.ft_moe_fp8block_decode.argtypes = [vp, i32, vp, vp, i32, ctypes.POINTER(_F8Experts),
                                           ctypes.POINTER(_F8Shared), f32, vp, vp, sz, vp]
    i64 = ctypes.c_int64
    lib.ft_nvfp4_linear_workspace_bytes.restype = sz
    lib.ft_nvfp4_linear_workspace_bytes.argtypes = [i32, i32]
    lib.ft_nvfp4_linear.restype = ctypes.c_int
    lib.ft_nvfp4_linear.argtypes = [vp, i32, i64, ctypes.POINTER(_Matrix), vp, i32, vp, sz, vp]
    lib.ft_kv_append.restype = ctypes.c_int
    lib.ft_kv_append.argtypes = [vp, i64, vp, i64, vp, i64, vp, i32, i32, ctypes.POINTER(_PagedKV),
                                 vp, i32, i32, vp, vp, vp, i32, i32, vp, vp]
    lib.ft_paged_attention_workspace_bytes.restype = sz
    lib.ft_paged_attention_workspace_bytes.argtypes = [i32, i32]
    lib.ft_paged_decode_attention.restype = ctypes.c_int
    lib.ft_paged_decode_attention.argtypes = [vp, i64, i32, i32, ctypes.POINTER(_PagedKV), vp, i32,
                                              vp, f32, i32, vp, vp, vp, sz, vp]
    lib.ft_residual_norm.restype = ctypes.c_int
    lib.ft_residual_norm.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, f32, f32, vp, vp, vp]
    lib.ft_residual_norm_backward_workspace_bytes.restype = sz
    lib.ft_residual_norm_backward_workspace_bytes.argtypes = [i32, i32]
    lib.ft_residual_norm_backward.restype = ctypes.c_int
    lib.ft_residual_norm_backward.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, f32,
                                              f32, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.ft_moe_debug_set_wait_limit.restype = ctypes.c_int
    lib.ft_moe_debug_set_wait_limit.argtypes = [ctypes.c_int64]
    return lib


_LIB = load_library()


def lib() -> ctypes.CDLL:
    return _LIB


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _stream(stream, dev=None) -> int:
    if stream is None:
        if dev is not None and torch._C._cuda_getDevice() == dev:
            return torch._C._cuda_getCurrentRawStream(dev)
        stream = torch.cuda.current_stream()
    if dev is not None and stream.device_index != dev:
        raise ValueError(f"the tensors are on cuda:{dev}, the stream on cuda:{stream.device_index} "
                         "(torch.cuda.set_device selects the current device)")
    return stream.cuda_stream


def _check(st: int, what: str):
    if st != FT_OK:
        detail = _LIB.ft_moe_last_cuda_error().decode() if st == 5 else ""
        raise FtError(st, what, detail)


# The kernels reach every tensor through its raw pointer, so a host tensor, a narrower
# element type, a strided view or a wrong shape would be read or written out of bounds on
# the GPU. _need refuses those before the call (a few hundred ns per tensor); the expert
# tensors are checked once, when their objects are built.
BF16_BITS = (torch.bfloat16, torch.int16, torch.uint16)   # bf16 values or their bit patterns
_F32 = (torch.float32,)
_I32 = (torch.int32,)


def _need(t, name, dev, dtypes, shape):
    """t on cuda:dev, of one of `dtypes` (None: any 1-byte type), contiguous, of `shape`
    (None: any)."""
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on cuda:{dev}, got one on {t.device}")
    if (t.element_size() != 1) if dtypes is None else (t.dtype not in dtypes):
        raise TypeError(f"{name}: element type {t.dtype} is not accepted here")
    if not t.is_contiguous():
        raise ValueError(f"{name}: the tensor must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _need_scalar(t, name, dev):
    _need(t, name, dev, _F32, None)
    if t.numel() != 1:
        raise ValueError(f"{name}: one float32 value expected, got {t.numel()}")


def _device_of(t, what) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{what}: CUDA tensors are required, got one on {t.device}")
    return dev


@dataclass(frozen=True)
class NvFP4Experts:
    """Routed experts on the device: w13 u8 [E,2I,H/2], s13 u8 [E,2I,H/16], g13 f32 [E],
    w2 u8 [E,H,I/2], s2 u8 [E,H,I/16], g2 f32 [E] (codes and scales: any 1-byte type).
    Checked when built: one device, contiguous, consistent shapes."""
    w13: torch.Tensor
    s13: torch.Tensor
    g13: torch.Tensor
    w2: torch.Tensor
    s2: torch.Tensor
    g2: torch.Tensor

    def __post_init__(self):
        dev = _device_of(self.w13, "NvFP4Experts")
        if self.w13.dim() != 3 or self.w2.dim() != 3:
            raise ValueError("NvFP4Experts: w13 [E,2I,H/2] and w2 [E,H,I/2] are 3-D")
        E, H, I = self.E, self.H, self.I
        _need(self.w13, "w13", dev, None, (E, 2 * I, H // 2))
        _need(self.s13, "s13", dev, None, (E, 2 * I, H // 16))
        _need(self.g13, "g13", dev, _F32, (E,))
        _need(self.w2, "w2", dev, None, (E, H, I // 2))
        _need(self.s2, "s2", dev, None, (E, H, I // 16))
        _need(self.g2, "g2", dev, _F32, (E,))
        object.__setattr__(self, "device_index", dev)
        object.__setattr__(self, "_cs", _Experts(E, H, I, _ptr(self.w13), _ptr(self.s13),
                                                 _ptr(self.g13), _ptr(self.w2), _ptr(self.s2),
                                                 _ptr(self.g2)))

    @property
    def E(self):
        return self.w13.shape[0]

    @property
    def H(self):
        return self.w2.shape[1]

    @property
    def I(self):
        return self.w13.shape[1] // 2

    def cstruct(self) -> _Experts:
        return self._cs


@dataclass(frozen=True)
class NvFP4Shared:
    """Shared expert on the device (no E dimension): w13 [2I,H/2], s13 [2I,H/16], w2 [H,I/2],
    s2 [H,I/16] (any 1-byte type), g13/g2 1-element f32 tensors and gate bf16 [H] (or a
    16-bit integer tensor holding the bf16 bits). Checked when built."""
    w13: torch.Tensor
    s13: torch.Tensor
    g13: torch.Tensor
    w2: torch.Tensor
    s2: torch.Tensor
    g2: torch.Tensor
    gate: torch.Tensor

    def __post_init__(self):
        dev = _device_of(self.w13, "NvFP4Shared")
        if self.w13.dim() != 2 or self.w2.dim() != 2:
            raise ValueError("NvFP4Shared: w13 [2I,H/2] and w2 [H,I/2] are 2-D")
        H, I = self.w2.shape[0], self.w13.shape[0] // 2
        _need(self.w13, "shared w13", dev, None, (2 * I, H // 2))
        _need(self.s13, "shared s13", dev, None, (2 * I, H // 16))
        _need(self.w2, "shared w2", dev, None, (H, I // 2))
        _need(self.s2, "shared s2", dev, None, (H, I // 16))
        _need_scalar(self.g13, "shared g13", dev)
        _need_scalar(self.g2, "shared g2", dev)
        _need(self.gate, "shared gate", dev, BF16_BITS, (H,))
        object.__setattr__(self, "device_index", dev)
        object.__setattr__(self, "H", H)
        object.__setattr__(self, "I", I)
        object.__setattr__(self, "_cs", _Shared(_ptr(self.w13), _ptr(self.s13), _ptr(self.g13),
                                                _ptr(self.w2), _ptr(self.s2), _ptr(self.g2),
                                                _ptr(self.gate)))

    def check_for(self, experts: NvFP4Experts):
        if (self.device_index, self.H, self.I) != (experts.device_index, experts.H, experts.I):
            raise ValueError("shared expert: H, I and the device must match the routed experts")

    def cstruct(self) -> _Shared:
        return self._cs


@dataclass(frozen=True)
class Fp8BlockExperts:
    """Block-FP8 routed experts on the device: w13 u8 [E,2I,H] (E4M3 codes), s13 f32
    [E,2I/128,H/128], w2 u8 [E,H,I], s2 f32 [E,H/128,I/128]. Checked when built."""
    w13: torch.Tensor
    s13: torch.Tensor
    w2: torch.Tensor
    s2: torch.Tensor

    def __post_init__(self):
        dev = _device_of(self.w13, "Fp8BlockExperts")
        if self.w13.dim() != 3 or self.w2.dim() != 3:
            raise ValueError("Fp8BlockExperts: w13 [E,2I,H] and w2 [E,H,I] are 3-D")
        E, H, I = self.w13.shape[0], self.w2.shape[1], self.w13.shape[1] // 2
        t = lambda n: -(-n // 128)
        _need(self.w13, "w13", dev, None, (E, 2 * I, H))
        _need(self.s13, "s13", dev, _F32, (E, t(2 * I), t(H)))
        _need(self.w2, "w2", dev, None, (E, H, I))
        _need(self.s2, "s2", dev, _F32, (E, t(H), t(I)))
        object.__setattr__(self, "device_index", dev)
        object.__setattr__(self, "E", E)
        object.__setattr__(self, "H", H)
        object.__setattr__(self, "I", I)
        object.__setattr__(self, "_cs", _F8Experts(E, H, I, _ptr(self.w13), _ptr(self.s13),
                                                   _ptr(self.w2), _ptr(self.s2)))

    def cstruct(self) -> _F8Experts:
        return self._cs


@dataclass(frozen=True)
class Fp8BlockShared:
    """Block-FP8 shared expert (no E dimension) and its gate vector bf16 [H]."""
    w13: torch.Tensor
    s13: torch.Tensor
    w2: torch.Tensor
    s2: torch.Tensor
    gate: torch.Tensor

    def __post_init__(self):
        dev = _device_of(self.w13, "Fp8BlockShared")
        H, I = self.w2.shape[0], self.w13.shape[0] // 2
        t = lambda n: -(-n // 128)
        _need(self.w13, "shared w13", dev, None, (2 * I, H))
        _need(self.s13, "shared s13", dev, _F32, (t(2 * I), t(H)))
        _need(self.w2, "shared w2", dev, None, (H, I))
        _need(self.s2, "shared s2", dev, _F32, (t(H), t(I)))
        _need(self.gate, "shared gate", dev, BF16_BITS, (H,))
        object.__setattr__(self, "device_index", dev)
        object.__setattr__(self, "H", H)
        object.__setattr__(self, "I", I)
        object.__setattr__(self, "_cs", _F8Shared(_ptr(self.w13), _ptr(self.s13), _ptr(self.w2),
                                                  _ptr(self.s2), _ptr(self.gate)))

    def check_for(self, experts):
        if (self.device_index, self.H, self.I) != (experts.device_index, experts.H, experts.I):
            raise ValueError("shared expert: H, I and the device must match the routed experts")

    def cstruct(self) -> _F8Shared:
        return self._cs


def abi_version() -> int:
    return _LIB.ft_moe_abi_version()


def status_string(st: int) -> str:
    return _LIB.ft_status_string(st).decode()


def route(logits: torch.Tensor, k: int, topk_idx=None, topk_w=None, stream=None):
    """ft_moe_route on fp32 logits [T, E] (device). Returns (idx int32 [T,k], w f32 [T,k])."""
    dev = _device_of(logits, "ft_moe_route")
    if logits.dim() != 2:
        raise ValueError("logits: [T, E] expected")
    _need(logits, "logits", dev, _F32, None)
    T, E = logits.shape
    if topk_idx is None:
        topk_idx = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    else:
        _need(topk_idx, "topk_idx", dev, _I32, (T, k))
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    else:
        _need(topk_w, "topk_w", dev, _F32, (T, k))
    st = _LIB.ft_moe_route(_ptr(logits), T, E, k, _ptr(topk_idx), _ptr(topk_w),
                           _stream(stream, dev))
    _check(st, "ft_moe_route")
    return topk_idx, topk_w


def router_logits(x, w_router, gate=None, logits=None, gate_dot=None, stream=None):
    """ft_moe_router_logits: bf16 x [T,H] and router weights [E,H] (and a bf16 gate [H]) ->
    (logits f32 [T,E], gate dots f32 [T] or None)."""
    dev = _device_of(x, "ft_moe_router_logits")
    if x.dim() != 2 or w_router.dim() != 2:
        raise ValueError("x [T, H] and w_router [E, H] expected")
    T, H = x.shape
    E = w_router.shape[0]
    _need(x, "x", dev, BF16_BITS, (T, H))
    _need(w_router, "w_router", dev, BF16_BITS, (E, H))
    if gate is not None:
        _need(gate, "gate", dev, BF16_BITS, (H,))
    if logits is None:
        logits = torch.empty((T, E), dtype=torch.float32, device=x.device)
    _need(logits, "logits", dev, _F32, (T, E))
    if gate is not None and gate_dot is None:
        gate_dot = torch.empty((T,), dtype=torch.float32, device=x.device)
    if gate_dot is not None:
        _need(gate_dot, "gate_dot", dev, _F32, (T,))
    st = _LIB.ft_moe_router_logits(_ptr(x), T, H, _ptr(w_router), E, _ptr(gate), _ptr(logits),
                                   _ptr(gate_dot), _stream(stream, dev))
    _check(st, "ft_moe_router_logits")
    return logits, gate_dot


def router_route(x, w_router, k, gate=None, stream=None):
    """ft_moe_router_route: the routing slots (idx int32 [T,k], w f32 [T,k]) from x and the
    router matrix; returns (idx, w, logits, gate dots or None)."""
    dev = _device_of(x, "ft_moe_router_route")
    T, H = x.shape
    E = w_router.shape[0]
    _need(x, "x", dev, BF16_BITS, (T, H))
    _need(w_router, "w_router", dev, BF16_BITS, (E, H))
    if gate is not None:
        _need(gate, "gate", dev, BF16_BITS, (H,))
    logits = torch.empty((T, E), dtype=torch.float32, device=x.device)
    gate_dot = torch.empty((T,), dtype=torch.float32, device=x.device) if gate is not None else None
    idx = torch.empty((T, k), dtype=torch.int32, device=x.device)
    w = torch.empty((T, k), dtype=torch.float32, device=x.device)
    st = _LIB.ft_moe_router_route(_ptr(x), T, H, _ptr(w_router), E, _ptr(gate), k, _ptr(logits),
                                  _ptr(gate_dot), _ptr(idx), _ptr(w), _stream(stream, dev))
    _check(st, "ft_moe_router_route")
    return idx, w, logits, gate_dot


def workspace_bytes(T, k, E, H, I, has_shared, prefill=False) -> int:
    return _LIB.ft_moe_workspace_bytes(T, k, E, H, I, int(bool(has_shared)), int(bool(prefill)))


def new_workspace(T, k, experts: NvFP4Experts, has_shared, prefill=False, device=None,
                  stream=None) -> torch.Tensor:
    n = workspace_bytes(T, k, experts.E, experts.H, experts.I, has_shared, prefill)
    if n == 0 and T == 0:   # an empty batch needs no workspace
        return torch.empty(0, dtype=torch.uint8, device=device or experts.w13.device)
    if n == 0:
        raise FtError(2, "ft_moe_workspace_bytes")
    ws = torch.empty(n + 256, dtype=torch.uint8, device=device or experts.w13.device)
    off = (-ws.data_ptr()) % 256                      # 256-byte aligned view
    ws = ws[off:off + n]
    _check(_LIB.ft_moe_workspace_init(_ptr(ws), n, _stream(stream)), "ft_moe_workspace_init")
    return ws


# Calls made without a workspace share one per (host thread, device, stream). Launches on one
# stream run in order, so a call never finds its workspace in use by an earlier call that is
# still running; a call of several launches is not one step for another thread, whose launches
# may come between them, so threads do not share. The workspace grows (a new, larger one) when a
# call needs more; nothing is allocated on calls that fit. The old one goes back to its stream's
# pool, and no graph holds its address: a call that is being captured takes a workspace from
# the capture's own pool, which lives as long as the graph.
class _Kept(threading.local):
    def __init__(self):
        self.by_stream = {}


_KEPT = _Kept()


def _new_scratch(n, dev, head=True):
    ws = torch.empty(n + 256, dtype=torch.uint8, device=torch.device("cuda", dev))
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + n]
    if head:
        _check(_LIB.ft_moe_workspace_init(_ptr(ws), min(n, WORKSPACE_HEAD_BYTES), _stream(None, dev)),
               "ft_moe_workspace_init")
    return ws


def _scratch(n, dev, head=False):
    """n bytes at least for a call on the current stream of cuda:dev. head: its counters are needed
    (zeroed in a captured workspace too; kept ones always are)."""
    if torch._C._cuda_isCurrentStreamCapturing():
        return _new_scratch(n, dev, head)
    kept, key = _KEPT.by_stream, (dev, torch._C._cuda_getCurrentRawStream(dev))
    ws = kept.get(key)
    if ws is None or ws.numel() < n:
        old, ws = ws, _new_scratch(n, dev)
        if old is not None:
            ws[:4].copy_(old[:4])   # the flags of earlier calls
        kept[key] = ws
    return ws


def default_workspace(T, k, experts: NvFP4Experts, has_shared, prefill=False, stream=None):
    """The workspace a call without one uses: kept per (host thread, device, stream) and reused,
    or, while the stream is captured, one of the capture's own."""
    if stream is not None:
        with torch.cuda.stream(stream):   # it belongs to the stream that uses it
            return default_workspace(T, k, experts, has_shared, prefill)
    n = workspace_bytes(T, k, experts.E, experts.H, experts.I, has_shared, prefill)
    if n == 0:
        return new_workspace(T, k, experts, has_shared, prefill)
    return _scratch(n, experts.device_index, True)


def _call_tensors(experts, shared, x, out, workspace, T_name="x"):
    """Checks shared by the layer calls: x [T,H] and out [T,H] (bf16 bits), the shared expert
    against the routed ones, the workspace (1-byte elements: numel() is its size in bytes).
    Returns (device, T, out)."""
    dev = experts.device_index
    if x.dim() != 2:
        raise ValueError(f"{T_name}: [T, H] expected")
    T = x.shape[0]
    _need(x, T_name, dev, BF16_BITS, (T, experts.H))
    if shared is not None:
        shared.check_for(experts)
    if out is None:
        out = torch.empty((T, experts.H), dtype=torch.bfloat16, device=x.device)
    else:
        _need(out, "out", dev, BF16_BITS, (T, experts.H))
    if workspace is not None:
        _need(workspace, "workspace", dev, None, None)
    return dev, T, out


def _slots(topk_idx, topk_w, T, dev):
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx: [T, k] expected")
    k = topk_idx.shape[1]
    _need(topk_idx, "topk_idx", dev, _I32, (T, k))
    _need(topk_w, "topk_w", dev, _F32, (T, k))
    return k


def _layer(fn, name, x, topk_idx, topk_w, experts, shared, limit, out, workspace, stream):
    dev, T, out = _call_tensors(experts, shared, x, out, workspace)
    k = _slots(topk_idx, topk_w, T, dev)
    ex = experts.cstruct()
    sh = shared.cstruct() if shared is not None else None
    st = fn(_ptr(x), T, _ptr(topk_idx), _ptr(topk_w), k, ctypes.byref(ex),
            ctypes.byref(sh) if sh is not None else None, float(limit), _ptr(out),
            _ptr(workspace), workspace.numel(), _stream(stream, dev))
    _check(st, name)
    return out


def decode(x, topk_idx, topk_w, experts, shared=None, limit=7.0, out=None, workspace=None,
           stream=None):
    """ft_moe_nvfp4_decode: x bf16 [T,H] (T <= 64) -> out bf16 [T,H]."""
    if workspace is None:
        workspace = default_workspace(x.shape[0], topk_idx.shape[1], experts, shared is not None,
                                      stream=stream)
    return _layer(_LIB.ft_moe_nvfp4_decode, "ft_moe_nvfp4_decode", x, topk_idx, topk_w,
                  experts, shared, limit, out, workspace, stream)


def decode_noalloc(x, topk_idx, topk_w, experts, shared=None, limit=7.0, out=None,
                   stream=None):
    """ft_moe_nvfp4_decode_noalloc: decode with the library's fixed scratch array (no
    workspace, no device allocation by the library)."""
    dev, T, out = _call_tensors(experts, shared, x, out, None)
    k = _slots(topk_idx, topk_w, T, dev)
    ex = experts.cstruct()
    sh = shared.cstruct() if shared is not None else None
    st = _LIB.ft_moe_nvfp4_decode_noalloc(_ptr(x), T, _ptr(topk_idx), _ptr(topk_w), k,
                                          ctypes.byref(ex),
                                          ctypes.byref(sh) if sh is not None else None,
                                          float(limit), _ptr(out), _stream(stream, dev))
    _check(st, "ft_moe_nvfp4_decode_noalloc")
    return out


def decode_routed(x, logits, k, experts, shared=None, limit=7.0, out=None, topk_idx=None,
                  topk_w=None, workspace=None, stream=None):
    """ft_moe_nvfp4_decode_routed: the layer from the router logits f32 [T,E] (T <= 64); one
    launch for T = 1. topk_idx / topk_w (int32 / f32 [T,k]), when given, receive the slots."""
    if workspace is None:
        workspace = default_workspace(x.shape[0], k, experts, shared is not None, stream=stream)
    dev, T, out = _call_tensors(experts, shared, x, out, workspace)
    _need(logits, "logits", dev, _F32, (T, experts.E))
    if topk_idx is not None:
        _need(topk_idx, "topk_idx", dev, _I32, (T, k))
    if topk_w is not None:
        _need(topk_w, "topk_w", dev, _F32, (T, k))
    ex = experts.cstruct()
    sh = shared.cstruct() if shared is not None else None
    st = _LIB.ft_moe_nvfp4_decode_routed(_ptr(x), T, _ptr(logits), k, ctypes.byref(ex),
                                         ctypes.byref(sh) if sh is not None else None,
                                         float(limit), _ptr(out), _ptr(topk_idx), _ptr(topk_w),
                                         _ptr(workspace), workspace.numel(), _stream(stream, dev))
    _check(st, "ft_moe_nvfp4_decode_routed")
    return out


def prefill(x, topk_idx, topk_w, experts, shared=None, limit=7.0, out=None, workspace=None,
            stream=None):
    """ft_moe_nvfp4_prefill: x bf16 [T,H] (any T) -> out bf16 [T,H]."""
    if workspace is None:
        workspace = default_workspace(x.shape[0], topk_idx.shape[1], experts, shared is not None,
                                      prefill=True, stream=stream)
    return _layer(_LIB.ft_moe_nvfp4_prefill, "ft_moe_nvfp4_prefill", x, topk_idx, topk_w,
                  experts, shared, limit, out, workspace, stream)


def _need_host(t, name, dtypes, shape):
    if t.device.type != "cpu":
        raise ValueError(f"{name}: expected a host tensor, got one on {t.device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: element type {t.dtype} is not accepted here")
    if not t.is_contiguous():
        raise ValueError(f"{name}: the tensor must be contiguous")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def layer_from_host(x_host, logits_host, k, experts, shared=None, limit=7.0, out_host=None,
                    x_dev=None, logits_dev=None, out_dev=None, topk_idx_dev=None,
                    topk_w_dev=None, workspace=None, stream=None):
    """ft_moe_layer_from_host: x bf16 [T,H] and logits f32 [T,E] in host memory (pinned for
    asynchronous copies) -> out_host bf16 [T,H], with the device buffers given (or made
    here). Everything is enqueued on the stream; the host output is ready once it is
    synchronised. Returns out_host."""
    dev = experts.device_index
    if x_host.dim() != 2:
        raise ValueError("x_host: [T, H] expected")
    T, H, E = x_host.shape[0], experts.H, experts.E
    _need_host(x_host, "x_host", BF16_BITS, (T, H))
    _need_host(logits_host, "logits_host", _F32, (T, E))
    if out_host is None:
        out_host = torch.empty((T, H), dtype=torch.bfloat16).pin_memory()
    else:
        _need_host(out_host, "out_host", BF16_BITS, (T, H))
    if shared is not None:
        shared.check_for(experts)
    cuda = torch.device("cuda", dev)
    x_dev = torch.empty((T, H), dtype=torch.bfloat16, device=cuda) if x_dev is None else x_dev
    logits_dev = (torch.empty((T, E), dtype=torch.float32, device=cuda) if logits_dev is None
                  else logits_dev)
    out_dev = torch.empty((T, H), dtype=torch.bfloat16, device=cuda) if out_dev is None else out_dev
    _need(x_dev, "x_dev", dev, BF16_BITS, (T, H))
    _need(logits_dev, "logits_dev", dev, _F32, (T, E))
    _need(out_dev, "out_dev", dev, BF16_BITS, (T, H))
    prefill = T > 64
    if prefill and topk_idx_dev is None:
        topk_idx_dev = torch.empty((T, k), dtype=torch.int32, device=cuda)
    if prefill and topk_w_dev is None:
        topk_w_dev = torch.empty((T, k), dtype=torch.float32, device=cuda)
    if topk_idx_dev is not None:
        _need(topk_idx_dev, "topk_idx_dev", dev, _I32, (T, k))
    if topk_w_dev is not None:
        _need(topk_w_dev, "topk_w_dev", dev, _F32, (T, k))
    if workspace is None:
        workspace = default_workspace(T, k, experts, shared is not None, prefill=prefill,
                                      stream=stream)
    _need(workspace, "workspace", dev, None, None)
    ex = experts.cstruct()
    sh = shared.cstruct() if shared is not None else None
    st = _LIB.ft_moe_layer_from_host(_ptr(x_host), _ptr(logits_host), T, k, ctypes.byref(ex),
                                     ctypes.byref(sh) if sh is not None else None, float(limit),
                                     _ptr(out_host), _ptr(x_dev), _ptr(logits_dev),
                                     _ptr(topk_idx_dev), _ptr(topk_w_dev), _ptr(out_dev),
                                     _ptr(workspace), workspace.numel(), _stream(stream, dev))
    _check(st, "ft_moe_layer_from_host")
    return out_host


def fp8block_workspace_bytes(T, k, E, H, I, has_shared) -> int:
    return _LIB.ft_moe_fp8block_workspace_bytes(T, k, E, H, I, int(bool(has_shared)))


def new_fp8block_workspace(T, k, experts: Fp8BlockExperts, has_shared, stream=None):
    n = fp8block_workspace_bytes(T, k, experts.E, experts.H, experts.I, has_shared)
    if n == 0:
        raise FtError(2, "ft_moe_fp8block_workspace_bytes")
    ws = torch.empty(n + 256, dtype=torch.uint8, device=experts.w13.device)
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + n]
    _check(_LIB.ft_moe_workspace_init(_ptr(ws), n, _stream(stream)), "ft_moe_workspace_init")
    return ws


def fp8block_decode(x, topk_idx, topk_w, experts: Fp8BlockExperts, shared=None, limit=7.0,
                    out=None, workspace=None, stream=None):
    """ft_moe_fp8block_decode: x bf16 [T,H] (T <= 64) with block-FP8 experts -> out bf16
    [T,H]."""
    if workspace is None:
        workspace = new_fp8block_workspace(x.shape[0], topk_idx.shape[1], experts,
                                           shared is not None, stream=stream)
    dev, T, out = _call_tensors(experts, shared, x, out, workspace)
    k = _slots(topk_idx, topk_w, T, dev)
    ex = experts.cstruct()
    sh = shared.cstruct() if shared is not None else None
    st = _LIB.ft_moe_fp8block_decode(_ptr(x), T, _ptr(topk_idx), _ptr(topk_w), k,
                                     ctypes.byref(ex), ctypes.byref(sh) if sh is not None else None,
                                     float(limit), _ptr(out), _ptr(workspace), workspace.numel(),
                                     _stream(stream, dev))
    _check(st, "ft_moe_fp8block_decode")
    return out


# ---------------------------------------------------------------- the decode block
# The operators between two layer calls: dense NVFP4 products, cache append, attention of one new
# token per sequence and the norms around the gated residual sum. Sizes come from the tensors;
# what the kernels require beyond them (multiples, ranges) is refused by the library with its
# status, what they would read out of bounds is refused here.
GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_ELEMENT = range(4)
_MAX_I32 = 2 ** 31 - 1   # sizes are 32-bit in the C ABI, and ctypes drops the bits above
_RES = (torch.bfloat16, torch.float32)


def _need_rows(t, name, dev, inner):
    """t on cuda:dev, bf16 bits [T, *inner] whose rows are contiguous: the distance between rows
    may be larger than a row (a slice of a wider tensor). Returns it, in elements."""
    shape = t.shape
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on cuda:{dev}, got one on {t.device}")
    if t.dtype not in BF16_BITS:
        raise TypeError(f"{name}: element type {t.dtype} is not accepted here")
    if shape[1:] != inner:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected [T, {', '.join(map(str, inner))}]")
    stride, last = t.stride(), inner[-1]
    row = last if len(inner) == 1 else inner[0] * last
    if (stride[-1] != 1 and last != 1) or (len(inner) == 2 and stride[1] != last and inner[0] != 1):
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    if shape[0] <= 1:
        return row
    if stride[0] < row:
        raise ValueError(f"{name}: the rows must not overlap")
    return stride[0]


@dataclass(frozen=True)
class NvFP4Linear:
    """A dense NVFP4 matrix on the device: codes u8 [N,K/2], scales u8 [N,K/16] (any 1-byte type),
    gscale a 1-element f32 tensor. Checked when built."""
    codes: torch.Tensor
    scales: torch.Tensor
    gscale: torch.Tensor

    def __post_init__(self):
        dev = _device_of(self.codes, "NvFP4Linear")
        if self.codes.dim() != 2:
            raise ValueError("NvFP4Linear: codes [N,K/2] are 2-D")
        N, K = self.codes.shape[0], self.codes.shape[1] * 2
        if K % 32 != 0 or K == 0 or N == 0:
            raise ValueError("NvFP4Linear: K is a multiple of 32, and N is not 0")
        if N > _MAX_I32 or K > _MAX_I32:
            raise ValueError(f"NvFP4Linear: [{N}, {K}] is too large")
        _need(self.codes, "codes", dev, None, (N, K // 2))
        _need(self.scales, "scales", dev, None, (N, K // 16))
        _need_scalar(self.gscale, "gscale", dev)
        object.__setattr__(self, "device_index", dev)
        object.__setattr__(self, "N", N)
        object.__setattr__(self, "K", K)
        object.__setattr__(self, "_cs", _Matrix(N, K, _ptr(self.codes), _ptr(self.scales),
                                                _ptr(self.gscale)))
        object.__setattr__(self, "_ref", ctypes.byref(self._cs))


def nvfp4_linear_workspace_bytes(T, K) -> int:
    return _LIB.ft_nvfp4_linear_workspace_bytes(T, K)


def nvfp4_linear(x, weight: NvFP4Linear, out=None, out_dtype=torch.bfloat16, workspace=None,
                 stream=None):
    """ft_nvfp4_linear: x bf16 [T,K] (T <= 64; rows may be slices of a wider tensor) -> W x_t,
    [T,N] in bf16, or in float32 (out_dtype, or the type of `out`)."""
    if stream is not None:
        with torch.cuda.stream(stream):   # what the call makes belongs to the stream that it runs on
            return nvfp4_linear(x, weight, out, out_dtype, workspace)
    dev = weight.device_index
    if x.dim() != 2:
        raise ValueError("x: [T, K] expected")
    stride = _need_rows(x, "x", dev, (weight.K,))
    T = x.shape[0]
    if out is None:
        if out_dtype not in _RES:
            raise TypeError(f"out_dtype: {out_dtype} is not accepted here")
        out = torch.empty((T, weight.N), dtype=out_dtype, device=x.device)
    else:
        _need(out, "out", dev, _RES, (T, weight.N))
    ws, ws_bytes = 0, 0
    if workspace is not None:
        _need(workspace, "workspace", dev, None, None)
        ws, ws_bytes = workspace.data_ptr(), workspace.numel()
    elif T > 8:   # fewer tokens need none
        n = _LIB.ft_nvfp4_linear_workspace_bytes(T, weight.K)
        if n > 0:
            workspace = _scratch(n, dev)
            ws, ws_bytes = workspace.data_ptr(), workspace.numel()
    st = _LIB.ft_nvfp4_linear(x.data_ptr(), T, stride, weight._ref, out.data_ptr(),
                              out.dtype is torch.float32, ws, ws_bytes, _stream(None, dev))
    _check(st, "ft_nvfp4_linear")
    return out


@dataclass(frozen=True)
class PagedKVCache:
    """A paged key-value cache on the device: k and v [num_pages, page_size, Hkv, D], bf16 or
    float8_e4m3fn (values are code * scale), elements of a head contiguous and the other strides
    free (a permuted view of [page, head, slot, d] storage is fine). Checked when built."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: float = 1.0
    v_scale: float = 1.0

    def __post_init__(self):
        dev = _device_of(self.k, "PagedKVCache")
        if self.k.dim() != 4 or self.k.shape != self.v.shape:
            raise ValueError("PagedKVCache: k and v [num_pages, page_size, Hkv, D] of one shape")
        if self.v.get_device() != dev:
            raise ValueError("PagedKVCache: k and v must be on one device")
        if self.k.dtype not in (torch.bfloat16, torch.float8_e4m3fn) or self.k.dtype != self.v.dtype:
            raise TypeError("PagedKVCache: k and v are both bfloat16 or both float8_e4m3fn")
        if self.k.stride(3) != 1 or self.v.stride(3) != 1:
            raise ValueError("PagedKVCache: the elements of a head must be contiguous")
        if max(self.k.shape) > _MAX_I32:
            raise ValueError(f"PagedKVCache: {tuple(self.k.shape)} is too large")
        f8 = self.k.dtype == torch.float8_e4m3fn
        object.__setattr__(self, "device_index", dev)
        object.__setattr__(self, "heads", tuple(self.k.shape[2:]))   # (Hkv, D)
        object.__setattr__(self, "_cs", _PagedKV(
            _ptr(self.k), _ptr(self.v), *self.k.shape, *self.k.stride()[:3], *self.v.stride()[:3],
            int(f8), float(self.k_scale), float(self.v_scale)))
        object.__setattr__(self, "_ref", ctypes.byref(self._cs))

    @property
    def page_size(self):
        return self._cs.page_size

    @property
    def Hkv(self):
        return self.heads[0]

    @property
    def D(self):
        return self.heads[1]


def kv_append(k, v, cache: PagedKVCache, block_table, positions, seq_ids=None, q=None, rope=None,
              q_out=None, workspace=None, stream=None):
    """ft_kv_append: k, v bf16 [T,Hkv,D] into the cache's slots of `positions` int32 [T] (of the
    sequences seq_ids int32 [T], or 0..T-1) through block_table int32 [B,width], k rotated by rope
    f32 [rows, R] (cos | sin; None: not at all). Returns the rotated q bf16 [T,Hq,D], or None
    without q. Rows of k, v and q may be slices of one projection's output. A token whose page,
    sequence or position lies outside its table stores nothing and flags it (get_error)."""
    if stream is not None:
        with torch.cuda.stream(stream):   # what the call makes belongs to the stream that it runs on
            return kv_append(k, v, cache, block_table, positions, seq_ids, q, rope, q_out, workspace)
    dev, inner = cache.device_index, cache.heads
    if k.dim() != 3 or block_table.dim() != 2:
        raise ValueError("k [T, Hkv, D] and block_table [B, width] expected")
    T, D = k.shape[0], inner[1]
    ks, vs = _need_rows(k, "k", dev, inner), _need_rows(v, "v", dev, inner)
    if v.shape[0] != T:
        raise ValueError("v: as many tokens as k expected")
    _need(block_table, "block_table", dev, _I32, None)
    _need(positions, "positions", dev, _I32, (T,))
    B, width = block_table.shape
    if T > _MAX_I32 or B > _MAX_I32 or width > _MAX_I32:
        raise ValueError(f"{T} tokens, block_table [{B}, {width}]: too large")
    if seq_ids is not None:
        _need(seq_ids, "seq_ids", dev, _I32, (T,))
    elif T > B:
        raise ValueError("seq_ids: required for more tokens than block_table has rows")
    Hq = qs = qp = qo = 0
    if q is not None:
        if q.dim() != 3 or q.shape[0] != T:
            raise ValueError("q: [T, Hq, D] expected")
        Hq = q.shape[1]
        qs = _need_rows(q, "q", dev, (Hq, D))
        if q_out is None:
            q_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=q.device)
        else:
            _need(q_out, "q_out", dev, BF16_BITS, (T, Hq, D))
        qp, qo = q.data_ptr(), q_out.data_ptr()
    rows = dim = rp = 0
    if rope is not None:
        if rope.dim() != 2:
            raise ValueError("rope: [rows, R] expected")
        _need(rope, "rope", dev, _F32, None)
        rows, dim = rope.shape
        if rows > _MAX_I32:
            raise ValueError(f"rope: {rows} rows are too many")
        rp = rope.data_ptr()
    if workspace is not None:
        _need(workspace, "workspace", dev, None, None)
        if workspace.numel() < WORKSPACE_HEAD_BYTES:
            raise ValueError("workspace: at least WORKSPACE_HEAD_BYTES expected")
    elif T > 0:
        workspace = _scratch(WORKSPACE_HEAD_BYTES, dev)   # for its flags
    st = _LIB.ft_kv_append(k.data_ptr(), ks, v.data_ptr(), vs, qp, qs, qo, T, Hq, cache._ref,
                           block_table.data_ptr(), B, width,
                           0 if seq_ids is None else seq_ids.data_ptr(), positions.data_ptr(), rp,
                           rows, dim, 0 if workspace is None else workspace.data_ptr(),
                           _stream(None, dev))
    if st != FT_OK:
        _check(st, "ft_kv_append")
    return q_out if q is not None else None


def paged_attention_workspace_bytes(B, D) -> int:
    return _LIB.ft_paged_attention_workspace_bytes(B, D)


@functools.lru_cache(maxsize=1024)
def _attention_bytes(B, D, dev) -> int:   # a size of the device's, asked for once
    n = _LIB.ft_paged_attention_workspace_bytes(B, D)
    if n == 0:
        raise FtError(2, "ft_paged_attention_workspace_bytes")
    return n


def paged_decode_attention(q, cache: PagedKVCache, block_table, seq_lens, scale=None, window=0,
                           out=None, lse=None, workspace=None, stream=None):
    """ft_paged_decode_attention: q bf16 [B,Hq,D], one new token per sequence, over the first
    seq_lens int32 [B] slots of each (the last `window` of them if window > 0) through block_table
    int32 [B,width]. scale: 1/sqrt(D) by default. Returns (out bf16 [B,Hq,D], lse f32 [B,Hq])."""
    if stream is not None:
        with torch.cuda.stream(stream):   # what the call makes belongs to the stream that it runs on
            return paged_decode_attention(q, cache, block_table, seq_lens, scale, window, out, lse,
                                          workspace)
    dev, D = cache.device_index, cache.heads[1]
    if q.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q [B, Hq, D] and block_table [B, width] expected")
    B, Hq, _ = q.shape
    qs = _need_rows(q, "q", dev, (Hq, D))
    _need(block_table, "block_table", dev, _I32, None)
    rows, width = block_table.shape
    if rows != B:
        raise ValueError(f"block_table: {rows} rows for {B} sequences")
    if B > _MAX_I32 or width > _MAX_I32 or window > _MAX_I32:
        raise ValueError(f"{B} sequences, {width} pages each, window {window}: out of range")
    _need(seq_lens, "seq_lens", dev, _I32, (B,))
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=q.device)
    else:
        _need(out, "out", dev, BF16_BITS, (B, Hq, D))
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    else:
        _need(lse, "lse", dev, _F32, (B, Hq))
    if workspace is not None:
        _need(workspace, "workspace", dev, None, None)
    elif B > 0:
        workspace = _scratch(_attention_bytes(B, D, dev), dev)
    st = _LIB.ft_paged_decode_attention(
        q.data_ptr(), qs, B, Hq, cache._ref, block_table.data_ptr(), width, seq_lens.data_ptr(),
        D ** -0.5 if scale is None else scale, window, out.data_ptr(), lse.data_ptr(),
        0 if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel(), _stream(None, dev))
    if st != FT_OK:
        _check(st, "ft_paged_decode_attention")
    return out, lse


def _norm_inputs(y, residual, w_post, w_pre, gate):
    """Checks shared by the norm and its gradient. Returns (device, T, H, gate kind, stream type)."""
    dev = _device_of(y, "ft_residual_norm")
    if y.dim() != 2:
        raise ValueError("y: [T, H] expected")
    T, H = both = y.shape
    if T > _MAX_I32:
        raise ValueError(f"y: {T} rows are too many")
    _need(y, "y", dev, BF16_BITS, None)
    res = torch.bfloat16
    if residual is not None:
        _need(residual, "residual", dev, _RES, both)
        res = residual.dtype
    if w_post is not None:
        _need(w_post, "w_post", dev, BF16_BITS, (H,))
    if w_pre is not None:
        _need(w_pre, "w_pre", dev, BF16_BITS, (H,))
    kind = GATE_NONE
    if gate is not None:
        shape = gate.shape
        if shape == both:
            kind = GATE_ELEMENT
        elif shape == (T, 1):
            kind = GATE_TOKEN
        elif shape == (H,):
            kind = GATE_CHANNEL
        else:
            raise ValueError(f"gate: shape {tuple(shape)}, expected ({H},), ({T}, 1) or ({T}, {H})")
        _need(gate, "gate", dev, BF16_BITS, None)
    return dev, T, H, kind, res


def residual_norm(y, residual=None, w_post=None, w_pre=None, gate=None, scale=1.0, eps=1e-6,
                  res_out=None, x_out=None, stream=None):
    """ft_residual_norm: r' = residual + scale * gate * norm(y, w_post) and x' = norm(r', w_pre) for
    y bf16 [T,H]; a weight that is None leaves its norm out. gate bf16 [H], [T,1] or [T,H].
    Returns (r' in the residual's type, x' bf16 or None without w_pre)."""
    if stream is not None:
        with torch.cuda.stream(stream):   # what the call makes belongs to the stream that it runs on
            return residual_norm(y, residual, w_post, w_pre, gate, scale, eps, res_out, x_out)
    dev, T, H, kind, res = _norm_inputs(y, residual, w_post, w_pre, gate)
    if res_out is None:
        res_out = torch.empty_like(y if residual is None else residual, dtype=res)
    else:
        _need(res_out, "res_out", dev, _RES if residual is None else (res,), (T, H))
        res = res_out.dtype
    x = 0
    if w_pre is None:
        x_out = None
    else:
        if x_out is None:
            x_out = torch.empty_like(y, dtype=torch.bfloat16)
        else:
            _need(x_out, "x_out", dev, BF16_BITS, (T, H))
        x = x_out.data_ptr()
    st = _LIB.ft_residual_norm(
        y.data_ptr(), 0 if residual is None else residual.data_ptr(),
        0 if w_post is None else w_post.data_ptr(), 0 if w_pre is None else w_pre.data_ptr(),
        0 if gate is None else gate.data_ptr(), kind, T, H, res is torch.float32, scale, eps,
        res_out.data_ptr(), x, _stream(None, dev))
    if st != FT_OK:
        _check(st, "ft_residual_norm")
    return res_out, x_out


class NormGradients(NamedTuple):
    """What residual_norm_backward returns; None for inputs that were None."""
    dy: torch.Tensor
    dresidual: torch.Tensor
    dw_post: torch.Tensor | None
    dw_pre: torch.Tensor | None
    dgate: torch.Tensor | None


@functools.lru_cache(maxsize=1024)
def _norm_backward_bytes(T, H, dev) -> int:
    n = _LIB.ft_residual_norm_backward_workspace_bytes(T, H)
    if n == 0:
        raise FtError(2, "ft_residual_norm_backward_workspace_bytes")
    return n


def residual_norm_backward(y, residual, d_r, d_x=None, w_post=None, w_pre=None, gate=None,
                           scale=1.0, eps=1e-6, workspace=None, stream=None) -> NormGradients:
    """ft_residual_norm_backward: the gradient of residual_norm for d_r (of r', its type; None: zero)
    and d_x (of x', bf16; required with w_pre): dy bf16, dresidual in the stream's type (the
    residual's, or d_r's without one), dw_post and dw_pre f32 [H], dgate f32 [H] or [T,1], or bf16
    [T,H]."""
    if stream is not None:
        with torch.cuda.stream(stream):   # what the call makes belongs to the stream that it runs on
            return residual_norm_backward(y, residual, d_r, d_x, w_post, w_pre, gate, scale, eps,
                                          workspace)
    dev, T, H, kind, res = _norm_inputs(y, residual, w_post, w_pre, gate)
    if d_r is not None:
        _need(d_r, "d_r", dev, _RES if residual is None else (res,), (T, H))
        res = d_r.dtype
    if w_pre is not None:
        if d_x is None:
            raise ValueError("d_x: required with w_pre")
        _need(d_x, "d_x", dev, BF16_BITS, (T, H))
    f32 = torch.float32
    dy = torch.empty_like(y, dtype=torch.bfloat16)
    dres = torch.empty_like(y, dtype=res)
    dw_post = dw_pre = dgate = None
    post = pre = dx = gp = dg = 0
    if w_post is not None:
        dw_post = torch.empty_like(w_post, dtype=f32)
        post = dw_post.data_ptr()
    if w_pre is not None:
        dw_pre = torch.empty_like(w_pre, dtype=f32)
        pre, dx = dw_pre.data_ptr(), d_x.data_ptr()
    if gate is not None:
        dgate = torch.empty_like(gate, dtype=torch.bfloat16 if kind == GATE_ELEMENT else f32)
        gp, dg = gate.data_ptr(), dgate.data_ptr()
    if workspace is not None:
        _need(workspace, "workspace", dev, None, None)
    elif T > 0:
        workspace = _scratch(_norm_backward_bytes(T, H, dev), dev)
    st = _LIB.ft_residual_norm_backward(
        y.data_ptr(), 0 if residual is None else residual.data_ptr(),
        0 if w_post is None else w_post.data_ptr(), 0 if w_pre is None else w_pre.data_ptr(), gp,
        kind, 0 if d_r is None else d_r.data_ptr(), dx, T, H, res is f32, scale, eps,
        dy.data_ptr(), dres.data_ptr(), post, pre, dg,
        0 if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel(), _stream(None, dev))
    if st != FT_OK:
        _check(st, "ft_residual_norm_backward")
    return NormGradients(dy, dres, dw_post, dw_pre, dgate)


def get_error(workspace=None, stream=None) -> int:
    """ft_moe_get_error: what the calls with this workspace have flagged since the last look, or,
    without one, those that this thread made on the stream (the current one) without a workspace.
    A captured call without a workspace has nowhere to flag: give it one."""
    if workspace is None:
        dev = torch.cuda.current_device() if stream is None else stream.device_index
        workspace = _KEPT.by_stream.get((dev, _stream(stream, dev)))
        if workspace is None:
            return FT_OK
    dev = _device_of(workspace, "ft_moe_get_error")
    return _LIB.ft_moe_get_error(_ptr(workspace), _stream(stream, dev))


def debug_set_wait_limit(iterations: int | None):
    """Test hook: how often a decode kernel polls for the other CTAs' results before it
    flags FT_ERR_TIMEOUT and goes on (None: the default bound)."""
    _check(_LIB.ft_moe_debug_set_wait_limit(-1 if iterations is None else int(iterations)),
           "ft_moe_debug_set_wait_limit")
