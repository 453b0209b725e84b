"""Thin ctypes binding over libjepa.so (the C ABI in include/jepa_cem.h).

Argument marshalling only: every step of the planning path runs in the library's CUDA
kernels. torch is used for device memory and streams. There is no fallback: if the
library is missing or fails to load, ``load()`` raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Dict, Optional

import numpy as np

from . import synthetic

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libjepa.so")
_lib = None

JEPA_OK = 0
STATUS = {0: "ok", 1: "invalid argument", 2: "shape", 3: "not loaded", 4: "out of memory",
          5: "CUDA error", 6: "timeout", 7: "unsupported"}
EXPORTS = ("jepa_create", "jepa_destroy", "jepa_last_error", "jepa_status_string",
           "jepa_weight_blob_bytes", "jepa_load_weights", "jepa_sample_actions", "jepa_philox4x32_10",
           "jepa_predictor_forward", "jepa_cem_select_refit", "jepa_cem_plan",
           "jepa_plan_kernel_count", "jepa_linear_bf16", "jepa_profile_enable",
           "jepa_profile_read", "jepa_sync_check", "jepa_energy_l1_noalloc",
           "jepa_attention_bf16", "jepa_cem_warm_start", "jepa_world_model_step",
           "jepa_cem_closed_loop", "jepa_linear_fp8", "jepa_quantize_rows_fp8",
           "jepa_set_use_graphs", "jepa_selftest_bounded_wait", "jepa_linear_resid_bf16",
           "jepa_linear_qkv_bf16", "jepa_rope_table", "jepa_rope_append_kv8", "jepa_kv8_read",
           "jepa_attention_kv8_workspace", "jepa_attention_kv8", "jepa_attention_packed",
           "jepa_rope_append_kv4", "jepa_kv4_read", "jepa_attention_kv4_workspace", "jepa_attention_kv4",
           "jepa_kv4_evict_workspace", "jepa_kv4_evict", "jepa_add_rmsnorm_fp8")


class JepaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [("layers", ctypes.c_int32), ("width", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("mlp", ctypes.c_int32), ("patch_tokens", ctypes.c_int32),
                ("embed_dim", ctypes.c_int32), ("action_dim", ctypes.c_int32),
                ("state_dim", ctypes.c_int32), ("max_horizon", ctypes.c_int32),
                ("precision", ctypes.c_int32), ("ln_eps", ctypes.c_float),
                ("max_chunk", ctypes.c_int32), ("mlp_kind", ctypes.c_int32)]

MLP_KINDS = {"gelu": 0, "gated": 1}
PRECISIONS = {"fp32": 0, "bf16": 1, "fp8": 2}


class Trace(ctypes.Structure):
    _fields_ = [("mu", ctypes.c_void_p), ("sigma", ctypes.c_void_p), ("actions", ctypes.c_void_p),
                ("energy", ctypes.c_void_p), ("elites", ctypes.c_void_p),
                ("winner", ctypes.c_void_p)]


class Kv8Struct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


class Kv4Struct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("k_unit", ctypes.c_void_p), ("v_unit", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


def load(path: str = _LIB_PATH):
    """Load the library (once) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first (__graft_entry__.build())")
    lib = ctypes.CDLL(path)
    P, I, U64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_float
    I64, D, Z, CACHE = ctypes.c_int64, ctypes.c_double, ctypes.c_size_t, ctypes.POINTER(Kv8Struct)
    CACHE4 = ctypes.POINTER(Kv4Struct)
    sig = {
        "jepa_create": ([ctypes.POINTER(Config), I, ctypes.POINTER(P)], I),
        "jepa_destroy": ([P], None),
        "jepa_last_error": ([P], ctypes.c_char_p),
        "jepa_status_string": ([I], ctypes.c_char_p),
        "jepa_weight_blob_bytes": ([ctypes.POINTER(Config)], ctypes.c_size_t),
        "jepa_load_weights": ([P, P, ctypes.c_size_t], I),
        "jepa_sample_actions": ([P, P, P, I, I, I, I, U64, P, P], I),
        "jepa_philox4x32_10": ([P, P, U64, I, P, P], I),
        "jepa_predictor_forward": ([P, P, P, P, I, I, I, P, P, P, P], I),
        "jepa_cem_select_refit": ([P, P, P, I, I, I, I, P, P, P, P], I),
        "jepa_cem_plan": ([P, P, P, P, P, P, I, I, I, I, I, U64, P, ctypes.POINTER(Trace), P], I),
        "jepa_plan_kernel_count": ([P, I, I, I, I, I, ctypes.POINTER(ctypes.c_int64)], I),
        "jepa_linear_bf16": ([P, P, P, P, I, I, I, I, P, P], I),
        "jepa_linear_resid_bf16": ([P, P, P, P, I, I, I, P, P], I),
        "jepa_linear_qkv_bf16": ([P, P, P, P, I, I, I, I, I, I, P, P, P], I),
        "jepa_profile_enable": ([P, I], I),
        "jepa_profile_read": ([P, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double),
                               ctypes.POINTER(ctypes.c_int64)], I),
        "jepa_sync_check": ([P, P], I),
        "jepa_attention_bf16": ([P, P, P, P, I, I, I, I, I, I, P], I),
        "jepa_energy_l1_noalloc": ([P, P, I, I, I, I, P, P, ctypes.c_char_p, ctypes.c_size_t], I),
        "jepa_cem_warm_start": ([P, P, P, P, I, I, P, P, P], I),
        "jepa_world_model_step": ([P, P, P, P, I, P, P, P, P, P], I),
        "jepa_cem_closed_loop": ([P, P, P, P, P, P, I, I, I, I, I, I, I, U64, P, P, P], I),
        "jepa_linear_fp8": ([P, P, P, P, P, P, I, I, I, I, P, P], I),
        "jepa_quantize_rows_fp8": ([P, P, I, I, P, P, P], I),
        "jepa_rope_table": ([P, I, I, D, D, P, P], I),
        "jepa_rope_append_kv8": ([P, CACHE, P, I64, P, I64, P, I64, I, I, P, P, F, P, I, I, I, P, P,
                                  P, P, P], I),
        "jepa_kv8_read": ([P, CACHE, P, P, I, P, P, P], I),
        "jepa_attention_kv8_workspace": ([P, CACHE, ctypes.POINTER(Z)], I),
        "jepa_attention_kv8": ([P, CACHE, P, I, I, P, F, I, P, P, P, Z, P], I),
        "jepa_attention_packed": ([P, P, I64, P, I64, P, I64, I, I, I, I, I, I, P, P, F, I, P, P, P],
                                  I),
        "jepa_rope_append_kv4": ([P, CACHE4, P, I64, P, I64, P, I64, I, I, P, P, F, P, I, I, I, P, P,
                                  P, P, P, P], I),
        "jepa_kv4_read": ([P, CACHE4, P, P, I, P, P, P], I),
        "jepa_attention_kv4_workspace": ([P, CACHE4, ctypes.POINTER(Z)], I),
        "jepa_attention_kv4": ([P, CACHE4, P, I, I, P, F, I, P, P, P, P, F, P, Z, P], I),
        "jepa_kv4_evict_workspace": ([P, CACHE4, I, ctypes.POINTER(Z)], I),
        "jepa_kv4_evict": ([P, CACHE4, P, P, I, I, CACHE4, P, P, P, Z, P], I),
        "jepa_add_rmsnorm_fp8": ([P, P, I, I64, P, I, I64, P, F, I, I, P, I64, P, P, P, P], I),
        "jepa_set_use_graphs": ([P, I], I),
        "jepa_selftest_bounded_wait": ([P, P], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def make_config(pc: synthetic.PredictorConfig, max_horizon: int = 1, max_chunk: int = 0) -> Config:
    return Config(pc.layers, pc.width, pc.heads, pc.mlp, pc.patch_tokens, pc.embed_dim,
                  pc.action_dim, pc.state_dim, max_horizon, PRECISIONS[pc.precision],
                  pc.ln_eps, max_chunk, MLP_KINDS[pc.mlp_kind])


def pack_weights(pc: synthetic.PredictorConfig, weights: Dict[str, np.ndarray]) -> bytes:
    """Weight blob: 64-byte header + fp32 tensors in canonical order (format only)."""
    hdr = struct.pack("<11i", 0x4150454A, 1, pc.layers, pc.width, pc.heads, pc.mlp,
                      pc.patch_tokens, pc.embed_dim, pc.action_dim, pc.state_dim,
                      MLP_KINDS[pc.mlp_kind]).ljust(64, b"\0")
    shapes = synthetic.weight_shapes(pc)
    parts = [hdr]
    for name in synthetic.weight_names(pc):
        w = np.ascontiguousarray(weights[name], dtype=np.float32)
        assert w.shape == shapes[name], (name, w.shape)
        parts.append(w.tobytes())
    return b"".join(parts)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_DTYPES = {"f32": ("float32",), "bf16": ("bfloat16", "int16", "uint16"), "u8": ("uint8", "float8_e4m3fn"),
           "i32": ("int32",), "u32": ("int32", "uint32")}


def _arg(t, name: str, kind: str, numel: int, host_ok: bool = False,
         optional: bool = False) -> Optional[int]:
    """Address of argument `t` after checking that it can hold `numel` elements of `kind`.

    A torch tensor must have that element type, be contiguous, hold at least `numel`
    elements and live on a CUDA device (or, where `host_ok`, in host memory); anything else
    raises JepaError(INVALID_ARG) before the library is called, so that no kernel reads or
    writes past a caller's buffer. A raw integer address is passed through unchecked: the
    caller vouches for its size and location. None is allowed only for optional arguments."""
    if t is None:
        if optional:
            return None
        raise JepaError(1, f"{name} is required")
    if isinstance(t, int):
        return t
    import torch
    if not isinstance(t, torch.Tensor):
        raise JepaError(1, f"{name}: expected a torch tensor or an integer address, got {type(t).__name__}")
    if str(t.dtype).replace("torch.", "") not in _DTYPES[kind]:
        raise JepaError(1, f"{name}: dtype {t.dtype} where {kind} is required")
    if not t.is_contiguous():
        raise JepaError(1, f"{name} must be contiguous")
    if not t.is_cuda and not host_ok:
        raise JepaError(1, f"{name} must be a CUDA tensor")
    if t.numel() < numel:
        raise JepaError(1, f"{name} holds {t.numel()} elements, {numel} are needed")
    return t.data_ptr()


class _Fast:
    """What the single-token entry points look up on every call, fetched once: a serving step
    makes a few such calls a layer, and its kernels take microseconds."""

    torch = None

    @classmethod
    def load(cls):
        import torch
        cls.u8 = frozenset(d for d in (torch.uint8, getattr(torch, "float8_e4m3fn", None)) if d)
        cls.bf16 = frozenset((torch.bfloat16, torch.int16, torch.uint16))
        cls.f32, cls.i32 = frozenset((torch.float32,)), frozenset((torch.int32,))
        cls.matrices = {torch.float32: 0, torch.bfloat16: 1}
        cls.kinds = {"u8": cls.u8, "bf16": cls.bf16, "f32": cls.f32, "i32": cls.i32}
        # the stream's address without a Stream object around it, where torch has that
        cls.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        cls.Tensor = torch.Tensor
        cls.torch = torch


def _dev(t, name: str, kind: str, numel: int, device: int) -> int:
    """Address of the device tensor `t`, checked as in _arg and for its device."""
    if (isinstance(t, _Fast.Tensor) and t.dtype in _Fast.kinds[kind] and t.get_device() == device
            and t.is_contiguous() and t.numel() >= numel):
        return t.data_ptr()
    at = _arg(t, name, kind, numel)
    if isinstance(t, _Fast.Tensor):
        raise JepaError(1, f"{name} is on {t.device}, the planner on cuda:{device}")
    return at


def _opt(t, name: str, kind: str, numel: int, device: int) -> Optional[int]:
    return None if t is None else _dev(t, name, kind, numel, device)


def _sized(t, name: str):
    """`t` itself, once it is a tensor: for arguments whose size the call goes by, where an address
    says too little."""
    if _Fast.torch is None:
        _Fast.load()
    if not isinstance(t, _Fast.Tensor):
        raise JepaError(1, f"{name}: expected a torch tensor, got {type(t).__name__}")
    return t


def _int32(n, name: str) -> int:
    """`n` itself, which the library takes as 32 bits (ctypes would cut off what is above them)."""
    if not -2 ** 31 <= n < 2 ** 31:
        raise JepaError(1, f"{name} out of range ({n})")
    return n


def _rows(t, name: str, device: Optional[int] = None):
    """(address, elements between tokens, tokens, heads, head_dim) of token rows [tokens, heads,
    head_dim]: a bf16 CUDA tensor whose heads lie back to back (a slice of a wider projection's
    rows is fine)."""
    if _Fast.torch is None:
        _Fast.load()
    if not isinstance(t, _Fast.Tensor) or t.dim() != 3:
        raise JepaError(1, f"{name}: expected a tensor [tokens, heads, head_dim]")
    if t.dtype not in _Fast.bf16:
        raise JepaError(1, f"{name}: dtype {t.dtype} where bf16 is required")
    n, heads, dim = t.shape
    st = t.stride()
    if (dim > 1 and st[2] != 1) or (heads > 1 and st[1] != dim):
        raise JepaError(1, f"{name}: the heads of a token must be contiguous")
    at = t.get_device()                  # -1: host memory
    if at < 0:
        raise JepaError(1, f"{name} must be a CUDA tensor")
    if device is not None and at != device:
        raise JepaError(1, f"{name} is on {t.device}, the planner on cuda:{device}")
    return t.data_ptr(), (st[0] if n > 1 else heads * dim), n, heads, dim


class KvCache8:
    """One layer's 8-bit paged key/value cache (jepa_kv8_cache of the C header) over tensors that
    the caller owns; the handle keeps them alive and checks them once.

    k, v: uint8 or float8_e4m3fn [num_pages, kv_heads, page_size, head_dim]; k_scale, v_scale:
    float32 [num_pages, kv_heads]; page_table: int32 [batch, max_pages]."""

    def __init__(self, k, v, k_scale, v_scale, page_table):
        for name, t in (("k", k), ("v", v), ("k_scale", k_scale), ("v_scale", v_scale),
                        ("page_table", page_table)):
            _sized(t, "KvCache8: " + name)
        if k.dim() != 4 or page_table.dim() != 2:
            raise JepaError(1, "KvCache8: k must be [num_pages, kv_heads, page_size, head_dim] and "
                               "page_table [batch, max_pages]")
        pages, heads, page, dim = k.shape
        if tuple(v.shape) != tuple(k.shape):
            raise JepaError(1, f"KvCache8: v has shape {tuple(v.shape)}, k {tuple(k.shape)}")
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if tuple(s.shape) != (pages, heads):
                raise JepaError(1, f"KvCache8: {name} must be [{pages}, {heads}]")
        if dim not in (64, 128) or page not in (16, 32, 64, 128):
            raise JepaError(2, "KvCache8: head_dim must be 64 or 128, page_size 16, 32, 64 or 128")
        self.tensors = (k, v, k_scale, v_scale, page_table)
        if len({t.device for t in self.tensors}) != 1:
            raise JepaError(1, "KvCache8: all tensors must be on one device")
        n = pages * heads
        batch, max_pages = page_table.shape
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page, dim
        self.batch, self.max_pages, self.device = batch, max_pages, k.device
        self.struct = Kv8Struct(
            _arg(k, "k", "u8", n * page * dim), _arg(v, "v", "u8", n * page * dim),
            _arg(k_scale, "k_scale", "f32", n), _arg(v_scale, "v_scale", "f32", n),
            _arg(page_table, "page_table", "i32", batch * max_pages), pages, page, heads, dim, batch,
            max_pages)
        self.ref = ctypes.byref(self.struct)
        self.index = k.get_device()

    def check(self, device: int):
        """Raises unless the cache lives on this device."""
        if self.index != device:
            raise JepaError(1, f"cache is on {self.device}, the planner on cuda:{device}")


class KvCache4:
    """One layer's 4-bit paged key/value cache (jepa_kv4_cache of the C header) over tensors that
    the caller owns; the handle keeps them alive and checks them once.

    k, v: uint8 [num_pages, kv_heads, page_size, head_dim / 2]; k_scale, v_scale: uint8 or
    float8_e4m3fn [num_pages, kv_heads, page_size, head_dim / 16]; page_table: int32 [batch,
    max_pages]; k_unit, v_unit: float32 [kv_heads], powers of two, or None (1)."""

    def __init__(self, k, v, k_scale, v_scale, page_table, k_unit=None, v_unit=None):
        for name, t in (("k", k), ("v", v), ("k_scale", k_scale), ("v_scale", v_scale),
                        ("page_table", page_table)):
            _sized(t, "KvCache4: " + name)
        if k.dim() != 4 or page_table.dim() != 2:
            raise JepaError(1, "KvCache4: k must be [num_pages, kv_heads, page_size, head_dim / 2] and "
                               "page_table [batch, max_pages]")
        pages, heads, page, half = k.shape
        dim = 2 * half
        if dim not in (64, 128) or page not in (16, 32, 64, 128):
            raise JepaError(2, "KvCache4: head_dim must be 64 or 128, page_size 16, 32, 64 or 128")
        if tuple(v.shape) != tuple(k.shape):
            raise JepaError(1, f"KvCache4: v has shape {tuple(v.shape)}, k {tuple(k.shape)}")
        for name, s in (("k_scale", k_scale), ("v_scale", v_scale)):
            if tuple(s.shape) != (pages, heads, page, dim // 16):
                raise JepaError(1, f"KvCache4: {name} must be [{pages}, {heads}, {page}, {dim // 16}]")
        for name, u in (("k_unit", k_unit), ("v_unit", v_unit)):
            if u is not None and tuple(_sized(u, "KvCache4: " + name).shape) != (heads,):
                raise JepaError(1, f"KvCache4: {name} must be [{heads}]")
        self.tensors = tuple(t for t in (k, v, k_scale, v_scale, page_table, k_unit, v_unit) if t is not None)
        if len({t.device for t in self.tensors}) != 1:
            raise JepaError(1, "KvCache4: all tensors must be on one device")
        n = pages * heads * page
        batch, max_pages = page_table.shape
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page, dim
        self.batch, self.max_pages, self.device = batch, max_pages, k.device
        self.struct = Kv4Struct(
            _arg(k, "k", "u8", n * half), _arg(v, "v", "u8", n * half),
            _arg(k_scale, "k_scale", "u8", n * dim // 16), _arg(v_scale, "v_scale", "u8", n * dim // 16),
            _arg(k_unit, "k_unit", "f32", heads, optional=True),
            _arg(v_unit, "v_unit", "f32", heads, optional=True),
            _arg(page_table, "page_table", "i32", batch * max_pages), pages, page, heads, dim, batch,
            max_pages)
        self.ref = ctypes.byref(self.struct)
        self.index = k.get_device()

    def check(self, device: int):
        """Raises unless the cache lives on this device."""
        if self.index != device:
            raise JepaError(1, f"cache is on {self.device}, the planner on cuda:{device}")


def _matrix(t, name: str, device: int, shape=None):
    """(address, 1 where bf16, elements between rows) of a float32 or bf16 CUDA tensor [rows, cols]
    (of this shape, where one is given) whose rows are contiguous (columns of a wider tensor are fine)."""
    if not isinstance(t, _Fast.Tensor) or t.dim() != 2:
        raise JepaError(1, f"{name}: expected a tensor [rows, cols]")
    if shape is not None and t.shape != shape:
        raise JepaError(1, f"{name} {tuple(t.shape)} does not fit x {tuple(shape)}")
    half = _Fast.matrices.get(t.dtype)
    if half is None:
        raise JepaError(1, f"{name}: dtype {t.dtype} where float32 or bfloat16 is required")
    if t.is_contiguous():
        stride = t.shape[1] if shape is None else shape[1]
    else:
        rows, cols = t.shape
        if cols > 1 and t.stride(1) != 1:
            raise JepaError(1, f"{name}: the elements of a row must be contiguous")
        stride = t.stride(0) if rows > 1 else cols
    if t.get_device() != device:
        raise JepaError(1, f"{name} is on {t.device}, the planner on cuda:{device}")
    return t.data_ptr(), half, stride


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def energy_l1_noalloc(z_pred, goal, B, N, P, E, energy, stream=None):
    """L1 energy of predicted frames without any device allocation (see the C header).

    For callers that cannot allocate device memory (a fixed memory budget owned by a host
    framework, or a control loop that must not allocate mid-episode). Raises JepaError with
    the library's message on failure, e.g. when B*N*ceil(P/32) exceeds the fixed scratch."""
    lib = load()
    if min(B, N, P, E) < 1:
        raise JepaError(1, "energy_l1_noalloc: B, N, P and E must be positive")
    zp = _arg(z_pred, "z_pred", "f32", B * N * P * E)
    gp = _arg(goal, "goal", "f32", B * P * E)
    ep = _arg(energy, "energy", "f32", B * N)
    buf = ctypes.create_string_buffer(256)
    st = lib.jepa_energy_l1_noalloc(zp, gp, B, N, P, E, ep, _stream(stream), buf, len(buf))
    if st != JEPA_OK:
        raise JepaError(st, buf.value.decode())


def _stream_on(stream, device: int) -> int:
    """The given stream, or the device's current one."""
    if stream is None:
        if _Fast.raw_stream is not None:
            return _Fast.raw_stream(device)
        return _Fast.torch.cuda.current_stream(device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _refuse(cache, other, what: str):
    """Refuses a cache of the other width, whose handle the library would not take."""
    if type(cache) is other:
        raise JepaError(1, f"{what}: got a {other.__name__}")


def _append_method(name: str):
    """Planner's append to one of the paged caches (jepa_<name> of the C header)."""
    eight = name.endswith("8")
    call, other = "jepa_" + name, KvCache4 if eight else KvCache8

    def append(self, q, k, v, rope_table, cu, start, cache, q_out, q_norm=None, k_norm=None,
               norm_eps=1e-6, interleaved=False, k_out=None, stream=None, rope_start=None):
        """Norm, rotate and append packed tokens: q [tokens, q_heads, head_dim] (or None with
        q_out None), k and v [tokens, kv_heads, head_dim]; rope_table [positions, rot] or None;
        rope_start [batch] (4-bit cache only): positions for the rotation where they are not start."""
        _refuse(cache, other, name)
        dev = self.device
        kp, ks, tokens, heads, dim = _rows(k, "k", dev)
        vp, vs, *v_shape = _rows(v, "v", dev)
        if v_shape != [tokens, heads, dim] or heads != cache.kv_heads or dim != cache.head_dim:
            raise JepaError(1, f"k {tuple(k.shape)} and v {tuple(v.shape)} do not fit the cache's "
                               f"{cache.kv_heads} heads of {cache.head_dim}")
        if (q is None) != (q_out is None):
            raise JepaError(1, "q and q_out are given together")
        qp, qs, q_heads, qo = None, 0, 0, None
        if q is not None:
            qp, qs, q_tokens, q_heads, q_dim = _rows(q, "q", dev)
            if q_tokens != tokens or q_dim != dim:
                raise JepaError(1, f"q {tuple(q.shape)} does not fit k {tuple(k.shape)}")
            qo = _dev(q_out, "q_out", "bf16", tokens * q_heads * dim, dev)
        positions = rot = 0
        if rope_table is not None:
            if _sized(rope_table, "rope_table").dim() != 2:
                raise JepaError(1, "rope_table must be [positions, rot]")
            positions, rot = rope_table.shape
        cache.check(dev)
        if tokens < 1:
            raise JepaError(1, "tokens must be >= 1 (got 0)")
        apart = ()
        if not eight:
            apart = (_opt(rope_start, "rope_start", "i32", cache.batch, dev),)
        elif rope_start is not None:
            raise JepaError(1, f"{name} takes no rope_start")
        st = getattr(self.lib, call)(
            self.h, cache.ref, qp, qs, kp, ks, vp, vs, tokens, q_heads,
            _opt(q_norm, "q_norm", "f32", dim, dev), _opt(k_norm, "k_norm", "f32", dim, dev), norm_eps,
            _opt(rope_table, "rope_table", "f32", positions * rot, dev), positions, rot,
            int(interleaved), _dev(cu, "cu", "i32", cache.batch + 1, dev),
            _dev(start, "start", "i32", cache.batch, dev), *apart, qo,
            _opt(k_out, "k_out", "bf16", tokens * heads * dim, dev), _stream_on(stream, dev))
        if st:
            self._check(st, name)

    append.__name__ = name
    append.__qualname__ = "Planner." + name
    return append


def _read_method(name: str):
    """Planner's read-back of one of the paged caches."""
    call, other = "jepa_" + name, KvCache4 if name.startswith("kv8") else KvCache8

    def read(self, cache, cu, first, k_out, v_out, stream=None):
        """Cached tokens as bf16 into k_out, v_out [tokens, kv_heads, head_dim]."""
        _refuse(cache, other, name)
        dev = self.device
        cache.check(dev)
        tokens = k_out.shape[0] if _sized(k_out, "k_out").dim() else 0
        if tokens < 1:
            raise JepaError(1, "tokens must be >= 1 (got 0)")
        n = tokens * cache.kv_heads * cache.head_dim
        st = getattr(self.lib, call)(
            self.h, cache.ref, _dev(cu, "cu", "i32", cache.batch + 1, dev),
            _dev(first, "first", "i32", cache.batch, dev), tokens, _dev(k_out, "k_out", "bf16", n, dev),
            _dev(v_out, "v_out", "bf16", n, dev), _stream_on(stream, dev))
        if st:
            self._check(st, name)

    read.__name__ = name
    read.__qualname__ = "Planner." + name
    return read


class Planner:
    """One library context (weights + workspaces + captured graphs) on one device."""

    def __init__(self, pc: synthetic.PredictorConfig, max_horizon: int = 1, device: int = 0,
                 max_chunk: int = 0):
        self.lib = load()
        self.pc = pc
        self.device = device
        self.cfg = make_config(pc, max_horizon, max_chunk)
        h = ctypes.c_void_p()
        st = self.lib.jepa_create(ctypes.byref(self.cfg), device, ctypes.byref(h))
        if st != JEPA_OK:
            raise JepaError(st, "jepa_create")
        self.h = h

    def _check(self, st: int, what: str):
        if st != JEPA_OK:
            raise JepaError(st, f"{what}: {self.lib.jepa_last_error(self.h).decode()}")

    def close(self):
        if getattr(self, "h", None):
            self.lib.jepa_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def blob_bytes(self) -> int:
        return self.lib.jepa_weight_blob_bytes(ctypes.byref(self.cfg))

    def load_weights(self, weights: Dict[str, np.ndarray]):
        blob = pack_weights(self.pc, weights)
        buf = ctypes.create_string_buffer(blob, len(blob))
        self._check(self.lib.jepa_load_weights(self.h, buf, len(blob)), "load_weights")

    def load_blob(self, blob: bytes):
        buf = ctypes.create_string_buffer(blob, len(blob))
        return self.lib.jepa_load_weights(self.h, buf, len(blob))

    def _dims(self, **sizes):
        for k, v in sizes.items():
            if int(v) < 1:
                raise JepaError(1, f"{k} must be >= 1 (got {v})")

    def sample_actions(self, mu, sigma, B, N, H, rnd, seed, actions, stream=None):
        self._dims(B=B, N=N, H=H)
        A = self.pc.action_dim
        self._check(self.lib.jepa_sample_actions(
            self.h, _arg(mu, "mu", "f32", B * H * A), _arg(sigma, "sigma", "f32", B * H * A), B, N,
            H, rnd, seed, _arg(actions, "actions", "f32", B * N * H * A), _stream(stream)),
            "sample_actions")

    def philox(self, counters, seed, n, out, stream=None):
        self._dims(n=n)
        self._check(self.lib.jepa_philox4x32_10(self.h, _arg(counters, "counters", "u32", 4 * n),
                                                seed, n, _arg(out, "out", "u32", 4 * n),
                                                _stream(stream)), "philox4x32_10")

    def predictor_forward(self, z_ctx, state0, actions, B, N, H, goal=None, z_pred=None,
                          energy=None, stream=None):
        self._dims(B=B, N=N, H=H)
        pc, PE = self.pc, self.pc.patch_tokens * self.pc.embed_dim
        self._check(self.lib.jepa_predictor_forward(
            self.h, _arg(z_ctx, "z_ctx", "f32", B * PE), _arg(state0, "state0", "f32", B * pc.state_dim),
            _arg(actions, "actions", "f32", B * N * H * pc.action_dim), B, N, H,
            _arg(goal, "goal", "f32", B * PE, optional=True),
            _arg(z_pred, "z_pred", "f32", B * N * PE, optional=True),
            _arg(energy, "energy", "f32", B * N, optional=True), _stream(stream)), "predictor_forward")

    def select_refit(self, energy, actions, B, N, H, K, mu_out, sigma_out, elites_out=None,
                     stream=None):
        self._dims(B=B, N=N, H=H, K=K)
        HA = H * self.pc.action_dim
        self._check(self.lib.jepa_cem_select_refit(
            self.h, _arg(energy, "energy", "f32", B * N), _arg(actions, "actions", "f32", B * N * HA),
            B, N, H, K, _arg(mu_out, "mu_out", "f32", B * HA), _arg(sigma_out, "sigma_out", "f32", B * HA),
            _arg(elites_out, "elites_out", "i32", B * K, optional=True), _stream(stream)),
            "select_refit")

    def plan(self, z0, state0, goal, mu0, sigma0, B, H, N, K, rounds, seed, action_out,
             trace: Optional[Dict[str, object]] = None, stream=None):
        """Inputs and action_out may be torch tensors (CUDA or host) or raw host/device
        addresses (int); the trace's buffers are CUDA tensors or device addresses."""
        self._dims(B=B, H=H, N=N, K=K, rounds=rounds)
        pc = self.pc
        PE, HA, R = pc.patch_tokens * pc.embed_dim, H * pc.action_dim, rounds
        tr = None
        if trace is not None:
            sizes = {"mu": ("f32", (R + 1) * B * HA), "sigma": ("f32", (R + 1) * B * HA),
                     "actions": ("f32", R * B * N * HA), "energy": ("f32", R * B * N),
                     "elites": ("i32", R * B * K), "winner": ("i32", B)}
            tr = Trace(*(_arg(trace.get(k), f"trace[{k}]", sizes[k][0], sizes[k][1], optional=True)
                         for k in ("mu", "sigma", "actions", "energy", "elites", "winner")))
        self._check(self.lib.jepa_cem_plan(
            self.h, _arg(z0, "z0", "f32", B * PE, host_ok=True),
            _arg(state0, "state0", "f32", B * pc.state_dim, host_ok=True),
            _arg(goal, "goal", "f32", B * PE, host_ok=True),
            _arg(mu0, "mu0", "f32", B * HA, host_ok=True),
            _arg(sigma0, "sigma0", "f32", B * HA, host_ok=True), B, H, N, K, rounds, seed,
            _arg(action_out, "action_out", "f32", B * pc.action_dim, host_ok=True),
            ctypes.byref(tr) if tr is not None else None, _stream(stream)), "cem_plan")

    def warm_start(self, mu_prev, mu_prior, sigma_prior, B, H, mu_out, sigma_out, stream=None):
        self._dims(B=B, H=H)
        n = B * H * self.pc.action_dim
        self._check(self.lib.jepa_cem_warm_start(
            self.h, _arg(mu_prev, "mu_prev", "f32", n), _arg(mu_prior, "mu_prior", "f32", n),
            _arg(sigma_prior, "sigma_prior", "f32", n), B, H, _arg(mu_out, "mu_out", "f32", n),
            _arg(sigma_out, "sigma_out", "f32", n), _stream(stream)), "cem_warm_start")

    def world_model_step(self, z, state, action, B, z_next, state_next, goal=None, distance=None,
                         stream=None):
        self._dims(B=B)
        pc, PE = self.pc, self.pc.patch_tokens * self.pc.embed_dim
        self._check(self.lib.jepa_world_model_step(
            self.h, _arg(z, "z", "f32", B * PE), _arg(state, "state", "f32", B * pc.state_dim),
            _arg(action, "action", "f32", B * pc.action_dim), B,
            _arg(goal, "goal", "f32", B * PE, optional=True), _arg(z_next, "z_next", "f32", B * PE),
            _arg(state_next, "state_next", "f32", B * pc.state_dim),
            _arg(distance, "distance", "f32", B, optional=True), _stream(stream)), "world_model_step")

    def closed_loop(self, z0, state0, goal, mu_prior, sigma_prior, B, H, N, K, rounds, steps,
                    warm, seed, actions_out, distance_out, stream=None):
        self._dims(B=B, H=H, N=N, K=K, rounds=rounds, steps=steps)
        pc = self.pc
        PE, HA = pc.patch_tokens * pc.embed_dim, H * pc.action_dim
        self._check(self.lib.jepa_cem_closed_loop(
            self.h, _arg(z0, "z0", "f32", B * PE, host_ok=True),
            _arg(state0, "state0", "f32", B * pc.state_dim, host_ok=True),
            _arg(goal, "goal", "f32", B * PE, host_ok=True),
            _arg(mu_prior, "mu_prior", "f32", B * HA, host_ok=True),
            _arg(sigma_prior, "sigma_prior", "f32", B * HA, host_ok=True), B, H, N, K, rounds, steps,
            int(warm), seed, _arg(actions_out, "actions_out", "f32", steps * B * pc.action_dim,
                                  host_ok=True),
            _arg(distance_out, "distance_out", "f32", steps * B, host_ok=True), _stream(stream)),
            "cem_closed_loop")

    def kernel_count(self, B, H, N, K, rounds) -> int:
        c = ctypes.c_int64()
        self._check(self.lib.jepa_plan_kernel_count(self.h, B, H, N, K, rounds, ctypes.byref(c)),
                    "plan_kernel_count")
        return c.value

    def linear_bf16(self, A, W, bias, M, N, K, gelu, out, stream=None):
        self._dims(M=M, N=N, K=K)
        n_out = N // 2 if int(gelu) == 2 else N
        self._check(self.lib.jepa_linear_bf16(
            self.h, _arg(A, "A", "bf16", M * K), _arg(W, "W", "bf16", N * K),
            _arg(bias, "bias", "f32", N, optional=True), M, N, K, int(gelu),
            _arg(out, "out", "f32", M * n_out), _stream(stream)), "linear_bf16")

    def linear_resid_bf16(self, A, W, bias, M, N, K, x, stream=None):
        self._dims(M=M, N=N, K=K)
        self._check(self.lib.jepa_linear_resid_bf16(
            self.h, _arg(A, "A", "bf16", M * K), _arg(W, "W", "bf16", N * K),
            _arg(bias, "bias", "f32", N, optional=True), M, N, K,
            _arg(x, "x", "f32", M * N), _stream(stream)), "linear_resid_bf16")

    def linear_qkv_bf16(self, A, W, bias, M, d, K, T, kv_rows, frame, q, kv, stream=None):
        self._dims(M=M, d=d, K=K, T=T, kv_rows=kv_rows)
        ncand = -(-int(M) // int(T))
        self._check(self.lib.jepa_linear_qkv_bf16(
            self.h, _arg(A, "A", "bf16", M * K), _arg(W, "W", "bf16", 3 * d * K),
            _arg(bias, "bias", "f32", 3 * d, optional=True), M, d, K, T, kv_rows, int(frame),
            _arg(q, "q", "bf16", M * d), _arg(kv, "kv", "bf16", ncand * kv_rows * 2 * d),
            _stream(stream)), "linear_qkv_bf16")

    def linear_fp8(self, A, a_scale, W, w_scale, bias, M, N, K, gelu, out, stream=None):
        self._dims(M=M, N=N, K=K)
        n_out = N // 2 if int(gelu) == 2 else N
        self._check(self.lib.jepa_linear_fp8(
            self.h, _arg(A, "A", "u8", M * K), _arg(a_scale, "a_scale", "f32", M),
            _arg(W, "W", "u8", N * K), _arg(w_scale, "w_scale", "f32", N),
            _arg(bias, "bias", "f32", N, optional=True), M, N, K, int(gelu),
            _arg(out, "out", "f32", M * n_out), _stream(stream)), "linear_fp8")

    def quantize_rows_fp8(self, x, rows, cols, codes, scales, stream=None):
        self._dims(rows=rows, cols=cols)
        self._check(self.lib.jepa_quantize_rows_fp8(
            self.h, _arg(x, "x", "f32", rows * cols), rows, cols,
            _arg(codes, "codes", "u8", rows * cols), _arg(scales, "scales", "f32", rows),
            _stream(stream)), "quantize_rows_fp8")

    def attention_bf16(self, q, kv, out, ncand, T, Lk, kv_rows, heads, d, stream=None):
        self._dims(ncand=ncand, T=T, Lk=Lk, kv_rows=kv_rows, heads=heads, d=d)
        self._check(self.lib.jepa_attention_bf16(
            self.h, _arg(q, "q", "bf16", ncand * T * d), _arg(kv, "kv", "bf16", ncand * kv_rows * 2 * d),
            _arg(out, "out", "bf16", ncand * T * d), ncand, T, Lk, kv_rows, heads, d,
            _stream(stream)), "attention_bf16")

    # ---- 8-bit paged key/value cache and the attention around it (see the C header) ----

    def rope_table(self, positions, rot, base=10000.0, factor=1.0, table=None, stream=None):
        """cos / sin table [positions, rot] for rope_append_kv8 (allocated when not given)."""
        self._dims(positions=positions, rot=rot)
        if _Fast.torch is None:
            _Fast.load()
        if table is None:
            table = _Fast.torch.empty(positions, rot, device=f"cuda:{self.device}")
        self._check(self.lib.jepa_rope_table(
            self.h, positions, rot, base, factor,
            _dev(table, "table", "f32", positions * rot, self.device),
            _stream_on(stream, self.device)), "rope_table")
        return table

    rope_append_kv8 = _append_method("rope_append_kv8")
    kv8_read = _read_method("kv8_read")

    def attention_kv8_workspace(self, cache: KvCache8) -> int:
        """Bytes of workspace that attention_kv8 needs."""
        n = ctypes.c_size_t()
        self._check(self.lib.jepa_attention_kv8_workspace(self.h, cache.ref, ctypes.byref(n)),
                    "attention_kv8_workspace")
        return n.value

    def attention_kv8(self, q, cache: KvCache8, kv_len, out, scale, workspace, causal=True, lse=None,
                      stream=None):
        """Attention of q [batch, q_tokens, q_heads, head_dim] over the cache; workspace: a uint8
        tensor of attention_kv8_workspace bytes, one for each call that may run at a time."""
        dev = self.device
        if getattr(q, "ndim", 0) != 4 or q.shape[0] != cache.batch or q.shape[3] != cache.head_dim:
            raise JepaError(1, f"q must be [{cache.batch}, q_tokens, q_heads, {cache.head_dim}]")
        cache.check(dev)
        batch, q_tokens, q_heads, dim = q.shape
        rows = batch * q_tokens * q_heads
        if rows < 1:
            raise JepaError(1, "q_tokens and q_heads must be >= 1")
        st = self.lib.jepa_attention_kv8(
            self.h, cache.ref, _dev(q, "q", "bf16", rows * dim, dev), q_tokens, q_heads,
            _dev(kv_len, "kv_len", "i32", batch, dev), scale, int(causal),
            _dev(out, "out", "bf16", rows * dim, dev), _opt(lse, "lse", "f32", rows, dev),
            _dev(_sized(workspace, "workspace"), "workspace", "u8", 0, dev), workspace.numel(),
            _stream_on(stream, dev))
        if st:
            self._check(st, "attention_kv8")

    def attention_packed(self, q, k, v, cu_q, cu_k, out, scale, frame=1, lse=None, stream=None):
        """Attention of packed prompts: q [tokens_q, q_heads, head_dim], k and v [tokens_k,
        kv_heads, head_dim]; cu_q, cu_k [batch + 1]."""
        dev = self.device
        qp, qs, tokens_q, q_heads, dim = _rows(q, "q", dev)
        kp, ks, tokens_k, kv_heads, k_dim = _rows(k, "k", dev)
        vp, vs, *v_shape = _rows(v, "v", dev)
        if v_shape != [tokens_k, kv_heads, k_dim] or k_dim != dim:
            raise JepaError(1, f"q {tuple(q.shape)}, k {tuple(k.shape)} and v {tuple(v.shape)} do not fit")
        batch = _sized(cu_q, "cu_q").numel() - 1
        if min(tokens_q, tokens_k, batch) < 1:
            raise JepaError(1, "tokens_q, tokens_k and batch must be >= 1")
        st = self.lib.jepa_attention_packed(
            self.h, qp, qs, kp, ks, vp, vs, tokens_q, tokens_k, batch, q_heads, kv_heads, dim,
            _dev(cu_q, "cu_q", "i32", batch + 1, dev), _dev(cu_k, "cu_k", "i32", batch + 1, dev), scale,
            frame, _dev(out, "out", "bf16", tokens_q * q_heads * dim, dev),
            _opt(lse, "lse", "f32", tokens_q * q_heads, dev), _stream_on(stream, dev))
        if st:
            self._check(st, "attention_packed")

    # ---- 4-bit paged key/value cache, eviction, and the norm ahead of 8-bit products ----

    rope_append_kv4 = _append_method("rope_append_kv4")
    kv4_read = _read_method("kv4_read")

    def attention_kv4_workspace(self, cache: KvCache4) -> int:
        """Bytes of workspace that attention_kv4 needs."""
        n = ctypes.c_size_t()
        self._check(self.lib.jepa_attention_kv4_workspace(self.h, cache.ref, ctypes.byref(n)),
                    "attention_kv4_workspace")
        return n.value

    def attention_kv4(self, q, cache: KvCache4, kv_len, out, scale, workspace, causal=True, lse=None,
                      mass=None, mass_out=None, decay=1.0, stream=None):
        """Attention of q [batch, q_tokens, q_heads, head_dim] over the cache; workspace: a uint8
        tensor of attention_kv4_workspace bytes, one for each call that may run at a time. With
        mass_out [batch, kv_heads, max_pages * page_size] (and lse), also decay * mass + the weights
        that the cached tokens received (mass None: zeros; the same tensor: in place)."""
        _refuse(cache, KvCache8, "attention_kv4")
        dev = self.device
        if getattr(q, "ndim", 0) != 4 or q.shape[0] != cache.batch or q.shape[3] != cache.head_dim:
            raise JepaError(1, f"q must be [{cache.batch}, q_tokens, q_heads, {cache.head_dim}]")
        cache.check(dev)
        batch, q_tokens, q_heads, dim = q.shape
        rows = batch * q_tokens * q_heads
        if rows < 1:
            raise JepaError(1, "q_tokens and q_heads must be >= 1")
        held = batch * cache.kv_heads * cache.max_pages * cache.page_size
        st = self.lib.jepa_attention_kv4(
            self.h, cache.ref, _dev(q, "q", "bf16", rows * dim, dev), q_tokens, q_heads,
            _dev(kv_len, "kv_len", "i32", batch, dev), scale, int(causal),
            _dev(out, "out", "bf16", rows * dim, dev), _opt(lse, "lse", "f32", rows, dev),
            _opt(mass, "mass", "f32", held, dev), _opt(mass_out, "mass_out", "f32", held, dev), decay,
            _dev(_sized(workspace, "workspace"), "workspace", "u8", 0, dev), workspace.numel(),
            _stream_on(stream, dev))
        if st:
            self._check(st, "attention_kv4")

    def kv4_evict_workspace(self, cache: KvCache4, keep: int) -> int:
        """Bytes of workspace that kv4_evict needs."""
        n = ctypes.c_size_t()
        self._check(self.lib.jepa_kv4_evict_workspace(self.h, cache.ref, _int32(keep, "keep"), ctypes.byref(n)),
                    "kv4_evict_workspace")
        return n.value

    def kv4_evict(self, cache: KvCache4, kv_len, mass, keep, recent, to: KvCache4, len_out, mass_out,
                  workspace, stream=None):
        """Keep the last `recent` tokens of each sequence and head and those with the largest mass,
        `keep` in all, as the tokens of `to`'s pages; len_out [batch], mass_out (or None) [batch,
        kv_heads, to.max_pages * to.page_size]; workspace: kv4_evict_workspace bytes."""
        _refuse(cache, KvCache8, "kv4_evict")
        _refuse(to, KvCache8, "kv4_evict")
        dev = self.device
        cache.check(dev)
        to.check(dev)
        heads = cache.batch * cache.kv_heads
        st = self.lib.jepa_kv4_evict(
            self.h, cache.ref, _dev(_sized(kv_len, "kv_len"), "kv_len", "i32", cache.batch, dev),
            _dev(mass, "mass", "f32", heads * cache.max_pages * cache.page_size, dev), _int32(keep, "keep"),
            _int32(recent, "recent"), to.ref, _dev(len_out, "len_out", "i32", cache.batch, dev),
            _opt(mass_out, "mass_out", "f32", heads * to.max_pages * to.page_size, dev),
            _dev(_sized(workspace, "workspace"), "workspace", "u8", 0, dev), workspace.numel(),
            _stream_on(stream, dev))
        if st:
            self._check(st, "kv4_evict")

    def add_rmsnorm_fp8(self, x, delta, weight, x_out, codes, scales, eps=1e-6, y=None, stream=None):
        """s = x + delta to x_out (None: not wanted; x: in place), its RMS norm times weight as e4m3
        codes [rows, cols] with scales [rows] (or both None), and as bf16 to y [rows, cols] (or None).
        x and x_out float32 or bf16 [rows, cols], delta either or None."""
        if _Fast.torch is None:
            _Fast.load()
        dev = self.device
        xp, xh, xs = _matrix(x, "x", dev)
        shape = x.shape
        rows, cols = shape
        dp, dh, ds = (None, 0, 0) if delta is None else _matrix(delta, "delta", dev, shape)
        op, oh, os_ = (None, xh, 0) if x_out is None else _matrix(x_out, "x_out", dev, shape)
        if oh != xh:
            raise JepaError(1, "x_out must have x's type")
        if rows < 1 or cols < 1:
            raise JepaError(1, "rows and cols must be >= 1")
        _int32(rows, "rows")
        n = rows * cols
        st = self.lib.jepa_add_rmsnorm_fp8(
            self.h, xp, xh, xs, dp, dh, ds, _dev(weight, "weight", "f32", cols, dev), eps, rows, cols, op,
            os_, _opt(codes, "codes", "u8", n, dev), _opt(scales, "scales", "f32", rows, dev),
            _opt(y, "y", "bf16", n, dev), _stream_on(stream, dev))
        if st:
            self._check(st, "add_rmsnorm_fp8")

    def set_use_graphs(self, on: bool):
        self._check(self.lib.jepa_set_use_graphs(self.h, int(on)), "set_use_graphs")

    def profile_enable(self, on: bool):
        self._check(self.lib.jepa_profile_enable(self.h, int(on)), "profile_enable")

    def profile_read(self):
        ms, fl, n = ctypes.c_double(), ctypes.c_double(), ctypes.c_int64()
        self._check(self.lib.jepa_profile_read(self.h, ctypes.byref(ms), ctypes.byref(fl),
                                               ctypes.byref(n)), "profile_read")
        return ms.value, fl.value, n.value

    def selftest_bounded_wait(self, stream=None):
        self._check(self.lib.jepa_selftest_bounded_wait(self.h, _stream(stream)),
                    "selftest_bounded_wait")

    def sync_check(self, stream=None):
        self._check(self.lib.jepa_sync_check(self.h, _stream(stream)), "sync_check")
