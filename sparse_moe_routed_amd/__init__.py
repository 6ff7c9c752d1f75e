"""Python binding of libmoe.so, the MI355X routed mixture-of-experts layer.

Argument marshalling only: every step of the layer runs in the HIP kernels of
libmoe.so (include/moe.h).  PyTorch supplies device memory and the current
HIP stream.  There is no fallback: if the library is missing or no GPU is
visible, the compute calls raise.

    import sparse_moe_routed_amd as moe
    router = moe.pack_router(w_r, b)                  # once per router matrix
    ids, gates = moe.route(x, router)                 # top-6 routing
    y = moe.forward(x, ids, gates, experts)           # routed experts
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("MOE_LIB") or os.path.join(_PKG, "libmoe.so")

OK, EINVAL, EUNSUPPORTED, EWORKSPACE, EHIP = 0, 1, 2, 3, 4
WFMT = {"bf16": 0, "fp8": 1, "nvfp4": 2, "fp8_block": 3, "int8": 4}
Y_BF16, Y_F32 = 0, 1


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_str(status)} (status {status})")


class Dims(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("ffn", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32)]


class Router(ctypes.Structure):
    _fields_ = [("w_packed", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class Experts(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("up", ctypes.c_void_p), ("down", ctypes.c_void_p),
                ("up_bs", ctypes.c_void_p), ("down_bs", ctypes.c_void_p),
                ("up_s", ctypes.c_void_p), ("down_s", ctypes.c_void_p)]


class Cache(ctypes.Structure):
    _fields_ = [("n_slots", ctypes.c_int32), ("host", Experts), ("up_s", ctypes.c_void_p),
                ("down_s", ctypes.c_void_p), ("slot_up", ctypes.c_void_p),
                ("slot_down", ctypes.c_void_p), ("slot_up_bs", ctypes.c_void_p),
                ("slot_down_bs", ctypes.c_void_p), ("slot_of", ctypes.c_void_p)]


class CacheStats(ctypes.Structure):
    _fields_ = [("touched", ctypes.c_int32), ("hits", ctypes.c_int32), ("misses", ctypes.c_int32),
                ("bytes_uploaded", ctypes.c_int64)]


class WsLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in
                ("counts", "offsets", "sorted_src", "inv", "act", "out_rows", "x_q", "act_q",
                 "scales", "total")]


# symbol name -> (restype, argtypes); must match include/moe.h
_SIGS = {
    "moe_abi_version": (ctypes.c_int32, []),
    "moe_status_str": (ctypes.c_char_p, [ctypes.c_int32]),
    "moe_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(Dims), ctypes.c_int32, ctypes.c_int32]),
    "moe_workspace_layout": (ctypes.c_int32, [ctypes.POINTER(Dims), ctypes.c_int32, ctypes.c_int32,
                                              ctypes.POINTER(WsLayout)]),
    "moe_router_pack": (ctypes.c_int32, [ctypes.POINTER(Dims), ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_void_p]),
    "moe_route_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(Dims), ctypes.c_int32]),
    "moe_route": (ctypes.c_int32, [ctypes.POINTER(Dims), ctypes.c_int32, ctypes.c_void_p,
                                   ctypes.POINTER(Router), ctypes.c_void_p, ctypes.c_void_p,
                                   ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "moe_forward": (ctypes.c_int32, [ctypes.POINTER(Dims), ctypes.c_int32, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(Experts),
                                     ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                     ctypes.c_size_t, ctypes.c_void_p]),
    "moe_forward_timed": (ctypes.c_int32, [ctypes.POINTER(Dims), ctypes.c_int32, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(Experts),
                                           ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                           ctypes.c_size_t, ctypes.c_void_p,
                                           ctypes.POINTER(ctypes.c_void_p), ctypes.c_int32]),
    "moe_shared_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(Dims), ctypes.c_int32,
                                                    ctypes.c_int32]),
    "moe_shared_forward": (ctypes.c_int32, [ctypes.POINTER(Dims), ctypes.c_int32, ctypes.c_void_p,
                                            ctypes.POINTER(Experts), ctypes.c_void_p, ctypes.c_int32,
                                            ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t,
                                            ctypes.c_void_p]),
    "moe_forward_noalloc": (ctypes.c_int32, [ctypes.POINTER(Dims), ctypes.c_int32, ctypes.c_void_p,
                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(Experts),
                                             ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]),
    "moe_cache_state_size": (ctypes.c_size_t, [ctypes.POINTER(Dims), ctypes.c_int32]),
    "moe_cache_init": (ctypes.c_int32, [ctypes.POINTER(Dims), ctypes.POINTER(Cache), ctypes.c_void_p,
                                        ctypes.c_size_t, ctypes.c_void_p]),
    "moe_forward_cached": (ctypes.c_int32, [ctypes.POINTER(Dims), ctypes.c_int32, ctypes.c_void_p,
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(Cache),
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                            ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                            ctypes.POINTER(CacheStats)]),
    "moe_quantize_experts": (ctypes.c_int32, [ctypes.POINTER(Dims), ctypes.c_int32, ctypes.c_void_p,
                                              ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_void_p, ctypes.c_void_p]),
    "moe_quantize_activation": (ctypes.c_int32, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                                 ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                                 ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                                 ctypes.c_void_p]),
    "moe_prenorm": (ctypes.c_int32, [ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p]),
    "moe_residual_add": (ctypes.c_int32, [ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p]),
    "moe_residual_prenorm": (ctypes.c_int32, [ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                              ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "moe_block_pack": (ctypes.c_int32, [ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "moe_block_packed_size": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32]),
    "moe_block_pack_codes": (ctypes.c_int32, [ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                              ctypes.c_void_p, ctypes.c_void_p]),
    "moe_block_quantize": (ctypes.c_int32, [ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "moe_block_matmul": (ctypes.c_int32, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
                         + [ctypes.c_void_p] * 6),
    "moe_block_linear_workspace_size": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32]),
    "moe_block_linear": (ctypes.c_int32, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32]
                         + [ctypes.c_void_p] * 5 + [ctypes.c_size_t, ctypes.c_void_p]),
    "moe_channel_pack": (ctypes.c_int32, [ctypes.c_int32, ctypes.c_int32] + [ctypes.c_void_p] * 4),
    "moe_channel_packed_size": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32]),
    "moe_channel_pack_codes": (ctypes.c_int32, [ctypes.c_int32, ctypes.c_int32] + [ctypes.c_void_p] * 3),
    "moe_channel_quantize": (ctypes.c_int32, [ctypes.c_int32, ctypes.c_int32] + [ctypes.c_void_p] * 4),
    "moe_channel_matmul": (ctypes.c_int32, [ctypes.c_int32] * 3 + [ctypes.c_void_p] * 5
                           + [ctypes.c_int32, ctypes.c_void_p]),
    "moe_channel_linear_workspace_size": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32]),
    "moe_channel_linear": (ctypes.c_int32, [ctypes.c_int32] * 3 + [ctypes.c_void_p] * 4
                           + [ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "moe_grouped_matmul": (ctypes.c_int32, [ctypes.c_int32] * 4 + [ctypes.c_void_p] * 4
                           + [ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p]),
    "moe_grouped_input_grad": (ctypes.c_int32, [ctypes.c_int32] * 4 + [ctypes.c_void_p] * 4
                               + [ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p]),
    "moe_grouped_weight_grad_workspace_size": (ctypes.c_size_t, [ctypes.c_int32] * 4),
    "moe_grouped_weight_grad": (ctypes.c_int32, [ctypes.c_int32] * 4 + [ctypes.c_void_p] * 4
                                + [ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t,
                                   ctypes.c_void_p]),
    "moe_group_rows_workspace_size": (ctypes.c_size_t, [ctypes.c_int32, ctypes.c_int32]),
    "moe_group_rows": (ctypes.c_int32, [ctypes.c_int32] * 2 + [ctypes.c_void_p] * 5
                       + [ctypes.c_size_t, ctypes.c_void_p]),
    "moe_layer_few_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(Dims), ctypes.c_int32,
                                                       ctypes.c_int32]),
    "moe_layer_few": (ctypes.c_int32, [ctypes.POINTER(Dims), ctypes.c_int32, ctypes.c_void_p,
                                       ctypes.POINTER(Router), ctypes.POINTER(Experts),
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t,
                                       ctypes.c_void_p]),
    "moe_residual_norm": (ctypes.c_int32, [ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                           ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_float, ctypes.c_float, ctypes.c_int32,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
}

_lib = None
ABI_VERSION = 9  # MOE_ABI_VERSION of include/moe.h this binding describes


def lib():
    """Load libmoe.so (built in-tree by build.py); raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run `python -m sparse_moe_routed_amd.build`")
        l = ctypes.CDLL(LIB_PATH)
        l.moe_abi_version.restype = ctypes.c_int32
        if l.moe_abi_version() != ABI_VERSION:
            raise ImportError(f"{LIB_PATH} has ABI version {l.moe_abi_version()}, this binding "
                              f"expects {ABI_VERSION}: rebuild with `python -m sparse_moe_routed_amd.build`")
        for name, (res, args) in _SIGS.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
    return _lib


def status_str(status: int) -> str:
    return lib().moe_status_str(int(status)).decode()


def _check(fn: str, status: int):
    if status != OK:
        raise MoeError(fn, status)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _dev(t: torch.Tensor, dtype, name: str, shape=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected dtype {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    if shape is not None and t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


@dataclass
class LayerDims:
    hidden: int = 2688
    ffn: int = 1856
    n_experts: int = 128
    top_k: int = 6

    def c(self) -> Dims:
        return Dims(self.hidden, self.ffn, self.n_experts, self.top_k)


@dataclass
class ExpertBank:
    """Device expert bank in one of the formats of WFMT (see moe_experts in moe.h)."""
    fmt: str
    up: torch.Tensor
    down: torch.Tensor
    up_bs: Optional[torch.Tensor] = None
    down_bs: Optional[torch.Tensor] = None
    up_s: Optional[torch.Tensor] = None
    down_s: Optional[torch.Tensor] = None

    def c(self) -> Experts:
        return Experts(WFMT[self.fmt], self.up.data_ptr(), self.down.data_ptr(),
                       self.up_bs.data_ptr() if self.up_bs is not None else None,
                       self.down_bs.data_ptr() if self.down_bs is not None else None,
                       self.up_s.data_ptr() if self.up_s is not None else None,
                       self.down_s.data_ptr() if self.down_s is not None else None)


@functools.lru_cache(maxsize=256)
def _bank_parts(fmt: str, E: int, H: int, F: int):
    """(field, dtype or None, bytes) of a bank's tensors."""
    n, code, scale = E * H * F, None, torch.float32
    if fmt == "bf16":
        return ("up", torch.bfloat16, 2 * n), ("down", torch.bfloat16, 2 * n)
    if fmt == "fp8":
        return ("up", code, n), ("down", code, n), ("up_s", scale, 4 * E), ("down_s", scale, 4 * E)
    if fmt == "nvfp4":
        return (("up", code, n // 2), ("down", code, n // 2), ("up_s", scale, 4 * E), ("down_s", scale, 4 * E),
                ("up_bs", code, n // 16), ("down_bs", code, n // 16))
    kh, kf = -(-H // 128), -(-F // 128)
    if fmt == "int8":
        return (("up", code, E * -(-F // 16) * kh * 2048), ("down", code, E * -(-H // 16) * kf * 2048),
                ("up_s", scale, 4 * E * F), ("down_s", scale, 4 * E * H))
    return (("up", code, E * -(-F // 16) * kh * 2048), ("down", code, E * -(-H // 16) * kf * 2048),
            ("up_s", scale, 4 * E * kh * kf), ("down_s", scale, 4 * E * kh * kf))


def _check_bank(bank: ExpertBank, dims: LayerDims, device: torch.device):
    """The bank's tensors are on the device and hold the layer's experts: the
    kernels read them by the dims alone."""
    for name, dtype, n in _bank_parts(bank.fmt, dims.n_experts, dims.hidden, dims.ffn):
        t = getattr(bank, name)
        if not (isinstance(t, torch.Tensor) and t.nbytes >= n and t.device == device and t.is_contiguous() and
                (dtype is None or t.dtype is dtype)):
            what = "None" if t is None else f"{tuple(t.shape)} {t.dtype} on {t.device}"
            raise ValueError(f"{name}: {what}; {dims} needs a contiguous {dtype or 'byte'} tensor of {n} bytes "
                             f"or more on {device}")


def abi_version() -> int:
    return lib().moe_abi_version()


def workspace_size(dims: LayerDims, fmt: str, max_tokens: int) -> int:
    d = dims.c()
    return int(lib().moe_workspace_size(ctypes.byref(d), WFMT[fmt], int(max_tokens)))


def workspace_layout(dims: LayerDims, fmt: str, T: int) -> dict:
    d = dims.c()
    out = WsLayout()
    _check("moe_workspace_layout", lib().moe_workspace_layout(ctypes.byref(d), WFMT[fmt], int(T),
                                                              ctypes.byref(out)))
    return {n: getattr(out, n) for n, _ in WsLayout._fields_}


def workspace(dims: LayerDims, fmt: str, max_tokens: int, device="cuda") -> torch.Tensor:
    return torch.empty(max(256, workspace_size(dims, fmt, max_tokens)), dtype=torch.uint8, device=device)


@dataclass
class PackedRouter:
    """Router matrix packed by moe_router_pack (bf16 [3, E, H]) and its bias."""
    w_packed: torch.Tensor
    bias: Optional[torch.Tensor] = None


def pack_router(w_r: torch.Tensor, bias: Optional[torch.Tensor] = None,
                dims: LayerDims = LayerDims()) -> PackedRouter:
    """moe_router_pack: fp32 [E, H] -> exact bf16 (hi, mid, lo) split."""
    _dev(w_r, torch.float32, "w_r", (dims.n_experts, dims.hidden))
    if bias is not None:
        _dev(bias, torch.float32, "bias", (dims.n_experts,))
    packed = torch.empty((3, dims.n_experts, dims.hidden), dtype=torch.bfloat16, device=w_r.device)
    d = dims.c()
    _check("moe_router_pack", lib().moe_router_pack(ctypes.byref(d), _ptr(w_r), _ptr(packed), _stream()))
    return PackedRouter(packed, bias)


def route_workspace(dims: LayerDims, max_tokens: int, device="cuda") -> torch.Tensor:
    d = dims.c()
    n = int(lib().moe_route_workspace_size(ctypes.byref(d), int(max_tokens)))
    return torch.empty(max(256, n), dtype=torch.uint8, device=device)


def route(x: torch.Tensor, router: PackedRouter, dims: LayerDims = LayerDims(),
          ids: Optional[torch.Tensor] = None, gates: Optional[torch.Tensor] = None,
          ws: Optional[torch.Tensor] = None):
    """moe_route: ids int32 [T, k], gates fp32 [T, k]."""
    T = x.shape[0]
    _dev(x, torch.bfloat16, "x", (T, dims.hidden))
    _dev(router.w_packed, torch.bfloat16, "w_packed", (3, dims.n_experts, dims.hidden))
    if router.bias is not None:
        _dev(router.bias, torch.float32, "bias", (dims.n_experts,))
    if ids is None:
        ids = torch.empty((T, dims.top_k), dtype=torch.int32, device=x.device)
    if gates is None:
        gates = torch.empty((T, dims.top_k), dtype=torch.float32, device=x.device)
    if ws is None:
        ws = route_workspace(dims, T, x.device)
    _dev(ids, torch.int32, "ids", (T, dims.top_k))
    _dev(gates, torch.float32, "gates", (T, dims.top_k))
    _dev(ws, torch.uint8, "ws")
    d = dims.c()
    r = Router(router.w_packed.data_ptr(),
               router.bias.data_ptr() if router.bias is not None else None)
    _check("moe_route", lib().moe_route(ctypes.byref(d), T, _ptr(x), ctypes.byref(r), _ptr(ids),
                                        _ptr(gates), _ptr(ws), ws.numel(), _stream()))
    return ids, gates


def forward(x: torch.Tensor, ids: torch.Tensor, gates: torch.Tensor, experts: ExpertBank,
            dims: LayerDims = LayerDims(), y_dtype: torch.dtype = torch.float32,
            ws: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_forward: y [T, H] in fp32 or bf16."""
    T = x.shape[0]
    _dev(x, torch.bfloat16, "x", (T, dims.hidden))
    _dev(ids, torch.int32, "ids", (T, dims.top_k))
    _dev(gates, torch.float32, "gates", (T, dims.top_k))
    if ws is None:
        ws = workspace(dims, experts.fmt, T, x.device)
    _dev(ws, torch.uint8, "ws")
    if y is None:
        y = torch.empty((T, dims.hidden), dtype=y_dtype, device=x.device)
    _dev(y, y_dtype, "y", (T, dims.hidden))
    _check_bank(experts, dims, x.device)
    yd = {torch.float32: Y_F32, torch.bfloat16: Y_BF16}[y_dtype]
    d = dims.c()
    e = experts.c()
    _check("moe_forward", lib().moe_forward(ctypes.byref(d), T, _ptr(x), _ptr(ids), _ptr(gates),
                                            ctypes.byref(e), _ptr(y), yd, _ptr(ws),
                                            ws.numel(), _stream()))
    return y


def shared_dims(hidden: int = 2688, ffn: int = 3712) -> LayerDims:
    """Dims of a shared expert: one expert that every token takes."""
    return LayerDims(hidden, ffn, 1, 1)


def shared_workspace(dims: LayerDims, fmt: str, max_tokens: int, device="cuda") -> torch.Tensor:
    d = dims.c()
    n = int(lib().moe_shared_workspace_size(ctypes.byref(d), WFMT[fmt], int(max_tokens)))
    if n == 0:
        raise ValueError(f"moe_shared_workspace_size: invalid dims {dims} or format {fmt}")
    return torch.empty(n, dtype=torch.uint8, device=device)


def shared_forward(x: torch.Tensor, expert: ExpertBank, dims: LayerDims,
                   y: Optional[torch.Tensor] = None, y_dtype: torch.dtype = torch.float32,
                   accumulate: bool = False, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_shared_forward: the shared expert on every token; with accumulate,
    added to the fp32 y given (the routed output, for the MoE block)."""
    T = x.shape[0]
    _dev(x, torch.bfloat16, "x", (T, dims.hidden))
    if y is None:
        if accumulate:
            raise ValueError("accumulate needs the y to add to")
        y = torch.empty((T, dims.hidden), dtype=y_dtype, device=x.device)
    _dev(y, y_dtype, "y", (T, dims.hidden))
    if ws is None:
        ws = shared_workspace(dims, expert.fmt, T, x.device)
    _dev(ws, torch.uint8, "ws")
    _check_bank(expert, dims, x.device)
    yd = {torch.float32: Y_F32, torch.bfloat16: Y_BF16}[y_dtype]
    d = dims.c()
    e = expert.c()
    _check("moe_shared_forward", lib().moe_shared_forward(
        ctypes.byref(d), T, _ptr(x), ctypes.byref(e), _ptr(y), yd, int(bool(accumulate)),
        _ptr(ws), ws.numel(), _stream()))
    return y


NOALLOC_SCRATCH_BYTES = 8 << 20  # MOE_NOALLOC_SCRATCH_BYTES of include/moe.h


def forward_noalloc(x: torch.Tensor, ids: torch.Tensor, gates: torch.Tensor, experts: ExpertBank,
                    dims: LayerDims = LayerDims(), y_dtype: torch.dtype = torch.float32,
                    y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_forward_noalloc: moe_forward with the library's fixed device
    scratch instead of a workspace (y is allocated here unless passed)."""
    T = x.shape[0]
    _dev(x, torch.bfloat16, "x", (T, dims.hidden))
    _dev(ids, torch.int32, "ids", (T, dims.top_k))
    _dev(gates, torch.float32, "gates", (T, dims.top_k))
    if y is None:
        y = torch.empty((T, dims.hidden), dtype=y_dtype, device=x.device)
    _dev(y, y_dtype, "y", (T, dims.hidden))
    _check_bank(experts, dims, x.device)
    yd = {torch.float32: Y_F32, torch.bfloat16: Y_BF16}[y_dtype]
    d = dims.c()
    e = experts.c()
    _check("moe_forward_noalloc", lib().moe_forward_noalloc(
        ctypes.byref(d), T, _ptr(x), _ptr(ids), _ptr(gates), ctypes.byref(e), _ptr(y), yd,
        _stream()))
    return y


N_STAGES = 6
STAGES = ("permute", "quant_x", "up", "quant_act", "down", "combine")
N_TIMED_EVENTS = N_STAGES + 5


def forward_timed(x: torch.Tensor, ids: torch.Tensor, gates: torch.Tensor, experts: ExpertBank,
                  events, dims: LayerDims = LayerDims(), y_dtype: torch.dtype = torch.float32,
                  ws: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_forward_timed: like forward, recording the caller's hipEvent_t handles
    (a sequence of N_STAGES + 1 ints) before each stage and after the last;
    N_TIMED_EVENTS handles add the up and down GEMM kernels' own start and end."""
    T = x.shape[0]
    if ws is None:
        ws = workspace(dims, experts.fmt, T, x.device)
    if y is None:
        y = torch.empty((T, dims.hidden), dtype=y_dtype, device=x.device)
    _dev(x, torch.bfloat16, "x", (T, dims.hidden))
    _dev(ids, torch.int32, "ids", (T, dims.top_k))
    _dev(gates, torch.float32, "gates", (T, dims.top_k))
    _dev(ws, torch.uint8, "ws")
    _dev(y, y_dtype, "y", (T, dims.hidden))
    _check_bank(experts, dims, x.device)
    yd = {torch.float32: Y_F32, torch.bfloat16: Y_BF16}[y_dtype]
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e) for e in events])
    d = dims.c()
    e = experts.c()
    _check("moe_forward_timed", lib().moe_forward_timed(
        ctypes.byref(d), T, _ptr(x), _ptr(ids), _ptr(gates), ctypes.byref(e), _ptr(y), yd,
        _ptr(ws), ws.numel(), _stream(), arr, len(events)))
    return y


class ExpertCache:
    """moe_cache: the bank's codes in pinned host memory and n_slots device
    slots that hold the experts batches select (least recently used replaced).
    Per-expert scales stay on the device."""

    def __init__(self, bank: ExpertBank, n_slots: int, dims: LayerDims = LayerDims()):
        _check_bank(bank, dims, bank.up.device)
        dev = bank.up.device

        def host(t):
            if t is None:
                return None
            h = torch.empty(t.shape, dtype=t.dtype, pin_memory=True)
            h.copy_(t)
            return h

        def slots(t):
            return None if t is None else torch.empty((n_slots,) + tuple(t.shape[1:]), dtype=t.dtype,
                                                       device=dev)

        self.fmt, self.n_slots, self.dims = bank.fmt, int(n_slots), dims
        self.host_up, self.host_down = host(bank.up), host(bank.down)
        self.host_up_bs, self.host_down_bs = host(bank.up_bs), host(bank.down_bs)
        self.up_s, self.down_s = bank.up_s, bank.down_s
        self.slot_up, self.slot_down = slots(bank.up), slots(bank.down)
        self.slot_up_bs, self.slot_down_bs = slots(bank.up_bs), slots(bank.down_bs)
        self.slot_of = torch.empty(dims.n_experts, dtype=torch.int32, device=dev)
        d = dims.c()
        self.state_bytes = int(lib().moe_cache_state_size(ctypes.byref(d), self.n_slots))
        if self.state_bytes == 0:
            raise ValueError(f"n_slots {n_slots} outside [top_k, n_experts]")
        self.state = (ctypes.c_uint64 * ((self.state_bytes + 7) // 8))()  # 8-byte aligned
        c = self.c()
        _check("moe_cache_init", lib().moe_cache_init(ctypes.byref(d), ctypes.byref(c), self.state,
                                                      self.state_bytes, _stream()))

    def c(self) -> Cache:
        p = lambda t: t.data_ptr() if t is not None else None
        h = Experts(WFMT[self.fmt], p(self.host_up), p(self.host_down), p(self.host_up_bs),
                    p(self.host_down_bs), None, None)
        return Cache(self.n_slots, h, p(self.up_s), p(self.down_s), p(self.slot_up),
                     p(self.slot_down), p(self.slot_up_bs), p(self.slot_down_bs), p(self.slot_of))


def forward_cached(x: torch.Tensor, ids: torch.Tensor, gates: torch.Tensor, cache: ExpertCache,
                   dims: LayerDims = LayerDims(), y_dtype: torch.dtype = torch.float32,
                   ws: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
    """moe_forward_cached: (y [T, H], stats dict); y equals forward() on the
    bank the cache was built from."""
    if dims != cache.dims:
        raise ValueError(f"dims: {dims}, the cache was built for {cache.dims}")
    T = x.shape[0]
    _dev(x, torch.bfloat16, "x", (T, dims.hidden))
    _dev(ids, torch.int32, "ids", (T, dims.top_k))
    _dev(gates, torch.float32, "gates", (T, dims.top_k))
    if ws is None:
        ws = workspace(dims, cache.fmt, T, x.device)
    _dev(ws, torch.uint8, "ws")
    if y is None:
        y = torch.empty((T, dims.hidden), dtype=y_dtype, device=x.device)
    _dev(y, y_dtype, "y", (T, dims.hidden))
    yd = {torch.float32: Y_F32, torch.bfloat16: Y_BF16}[y_dtype]
    d = dims.c()
    c = cache.c()
    st = CacheStats()
    _check("moe_forward_cached", lib().moe_forward_cached(
        ctypes.byref(d), T, _ptr(x), _ptr(ids), _ptr(gates), ctypes.byref(c), cache.state, _ptr(y),
        yd, _ptr(ws), ws.numel(), _stream(), ctypes.byref(st)))
    return y, {"touched": st.touched, "hits": st.hits, "misses": st.misses,
               "bytes_uploaded": st.bytes_uploaded}


def quantize_experts(up: torch.Tensor, down: torch.Tensor, fmt: str,
                     dims: LayerDims = LayerDims()) -> ExpertBank:
    """moe_quantize_experts: pack a bf16 bank [E,F,H] / [E,H,F] into fp8, nvfp4,
    fp8_block or int8."""
    if fmt == "bf16":
        return ExpertBank("bf16", up, down)
    E, F, H = dims.n_experts, dims.ffn, dims.hidden
    _dev(up, torch.bfloat16, "up", (E, F, H))
    _dev(down, torch.bfloat16, "down", (E, H, F))
    dev = up.device
    if fmt == "fp8":
        up_q = torch.empty((E, F, H), dtype=torch.uint8, device=dev)
        # down codes: per-expert byte arrays in the panel layout (moe.h)
        down_q = torch.empty((E, H * F), dtype=torch.uint8, device=dev)
        up_bs = down_bs = None
    elif fmt == "nvfp4":
        # per-expert byte arrays in the panel layout of moe_experts (moe.h)
        up_q = torch.empty((E, F * H // 2), dtype=torch.uint8, device=dev)
        down_q = torch.empty((E, H * F // 2), dtype=torch.uint8, device=dev)
        up_bs = torch.empty((E, F * H // 16), dtype=torch.uint8, device=dev)
        down_bs = torch.empty((E, H * F // 16), dtype=torch.uint8, device=dev)
    elif fmt == "fp8_block":
        up_q = torch.empty((E, block_packed_size(F, H)), dtype=torch.uint8, device=dev)
        down_q = torch.empty((E, block_packed_size(H, F)), dtype=torch.uint8, device=dev)
        up_bs = down_bs = None
    elif fmt == "int8":
        up_q = torch.empty((E, channel_packed_size(F, H)), dtype=torch.int8, device=dev)
        down_q = torch.empty((E, channel_packed_size(H, F)), dtype=torch.int8, device=dev)
        up_bs = down_bs = None
    else:
        raise ValueError(fmt)
    nf, nh = (-(-F // 128), -(-H // 128))
    up_shape = {"fp8_block": (E, nf, nh), "int8": (E, F)}.get(fmt, (E,))
    down_shape = {"fp8_block": (E, nh, nf), "int8": (E, H)}.get(fmt, (E,))
    up_s = torch.empty(up_shape, dtype=torch.float32, device=dev)
    down_s = torch.empty(down_shape, dtype=torch.float32, device=dev)
    d = dims.c()
    _check("moe_quantize_experts", lib().moe_quantize_experts(
        ctypes.byref(d), WFMT[fmt], _ptr(up), _ptr(down), _ptr(up_q), _ptr(down_q),
        _ptr(up_bs), _ptr(down_bs), _ptr(up_s), _ptr(down_s), _stream()))
    return ExpertBank(fmt, up_q, down_q, up_bs, down_bs, up_s, down_s)


def quantize_activation(x: torch.Tensor, fmt: str):
    """moe_quantize_activation: (codes, block scales or None, scale fp32[1]; fp8_block:
    [ceil(cols / 128), rows]; int8: [rows])."""
    rows, cols = x.shape
    _dev(x, torch.bfloat16, "x")
    dev = x.device
    if fmt in ("fp8", "fp8_block", "int8"):
        codes = torch.empty((rows, cols), dtype=torch.int8 if fmt == "int8" else torch.uint8, device=dev)
        bs = None
    elif fmt == "nvfp4":
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
        bs = torch.empty((rows, cols // 16), dtype=torch.uint8, device=dev)
    else:
        raise ValueError(fmt)
    shape = {"fp8_block": (-(-cols // 128), rows), "int8": (rows,)}.get(fmt, (1,))
    scale = torch.empty(shape, dtype=torch.float32, device=dev)
    ws = torch.empty(256, dtype=torch.uint8, device=dev)
    _check("moe_quantize_activation", lib().moe_quantize_activation(
        WFMT[fmt], rows, cols, _ptr(x), _ptr(codes), _ptr(bs), _ptr(scale), _ptr(ws), 256, _stream()))
    return codes, bs, scale


def prenorm(x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    T, H = x.shape
    _dev(x, torch.bfloat16, "x")
    if out is None:
        out = torch.empty_like(x)
    _check("moe_prenorm", lib().moe_prenorm(T, H, _ptr(x), _ptr(out), _stream()))
    return out


def residual_add(x: torch.Tensor, y: torch.Tensor) -> torch.Tensor:
    T, H = x.shape
    _dev(x, torch.bfloat16, "x")
    _dev(y, torch.float32, "y", (T, H))
    _check("moe_residual_add", lib().moe_residual_add(T, H, _ptr(x), _ptr(y), _stream()))
    return x


def residual_prenorm(x: torch.Tensor, y: torch.Tensor,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_residual_prenorm: x <- bf16(x + y) in place, returns prenorm(x) in out."""
    T, H = x.shape
    _dev(x, torch.bfloat16, "x")
    _dev(y, torch.float32, "y", (T, H))
    if out is None:
        out = torch.empty_like(x)
    _dev(out, torch.bfloat16, "out", (T, H))
    _check("moe_residual_prenorm",
           lib().moe_residual_prenorm(T, H, _ptr(x), _ptr(y), _ptr(out), _stream()))
    return out


GATE_NONE, GATE_TOKEN, GATE_CHANNEL, GATE_ELEMENT = 0, 1, 2, 3


def _launch(name: str, fn, index: int, *args):
    """fn(*args, the current stream of device `index`), with that device current."""
    here = torch._C._cuda_getDevice()
    if here != index:
        torch._C._cuda_setDevice(index)
    try:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    finally:
        if here != index:
            torch._C._cuda_setDevice(here)
    if status != OK:
        raise MoeError(name, status)


def _same_device(device: torch.device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name}: on {t.device}, x is on {device}")


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _arg(t, dtype, name: str, shape, device: torch.device):
    """_dev and _same_device in one look, for calls whose kernels are shorter than
    their arguments' checks: a microsecond of a call with seven tensors."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and
            t.device == device and t.is_contiguous()):
        _dev(t, dtype, name, shape)
        _same_device(device, **{name: t})


_Y_DTYPES = {torch.float32: Y_F32, torch.bfloat16: Y_BF16}


def residual_norm(x: torch.Tensor, y: Optional[torch.Tensor], out: Optional[torch.Tensor] = None,
                  x_out: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                  post_weight: Optional[torch.Tensor] = None,
                  pre_weight: Optional[torch.Tensor] = None, scale: float = 1.0,
                  eps: float = 1e-6, post_norm: bool = True, pre_norm: bool = True):
    """moe_residual_norm: (x', out).  x' goes into x_out, or into x itself when
    it is None; with pre_norm=False there is no out (None).  The gate's shape
    says its kind: [T, 1], [H] or [T, H].  Without a block output (y=None) x
    stays and out is its pre-norm."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x: expected a [T, H] tensor")
    T, H = rows = x.shape
    _dev(x, torch.bfloat16, "x")
    dev = x.device
    kind, yd = GATE_NONE, Y_F32
    if y is not None:
        yd = _Y_DTYPES.get(y.dtype)
        if yd is None:
            raise ValueError(f"y: expected float32 or bfloat16, got {y.dtype}")
        _arg(y, y.dtype, "y", rows, dev)
        if x_out is None:
            x_out = x
        else:
            _arg(x_out, torch.bfloat16, "x_out", rows, dev)
    elif x_out is not None or gate is not None or post_weight is not None:
        raise ValueError("x_out, gate and post_weight need a block output y")
    if gate is not None:
        shape = gate.shape
        kind = (GATE_TOKEN if shape == (T, 1) else GATE_CHANNEL if shape == (H,) else
                GATE_ELEMENT if shape == rows else None)
        if kind is None:
            raise ValueError(f"gate: expected shape ({T}, 1), ({H},) or ({T}, {H}), got {tuple(gate.shape)}")
        _arg(gate, torch.float32, "gate", shape, dev)
    if post_weight is not None:
        _arg(post_weight, torch.float32, "post_weight", (H,), dev)
    if pre_weight is not None:
        _arg(pre_weight, torch.float32, "pre_weight", (H,), dev)
    if pre_norm and out is None:
        out = torch.empty_like(x)
    if out is not None:
        if not pre_norm:
            raise ValueError("out: given with pre_norm=False")
        _arg(out, torch.bfloat16, "out", rows, dev)
    _launch("moe_residual_norm", lib().moe_residual_norm, dev.index,
            T, H, x.data_ptr(), _p(y), yd, _p(gate), kind, _p(post_weight), _p(pre_weight), scale, eps,
            1 if post_norm else 0, _p(x_out), _p(out))
    return (x if y is None else x_out), out


FEW_TOKENS = 16  # MOE_FEW_TOKENS of include/moe.h


def layer_few_workspace(dims: LayerDims, fmt: str, max_tokens: int = FEW_TOKENS,
                        device="cuda") -> torch.Tensor:
    d = dims.c()
    n = int(lib().moe_layer_few_workspace_size(ctypes.byref(d), WFMT[fmt], int(max_tokens)))
    if n == 0:
        raise ValueError(f"moe_layer_few_workspace_size: invalid dims {dims}, format {fmt} or "
                         f"max_tokens {max_tokens} (at most {FEW_TOKENS})")
    return torch.empty(n, dtype=torch.uint8, device=device)


def layer_few(x: torch.Tensor, router: PackedRouter, experts: ExpertBank,
              dims: LayerDims = LayerDims(), y_dtype: torch.dtype = torch.float32,
              ids: Optional[torch.Tensor] = None, gates: Optional[torch.Tensor] = None,
              ws: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
    """moe_layer_few: route and forward of at most FEW_TOKENS tokens, in two
    kernels where that is faster; (y [T, H], ids int32 [T, k], gates fp32 [T, k])."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x: expected a [T, H] tensor")
    T, dev = x.shape[0], x.device
    _dev(x, torch.bfloat16, "x", (T, dims.hidden))
    _arg(router.w_packed, torch.bfloat16, "w_packed", (3, dims.n_experts, dims.hidden), dev)
    if router.bias is not None:
        _arg(router.bias, torch.float32, "bias", (dims.n_experts,), dev)
    _check_bank(experts, dims, dev)
    if ids is None:
        ids = torch.empty((T, dims.top_k), dtype=torch.int32, device=dev)
    else:
        _arg(ids, torch.int32, "ids", (T, dims.top_k), dev)
    if gates is None:
        gates = torch.empty((T, dims.top_k), dtype=torch.float32, device=dev)
    else:
        _arg(gates, torch.float32, "gates", (T, dims.top_k), dev)
    if y is None:
        y = torch.empty((T, dims.hidden), dtype=y_dtype, device=dev)
    else:
        _arg(y, y_dtype, "y", (T, dims.hidden), dev)
    if ws is None:
        ws = layer_few_workspace(dims, experts.fmt, min(T, FEW_TOKENS), dev)
    else:
        _arg(ws, torch.uint8, "ws", getattr(ws, "shape", None), dev)
    yd = _Y_DTYPES[y_dtype]
    d = dims.c()
    r = Router(router.w_packed.data_ptr(),
               router.bias.data_ptr() if router.bias is not None else None)
    e = experts.c()
    _launch("moe_layer_few", lib().moe_layer_few, dev.index,
            ctypes.byref(d), T, x.data_ptr(), ctypes.byref(r), ctypes.byref(e), ids.data_ptr(),
            gates.data_ptr(), y.data_ptr(), yd, ws.data_ptr(), ws.numel())
    return y, ids, gates


BLOCK_FEW_ROWS = 32  # MOE_BLOCK_FEW_ROWS of include/moe.h


@dataclass
class BlockWeight:
    """A weight of `shape` (N, K) packed by moe_block_pack: E4M3 codes u8
    [block_packed_size(N, K)] and one fp32 scale per 128 x 128 block,
    [ceil(N / 128), ceil(K / 128)]."""
    codes: torch.Tensor
    scales: torch.Tensor
    shape: tuple


def block_packed_size(N: int, K: int) -> int:
    n = int(lib().moe_block_packed_size(int(N), int(K)))
    if n == 0:
        raise ValueError(f"moe_block_packed_size: invalid N {N} or K {K} (K % 16 == 0)")
    return n


def _matrix(t: torch.Tensor, dtype, name: str):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name}: expected a matrix")
    return _dev(t, dtype, name)


def block_pack(w: torch.Tensor) -> BlockWeight:
    """moe_block_pack: bf16 [N, K] -> E4M3 codes with a scale per 128 x 128 block."""
    N, K = _matrix(w, torch.bfloat16, "w").shape
    codes = torch.empty(block_packed_size(N, K), dtype=torch.uint8, device=w.device)
    scales = torch.empty((-(-N // 128), -(-K // 128)), dtype=torch.float32, device=w.device)
    _launch("moe_block_pack", lib().moe_block_pack, w.device.index,
            N, K, w.data_ptr(), codes.data_ptr(), scales.data_ptr())
    return BlockWeight(codes, scales, (N, K))


def block_pack_codes(codes: torch.Tensor, scales: torch.Tensor) -> BlockWeight:
    """moe_block_pack_codes: row-major E4M3 codes [N, K] (u8 or float8_e4m3fn) and
    their block scales fp32 [ceil(N / 128), ceil(K / 128)], as a checkpoint holds
    them."""
    if isinstance(codes, torch.Tensor) and codes.dtype == torch.float8_e4m3fn:
        codes = codes.view(torch.uint8)
    N, K = _matrix(codes, torch.uint8, "codes").shape
    _dev(scales, torch.float32, "scales", (-(-N // 128), -(-K // 128)))
    _same_device(codes.device, scales=scales)
    packed = torch.empty(block_packed_size(N, K), dtype=torch.uint8, device=codes.device)
    _launch("moe_block_pack_codes", lib().moe_block_pack_codes, codes.device.index,
            N, K, codes.data_ptr(), packed.data_ptr())
    return BlockWeight(packed, scales, (N, K))


def block_quantize(x: torch.Tensor):
    """moe_block_quantize: bf16 [M, K] -> (codes u8 [M, K], scales fp32
    [ceil(K / 128), M])."""
    M, K = _matrix(x, torch.bfloat16, "x").shape
    codes = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    scales = torch.empty((-(-K // 128), M), dtype=torch.float32, device=x.device)
    _launch("moe_block_quantize", lib().moe_block_quantize, x.device.index,
            M, K, x.data_ptr(), codes.data_ptr(), scales.data_ptr())
    return codes, scales


def _block_operands(rows: torch.Tensor, weight: BlockWeight, y: Optional[torch.Tensor]):
    M, K = rows.shape
    N = weight.shape[0]
    if weight.shape[1] != K:
        raise ValueError(f"weight: K is {weight.shape[1]}, the rows have {K}")
    dev = rows.device
    _arg(weight.codes, torch.uint8, "weight.codes", ((N + 15) // 16 * -(-K // 128) * 2048,), dev)
    _arg(weight.scales, torch.float32, "weight.scales", (-(-N // 128), -(-K // 128)), dev)
    if y is None:
        y = rows.new_empty((M, N), dtype=torch.bfloat16)
    else:
        _arg(y, torch.bfloat16, "y", (M, N), dev)
    return M, N, K, y


def block_matmul(codes: torch.Tensor, scales: torch.Tensor, weight: BlockWeight,
                 y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_block_matmul: bf16 [M, N] from codes and scales of block_quantize."""
    _matrix(codes, torch.uint8, "codes")
    M, N, K, y = _block_operands(codes, weight, y)
    _dev(scales, torch.float32, "scales", (-(-K // 128), M))
    _same_device(codes.device, scales=scales)
    _launch("moe_block_matmul", lib().moe_block_matmul, codes.device.index,
            M, N, K, codes.data_ptr(), scales.data_ptr(), weight.codes.data_ptr(),
            weight.scales.data_ptr(), y.data_ptr())
    return y


@functools.lru_cache(maxsize=256)
def _block_linear_bytes(max_rows: int, K: int) -> int:
    return int(lib().moe_block_linear_workspace_size(max_rows, K))


def block_linear_workspace(max_rows: int, K: int, device="cuda") -> torch.Tensor:
    n = _block_linear_bytes(int(max_rows), int(K))
    if n == 0:
        raise ValueError(f"moe_block_linear_workspace_size: invalid rows {max_rows} or K {K}")
    return torch.empty(n, dtype=torch.uint8, device=device)


def block_linear(x: torch.Tensor, weight: BlockWeight, y: Optional[torch.Tensor] = None,
                 ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_block_linear: bf16 [M, N] = x [M, K] quantised by rows, times the weight."""
    _matrix(x, torch.bfloat16, "x")
    M, N, K, y = _block_operands(x, weight, y)
    if ws is not None:
        _dev(ws, torch.uint8, "ws")
        _same_device(x.device, ws=ws)
    elif M > BLOCK_FEW_ROWS:
        ws = block_linear_workspace(M, K, x.device)
    _launch("moe_block_linear", lib().moe_block_linear, x.device.index,
            M, N, K, x.data_ptr(), weight.codes.data_ptr(), weight.scales.data_ptr(), y.data_ptr(),
            _p(ws), 0 if ws is None else ws.numel())
    return y


CHANNEL_FEW_ROWS = 32  # MOE_CHANNEL_FEW_ROWS of include/moe.h


@dataclass
class ChannelWeight:
    """A weight of `shape` (N, K) packed by moe_channel_pack: 8-bit integer codes
    [channel_packed_size(N, K)] and one fp32 scale per output channel, [N]."""
    codes: torch.Tensor
    scales: torch.Tensor
    shape: tuple


def channel_packed_size(N: int, K: int) -> int:
    n = int(lib().moe_channel_packed_size(int(N), int(K)))
    if n == 0:
        raise ValueError(f"moe_channel_packed_size: invalid N {N} or K {K} (K % 16 == 0, K <= 65536)")
    return n


def channel_pack(w: torch.Tensor) -> ChannelWeight:
    """moe_channel_pack: bf16 [N, K] -> 8-bit integer codes with a scale per row."""
    N, K = _matrix(w, torch.bfloat16, "w").shape
    codes = torch.empty(channel_packed_size(N, K), dtype=torch.int8, device=w.device)
    scales = torch.empty(N, dtype=torch.float32, device=w.device)
    _launch("moe_channel_pack", lib().moe_channel_pack, w.device.index,
            N, K, w.data_ptr(), codes.data_ptr(), scales.data_ptr())
    return ChannelWeight(codes, scales, (N, K))


def channel_pack_codes(codes: torch.Tensor, scales: torch.Tensor) -> ChannelWeight:
    """moe_channel_pack_codes: row-major int8 codes [N, K] and their channel scales
    fp32 [N], as a checkpoint holds them."""
    N, K = _matrix(codes, torch.int8, "codes").shape
    _arg(scales, torch.float32, "scales", (N,), codes.device)
    packed = torch.empty(channel_packed_size(N, K), dtype=torch.int8, device=codes.device)
    _launch("moe_channel_pack_codes", lib().moe_channel_pack_codes, codes.device.index,
            N, K, codes.data_ptr(), packed.data_ptr())
    return ChannelWeight(packed, scales, (N, K))


def channel_quantize(x: torch.Tensor):
    """moe_channel_quantize: bf16 [M, K] -> (codes int8 [M, K], scales fp32 [M])."""
    M, K = _matrix(x, torch.bfloat16, "x").shape
    codes = torch.empty((M, K), dtype=torch.int8, device=x.device)
    scales = torch.empty(M, dtype=torch.float32, device=x.device)
    _launch("moe_channel_quantize", lib().moe_channel_quantize, x.device.index,
            M, K, x.data_ptr(), codes.data_ptr(), scales.data_ptr())
    return codes, scales


def _out(out: Optional[torch.Tensor], dtype: Optional[torch.dtype], name: str, shape, like: torch.Tensor):
    """(output tensor, its MOE_Y_*): `out` as given, whose dtype must be `dtype` unless
    that is None, or a new one (bf16 for None)."""
    if out is None:
        out = like.new_empty(shape, dtype=torch.bfloat16 if dtype is None else dtype)
        yd = _Y_DTYPES.get(out.dtype)
    else:
        yd = _Y_DTYPES.get(out.dtype) if isinstance(out, torch.Tensor) else None
        if yd is not None:
            _arg(out, out.dtype if dtype is None else dtype, name, shape, like.device)
    if yd is None:
        raise ValueError(f"{name}: expected float32 or bfloat16")
    return out, yd


def _channel_operands(rows: torch.Tensor, weight: ChannelWeight, y, y_dtype):
    M, K = rows.shape
    N = weight.shape[0]
    if weight.shape[1] != K:
        raise ValueError(f"weight: K is {weight.shape[1]}, the rows have {K}")
    dev = rows.device
    _arg(weight.codes, torch.int8, "weight.codes", ((N + 15) // 16 * -(-K // 128) * 2048,), dev)
    _arg(weight.scales, torch.float32, "weight.scales", (N,), dev)
    y, yd = _out(y, y_dtype, "y", (M, N), rows)
    return M, N, K, y, yd


def channel_matmul(codes: torch.Tensor, scales: torch.Tensor, weight: ChannelWeight,
                   y: Optional[torch.Tensor] = None, y_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """moe_channel_matmul: [M, N] in bf16 (or y_dtype) from codes and scales of
    channel_quantize."""
    _matrix(codes, torch.int8, "codes")
    M, N, K, y, yd = _channel_operands(codes, weight, y, y_dtype)
    _arg(scales, torch.float32, "scales", (M,), codes.device)
    _launch("moe_channel_matmul", lib().moe_channel_matmul, codes.device.index,
            M, N, K, codes.data_ptr(), scales.data_ptr(), weight.codes.data_ptr(),
            weight.scales.data_ptr(), y.data_ptr(), yd)
    return y


@functools.lru_cache(maxsize=256)
def _channel_linear_bytes(max_rows: int, K: int) -> int:
    return int(lib().moe_channel_linear_workspace_size(max_rows, K))


def channel_linear_workspace(max_rows: int, K: int, device="cuda") -> torch.Tensor:
    n = _channel_linear_bytes(int(max_rows), int(K))
    if n == 0:
        raise ValueError(f"moe_channel_linear_workspace_size: invalid rows {max_rows} or K {K}")
    return torch.empty(n, dtype=torch.uint8, device=device)


def channel_linear(x: torch.Tensor, weight: ChannelWeight, y: Optional[torch.Tensor] = None,
                   y_dtype: Optional[torch.dtype] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_channel_linear: [M, N] in bf16 (or y_dtype) = x [M, K] quantised by rows,
    times the weight."""
    _matrix(x, torch.bfloat16, "x")
    M, N, K, y, yd = _channel_operands(x, weight, y, y_dtype)
    if ws is not None:
        _arg(ws, torch.uint8, "ws", getattr(ws, "shape", None), x.device)
    elif M > CHANNEL_FEW_ROWS:
        ws = channel_linear_workspace(M, K, x.device)
    _launch("moe_channel_linear", lib().moe_channel_linear, x.device.index,
            M, N, K, x.data_ptr(), weight.codes.data_ptr(), weight.scales.data_ptr(), y.data_ptr(), yd,
            _p(ws), 0 if ws is None else ws.numel())
    return y


# ---- products grouped by expert
def group_rows(ids: torch.Tensor, n_experts: int):
    """moe_group_rows: (offsets int32 [n_experts + 1], src int32 [R], inv int32 of ids'
    shape) of the R = ids.numel() rows that ids int32 (e.g. [T, k] of route) name:
    row i of the sorted rows is flat entry src[i], entry j is sorted row inv[j]
    (-1: an id outside [0, n_experts); src is 0 behind the last row there is)."""
    if not isinstance(ids, torch.Tensor):
        raise ValueError("ids: expected a tensor")
    _dev(ids, torch.int32, "ids")
    R, dev = ids.numel(), ids.device
    n = int(lib().moe_group_rows_workspace_size(int(n_experts), R))
    if n == 0:
        raise ValueError(f"moe_group_rows_workspace_size: invalid n_experts {n_experts} or rows {R}")
    offsets = torch.empty(n_experts + 1, dtype=torch.int32, device=dev)
    src = torch.zeros(R, dtype=torch.int32, device=dev)
    inv = torch.empty(ids.shape, dtype=torch.int32, device=dev)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _launch("moe_group_rows", lib().moe_group_rows, dev.index,
            R, n_experts, ids.data_ptr(), offsets.data_ptr(), src.data_ptr(), inv.data_ptr(), ws.data_ptr(), n)
    return offsets, src, inv


def _grouped_operands(rows: torch.Tensor, name: str, w: torch.Tensor, offsets: torch.Tensor, axis: int):
    """(R, E, N, K) of rows [R, w.shape[axis]] and w [E, N, K]."""
    R, width = _matrix(rows, torch.bfloat16, name).shape
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise ValueError("w: expected a [E, N, K] tensor")
    E, N, K = shape = w.shape
    _arg(w, torch.bfloat16, "w", shape, rows.device)
    if shape[axis] != width:
        raise ValueError(f"{name}: {width} columns, w is {tuple(shape)}")
    _arg(offsets, torch.int32, "offsets", (E + 1,), rows.device)
    return R, E, N, K


def grouped_matmul(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, y: Optional[torch.Tensor] = None,
                   y_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """moe_grouped_matmul: y [R, N] with y[r] = w[e] x[r] for the rows offsets[e] to
    offsets[e + 1] of expert e; x bf16 [R, K], w bf16 [E, N, K].  Rows before
    offsets[0] and behind offsets[E] stay as they are in a y that is given and are zero
    in a new one.  (With gradients: grouped_linear.)"""
    R, E, N, K = _grouped_operands(x, "x", w, offsets, 2)
    fresh = y is None
    y, yd = _out(y, y_dtype, "y", (R, N), x)
    _launch("moe_grouped_matmul", lib().moe_grouped_matmul, x.device.index,
            R, E, N, K, x.data_ptr(), w.data_ptr(), offsets.data_ptr(), y.data_ptr(), yd, 1 if fresh else 0)
    return y


def grouped_input_grad(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                       dx: Optional[torch.Tensor] = None, dx_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """moe_grouped_input_grad: dx [R, K] with dx[r] = dy[r] w[e]; dy bf16 [R, N], w bf16
    [E, N, K].  Rows before offsets[0] and behind offsets[E] as in grouped_matmul."""
    R, E, N, K = _grouped_operands(dy, "dy", w, offsets, 1)
    fresh = dx is None
    dx, yd = _out(dx, dx_dtype, "dx", (R, K), dy)
    _launch("moe_grouped_input_grad", lib().moe_grouped_input_grad, dy.device.index,
            R, E, N, K, dy.data_ptr(), w.data_ptr(), offsets.data_ptr(), dx.data_ptr(), yd, 1 if fresh else 0)
    return dx


@functools.lru_cache(maxsize=256)
def _weight_grad_bytes(R: int, E: int, N: int, K: int) -> int:
    return int(lib().moe_grouped_weight_grad_workspace_size(R, E, N, K))


def grouped_weight_grad(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor,
                        dw: Optional[torch.Tensor] = None, dw_dtype: Optional[torch.dtype] = None,
                        accumulate: bool = False, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_grouped_weight_grad: dw [E, N, K] with dw[e] = dy[rows of e]^T x[rows of e],
    in bf16 (or dw_dtype); with accumulate added to the fp32 dw given.  dy bf16
    [R, N], x bf16 [R, K].  ws: a uint8 workspace, allocated here where the sizes need
    one and none is given."""
    R, N = _matrix(dy, torch.bfloat16, "dy").shape
    dev = dy.device
    _arg(x, torch.bfloat16, "x", (R, _matrix(x, torch.bfloat16, "x").shape[1]), dev)
    K = x.shape[1]
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets: expected an int32 [E + 1] tensor")
    E = offsets.numel() - 1
    _arg(offsets, torch.int32, "offsets", (E + 1,), dev)
    if accumulate and dw is None:
        raise ValueError("accumulate needs the dw to add to")
    dw, yd = _out(dw, dw_dtype, "dw", (E, N, K), dy)
    if ws is not None:
        _arg(ws, torch.uint8, "ws", getattr(ws, "shape", None), dev)
    else:
        n = _weight_grad_bytes(R, E, N, K)
        if n > 256:
            ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _launch("moe_grouped_weight_grad", lib().moe_grouped_weight_grad, dev.index,
            R, E, N, K, dy.data_ptr(), x.data_ptr(), offsets.data_ptr(), dw.data_ptr(), yd, 1 if accumulate else 0,
            _p(ws), 0 if ws is None else ws.numel())
    return dw


class _GroupedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets):
        ctx.save_for_backward(x, w, offsets)
        return grouped_matmul(x, w, offsets)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        if dy.data_ptr() % 16:  # a part of another gradient, which may begin anywhere
            dy = dy.clone()
        dx = grouped_input_grad(dy, w, offsets) if ctx.needs_input_grad[0] else None
        dw = grouped_weight_grad(dy, x, offsets) if ctx.needs_input_grad[1] else None
        return dx, dw, None


def grouped_linear(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor) -> torch.Tensor:
    """grouped_matmul with gradients (torch autograd): bf16 y [R, N] of x bf16 [R, K] and
    w bf16 [E, N, K], dx and dw in bf16; rows of no expert have y and dx of zero, so that
    offsets may be those of some of the experts, off[lo:hi + 1].  The forward can be captured in a graph; a
    captured backward is to call grouped_input_grad and grouped_weight_grad themselves,
    since autograd's own bookkeeping of leaves does not belong in one."""
    return _GroupedLinear.apply(x, w, offsets)
