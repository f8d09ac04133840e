"""Thin Python binding of libtb_b200.so (include/tb.h).

Argument marshalling only: tensors are passed as raw device pointers with
the current CUDA stream of their device; every computation runs in the
library's kernels.  There is no host fallback: if the shared library is
missing or cannot be loaded, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib
import os

import torch

from decode_gemv_tb_b200.build import bind_tag

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libtb_b200.so")

TERNARY, INT2, INT3 = 0, 1, 2
TERNARY_B3 = 3  # the ternary grid, 5 codes per byte
MX4 = 4  # microscaled 4-bit floats: the expert layer and tb_mx4_*
F32, BF16 = 0, 1
MAX_LAYER_ITEMS = 16
FLAG_OVERLAP_PREVIOUS = 1
FLAG_TEST_STALL = 0x80000000  # test hook: the batch-1 kernel's waits give up (see include/tb.h)
NOALLOC_SCRATCH_BYTES = 4 << 20  # TB_NOALLOC_SCRATCH_BYTES

STATUS = {0: "TB_OK", 1: "TB_ERR_ARG", 2: "TB_ERR_SHAPE", 3: "TB_ERR_ALIGN", 4: "TB_ERR_UNSUPPORTED", 5: "TB_ERR_CUDA",
          6: "TB_ERR_TIMEOUT"}

# every entry point the header declares: (name, restype, argtypes)
_P, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
SIGNATURES = {
    "tb_version": (ctypes.c_int, []),
    "tb_status_string": (ctypes.c_char_p, [_I32]),
    "tb_packed_bytes": (_SZ, [_I32, _I64, _I64]),
    "tb_scale_bytes": (_SZ, [_I64, _I64]),
    "tb_scales_absmax": (_I32, [_P, _I32, _I64, _I64, _I32, _P, _P]),
    "tb_pack": (_I32, [_P, _I32, _I64, _I64, _I32, _P, _P, _P, _P]),
    "tb_unpack": (_I32, [_P, _I32, _I64, _I64, _P, _P]),
    "tb_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "tb_layer_workspace_bytes": (_SZ, [_P, _I32]),
    "tb_gemv": (_I32, [_P, _I32, _P, _P, _P, _I32, _I64, _I64, _P, _SZ, _P]),
    "tb_gemm": (_I32, [_P, _I32, _P, _P, _I64, _P, _I32, _I64, _I64, _I64, _I64, _P, _SZ, _P]),
    "tb_layer_gemv": (_I32, [_P, _I32, ctypes.c_uint, _P, _SZ, _P]),
    "tb_gemv_noalloc": (_I32, [_P, _I32, _P, _P, _P, _I32, _I64, _I64, _P]),
    "tb_wait_timeouts": (ctypes.c_uint, []),
    "tb_sync_status": (_I32, [_P]),
    "tb_gate_up_workspace_bytes": (_SZ, [_P, _P]),
    "tb_gate_up_silu": (_I32, [_P, _P, _P, ctypes.c_uint, _P, _SZ, _P]),
    "tb_mx4_code_bytes": (_SZ, [_I64, _I64]),
    "tb_mx4_scale_bytes": (_SZ, [_I64, _I64]),
    "tb_mx4_quantize": (_I32, [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _P]),
    "tb_mx4_dequantize": (_I32, [_P, _P, _I64, _I64, _P, _I32, _I64, _P]),
    "tb_moe_route": (_I32, [_P, _I64, _P, _I64, _I64, _I64, _I32, _I32, _P, _P, _P]),
    "tb_moe_workspace_bytes": (_SZ, [_P, _I64, _I32]),
    "tb_moe": (_I32, [_P, _P, _I64, _P, _P, _I64, _I32, _P, _I32, _I64, ctypes.c_uint, _P, _SZ, _P]),
    "tb_mx4_gemm": (_I32, [_P, _P, _P, _P, _P, _I32, _I64, _I64, _I64, _I64, ctypes.c_uint, _P]),
}


# entry points called by _tb_bind.so, and the text of their statuses, in the order that its init takes
BOUND = ("tb_mx4_quantize", "tb_mx4_dequantize", "tb_mx4_gemm", "tb_moe_route", "tb_moe", "tb_status_string")


class Linear(ctypes.Structure):
    """tb_linear_t"""
    _fields_ = [("packed", _P), ("scales", _P), ("x", _P), ("y", _P), ("N", _I64), ("K", _I64),
                ("grid", ctypes.c_int32), ("y_dtype", ctypes.c_int32)]


class MoE(ctypes.Structure):
    """tb_moe_t"""
    _fields_ = [("gate", _P), ("up", _P), ("down", _P), ("gate_scales", _P), ("up_scales", _P), ("down_scales", _P),
                ("gate_grid", ctypes.c_int32), ("up_grid", ctypes.c_int32), ("down_grid", ctypes.c_int32),
                ("E", ctypes.c_int32), ("H", _I64), ("I", _I64)]


class TBError(RuntimeError):
    pass


_lib = None
_bind = None  # _tb_bind.so, the calls that do not go through ctypes


class _NoBind:
    """In the place of _tb_bind.so where that cannot be loaded: its calls raise, the others do not need it."""

    def __init__(self, why: str):
        self._why = f"_tb_bind.so: {why}; run `python -m decode_gemv_tb_b200.build`"

    def __getattr__(self, name):
        raise TBError(self._why)


def _load_bind(lib: ctypes.CDLL):
    try:
        bind = importlib.import_module("decode_gemv_tb_b200._tb_bind")
    except ImportError as e:
        return _NoBind(str(e))
    built_for = getattr(bind, "built_for", "another version of this package")
    if built_for != bind_tag():
        return _NoBind(f"built for {built_for}, not for {bind_tag()}")
    bind.init(TBError, *(ctypes.cast(getattr(lib, name), _P).value for name in BOUND))
    return bind


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the shared library (raises if it is missing).  _tb_bind.so is loaded beside it where it can be; without it
    the 4-bit and expert-layer calls raise."""
    global _lib, _bind
    if _lib is None:
        if not os.path.exists(path):
            raise TBError(f"libtb_b200.so not built at {path}; run `python -m decode_gemv_tb_b200.build`")
        lib = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _bind, _lib = _load_bind(lib), lib
    return _lib


def _check(rc: int, what: str):
    if rc != 0:
        msg = load().tb_status_string(rc).decode()
        raise TBError(f"{what}: {STATUS.get(rc, rc)} ({msg})")


def _dev(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise TBError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise TBError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _wdtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TBError(f"weights must be float32 or bfloat16, got {t.dtype}")


def _ydtype(dt) -> int:
    if dt == torch.float32:
        return F32
    if dt == torch.bfloat16:
        return BF16
    raise TBError(f"output dtype must be float32 or bfloat16, got {dt}")


def _bits(t: torch.Tensor, name: str) -> int:
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TBError(f"{name} must hold bf16 bit patterns")
    return _dev(t, name)


# ---- sizes -----------------------------------------------------------------

def wait_timeouts() -> int:
    """Bounded device waits that gave up since the last call (synchronizes)."""
    return int(load().tb_wait_timeouts())


def sync_status(stream: int | None = None) -> int:
    """tb_sync_status on the current stream: 0 (TB_OK), 6 (TB_ERR_TIMEOUT) or 5."""
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    return int(load().tb_sync_status(stream))


def version() -> int:
    return load().tb_version()


def packed_bytes(grid: int, N: int, K: int) -> int:
    return int(load().tb_packed_bytes(grid, N, K))


def scale_bytes(N: int, K: int) -> int:
    return int(load().tb_scale_bytes(N, K))


# ---- entry points -----------------------------------------------------------

def tb_scales_absmax(W: torch.Tensor, grid: int, scales: torch.Tensor | None = None) -> torch.Tensor:
    N, K = W.shape
    if scales is None:
        scales = torch.empty((N, K // 128), dtype=torch.bfloat16, device=W.device)
    _check(load().tb_scales_absmax(_dev(W, "W"), _wdtype(W), N, K, grid, _bits(scales, "scales"), _stream(W)),
           "tb_scales_absmax")
    return scales


def tb_pack(W: torch.Tensor, grid: int, scales: torch.Tensor, packed: torch.Tensor | None = None,
            bad_count: torch.Tensor | None = None) -> torch.Tensor:
    N, K = W.shape
    if packed is None:
        packed = torch.empty(packed_bytes(grid, N, K), dtype=torch.uint8, device=W.device)
    bc = 0 if bad_count is None else _dev(bad_count, "bad_count")
    _check(load().tb_pack(_dev(W, "W"), _wdtype(W), N, K, grid, _bits(scales, "scales"), _dev(packed, "packed"),
                          bc, _stream(W)), "tb_pack")
    return packed


def tb_unpack(packed: torch.Tensor, grid: int, N: int, K: int, codes: torch.Tensor | None = None) -> torch.Tensor:
    if codes is None:
        codes = torch.empty((N, K), dtype=torch.int8, device=packed.device)
    _check(load().tb_unpack(_dev(packed, "packed"), grid, N, K, _dev(codes, "codes"), _stream(packed)), "tb_unpack")
    return codes


def workspace_bytes(M: int, N: int, K: int) -> int:
    return int(load().tb_workspace_bytes(M, N, K))


def workspace(nbytes: int, device) -> torch.Tensor:
    """Caller-owned scratch for the products (256-byte aligned), zero-filled
    once as the batch-1 kernel's counters require (calls leave it zero)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def tb_gemv(packed: torch.Tensor, grid: int, scales: torch.Tensor, x: torch.Tensor, N: int, K: int,
            y: torch.Tensor | None = None, out_dtype=torch.float32, ws: torch.Tensor | None = None) -> torch.Tensor:
    if y is None:
        y = torch.empty(N, dtype=out_dtype, device=x.device)
    if ws is None:
        ws = workspace(workspace_bytes(1, N, K), x.device)
    _check(load().tb_gemv(_dev(packed, "packed"), grid, _bits(scales, "scales"), _bits(x, "x"), _dev(y, "y"),
                          _ydtype(y.dtype), N, K, _dev(ws, "workspace"), ws.numel(), _stream(x)), "tb_gemv")
    return y


def tb_gemv_noalloc(packed: torch.Tensor, grid: int, scales: torch.Tensor, x: torch.Tensor, N: int, K: int,
                    y: torch.Tensor) -> torch.Tensor:
    """tb_gemv over the library's fixed device scratch: no workspace, and
    the caller provides y, so the call itself allocates nothing."""
    _check(load().tb_gemv_noalloc(_dev(packed, "packed"), grid, _bits(scales, "scales"), _bits(x, "x"),
                                  _dev(y, "y"), _ydtype(y.dtype), N, K, _stream(x)), "tb_gemv_noalloc")
    return y


def tb_gemm(packed: torch.Tensor, grid: int, scales: torch.Tensor, X: torch.Tensor, N: int, K: int,
            Y: torch.Tensor | None = None, out_dtype=torch.float32, ws: torch.Tensor | None = None) -> torch.Tensor:
    M = X.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=out_dtype, device=X.device)
    if ws is None:
        ws = workspace(workspace_bytes(M, N, K), X.device)
    _check(load().tb_gemm(_dev(packed, "packed"), grid, _bits(scales, "scales"), _bits(X, "X"), X.stride(0),
                          _dev(Y, "Y"), _ydtype(Y.dtype), Y.stride(0), M, N, K, _dev(ws, "workspace"), ws.numel(),
                          _stream(X)), "tb_gemm")
    return Y


def linear_items(items) -> ctypes.Array:
    """Build a tb_linear_t array from (packed, grid, scales, x, y, N, K)."""
    arr = (Linear * len(items))()
    for i, (packed, grid, scales, x, y, N, K) in enumerate(items):
        arr[i] = Linear(_dev(packed, "packed"), _bits(scales, "scales"), _bits(x, "x"), _dev(y, "y"), N, K, grid,
                        _ydtype(y.dtype))
    return arr


def layer_workspace_bytes(arr: ctypes.Array) -> int:
    return int(load().tb_layer_workspace_bytes(ctypes.cast(arr, ctypes.c_void_p), len(arr)))


def tb_layer_gemv(items, ws: torch.Tensor | None = None, flags: int = 0, stream: int | None = None) -> None:
    """items: list of (packed, grid, scales, x, y, N, K), or a prebuilt
    linear_items() array (reused without re-marshalling)."""
    arr = items if isinstance(items, ctypes.Array) else linear_items(items)
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    if ws is None:
        ws = workspace(layer_workspace_bytes(arr), torch.device("cuda", torch.cuda.current_device()))
    _check(load().tb_layer_gemv(ctypes.cast(arr, ctypes.c_void_p), len(arr), flags, ws.data_ptr(), ws.numel(),
                                stream), "tb_layer_gemv")


def gate_up_workspace_bytes(gate, up) -> int:
    """Workspace bytes of tb_gate_up_silu for gate, up: (packed, grid, scales, x, y, N, K)."""
    arr = linear_items([gate, up])
    return int(load().tb_gate_up_workspace_bytes(ctypes.cast(ctypes.byref(arr, 0), ctypes.c_void_p),
                                                  ctypes.cast(ctypes.byref(arr, ctypes.sizeof(Linear)), ctypes.c_void_p)))


def tb_gate_up_silu(gate, up, h: torch.Tensor, ws: torch.Tensor | None = None, flags: int = 0,
                    stream: int | None = None) -> torch.Tensor:
    """gate, up: (packed, grid, scales, x, y, N, K) of equal N and K; writes
    their y and h = bf16(silu(gate) * up) ([N] bf16)."""
    arr = linear_items([gate, up])
    if h.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TBError("h must hold bf16")
    g_ptr = ctypes.cast(ctypes.byref(arr, 0), ctypes.c_void_p)
    u_ptr = ctypes.cast(ctypes.byref(arr, ctypes.sizeof(Linear)), ctypes.c_void_p)
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    if ws is None:
        ws = workspace(load().tb_gate_up_workspace_bytes(g_ptr, u_ptr), torch.device("cuda", torch.cuda.current_device()))
    _check(load().tb_gate_up_silu(g_ptr, u_ptr, _dev(h, "h"), flags, ws.data_ptr(), ws.numel(), stream),
           "tb_gate_up_silu")
    return h


# ---- microscaled 4-bit floats -------------------------------------------------

def _same_device(first: torch.Tensor, *rest) -> int:
    """The library launches on the current device: every tensor has to live there.  Returns its index."""
    dev = first.get_device()  # -1: not a CUDA tensor
    if dev < 0:
        raise TBError("tensors must be CUDA tensors")
    if dev != torch._C._cuda_getDevice():
        raise TBError(f"tensors on cuda:{dev}, but the current device is cuda:{torch.cuda.current_device()}")
    for t in rest:
        if t is not None and t.get_device() != dev:
            raise TBError(f"tensors on different devices: cuda:{dev} and {t.device}")
    return dev


def _allocating(stream: int | None):
    """What is allocated for a call on `stream` belongs to that stream: its memory is not one that other work still uses,
    and is not given to other work while the call runs."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(torch.cuda.ExternalStream(stream))


def _bytes(t: torch.Tensor, name: str, need: int) -> int:
    if t.dtype != torch.uint8 or t.numel() < need:
        raise TBError(f"{name} must hold at least {need} bytes as uint8")
    if not t.is_contiguous():
        raise TBError(f"{name} must be contiguous")
    return t.data_ptr()


def mx4_code_bytes(N: int, K: int) -> int:
    return int(load().tb_mx4_code_bytes(N, K))


def mx4_scale_bytes(N: int, K: int) -> int:
    return int(load().tb_mx4_scale_bytes(N, K))


def _mx4_sizes(N: int, K: int):
    if N < 1 or K < 32 or K % 32:
        raise TBError(f"MX4 needs N >= 1 and K a positive multiple of 32, got {N} x {K}")
    return N * (K // 2), 512 * (-(-N // 128)) * (-(-K // 128))


def tb_mx4_quantize(W: torch.Tensor, codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                    bad_count: torch.Tensor | None = None, stream: int | None = None):
    """W [N][K] (rows may be strided) -> codes [N][K/2] uint8 and the scale tiles (uint8)."""
    load()
    if codes is None or scales is None:
        N, K = W.shape
        _, ns = _mx4_sizes(N, K)
        with _allocating(stream):
            if codes is None:
                codes = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device)
            if scales is None:
                scales = torch.empty(ns, dtype=torch.uint8, device=W.device)
    _bind.mx4_quantize(W, codes, scales, bad_count, stream)
    return codes, scales


def tb_mx4_dequantize(codes: torch.Tensor, scales: torch.Tensor, N: int, K: int, W: torch.Tensor | None = None,
                      out_dtype=torch.bfloat16, stream: int | None = None) -> torch.Tensor:
    """The values that MX4 codes stand for, [N][K] fp32 or bf16."""
    load()
    if W is None:
        _mx4_sizes(N, K)
        with _allocating(stream):
            W = torch.empty((N, K), dtype=out_dtype, device=codes.device)
    _bind.mx4_dequantize(codes, scales, N, K, W, stream)
    return W


def tb_mx4_gemm(w_codes: torch.Tensor, w_scales: torch.Tensor, x_codes: torch.Tensor, x_scales: torch.Tensor,
                M: int, N: int, K: int, Y: torch.Tensor | None = None, out_dtype=torch.float32, flags: int = 0,
                stream: int | None = None) -> torch.Tensor:
    """Y [M][N] = X W^T of two MX4 tensors (N rows of W, M rows of X, K columns)."""
    load()
    if Y is None:
        with _allocating(stream):
            Y = torch.empty((M, N), dtype=out_dtype, device=x_codes.device)
    _bind.mx4_gemm(w_codes, w_scales, x_codes, x_scales, M, N, K, Y, flags, stream)
    return Y


# ---- mixture-of-experts layer ---------------------------------------------------

MOE_MAX_TOKENS, MOE_MAX_TOPK, MOE_MAX_EXPERTS = 64, 16, 512


def tb_moe_route(x: torch.Tensor, router: torch.Tensor, k: int, renormalize: bool = True,
                 ids: torch.Tensor | None = None, weights: torch.Tensor | None = None, stream: int | None = None):
    """x [T][H] (rows may be strided), router [E][H], both bf16 -> the k best experts of every token, ids [T][k]
    int32, and their softmax weights [T][k] fp32."""
    load()
    if ids is None or weights is None:
        with _allocating(stream):
            if ids is None:
                ids = torch.empty((x.shape[0], k), dtype=torch.int32, device=x.device)
            if weights is None:
                weights = torch.empty((x.shape[0], k), dtype=torch.float32, device=x.device)
    _bind.moe_route(x, router, k, renormalize, ids, weights, stream)
    return ids, weights


class MoELayer:
    """A tb_moe_t and the tensors it points to."""

    def __init__(self, desc: MoE, tensors, device):
        self.desc, self.tensors, self.device, self.H = desc, tensors, device, desc.H
        self.ptr = ctypes.addressof(desc)


def moe_layer(gate, up, down, E: int, H: int, I: int) -> MoELayer:
    """Describe E stacked experts.  gate, up, down: (packed, scales, grid) of the [E*I][H], [E*I][H] and [E*H][I]
    matrices, as tb_pack (or tb_mx4_quantize) leaves them."""
    mats = []
    for name, (packed, scales, grid), (N, K) in zip(("gate", "up", "down"), (gate, up, down),
                                                    ((E * I, H), (E * I, H), (E * H, I))):
        _same_device(gate[0], packed, scales)
        if grid == MX4:
            nc, ns = _mx4_sizes(N, K)
            mats.append((_bytes(packed, name, nc), _bytes(scales, f"{name} scales", ns)))
        else:
            if grid != TERNARY_B3 and scales.numel() < N * (K // 128):
                raise TBError(f"{name} scales must hold {N} x {K // 128} values")
            mats.append((_bytes(packed, name, packed_bytes(grid, N, K)), _bits(scales, f"{name} scales")))
    desc = MoE(*(m[0] for m in mats), *(m[1] for m in mats), gate[2], up[2], down[2], E, H, I)
    return MoELayer(desc, (gate, up, down), gate[0].get_device())


def moe_workspace_bytes(layer: MoELayer, T: int, k: int) -> int:
    return int(load().tb_moe_workspace_bytes(layer.ptr, T, k))


def tb_moe(layer: MoELayer, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, y: torch.Tensor | None = None,
           out_dtype=torch.float32, ws: torch.Tensor | None = None, flags: int = 0, stream: int | None = None) -> torch.Tensor:
    """y [T][H] = the routed experts' MLP of x [T][H] (bf16, rows may be strided), summed with the weights."""
    load()
    if y is None or ws is None:
        with _allocating(stream):
            if y is None:
                y = torch.empty((ids.shape[0], layer.H), dtype=out_dtype, device=x.device)
            if ws is None:
                # data only: nothing of it has to be zero, and no other call shares it
                ws = torch.empty(moe_workspace_bytes(layer, *ids.shape), dtype=torch.uint8, device=x.device)
    _bind.moe(layer.ptr, layer.H, layer.device, x, ids, weights, y, ws, flags, stream)
    return y
