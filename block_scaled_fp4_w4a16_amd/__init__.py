"""Python binding of the fp4w4a16 C ABI (block-scaled 4-bit weights x bf16 activations on gfx950).

Argument marshalling only: every function below checks tensor devices, dtypes and sizes,
passes raw device pointers and the current HIP stream to the C entry point of the same
name in libfp4w4a16.so, and raises RuntimeError on a negative status (the MXFP4 operators
do so in _fp4bind.so, the binding's native half). All computation runs in the library's HIP
kernels; there is no fallback path. Importing this package without the C library fails loudly;
without the native half, the MXFP4 calls do.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp4w4a16.so")

FORMATS = {"nvfp4": 1, "rocmfp4_dual": 2, "rocmfp4_fast": 3, "q4_0": 4}
BLOCK_BYTES = {"rocmfp4_dual": 18, "rocmfp4_fast": 17, "q4_0": 18}
GEMV_MAX_M = 16

_c = ctypes.c_int
_i64 = ctypes.c_int64
_p = ctypes.c_void_p
_f = ctypes.c_float

GEMV_MAX_ITEMS = 32


class GemvItem(ctypes.Structure):
    """Mirror of `fp4_gemv_item` (one matrix of a w4a16_gemv_batched call)."""
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("x_bf16", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("global_scale", ctypes.c_float)]


class Mx(ctypes.Structure):
    """Mirror of `fp4_mx` (an MXFP4 operand in device memory)."""
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("ldq", ctypes.c_int64), ("lds", ctypes.c_int64)]


_mx = ctypes.POINTER(Mx)
_SIGS = {
    "fp4_abi_version": (_c, []),
    "fp4_status_string": (ctypes.c_char_p, [_c]),
    "fp4_layout_bytes": (_c, [_c, _i64, _i64, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]),
    "fp4_pack_layout": (_c, [_c, _i64, _i64, _p, _p, _p, _p, _c, _p]),
    "w4a16_gemv": (_c, [_c, _i64, _i64, _i64, _p, _p, _f, _p, _p, _p]),
    "w4a16_gemv_batched": (_c, [_c, _i64, _c, ctypes.POINTER(GemvItem), _p]),
    "w4a16_gemm": (_c, [_c, _i64, _i64, _i64, _p, _p, _f, _p, _p, _p]),
    "w4a16_midm": (_c, [_c, _i64, _i64, _i64, _p, _p, _f, _p, _p, _p]),
    "w4a16_matmul": (_c, [_c, _i64, _i64, _i64, _p, _p, _f, _p, _p, _p]),
    "w4a16_gemm_ws": (_c, [_c, _i64, _i64, _i64, _p, _p, _f, _p, _p, _p, ctypes.c_size_t, _p]),
    "w4a16_matmul_ws": (_c, [_c, _i64, _i64, _i64, _p, _p, _f, _p, _p, _p, ctypes.c_size_t, _p]),
    "w4a16_gemm_workspace_bytes": (_i64, [_c, _i64, _i64, _i64]),
    "w4a16_matmul_workspace_bytes": (_i64, [_c, _i64, _i64, _i64]),
    "w4a16_gemm_noalloc": (_c, [_c, _i64, _i64, _i64, _p, _p, _f, _p, _p, _p]),
    "fp4_dequant_f32": (_c, [_c, _i64, _i64, _p, _p, _f, _p, _p]),
    "fp4_quantize_nvfp4": (_c, [_i64, _i64, _p, _p, _p, _p, _p]),
    "fp4_quantize_rocmfp4": (_c, [_c, _i64, _i64, _p, _p, _p, _p]),
    "fp4_quantize_q4_0": (_c, [_i64, _i64, _p, _p, _p]),
    "fp4_quantize_mxfp4": (_c, [_c, _i64, _i64, _p, _i64, _mx, _mx, _p]),
    "fp4_dequant_mxfp4": (_c, [_c, _i64, _i64, _mx, _p, _i64, _p]),
    "w4a4_matmul": (_c, [_c, _i64, _i64, _i64, _mx, _mx, _p, _i64, _p, ctypes.c_size_t, _p]),
    "w4a4_matmul_workspace_bytes": (_i64, [_i64, _i64, _i64]),
    "w4a4_linear": (_c, [_c, _c, _i64, _i64, _i64, _p, _i64, _mx, _p, _i64, _p, ctypes.c_size_t, _p]),
    "w4a4_linear_workspace_bytes": (_i64, [_i64, _i64, _i64]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with block_scaled_fp4_w4a16_amd/build.py "
                              "(or __graft_entry__.build())")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(h, name)
            fn.restype = res
            fn.argtypes = args
        _lib = h
    return _lib


lib()  # fail at import time when the HIP library is absent

class _MissingNative:
    """Stands for _fp4bind.so where it cannot be loaded: the W4A16 calls need only the C library and work without it,
    each MXFP4 call raises."""

    def __init__(self, cause: ImportError):
        self._cause = cause

    def __getattr__(self, name):
        if name.startswith("__"):
            raise AttributeError(name)
        raise ImportError("the MXFP4 operators need _fp4bind.so, built for the installed torch: build it with "
                          f"block_scaled_fp4_w4a16_amd/build.py (or __graft_entry__.build()); {self._cause}") from self._cause


try:
    from . import _fp4bind as _native  # noqa: E402  (links libfp4w4a16.so, loaded above)
except ImportError as _cause:  # not built, or built for another torch
    _native = _MissingNative(_cause)


def _fmt(fmt) -> int:
    if isinstance(fmt, str):
        if fmt not in FORMATS:
            raise ValueError(f"unknown format {fmt!r}; expected one of {sorted(FORMATS)}")
        return FORMATS[fmt]
    return int(fmt)


def _check(rc: int, what: str):
    if rc != 0:
        raise RuntimeError(f"{what}: {lib().fp4_status_string(rc).decode()} (status {rc})")


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError("tensors must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def _device(*ts) -> torch.device:
    """The one GPU that every given tensor (None entries skipped) lives on; the call runs there."""
    devs = {t.device for t in ts if isinstance(t, torch.Tensor)}
    if len(devs) != 1:
        raise ValueError(f"tensors must all live on one GPU (got {sorted(str(d) for d in devs)})")
    d = devs.pop()
    if d.type != "cuda":
        raise ValueError("tensors must live on the GPU")
    return d


@functools.lru_cache(maxsize=4096)
def _plane_bytes(f: int, N: int, K: int) -> tuple[int, int]:
    q = ctypes.c_size_t()
    s = ctypes.c_size_t()
    _check(lib().fp4_layout_bytes(f, N, K, ctypes.byref(q), ctypes.byref(s)), "fp4_layout_bytes")
    return q.value, s.value


def _check_planes(f: int, N: int, K: int, q, s):
    qb, sb = _plane_bytes(f, N, K)
    if _nbytes(q) < qb or _nbytes(s) < sb:
        raise ValueError(f"packed planes too small for N={N} K={K}: need {qb} + {sb} bytes, "
                         f"got {_nbytes(q)} + {_nbytes(s)}")


def fp4_abi_version() -> int:
    return lib().fp4_abi_version()


def fp4_status_string(status: int) -> str:
    return lib().fp4_status_string(status).decode()


def fp4_layout_bytes(fmt, N: int, K: int) -> tuple[int, int]:
    q = ctypes.c_size_t()
    s = ctypes.c_size_t()
    _check(lib().fp4_layout_bytes(_fmt(fmt), N, K, ctypes.byref(q), ctypes.byref(s)), "fp4_layout_bytes")
    return q.value, s.value


def fp4_pack_layout(fmt, N, K, src_q, src_s, dst_q, dst_s, validate=False, stream=None):
    """Canonical bytes -> kernel layout. validate=True first checks every scale code on the device
    (waits for the stream) and raises RuntimeError with the library's FP4_ERR_INVALID_SCALE status,
    leaving dst_q / dst_s untouched, if one is NaN (or, for Q4_0, not finite)."""
    f = _fmt(fmt)
    dev = _device(src_q, src_s, dst_q, dst_s)
    if N > 0 and K > 0 and K % 16 == 0:
        if f == 1:
            need = (N * K // 2, N * K // 16)
            if _nbytes(src_q) < need[0] or (src_s is not None and _nbytes(src_s) < need[1]):
                raise ValueError(f"canonical NVFP4 planes too small: need {need[0]} + {need[1]} bytes")
        elif K % 32 == 0 and f in (2, 3, 4):
            need = N * (K // 32) * {2: 18, 3: 17, 4: 18}[f]
            if _nbytes(src_q) < need:
                raise ValueError(f"canonical blocks too small: need {need} bytes, got {_nbytes(src_q)}")
        if f in (1, 2, 3, 4) and (f == 1 or K % 32 == 0):
            _check_planes(f, N, K, dst_q, dst_s)
    with torch.cuda.device(dev):
        _check(lib().fp4_pack_layout(f, N, K, _ptr(src_q), _ptr(src_s), _ptr(dst_q), _ptr(dst_s), int(bool(validate)),
                                     _stream(stream)), "fp4_pack_layout")


def _product(name, fmt, M, N, K, q, s, global_scale, x, y, stream):
    if x.dtype != torch.bfloat16 or y.dtype != torch.float32:
        raise TypeError("x must be bfloat16 and y float32")
    if x.numel() < M * K or y.numel() < M * N:
        raise ValueError("x or y is smaller than M x K / M x N")
    f = _fmt(fmt)
    dev = _device(q, s, x, y)
    if M > 0 and N > 0 and K > 0:
        _check_planes(f, N, K, q, s)
    with torch.cuda.device(dev):
        _check(getattr(lib(), name)(f, M, N, K, _ptr(q), _ptr(s), float(global_scale), _ptr(x), _ptr(y),
                                    _stream(stream)), name)


def w4a16_gemv(fmt, M, N, K, q, s, global_scale, x, y, stream=None):
    _product("w4a16_gemv", fmt, M, N, K, q, s, global_scale, x, y, stream)


def w4a16_gemv_batched(fmt, M, items, stream=None):
    """items: sequence of (q, s, global_scale, x, y, N, K), one per matrix; all share fmt and M."""
    arr = (GemvItem * max(1, len(items)))()
    f = _fmt(fmt)
    tensors = []
    for i, (q, s, g, x, y, n, k) in enumerate(items):
        if x.dtype != torch.bfloat16 or y.dtype != torch.float32:
            raise TypeError("x must be bfloat16 and y float32")
        if x.numel() < M * k or y.numel() < M * n:
            raise ValueError("x or y is smaller than M x K / M x N")
        if M > 0 and n > 0 and k > 0:
            _check_planes(f, n, k, q, s)
        tensors += [q, s, x, y]
        arr[i] = GemvItem(_ptr(q), _ptr(s), _ptr(x), _ptr(y), n, k, float(g))
    with torch.cuda.device(_device(*tensors) if tensors else torch.cuda.current_device()):
        _check(lib().w4a16_gemv_batched(f, M, len(items), arr, _stream(stream)), "w4a16_gemv_batched")


def _workspace_bytes(name, fmt, M, N, K, device=None) -> int:
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        n = int(getattr(lib(), name)(_fmt(fmt), M, N, K))
    _check(n if n < 0 else 0, name)
    return n


def w4a16_gemm_workspace_bytes(fmt, M, N, K, device=None) -> int:
    """Workspace bytes w4a16_gemm_ws would use for this shape on `device` (default: the current one)."""
    return _workspace_bytes("w4a16_gemm_workspace_bytes", fmt, M, N, K, device)


def w4a16_matmul_workspace_bytes(fmt, M, N, K, device=None) -> int:
    """Workspace bytes w4a16_matmul_ws can use for this shape on `device` (0: it takes none)."""
    return _workspace_bytes("w4a16_matmul_workspace_bytes", fmt, M, N, K, device)


def _product_ws(name, fmt, M, N, K, q, s, global_scale, x, y, stream, workspace):
    """A product entry point that takes a workspace: `workspace` (a uint8 CUDA tensor) or, by default, one
    of the size the library asks for, allocated here from torch's caching allocator on the launch stream."""
    if x.dtype != torch.bfloat16 or y.dtype != torch.float32:
        raise TypeError("x must be bfloat16 and y float32")
    if x.numel() < M * K or y.numel() < M * N:
        raise ValueError("x or y is smaller than M x K / M x N")
    f = _fmt(fmt)
    dev = _device(q, s, x, y)
    if M > 0 and N > 0 and K > 0:
        _check_planes(f, N, K, q, s)
    with torch.cuda.device(dev):
        st = _stream(stream)
        if workspace is None and M > 0:
            query = "w4a16_gemm_workspace_bytes" if name == "w4a16_gemm_ws" else "w4a16_matmul_workspace_bytes"
            nbytes = _workspace_bytes(query, f, M, N, K, dev)
            if nbytes > 0:
                workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
                if stream is not None:
                    # the kernels run on `stream`, not necessarily the one the allocator recorded
                    ext = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(st)
                    workspace.record_stream(ext)
        ws_ptr, ws_bytes = (None, 0) if workspace is None else (_ptr(workspace), _nbytes(workspace))
        _check(getattr(lib(), name)(f, M, N, K, _ptr(q), _ptr(s), float(global_scale), _ptr(x), _ptr(y), ws_ptr,
                                    ws_bytes, st), name)


def w4a16_gemm(fmt, M, N, K, q, s, global_scale, x, y, stream=None, workspace=None):
    """The prefill product through w4a16_gemm_ws (K parts in a workspace where the launch rules split K)."""
    _product_ws("w4a16_gemm_ws", fmt, M, N, K, q, s, global_scale, x, y, stream, workspace)


def w4a16_gemm_noworkspace(fmt, M, N, K, q, s, global_scale, x, y, stream=None):
    """The C entry point w4a16_gemm itself (no workspace: at most the two-part atomic split)."""
    _product("w4a16_gemm", fmt, M, N, K, q, s, global_scale, x, y, stream)


def w4a16_gemm_noalloc(fmt, M, N, K, q, s, global_scale, x, y, stream=None):
    _product("w4a16_gemm_noalloc", fmt, M, N, K, q, s, global_scale, x, y, stream)


def w4a16_midm(fmt, M, N, K, q, s, global_scale, x, y, stream=None):
    _product("w4a16_midm", fmt, M, N, K, q, s, global_scale, x, y, stream)


def w4a16_matmul(fmt, M, N, K, q, s, global_scale, x, y, stream=None, workspace=None):
    """Dispatch on M through w4a16_matmul_ws (the prefill path with a workspace)."""
    _product_ws("w4a16_matmul_ws", fmt, M, N, K, q, s, global_scale, x, y, stream, workspace)


def fp4_dequant_f32(fmt, N, K, q, s, global_scale, w, stream=None):
    if w.dtype != torch.float32 or w.numel() < N * K:
        raise ValueError("w must be float32 with N x K elements")
    f = _fmt(fmt)
    dev = _device(q, s, w)
    if N > 0 and K > 0:
        _check_planes(f, N, K, q, s)
    with torch.cuda.device(dev):
        _check(lib().fp4_dequant_f32(f, N, K, _ptr(q), _ptr(s), float(global_scale), _ptr(w), _stream(stream)),
               "fp4_dequant_f32")


def fp4_quantize_nvfp4(N, K, w, wq, ws, g_out, stream=None):
    if w.dtype != torch.float32 or g_out.dtype != torch.float32:
        raise TypeError("w and g_out must be float32")
    if w.numel() < N * K or wq.numel() < N * K // 2 or ws.numel() < N * K // 16 or g_out.numel() < 1:
        raise ValueError("buffer too small")
    with torch.cuda.device(_device(w, wq, ws, g_out)):
        _check(lib().fp4_quantize_nvfp4(N, K, _ptr(w), _ptr(wq), _ptr(ws), _ptr(g_out), _stream(stream)),
               "fp4_quantize_nvfp4")


def fp4_quantize_rocmfp4(fmt, N, K, w, importance, blocks, stream=None):
    if w.dtype != torch.float32 or (importance is not None and importance.dtype != torch.float32):
        raise TypeError("w and importance must be float32")
    f = _fmt(fmt)
    bb = 18 if f == 2 else 17
    if w.numel() < N * K or blocks.numel() < N * (K // 32) * bb:
        raise ValueError("buffer too small")
    with torch.cuda.device(_device(w, importance, blocks)):
        _check(lib().fp4_quantize_rocmfp4(f, N, K, _ptr(w), _ptr(importance), _ptr(blocks), _stream(stream)),
               "fp4_quantize_rocmfp4")


def fp4_quantize_q4_0(N, K, w, blocks, stream=None):
    if w.dtype != torch.float32:
        raise TypeError("w must be float32")
    if w.numel() < N * K or blocks.numel() < N * (K // 32) * 18:
        raise ValueError("buffer too small")
    with torch.cuda.device(_device(w, blocks)):
        _check(lib().fp4_quantize_q4_0(N, K, _ptr(w), _ptr(blocks), _stream(stream)), "fp4_quantize_q4_0")


# ----------------------------------------------------------------------------------------------
# Convenience: a packed weight in kernel layout (allocation through torch, compute in the library)
# ----------------------------------------------------------------------------------------------

@dataclass
class PackedWeight:
    fmt: str
    N: int
    K: int
    q: torch.Tensor          # nibble plane (uint8)
    s: torch.Tensor          # scale plane (uint8)
    global_scale: float

    @staticmethod
    def empty(fmt: str, N: int, K: int, global_scale: float = 1.0, device="cuda") -> "PackedWeight":
        qb, sb = fp4_layout_bytes(fmt, N, K)
        return PackedWeight(fmt, N, K, torch.empty(qb, dtype=torch.uint8, device=device),
                            torch.empty(sb, dtype=torch.uint8, device=device), float(global_scale))

    @staticmethod
    def from_canonical(fmt: str, N: int, K: int, src_q: torch.Tensor, src_s: torch.Tensor | None,
                       global_scale: float = 1.0, stream=None, validate: bool = False) -> "PackedWeight":
        pw = PackedWeight.empty(fmt, N, K, global_scale, device=src_q.device)
        fp4_pack_layout(fmt, N, K, src_q, src_s, pw.q, pw.s, validate, stream)
        return pw

    @staticmethod
    def quantize(fmt: str, w: torch.Tensor, importance: torch.Tensor | None = None, stream=None) -> "PackedWeight":
        """Pack fp32 weights [N, K] on the GPU with the device packer, then repack to kernel layout."""
        N, K = w.shape
        w = w.contiguous()
        if fmt == "nvfp4":
            wq = torch.empty(N * K // 2, dtype=torch.uint8, device=w.device)
            ws = torch.empty(N * K // 16, dtype=torch.uint8, device=w.device)
            g = torch.empty(1, dtype=torch.float32, device=w.device)
            fp4_quantize_nvfp4(N, K, w, wq, ws, g, stream)
            gs = float(g.item())
            return PackedWeight.from_canonical(fmt, N, K, wq, ws, gs, stream=stream)
        blocks = torch.empty(N * (K // 32) * BLOCK_BYTES[fmt], dtype=torch.uint8, device=w.device)
        if fmt == "q4_0":
            if importance is not None:
                raise ValueError("the Q4_0 packer takes no importance")
            fp4_quantize_q4_0(N, K, w, blocks, stream)
        else:
            fp4_quantize_rocmfp4(fmt, N, K, w, importance, blocks, stream)
        return PackedWeight.from_canonical(fmt, N, K, blocks, None, 1.0, stream=stream)

    def matmul(self, x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """x W^T [M, N]; outside autograd: the result has no gradient, whether or not x requires one."""
        M = x.shape[0]
        if x.shape[-1] != self.K:
            raise ValueError("x's last dimension must be K")
        if out is None:
            out = torch.empty(M, self.N, dtype=torch.float32, device=x.device)
        w4a16_matmul(self.fmt, M, self.N, self.K, self.q, self.s, self.global_scale, x.contiguous(), out, stream)
        return out

    def dequant(self, stream=None) -> torch.Tensor:
        w = torch.empty(self.N, self.K, dtype=torch.float32, device=self.q.device)
        fp4_dequant_f32(self.fmt, self.N, self.K, self.q, self.s, self.global_scale, w, stream)
        return w


# ----------------------------------------------------------------------------------------------
# MXFP4 on both sides (W4A4): quantisation, products, a trainable linear layer. torch.jit.trace and make_fx would record
# the allocations without the kernels: every call refuses to be traced.
# ----------------------------------------------------------------------------------------------

def fp4_quantize_mxfp4(M, K, x, q=None, s=None, qt=None, st=None, stream=None):
    """x [M, K] (float32, bfloat16 or float16; rows may be strided) -> MXFP4 along its rows into q [M, 16 ceil(K/32)] and
    s [M, ceil(K/32)], and / or along its columns into qt [K, 16 ceil(M/32)] and st [K, ceil(M/32)] (the transposed
    operand). One of the two pairs may be None. Rows of the scales lie a multiple of 4 bytes apart, and the bytes of s and
    of st between a row's last scale and the next multiple of 4 are written as zeros."""
    _native.quantize(M, K, x, q, s, qt, st, stream)


def fp4_dequant_mxfp4(M, K, q, s, out, stream=None):
    """The values of an MXFP4 operand into out [M, K] (float32 or bfloat16; rows may be strided)."""
    _native.dequant(M, K, q, s, out, stream)


def _mx_workspace_bytes(name, M, N, K, device) -> int:
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        n = int(getattr(lib(), name)(M, N, K))
    _check(n if n < 0 else 0, name)
    return n


def w4a4_matmul_workspace_bytes(M, N, K, device=None) -> int:
    """Workspace bytes w4a4_matmul can use for this shape on `device` (default: the current one)."""
    return _mx_workspace_bytes("w4a4_matmul_workspace_bytes", M, N, K, device)


def w4a4_linear_workspace_bytes(M, N, K, device=None) -> int:
    """Workspace bytes of w4a4_linear for this shape on `device` (default: the current one)."""
    return _mx_workspace_bytes("w4a4_linear_workspace_bytes", M, N, K, device)


def w4a4_matmul(M, N, K, aq, a_s, bq, bs, y, stream=None, workspace=None):
    """y [M, N] (float32, bfloat16 or float16; rows may be strided) = A B^T of two MXFP4 operands of depth K.
    `workspace`: a uint8 CUDA tensor, by default one of the size the library asks for, allocated here."""
    _native.matmul(M, N, K, aq, a_s, bq, bs, y, stream, workspace)


def w4a4_linear(M, N, K, x, bq, bs, y, stream=None, workspace=None):
    """y [M, N] = Q(x) B^T: dense x [M, K] quantised along its rows, times an MXFP4 operand of depth K. No
    gradient is computed: x or y that requires one is refused while gradients are enabled."""
    _native.linear(M, N, K, x, bq, bs, y, stream, workspace)


@dataclass
class MXTensor:
    """An MXFP4 operand: `rows` rows of `K` values, blocks of 32 along K (the last one padded with zeros).

    A `stream` given to a method (a torch stream or a raw handle, of the tensors' GPU; None: the current one) takes the
    place of the current stream for the whole call, its copies and allocations included: inputs have to be ready on it, and
    to live until it has read them (`record_stream` where they may be freed earlier), and a result made for it is used
    elsewhere as any tensor made under `torch.cuda.stream(stream)`."""
    codes: torch.Tensor      # uint8 [rows, 16 ceil(K / 32)], element 2j in the low half of byte j
    scales: torch.Tensor     # uint8 [rows, ceil(K / 32)], E8M0; rows a multiple of 4 bytes apart
    rows: int
    K: int

    @staticmethod
    def empty(rows: int, K: int, device="cuda") -> "MXTensor":
        if rows < 0 or K < 1:
            raise ValueError(f"an MXFP4 operand needs rows >= 0 and K >= 1, not {rows} and {K}")
        nb = (K + 31) // 32
        scales = torch.empty(rows, (nb + 3) // 4 * 4, dtype=torch.uint8, device=device)
        return MXTensor(torch.empty(rows, 16 * nb, dtype=torch.uint8, device=device), scales[:, :nb], rows, K)

    @staticmethod
    def from_canonical(codes: torch.Tensor, scales: torch.Tensor, K: int | None = None) -> "MXTensor":
        """Codes [rows, K / 2] and E8M0 scales [rows, K / 32] as checkpoints hold them. The tensors are used as they are
        where their rows are aligned (codes to 16 bytes, scales to 4), and copied otherwise. K that is not a multiple of 32
        leaves codes past K in each row's last block, which have to be zeros: products do not mask them."""
        return MXTensor(*_native.from_canonical(codes, scales, K))

    @staticmethod
    def quantize(x: torch.Tensor, stream=None) -> "MXTensor":
        """x [..., K] along its last axis."""
        rows, k, q, s, _, _ = _native.quantize_new(x, True, False, stream)
        return MXTensor(q, s, rows, k)

    @staticmethod
    def quantize_t(x: torch.Tensor, stream=None) -> "MXTensor":
        """x [..., K], seen as a matrix, along its columns: the operand of K rows that stands for its transpose."""
        rows, k, _, _, q, s = _native.quantize_new(x, False, True, stream)
        return MXTensor(q, s, k, rows)

    @staticmethod
    def quantize_both(x: torch.Tensor, stream=None) -> tuple["MXTensor", "MXTensor"]:
        """(quantize(x), quantize_t(x)) from one reading of x."""
        rows, k, q, s, qt, st = _native.quantize_new(x, True, True, stream)
        return MXTensor(q, s, rows, k), MXTensor(qt, st, k, rows)

    def dequant(self, dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
        return _native.dequant_new(self.codes, self.scales, self.rows, self.K, dtype, stream)

    def matmul(self, x, out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32,
               stream=None, workspace: torch.Tensor | None = None) -> torch.Tensor:
        """x self^T [M, rows], self the weights: x an MXTensor of the same K, or dense [M, K], quantised on the way. No
        gradient is computed: dense x (or `out`) that requires one is refused while gradients are enabled."""
        if isinstance(x, MXTensor):
            if x.K != self.K:
                raise ValueError(f"depths differ: {x.K} and {self.K}")
            return _native.matmul_new(x.codes, x.scales, x.rows, self.codes, self.scales, self.rows, self.K, out, out_dtype,
                                      stream, workspace)
        return _native.linear_new(x, self.codes, self.scales, self.rows, self.K, out, out_dtype, stream, workspace)


def mx_linear(x: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
    """x [..., K] times w [N, K] transposed, both quantised to MXFP4 in the call, in x's type; differentiable once in both.

    Rounding to MXFP4 counts as the identity in the backward pass, whose products are MXFP4 too: with g the gradient of
    the result, dx = Q(g) Q(w^T)^T in x's type and dw = Q(g^T) Q(x^T)^T in w's, every operand quantised along the axis that
    its product contracts. x and w are float32, bfloat16 or float16 on one GPU.

    A step captured into a graph takes its gradients with torch.autograd.grad; torch's accumulation into `.grad` joins the
    stream on which an eager step that is still alive first used the leaf, which a capture cannot do."""
    return _native.mx_linear(x, w)
