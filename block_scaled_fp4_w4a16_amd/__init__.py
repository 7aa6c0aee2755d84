"""Python binding of the fp4w4a16 C ABI (block-scaled 4-bit weights x bf16 activations on gfx950).

Argument marshalling only: every function below checks tensor devices, dtypes and sizes,
passes raw device pointers and the current HIP stream to the C entry point of the same
name in libfp4w4a16.so, and raises RuntimeError on a negative status. All computation
runs in the library's HIP kernels; there is no fallback path. Importing this package
without the built library fails loudly.
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
# MXFP4 on both sides (W4A4): quantisation, products, a trainable linear layer
# ----------------------------------------------------------------------------------------------

DENSE_TYPES = {torch.float32: 1, torch.bfloat16: 2, torch.float16: 3}
MX_BLOCK = 32


def _dense_type(t: torch.Tensor, what: str, allowed=DENSE_TYPES) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor")
    if t.dtype not in allowed:
        raise TypeError(f"{what} must be one of {sorted(str(d) for d in allowed)}, not {t.dtype}")
    return allowed[t.dtype]


def _rows_of(t: torch.Tensor, rows: int, cols: int, what: str) -> int:
    """Row stride (in elements) of a [rows, cols] matrix whose rows are contiguous."""
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError(f"{what} must have shape [{rows}, {cols}], not {list(t.shape)}")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: the elements of a row must be contiguous")
    if rows > 1 and t.stride(0) < cols:
        raise ValueError(f"{what}: rows overlap")
    return t.stride(0) if rows > 1 else max(cols, 1)


def _blocks(k: int) -> int:
    return (k + MX_BLOCK - 1) // MX_BLOCK


def _mx_struct(q, s, rows: int, k: int, what: str) -> Mx:
    """The C operand of codes q [rows, 16 ceil(k / 32)] and scales s [rows, ceil(k / 32)] (uint8; row strides free)."""
    nb = _blocks(k)
    if q.dtype != torch.uint8 or s.dtype != torch.uint8:
        raise TypeError(f"{what}: codes and scales must be uint8")
    ldq = _rows_of(q, rows, 16 * nb, f"{what} codes")
    lds = _rows_of(s, rows, nb, f"{what} scales")
    if rows == 1:
        lds = (nb + 3) // 4 * 4
    # scale rows are read in whole dwords
    end = s.storage_offset() + (rows - 1) * lds + (nb + 3) // 4 * 4
    if rows > 0 and end > s.untyped_storage().nbytes():
        raise ValueError(f"{what} scales: the last row must be readable up to a multiple of 4 bytes")
    return Mx(q.data_ptr(), s.data_ptr(), ldq, lds)


def fp4_quantize_mxfp4(M, K, x, q=None, s=None, qt=None, st=None, stream=None):
    """x [M, K] (float32, bfloat16 or float16; rows may be strided) -> MXFP4 along its rows into q [M, 16 ceil(K/32)] and
    s [M, ceil(K/32)], and / or along its columns into qt [K, 16 ceil(M/32)] and st [K, ceil(M/32)] (the transposed
    operand). One of the two pairs may be None. Rows of the scales lie a multiple of 4 bytes apart."""
    ty = _dense_type(x, "x")
    ldx = _rows_of(x, M, K, "x")
    if (q is None) != (s is None) or (qt is None) != (st is None):
        raise ValueError("codes and scales come in pairs")
    dev = _device(x, q, s, qt, st)
    rows = _mx_struct(q, s, M, K, "rows") if q is not None else None
    cols = _mx_struct(qt, st, K, M, "columns") if qt is not None else None
    with torch.cuda.device(dev):
        _check(lib().fp4_quantize_mxfp4(ty, M, K, x.data_ptr(), ldx, rows, cols, _stream(stream)), "fp4_quantize_mxfp4")


def fp4_dequant_mxfp4(M, K, q, s, out, stream=None):
    """The values of an MXFP4 operand into out [M, K] (float32 or bfloat16; rows may be strided)."""
    ty = _dense_type(out, "out", {torch.float32: 1, torch.bfloat16: 2})
    ldo = _rows_of(out, M, K, "out")
    dev = _device(q, s, out)
    a = _mx_struct(q, s, M, K, "operand")
    with torch.cuda.device(dev):
        _check(lib().fp4_dequant_mxfp4(ty, M, K, a, out.data_ptr(), ldo, _stream(stream)), "fp4_dequant_mxfp4")


@functools.lru_cache(maxsize=4096)
def _mx_workspace_bytes(name: str, M: int, N: int, K: int, device: int) -> int:
    with torch.cuda.device(device):
        n = int(getattr(lib(), name)(M, N, K))
    _check(n if n < 0 else 0, name)
    return n


def w4a4_matmul_workspace_bytes(M, N, K, device=None) -> int:
    """Workspace bytes w4a4_matmul can use for this shape on `device` (default: the current one)."""
    return _mx_workspace_bytes("w4a4_matmul_workspace_bytes", M, N, K, _device_index(device))


def w4a4_linear_workspace_bytes(M, N, K, device=None) -> int:
    """Workspace bytes of w4a4_linear for this shape on `device` (default: the current one)."""
    return _mx_workspace_bytes("w4a4_linear_workspace_bytes", M, N, K, _device_index(device))


def _device_index(device) -> int:
    if device is None:
        return torch.cuda.current_device()
    d = torch.device(device)
    return d.index if d.index is not None else torch.cuda.current_device()


def _mx_workspace(name, M, N, K, dev, stream, st, workspace):
    """(pointer, bytes, tensor) of the given workspace or of one allocated here as the library asks."""
    if workspace is None:
        nbytes = _mx_workspace_bytes(name, M, N, K, dev.index) if M > 0 else 0
        if nbytes == 0:
            return None, 0, None
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        if stream is not None:
            # the kernels run on `stream`, not necessarily the one the allocator recorded
            ext = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(st)
            workspace.record_stream(ext)
    elif workspace.device != dev:
        raise ValueError("the workspace must live on the tensors' GPU")
    return _ptr(workspace), _nbytes(workspace), workspace


def w4a4_matmul(M, N, K, aq, a_s, bq, bs, y, stream=None, workspace=None):
    """y [M, N] (float32, bfloat16 or float16; rows may be strided) = A B^T of two MXFP4 operands of depth K."""
    ty = _dense_type(y, "y")
    ldy = _rows_of(y, M, N, "y")
    dev = _device(aq, a_s, bq, bs, y)
    a, b = _mx_struct(aq, a_s, M, K, "A"), _mx_struct(bq, bs, N, K, "B")
    with torch.cuda.device(dev):
        st = _stream(stream)
        ws, nbytes, keep = _mx_workspace("w4a4_matmul_workspace_bytes", M, N, K, dev, stream, st, workspace)
        _check(lib().w4a4_matmul(ty, M, N, K, a, b, y.data_ptr(), ldy, ws, nbytes, st), "w4a4_matmul")


def w4a4_linear(M, N, K, x, bq, bs, y, stream=None, workspace=None):
    """y [M, N] = Q(x) B^T: dense x [M, K] quantised along its rows, times an MXFP4 operand of depth K."""
    tx, ty = _dense_type(x, "x"), _dense_type(y, "y")
    ldx, ldy = _rows_of(x, M, K, "x"), _rows_of(y, M, N, "y")
    dev = _device(x, bq, bs, y)
    b = _mx_struct(bq, bs, N, K, "B")
    with torch.cuda.device(dev):
        st = _stream(stream)
        ws, nbytes, keep = _mx_workspace("w4a4_linear_workspace_bytes", M, N, K, dev, stream, st, workspace)
        _check(lib().w4a4_linear(tx, ty, M, N, K, x.data_ptr(), ldx, b, y.data_ptr(), ldy, ws, nbytes, st), "w4a4_linear")


def _as_rows(x: torch.Tensor) -> torch.Tensor:
    """x [..., K] as a matrix whose rows are contiguous (a copy only where the strides ask for one)."""
    x = x.reshape(-1, x.shape[-1]) if x.dim() != 2 else x
    ok = (x.shape[1] <= 1 or x.stride(1) == 1) and (x.shape[0] <= 1 or x.stride(0) >= x.shape[1])
    return x if ok else x.contiguous()


@dataclass
class MXTensor:
    """An MXFP4 operand: `rows` rows of `K` values, blocks of 32 along K (the last one padded with zeros)."""
    codes: torch.Tensor      # uint8 [rows, 16 ceil(K / 32)], element 2j in the low half of byte j
    scales: torch.Tensor     # uint8 [rows, ceil(K / 32)], E8M0; rows a multiple of 4 bytes apart
    rows: int
    K: int

    @staticmethod
    def empty(rows: int, K: int, device="cuda") -> "MXTensor":
        if rows < 0 or K < 1:
            raise ValueError(f"an MXFP4 operand needs rows >= 0 and K >= 1, not {rows} and {K}")
        nb = _blocks(K)
        scales = torch.empty(rows, (nb + 3) // 4 * 4, dtype=torch.uint8, device=device)
        return MXTensor(torch.empty(rows, 16 * nb, dtype=torch.uint8, device=device), scales[:, :nb], rows, K)

    @staticmethod
    def from_canonical(codes: torch.Tensor, scales: torch.Tensor, K: int | None = None) -> "MXTensor":
        """Codes [rows, K / 2] and E8M0 scales [rows, K / 32] as checkpoints hold them. The tensors are used as they are
        where their rows are aligned (codes to 16 bytes, scales to 4), and copied otherwise."""
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales must be uint8")
        if codes.dim() != 2 or scales.dim() != 2 or codes.shape[0] != scales.shape[0]:
            raise ValueError("codes and scales must be matrices with the same number of rows")
        K = codes.shape[1] * 2 if K is None else K
        rows, nb = codes.shape[0], _blocks(K)
        if K < 1 or codes.shape[1] != 16 * nb or scales.shape[1] != nb:
            raise ValueError(f"K = {K} needs {16 * nb} bytes of codes and {nb} scales a row, "
                             f"not {codes.shape[1]} and {scales.shape[1]}")
        _device(codes, scales)
        t = MXTensor.empty(rows, K, device=codes.device)
        if codes.stride(1) == 1 and (rows <= 1 or (codes.stride(0) % 16 == 0 and codes.stride(0) >= 16 * nb)) \
                and codes.data_ptr() % 16 == 0:
            t.codes = codes
        else:
            t.codes.copy_(codes)
        end = scales.storage_offset() + (rows - 1) * scales.stride(0) + (nb + 3) // 4 * 4
        if (nb <= 1 or scales.stride(1) == 1) and (rows <= 1 or (scales.stride(0) % 4 == 0 and scales.stride(0) >= nb)) \
                and scales.data_ptr() % 4 == 0 and end <= scales.untyped_storage().nbytes():
            t.scales = scales
        else:
            t.scales.copy_(scales)
        return t

    @staticmethod
    def quantize(x: torch.Tensor, stream=None) -> "MXTensor":
        """x [..., K] along its last axis."""
        x = _as_rows(x)
        t = MXTensor.empty(x.shape[0], x.shape[1], device=x.device)
        fp4_quantize_mxfp4(x.shape[0], x.shape[1], x, t.codes, t.scales, stream=stream)
        return t

    @staticmethod
    def quantize_t(x: torch.Tensor, stream=None) -> "MXTensor":
        """x [..., K], seen as a matrix, along its columns: the operand of K rows that stands for its transpose."""
        x = _as_rows(x)
        t = MXTensor.empty(x.shape[1], x.shape[0], device=x.device)
        fp4_quantize_mxfp4(x.shape[0], x.shape[1], x, None, None, t.codes, t.scales, stream=stream)
        return t

    @staticmethod
    def quantize_both(x: torch.Tensor, stream=None) -> tuple["MXTensor", "MXTensor"]:
        """(quantize(x), quantize_t(x)) from one reading of x."""
        x = _as_rows(x)
        r = MXTensor.empty(x.shape[0], x.shape[1], device=x.device)
        c = MXTensor.empty(x.shape[1], x.shape[0], device=x.device)
        fp4_quantize_mxfp4(x.shape[0], x.shape[1], x, r.codes, r.scales, c.codes, c.scales, stream=stream)
        return r, c

    def dequant(self, dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
        out = torch.empty(self.rows, self.K, dtype=dtype, device=self.codes.device)
        fp4_dequant_mxfp4(self.rows, self.K, self.codes, self.scales, out, stream)
        return out

    def matmul(self, x, out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float32,
               stream=None, workspace: torch.Tensor | None = None) -> torch.Tensor:
        """x self^T [M, rows], self the weights: x an MXTensor of the same K, or dense [M, K], quantised on the way."""
        if isinstance(x, MXTensor):
            if x.K != self.K:
                raise ValueError(f"depths differ: {x.K} and {self.K}")
            m = x.rows
        else:
            if x.dim() != 2 or x.shape[1] != self.K:
                raise ValueError("x must be [M, K] with the weights' K")
            m = x.shape[0]
        if out is None:
            out = torch.empty(m, self.rows, dtype=out_dtype, device=self.codes.device)
        if isinstance(x, MXTensor):
            w4a4_matmul(m, self.rows, self.K, x.codes, x.scales, self.codes, self.scales, out, stream, workspace)
        else:
            w4a4_linear(m, self.rows, self.K, _as_rows(x), self.codes, self.scales, out, stream, workspace)
        return out


class _MxLinear(torch.autograd.Function):
    """y = Q(x) Q(w)^T. Rounding to MXFP4 counts as the identity in the backward pass, whose products are MXFP4 too:
    dx = Q(g) Q(w^T)^T contracts N, dw = Q(g^T) Q(x^T)^T contracts the rows of x, each operand quantised along the axis
    contracted. The transposed operands are made with the forward ones, from one reading of x and of w."""

    @staticmethod
    def forward(ctx, x, w):
        rows = _as_rows(x)
        need_dx, need_dw = ctx.needs_input_grad
        ctx.shape, ctx.w_dtype, ctx.x_dtype = x.shape, w.dtype, x.dtype
        xq, xt = MXTensor.quantize_both(rows) if need_dw and rows.shape[0] else (MXTensor.quantize(rows), None)
        wm = _as_rows(w)
        wq, wt = MXTensor.quantize_both(wm) if need_dx else (MXTensor.quantize(wm), None)
        empty = torch.empty(0, dtype=torch.uint8, device=x.device)
        ctx.save_for_backward(xt.codes if xt else empty, xt.scales if xt else empty, wt.codes if wt else empty,
                              wt.scales if wt else empty)
        return wq.matmul(xq, out_dtype=x.dtype).reshape(*x.shape[:-1], w.shape[0])

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        xc, xs, wc, ws = ctx.saved_tensors
        g = _as_rows(g)
        m, n = g.shape
        k = ctx.shape[-1]
        need_dx, need_dw = ctx.needs_input_grad
        dx = dw = None
        if m == 0:
            dx = torch.empty(ctx.shape, dtype=ctx.x_dtype, device=g.device) if need_dx else None
            dw = torch.zeros(n, k, dtype=ctx.w_dtype, device=g.device) if need_dw else None
            return dx, dw
        gq = gt = None
        if need_dx and need_dw:
            gq, gt = MXTensor.quantize_both(g)
        elif need_dx:
            gq = MXTensor.quantize(g)
        elif need_dw:
            gt = MXTensor.quantize_t(g)
        if need_dx:
            dx = MXTensor(wc, ws, k, n).matmul(gq, out_dtype=ctx.x_dtype).reshape(ctx.shape)
        if need_dw:
            dw = MXTensor(xc, xs, k, m).matmul(gt, out_dtype=ctx.w_dtype)
        return dx, dw


def mx_linear(x: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
    """x [..., K] times w [N, K] transposed, both quantised to MXFP4 in the call, in x's type; differentiable in both.
    x and w are float32, bfloat16 or float16 on one GPU; dx has x's type and dw has w's."""
    _dense_type(x, "x")
    _dense_type(w, "w")
    _device(x, w)
    if x.dim() < 1 or w.dim() != 2 or x.shape[-1] != w.shape[1]:
        raise ValueError(f"x [..., K] and w [N, K] expected, not {list(x.shape)} and {list(w.shape)}")
    if w.shape[0] < 1 or w.shape[1] < 1:
        raise ValueError("w has no rows or no columns")
    return _MxLinear.apply(x, w)
