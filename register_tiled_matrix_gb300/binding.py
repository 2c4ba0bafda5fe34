"""ctypes binding of libgemm_gb300.so: argument marshalling only.

Every step of the product runs in the library's CUDA kernels; this module
checks tensor metadata, allocates the output with torch when the caller gives
none, passes raw device pointers and the current torch stream, and turns a
non-zero status into an exception. There is no CPU fallback: if the library
is missing the calls raise.
"""

from __future__ import annotations

import ctypes
import os
import re
from typing import Callable, List, Optional, Tuple

import torch

from . import native_build as _build

STATUS = {
    0: "GEMM_OK",
    -1: "GEMM_ERR_INVALID_ARG",
    -2: "GEMM_ERR_ALIGNMENT",
    -3: "GEMM_ERR_LAUNCH",
    -4: "GEMM_ERR_TIMEOUT",
    -5: "GEMM_ERR_DEVICE",
}

_lib: Optional[ctypes.CDLL] = None


class GemmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


def library_path() -> str:
    return _build.LIB


def load_library() -> ctypes.CDLL:
    """Load the built library (build it first with register_tiled_matrix_gb300.build())."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"CUDA library {path} is not built: call register_tiled_matrix_gb300.build() "
                "(nvcc, sm_103a) first; there is no fallback implementation")
        lib = ctypes.CDLL(path)
        i64, p = ctypes.c_int64, ctypes.c_void_p
        for name in ("gemm_f32", "gemm_bf16f32", "gemm_f16f32"):
            f = getattr(lib, name)
            f.argtypes = [i64, i64, i64, p, p, p, p]
            f.restype = ctypes.c_int
        lib.gemm_f32_workspace_bytes.argtypes = [i64, i64, i64]
        lib.gemm_f32_workspace_bytes.restype = ctypes.c_int64
        lib.gemm_f32_schedule.argtypes = [i64, i64, i64, ctypes.c_int,
                                          ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]
        lib.gemm_f32_schedule.restype = ctypes.c_int
        lib.gemm_f32_ws.argtypes = [i64, i64, i64, p, p, p, p, i64, p]
        lib.gemm_f32_ws.restype = ctypes.c_int
        lib.gemm_bf16f32_workspace_bytes.argtypes = [i64, i64, i64]
        lib.gemm_bf16f32_workspace_bytes.restype = ctypes.c_int64
        for name in ("gemm_bf16f32_ws", "gemm_f16f32_ws"):
            f = getattr(lib, name)
            f.argtypes = [i64, i64, i64, p, p, p, p, i64, p]
            f.restype = ctypes.c_int
        lib.gemm_f32_ladder.argtypes = [ctypes.c_int, i64, i64, i64, p, p, p, p]
        lib.gemm_f32_ladder.restype = ctypes.c_int
        lib.gemm_bf16f32_selftest_timeout.argtypes = [i64, i64, i64, p, p, p, i64, p]
        lib.gemm_bf16f32_selftest_timeout.restype = ctypes.c_int
        lib.gemm_f32_selftest_timeout.argtypes = [i64, i64, i64, p, p, p, i64, p]
        lib.gemm_f32_selftest_timeout.restype = ctypes.c_int
        c_int = ctypes.c_int
        for name, args in (("gemm_w4_codes_bytes", [i64, i64]), ("gemm_q8_codes_bytes", [i64, i64]),
                           ("gemm_w4_workspace_bytes", [i64, i64, i64]),
                           ("gemm_q8t_workspace_bytes", [i64, i64, i64])):
            f = getattr(lib, name)
            f.argtypes, f.restype = args, i64
        lib.gemm_w4_pack.argtypes = [i64, i64, p, p, p]
        lib.gemm_w4_pack.restype = c_int
        for t in ("bf16", "f16"):
            for name, args in ((f"gemm_{t}_w4_quantize", [i64, i64, c_int, p, p, p, p, p]),
                               (f"gemm_{t}_w4_dequantize", [i64, i64, c_int, p, p, p, p, p]),
                               (f"gemm_{t}_q8_quantize", [i64, i64, p, p, p, p]),
                               (f"gemm_{t}_q8_dequantize", [i64, i64, p, p, p, p]),
                               (f"gemm_{t}w4f32", [i64] * 3 + [p] * 4 + [c_int, p, p, i64, p]),
                               (f"gemm_q8t{t}f32", [i64] * 3 + [p] * 5 + [i64, p])):
                f = getattr(lib, name)
                f.argtypes, f.restype = args, c_int
        lib.gemm_bf16w4f32_selftest_timeout.argtypes = [i64] * 3 + [p] * 4 + [c_int, p, i64, p]
        lib.gemm_bf16w4f32_selftest_timeout.restype = c_int
        lib.gemm_q8tbf16f32_selftest_timeout.argtypes = [i64] * 3 + [p] * 4 + [i64, p]
        lib.gemm_q8tbf16f32_selftest_timeout.restype = c_int
        f32 = ctypes.c_float
        lib.gemm_f8_pitch.argtypes = [i64]
        lib.gemm_route_rows.argtypes = [i64] * 4
        lib.gemm_route_workspace_bytes.argtypes = [i64, i64]
        for name in ("gemm_f8_pitch", "gemm_route_rows", "gemm_route_workspace_bytes"):
            getattr(lib, name).restype = i64
        operands = [p, i64, p, p, i64, p, p]  # two of (codes, pitch, scales), the result
        for name, args in [("gemm_f8w8f32_selftest_timeout", [i64] * 3 + operands + [i64, p]),
                           ("gemm_experts_join", [i64] * 4 + [p] * 5)]:
            f = getattr(lib, name)
            f.argtypes, f.restype = args, c_int
        for name in ("gemm_f8w8f32", "gemm_f8w8tf32", "gemm_f8tf8f32"):
            for entry, args in ((name, [i64] * 3 + operands + [p]),
                                (f"{name}_experts", [i64] * 4 + [p] + operands + [p])):
                f = getattr(lib, entry)
                f.argtypes, f.restype = args, c_int
        for t in ("f32", "bf16", "f16"):
            for name, args in ((f"gemm_{t}_f8_quantize", [i64, i64, p, i64, p, i64] + [p] * 6),
                               (f"gemm_{t}_f8_quantize_tiles", [i64] * 3 + [p] * 4),
                               (f"gemm_{t}_f8_dequantize", [i64] * 3 + [c_int, p, i64, p, p, p]),
                               (f"gemm_{t}_route", [i64] * 3 + [p, p, i64, i64, c_int, c_int, f32,
                                                                i64] + [p] * 6 + [i64, p]),
                               (f"gemm_{t}_route_backward", [i64] * 3 + [p, c_int, c_int, f32] +
                                [p] * 4),
                               (f"gemm_{t}_experts_join_backward", [i64] * 4 + [p] * 5)):
                f = getattr(lib, name)
                f.argtypes, f.restype = args, c_int
        lib.gemm_fp32_pipe_peak.argtypes = [i64, ctypes.c_int, p, ctypes.POINTER(ctypes.c_double),
                                            p]
        lib.gemm_fp32_pipe_peak.restype = ctypes.c_int
        lib.gemm_get_device_error.argtypes = [p]
        lib.gemm_get_device_error.restype = ctypes.c_int
        lib.gemm_status_string.argtypes = [ctypes.c_int]
        lib.gemm_status_string.restype = ctypes.c_char_p
        _lib = lib
    return _lib


def header_symbols() -> List[str]:
    """Names of the functions declared in include/gemm.h."""
    path = os.path.join(_build.INCLUDE, "gemm.h")
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(gemm_\w+)\s*\(", text)))


def status_string(status: int) -> str:
    return load_library().gemm_status_string(int(status)).decode()


def _check(status: int) -> None:
    if status != 0:
        raise GemmError(status, status_string(status))


# The current stream's handle without building a torch.cuda.Stream object
# (about a microsecond per call); the public API where the accessor is absent.
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream: Optional[torch.cuda.Stream], device: Optional[int] = None) -> int:
    if stream is not None:
        return int(stream.cuda_stream)
    if _raw_current_stream is not None:
        return int(_raw_current_stream(torch.cuda.current_device() if device is None else device))
    return int(torch.cuda.current_stream().cuda_stream)


class _SameDevice:
    """The device guard of a call whose tensors are on the current device: none."""

    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_SAME_DEVICE = _SameDevice()


def _on_device(t: torch.Tensor):
    """A context that makes t's device current for the call (switching only when
    it is not current already: the switch and switch back cost microseconds)."""
    idx = t.get_device()
    return _SAME_DEVICE if idx == torch.cuda.current_device() else torch.cuda.device(idx)


def _library() -> ctypes.CDLL:
    return _lib if _lib is not None else load_library()


def _prepare(A: torch.Tensor, B: torch.Tensor, dtype: torch.dtype,
             out: Optional[torch.Tensor]) -> torch.Tensor:
    for name, t in (("A", A), ("B", B)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.dim() != 2 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 2-D (row-major) matrix")
    M, K = A.shape
    K2, N = B.shape
    if K2 != K:
        raise ValueError(f"inner dimensions differ: A is {M}x{K}, B is {K2}x{N}")
    if A.device != B.device:
        raise ValueError("A and B must be on the same device")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
    elif (out.dtype != torch.float32 or out.shape != (M, N) or not out.is_contiguous()
          or out.device != A.device):
        raise ValueError("out must be a contiguous float32 M x N tensor on A's device")
    return out


def gemm_f32(A: torch.Tensor, B: torch.Tensor, out: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """C = A @ B on the SIMT FP32 register-tiled kernel (fp32 in, fp32 out)."""
    C = _prepare(A, B, torch.float32, out)
    M, K = A.shape
    N = B.shape[1]
    with _on_device(A):
        _check(_library().gemm_f32(M, N, K, A.data_ptr(), B.data_ptr(), C.data_ptr(),
                                       _stream_handle(stream, A.get_device())))
    return C


F32_KINDS = {0: "none", 1: "tiles", 2: "tiles+cluster-split", 3: "tiles+workspace-split",
             4: "column-strips", 5: "tiles+tail-cluster-split", 6: "tall-tiles",
             7: "tall-tiles+cluster-split", 8: "wide-tiles", 9: "wide-tiles+cluster-split",
             10: "tiles+stream-k"}


def gemm_f32_schedule(M: int, N: int, K: int, workspace: bool = False) -> Tuple[str, int]:
    """(kind, splits): how gemm_f32 (or gemm_f32_ws, workspace=True) computes this
    shape on the current device; kind is a value of F32_KINDS."""
    kind, splits = ctypes.c_int(-1), ctypes.c_int(0)
    _check(load_library().gemm_f32_schedule(int(M), int(N), int(K), 1 if workspace else 0,
                                            ctypes.byref(kind), ctypes.byref(splits)))
    return F32_KINDS[kind.value], splits.value


def gemm_f32_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace bytes gemm_f32_ws uses for this shape on the current device (0: none)."""
    n = int(load_library().gemm_f32_workspace_bytes(int(M), int(N), int(K)))
    _check(n if n < 0 else 0)
    return n


def gemm_f32_ws(A: torch.Tensor, B: torch.Tensor, out: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """C = A @ B, splitting K over a workspace when the shape has too few C tiles.

    `workspace` is a CUDA tensor of at least gemm_f32_workspace_bytes(M, N, K)
    bytes; when None, one is allocated with torch for this call."""
    C = _prepare(A, B, torch.float32, out)
    M, K = A.shape
    N = B.shape[1]
    with _on_device(A):
        if workspace is None:
            need = gemm_f32_workspace_bytes(M, N, K)
            workspace = torch.empty(max(need // 4, 1), dtype=torch.float32, device=A.device)
        if not workspace.is_cuda or workspace.device != A.device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor on A's device")
        nbytes = workspace.numel() * workspace.element_size()
        _check(_library().gemm_f32_ws(M, N, K, A.data_ptr(), B.data_ptr(), C.data_ptr(),
                                      workspace.data_ptr(), nbytes,
                                      _stream_handle(stream, A.get_device())))
    return C


LADDER = {0: "naive", 1: "shared-tiled 32x32", 2: "register-tiled 64x64, 4x4/thread",
          3: "register-tiled 128x128, 8x8/thread (gemm_f32)",
          4: "register-tiled 16x16, 1x1/thread (rung 2's kernel, T=1)",
          5: "register-tiled 32x32, 2x2/thread (rung 2's kernel, T=2)",
          6: "register-tiled 128x128, 8x8/thread (rung 2's kernel, T=8)"}


def gemm_f32_ladder(rung: int, A: torch.Tensor, B: torch.Tensor,
                    out: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """C = A @ B with rung `rung` of the page's ablation ladder (see LADDER)."""
    C = _prepare(A, B, torch.float32, out)
    M, K = A.shape
    N = B.shape[1]
    with _on_device(A):
        _check(load_library().gemm_f32_ladder(int(rung), M, N, K, A.data_ptr(), B.data_ptr(),
                                              C.data_ptr(), _stream_handle(stream, A.get_device())))
    return C


def gemm_bf16f32(A: torch.Tensor, B: torch.Tensor, out: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """C = A @ B on the tcgen05 tensor-core kernel (bf16 in, fp32 accumulate and out)."""
    C = _prepare(A, B, torch.bfloat16, out)
    M, K = A.shape
    N = B.shape[1]
    with _on_device(A):
        _check(_library().gemm_bf16f32(M, N, K, A.data_ptr(), B.data_ptr(), C.data_ptr(),
                                           _stream_handle(stream, A.get_device())))
    return C


def gemm_f16f32(A: torch.Tensor, B: torch.Tensor, out: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """C = A @ B on the tcgen05 tensor-core kernel (fp16 in, fp32 accumulate and out)."""
    C = _prepare(A, B, torch.float16, out)
    M, K = A.shape
    N = B.shape[1]
    with _on_device(A):
        _check(_library().gemm_f16f32(M, N, K, A.data_ptr(), B.data_ptr(), C.data_ptr(),
                                          _stream_handle(stream, A.get_device())))
    return C


def gemm_bf16f32_workspace_bytes(M: int, N: int, K: int) -> int:
    """Largest workspace gemm_bf16f32_ws / gemm_f16f32_ws may use for this shape (0: none)."""
    n = int(load_library().gemm_bf16f32_workspace_bytes(int(M), int(N), int(K)))
    _check(n if n < 0 else 0)
    return n


def _rows_on_16_bytes(t: torch.Tensor) -> bool:
    return t.shape[1] % 8 == 0 and t.data_ptr() % 16 == 0


def _gemm_2byte_ws(entry: str, A: torch.Tensor, B: torch.Tensor, dtype: torch.dtype,
                   out: Optional[torch.Tensor], workspace: Optional[torch.Tensor],
                   stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    C = _prepare(A, B, dtype, out)
    M, K = A.shape
    N = B.shape[1]
    with _on_device(A):
        if workspace is None and M > 128 and not (_rows_on_16_bytes(A) and _rows_on_16_bytes(B)):
            workspace = torch.empty(gemm_bf16f32_workspace_bytes(M, N, K), dtype=torch.uint8,
                                    device=A.device)
        ptr, nbytes = 0, 0
        if workspace is not None:
            if (not workspace.is_cuda or workspace.device != A.device
                    or not workspace.is_contiguous()):
                raise ValueError("workspace must be a contiguous CUDA tensor on A's device")
            ptr, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        _check(getattr(_library(), entry)(M, N, K, A.data_ptr(), B.data_ptr(), C.data_ptr(),
                                          ptr, nbytes, _stream_handle(stream, A.get_device())))
    return C


def gemm_bf16f32_ws(A: torch.Tensor, B: torch.Tensor, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """gemm_bf16f32, re-pitching operands whose rows are not 16-byte aligned into
    `workspace` (a CUDA tensor of at least gemm_bf16f32_workspace_bytes(M, N, K)
    bytes; allocated with torch for this call when None and a copy is needed)."""
    return _gemm_2byte_ws("gemm_bf16f32_ws", A, B, torch.bfloat16, out, workspace, stream)


def gemm_f16f32_ws(A: torch.Tensor, B: torch.Tensor, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """gemm_f16f32 with the workspace rule of gemm_bf16f32_ws."""
    return _gemm_2byte_ws("gemm_f16f32_ws", A, B, torch.float16, out, workspace, stream)


# ---------------------------------------------------------------- low-bit operands

W4_BLOCK = 128  # k per 64-byte block of packed 4-bit codes
W4_GROUPS = (32, 64, 128)
Q8_ROWS = 128   # rows sharing a scale
_TYPE_NAMES = {torch.bfloat16: "bf16", torch.float16: "f16"}


def _type_name(dtype: torch.dtype) -> str:
    try:
        return _TYPE_NAMES[dtype]
    except KeyError:
        raise ValueError(f"the type must be torch.bfloat16 or torch.float16, got {dtype}") from None


def _need(name: str, t: torch.Tensor, dtype: torch.dtype, shape, device=None) -> None:
    if (type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and (t.device == device if device is not None else t.is_cuda) and t.is_cuda):
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {' x '.join(map(str, shape))} tensor, "
                         f"got {' x '.join(map(str, t.shape))}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _matrix(name: str, t: torch.Tensor) -> Tuple[int, int]:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D (row-major) matrix")
    return t.shape


def _empty(like: torch.Tensor, shape, dtype: torch.dtype,
           stream: Optional[torch.cuda.Stream]) -> torch.Tensor:
    """Memory on like's device, of the stream the call runs on, so that it is reused in
    that stream's order."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _call(entry: str, device: int, stream: Optional[torch.cuda.Stream], *args) -> None:
    """entry(*args, stream) with `device` current (switched to only when it is not)."""
    f = getattr(_lib or load_library(), entry)
    if device == torch.cuda.current_device():
        status = f(*args, _stream_handle(stream, device))
    else:
        with torch.cuda.device(device):
            status = f(*args, _stream_handle(stream, device))
    if status:
        _check(status)


def _plain(t, dtype: torch.dtype, device: int) -> bool:
    return (type(t) is torch.Tensor and t.dtype is dtype and t.get_device() == device
            and t.is_contiguous())


def _w4_check(codes, scales, zeros, K: int, group: int, device) -> int:
    """Checks the three parts of a 4-bit weight with K rows; returns its columns."""
    if group not in W4_GROUPS:
        raise ValueError(f"group must be one of {W4_GROUPS}, got {group}")
    N = _matrix("codes", codes)[0]
    _need("codes", codes, torch.uint8, (N, (K + W4_BLOCK - 1) // W4_BLOCK * 64), device)
    meta = ((K + group - 1) // group, N)
    _matrix("scales", scales)
    _type_name(scales.dtype)
    _need("scales", scales, scales.dtype, meta, device)
    if zeros is not None:
        _need("zeros", zeros, torch.uint8, meta, device)
    return N


def gemm_w4_quantize(W: torch.Tensor, group: int = 128, zeros: bool = True,
                     stream: Optional[torch.cuda.Stream] = None
                     ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """(codes, scales, zero points) of a bf16 or fp16 K x N weight in 4 bits, `group`
    (32, 64 or 128) consecutive k of a column to a scale; zeros=False: symmetric
    codes around 8 and None for the zero points. Layout: include/gemm.h."""
    K, N = _matrix("W", W)
    name = _type_name(W.dtype)
    if group not in W4_GROUPS:
        raise ValueError(f"group must be one of {W4_GROUPS}, got {group}")
    codes = _empty(W, (N, (K + W4_BLOCK - 1) // W4_BLOCK * 64), torch.uint8, stream)
    meta = ((K + group - 1) // group, N)
    scales = _empty(W, meta, W.dtype, stream)
    zp = _empty(W, meta, torch.uint8, stream) if zeros else None
    _call(f"gemm_{name}_w4_quantize", W.get_device(), stream, K, N, group, W.data_ptr(),
          codes.data_ptr(), scales.data_ptr(), zp.data_ptr() if zeros else 0)
    return codes, scales, zp


def gemm_w4_pack(q: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Packed codes of a K x N uint8 tensor of 4-bit codes, one a byte (weights
    quantised elsewhere)."""
    K, N = _matrix("q", q)
    _need("q", q, torch.uint8, (K, N))
    codes = _empty(q, (N, (K + W4_BLOCK - 1) // W4_BLOCK * 64), torch.uint8, stream)
    _call("gemm_w4_pack", q.get_device(), stream, K, N, q.data_ptr(), codes.data_ptr())
    return codes


def gemm_w4_dequantize(codes: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor],
                       K: int, group: int = 128, out: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The K x N weight (q - z) * s in the scales' type."""
    _matrix("codes", codes)
    N = _w4_check(codes, scales, zeros, K, group, codes.device)
    if out is None:
        out = _empty(codes, (K, N), scales.dtype, stream)
    else:
        _need("out", out, scales.dtype, (K, N), codes.device)
    _call(f"gemm_{_type_name(scales.dtype)}_w4_dequantize", codes.get_device(), stream, K, N, group,
          codes.data_ptr(), scales.data_ptr(), 0 if zeros is None else zeros.data_ptr(),
          out.data_ptr())
    return out


def _workspace(workspace: Optional[torch.Tensor], operand: torch.Tensor, entry: str, size,
               stream) -> Tuple[int, int, Optional[torch.Tensor]]:
    """(pointer, bytes, tensor) of the caller's workspace, or of one made for this call
    when the 2-byte operand's rows are off 16-byte boundaries."""
    if workspace is None:
        need = 0 if _rows_on_16_bytes(operand) else int(getattr(_library(), entry)(*size))
        if need <= 0:
            return 0, 0, None
        workspace = _empty(operand, (need,), torch.uint8, stream)
    elif (not isinstance(workspace, torch.Tensor) or not workspace.is_cuda
          or workspace.device != operand.device or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous CUDA tensor on {operand.device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _w4_product(entry: str, dtype: torch.dtype, A, codes, scales, zeros, group, out, workspace,
                stream) -> torch.Tensor:
    # One look at everything a valid call passes (a decoded token's call takes little
    # longer than its kernel); what fails it is looked at part by part for its message.
    device = A.get_device() if type(A) is torch.Tensor else -1
    fine = (device >= 0 and group in W4_GROUPS and _plain(A, dtype, device)
            and _plain(codes, torch.uint8, device) and _plain(scales, dtype, device)
            and A.dim() == 2 and codes.dim() == 2)
    if fine:
        M, K = A.shape
        N, row = codes.shape
        meta = ((K + group - 1) // group, N)
        fine = (row == (K + W4_BLOCK - 1) // W4_BLOCK * 64 and scales.shape == meta
                and (zeros is None or (_plain(zeros, torch.uint8, device) and zeros.shape == meta)))
    if not fine:
        M, K = _matrix("A", A)
        _need("A", A, dtype, (M, K))
        _need("scales", scales, dtype, _matrix("scales", scales), A.device)
        N = _w4_check(codes, scales, zeros, K, group, A.device)
    if out is None:
        out = _empty(A, (M, N), torch.float32, stream)
    else:
        _need("out", out, torch.float32, (M, N), A.device)
    ptr, nbytes, workspace = _workspace(workspace, A, "gemm_w4_workspace_bytes", (M, N, K), stream)
    _call(entry, A.get_device(), stream, M, N, K, A.data_ptr(), codes.data_ptr(),
          scales.data_ptr(), 0 if zeros is None else zeros.data_ptr(), group, out.data_ptr(), ptr,
          nbytes)
    return out


def gemm_bf16w4f32(A: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                   zeros: Optional[torch.Tensor] = None, group: int = 128,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """C = A @ W (fp32) with bf16 A (M x K) and W (K x N) in 4 bits, as gemm_w4_quantize
    gives it. `workspace` (a CUDA tensor of gemm_w4_workspace_bytes(M, N, K) bytes)
    is allocated for this call when None and the call can use one."""
    return _w4_product("gemm_bf16w4f32", torch.bfloat16, A, codes, scales, zeros, group, out,
                       workspace, stream)


def gemm_f16w4f32(A: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                  zeros: Optional[torch.Tensor] = None, group: int = 128,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """gemm_bf16w4f32 for fp16 A and scales."""
    return _w4_product("gemm_f16w4f32", torch.float16, A, codes, scales, zeros, group, out,
                       workspace, stream)


def gemm_w4_workspace_bytes(M: int, N: int, K: int) -> int:
    """Largest workspace gemm_bf16w4f32 / gemm_f16w4f32 can use for this shape (0: none)."""
    n = int(load_library().gemm_w4_workspace_bytes(int(M), int(N), int(K)))
    _check(n if n < 0 else 0)
    return n


def gemm_q8_quantize(X: torch.Tensor, stream: Optional[torch.cuda.Stream] = None
                     ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(codes, scales): a bf16 or fp16 M x K activation saved in 8 bits, one scale
    for each column of 128 rows. codes: int8, M x ceil16(K); scales: fp32."""
    M, K = _matrix("X", X)
    name = _type_name(X.dtype)
    codes = _empty(X, (M, (K + 15) // 16 * 16), torch.int8, stream)
    scales = _empty(X, ((M + Q8_ROWS - 1) // Q8_ROWS, K), torch.float32, stream)
    _call(f"gemm_{name}_q8_quantize", X.get_device(), stream, M, K, X.data_ptr(),
          codes.data_ptr(), scales.data_ptr())
    return codes, scales


def _q8_check(codes, scales, M: int, K: int, device) -> None:
    _need("codes", codes, torch.int8, (M, (K + 15) // 16 * 16), device)
    _need("scales", scales, torch.float32, ((M + Q8_ROWS - 1) // Q8_ROWS, K), device)


def gemm_q8_dequantize(codes: torch.Tensor, scales: torch.Tensor, M: int, K: int,
                       dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The saved M x K activation, codes * scales, in `dtype` (bf16 or fp16)."""
    name = _type_name(dtype)
    _matrix("codes", codes)
    _q8_check(codes, scales, M, K, codes.device)
    if out is None:
        out = _empty(codes, (M, K), dtype, stream)
    else:
        _need("out", out, dtype, (M, K), codes.device)
    _call(f"gemm_{name}_q8_dequantize", codes.get_device(), stream, M, K, codes.data_ptr(),
          scales.data_ptr(), out.data_ptr())
    return out


def _q8t_product(entry: str, dtype: torch.dtype, codes, scales, dY, out, workspace,
                 stream) -> torch.Tensor:
    M, N = _matrix("dY", dY)
    K = _matrix("scales", scales)[1]
    _need("dY", dY, dtype, (M, N))
    _q8_check(codes, scales, M, K, dY.device)
    if out is None:
        out = _empty(dY, (K, N), torch.float32, stream)
    else:
        _need("out", out, torch.float32, (K, N), dY.device)
    ptr, nbytes, workspace = _workspace(workspace, dY, "gemm_q8t_workspace_bytes", (M, N, K), stream)
    _call(entry, dY.get_device(), stream, M, N, K, codes.data_ptr(), scales.data_ptr(),
          dY.data_ptr(), out.data_ptr(), ptr, nbytes)
    return out


def gemm_q8tbf16f32(codes: torch.Tensor, scales: torch.Tensor, dY: torch.Tensor,
                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """dW = X^T @ dY (K x N, fp32): the weight gradient of Y = X @ W from X as
    gemm_q8_quantize saved it and a bf16 dY (M x N). `workspace` (a CUDA tensor of
    gemm_q8t_workspace_bytes(M, N, K) bytes) is allocated for this call when None
    and the call can use one."""
    return _q8t_product("gemm_q8tbf16f32", torch.bfloat16, codes, scales, dY, out, workspace,
                        stream)


def gemm_q8tf16f32(codes: torch.Tensor, scales: torch.Tensor, dY: torch.Tensor,
                   out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """gemm_q8tbf16f32 for fp16 dY."""
    return _q8t_product("gemm_q8tf16f32", torch.float16, codes, scales, dY, out, workspace, stream)


def gemm_q8t_workspace_bytes(M: int, N: int, K: int) -> int:
    """Largest workspace gemm_q8tbf16f32 / gemm_q8tf16f32 can use for this shape (0: none)."""
    n = int(load_library().gemm_q8t_workspace_bytes(int(M), int(N), int(K)))
    _check(n if n < 0 else 0)
    return n


def gemm_bf16w4f32_selftest_timeout(A, codes, scales, zeros, group: int, out: torch.Tensor,
                                    wait_limit_ns: int) -> None:
    """Launch the 4-bit tensor-core kernel with its loads muted so every bounded wait runs out."""
    M, K = _matrix("A", A)
    _need("A", A, torch.bfloat16, (M, K))
    N = _w4_check(codes, scales, zeros, K, group, A.device)
    _need("out", out, torch.float32, (M, N), A.device)
    _call("gemm_bf16w4f32_selftest_timeout", A.get_device(), None, M, N, K, A.data_ptr(),
          codes.data_ptr(), scales.data_ptr(), 0 if zeros is None else zeros.data_ptr(), group,
          out.data_ptr(), int(wait_limit_ns))


def gemm_q8tbf16f32_selftest_timeout(codes, scales, dY, out: torch.Tensor,
                                     wait_limit_ns: int) -> None:
    """Launch the 8-bit weight-gradient kernel with its loads muted so every bounded wait runs out."""
    M, N = _matrix("dY", dY)
    K = _matrix("scales", scales)[1]
    _need("dY", dY, torch.bfloat16, (M, N))
    _q8_check(codes, scales, M, K, dY.device)
    _need("out", out, torch.float32, (K, N), dY.device)
    _call("gemm_q8tbf16f32_selftest_timeout", dY.get_device(), None, M, N, K, codes.data_ptr(),
          scales.data_ptr(), dY.data_ptr(), out.data_ptr(), int(wait_limit_ns))


def gemm_bf16f32_selftest_timeout(A: torch.Tensor, B: torch.Tensor, out: torch.Tensor,
                                  wait_limit_ns: int,
                                  stream: Optional[torch.cuda.Stream] = None) -> None:
    """Launch the bf16 kernel with its loads muted so every bounded wait runs out."""
    C = _prepare(A, B, torch.bfloat16, out)
    M, K = A.shape
    N = B.shape[1]
    with _on_device(A):
        _check(load_library().gemm_bf16f32_selftest_timeout(
            M, N, K, A.data_ptr(), B.data_ptr(), C.data_ptr(), int(wait_limit_ns),
            _stream_handle(stream)))


def gemm_f32_selftest_timeout(A: torch.Tensor, B: torch.Tensor, out: torch.Tensor,
                              wait_limit_ns: int,
                              stream: Optional[torch.cuda.Stream] = None) -> None:
    """Launch gemm_f32's TMA-fed kernel with its loads muted so every bounded wait runs out."""
    C = _prepare(A, B, torch.float32, out)
    M, K = A.shape
    N = B.shape[1]
    with _on_device(A):
        _check(load_library().gemm_f32_selftest_timeout(
            M, N, K, A.data_ptr(), B.data_ptr(), C.data_ptr(), int(wait_limit_ns),
            _stream_handle(stream)))


def get_device_error(stream: Optional[torch.cuda.Stream] = None) -> int:
    """Synchronise the stream; return and clear the device error word."""
    return int(load_library().gemm_get_device_error(_stream_handle(stream)))


def fp32_pipe_peak(iters: int = 20000, packed: bool = False, repeats: int = 5,
                   device: Optional[torch.device] = None) -> dict:
    """Measured throughput of the FP32 FMA pipes (gemm_fp32_pipe_peak).

    Times `repeats` launches with CUDA events on the current stream after one
    warm-up launch and returns the best: {"tflops", "ms", "sm_mhz"} where
    sm_mhz is the SM clock the launch ran at (clock cycles over global-timer
    nanoseconds, read by the kernel)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    lib = load_library()
    best = None
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev)
        clk = torch.zeros(2, dtype=torch.int64, device=dev)
        flops = ctypes.c_double(0.0)
        for r in range(repeats + 1):
            clk.zero_()
            e0 = torch.cuda.Event(enable_timing=True)
            e1 = torch.cuda.Event(enable_timing=True)
            e0.record(stream)
            _check(lib.gemm_fp32_pipe_peak(int(iters), 1 if packed else 0, clk.data_ptr(),
                                           ctypes.byref(flops), int(stream.cuda_stream)))
            e1.record(stream)
            stream.synchronize()
            if r == 0:
                continue  # warm-up launch
            ms = e0.elapsed_time(e1)
            cycles, ns = (int(v) for v in clk.cpu().tolist())
            res = {"tflops": flops.value / (ms * 1e-3) / 1e12, "ms": ms,
                   "sm_mhz": (cycles / ns * 1e3) if ns > 0 else None}
            if best is None or res["tflops"] > best["tflops"]:
                best = res
    return best
