"""ctypes binding of the 8-bit floating-point products and of the experts' layer: argument
marshalling only, as binding.py does it for the other entry points.

Codes are torch.float8_e4m3fn tensors of the operand's shape whose rows may be padded: a row's
values are neighbours, rows are a multiple of 16 bytes apart and start on 16-byte boundaries (a
contiguous tensor whose row length is a multiple of 16 is fine as it is). Layouts, formulas and
rules: include/gemm.h.
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import binding as _binding
from .binding import _call, _check, _empty, _need, load_library

F8_BLOCK = 128  # values that share a scale
F8_KINDS = {"rows": 0, "columns": 1, "tiles": 2}
_F8 = torch.float8_e4m3fn
_NAMES = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}
_SCORES = ("softmax", "sigmoid")

Stream = Optional[torch.cuda.Stream]


def _blocks(n: int) -> int:
    return (n + F8_BLOCK - 1) // F8_BLOCK


def _name(dtype) -> str:
    try:
        return _NAMES[dtype]
    except (KeyError, TypeError):
        raise ValueError("the type must be torch.float32, torch.bfloat16 or torch.float16, "
                         f"got {dtype}") from None


def _tensor(name: str, t, dims: int) -> torch.Size:
    """The shape of a contiguous CUDA tensor with so many dimensions."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != dims or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dims}-D tensor")
    return t.shape


def _whole(name: str, v, low: int, high: int) -> int:
    if isinstance(v, bool) or not isinstance(v, int) or not low <= v <= high:
        raise ValueError(f"{name} must be a whole number from {low} to {high}, got {v!r}")
    return v


def _codes(name: str, t, dims: int = 2, device: int = -1) -> int:
    """Checks codes (on the device with that index) and returns the bytes between their rows."""
    # One look at what a call that is in order passes (a decoded token's call takes little
    # longer than its kernel); what fails it is looked at part by part for its message.
    if type(t) is torch.Tensor and t.dtype is _F8 and t.dim() == dims and t.get_device() == device:
        shape, strides = t.shape, t.stride()
        cols, rows, ld = shape[-1], shape[-2], strides[-2]
        if rows == 1 and dims == 2:
            ld = (cols + 15) // 16 * 16
        if (strides[-1] == 1 and ld % 16 == 0 and ld >= cols > 1 and rows > 0
                and t.data_ptr() % 16 == 0
                and (dims == 2 or (rows > 1 and strides[0] == rows * ld and shape[0] > 0))):
            return ld
    return _codes_in_detail(name, t, dims, device)


def _codes_in_detail(name: str, t, dims: int, device: int) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != _F8:
        raise ValueError(f"{name} must be {_F8}, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must be a {dims}-D tensor, got {' x '.join(map(str, t.shape))}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}, got {t.device}")
    if t.numel() == 0:
        return (t.shape[-1] + 15) // 16 * 16
    rows, cols = t.shape[-2:]
    # The stride of a dimension of length 1 says nothing; any other one is the pitch as it is (0,
    # a repeated row's, is refused below).
    ld = (t.stride(-2) if rows > 1 else t.stride(-3) if dims == 3 and t.shape[0] > 1
          else (cols + 15) // 16 * 16)
    if ((cols > 1 and t.stride(-1) != 1) or ld % 16 or ld < cols or t.data_ptr() % 16
            or (dims == 3 and t.shape[0] > 1 and t.stride(0) != rows * ld)):
        raise ValueError(f"{name}: a row's codes must be neighbours, rows a multiple of 16 bytes "
                         "apart and on 16-byte boundaries, matrices one after another")
    return ld


def _new_codes(like: torch.Tensor, shape, stream: Stream) -> torch.Tensor:
    """Memory for codes whose rows are padded to 16 bytes, as a view of the shape."""
    cols = shape[-1]
    pitch = (cols + 15) // 16 * 16
    held = _empty(like, (*shape[:-1], pitch), _F8, stream)
    return held if pitch == cols else held.narrow(-1, 0, cols)


def _index(t) -> int:
    """The index of a tensor's CUDA device, -1 where it is none."""
    return t.get_device() if isinstance(t, torch.Tensor) else -1


def _floats(name: str, t, shape, device: int) -> int:
    """Checks contiguous fp32 values of a shape and returns their address."""
    if (type(t) is torch.Tensor and t.dtype is torch.float32 and t.get_device() == device
            and t.shape == shape and t.is_contiguous()):
        return t.data_ptr()
    _need(name, t, torch.float32, shape, torch.device("cuda", device))
    return t.data_ptr()


def _out(out, like: torch.Tensor, shape, stream: Stream, dtype=torch.float32) -> torch.Tensor:
    if out is None:
        return _empty(like, shape, dtype, stream)
    _need("out", out, dtype, shape, like.device)
    return out


def gemm_f8_quantize(X: torch.Tensor, kind: str = "rows", gather: Optional[torch.Tensor] = None,
                     fan: int = 1, factors: Optional[torch.Tensor] = None, stream: Stream = None
                     ) -> Tuple[torch.Tensor, ...]:
    """(codes, scales) of an fp32, bf16 or fp16 M x K matrix in e4m3 with a power-of-two scale
    for 128 values of a row (kind "rows") or of a column ("columns"); "both": (codes, scales) of
    each, from one reading. With `gather` (int32) row i of the result is X's row gather[i] // fan,
    times factors.flatten()[gather[i]] where factors (fp32, M * fan of them) is given, and zeros
    where gather[i] names none: what gemm_route's rows and weights are for."""
    source, K = _tensor("X", X, 2)
    name = _name(X.dtype)
    if kind not in ("rows", "columns", "both"):
        raise ValueError(f"kind must be rows, columns or both, got {kind!r}")
    if type(fan) is not int or fan != 1:
        _whole("fan", fan, 1, 1 << 20)
    M = source
    if gather is not None:
        M = _tensor("gather", gather, 1)[0]
        _need("gather", gather, torch.int32, (M,), X.device)
    elif fan != 1 or factors is not None:
        raise ValueError("fan and factors go with gather")
    if factors is not None:
        if not isinstance(factors, torch.Tensor):
            raise ValueError("factors must be a CUDA tensor")
        if factors.numel() != source * fan:
            raise ValueError(f"factors must have {source * fan} values, got {factors.numel()}")
        _need("factors", factors, torch.float32, factors.shape, X.device)
    got, pointers = (), ()
    if kind != "columns":
        codes = _new_codes(X, (M, K), stream)
        scales = _empty(X, (M, _blocks(K)), torch.float32, stream)
        got, pointers = (codes, scales), (codes.data_ptr(), scales.data_ptr())
    else:
        pointers = (0, 0)
    if kind != "rows":
        codes = _new_codes(X, (M, K), stream)
        scales = _empty(X, (_blocks(M), K), torch.float32, stream)
        got, pointers = got + (codes, scales), pointers + (codes.data_ptr(), scales.data_ptr())
    else:
        pointers += (0, 0)
    _call(f"gemm_{name}_f8_quantize", X.get_device(), stream, M, K, X.data_ptr(), source,
          0 if gather is None else gather.data_ptr(), fan,
          0 if factors is None else factors.data_ptr(), *pointers)
    return got


def gemm_f8_quantize_tiles(W: torch.Tensor, stream: Stream = None
                           ) -> Tuple[torch.Tensor, torch.Tensor]:
    """(codes, scales) of an fp32, bf16 or fp16 weight, K x N or E x K x N, in e4m3 with a
    power-of-two scale for each 128 x 128 tile."""
    shape = _tensor("W", W, 3 if isinstance(W, torch.Tensor) and W.dim() == 3 else 2)
    name = _name(W.dtype)
    E = shape[0] if len(shape) == 3 else 1
    K, N = shape[-2:]
    codes = _new_codes(W, tuple(shape), stream)
    scales = _empty(W, (*shape[:-2], _blocks(K), _blocks(N)), torch.float32, stream)
    _call(f"gemm_{name}_f8_quantize_tiles", W.get_device(), stream, E, K, N, W.data_ptr(),
          codes.data_ptr(), scales.data_ptr())
    return codes, scales


def gemm_f8_dequantize(codes: torch.Tensor, scales: torch.Tensor, kind: str = "rows",
                       dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                       stream: Stream = None) -> torch.Tensor:
    """The values codes * scales in `dtype` (fp32, bf16 or fp16) of codes held by "rows",
    "columns" or "tiles" (these E x K x N too)."""
    name = _name(dtype)
    if kind not in F8_KINDS:
        raise ValueError(f"kind must be one of {tuple(F8_KINDS)}, got {kind!r}")
    dims = 3 if kind == "tiles" and isinstance(codes, torch.Tensor) and codes.dim() == 3 else 2
    device = _index(codes)
    ld = _codes("codes", codes, dims, device)
    shape = codes.shape
    M, K = shape[-2:]
    held = ((M, _blocks(K)) if kind == "rows" else (_blocks(M), K) if kind == "columns"
            else (*shape[:-2], _blocks(M), _blocks(K)))
    scales_at = _floats("scales", scales, held, device)
    out = _out(out, codes, shape, stream, dtype)
    _call(f"gemm_{name}_f8_dequantize", device, stream, shape[0] if dims == 3 else 1, M, K,
          F8_KINDS[kind], codes.data_ptr(), ld, scales_at, out.data_ptr())
    return out


_FORWARD, _INPUT, _WEIGHT = "gemm_f8w8f32", "gemm_f8w8tf32", "gemm_f8tf8f32"


def _product(entry: str, names, A, a_scales, B, b_scales, out, stream: Stream,
             offsets=None, experts: bool = False):
    """Checks both operands of a product, names (A's, B's), and makes the call."""
    weight = entry is _WEIGHT
    device = _index(A)
    lda = _codes(names[0], A, 2, device)
    ldb = _codes(names[1], B, 3 if experts and not weight else 2, device)
    rows, mid = A.shape
    shape = B.shape
    K, N = shape[-2:]
    head = ()
    if experts:
        count = _tensor("offsets", offsets, 1)[0]
        _need("offsets", offsets, torch.int32, (count,), A.device)
        E = count - 1 if weight else shape[0]
        if count != E + 1 or E < 1:
            raise ValueError(f"offsets must have an entry more than there are experts, got {count}")
        head = (E, offsets.data_ptr())
    # sizes M (R), N, K as the C entry names them
    if weight:
        if shape[0] != rows:
            raise ValueError(f"{names[0]} and {names[1]} must have as many rows, got {rows} and "
                             f"{shape[0]}")
        K = mid
        a_shape, b_shape = (_blocks(rows), K), (_blocks(rows), N)
        result = (E, K, N) if experts else (K, N)
    else:
        if mid != (K if entry is _FORWARD else N):
            raise ValueError(f"{names[0]} is {rows} x {mid}, {names[1]} {K} x {N}: the sizes "
                             "summed over differ")
        a_shape, b_shape = (rows, _blocks(mid)), (*shape[:-2], _blocks(K), _blocks(N))
        result = (rows, N if entry is _FORWARD else K)
    a_at = _floats(f"{names[0]}'s scales", a_scales, a_shape, device)
    b_at = _floats(f"{names[1]}'s scales", b_scales, b_shape, device)
    out = _out(out, A, result, stream)
    _call(f"{entry}_experts" if experts else entry, device, stream, rows, N, K, *head,
          A.data_ptr(), lda, a_at, B.data_ptr(), ldb, b_at, out.data_ptr())
    return out


def gemm_f8w8f32(A: torch.Tensor, a_scales: torch.Tensor, W: torch.Tensor, w_scales: torch.Tensor,
                 out: Optional[torch.Tensor] = None, stream: Stream = None) -> torch.Tensor:
    """C = A @ W (fp32): A (M x K) as gemm_f8_quantize holds it by rows, W (K x N) by tiles."""
    return _product(_FORWARD, ("A", "W"), A, a_scales, W, w_scales, out, stream)


def gemm_f8w8tf32(dY: torch.Tensor, y_scales: torch.Tensor, W: torch.Tensor,
                  w_scales: torch.Tensor, out: Optional[torch.Tensor] = None,
                  stream: Stream = None) -> torch.Tensor:
    """dX = dY @ W^T (fp32), the input's gradient: dY (M x N) by rows, W (K x N) by tiles."""
    return _product(_INPUT, ("dY", "W"), dY, y_scales, W, w_scales, out, stream)


def gemm_f8tf8f32(X: torch.Tensor, x_scales: torch.Tensor, dY: torch.Tensor,
                  y_scales: torch.Tensor, out: Optional[torch.Tensor] = None,
                  stream: Stream = None) -> torch.Tensor:
    """dW = X^T @ dY (K x N, fp32), the weight's gradient: X (M x K) and dY (M x N) by columns."""
    return _product(_WEIGHT, ("X", "dY"), X, x_scales, dY, y_scales, out, stream)


def gemm_f8w8f32_experts(A: torch.Tensor, a_scales: torch.Tensor, W: torch.Tensor,
                         w_scales: torch.Tensor, offsets: torch.Tensor,
                         out: Optional[torch.Tensor] = None, stream: Stream = None) -> torch.Tensor:
    """gemm_f8w8f32 of each expert: rows offsets[e] .. offsets[e + 1] - 1 of A (R x K) times W[e]
    (W: E x K x N). Rows of the result in no expert's part are left as they were."""
    return _product(_FORWARD, ("A", "W"), A, a_scales, W, w_scales, out, stream,
                    offsets, True)


def gemm_f8w8tf32_experts(dY: torch.Tensor, y_scales: torch.Tensor, W: torch.Tensor,
                          w_scales: torch.Tensor, offsets: torch.Tensor,
                          out: Optional[torch.Tensor] = None, stream: Stream = None
                          ) -> torch.Tensor:
    """gemm_f8w8tf32 of each expert: its rows of dY (R x N) times W[e]^T."""
    return _product(_INPUT, ("dY", "W"), dY, y_scales, W, w_scales, out, stream,
                    offsets, True)


def gemm_f8tf8f32_experts(X: torch.Tensor, x_scales: torch.Tensor, dY: torch.Tensor,
                          y_scales: torch.Tensor, offsets: torch.Tensor,
                          out: Optional[torch.Tensor] = None, stream: Stream = None
                          ) -> torch.Tensor:
    """gemm_f8tf8f32 of each expert (E x K x N, fp32) over its rows of X (R x K) and dY (R x N);
    zeros for an expert without rows. The offsets are multiples of 128 (gemm_route's align)."""
    return _product(_WEIGHT, ("X", "dY"), X, x_scales, dY, y_scales, out, stream,
                    offsets, True)


def gemm_f8w8f32_selftest_timeout(A, a_scales, W, w_scales, out: torch.Tensor,
                                  wait_limit_ns: int) -> None:
    """Launch gemm_f8w8f32's kernel with its loads muted so every bounded wait runs out."""
    device = _index(A)
    lda, ldw = _codes("A", A, 2, device), _codes("W", W, 2, device)
    M, K = A.shape
    N = W.shape[1]
    a_at = _floats("A's scales", a_scales, (M, _blocks(K)), device)
    w_at = _floats("W's scales", w_scales, (_blocks(K), _blocks(N)), device)
    _need("out", out, torch.float32, (M, N), A.device)
    _call("gemm_f8w8f32_selftest_timeout", device, None, M, N, K, A.data_ptr(), lda, a_at,
          W.data_ptr(), ldw, w_at, out.data_ptr(), int(wait_limit_ns))


# ---------------------------------------------------------------- routing and joining


def gemm_route_rows(T: int, E: int, k: int, align: int = 128) -> int:
    """Entries of gemm_route's rows: the most that any routing of T tokens to k of E needs."""
    n = int(load_library().gemm_route_rows(int(T), int(E), int(k), int(align)))
    _check(n if n < 0 else 0)
    return n


def _route_rows(T: int, E: int, k: int, align: int) -> int:
    """gemm_route_rows of sizes in order, without a call into the library."""
    return T * k + min(E, T * k) * (align - 1)


def _score(score) -> int:
    if score not in _SCORES:
        raise ValueError(f"score must be one of {_SCORES}, got {score!r}")
    return _SCORES.index(score)


def gemm_route(logits: torch.Tensor, k: int, bias: Optional[torch.Tensor] = None,
               score: str = "softmax", groups: int = 1, top_groups: int = 1,
               renormalise: bool = True, scale: float = 1.0, align: int = 128,
               stream: Stream = None) -> Tuple[torch.Tensor, ...]:
    """(experts, weights, slots, rows, offsets) of T tokens from their logits (T x E; fp32, bf16
    or fp16): each token's k best experts by score + bias (int32, T x k), their weights (fp32,
    T x k: the scores, renormalised to sum to `scale` or times it), and the order by expert that
    the experts' products work in, each expert's part padded to a multiple of `align`: a slot's
    row (slots, T x k), the slot of each row (rows, -1 for none), and where each expert's rows
    start (offsets, E + 1). With groups > 1 only the experts of the top_groups groups whose two
    best scores sum highest take part. 128 rows aligned is what gemm_f8tf8f32_experts needs; 1
    makes the shortest order."""
    T, E = _tensor("logits", logits, 2)
    name = _name(logits.dtype)
    for what, v, most in (("k", k, 32), ("groups", groups, 32), ("top_groups", top_groups, 32),
                          ("align", align, 1024)):
        if type(v) is not int or not 1 <= v <= most:
            _whole(what, v, 1, most)
    sigmoid = _score(score)
    if bias is not None:
        _need("bias", bias, torch.float32, (E,), logits.device)
    R = _route_rows(T, E, k, align)
    need = int((_binding._lib or load_library()).gemm_route_workspace_bytes(T, E))
    experts = _empty(logits, (T, k), torch.int32, stream)
    slots = _empty(logits, (T, k), torch.int32, stream)
    weights = _empty(logits, (T, k), torch.float32, stream)
    rows = _empty(logits, (R,), torch.int32, stream)
    offsets = _empty(logits, (E + 1,), torch.int32, stream)
    workspace = _empty(logits, (need // 4,), torch.int32, stream) if need > 0 else None
    _call(f"gemm_{name}_route", logits.get_device(), stream, T, E, k, logits.data_ptr(),
          0 if bias is None else bias.data_ptr(), groups, top_groups, sigmoid,
          1 if renormalise else 0, float(scale), align, experts.data_ptr(), weights.data_ptr(),
          slots.data_ptr(), rows.data_ptr(), offsets.data_ptr(),
          0 if workspace is None else workspace.data_ptr(), max(need, 0))
    return experts, weights, slots, rows, offsets


def gemm_route_backward(logits: torch.Tensor, experts: torch.Tensor, dweights: torch.Tensor,
                        score: str = "softmax", renormalise: bool = True, scale: float = 1.0,
                        out: Optional[torch.Tensor] = None, stream: Stream = None) -> torch.Tensor:
    """dlogits (T x E, fp32) from the gradient of gemm_route's weights and the experts it chose."""
    T, E = _tensor("logits", logits, 2)
    name = _name(logits.dtype)
    k = _tensor("experts", experts, 2)[1]
    _need("experts", experts, torch.int32, (T, k), logits.device)
    _need("dweights", dweights, torch.float32, (T, k), logits.device)
    sigmoid = _score(score)
    out = _out(out, logits, (T, E), stream)
    _call(f"gemm_{name}_route_backward", logits.get_device(), stream, T, E, k, logits.data_ptr(),
          sigmoid, 1 if renormalise else 0, float(scale), experts.data_ptr(), dweights.data_ptr(),
          out.data_ptr())
    return out


def gemm_experts_join(C: torch.Tensor, slots: torch.Tensor, weights: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, stream: Stream = None) -> torch.Tensor:
    """Y (T x N, fp32) = sum over j of weights[t][j] * C[slots[t][j]]: the experts' products back
    in the tokens' order. Without weights the plain sum (an input's gradient)."""
    R, N = _tensor("C", C, 2)
    _need("C", C, torch.float32, (R, N))
    T, k = _tensor("slots", slots, 2)
    _need("slots", slots, torch.int32, (T, k), C.device)
    if weights is not None:
        _need("weights", weights, torch.float32, (T, k), C.device)
    out = _out(out, C, (T, N), stream)
    _call("gemm_experts_join", C.get_device(), stream, T, N, k, R, C.data_ptr(), slots.data_ptr(),
          0 if weights is None else weights.data_ptr(), out.data_ptr())
    return out


def gemm_experts_join_backward(dY: torch.Tensor, C: torch.Tensor, slots: torch.Tensor,
                               out: Optional[torch.Tensor] = None, stream: Stream = None
                               ) -> torch.Tensor:
    """dweights (T x k, fp32): dweights[t][j] = dY[t] . C[slots[t][j]], dY fp32, bf16 or fp16."""
    T, N = _tensor("dY", dY, 2)
    name = _name(dY.dtype)
    R = _tensor("C", C, 2)[0]
    _need("C", C, torch.float32, (R, N), dY.device)
    k = _tensor("slots", slots, 2)[1]
    _need("slots", slots, torch.int32, (T, k), dY.device)
    out = _out(out, dY, (T, k), stream)
    _call(f"gemm_{name}_experts_join_backward", dY.get_device(), stream, T, N, k, R,
          dY.data_ptr(), C.data_ptr(), slots.data_ptr(), out.data_ptr())
    return out
