"""Python binding of ``libmxfp4.so`` (the C ABI in include/mxfp4.h): the MXFP4
linear layer and its mixture-of-experts form.

Argument marshalling only, as in ``w4a16``: torch supplies device memory and
the current stream, the library's HIP kernels compute.  There is no fallback:
a missing library or a non-gfx950 device is an error.

    codes, scales = quantize(W)                 # W [N, K] fp16 / bf16 / fp32
    Y = linear(X, codes, scales)                # X [M, K] fp16 / bf16 -> [M, N]
    a, sa = quantize(X)
    Y = matmul(a, sa, codes, scales)            # both operands in 4 bits

    ids, weights = route(logits, k)             # logits [T, E]
    p = plan(ids, E)                            # rows ordered by expert
    H = grouped_linear(X, c1, s1, p.offsets, tokens=p.tokens, swiglu=True)
    H = grouped_linear(H, c2, s2, p.offsets, dtype=torch.float32)
    out = combine(H, p.positions, weights, dtype=X.dtype)       # [T, N]
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple

import torch

LIBRARY = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmxfp4.so")

BLOCK = 32                       # columns per scale
MAX_EXPERTS = 1024
MAX_CHOICES = 32
_FLOATS = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
_HALVES = {torch.float16: 0, torch.bfloat16: 1}
_FP32_ROWS = 16                  # added to a dtype: the experts' rows are fp32

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_size = ctypes.c_size_t
_SIGNATURES = {
    "mxfp4_quantize": [_p, _int, _i64, _i64, _i64, _p, _p, _p],
    "mxfp4_dequantize": [_p, _p, _i64, _i64, _p, _int, _p],
    "mxfp4_linear": [_p, _int, _i64, _i64, _p, _p, _i64, _i64, _p, _p, _size, _p],
    "mxfp4_matmul": [_p, _p, _i64, _p, _p, _i64, _i64, _p, _int, _p, _size, _p],
    "mxfp4_grouped_linear": [_p, _int, _i64, _i64, _p, _i64, _p, _p, _p, _i64, _i64, _i64, _int,
                             _p, _p],
    "moe_route": [_p, _int, _i64, _i64, _i64, _i64, _int, _p, _p, _p],
    "moe_plan": [_p, _i64, _i64, _i64, _p, _p, _p, _p, _size, _p],
    "moe_combine": [_p, _int, _i64, _i64, _p, _p, _i64, _i64, _p, _p],
}
_SIZES = ("mxfp4_linear_workspace_bytes", "mxfp4_matmul_workspace_bytes",
          "moe_plan_workspace_bytes")
_lib = None


class MXFP4Error(RuntimeError):
    """A non-zero status from the library."""

    def __init__(self, fn: str, status: int):
        super().__init__("%s failed: status %d (%s)" % (fn, status, status_string(status)))
        self.status = status


def library() -> ctypes.CDLL:
    """The loaded library (loaded on first use; raises if it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIBRARY):
            raise ImportError("%s is not built: run python -m weight_only_int4_gemv_amd.build"
                              % LIBRARY)
        lib = ctypes.CDLL(LIBRARY)
        for name, args in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, _int
        for name in _SIZES:
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = [_i64, _i64, _i64], _size
        lib.mxfp4_status_string.argtypes = [_int]
        lib.mxfp4_status_string.restype = ctypes.c_char_p
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return library().mxfp4_status_string(int(status)).decode()


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise MXFP4Error(fn, status)


def _need(t, name: str, dtypes, ndim: int, dense: bool = True) -> None:
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.is_cuda
            and (not ndim or t.dim() == ndim) and (not dense or t.is_contiguous())):
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a torch.Tensor" % name)
    if t.dtype not in dtypes:
        raise ValueError("%s must be one of %s, got %s"
                         % (name, ", ".join(str(d) for d in dtypes), t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be on the GPU, got %s" % (name, t.device))
    if ndim and t.dim() != ndim:
        raise ValueError("%s must have %d dims, got shape %s" % (name, ndim, tuple(t.shape)))
    if dense and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


_U8 = (torch.uint8,)
_I32 = (torch.int32,)
_F32 = (torch.float32,)


def _stream(*tensors) -> int:
    """The current stream; every tensor has to be on its device."""
    index = torch.cuda.current_device()
    for t in tensors:
        if t.get_device() != index:
            raise ValueError("tensors must be on the current device cuda:%d, got %s"
                             % (index, t.device))
    # The handle alone: torch.cuda.current_stream builds a Stream object first,
    # 1 us of the 8 a small call takes.
    return torch._C._cuda_getCurrentRawStream(index)


def _row_stride(t: torch.Tensor, name: str) -> int:
    """Elements between the rows of a 2-d tensor whose rows are dense."""
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError("the rows of %s must be dense, got strides %s" % (name, t.stride()))
    if rows <= 1 or cols == 0:
        return cols
    if t.stride(0) < cols:
        raise ValueError("the rows of %s overlap: strides %s" % (name, t.stride()))
    return t.stride(0)


def _out(t, shape, dtype, like: torch.Tensor, name: str) -> torch.Tensor:
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    _need(t, name, (dtype,), len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, want %s" % (name, tuple(t.shape), tuple(shape)))
    return t


def _weights(codes: torch.Tensor, scales: torch.Tensor, ndim: int, name: str = ""):
    """The shape [..., K] of an MXFP4 matrix."""
    _need(codes, name + "codes", _U8, ndim)
    _need(scales, name + "scales", _U8, ndim)
    *lead, half = codes.shape
    K = half * 2
    if K % BLOCK or scales.shape != (*lead, K // BLOCK):
        raise ValueError("%sscales shape %s does not match %scodes %s (blocks of %d columns)"
                         % (name, tuple(scales.shape), name, tuple(codes.shape), BLOCK))
    return (*lead, K)


def quantize(X: torch.Tensor, codes: torch.Tensor = None, scales: torch.Tensor = None):
    """X fp16, bf16 or fp32 [..., K] -> (codes uint8 [..., K/2], scales uint8
    [..., K/32]); K % 32 == 0.  X is dense, or 2-d with dense rows further apart
    (a row stride of whole 16 bytes).  A block with an infinity or a NaN gets the
    NaN scale 255."""
    lib = library()
    _need(X, "X", _FLOATS, 0, dense=False)
    if X.dim() < 1 or X.shape[-1] % BLOCK:
        raise ValueError("the last dim of X must be a multiple of %d, got shape %s"
                         % (BLOCK, tuple(X.shape)))
    K = X.shape[-1]
    if X.dim() == 2:
        rows, stride = X.shape[0], _row_stride(X, "X")
    else:
        _need(X, "X", _FLOATS, 0)
        rows, stride = (X.numel() // K if K else 0), K
    lead = tuple(X.shape[:-1])
    codes = _out(codes, lead + (K // 2,), torch.uint8, X, "codes")
    scales = _out(scales, lead + (K // BLOCK,), torch.uint8, X, "scales")
    _check("mxfp4_quantize",
           lib.mxfp4_quantize(X.data_ptr(), _FLOATS[X.dtype], rows, K, stride, codes.data_ptr(),
                              scales.data_ptr(), _stream(X, codes, scales)))
    return codes, scales


def dequantize(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
               Y: torch.Tensor = None) -> torch.Tensor:
    """The values of MXFP4 codes and scales, [..., K] of dtype (fp16, bf16, fp32).
    Y starts on 16 bytes."""
    lib = library()
    if dtype not in _FLOATS:
        raise ValueError("dtype must be fp16, bf16 or fp32, got %s" % dtype)
    shape = _weights(codes, scales, 0)
    Y = _out(Y, shape, dtype, codes, "Y")
    K = shape[-1]
    _check("mxfp4_dequantize",
           lib.mxfp4_dequantize(codes.data_ptr(), scales.data_ptr(),
                                Y.numel() // K if K else 0, K, Y.data_ptr(), _FLOATS[dtype],
                                _stream(codes, scales, Y)))
    return Y


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(fn: str, a: int, b: int, c: int) -> int:
    return getattr(library(), fn)(a, b, c)


def _workspace(need: int, given, like: torch.Tensor):
    """(pointer, bytes, tensors to check) of a workspace: the caller's, or one
    from torch's allocator, which holds it for the current stream's order."""
    if given is not None:
        _need(given, "workspace", _U8, 1)
        return given.data_ptr(), given.numel(), (given,)
    if need == 0:
        return None, 0, ()
    ws = like.new_empty(need, dtype=torch.uint8)
    return ws.data_ptr(), need, (ws,)


def linear_workspace(M: int, N: int, K: int, device="cuda") -> torch.Tensor:
    """A workspace for linear() (uint8, at least 1 byte)."""
    n = _workspace_bytes("mxfp4_linear_workspace_bytes", M, N, K)
    return torch.empty(max(1, n), dtype=torch.uint8, device=device)


def linear(X: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, Y: torch.Tensor = None,
           workspace: torch.Tensor = None) -> torch.Tensor:
    """X fp16 or bf16 [M, K] times MXFP4 weights [N, K] -> Y [M, N] of X's dtype.
    X's rows are dense and a multiple of 8 elements apart.  workspace: from
    linear_workspace(), else allocated per call where the shape uses one."""
    lib = library()
    N, K = _weights(codes, scales, 2)
    _need(X, "X", _HALVES, 2, dense=False)
    M = X.shape[0]
    if X.shape[1] != K:
        raise ValueError("X has %d columns, K = %d" % (X.shape[1], K))
    stride = _row_stride(X, "X")
    Y = _out(Y, (M, N), X.dtype, X, "Y")
    ws, ws_bytes, keep = _workspace(_workspace_bytes("mxfp4_linear_workspace_bytes", M, N, K),
                                    workspace, X)
    _check("mxfp4_linear",
           lib.mxfp4_linear(X.data_ptr(), _HALVES[X.dtype], M, stride, codes.data_ptr(),
                            scales.data_ptr(), N, K, Y.data_ptr(), ws, ws_bytes,
                            _stream(X, codes, scales, Y, *keep)))
    return Y


def matmul_workspace(M: int, N: int, K: int, device="cuda") -> torch.Tensor:
    """A workspace for matmul() (uint8, at least 1 byte)."""
    n = _workspace_bytes("mxfp4_matmul_workspace_bytes", M, N, K)
    return torch.empty(max(1, n), dtype=torch.uint8, device=device)


def matmul(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor,
           b_scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16, Y: torch.Tensor = None,
           workspace: torch.Tensor = None) -> torch.Tensor:
    """MXFP4 A [M, K] times MXFP4 B [N, K], Y[m, n] = sum_k A[m, k] B[n, k], of
    dtype fp16, bf16 or fp32.  workspace: from matmul_workspace(), else
    allocated per call where the shape uses one."""
    lib = library()
    if dtype not in _FLOATS:
        raise ValueError("dtype must be fp16, bf16 or fp32, got %s" % dtype)
    M, K = _weights(a_codes, a_scales, 2, "a_")
    N, Kb = _weights(b_codes, b_scales, 2, "b_")
    if K != Kb:
        raise ValueError("A has %d columns, B has %d" % (K, Kb))
    Y = _out(Y, (M, N), dtype, a_codes, "Y")
    ws, ws_bytes, keep = _workspace(_workspace_bytes("mxfp4_matmul_workspace_bytes", M, N, K),
                                    workspace, a_codes)
    _check("mxfp4_matmul",
           lib.mxfp4_matmul(a_codes.data_ptr(), a_scales.data_ptr(), M, b_codes.data_ptr(),
                            b_scales.data_ptr(), N, K, Y.data_ptr(), _FLOATS[dtype], ws, ws_bytes,
                            _stream(a_codes, a_scales, b_codes, b_scales, Y,
                                    *keep)))
    return Y


def route(logits: torch.Tensor, k: int, renormalize: bool = True, ids: torch.Tensor = None,
          weights: torch.Tensor = None):
    """Router logits [T, E] (fp16, bf16 or fp32, dense rows) -> (ids int32 [T, k],
    weights fp32 [T, k]): the k largest logits of each token in falling order,
    ties to the lowest expert, and their softmax over the chosen (renormalize)
    or over all experts.  Experts at -inf are never chosen: id -1, weight 0."""
    lib = library()
    _need(logits, "logits", _FLOATS, 2, dense=False)
    T, E = logits.shape
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError("logits have %d experts, want 1 to %d" % (E, MAX_EXPERTS))
    if not 1 <= k <= min(E, MAX_CHOICES):
        raise ValueError("k = %d, want 1 to min(%d experts, %d)" % (k, E, MAX_CHOICES))
    stride = _row_stride(logits, "logits")
    ids = _out(ids, (T, k), torch.int32, logits, "ids")
    weights = _out(weights, (T, k), torch.float32, logits, "weights")
    _check("moe_route",
           lib.moe_route(logits.data_ptr(), _FLOATS[logits.dtype], T, E, stride, k,
                         1 if renormalize else 0, ids.data_ptr(), weights.data_ptr(),
                         _stream(logits, ids, weights)))
    return ids, weights


class Plan(NamedTuple):
    """Choices ordered by expert: expert e owns the rows offsets[e] up to
    offsets[e + 1]; tokens[row] is a row's token (-1 from offsets[E] on),
    positions[t, j] the row of choice j of token t (-1: no choice)."""
    offsets: torch.Tensor       # int32 [E + 1]
    tokens: torch.Tensor        # int32 [T k]
    positions: torch.Tensor     # int32 [T, k]


def plan(ids: torch.Tensor, E: int, workspace: torch.Tensor = None) -> Plan:
    """ids int32 [T, k] -> Plan.  Ids outside [0, E) are no choice (a slice of
    the experts is planned by subtracting its first expert from the ids).
    workspace: uint8 of moe_plan_workspace_bytes, else allocated per call where
    the size uses one."""
    lib = library()
    _need(ids, "ids", _I32, 2)
    T, k = ids.shape
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError("E = %d, want 1 to %d" % (E, MAX_EXPERTS))
    if not 1 <= k <= MAX_CHOICES:
        raise ValueError("ids have %d choices a token, want 1 to %d" % (k, MAX_CHOICES))
    offsets, tokens, positions = ids.new_empty(E + 1), ids.new_empty(T * k), ids.new_empty((T, k))
    ws, ws_bytes, keep = _workspace(_workspace_bytes("moe_plan_workspace_bytes", T, k, E),
                                    workspace, ids)
    _check("moe_plan",
           lib.moe_plan(ids.data_ptr(), T, k, E, offsets.data_ptr(), tokens.data_ptr(),
                        positions.data_ptr(), ws, ws_bytes,
                        _stream(ids, *keep)))
    return Plan(offsets, tokens, positions)


def grouped_linear(X: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                   offsets: torch.Tensor, tokens: torch.Tensor = None, swiglu: bool = False,
                   Y: torch.Tensor = None, dtype: torch.dtype = None) -> torch.Tensor:
    """Row r of Y = its row of X (tokens[r], or r) times the MXFP4 weights
    [E, N, K] of the expert e with offsets[e] <= r < offsets[e + 1]; rows of no
    expert are 0.  Y is [R, N] of X's dtype, R = len(tokens) or X's rows.
    swiglu: the weights are gate rows, then up rows, and Y = silu(gate) * up
    is [R, N / 2].  dtype: Y's, X's (the default) or, without swiglu, fp32, for
    combine to round a token's sum once."""
    lib = library()
    E, N, K = _weights(codes, scales, 3)
    _need(X, "X", _HALVES, 2, dense=False)
    if X.shape[1] != K:
        raise ValueError("X has %d columns, K = %d" % (X.shape[1], K))
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError("codes hold %d experts, want 1 to %d" % (E, MAX_EXPERTS))
    if swiglu and N % 2:
        raise ValueError("swiglu takes an even number of weight rows, got %d" % N)
    if dtype not in (None, X.dtype) and (swiglu or dtype != torch.float32):
        raise ValueError("dtype must be %s%s, got %s"
                         % (X.dtype, "" if swiglu else " or torch.float32", dtype))
    rows32 = dtype == torch.float32
    _need(offsets, "offsets", _I32, 1)
    if offsets.shape[0] != E + 1:
        raise ValueError("offsets has %d entries, want %d" % (offsets.shape[0], E + 1))
    R = X.shape[0]
    if tokens is not None:
        _need(tokens, "tokens", _I32, 1)
        R = tokens.shape[0]
    stride = _row_stride(X, "X")
    Y = _out(Y, (R, N // 2 if swiglu else N), dtype or X.dtype, X, "Y")
    _check("mxfp4_grouped_linear",
           lib.mxfp4_grouped_linear(X.data_ptr(), _HALVES[X.dtype] + (_FP32_ROWS if rows32 else 0),
                                    X.shape[0], stride,
                                    tokens.data_ptr() if tokens is not None else None, R,
                                    codes.data_ptr(), scales.data_ptr(), offsets.data_ptr(), E, N,
                                    K, 1 if swiglu else 0, Y.data_ptr(),
                                    _stream(X, codes, scales, offsets, Y,
                                            *(() if tokens is None else (tokens,)))))
    return Y


def combine(Y: torch.Tensor, positions: torch.Tensor, weights: torch.Tensor,
            out: torch.Tensor = None, dtype: torch.dtype = None) -> torch.Tensor:
    """out[t] = sum over j of weights[t, j] * Y[positions[t, j]] (fp32 sums, j
    rising; a position outside Y adds nothing): Y fp16, bf16 or fp32 [R, N],
    positions int32 and weights fp32 [T, k] -> [T, N] of Y's dtype, for fp32 Y of
    dtype (fp16 or bf16)."""
    lib = library()
    _need(Y, "Y", _FLOATS, 2)
    rows32 = Y.dtype == torch.float32
    dtype = dtype or Y.dtype
    if dtype not in _HALVES or not rows32 and dtype != Y.dtype:
        raise ValueError("dtype must be %s, got %s"
                         % ("fp16 or bf16 for fp32 Y" if rows32 else Y.dtype, dtype))
    _need(positions, "positions", _I32, 2)
    _need(weights, "weights", _F32, 2)
    if positions.shape != weights.shape:
        raise ValueError("positions shape %s, weights %s"
                         % (tuple(positions.shape), tuple(weights.shape)))
    R, N = Y.shape
    T, k = positions.shape
    if not 1 <= k <= MAX_CHOICES:
        raise ValueError("positions have %d choices a token, want 1 to %d" % (k, MAX_CHOICES))
    out = _out(out, (T, N), dtype, Y, "out")
    _check("moe_combine",
           lib.moe_combine(Y.data_ptr(), _HALVES[dtype] + (_FP32_ROWS if rows32 else 0), R, N,
                           positions.data_ptr(), weights.data_ptr(), T, k, out.data_ptr(),
                           _stream(Y, positions, weights, out)))
    return out
