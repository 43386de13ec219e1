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

Products with an epilogue, and the backward pass (weights stay codes: gradients go to
activations, biases and the router):

    Y, Z = linear_act(X, codes, scales, bias, activation="gelu", residual=R, save=True)
    dZ, dbias = activation_grad(dY, Z, "gelu")
    dX = linear_grad(dZ, codes, scales)

    H, Z = grouped_linear_act(X, c1, s1, p.offsets, tokens=p.tokens, bias=b1,
                              activation="swiglu", save=True)
    rows, dweights = combine_grad(dout, Y, p.tokens, p.positions, weights)
    dH = grouped_linear_grad(rows, c2, s2, p.offsets)
    dZ, db1 = activation_grad(dH, Z, "swiglu", offsets=p.offsets)
    dX = grouped_linear_grad(dZ, c1, s1, p.offsets, dtype=torch.float32)
    dx = combine(dX, p.positions, torch.ones_like(weights), dtype=X.dtype)
    loss, counts = balance(logits, ids)
    dlogits = route_grad(logits, ids, dweights, counts=counts, dloss=dloss)
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
ACTIVATIONS = ("none", "relu", "silu", "gelu", "gelu_tanh", "swiglu")
_ACT = {name: i for i, name in enumerate(ACTIVATIONS)}
_SWIGLU = _ACT["swiglu"]

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
    "mxfp4_linear_act": [_p, _int, _i64, _i64, _p, _p, _i64, _i64, _p, _int, _p, _i64, _p, _p, _p,
                         _size, _p],
    "mxfp4_grouped_linear_act": [_p, _int, _i64, _i64, _p, _i64, _p, _p, _p, _i64, _i64, _i64, _p,
                                 _int, _p, _p, _p],
    "mxfp4_activation_grad": [_p, _int, _i64, _i64, _p, _i64, _i64, _int, _p, _i64, _p, _p, _p,
                              _size, _p],
    "mxfp4_linear_grad": [_p, _int, _i64, _i64, _p, _p, _i64, _i64, _p, _p, _size, _p],
    "mxfp4_grouped_linear_grad": [_p, _int, _i64, _i64, _p, _p, _p, _i64, _i64, _i64, _p, _p],
    "moe_balance": [_p, _int, _i64, _i64, _i64, _p, _i64, _p, _p, _p, _size, _p],
    "moe_route_grad": [_p, _int, _i64, _i64, _i64, _p, _i64, _p, _int, _p, _p, _p, _p],
    "moe_combine_grad": [_p, _int, _i64, _i64, _p, _i64, _p, _p, _p, _i64, _p, _p, _p],
}
_SIZES = ("mxfp4_linear_workspace_bytes", "mxfp4_matmul_workspace_bytes",
          "moe_plan_workspace_bytes", "mxfp4_linear_act_workspace_bytes",
          "mxfp4_activation_grad_workspace_bytes",
          "mxfp4_linear_grad_workspace_bytes", "moe_balance_workspace_bytes")
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
    if t.is_contiguous():
        return t.shape[1]
    rows, cols = t.shape
    if rows and cols > 1 and t.stride(1) != 1:
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


def _out_like(t, like: torch.Tensor, name: str) -> torch.Tensor:
    """_out() with the shape and dtype of `like`: 0.4 us less where that is contiguous."""
    if t is None and like.is_contiguous():
        return torch.empty_like(like)
    return _out(t, like.shape, like.dtype, like, name)


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


# ------------------------------------------- products with an epilogue, gradients

def _activation(name, N: int) -> int:
    act = _ACT.get("none" if name is None else name)
    if act is None:
        raise ValueError("activation must be one of %s, got %r" % (", ".join(ACTIVATIONS), name))
    if act == _SWIGLU and N % 2:
        raise ValueError("swiglu takes an even number of gate and up columns, got %d" % N)
    return act


def _ptr(t):
    return None if t is None else t.data_ptr()


def _given(*tensors):
    return tuple(t for t in tensors if t is not None)


def _bias(bias, shape, X: torch.Tensor) -> None:
    if bias is None:
        return
    _need(bias, "bias", (X.dtype,), len(shape))
    if tuple(bias.shape) != shape:
        raise ValueError("bias has shape %s, want %s" % (tuple(bias.shape), shape))


def linear_act_workspace(M: int, N: int, K: int, device="cuda") -> torch.Tensor:
    """A workspace for linear_act() (uint8, at least 1 byte)."""
    n = _workspace_bytes("mxfp4_linear_act_workspace_bytes", M, N, K)
    return torch.empty(max(1, n), dtype=torch.uint8, device=device)


def linear_act(X: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
               bias: torch.Tensor = None, activation: str = None, residual: torch.Tensor = None,
               save: bool = False, Y: torch.Tensor = None, Z: torch.Tensor = None,
               workspace: torch.Tensor = None):
    """Y = activation(X W^T + bias) + residual: X fp16 or bf16 [M, K] (rows as in
    linear()), MXFP4 weights [N, K], bias [N] and residual [M, F] (dense rows) of X's
    dtype or None.  activation: one of ACTIVATIONS; swiglu takes weights of gate rows,
    then up rows, F = N / 2, otherwise F = N.  Y [M, F] is of X's dtype; with save (or
    Z given) the result is (Y, Z), Z [M, N] what the activation was applied to.
    workspace: from linear_act_workspace(), else allocated per call where the shape uses
    one."""
    lib = library()
    N, K = _weights(codes, scales, 2)
    _need(X, "X", _HALVES, 2, dense=False)
    M = X.shape[0]
    if X.shape[1] != K:
        raise ValueError("X has %d columns, K = %d" % (X.shape[1], K))
    act = _activation(activation, N)
    F = N // 2 if act == _SWIGLU else N
    stride = _row_stride(X, "X")
    _bias(bias, (N,), X)
    r_stride = F
    if residual is not None:
        _need(residual, "residual", (X.dtype,), 2, dense=False)
        if tuple(residual.shape) != (M, F):
            raise ValueError("residual has shape %s, want %s" % (tuple(residual.shape), (M, F)))
        r_stride = _row_stride(residual, "residual")
    Y = _out(Y, (M, F), X.dtype, X, "Y")
    save = save or Z is not None
    if save:
        Z = _out(Z, (M, N), X.dtype, X, "Z")
    ws, ws_bytes, keep = _workspace(_workspace_bytes("mxfp4_linear_act_workspace_bytes", M, N, K),
                                    workspace, X)
    _check("mxfp4_linear_act",
           lib.mxfp4_linear_act(X.data_ptr(), _HALVES[X.dtype], M, stride, codes.data_ptr(),
                                scales.data_ptr(), N, K, _ptr(bias), act, _ptr(residual), r_stride,
                                Y.data_ptr(), _ptr(Z), ws, ws_bytes,
                                _stream(X, codes, scales, Y, *_given(bias, residual, Z), *keep)))
    return (Y, Z) if save else Y


def grouped_linear_act(X: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                       offsets: torch.Tensor, tokens: torch.Tensor = None,
                       bias: torch.Tensor = None, activation: str = None, save: bool = False,
                       Y: torch.Tensor = None, Z: torch.Tensor = None,
                       dtype: torch.dtype = None):
    """grouped_linear() with the epilogue of linear_act() (no residual), each expert
    with its bias, [E, N] of X's dtype or None.  Y [R, F] of dtype: X's (the default)
    or fp32; with save (or Z given) the result is (Y, Z), Z [R, N] of X's dtype.  Rows
    of no expert are 0 in both."""
    lib = library()
    E, N, K = _weights(codes, scales, 3)
    _need(X, "X", _HALVES, 2, dense=False)
    if X.shape[1] != K:
        raise ValueError("X has %d columns, K = %d" % (X.shape[1], K))
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError("codes hold %d experts, want 1 to %d" % (E, MAX_EXPERTS))
    act = _activation(activation, N)
    F = N // 2 if act == _SWIGLU else N
    if dtype not in (None, X.dtype, torch.float32):
        raise ValueError("dtype must be %s or torch.float32, got %s" % (X.dtype, dtype))
    rows32 = dtype == torch.float32
    _need(offsets, "offsets", _I32, 1)
    if offsets.shape[0] != E + 1:
        raise ValueError("offsets has %d entries, want %d" % (offsets.shape[0], E + 1))
    R = X.shape[0]
    if tokens is not None:
        _need(tokens, "tokens", _I32, 1)
        R = tokens.shape[0]
    stride = _row_stride(X, "X")
    _bias(bias, (E, N), X)
    Y = _out(Y, (R, F), dtype or X.dtype, X, "Y")
    save = save or Z is not None
    if save:
        Z = _out(Z, (R, N), X.dtype, X, "Z")
    _check("mxfp4_grouped_linear_act",
           lib.mxfp4_grouped_linear_act(X.data_ptr(),
                                        _HALVES[X.dtype] + (_FP32_ROWS if rows32 else 0),
                                        X.shape[0], stride, _ptr(tokens), R, codes.data_ptr(),
                                        scales.data_ptr(), offsets.data_ptr(), E, N, K,
                                        _ptr(bias), act, Y.data_ptr(), _ptr(Z),
                                        _stream(X, codes, scales, offsets, Y,
                                                *_given(tokens, bias, Z))))
    return (Y, Z) if save else Y


def activation_grad(dY: torch.Tensor, Z: torch.Tensor, activation: str,
                    offsets: torch.Tensor = None, bias: bool = True, dZ: torch.Tensor = None,
                    dbias: torch.Tensor = None, workspace: torch.Tensor = None):
    """dZ = dY * activation'(Z) and the bias's gradient, the sum of dZ's rows before
    their rounding: dY fp16 or bf16 [R, F] and Z [R, N] of that dtype (dense rows; F =
    N / 2 with swiglu) -> (dZ [R, N], dbias fp32 [N], with offsets int32 [E + 1] by
    expert, [E, N]); without bias dZ alone.  workspace: uint8 of
    mxfp4_activation_grad_workspace_bytes, else allocated per call where used."""
    lib = library()
    _need(dY, "dY", _HALVES, 2, dense=False)
    _need(Z, "Z", (dY.dtype,), 2, dense=False)
    R, N = Z.shape
    act = _activation(activation, N)
    F = N // 2 if act == _SWIGLU else N
    if tuple(dY.shape) != (R, F):
        raise ValueError("dY has shape %s, want %s" % (tuple(dY.shape), (R, F)))
    y_stride, z_stride = _row_stride(dY, "dY"), _row_stride(Z, "Z")
    E, shape = 0, (N,)
    if offsets is not None:
        _need(offsets, "offsets", _I32, 1)
        E = offsets.shape[0] - 1
        if not 1 <= E <= MAX_EXPERTS:
            raise ValueError("offsets are of %d experts, want 1 to %d" % (E, MAX_EXPERTS))
        shape = (E, N)
    dZ = _out_like(dZ, Z, "dZ")
    bias = bias or dbias is not None
    ws, ws_bytes, keep = None, 0, ()
    if bias:
        dbias = _out(dbias, shape, torch.float32, dY, "dbias")
        ws, ws_bytes, keep = _workspace(
            _workspace_bytes("mxfp4_activation_grad_workspace_bytes", R, N, E), workspace, dY)
    _check("mxfp4_activation_grad",
           lib.mxfp4_activation_grad(dY.data_ptr(), _HALVES[dY.dtype], R, y_stride, Z.data_ptr(),
                                     z_stride, N, act, _ptr(offsets), E, dZ.data_ptr(),
                                     _ptr(dbias), ws, ws_bytes,
                                     _stream(dY, Z, dZ, *_given(offsets, dbias), *keep)))
    return (dZ, dbias) if bias else dZ


def linear_grad_workspace(M: int, N: int, K: int, device="cuda") -> torch.Tensor:
    """A workspace for linear_grad() (uint8, at least 1 byte)."""
    n = _workspace_bytes("mxfp4_linear_grad_workspace_bytes", M, N, K)
    return torch.empty(max(1, n), dtype=torch.uint8, device=device)


def linear_grad(dY: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                dX: torch.Tensor = None, workspace: torch.Tensor = None) -> torch.Tensor:
    """The gradient of linear() with respect to X: dY fp16 or bf16 [M, N] (dense rows)
    times MXFP4 weights [N, K] -> dX [M, K] of dY's dtype, on 16 bytes.  More than
    16 rows are read fastest where N is a multiple of 8 and rows start on 16 bytes (3001 of
    them take three to four times as long elsewhere).  workspace: from linear_grad_workspace(), else
    allocated per call where the shape uses one."""
    lib = library()
    N, K = _weights(codes, scales, 2)
    _need(dY, "dY", _HALVES, 2, dense=False)
    M = dY.shape[0]
    if dY.shape[1] != N:
        raise ValueError("dY has %d columns, N = %d" % (dY.shape[1], N))
    stride = _row_stride(dY, "dY")
    dX = _out(dX, (M, K), dY.dtype, dY, "dX")
    ws, ws_bytes, keep = _workspace(_workspace_bytes("mxfp4_linear_grad_workspace_bytes", M, N, K),
                                    workspace, dY)
    _check("mxfp4_linear_grad",
           lib.mxfp4_linear_grad(dY.data_ptr(), _HALVES[dY.dtype], M, stride, codes.data_ptr(),
                                 scales.data_ptr(), N, K, dX.data_ptr(), ws, ws_bytes,
                                 _stream(dY, codes, scales, dX, *keep)))
    return dX


def grouped_linear_grad(dY: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                        offsets: torch.Tensor, dX: torch.Tensor = None,
                        dtype: torch.dtype = None) -> torch.Tensor:
    """The gradient of grouped_linear()'s product with respect to its rows: row r of dX
    = row r of dY (fp16 or bf16 [R, N]) times the MXFP4 weights [E, N, K] of its expert;
    rows of no expert are 0.  dX [R, K] of dtype: dY's (the default) or fp32, for
    combine() with weights of 1, which gives the gradient of a gathered X."""
    lib = library()
    E, N, K = _weights(codes, scales, 3)
    _need(dY, "dY", _HALVES, 2, dense=False)
    R = dY.shape[0]
    if dY.shape[1] != N:
        raise ValueError("dY has %d columns, N = %d" % (dY.shape[1], N))
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError("codes hold %d experts, want 1 to %d" % (E, MAX_EXPERTS))
    if dtype not in (None, dY.dtype, torch.float32):
        raise ValueError("dtype must be %s or torch.float32, got %s" % (dY.dtype, dtype))
    rows32 = dtype == torch.float32
    _need(offsets, "offsets", _I32, 1)
    if offsets.shape[0] != E + 1:
        raise ValueError("offsets has %d entries, want %d" % (offsets.shape[0], E + 1))
    stride = _row_stride(dY, "dY")
    dX = _out(dX, (R, K), dtype or dY.dtype, dY, "dX")
    _check("mxfp4_grouped_linear_grad",
           lib.mxfp4_grouped_linear_grad(dY.data_ptr(),
                                         _HALVES[dY.dtype] + (_FP32_ROWS if rows32 else 0), R,
                                         stride, codes.data_ptr(), scales.data_ptr(),
                                         offsets.data_ptr(), E, N, K, dX.data_ptr(),
                                         _stream(dY, codes, scales, offsets, dX)))
    return dX


def _router(logits: torch.Tensor, ids):
    """(T, E, k, row stride) of logits [T, E] and ids [T, k] (None: k = 1)."""
    _need(logits, "logits", _FLOATS, 2, dense=False)
    T, E = logits.shape
    if not 1 <= E <= MAX_EXPERTS:
        raise ValueError("logits have %d experts, want 1 to %d" % (E, MAX_EXPERTS))
    k = 1
    if ids is not None:
        _need(ids, "ids", _I32, 2)
        k = ids.shape[1]
        if ids.shape[0] != T or not 1 <= k <= MAX_CHOICES:
            raise ValueError("ids have shape %s, want (%d, 1 to %d)"
                             % (tuple(ids.shape), T, MAX_CHOICES))
    return T, E, k, _row_stride(logits, "logits")


def balance(logits: torch.Tensor, ids: torch.Tensor, loss: torch.Tensor = None,
            counts: torch.Tensor = None, workspace: torch.Tensor = None):
    """The balance loss E sum_e (c_e / C) (mean of softmax(logits)[:, e]) of a routing:
    logits [T, E] (fp16, bf16 or fp32, dense rows), ids int32 [T, k] -> (loss fp32 [],
    counts int32 [E + 1]): counts[e] = c_e the choices of expert e, C their sum,
    counts[E] the tokens with a usable expert, over which the mean is taken.
    workspace: uint8 of moe_balance_workspace_bytes, else allocated per call."""
    lib = library()
    _need(ids, "ids", _I32, 2)
    T, E, k, stride = _router(logits, ids)
    loss = _out(loss, (), torch.float32, logits, "loss")
    counts = _out(counts, (E + 1,), torch.int32, logits, "counts")
    ws, ws_bytes, keep = _workspace(_workspace_bytes("moe_balance_workspace_bytes", T, E, k),
                                    workspace, logits)
    _check("moe_balance",
           lib.moe_balance(logits.data_ptr(), _FLOATS[logits.dtype], T, E, stride, ids.data_ptr(),
                           k, loss.data_ptr(), counts.data_ptr(), ws, ws_bytes,
                           _stream(logits, ids, loss, counts, *keep)))
    return loss, counts


def route_grad(logits: torch.Tensor, ids: torch.Tensor = None, dweights: torch.Tensor = None,
               renormalize: bool = True, counts: torch.Tensor = None, dloss: torch.Tensor = None,
               dlogits: torch.Tensor = None) -> torch.Tensor:
    """dlogits [T, E] of the logits' dtype: the gradient of route()'s weights for ids
    int32 [T, k] and dweights fp32 [T, k] (None: no such part), plus dloss (fp32, one
    value) times the gradient of balance()'s loss for its counts (None: no such part).
    The choices and the counts are constants.  A NaN or +inf makes all gradients of its
    row NaN; with renormalize and without counts only the chosen experts' logits matter,
    and only their gradients become NaN."""
    lib = library()
    T, E, k, stride = _router(logits, ids)
    if dweights is None and counts is None:
        raise ValueError("dweights or counts must be given")
    if dweights is not None:
        if ids is None:
            raise ValueError("dweights need ids")
        _need(dweights, "dweights", _F32, 2)
        if dweights.shape != ids.shape:
            raise ValueError("dweights shape %s, ids %s"
                             % (tuple(dweights.shape), tuple(ids.shape)))
    if (counts is None) != (dloss is None):
        raise ValueError("counts and dloss go together")
    if counts is not None:
        _need(counts, "counts", _I32, 1)
        _need(dloss, "dloss", _F32, 0)
        if counts.shape[0] != E + 1 or dloss.numel() != 1:
            raise ValueError("counts have %d entries, want %d; dloss %d, want 1"
                             % (counts.shape[0], E + 1, dloss.numel()))
    dlogits = _out_like(dlogits, logits, "dlogits")
    _check("moe_route_grad",
           lib.moe_route_grad(logits.data_ptr(), _FLOATS[logits.dtype], T, E, stride, _ptr(ids), k,
                              _ptr(dweights), 1 if renormalize else 0, _ptr(counts), _ptr(dloss),
                              dlogits.data_ptr(),
                              _stream(logits, dlogits, *_given(ids, dweights, counts, dloss))))
    return dlogits


def combine_grad(dout: torch.Tensor, Y: torch.Tensor, tokens: torch.Tensor,
                 positions: torch.Tensor, weights: torch.Tensor, dY: torch.Tensor = None,
                 dweights: torch.Tensor = None):
    """The gradient of combine(): dout fp16 or bf16 [T, N], Y [R, N] of that dtype or
    fp32, tokens and positions of the plan, weights fp32 [T, k] -> (dY [R, N] of dout's
    dtype, 0 in rows of no choice; dweights fp32 [T, k], 0 for no choice)."""
    lib = library()
    _need(dout, "dout", _HALVES, 2)
    _need(Y, "Y", (dout.dtype, torch.float32), 2)
    _need(tokens, "tokens", _I32, 1)
    _need(positions, "positions", _I32, 2)
    _need(weights, "weights", _F32, 2)
    T, N = dout.shape
    R, columns = Y.shape
    choices = positions.shape
    k = choices[1]
    if columns != N or tokens.shape[0] != R:
        raise ValueError("Y has shape %s, want (%d tokens of the plan, %d)"
                         % (tuple(Y.shape), tokens.shape[0], N))
    if choices != weights.shape or choices[0] != T:
        raise ValueError("positions shape %s, weights %s, want (%d, k)"
                         % (tuple(positions.shape), tuple(weights.shape), T))
    if not 1 <= k <= MAX_CHOICES:
        raise ValueError("positions have %d choices a token, want 1 to %d" % (k, MAX_CHOICES))
    rows32 = Y.dtype == torch.float32
    dY = _out(dY, (R, N), dout.dtype, dout, "dY") if rows32 else _out_like(dY, Y, "dY")
    dweights = _out_like(dweights, weights, "dweights")
    _check("moe_combine_grad",
           lib.moe_combine_grad(dout.data_ptr(), _HALVES[dout.dtype] + (_FP32_ROWS if rows32 else 0),
                                T, N, Y.data_ptr(), R, tokens.data_ptr(), positions.data_ptr(),
                                weights.data_ptr(), k, dY.data_ptr(), dweights.data_ptr(),
                                _stream(dout, Y, tokens, positions, weights, dY, dweights)))
    return dY, dweights
