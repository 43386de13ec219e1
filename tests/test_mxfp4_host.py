"""The MXFP4 C ABI on the host: symbols, sizes and refusals (no kernel is
launched: without a device a call that passes the checks reports DEVICE), the
binding's own refusals, and the 64-bit reference the GPU tests use."""
import math
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import mxfp4_reference as ref
from weight_only_int4_gemv_amd import mxfp4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mxfp4.h")
OK, INVALID, SHAPE, MISALIGNED, DEVICE = 0, 1, 2, 3, 4
FAKE = 0x10000000            # addresses that are only ever compared
A, B, C, D, F = (FAKE * i for i in range(1, 6))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(mxfp4.LIBRARY):
        from weight_only_int4_gemv_amd import build
        build.build()
    return mxfp4.library()


def test_every_declared_symbol_is_exported(lib):
    text = open(HEADER).read()
    names = set(re.findall(r"^\s*[\w\s\*]+?\b((?:mxfp4|moe)_\w+)\s*\(", text, re.M))
    assert names == set(mxfp4._SIGNATURES) | set(mxfp4._SIZES) | {"mxfp4_status_string"}
    out = subprocess.run(["nm", "-D", "--defined-only", mxfp4.LIBRARY], check=True,
                         capture_output=True, text=True).stdout
    assert names <= set(re.findall(r"\bT (\w+)$", out, re.M))
    assert "torch" not in text and "hip_runtime" not in text


def test_status_strings(lib):
    assert len({mxfp4.status_string(s) for s in range(6)}) == 6
    assert mxfp4.status_string(99) == "unknown status"


def test_quantize_refusals(lib):
    q = lib.mxfp4_quantize
    assert q(A, 3, 4, 64, 64, B, C, None) == INVALID             # dtype
    assert q(A, 0, -1, 64, 64, B, C, None) == INVALID
    assert q(A, 0, (1 << 24) + 1, 64, 64, B, C, None) == INVALID
    assert q(A, 0, 4, 48, 48, B, C, None) == SHAPE
    assert q(A, 0, 4, -32, 32, B, C, None) == INVALID
    assert q(A, 0, 4, 64, 32, B, C, None) == INVALID             # stride < K
    assert q(A, 0, 4, 64, 1 << 40, B, C, None) == INVALID
    for bad in ((None, B, C), (A, None, C), (A, B, None)):
        assert q(bad[0], 0, 4, 64, 64, bad[1], bad[2], None) == INVALID
    assert q(A + 8, 0, 4, 64, 64, B, C, None) == MISALIGNED
    assert q(A, 0, 4, 64, 68, B, C, None) == MISALIGNED          # rows off 16 bytes
    assert q(A, 2, 4, 64, 66, B, C, None) == MISALIGNED
    assert q(A, 0, 4, 64, 64, B + 4, C, None) == MISALIGNED
    assert q(A, 0, 4, 64, 64, A + 496, C, None) == INVALID       # overlap
    assert q(A, 0, 4, 64, 64, B, B + 127, None) == INVALID
    assert q(None, 0, 0, 64, 64, None, None, None) == OK
    assert q(None, 0, 4, 0, 0, None, None, None) == OK


def test_dequantize_refusals(lib):
    d = lib.mxfp4_dequantize
    assert d(A, B, 4, 64, C, 5, None) == INVALID
    assert d(A, B, 4, 40, C, 0, None) == SHAPE
    assert d(A, B, -4, 64, C, 0, None) == INVALID
    assert d(None, B, 4, 64, C, 0, None) == INVALID
    assert d(A, B, 4, 64, C + 2, 0, None) == MISALIGNED
    assert d(A, B, 4, 64, A + 64, 0, None) == INVALID
    assert d(None, None, 0, 64, None, 0, None) == OK


def test_linear_refusals(lib):
    def call(X=A, dt=0, M=4, xs=64, c=B, s=C, N=8, K=64, Y=D, ws=None, wb=0):
        return lib.mxfp4_linear(X, dt, M, xs, c, s, N, K, Y, ws, wb, None)
    assert call(dt=2) == INVALID and call(dt=-1) == INVALID
    assert call(M=-1) == INVALID and call(N=-1) == INVALID and call(N=1 << 25) == INVALID
    assert call(K=80) == SHAPE and call(K=-32) == INVALID and call(K=1 << 25) == INVALID
    assert call(xs=32) == INVALID and call(xs=68) == MISALIGNED
    assert call(X=A + 8) == MISALIGNED and call(c=B + 8) == MISALIGNED
    assert call(Y=D + 1) == MISALIGNED
    assert call(X=None) == INVALID and call(c=None) == INVALID and call(s=None) == INVALID
    assert call(Y=None) == INVALID
    assert call(Y=A + 256) == INVALID and call(Y=B + 128) == INVALID and call(Y=C) == INVALID
    assert call(wb=16) == INVALID and call(ws=F + 8, wb=64) == MISALIGNED
    assert call(M=0, X=None, Y=None) == OK and call(N=0, c=None, s=None, Y=None) == OK


def test_matmul_refusals(lib):
    def call(ac=A, sa=B, M=4, bc=C, sb=D, N=8, K=64, Y=F, dt=0, ws=None, wb=0):
        return lib.mxfp4_matmul(ac, sa, M, bc, sb, N, K, Y, dt, ws, wb, None)
    assert call(dt=3) == INVALID and call(M=-1) == INVALID and call(N=-2) == INVALID
    assert call(K=33) == SHAPE
    assert call(ac=A + 4) == MISALIGNED and call(bc=C + 4) == MISALIGNED
    assert call(Y=F + 1) == MISALIGNED and call(Y=F + 2, dt=2) == MISALIGNED
    for name in ("ac", "sa", "bc", "sb", "Y"):
        assert call(**{name: None}) == INVALID
    assert call(Y=A + 64) == INVALID and call(Y=D) == INVALID
    assert call(ws=F * 2 + 1, wb=64) == MISALIGNED
    assert call(M=0, Y=None) == OK


def test_route_refusals(lib):
    def call(x=A, dt=0, T=4, E=8, st=8, k=2, ids=B, w=C):
        return lib.moe_route(x, dt, T, E, st, k, 1, ids, w, None)
    assert call(dt=3) == INVALID and call(T=-1) == INVALID
    assert call(E=0, st=0, k=1) == INVALID and call(E=1025, st=1025) == INVALID
    assert call(k=0) == INVALID and call(k=9) == INVALID and call(E=64, st=64, k=33) == INVALID
    assert call(st=7) == INVALID
    assert call(x=A + 1) == MISALIGNED and call(x=A + 2, dt=2) == MISALIGNED
    assert call(ids=B + 2) == MISALIGNED and call(w=C + 2) == MISALIGNED
    assert call(x=None) == INVALID and call(ids=None) == INVALID and call(w=None) == INVALID
    assert call(ids=A) == INVALID and call(ids=C) == INVALID
    assert call(T=0, x=None, ids=None, w=None) == OK


def test_plan_refusals(lib):
    def call(ids=A, T=4, k=2, E=8, off=B, tok=C, pos=D, ws=None, wb=0):
        return lib.moe_plan(ids, T, k, E, off, tok, pos, ws, wb, None)
    assert call(T=-1) == INVALID and call(k=0) == INVALID and call(k=33) == INVALID
    assert call(E=0) == INVALID and call(E=1025) == INVALID
    assert call(T=1 << 23, k=4) == INVALID                       # T k too large
    for name in ("ids", "off", "tok", "pos"):
        assert call(**{name: None}) == INVALID
    assert call(off=B + 2) == MISALIGNED
    assert call(tok=A) == INVALID and call(pos=C) == INVALID
    need = lib.moe_plan_workspace_bytes(100000, 2, 8)
    assert need > 0 and lib.moe_plan_workspace_bytes(4, 2, 8) == 0
    assert lib.moe_plan_workspace_bytes(-4, 2, 8) == 0
    assert call(T=100000) == INVALID                             # workspace missing
    assert call(T=100000, ws=F, wb=need - 1) == INVALID
    assert call(T=100000, ws=F + 1, wb=need) == MISALIGNED


def test_grouped_refusals(lib):
    def call(X=A, dt=0, xr=4, xs=64, tok=None, R=4, c=B, s=C, off=D, E=2, N=8, K=64, sw=0, Y=F):
        return lib.mxfp4_grouped_linear(X, dt, xr, xs, tok, R, c, s, off, E, N, K, sw, Y, None)
    assert call(dt=2) == INVALID and call(xr=-1) == INVALID and call(R=-1) == INVALID
    assert call(E=0) == INVALID and call(E=1025) == INVALID and call(N=-2) == INVALID
    assert call(K=63) == SHAPE and call(N=7, sw=1) == SHAPE
    assert call(xs=32) == INVALID and call(xs=68) == MISALIGNED
    assert call(R=5) == INVALID                                  # fewer rows than R, no tokens
    assert call(X=None) == INVALID and call(off=None) == INVALID and call(Y=None) == INVALID
    assert call(c=None) == INVALID and call(s=None) == INVALID
    assert call(X=A + 2) == MISALIGNED and call(c=B + 1) == MISALIGNED
    assert call(off=D + 2) == MISALIGNED and call(tok=F * 2 + 2, R=9) == MISALIGNED
    assert call(Y=A) == INVALID and call(Y=B + 256) == INVALID and call(Y=D) == INVALID
    assert call(R=0, Y=None) == OK and call(N=0, Y=None) == OK


def test_combine_refusals(lib):
    def call(Y=A, dt=0, R=4, N=8, pos=B, w=C, T=2, k=2, out=D):
        return lib.moe_combine(Y, dt, R, N, pos, w, T, k, out, None)
    assert call(dt=2) == INVALID and call(R=-1) == INVALID and call(N=-1) == INVALID
    assert call(k=0) == INVALID and call(k=33) == INVALID and call(T=-1) == INVALID
    for name in ("Y", "pos", "w", "out"):
        assert call(**{name: None}) == INVALID
    assert call(Y=A + 1) == MISALIGNED and call(pos=B + 2) == MISALIGNED
    assert call(out=A) == INVALID and call(out=C) == INVALID
    assert call(T=0, out=None) == OK and call(N=0, out=None) == OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")
def test_valid_calls_reach_the_device_check(lib):
    assert lib.mxfp4_quantize(A, 0, 4, 64, 72, B, C, None) == DEVICE
    assert lib.mxfp4_dequantize(A, B, 4, 64, C, 2, None) == DEVICE
    assert lib.mxfp4_linear(A, 1, 4, 64, B, C, 8, 64, D, None, 0, None) == DEVICE
    assert lib.mxfp4_linear(None, 1, 4, 0, None, None, 8, 0, D, None, 0, None) == DEVICE
    assert lib.mxfp4_matmul(A, B, 4, C, D, 8, 64, F, 2, None, 0, None) == DEVICE
    assert lib.moe_route(A, 2, 4, 8, 9, 8, 0, B, C, None) == DEVICE
    assert lib.moe_plan(None, 0, 2, 8, B, None, None, None, 0, None) == DEVICE
    assert lib.mxfp4_grouped_linear(A, 0, 1, 64, F * 2, 9, B, C, D, 2, 8, 64, 1, F, None) == DEVICE
    assert lib.moe_combine(None, 0, 0, 8, B, C, 2, 2, D, None) == DEVICE


def test_binding_refuses_host_and_odd_tensors(lib):
    x = torch.zeros(4, 64, dtype=torch.float16)
    u = torch.zeros(4, 32, dtype=torch.uint8)
    for call in (lambda: mxfp4.quantize(x), lambda: mxfp4.quantize([1.0]),
                 lambda: mxfp4.quantize(x.double()), lambda: mxfp4.dequantize(u, u),
                 lambda: mxfp4.linear(x, u, u), lambda: mxfp4.matmul(u, u, u, u),
                 lambda: mxfp4.matmul(u, u, u, u, dtype=torch.int8),
                 lambda: mxfp4.route(x, 2), lambda: mxfp4.plan(u, 2),
                 lambda: mxfp4.grouped_linear(x, u, u, u), lambda: mxfp4.combine(x, u, u)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------- the reference, by other means

def test_reference_quantizer_on_a_hand_worked_block():
    x = np.zeros((1, 32))
    x[0, :8] = [6.0, -5.0, 0.25, 0.75, -0.25, 3.5, 2.5, -0.0]     # peak 6: E = 0
    nib, s = ref.quantize(x)
    assert s[0, 0] == 127
    # ties: 5 -> 4 (code 6), 0.25 -> 0, 0.75 -> 1, 3.5 -> 4, 2.5 -> 2
    assert nib[0, :8].tolist() == [7, 14, 0, 2, 8, 6, 4, 8]
    assert ref.values(ref.pack(nib), s)[0, :7].tolist() == [6, -4, 0, 1, 0, 4, 2]


@pytest.mark.parametrize("peak,E", [(1.0, -2), (7.99, 0), (8.0, 1), (3.999, -1), (2.0 ** -140, -127),
                                    (2.0 ** 127, 125), (0.0, 0)])
def test_reference_scale(peak, E):
    x = np.full((1, 32), peak)
    nib, s = ref.quantize(x)
    assert int(s[0, 0]) - 127 == E
    if peak > 2.0 ** -126:
        assert (np.abs(ref.values(ref.pack(nib), s) - x) <= peak / 4).all()


def test_reference_rounds_to_the_nearest_value():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((8, 64))
    nib, s = ref.quantize(x)
    v = ref.values(ref.pack(nib), s)
    grid = ref.CODE_VALUES[None, None, :] * np.exp2(np.repeat(s.astype(float) - 127, 32, 1))[..., None]
    assert (np.abs(v - x) <= np.abs(grid - x[..., None]).min(axis=2)).all()


def test_reference_routing_and_plan():
    x = np.array([[1.0, 3.0, 3.0, -np.inf], [-np.inf] * 4, [0.0, np.nan, 1.0, 2.0]])
    ids, w = ref.route(x, 2, True)
    assert ids.tolist() == [[1, 2], [-1, -1], [1, 3]]
    assert w[0].tolist() == [0.5, 0.5] and w[1].tolist() == [0, 0] and np.isnan(w[2]).all()
    assert math.isclose(ref.route(x, 3, False)[1][0].sum(), 1.0)
    off, tok, pos = ref.plan(np.array([[1, 0], [-1, 1], [0, 7]]), 2)
    assert off.tolist() == [0, 2, 4]
    assert tok.tolist() == [0, 2, 0, 1, -1, -1]
    assert pos.tolist() == [[2, 0], [-1, 3], [1, -1]]
