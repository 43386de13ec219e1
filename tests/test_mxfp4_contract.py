"""What include/mxfp4.h promises, on the host: refusals of the entry points that
test_mxfp4_host does not reach (no kernel is launched)."""
import os
import re

import pytest
import torch

from test_mxfp4_host import A, B, C, D, DEVICE, F, INVALID, MISALIGNED, OK, ROOT, lib  # noqa: F401
from weight_only_int4_gemv_amd import build, mxfp4

ROWS = 16                            # MXFP4_FP32_ROWS
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not real")


# ------------------------------------------------------------- fp32 expert rows

def grouped(lib, dt=ROWS, R=4, N=8, sw=0, Y=F):  # noqa: F811
    return lib.mxfp4_grouped_linear(A, dt, 4, 64, None, R, B, C, D, 2, N, 64, sw, Y, None)


def combine(lib, dt=ROWS, Y=A, R=4, out=D):  # noqa: F811
    return lib.moe_combine(Y, dt, R, 8, B, C, 2, 2, out, None)


def test_fp32_rows_refusals(lib):  # noqa: F811
    for dt in (ROWS + 2, ROWS + 3, 2 * ROWS, ROWS - 1, -1, -ROWS, 2 ** 31 - 1, -2 ** 31):
        assert grouped(lib, dt) == INVALID and combine(lib, dt) == INVALID
    assert grouped(lib, sw=1) == INVALID
    assert grouped(lib, Y=F + 2) == MISALIGNED and combine(lib, Y=A + 2) == MISALIGNED
    # Y's bytes count as fp32: 4 x 8 rows reach 128 bytes
    assert grouped(lib, Y=A - 124) == INVALID and combine(lib, out=A + 124) == INVALID
    assert grouped(lib, R=0) == OK


@no_gpu
def test_fp32_rows_reach_the_device_check(lib):  # noqa: F811
    for dt in (ROWS, ROWS + 1):
        assert grouped(lib, dt) == DEVICE and combine(lib, dt) == DEVICE
        assert grouped(lib, dt, Y=F + 4) == DEVICE and combine(lib, dt, Y=A + 4) == DEVICE
        assert combine(lib, dt, out=A + 128) == DEVICE


# ------------------------------------------------------------- inline assembly

def test_assembly_names_the_registers_it_writes():
    """Every asm block that moves a value into m0 says so to the compiler."""
    found = 0
    for name in os.listdir(build.CSRC):
        text = open(os.path.join(build.CSRC, name)).read()
        for block in re.findall(r"asm volatile\((.*?)\);", text, re.S):
            if "s_mov_b32 m0" in block:
                found += 1
                assert '"m0"' in block.rsplit(":", 1)[1], (name, block)
    assert found >= 2


# ------------------------------------------------------------------- alignment

def words(*path):
    text = open(os.path.join(ROOT, *path)).read()
    return " ".join(re.sub(r"^\s*[*#/]+", "", text, flags=re.M).split())


@no_gpu
def test_dequantize_alignment_is_as_documented(lib):  # noqa: F811
    """Y of mxfp4_dequantize takes 16 bytes, as X and the codes do; the outputs of the
    other entry points their element size."""
    assert "X, its row stride in bytes, codes and the Y of mxfp4_dequantize 16" in \
        words("include", "mxfp4.h")
    assert "Y starts on 16 bytes" in " ".join(mxfp4.dequantize.__doc__.split())
    for dt, size in ((0, 2), (1, 2), (2, 4)):
        for at in (size, 8):
            assert lib.mxfp4_dequantize(A, B, 4, 64, C + at, dt, None) == MISALIGNED
        assert lib.mxfp4_dequantize(A, B, 4, 64, C + 16, dt, None) == DEVICE
    assert lib.mxfp4_linear(A, 1, 4, 64, B, C, 8, 64, D + 2, None, 0, None) == DEVICE
    assert lib.mxfp4_matmul(A, B, 4, C, D, 8, 64, F + 4, 2, None, 0, None) == DEVICE
    assert lib.moe_combine(A + 2, 0, 4, 8, B, C, 2, 2, D + 2, None) == DEVICE


def test_every_vector_type_is_used():
    sources = "".join(open(os.path.join(build.CSRC, n)).read() for n in os.listdir(build.CSRC)
                      if n.startswith(("mxfp4", "moe")))
    types = re.findall(r"typedef \w+ (\w+) __attribute__", sources)
    assert len(types) > 5
    assert [t for t in types if len(re.findall(r"\b%s\b" % t, sources)) < 2] == []


# ------------------------------------------------------------------ workspaces

@no_gpu
@pytest.mark.parametrize("name", ["linear", "matmul"])
def test_workspace_rules(lib, name):  # noqa: F811
    """Where K is split: too few bytes, memory off 16 bytes or over another tensor are
    refused, NULL and larger memory are not."""
    M, N, K = 50, 512, 8192
    need = getattr(lib, "mxfp4_%s_workspace_bytes" % name)(M, N, K)
    assert need > 0 and need % (M * N * 4) == 0
    far = 8 * F

    def call(ws, bytes_):
        if name == "linear":
            return lib.mxfp4_linear(A, 0, M, K, B, C, N, K, D, ws, bytes_, None)
        return lib.mxfp4_matmul(A, B, M, C, D, N, K, F, 0, ws, bytes_, None)
    assert call(far, need) == DEVICE and call(far, need + 5) == DEVICE and call(None, 0) == DEVICE
    assert call(far, need - 1) == INVALID and call(far, 0) == INVALID and call(None, need) == INVALID
    assert call(far + 8, need) == MISALIGNED
    for other in (A, B, C, D):
        assert call(other + 16, need) == INVALID and call(other - need + 16, need) == INVALID


def test_sizes_out_of_range_need_no_workspace(lib):  # noqa: F811
    for fn in (lib.mxfp4_linear_workspace_bytes, lib.mxfp4_matmul_workspace_bytes):
        for M, N, K in ((-1, 8, 32), (8, -1, 32), (8, 8, -32), (8, 8, 33), (1 << 25, 8, 32),
                        (8, 1 << 25, 32), (8, 8, 1 << 25), (0, 8, 64), (8, 0, 64), (8, 8, 0)):
            assert fn(M, N, K) == 0
