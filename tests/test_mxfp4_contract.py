"""What include/mxfp4.h promises, on the host: refusals of the entry points that
test_mxfp4_host does not reach (no kernel is launched)."""
import os
import re

import pytest
import torch

from test_mxfp4_host import A, B, C, D, DEVICE, F, INVALID, MISALIGNED, OK, lib  # noqa: F401
from weight_only_int4_gemv_amd import build

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
