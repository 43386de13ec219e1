"""Checks on the gfx950 assembly of the MXFP4 and expert kernels (no GPU needed):
no scratch memory, no packed-fp32 arithmetic, and no matrix-core result read
before its wait states (the checks of test_build_no_scratch, with the counts the
compiler pads to inside a basic block for the instructions used here)."""
import os
import re
import tempfile
from concurrent.futures import ThreadPoolExecutor

import pytest

import test_build_no_scratch as base
from weight_only_int4_gemv_amd import build as B

WAIT_STATES = {"v_mfma_f32_16x16x32_f16": 8, "v_mfma_f32_16x16x32_bf16": 8,
               "v_mfma_f32_32x32x16_f16": 12, "v_mfma_f32_32x32x16_bf16": 12,
               "v_mfma_scale_f32_16x16x128_f8f6f4": 8, "v_mfma_scale_f32_32x32x64_f8f6f4": 12}

pytestmark = base.pytestmark


@pytest.fixture(scope="module")
def assembly():
    sources = [os.path.join(B.CSRC, s) for s in B.MXFP4_SOURCES]
    with tempfile.TemporaryDirectory(prefix="mxfp4_asm_") as tmp:
        with ThreadPoolExecutor(max_workers=4) as ex:
            return dict(zip(B.MXFP4_SOURCES, ex.map(lambda s: base._assemble(s, tmp), sources)))


def test_no_kernel_uses_scratch(assembly):
    kernels = []
    for text in assembly.values():
        kernels += [(m.group(1), int(m.group(2))) for m in re.finditer(
            r"\.name:\s+(\S+)\s*\n(?:.*\n)*?\s*\.private_segment_fixed_size:\s+(\d+)", text)]
    assert len(kernels) > 20, "kernel metadata not found"
    bad = [k for k in kernels if k[1] > 0]
    assert not bad, "kernels using scratch: %s" % bad


def test_no_packed_fp32(assembly):
    for src, text in assembly.items():
        assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", text), src


def test_no_mfma_result_read_too_early(assembly, monkeypatch):
    monkeypatch.setattr(base, "MFMA_WAIT_STATES", WAIT_STATES)
    total, bad = 0, []
    for src, text in assembly.items():
        for m in re.finditer(r"^(_Z\w+):", text, re.M):
            end = text.find(".Lfunc_end", m.end())
            found, count = base.mfma_hazards(text[m.end():end])
            total += count
            bad += [(src, m.group(1)[:60]) + f for f in found[:2]]
    assert total > 100, "MFMA instructions not found"
    assert not bad, "MFMA results read before their wait states: %s" % bad[:6]
