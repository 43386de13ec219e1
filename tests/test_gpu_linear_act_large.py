"""GELU and SiLU behind products of thousands of columns (the two largest tilings), on the GPU
against the plain 64-bit form with torch's complementary error function of doubles."""
import math

import numpy as np
import pytest

import mxfp4_grad_reference as gref
from test_gpu_linear_act import HALVES, check_linear, mx, say  # noqa: F401

torch = pytest.importorskip("torch")


def erfc(z):
    return torch.special.erfc(torch.from_numpy(np.ascontiguousarray(z))).numpy()


def test_erfc_is_math_s():
    z = np.concatenate([np.linspace(-7, 26, 3301), [0.0, np.inf, -np.inf]])
    want = np.array([math.erfc(v) for v in z])
    assert (np.abs(erfc(z) - want) <= 2.0 ** -44 * want).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("M,N,K", [(640, 6656, 64), (2049, 4096, 32)])
def test_many_rows_and_columns(mx, monkeypatch, dtype, act, M, N, K):  # noqa: F811
    say("linear_act %s %s M=%d N=%d K=%d" % (dtype, act, M, N, K))
    monkeypatch.setattr(gref, "_erfc", erfc)
    check_linear(mx, np.random.default_rng([M, N, K]), M, N, K, dtype, act, bias=True, residual=M % 2 == 1,
                 save=True)
