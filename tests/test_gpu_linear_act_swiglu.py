"""SwiGLU where tiles of 64 x 128 would be the fastest but have no place for a gate and its up rows:
K slices of them, other tilings, and no workspace, on the GPU against plain 64-bit forms."""
import numpy as np
import pytest

import mxfp4_grad_reference as gref
import mxfp4_reference as ref
from test_gpu_linear_act import HALVES, check_linear, gpu, mx, say, weights  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M,N,K", [(64, 512, 2048), (97, 130, 1376), (300, 512, 2048), (701, 2050, 2048),
                                   (128, 4096, 256), (701, 7168, 2048), (100, 14336, 2048)])
def test_swiglu_in_every_choice(mx, dtype, M, N, K):  # noqa: F811
    say("swiglu %s M=%d N=%d K=%d" % (dtype, M, N, K))
    rng = np.random.default_rng([M, N, K])
    check_linear(mx, rng, M, N, K, dtype, "swiglu", residual=True, save=True)
    if M * N < 1 << 19:                                     # scales on both sides of fp16's range
        check_linear(mx, rng, M, N, K, dtype, "swiglu", bias=False, save=False, low=98, high=124)


@pytest.mark.parametrize("dtype", HALVES)
def test_swiglu_without_a_workspace(mx, dtype):  # noqa: F811
    """The same product with workspace NULL is not split."""
    M, N, K = 97, 520, 2048
    say("swiglu without a workspace %s" % dtype)
    lib = mx.library()
    assert lib.mxfp4_linear_act_workspace_bytes(M, N, K) > 0
    rng = np.random.default_rng(4)
    codes, scales = weights(rng, (N, K))
    x = gpu(rng.standard_normal((M, K)), dtype)
    c, s = gpu(codes), gpu(scales)
    y = torch.empty((M, N // 2), dtype=dtype, device="cuda")
    z = torch.empty((M, N), dtype=dtype, device="cuda")
    status = lib.mxfp4_linear_act(x.data_ptr(), 0 if dtype == torch.float16 else 1, M, K, c.data_ptr(),
                                  s.data_ptr(), N, K, None, 5, None, 0, y.data_ptr(), z.data_ptr(), None,
                                  0, torch.cuda.current_stream().cuda_stream)
    assert status == 0
    want_z, mags = ref.product(ref.f64(x), ref.values(codes, scales))
    bz = ref.sum_bound(K, mags)
    want, by = gref.epilogue(want_z, bz, "swiglu")
    ref.check(z, want_z, bz + ref.rounded(np.abs(want_z) + bz, dtype), dtype)
    ref.check(y, want, by + ref.rounded(np.abs(want) + by, dtype), dtype)
