"""Weight-only MXFP4 products at the ends of the scale range, for every kernel: weights
of 2^128 and more, which neither bf16 nor fp32 holds (scale bytes 253 and 254), next to
the smallest ones and to zeros in X, against the 64-bit reference (bounds derived in
mxfp4_reference)."""
import numpy as np
import pytest

import mxfp4_reference as ref
from test_gpu_moe import check_grouped, experts
from test_gpu_mxfp4 import HALVES, check_linear, check_matmul, gpu, mx, random_weight, say  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

# One shape for each kernel: stream with one and four weight tiles a block, then the
# 32 x 256, 64 x 128, 64 x 256 and 128 x 256 blocks.
SHAPES = {"stream 1": (9, 70), "stream 4": (3, 12300), "32x256": (19, 530), "64x128": (70, 300),
          "64x256": (449, 8200), "128x256": (1030, 7201)}
K = 224                                                   # an odd number of blocks


def one_hot(M, dtype, seed):
    """Rows with 2^-3 in one column: every product of 2^-131 (the least code under the
    least scale) up to 6 * 2^124 is exact in bf16."""
    cols = np.random.default_rng(seed).integers(0, K, M)
    x = np.zeros((M, K))
    x[np.arange(M), cols] = 0.125
    return gpu(x, dtype), cols


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("low,high", [(0, 3), (250, 254), (0, 254)])
def test_one_hot_picks_any_weight(mx, dtype, name, low, high):  # noqa: F811
    """One product, no error: y is the weight over 8, rounded once; a zero in X takes
    nothing from the largest weights."""
    M, N = SHAPES[name]
    say("scale ends one-hot %s %s %d..%d" % (dtype, name, low, high))
    codes, scales = random_weight(np.random.default_rng([M, N, high]), N, K, low, high)
    x, cols = one_hot(M, dtype, M)
    y = mx.linear(x, gpu(codes), gpu(scales)).cpu()
    want = torch.from_numpy(ref.values(codes, scales).T[cols] / 8).to(dtype)
    assert not torch.isnan(y).any()
    assert torch.equal(y, want)


@pytest.mark.parametrize("name", list(SHAPES))
@pytest.mark.parametrize("low,high", [(250, 254), (120, 254), (0, 254)])
def test_sums_of_large_weights(mx, name, low, high):  # noqa: F811
    """bf16 X small enough that every sum is finite."""
    M, N = SHAPES[name]
    say("scale ends sums %s %d..%d" % (name, low, high))
    rng = np.random.default_rng([M, N, low])
    codes, scales = random_weight(rng, N, K, low, high)
    x = gpu(rng.standard_normal((M, K)) * 2.0 ** -20, torch.bfloat16)
    y = check_linear(mx, x, codes, scales)
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("name", list(SHAPES))
def test_zeros_meet_the_largest_weights(mx, dtype, name):  # noqa: F811
    """X is 0 where the weights are largest, ordinary elsewhere: ordinary outputs."""
    M, N = SHAPES[name]
    say("scale ends zeros %s %s" % (dtype, name))
    rng = np.random.default_rng([M, N])
    codes, scales = random_weight(rng, N, K, 112, 122)
    scales[::3, 2], scales[1::5, 6] = 254, 253
    x = rng.standard_normal((M, K))
    x[:, 64:96], x[:, 192:224] = 0, 0
    check_linear(mx, gpu(x, dtype), codes, scales)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("name", ["stream 1", "64x128"])
def test_not_finite_x_meets_the_largest_weights(mx, dtype, name):  # noqa: F811
    """An infinity takes the weight's sign, NaN where the weight is 0; a NaN scale stays."""
    M, N = SHAPES[name]
    say("scale ends not finite %s %s" % (dtype, name))
    rng = np.random.default_rng([M, N])
    codes, scales = random_weight(rng, N, K, 252, 254)
    scales[7, 0] = 255
    x = np.zeros((M, K))
    x[0, 70], x[1, 3], x[2, 200] = np.inf, np.nan, -np.inf
    y = ref.f64(mx.linear(gpu(x, dtype), gpu(codes), gpu(scales)))
    keep = np.arange(N) != 7
    w = ref.values(codes, scales)
    with np.errstate(all="ignore"):
        assert np.array_equal(y[0, keep], w[keep, 70] * np.inf, equal_nan=True)
        assert np.array_equal(y[2, keep], w[keep, 200] * -np.inf, equal_nan=True)
    assert np.isnan(y[1]).all() and np.isnan(y[:, 7]).all() and (y[3:, keep] == 0).all()


def test_k_slices_of_the_largest_weights(mx):  # noqa: F811
    """Partial sums through the workspace, some slices with the largest weights only."""
    rng = np.random.default_rng(1)
    M, N, k = 19, 530, 4128
    codes, scales = random_weight(rng, N, k, 230, 240)
    scales[::2, 40:60] = 254
    x = gpu(rng.standard_normal((M, k)) * 2.0 ** -20, torch.bfloat16)
    assert mx.linear_workspace(M, N, k).numel() > 1
    say("scale ends slices")
    assert torch.isfinite(check_linear(mx, x, codes, scales)).all()


# Rows of each expert: less than one on average (stream), then each block size.
GROUPS = {"stream": [1, 0, 0, 2, 0, 0], "32x256": [0, 33, 5, 20], "64x256": [131, 0, 64, 3],
          "128x256": [400, 129, 0, 260]}


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("name", list(GROUPS))
def test_grouped_rows_of_no_token_stay_zero(mx, dtype, name):  # noqa: F811
    """A token outside X is a row of zeros whatever the weights."""
    say("scale ends tokens %s %s" % (dtype, name))
    rng = np.random.default_rng(len(name))
    counts = GROUPS[name]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    codes, scales = experts(rng, len(counts), 140, K, 250, 254)
    tokens = np.where(rng.random(offsets[-1]) < 0.5, -1, 0)
    y = mx.grouped_linear(gpu(np.zeros((1, K)), dtype), gpu(codes), gpu(scales),
                          gpu(offsets, torch.int32), tokens=gpu(tokens, torch.int32))
    assert (y == 0).all()


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("swiglu", [False, True])
def test_grouped_large_weights(mx, name, swiglu):  # noqa: F811
    """bf16 rows small enough that every sum and product is finite."""
    say("scale ends grouped %s swiglu=%s" % (name, swiglu))
    rng = np.random.default_rng([len(name), swiglu])
    counts = GROUPS[name]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    codes, scales = experts(rng, len(counts), 140, K, 112, 122)
    if swiglu:
        scales[:, 75::3, 1::2] = 254                      # up rows
    else:
        scales[::2, ::3, 1::2] = 253
        scales[1::2, 1::4, 0] = 254
    x = gpu(rng.standard_normal((offsets[-1], K)) * 2.0 ** -20, torch.bfloat16)
    y = check_grouped(mx, x, codes, scales, offsets, swiglu=swiglu)
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("M,N", [(3, 40), (100, 90), (300, 300)])
def test_matmul_of_large_scales(mx, M, N):  # noqa: F811
    """The 4-bit product applies the scales in the instruction: finite where the sum is."""
    say("scale ends matmul M=%d" % M)
    rng = np.random.default_rng([M, N])
    check_matmul(mx, *random_weight(rng, M, K, 90, 100), *random_weight(rng, N, K, 250, 254),
                 torch.bfloat16)
