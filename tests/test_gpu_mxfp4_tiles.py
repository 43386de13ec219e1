"""The tiled weight-only MXFP4 kernels where their tiles, K slices, scale chunks and
stores end unevenly, against the 64-bit reference (bounds derived in mxfp4_reference)."""
import numpy as np
import pytest

import mxfp4_reference as ref
from test_gpu_moe import check_grouped, experts
from test_gpu_mxfp4 import HALVES, check_linear, gpu, mx, random_weight, say  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

# One shape for each block size: 32 x 256, 64 x 128, 64 x 256 and 128 x 256.
DENSE = {"32x256": (19, 530), "64x128": (70, 300), "64x256": (449, 8200), "128x256": (1030, 7201)}


def dense(rng, name, K, dtype, low=110, high=124):
    M, N = DENSE[name]
    return gpu(rng.standard_normal((M, K)), dtype), random_weight(rng, N, K, low, high)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("name", list(DENSE))
@pytest.mark.parametrize("K", [32, 96, 288, 480])
def test_every_tile_size(mx, dtype, name, K):  # noqa: F811
    """K one block past whole steps and scale chunks of 8 and 16 blocks."""
    say("tiles %s %s K=%d" % (name, dtype, K))
    x, (codes, scales) = dense(np.random.default_rng([K, len(name)]), name, K, dtype)
    check_linear(mx, x, codes, scales)


@pytest.mark.parametrize("name", ["32x256", "64x128"])
@pytest.mark.parametrize("K", [2016, 2048, 2080, 4128, 5216])
def test_scales_held_past_64_blocks(mx, name, K):  # noqa: F811
    """With and without K slices: 64 blocks of scales are held at a time."""
    say("scales %s K=%d" % (name, K))
    M, N = DENSE[name]
    rng = np.random.default_rng([K, M])
    x, (codes, scales) = dense(rng, name, K, torch.bfloat16)
    need = mx.linear_workspace(M, N, K).numel()
    assert need > 1                                       # this shape is split
    y = check_linear(mx, x, codes, scales)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")      # NaN
    assert torch.equal(y, mx.linear(x, gpu(codes), gpu(scales), workspace=ws))
    # The unsplit product through the C ABI (no workspace).
    c, s, z = gpu(codes), gpu(scales), torch.empty_like(y)
    status = mx.library().mxfp4_linear(x.data_ptr(), 1, M, K, c.data_ptr(), s.data_ptr(), N, K,
                                       z.data_ptr(), None, 0, torch.cuda.current_stream().cuda_stream)
    assert status == 0
    w = ref.values(codes, scales)
    want, mags = ref.product(ref.f64(x), w)
    bound = ref.sum_bound(K, mags)
    ref.check(z, want, bound + ref.rounded(np.abs(want) + bound, x.dtype), x.dtype)


@pytest.mark.parametrize("name", list(DENSE))
@pytest.mark.parametrize("at", [0, 3, 9])
def test_fp16_weights_leave_its_range_midway(mx, name, at):  # noqa: F811
    """From block `at` on some rows' scales pass fp16's range, later ones return."""
    say("midway %s at=%d" % (name, at))
    rng = np.random.default_rng([at, len(name)])
    x, (codes, scales) = dense(rng, name, 416, torch.float16)
    scales[3::7, at:at + 2] = 150
    scales[5::11, at + 1] = 60
    check_linear(mx, x, codes, scales)


@pytest.mark.parametrize("name", list(DENSE))
def test_unaligned_scales_and_outputs(mx, name):  # noqa: F811
    """Scales at an odd address, Y at an odd element, an odd row length."""
    M, N = DENSE[name]
    rng = np.random.default_rng(M)
    x, (codes, scales) = dense(rng, name, 352, torch.bfloat16)
    s = torch.empty(N * 11 + 1, dtype=torch.uint8, device="cuda")[1:].view(N, 11)
    s.copy_(gpu(scales))
    out = torch.full((M * N + 9,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = out[3:3 + M * N].view(M, N)
    say("unaligned %s" % name)
    mx.linear(x, gpu(codes), s, Y=y)
    assert (out[:3] == 7).all() and (out[3 + M * N:] == 7).all()
    assert torch.equal(y, mx.linear(x, gpu(codes), gpu(scales)))


# Mean rows per expert in the range of each block size; uneven, with empty experts.
GROUPS = {"32x256": [0, 33, 5, 20], "64x256": [131, 0, 64, 3], "128x256": [400, 129, 0, 260]}


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("F,K,swiglu", [(129, 288, True), (300, 480, True), (270, 2080, False)])
def test_grouped_tile_sizes(mx, dtype, name, F, K, swiglu):  # noqa: F811
    say("grouped %s %s F=%d K=%d" % (name, dtype, F, K))
    rng = np.random.default_rng([F, K, len(name)])
    offsets = np.concatenate([[0], np.cumsum(GROUPS[name])])
    codes, scales = experts(rng, 4, 2 * F if swiglu else F, K, 112, 122)
    x = gpu(rng.standard_normal((50, K)), dtype)
    tokens = rng.integers(0, 50, int(offsets[-1]) + 3)
    tokens[::17] = -1
    check_grouped(mx, x, codes, scales, offsets, tokens=tokens, swiglu=swiglu)


@pytest.mark.parametrize("name", list(GROUPS))
def test_grouped_fp16_range_midway(mx, name):  # noqa: F811
    rng = np.random.default_rng(len(name))
    offsets = np.concatenate([[0], np.cumsum(GROUPS[name])])
    codes, scales = experts(rng, 4, 140, 352, 112, 122)
    scales[1, 2::5, 4:6] = 148
    scales[3, ::9, 7] = 20
    check_grouped(mx, gpu(rng.standard_normal((int(offsets[-1]), 352)), torch.float16), codes,
                  scales, offsets)


@pytest.mark.parametrize("E", [63, 200, 1024])
def test_grouped_many_experts(mx, E):  # noqa: F811
    """More groups than a wave scans at once; most experts empty."""
    rng = np.random.default_rng(E)
    counts = np.where(rng.random(E) < 0.9, 0, rng.integers(1, 60, E))
    counts[-1] = E + 40                                    # at least a row per expert on average
    counts[0] = 3
    offsets = np.concatenate([[0], np.cumsum(counts)])
    codes, scales = experts(rng, E, 34, 64, 112, 122)
    say("many experts E=%d rows=%d" % (E, offsets[-1]))
    check_grouped(mx, gpu(rng.standard_normal((int(offsets[-1]), 64)), torch.bfloat16), codes,
                  scales, offsets)


@pytest.mark.parametrize("offsets", [[-5, 40, 20, 900], [0, 0, 0, 0], [70, 70, 70, 70],
                                     [2 ** 31 - 1, -2 ** 31, 5, 2 ** 31 - 1]])
@pytest.mark.parametrize("rows", [2, 70, 500, 700])
def test_grouped_bad_offsets_stay_inside(mx, offsets, rows):  # noqa: F811
    """Entries outside [0, R] are clamped, a falling pair is an empty expert."""
    rng = np.random.default_rng(rows)
    codes, scales = experts(rng, 3, 50, 96)
    x = gpu(rng.standard_normal((rows, 96)), torch.bfloat16)
    say("offsets %s rows=%d" % (offsets, rows))
    y = ref.f64(mx.grouped_linear(x, gpu(codes), gpu(scales), gpu(np.array(offsets), torch.int32)))
    assert np.isfinite(y).all()
    lo = np.clip(offsets, 0, rows)
    assert (y[:lo[0]] == 0).all()
    if (np.diff(lo) >= 0).all():
        want = np.zeros((rows, 50))
        mags = np.zeros((rows, 50))
        for e in range(3):
            want[lo[e]:lo[e + 1]], mags[lo[e]:lo[e + 1]] = ref.product(
                ref.f64(x)[lo[e]:lo[e + 1]], ref.values(codes[e], scales[e]))
        bound = ref.sum_bound(96, mags)
        ref.check(torch.from_numpy(y).bfloat16(), want, bound + ref.rounded(np.abs(want) + bound, x.dtype),
                  x.dtype)


def test_example_runs():
    from weight_only_int4_gemv_amd import moe_example
    error = moe_example.run(tokens=37, experts=8, choices=2, hidden=256, inner=160, seed=3)
    # |error| of the layer's outputs against the 64-bit layer on the quantized weights,
    # relative to the largest output: bf16 rounds the hidden rows, their outputs and the
    # sum (2^-8 each), the fp32 sums are far below.
    assert error <= 4 * 2.0 ** -8
