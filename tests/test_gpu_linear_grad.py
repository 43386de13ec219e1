"""The gradient through the MXFP4 product on the GPU against the plain 64-bit form (bounds
derived in mxfp4_reference), and against differences of the product itself."""
import numpy as np
import pytest

import mxfp4_reference as ref
from test_gpu_linear_act import HALVES, RAGGED, gpu, mx, ranges, say, weights  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def expect(dy, codes, scales, dtype):
    """(dX, its bound) of float64 dy."""
    w = ref.values(codes, scales)
    want, mags = ref.product(dy, w.T)
    return want, ref.sum_bound(dy.shape[1], mags) + ref.rounded(np.abs(want), dtype)


def check_grad(mx, dy, codes, scales, **more):  # noqa: F811
    got = mx.linear_grad(dy, gpu(codes), gpu(scales), **more)
    ref.check(got, *expect(ref.f64(dy), codes, scales, dy.dtype), dy.dtype)
    return got


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 4096, 64), (2, 33, 288), (16, 4096, 512), (17, 100, 96),
                                   (32, 2047, 256), (33, 64, 4128), (64, 8, 1024), (100, 2056, 160),
                                   (129, 517, 544), (300, 96, 8192), (1030, 72, 4096), (4100, 40, 1056),
                                   (260, 4096, 320)])
def test_linear_grad(mx, dtype, M, N, K):  # noqa: F811
    say("linear_grad %s M=%d N=%d K=%d" % (dtype, M, N, K))
    rng = np.random.default_rng([M, N, K])
    codes, scales = weights(rng, (N, K))
    check_grad(mx, gpu(rng.standard_normal((M, N)), dtype), codes, scales)


# Rows that fill the chip once with blocks of 128, 96, 64 and 32 rows.
TILES = [65500, 49100, 32700, 16300]


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M", TILES)
@pytest.mark.parametrize("N,K", [(392, 256), (331, 224), (200, 160)])
def test_every_tiling(mx, dtype, M, N, K):  # noqa: F811
    """Several steps of each; rows of dY on 16 bytes and not, scales on words and not, ends of the
    rows, the weight rows and the columns inside a tile."""
    say("linear_grad tilings %s M=%d N=%d K=%d" % (dtype, M, N, K))
    rng = np.random.default_rng([M, N])
    codes, scales = weights(rng, (N, K))
    check_grad(mx, gpu(rng.standard_normal((M, N)), dtype), codes, scales)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M", TILES)
@pytest.mark.parametrize("low,high", [(90, 120), (118, 150), (0, 3)])
def test_every_tiling_scale_ranges(mx, dtype, M, low, high):  # noqa: F811
    say("linear_grad tilings scales %s M=%d %d..%d" % (dtype, M, low, high))
    rng = np.random.default_rng([M, low])
    N, K = 264, 128
    codes, scales = weights(rng, (N, K), 118, 126)
    scales[150:] = weights(rng, (N - 150, K), low, high)[1]      # from the third step on
    dy = gpu(rng.standard_normal((M, N)) * 2.0 ** -6, dtype)
    check_grad(mx, dy, codes, scales)
    scales[190, 1], scales[7, 3] = 254, 253
    check_grad(mx, dy, codes, scales)
    scales[263, 2] = 255
    assert mx.linear_grad(dy, gpu(codes), gpu(scales))[:, 64:96].isnan().all()


@pytest.mark.parametrize("M", [4, 50, 300])
def test_scales_at_any_byte(mx, M):  # noqa: F811
    rng = np.random.default_rng(M)
    codes, scales = weights(rng, (520, 512))
    room = torch.empty(scales.size + 3, dtype=torch.uint8, device="cuda")
    dy = gpu(rng.standard_normal((M, 520)), torch.bfloat16)
    want = mx.linear_grad(dy, gpu(codes), gpu(scales))
    for at in (1, 2, 3):
        view = room[at:at + scales.size].view(scales.shape)
        view.copy_(gpu(scales))
        assert torch.equal(mx.linear_grad(dy, gpu(codes), view), want)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M", [3, 40, 200])
def test_strides_and_alignment(mx, dtype, M):  # noqa: F811
    """Rows of dY at any element; what stands between and behind them is not read as data."""
    say("linear_grad strides %s M=%d" % (dtype, M))
    rng = np.random.default_rng(M)
    for N, left, right in ((64, 0, 8), (64, 8, 0), (64, 1, 0), (67, 0, 5), (67, 0, 0), (60, 0, 4)):
        codes, scales = weights(rng, (N, 96))
        room = torch.full((M, left + N + right), float("nan"), dtype=dtype, device="cuda")
        dy = room[:, left:left + N]
        dy.copy_(gpu(rng.standard_normal((M, N))))
        check_grad(mx, dy, codes, scales)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M", [2, 70, 300])
@pytest.mark.parametrize("low,high", [(90, 120), (118, 150), (0, 60), (0, 3), (200, 252)])
def test_scale_ranges(mx, dtype, M, low, high):  # noqa: F811
    """Scales inside and outside fp16's range, mixed within a step."""
    say("linear_grad scales %s M=%d %d..%d" % (dtype, M, low, high))
    rng = np.random.default_rng([M, low])
    codes, scales = weights(rng, (200, 320), low, high)
    dy = rng.standard_normal((M, 200)) * (2.0 ** -14 if high > 200 else 1.0)
    check_grad(mx, gpu(dy, dtype), codes, scales)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M", [2, 70, 300])
def test_far_and_nan_scales(mx, dtype, M):  # noqa: F811
    """Scale bytes 253 and 254 (weights past bf16) enter exactly, 255 makes its block's columns
    NaN, wherever a step first meets them."""
    say("linear_grad far scales %s M=%d" % (dtype, M))
    rng = np.random.default_rng(M)
    N, K = 330, 320
    codes, scales = weights(rng, (N, K))
    scales[300, 4] = 253
    scales[17, 0] = 254
    dy = rng.standard_normal((M, N)) * 2.0 ** -10
    check_grad(mx, gpu(dy, dtype), codes, scales)
    scales[40, 7] = 255
    got = check_grad(mx, gpu(dy, dtype), codes, scales)
    # fp16 overflows to infinity where a weight of 2^126 or more meets 2^-10
    assert got[:, 224:256].isnan().all() and not got[:, :224].isnan().any()


@pytest.mark.parametrize("M", [1, 50, 400])
def test_not_finite_rows_stay_rows(mx, M):  # noqa: F811
    rng = np.random.default_rng(M)
    codes, scales = (gpu(t) for t in weights(rng, (96, 256)))
    dy = gpu(rng.standard_normal((M + 2, 96)), torch.bfloat16)
    clean = mx.linear_grad(dy, codes, scales)
    dy[M // 2, 5], dy[M + 1, 9] = float("nan"), float("inf")
    got = mx.linear_grad(dy, codes, scales)
    assert got[M // 2].isnan().all() and not got[M + 1].isfinite().any()
    rest = [r for r in range(M + 2) if r not in (M // 2, M + 1)]
    assert torch.equal(got[rest], clean[rest])


def test_empty_sizes(mx):  # noqa: F811
    u = torch.empty((0, 32), dtype=torch.uint8, device="cuda")
    s = torch.empty((0, 2), dtype=torch.uint8, device="cuda")
    dy = torch.empty((5, 0), dtype=torch.bfloat16, device="cuda")
    assert torch.equal(mx.linear_grad(dy, u, s), torch.zeros((5, 64), dtype=dy.dtype, device="cuda"))
    none = torch.empty((7, 0), dtype=torch.uint8, device="cuda")
    assert mx.linear_grad(torch.ones((5, 7), dtype=dy.dtype, device="cuda"), none, none).shape == (5, 0)
    codes, scales = (gpu(t) for t in weights(np.random.default_rng(1), (7, 64)))
    assert mx.linear_grad(torch.empty((0, 7), dtype=dy.dtype, device="cuda"), codes,
                          scales).shape == (0, 64)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M", [4, 40])
def test_slices_and_workspaces(mx, dtype, M):  # noqa: F811
    """N slices through a dirty, larger workspace, and none; twice the same."""
    N, K = 8192, 256
    need = mx.library().mxfp4_linear_grad_workspace_bytes(M, N, K)
    assert need > 0
    rng = np.random.default_rng(M)
    codes, scales = weights(rng, (N, K))
    dy = gpu(rng.standard_normal((M, N)), dtype)
    ws = torch.full((need + 32,), 255, dtype=torch.uint8, device="cuda")
    first = check_grad(mx, dy, codes, scales, workspace=ws)
    assert torch.equal(first, mx.linear_grad(dy, gpu(codes), gpu(scales)))
    c, s, dx = gpu(codes), gpu(scales), torch.empty_like(first)
    assert mx.library().mxfp4_linear_grad(dy.data_ptr(), 0 if dtype == torch.float16 else 1, M, N,
                                          c.data_ptr(), s.data_ptr(), N, K, dx.data_ptr(), None, 0,
                                          torch.cuda.current_stream().cuda_stream) == 0
    ref.check(dx, *expect(ref.f64(dy), codes, scales, dtype), dtype)


def test_writes_only_its_output(mx):  # noqa: F811
    rng = np.random.default_rng(2)
    for M in (3, 45, 200):
        codes, scales = (gpu(t) for t in weights(rng, (70, 96)))
        room = torch.full((M + 2, 96), float("nan"), dtype=torch.float16, device="cuda")
        mx.linear_grad(gpu(rng.standard_normal((M, 70)), torch.float16), codes, scales, dX=room[1:-1])
        assert room[0].isnan().all() and room[-1].isnan().all() and room[1:-1].isfinite().all()


def test_is_the_product_s_difference(mx):  # noqa: F811
    """<linear(x + d) - linear(x), dY> = <d, linear_grad(dY)>: d and x are powers of two, so that
    the differences of the 32-bit sums are the product's own."""
    rng = np.random.default_rng(9)
    M, N, K = 24, 160, 128
    codes, scales = weights(rng, (N, K), 124, 127)
    c, s = gpu(codes), gpu(scales)
    dy = rng.choice([-1.0, 1.0, 2.0], (M, N))
    x, d = rng.choice([-1.0, 1.0], (M, K)), np.zeros((M, K))
    d[:, ::5] = 1.0
    both = [ref.f64(mx.grouped_linear(gpu(v, torch.bfloat16), c[None], s[None],
                                      gpu(np.array([0, M], dtype=np.int32)), dtype=torch.float32))
            for v in (x + d, x)]
    left = ((both[0] - both[1]) * dy).sum(axis=1)
    grad = ref.f64(mx.grouped_linear_grad(gpu(dy, torch.bfloat16), c[None], s[None],
                                          gpu(np.array([0, M], dtype=np.int32)), dtype=torch.float32))
    # small multiples of 2^-4 below 2^12: every sum is exact
    assert np.array_equal(left, (d * grad).sum(axis=1))


# -------------------------------------------------------------------- experts

@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("name", list(RAGGED))
@pytest.mark.parametrize("N,K", [(40, 96), (129, 288), (64, 1056)])
def test_grouped_linear_grad(mx, dtype, name, N, K):  # noqa: F811
    say("grouped_linear_grad %s %s N=%d K=%d" % (dtype, name, N, K))
    for scale in (1, 3, 14):
        offsets = [o * scale for o in RAGGED[name]]
        E, R = 4, 80 * scale
        rng = np.random.default_rng([N, K, scale])
        codes, scales = weights(rng, (E, N, K))
        dy = gpu(rng.standard_normal((R, N)), dtype)
        want, bound = np.zeros((R, K)), np.zeros((R, K))
        for e, (lo, hi) in enumerate(ranges(offsets, R)):
            want[lo:hi], mags = ref.product(ref.f64(dy)[lo:hi], ref.values(codes[e], scales[e]).T)
            bound[lo:hi] = ref.sum_bound(N, mags)
        o = gpu(np.array(offsets, dtype=np.int32))
        for out in (dtype, torch.float32):
            got = mx.grouped_linear_grad(dy, gpu(codes), gpu(scales), o, dtype=out)
            ref.check(got, want, bound + ref.rounded(np.abs(want), out), out)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("rows", [(3, 0, 17, 1), (17, 0, 33, 1), (40, 31, 50, 1), (97, 65, 1, 100),
                                  (129, 40, 250, 3)])
@pytest.mark.parametrize("N,pad", [(320, 8), (333, 3)])
def test_part_filled_tiles(mx, dtype, rows, N, pad):  # noqa: F811
    """Tiles of every height with fewer rows than they hold, rows of dY apart with NaN between: an
    expert's last row, which may stand for those that are not there, changes no other row, nor does a
    neighbour's."""
    K, R = 544, sum(rows)
    say("part-filled tiles %s %s N=%d" % (dtype, rows, N))
    rng = np.random.default_rng([N, R])
    codes, scales = weights(rng, (4, N, K))
    offsets = np.concatenate([[0], np.cumsum(rows)])
    room = torch.full((R, N + pad), float("nan"), dtype=dtype, device="cuda")
    dy = room[:, :N]
    dy.copy_(gpu(rng.standard_normal((R, N)), dtype))
    args = gpu(codes), gpu(scales), gpu(offsets.astype(np.int32))
    got = mx.grouped_linear_grad(dy, *args)
    for e in range(4):
        lo, hi = offsets[e], offsets[e + 1]
        ref.check(got[lo:hi], *expect(ref.f64(dy[lo:hi]), codes[e], scales[e], dtype), dtype)
    last = torch.tensor([int(offsets[e + 1]) - 1 for e in range(4) if rows[e]], device="cuda")
    dy[last] = float("nan")
    spoilt = mx.grouped_linear_grad(dy, *args)
    assert spoilt[last].isnan().all()
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[last] = False
    assert torch.equal(spoilt[keep], got[keep])


def test_grouped_experts_past_32_bits(mx):  # noqa: F811
    """Codes of more than 2^32 bytes: the last experts' weights lie past 32-bit offsets."""
    E, N, K = 5, 65536, 32768
    rng = np.random.default_rng(4)
    codes = torch.zeros((E, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((E, N, K // 32), 127, dtype=torch.uint8, device="cuda")
    part, ps = weights(rng, (64, K))
    codes[4, -64:], scales[4, -64:] = gpu(part), gpu(ps)
    for rows in (4, 40):
        dy = torch.zeros((rows, N), dtype=torch.bfloat16, device="cuda")
        dy[:, -64:] = gpu(rng.standard_normal((rows, 64)))
        offsets = gpu(np.array([0, 0, 0, 0, 0, rows], dtype=np.int32))
        got = mx.grouped_linear_grad(dy, codes, scales, offsets)
        want, bound = expect(ref.f64(dy[:, -64:]), part, ps, torch.bfloat16)
        ref.check(got, want, bound + 0 * want, torch.bfloat16)
