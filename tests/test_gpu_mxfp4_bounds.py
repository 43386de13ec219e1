"""Offsets that fall, offsets past 32 bits, workspaces that are too small: the MXFP4 and
expert operators at the edges of their memory, against the 64-bit reference (bounds
derived in mxfp4_reference)."""
import numpy as np
import pytest

import mxfp4_reference as ref
from test_gpu_moe import check_grouped, check_plan, experts
from test_gpu_mxfp4 import HALVES, check_linear, gpu, mx, random_weight, say  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


# ------------------------------------------------------------- any offsets at all

@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("offsets", [[-5, 40, 20, 900], [0, 0, 0, 0], [70, 70, 70, 70], [9, 3, 60, 1],
                                     [2 ** 31 - 1, -2 ** 31, 5, 2 ** 31 - 1], [1, 69, 2, 68]])
@pytest.mark.parametrize("rows", [2, 70, 500, 700])       # each kernel
@pytest.mark.parametrize("swiglu", [False, True])
def test_every_row_is_written_once(mx, dtype, offsets, rows, swiglu):  # noqa: F811
    """An entry counts as at least 0 and those before it, at most R: a falling pair is
    an empty expert, rows of no expert are 0, and no row keeps what it held."""
    say("offsets %s rows=%d %s" % (offsets, rows, dtype))
    rng = np.random.default_rng(rows)
    codes, scales = experts(rng, 3, 50, 96, 112, 122)
    x = gpu(rng.standard_normal((rows, 96)), dtype)
    y = torch.full((rows, 25 if swiglu else 50), float("nan"), dtype=dtype, device="cuda")
    mx.grouped_linear(x, gpu(codes), gpu(scales), gpu(np.array(offsets), torch.int32), swiglu=swiglu,
                      Y=y)
    starts = np.maximum.accumulate(np.clip(offsets, 0, rows))
    h, bound = np.zeros((rows, 50)), np.zeros((rows, 50))
    for e in range(3):
        own = slice(starts[e], starts[e + 1])
        h[own], mags = ref.product(ref.f64(x)[own], ref.values(codes[e], scales[e]))
        bound[own] = ref.sum_bound(96, mags)
    if swiglu:
        h, bound = ref.swiglu(h, bound)
    ref.check(y, h, bound + ref.rounded(np.abs(h) + bound, dtype), dtype)
    assert (y[:starts[0]] == 0).all() and (y[starts[3]:] == 0).all()


# -------------------------------------------------- few experts, many experts

@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("counts", [[1, 0, 2, 0, 1, 0, 0, 0], [3, 9, 0, 17, 1, 40, 2, 8], [64] * 8])
def test_few_experts_of_a_long_k(mx, dtype, counts):  # noqa: F811
    """Eight experts of 14336 columns: less than a row each, ten, and 64."""
    say("long K %s rows=%d" % (dtype, sum(counts)))
    rng = np.random.default_rng(sum(counts))
    codes, scales = experts(rng, 8, 100, 14336, 112, 122)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    check_grouped(mx, gpu(rng.standard_normal((offsets[-1], 14336)), dtype), codes, scales, offsets)


@pytest.mark.parametrize("E,mean", [(129, 1), (256, 5), (256, 40), (200, 200), (1024, 30)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_many_experts_of_every_block_size(mx, E, mean, swiglu):  # noqa: F811
    """Groups past one and two scans of 64, uneven, for each kernel."""
    rng = np.random.default_rng([E, mean])
    counts = rng.integers(0, 2 * mean + 1, E)
    counts[rng.random(E) < 0.2] = 0
    counts[E // 2] += max(0, E * mean - counts.sum())     # the mean, by one large expert
    offsets = np.concatenate([[0], np.cumsum(counts)])
    say("many experts E=%d rows=%d" % (E, offsets[-1]))
    codes, scales = experts(rng, E, 40, 64, 112, 122)
    x = gpu(rng.standard_normal((500, 64)), torch.bfloat16)
    check_grouped(mx, x, codes, scales, offsets, tokens=rng.integers(-1, 501, offsets[-1]),
                  swiglu=swiglu)


# --------------------------------------------------------------- past 32 bits

@pytest.mark.parametrize("M", [2, 9, 16, 20])
def test_far_rows_of_x(mx, M):  # noqa: F811
    """The stream kernel (to 16 rows) and the 32 x 256 block: rows of X that begin past
    2^32 elements.  Their outputs cannot: M N stays below 2^29."""
    say("far rows M=%d" % M)
    rng = np.random.default_rng(M)
    stride = min((1 << 33) // (M - 1) // 8 * 8, 1 << 32)
    assert (M - 1) * stride >= 1 << 32
    big = torch.empty((M - 1) * stride + 96, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((M, 96), (stride, 1))
    x.copy_(gpu(rng.standard_normal((M, 96)), torch.bfloat16))
    check_linear(mx, x, *random_weight(rng, 300, 96))


@pytest.mark.parametrize("per", [1, 40, 200])
def test_far_tokens(mx, per):  # noqa: F811
    """Gathered rows of X past 2^31 elements, for each kernel."""
    say("far tokens per=%d" % per)
    stride, rows = 1 << 20, 2100
    big = torch.empty((rows - 1) * stride + 64, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((rows, 64), (stride, 1))
    x.fill_(0)
    x[rows - 1] = 1
    x[7] = 2
    codes = torch.full((3, 40, 32), 0x22, dtype=torch.uint8, device="cuda")       # ones
    scales = torch.full((3, 40, 2), 127, dtype=torch.uint8, device="cuda")
    R = 2 if per == 1 else 3 * per
    tokens = torch.full((R,), rows - 1, dtype=torch.int32, device="cuda")
    tokens[1] = 7
    offsets = torch.tensor([0, R, R, R], dtype=torch.int32, device="cuda")
    y = mx.grouped_linear(x, codes, scales, offsets, tokens=tokens)
    want = torch.full_like(y, 64.0)
    want[1] = 128
    assert torch.equal(y, want)


def test_far_outputs_of_the_small_tiling(mx):  # noqa: F811
    """64 columns and as many rows as there may be: bytes past 2^32 (2^30 elements of
    fp32; more cannot be reached with 64 columns)."""
    M, N = 1 << 24, 64
    say("far outputs M=%d" % M)
    a = torch.zeros((M, 16), dtype=torch.uint8, device="cuda")
    sa = torch.full((M, 1), 127, dtype=torch.uint8, device="cuda")
    a[-1], a[5] = 0x22, 0x44
    b = torch.full((N, 16), 0x22, dtype=torch.uint8, device="cuda")
    sb = torch.full((N, 1), 127, dtype=torch.uint8, device="cuda")
    y = mx.matmul(a, sa, b, sb, dtype=torch.float32)
    assert (y[-1] == 32).all() and (y[5] == 64).all()
    assert int(torch.count_nonzero(y[1 << 20:])) == N and int(torch.count_nonzero(y[:1 << 20])) == N


@pytest.mark.parametrize("dtype", HALVES + [torch.float32])
def test_far_rows_of_the_quantizer(mx, dtype):  # noqa: F811
    """Dense past 2^31 elements, and rows that lie past 2^32, there and back."""
    say("far quantizer %s" % dtype)
    K = 1 << 15
    x = torch.zeros(((1 << 16) + 3, K), dtype=dtype, device="cuda")
    last = gpu(np.random.default_rng(1).standard_normal((2, K)), dtype)
    x[-2:] = last
    codes, scales = mx.quantize(x)
    nib, s = ref.quantize(ref.f64(last))
    assert np.array_equal(codes[-2:].cpu().numpy(), ref.pack(nib))
    assert np.array_equal(scales[-2:].cpu().numpy(), s)
    assert int(torch.count_nonzero(codes[:-2])) == 0 and (scales[:-2] == 127).all()
    y = mx.dequantize(codes, scales, dtype=dtype)
    assert torch.equal(y[-2:].cpu(), torch.from_numpy(ref.values(ref.pack(nib), s)).to(dtype))
    assert int(torch.count_nonzero(y[:-2])) == 0
    del y, codes, scales
    two = x.view(-1).as_strided((2, 64), ((1 << 31) + 64, 1))
    codes, scales = mx.quantize(two)
    nib, s = ref.quantize(ref.f64(two))
    assert np.array_equal(codes.cpu().numpy(), ref.pack(nib)) and np.array_equal(scales.cpu().numpy(), s)


def test_far_rows_of_the_weighted_sum(mx):  # noqa: F811
    """Rows of Y and of the result past 2^31 elements."""
    say("far weighted sum")
    R, N = (1 << 16) + 9, 1 << 15
    y = torch.zeros((R, N), dtype=torch.bfloat16, device="cuda")
    y[-1], y[3] = 2, 8
    pos = torch.full((R, 1), -1, dtype=torch.int32, device="cuda")
    pos[0], pos[-1] = R - 1, 3
    out = mx.combine(y, pos, torch.full((R, 1), 0.5, device="cuda"))
    assert (out[0] == 1).all() and (out[-1] == 4).all()
    assert int(torch.count_nonzero(out[1:-1])) == 0


def test_far_rows_of_the_router(mx):  # noqa: F811
    say("far router")
    T, E = 1 << 23, 260
    x = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    x[-1, 259], x[-1, 7], x[0, 100] = 2, 1, 3
    ids, w = mx.route(x, 2)
    assert ids[-1].tolist() == [259, 7] and ids[0].tolist() == [100, 0]
    assert (ids[1:-1] == torch.tensor([0, 1], dtype=torch.int32, device="cuda")).all()
    assert (w[1:-1] == 0.5).all()


def test_largest_plan(mx):  # noqa: F811
    """2^24 choices, in 4096 blocks."""
    say("largest plan")
    check_plan(mx, np.random.default_rng(2).integers(-1, 64, (1 << 22, 4)), 64)


# ---------------------------------------------------------------- workspaces

def test_a_workspace_too_small_is_refused(mx):  # noqa: F811
    M, N, K = 50, 512, 8192
    rng = np.random.default_rng(3)
    c, s = (gpu(t) for t in random_weight(rng, N, K))
    x = gpu(rng.standard_normal((M, K)), torch.bfloat16)
    a, sa = mx.quantize(x)
    for call, ws in ((lambda w: mx.linear(x, c, s, workspace=w), mx.linear_workspace(M, N, K)),
                     (lambda w: mx.matmul(a, sa, c, s, workspace=w), mx.matmul_workspace(M, N, K))):
        assert ws.numel() > 1
        with pytest.raises(mx.MXFP4Error) as e:
            call(ws[:-1])
        assert e.value.status == 1
        with pytest.raises(mx.MXFP4Error) as e:
            call(torch.cat((ws, ws))[8:])
        assert e.value.status == 3
        y = call(ws)
        # larger memory, whatever it holds, and what lies behind it
        more = torch.full((ws.numel() + 64,), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(call(more), y) and (more[-64:] == 255).all()
