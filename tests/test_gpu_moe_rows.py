"""Experts' rows kept in fp32 up to the weighted sum, against the plain 64-bit
reference (bounds derived in mxfp4_reference)."""
import numpy as np
import pytest

import mxfp4_reference as ref
from test_gpu_moe import RAGGED, experts, gpu, mx, say  # noqa: F401
from test_gpu_mxfp4_tiles import GROUPS

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

HALVES = [torch.float16, torch.bfloat16]
F32 = torch.float32
COUNTS = dict(GROUPS, decode=RAGGED["decode"], larger=RAGGED["larger"])


def product(x, codes, scales, offsets):
    """(rows, bound on fp32 sums) in 64 bits."""
    R, N = len(x), codes.shape[1]
    h, bound = np.zeros((R, N)), np.zeros((R, N))
    for e in range(len(codes)):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            h[lo:hi], mags = ref.product(x[lo:hi], ref.values(codes[e], scales[e]))
            bound[lo:hi] = ref.sum_bound(x.shape[1], mags)
    return h, bound


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("N,K", [(96, 128), (129, 352), (300, 1056)])
def test_rows_in_fp32(mx, dtype, name, N, K):  # noqa: F811
    """No rounding to 16 bits: the bound is that of the fp32 sums alone."""
    say("fp32 rows %s %s N=%d K=%d" % (dtype, name, N, K))
    rng = np.random.default_rng([N, K, len(name)])
    offsets = np.concatenate([[0], np.cumsum(COUNTS[name])])
    codes, scales = experts(rng, len(offsets) - 1, N, K)
    x = gpu(rng.standard_normal((offsets[-1] + 3, K)), dtype)     # three rows of no expert
    args = x, gpu(codes), gpu(scales), gpu(offsets, torch.int32)
    y = mx.grouped_linear(*args, dtype=F32)
    assert y.dtype == F32
    want, bound = product(ref.f64(x), codes, scales, offsets)
    ref.check(y, want, bound + ref.rounded(np.abs(want) + bound, F32), F32)
    assert (y[-3:] == 0).all()
    # the 16-bit rows are these, rounded
    assert torch.equal(mx.grouped_linear(*args), y.to(dtype))
    # any element-aligned Y, and nothing around it
    out = torch.full((y.numel() + 9,), 7.0, device="cuda")
    inner = out[3:3 + y.numel()].view(y.shape)
    mx.grouped_linear(*args, Y=inner, dtype=F32)
    assert torch.equal(inner, y) and (out[:3] == 7).all() and (out[3 + y.numel():] == 7).all()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (3, 6, 64), (70, 2, 1001), (300, 8, 776)])
@pytest.mark.parametrize("at", [0, 1])
def test_combine_fp32_rows(mx, dtype, T, k, N, at):  # noqa: F811
    say("combine fp32 rows %s T=%d k=%d N=%d" % (dtype, T, k, N))
    rng = np.random.default_rng([T, k, N])
    R = T * k
    y = torch.empty(R * N + at, device="cuda")[at:].view(R, N)
    y.copy_(gpu(rng.standard_normal((R, N)), F32))
    pos = rng.permutation(R).reshape(T, k)
    pos = np.where(rng.random((T, k)) < 0.15, rng.choice([-1, R, 2 ** 31 - 1, -2 ** 31]), pos)
    w = gpu(rng.random((T, k)), F32)
    out = mx.combine(y, gpu(pos, torch.int32), w, dtype=dtype)
    check_sum(out, ref.f64(y), np.zeros((R, N)), pos, ref.f64(w), dtype)


def check_sum(out, rows, bound, pos, w, dtype):
    """out against the weighted sum of rows known to `bound`: k products and sums in
    fp32, one rounding."""
    T, k = pos.shape
    want, b, mags = (np.zeros((T, rows.shape[1])) for _ in range(3))
    for j in range(k):
        used = (pos[:, j] >= 0) & (pos[:, j] < len(rows))
        want[used] += w[used, j:j + 1] * rows[pos[used, j]]
        mags[used] += np.abs(w[used, j:j + 1]) * np.abs(rows[pos[used, j]])
        b[used] += np.abs(w[used, j:j + 1]) * bound[pos[used, j]]
    b += (k + 2) * 2.0 ** -24 * (mags + b)
    assert out.dtype == dtype
    ref.check(out, want, b + ref.rounded(np.abs(want) + b, dtype), dtype)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("T,E,k", [(4, 16, 3), (120, 4, 2), (300, 8, 8)])
def test_down_projection_rounds_once(mx, dtype, T, E, k):  # noqa: F811
    """The product by expert and the sum over a token's experts, as one: a single
    rounding to 16 bits, also where the experts' rows nearly cancel."""
    say("down rounds once %s T=%d E=%d k=%d" % (dtype, T, E, k))
    rng = np.random.default_rng([T, E, k])
    K, N = 224, 140
    ids, w = mx.route(gpu(rng.standard_normal((T, E)), F32), k)
    p = mx.plan(ids, E)
    x = gpu(rng.standard_normal((T * k, K)), dtype)
    codes, scales = experts(rng, E, N, K, 112, 122)
    y = mx.grouped_linear(x, gpu(codes), gpu(scales), p.offsets, dtype=F32)
    out = mx.combine(y, p.positions, w, dtype=dtype)
    rows, bound = product(ref.f64(x), codes, scales, p.offsets.cpu().numpy())
    bound += 2.0 ** -24 * (np.abs(rows) + bound)              # y is stored in fp32
    check_sum(out, rows, bound, p.positions.cpu().numpy(), ref.f64(w), dtype)


def test_dtype_refusals(mx):  # noqa: F811
    c = torch.zeros(2, 8, 32, dtype=torch.uint8, device="cuda")
    s = torch.zeros(2, 8, 2, dtype=torch.uint8, device="cuda")
    x = torch.zeros(5, 64, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    pos, w = off[None], torch.zeros(1, 3, device="cuda")
    y32 = torch.zeros(5, 8, device="cuda")
    for call in (lambda: mx.grouped_linear(x, c, s, off, dtype=torch.float16),
                 lambda: mx.grouped_linear(x, c, s, off, dtype=F32, swiglu=True),
                 lambda: mx.grouped_linear(x, c, s, off, dtype=torch.float64),
                 lambda: mx.grouped_linear(x, c, s, off, Y=y32),
                 lambda: mx.grouped_linear(x, c, s, off, Y=y32.bfloat16(), dtype=F32),
                 lambda: mx.combine(y32, pos, w), lambda: mx.combine(y32, pos, w, dtype=F32),
                 lambda: mx.combine(x, pos, w, dtype=torch.float16),
                 lambda: mx.combine(y32, pos, w, dtype=x.dtype, out=y32[:1])):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("T", [1, 16, 300])
def test_example_router_is_not_quantized(T):
    """The example's layer takes the experts that its router, as given, chooses."""
    from weight_only_int4_gemv_amd import moe_example, mxfp4
    say("example router T=%d" % T)
    rng = np.random.default_rng(T)
    E, K, F = 16, 256, 32
    router = gpu(rng.standard_normal((E, K)) / K ** 0.5, torch.bfloat16)
    layer = moe_example.Layer(gpu(rng.standard_normal((E, 2 * F, K)), torch.bfloat16),
                              gpu(rng.standard_normal((E, K, F)), torch.bfloat16), router, 3)
    x = gpu(rng.standard_normal((T, K)), torch.bfloat16)
    logits = layer.logits(x)
    want, mags = ref.product(ref.f64(x), ref.f64(router))
    # fp32 sums of any order: a rounding for each product and sum
    bound = K * 2.0 ** -23 * mags
    assert (np.abs(ref.f64(logits) - want) <= bound).all()
    ids, weights = mxfp4.route(logits, 3)
    want_ids, want_weights = ref.route(want, 3, True)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    # |dw| <= 2 w (1 - w) max |dl| for a softmax, whose own terms are a few units off
    assert np.abs(ref.f64(weights) - want_weights).max() <= bound.max() / 2 + 2.0 ** -20
