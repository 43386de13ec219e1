"""MXFP4 quantizer, dequantizer and products on the GPU against the plain 64-bit
reference (bounds derived in mxfp4_reference)."""
import numpy as np
import pytest

import mxfp4_reference as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

FLOATS = [torch.float16, torch.bfloat16, torch.float32]
HALVES = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def mx():
    assert torch.cuda.is_available()
    from weight_only_int4_gemv_amd import mxfp4
    mxfp4.library()
    return mxfp4


def say(msg):
    print("[case] " + msg, flush=True)


def gpu(x, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda", dtype)


def random_weight(rng, N, K, low=110, high=127):
    """Packed codes and scale bytes, every code and the scales low..high."""
    return (rng.integers(0, 256, (N, K // 2), dtype=np.uint8),
            rng.integers(low, high + 1, (N, K // 32)).astype(np.uint8))


def check_quantize(mx, x):
    codes, scales = mx.quantize(x)
    nib, s = ref.quantize(ref.f64(x).reshape(-1, x.shape[-1]))
    assert np.array_equal(scales.cpu().numpy().reshape(s.shape), s)
    assert np.array_equal(codes.cpu().numpy().reshape(-1, x.shape[-1] // 2), ref.pack(nib))


# ---------------------------------------------------------------- quantizer

@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 96), (17, 4096), (129, 1184), (1000, 64), (5, 20000 * 32)])
def test_quantize_random(mx, dtype, rows, K):
    say("quantize %s %dx%d" % (dtype, rows, K))
    rng = np.random.default_rng([rows, K])
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-12, 13, (rows, 1)))
    check_quantize(mx, gpu(x, dtype))


@pytest.mark.parametrize("dtype", HALVES)
def test_quantize_every_16_bit_pattern(mx, dtype):
    """Each pattern leads a block of smaller values, and fills blocks with its neighbours."""
    say("quantize all patterns %s" % dtype)
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    every = bits.view(dtype)
    check_quantize(mx, every.view(-1, 32).cuda())
    lead = every[:, None].repeat(1, 32)
    factor = torch.tensor([1.0] + [0.9 ** i for i in range(1, 32)], dtype=torch.float64)
    rest = (lead.double() * factor * torch.where(torch.arange(32) % 3 == 0, -1.0, 1.0))
    check_quantize(mx, rest.to(dtype).cuda())


def test_quantize_ties_and_borders(mx):
    """Every midpoint of the grid and its fp32 neighbours, under every peak binade
    that keeps them representable, with both signs."""
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=np.float32)
    vals = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(9)),
                           [6.0, 5.99, 0.0]]).astype(np.float32)
    block = np.concatenate([vals, np.full(32 - 1 - len(vals), 1.0, np.float32), [4.0]])
    rows = [np.ldexp(block * sign, e).astype(np.float32) for e in range(-120, 125, 7)
            for sign in (1, -1)]
    say("quantize ties")
    check_quantize(mx, gpu(np.stack(rows)))


@pytest.mark.parametrize("dtype", FLOATS)
def test_quantize_special_blocks(mx, dtype):
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    sub = 2.0 ** {torch.float16: -24, torch.bfloat16: -133, torch.float32: -149}[dtype]
    x = torch.zeros(12, 64, dtype=torch.float64)
    x[1, :32] = -0.0
    x[2, 5], x[2, 40] = float("inf"), 1.0
    x[3, 31], x[3, 32] = float("nan"), -2.0
    x[4, 7] = -float("inf")
    x[5] = big
    x[6, ::2], x[6, 1::2] = tiny, -tiny / 2
    x[7] = sub
    x[8, 0], x[8, 1:] = big, sub
    x[9, 63] = 3 * sub
    x[10, :32] = torch.linspace(-7.9, 7.9, 32)
    x[11, 1], x[11, 33] = 1.0, float("nan")
    say("quantize special %s" % dtype)
    check_quantize(mx, x.to(dtype).cuda())


@pytest.mark.parametrize("dtype", FLOATS)
def test_quantize_strided_and_3d(mx, dtype):
    rng = np.random.default_rng(3)
    say("quantize strided %s" % dtype)
    wide = gpu(rng.standard_normal((37, 352)), dtype)
    check_quantize(mx, wide[:, :160])
    check_quantize(mx, wide[::3, 32:320])
    check_quantize(mx, wide[5:6, 64:128])
    cube = gpu(rng.standard_normal((3, 5, 64)), dtype)
    codes, scales = mx.quantize(cube)
    assert codes.shape == (3, 5, 32) and scales.shape == (3, 5, 2)
    check_quantize(mx, cube)
    assert mx.quantize(cube[:0])[0].shape == (0, 5, 32)


@pytest.mark.parametrize("dtype", FLOATS)
def test_dequantize_every_code_and_scale(mx, dtype):
    say("dequantize %s" % dtype)
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))          # 512 columns
    scales = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, 16))
    got = mx.dequantize(gpu(codes), gpu(scales), dtype=dtype).cpu()
    with np.errstate(all="ignore"):
        want = torch.from_numpy(ref.values(codes, scales)).to(dtype)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok], want[ok])


# ------------------------------------------------------------------- linear

LINEAR_SHAPES = [(1, 1, 32), (1, 33, 96), (2, 14336, 64), (1, 257, 4096), (3, 100, 1184), (16, 64, 512),
                 (17, 31, 2080), (33, 130, 160), (50, 512, 1440), (64, 96, 4064), (65, 200, 256),
                 (129, 129, 1056), (200, 300, 704), (257, 513, 96), (300, 640, 4096), (1, 5, 0)]


def check_linear(mx, x, codes, scales, **kw):
    y = mx.linear(x, gpu(codes), gpu(scales), **kw)
    w = ref.values(codes, scales)
    want, mags = ref.product(ref.f64(x), w)
    bound = ref.sum_bound(w.shape[1], mags)
    ref.check(y, want, bound + ref.rounded(np.abs(want) + bound, x.dtype), x.dtype)
    return y


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M,N,K", LINEAR_SHAPES)
def test_linear(mx, dtype, M, N, K):
    say("linear %s M=%d N=%d K=%d" % (dtype, M, N, K))
    rng = np.random.default_rng([M, N, K])
    codes, scales = random_weight(rng, N, K)
    check_linear(mx, gpu(rng.standard_normal((M, K)), dtype), codes, scales)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M", [1, 20, 40, 150, 400])
@pytest.mark.parametrize("low,high", [(0, 20), (90, 110), (100, 108), (136, 146), (0, 160)])
def test_linear_scale_ranges(mx, dtype, M, low, high):
    """Scales around and far past the fp16 range, tiny and huge together."""
    say("linear scales %s M=%d %d..%d" % (dtype, M, low, high))
    rng = np.random.default_rng([M, low, high])
    codes, scales = random_weight(rng, 150, 544, low, high)
    x = rng.standard_normal((M, 544)) * 2.0 ** (8 if dtype == torch.float16 else 80)
    check_linear(mx, gpu(x, dtype), codes, scales)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M", [1, 9, 70, 330])
def test_linear_one_hot_is_exact(mx, dtype, M):
    """A one-hot row picks one weight: no error at all (weights that fit dtype)."""
    rng = np.random.default_rng(M)
    N, K = 70, 1120
    codes, scales = random_weight(rng, N, K, 116, 130)
    cols = rng.integers(0, K, M)
    x = np.zeros((M, K))
    x[np.arange(M), cols] = 1
    say("linear one-hot %s M=%d" % (dtype, M))
    y = mx.linear(gpu(x, dtype), gpu(codes), gpu(scales))
    assert np.array_equal(ref.f64(y), ref.values(codes, scales).T[cols])


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M", [3, 40, 290])
@pytest.mark.parametrize("wide", [False, True])
def test_linear_not_finite(mx, dtype, M, wide):
    """Infinities and NaN in X stay in their rows, a NaN scale in its column."""
    rng = np.random.default_rng([M, wide])
    N, K = 100, 320
    codes, scales = random_weight(rng, N, K, *((60, 150) if wide else (118, 124)))
    codes = np.where(codes & 7 == 0, codes | 1, codes)
    codes = np.where(codes & 0x70 == 0, codes | 0x10, codes)       # inf times 0 is tested below
    x = rng.standard_normal((M, K))
    x[0, 7], x[1, 300], x[2, 11], x[2, 12] = np.inf, np.nan, np.inf, -np.inf
    scales[5, 3] = 255
    say("linear not finite %s M=%d" % (dtype, M))
    y = ref.f64(mx.linear(gpu(x, dtype), gpu(codes), gpu(scales)))
    keep = np.arange(N) != 5
    w = ref.values(codes, scales)
    assert np.isnan(y[:, 5]).all() and np.isnan(y[1]).all()
    assert np.array_equal(y[0, keep], np.sign(w[keep, 7]) * np.inf)
    differ = np.sign(w[:, 11]) == np.sign(w[:, 12])                # inf - inf
    assert np.isnan(y[2, keep & differ]).all()
    rest = np.arange(M) > 2
    xr = ref.f64(gpu(x, dtype))[rest]
    want, mags = ref.product(xr, w[keep])
    bound = ref.sum_bound(K, mags)
    ref.check(torch.from_numpy(y[rest][:, keep]).to(dtype), want,
              bound + ref.rounded(np.abs(want) + bound, dtype), dtype)
    codes[:] = 0
    y = ref.f64(mx.linear(gpu(x, dtype), gpu(codes), gpu(scales)))
    assert np.isnan(y[:3]).all() and (y[3:, keep] == 0).all()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M,stride", [(1, 999), (7, 328), (70, 640), (300, 352)])
def test_linear_strided_rows(mx, dtype, M, stride):
    """Rows of a wider tensor whose other columns hold NaN."""
    rng = np.random.default_rng([M, stride])
    K = 320
    wide = torch.full((M + 1, stride), float("nan"), dtype=dtype, device="cuda")
    x = gpu(rng.standard_normal((M, K)), dtype)
    wide[:M, :K] = x
    codes, scales = random_weight(rng, 77, K)
    say("linear strided %s M=%d" % (dtype, M))
    out = torch.full((M, 77), float("nan"), dtype=dtype, device="cuda")
    y = check_linear(mx, wide[:M, :K], codes, scales, Y=out)
    assert y is out and torch.equal(y, mx.linear(x, gpu(codes), gpu(scales)))


@pytest.mark.parametrize("M", [1, 50, 300])
def test_linear_writes_only_its_output(mx, M):
    rng = np.random.default_rng(M)
    N, K = 203, 416
    codes, scales = random_weight(rng, N, K)
    buf = torch.full((M * N + 64,), 7.0, dtype=torch.float16, device="cuda")
    mx.linear(gpu(rng.standard_normal((M, K)), torch.float16), gpu(codes), gpu(scales),
              Y=buf[32:32 + M * N].view(M, N))
    assert (buf[:32] == 7).all() and (buf[32 + M * N:] == 7).all()


# ------------------------------------------------------------------- matmul

MATMUL_SHAPES = [(1, 1, 32), (5, 70, 96), (31, 33, 64), (64, 64, 256), (65, 129, 544), (130, 257, 1184),
                 (200, 96, 4096), (256, 256, 512), (300, 520, 288), (513, 260, 800), (1, 300, 2080),
                 (3, 5, 0)]


def check_matmul(mx, a, sa, b, sb, dtype):
    y = mx.matmul(gpu(a), gpu(sa), gpu(b), gpu(sb), dtype=dtype)
    va, vb = ref.values(a, sa), ref.values(b, sb)
    want, mags = ref.product(va, vb)
    bound = ref.sum_bound(va.shape[1], mags)
    ref.check(y, want, bound + ref.rounded(np.abs(want) + bound, dtype), dtype)


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("M,N,K", MATMUL_SHAPES)
def test_matmul(mx, dtype, M, N, K):
    say("matmul %s M=%d N=%d K=%d" % (dtype, M, N, K))
    rng = np.random.default_rng([M, N, K])
    check_matmul(mx, *random_weight(rng, M, K, 120, 132), *random_weight(rng, N, K, 112, 124), dtype)


@pytest.mark.parametrize("M,N", [(3, 40), (100, 90), (300, 300)])
def test_matmul_scale_extremes(mx, M, N):
    """Scales of the whole byte range whose products stay in fp32's."""
    rng = np.random.default_rng([M, N])
    K = 352
    a, sa = random_weight(rng, M, K, 1, 254)
    b, _ = random_weight(rng, N, K)
    # a block's two scales multiply to 2^-20 .. 2^0 of each other's middle
    sa[:] = sa[:1]
    sb = np.clip(254 - sa[:1].astype(int) - rng.integers(0, 20, (N, K // 32)), 0, 254).astype(np.uint8)
    say("matmul extremes M=%d N=%d" % (M, N))
    check_matmul(mx, a, sa, b, sb, torch.float32)


@pytest.mark.parametrize("M,N", [(3, 40), (100, 90), (300, 300)])
def test_matmul_nan_scales(mx, M, N):
    rng = np.random.default_rng([M, N])
    a, sa = random_weight(rng, M, 224, 120, 130)
    b, sb = random_weight(rng, N, 224, 120, 130)
    sa[1, 6], sb[N - 1, 0] = 255, 255
    say("matmul NaN M=%d N=%d" % (M, N))
    check_matmul(mx, a, sa, b, sb, torch.bfloat16)


@pytest.mark.parametrize("dtype", HALVES)
def test_quantize_then_matmul_is_the_product_of_values(mx, dtype):
    rng = np.random.default_rng(9)
    x = gpu(rng.standard_normal((70, 480)), dtype)
    w = gpu(rng.standard_normal((90, 480)) * 0.02, torch.float32)
    (a, sa), (b, sb) = mx.quantize(x), mx.quantize(w)
    y = mx.matmul(a, sa, b, sb, dtype=torch.float32)
    va, vb = (ref.f64(mx.dequantize(c, s, dtype=torch.float32)) for c, s in ((a, sa), (b, sb)))
    want, mags = ref.product(va, vb)
    bound = ref.sum_bound(480, mags)
    ref.check(y, want, bound + ref.rounded(np.abs(want) + bound, torch.float32), torch.float32)


# --------------------------------------------------- refusals, streams, graphs

def test_binding_refusals(mx):
    x = torch.zeros(4, 64, dtype=torch.float16, device="cuda")
    c = torch.zeros(8, 32, dtype=torch.uint8, device="cuda")
    s = torch.zeros(8, 2, dtype=torch.uint8, device="cuda")
    bad = [lambda: mx.quantize(x[:, :40]), lambda: mx.quantize(x.t()),
           lambda: mx.quantize(x[:1].expand(4, 64)), lambda: mx.quantize(x, codes=c),
           lambda: mx.dequantize(c, s[:, :1]), lambda: mx.dequantize(c, s, dtype=torch.float64),
           lambda: mx.linear(x[:, :32], c, s), lambda: mx.linear(x.float(), c, s),
           lambda: mx.linear(x, c, s[:4]), lambda: mx.linear(x, c[::2], s[::2]),
           lambda: mx.linear(x[0], c, s), lambda: mx.linear(x, c, s, Y=x),
           lambda: mx.matmul(c, s, c[:, :16].contiguous(), s[:, :1].contiguous()),
           lambda: mx.linear(x, c, s, workspace=x)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    wide = torch.zeros(4, 70, dtype=torch.float16, device="cuda")
    with pytest.raises(mx.MXFP4Error) as e:        # rows 140 bytes apart
        mx.linear(wide[:, :64], c, s)
    assert e.value.status == 3


@pytest.mark.parametrize("M", [1, 60, 300])
def test_linear_on_another_stream(mx, M):
    rng = np.random.default_rng(M)
    codes, scales = random_weight(rng, 256, 2048)
    c, s = gpu(codes), gpu(scales)
    x = gpu(rng.standard_normal((M, 2048)), torch.bfloat16)
    want = mx.linear(x, c, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = mx.linear(x + 0, c, s)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, want)


@pytest.mark.parametrize("M", [1, 60, 300])
def test_products_replay_from_a_graph(mx, M):
    rng = np.random.default_rng(M)
    N, K = 260, 2080
    codes, scales = random_weight(rng, N, K)
    c, s = gpu(codes), gpu(scales)
    x = gpu(rng.standard_normal((M, K)), torch.bfloat16)
    say("graph M=%d" % M)

    def step():
        a, sa = mx.quantize(x)
        return mx.linear(x, c, s), mx.matmul(a, sa, c, s), mx.dequantize(a, sa)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for rep in range(4):
        x.copy_(gpu(np.random.default_rng([M, rep]).standard_normal((M, K)), torch.bfloat16))
        want = [t.clone() for t in step()]
        for t in outs:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b), "replay %d" % rep


@pytest.mark.parametrize("M", [2, 100, 400])
def test_products_are_deterministic(mx, M):
    rng = np.random.default_rng(M)
    codes, scales = random_weight(rng, 300, 4096)
    c, s = gpu(codes), gpu(scales)
    x = gpu(rng.standard_normal((M, 4096)), torch.float16)
    a, sa = mx.quantize(x)
    y, z = mx.linear(x, c, s), mx.matmul(a, sa, c, s)
    for _ in range(5):
        assert torch.equal(mx.linear(x, c, s), y) and torch.equal(mx.matmul(a, sa, c, s), z)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_offsets_past_32_bits(mx, M):
    """Rows of X more than 2^31 elements in, outputs more than 2^31 elements in."""
    say("offsets M=%d" % M)
    rng = np.random.default_rng(M)
    stride = (1 << 33) // max(M, 2) // 8 * 8
    big = torch.empty((M - 1) * stride + 64, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((M, 64), (stride, 1))
    x.copy_(gpu(rng.standard_normal((M, 64)), torch.bfloat16))
    codes, scales = random_weight(rng, 96, 64)
    check_linear(mx, x, codes, scales)
    del big, x
    N = (1 << 32) // M // 2 + 40                       # M N past 2^31
    if M > 1 and N < 1 << 24:
        codes = torch.zeros((N, 16), dtype=torch.uint8, device="cuda")
        scales = torch.full((N, 1), 127, dtype=torch.uint8, device="cuda")
        codes[-1] = 0x22                               # ones
        y = mx.linear(torch.ones((M, 32), dtype=torch.bfloat16, device="cuda"), codes, scales)
        a, sa = mx.quantize(torch.ones((M, 32), dtype=torch.bfloat16, device="cuda"))
        z = mx.matmul(a, sa, codes, scales)
        for t in (y, z):
            assert (t[:, -1] == 32).all() and (t[-1, :-1] == 0).all() and t[M // 2, 5] == 0
