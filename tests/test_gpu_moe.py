"""Routing, planning, the ragged expert product and the weighted sum on the GPU
against the plain 64-bit reference (bounds derived in mxfp4_reference)."""
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


# -------------------------------------------------------------------- routing

def check_route(mx, logits, k, renormalize):
    ids, weights = mx.route(logits, k, renormalize=renormalize)
    x = ref.f64(logits)
    want_ids, want = ref.route(x, k, renormalize)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    got = ref.f64(weights)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    # the difference to the peak is rounded once and enters the exponential, whose own
    # error is a few units; a sum of E terms; the division
    with np.errstate(all="ignore"):
        arg = np.abs(np.log(np.where(want > 0, want, 1)))
    bound = want * (x.shape[1] + 16 + 2 * arg + 2 * np.log(x.shape[1] + 1)) * 2.0 ** -24 + 2.0 ** -126
    ok = np.isnan(want) | (np.abs(got - want) <= bound)
    assert ok.all()
    assert (got[want_ids < 0] == 0).all()


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (5, 8, 8), (64, 64, 6), (33, 65, 1), (100, 128, 8),
                                   (17, 130, 32), (9, 256, 9), (40, 300, 4), (7, 1024, 32), (1000, 60, 4)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route(mx, dtype, T, E, k, renormalize):
    say("route %s T=%d E=%d k=%d" % (dtype, T, E, k))
    rng = np.random.default_rng([T, E, k])
    x = rng.standard_normal((T, E)) * 3
    x[::2] = np.round(x[::2])                              # many ties
    check_route(mx, gpu(x, dtype), k, renormalize)


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("E", [5, 64, 100, 200, 700])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_masks_and_specials(mx, dtype, E, renormalize):
    say("route specials %s E=%d" % (dtype, E))
    rng = np.random.default_rng(E)
    low = torch.finfo(dtype).min
    x = rng.standard_normal((14, E))
    x[0] = -np.inf
    x[1, 1:] = -np.inf
    x[2, ::2] = -np.inf
    x[3] = low
    x[4, 1:] = low
    x[5, 2] = np.nan
    x[6, 0] = np.inf
    x[7, 1], x[7, 4] = np.inf, np.inf
    x[8] = 0.0
    x[8, 1::2] = -0.0
    x[9] = np.nan
    x[10] = np.inf
    x[11, 0], x[11, 3] = -np.inf, np.nan
    x[12, :-1] = -np.inf
    x[13] = 60000.0
    check_route(mx, gpu(x, dtype), min(E, 4), renormalize)


@pytest.mark.parametrize("dtype", FLOATS)
def test_route_strided(mx, dtype):
    wide = torch.full((21, 90), float("inf"), dtype=dtype, device="cuda")
    wide[:, :63] = gpu(np.random.default_rng(1).standard_normal((21, 63)), dtype)
    check_route(mx, wide[:, :63], 5, True)
    check_route(mx, wide[:, 1:63], 5, False)
    check_route(mx, wide[::4, 1:62], 5, False)


# ----------------------------------------------------------------------- plan

def check_plan(mx, ids, E, **kw):
    p = mx.plan(gpu(ids, torch.int32), E, **kw)
    for got, want in zip(p, ref.plan(ids, E)):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("T,k,E", [(0, 2, 8), (1, 1, 1), (3, 6, 64), (64, 1, 3), (65, 2, 65), (500, 8, 60),
                                   (512, 8, 64), (513, 8, 1024), (2000, 4, 128), (8191, 8, 128),
                                   (40000, 3, 1000), (131, 32, 300)])
def test_plan(mx, T, k, E):
    say("plan T=%d k=%d E=%d" % (T, k, E))
    rng = np.random.default_rng([T, k, E])
    ids = rng.integers(0, E, (T, k))
    check_plan(mx, ids, E)
    ids = np.where(rng.random((T, k)) < 0.2, rng.choice([-1, E, E + 7, -2 ** 31, 2 ** 31 - 1], (T, k)), ids)
    check_plan(mx, ids, E)


@pytest.mark.parametrize("T,k", [(70, 4), (6000, 4)])
def test_plan_uneven(mx, T, k):
    check_plan(mx, np.full((T, k), 5), 9)
    check_plan(mx, np.full((T, k), -1), 9)
    check_plan(mx, np.arange(T * k).reshape(T, k) // 1000, 9)
    n = mx.library().moe_plan_workspace_bytes(T, k, 9)
    ws = torch.full((max(n, 1),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):                                   # a dirty workspace, reused
        check_plan(mx, np.arange(T * k).reshape(T, k) * 7 % 11 - 1, 9, workspace=ws)


# ------------------------------------------------------------ expert products

def experts(rng, E, N, K, low=110, high=127):
    return (rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8),
            rng.integers(low, high + 1, (E, N, K // 32)).astype(np.uint8))


def check_grouped(mx, x, codes, scales, offsets, tokens=None, swiglu=False, **kw):
    E, N = codes.shape[:2]
    K = x.shape[1]
    y = mx.grouped_linear(x, gpu(codes), gpu(scales), gpu(offsets, torch.int32),
                          tokens=None if tokens is None else gpu(tokens, torch.int32),
                          swiglu=swiglu, **kw)
    xv = ref.f64(x)
    if tokens is not None:
        inside = (tokens >= 0) & (tokens < len(xv))
        rows = np.zeros((len(tokens), K))
        rows[inside] = xv[tokens[inside]]
        xv = rows
    R = len(xv)
    h, bound = np.zeros((R, N)), np.zeros((R, N))
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            h[lo:hi], mags = ref.product(xv[lo:hi], ref.values(codes[e], scales[e]))
            bound[lo:hi] = ref.sum_bound(K, mags)
    if swiglu:
        h, bound = ref.swiglu(h, bound)
    ref.check(y, h, bound + ref.rounded(np.abs(h) + bound, x.dtype), x.dtype)
    return y


# rows of each expert
RAGGED = {
    "one row": [0, 1, 0],
    "decode": [1, 0, 0, 2, 1, 0, 1, 3, 0, 0, 1],
    "all in one": [0, 0, 150, 0],
    "around tiles": [15, 16, 17, 0, 31, 32, 33, 1],
    "large": [63, 64, 65, 130, 0, 257, 1],
    "larger": [300, 5, 700],
    "none": [0, 0],
}


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("name", list(RAGGED))
@pytest.mark.parametrize("N,K", [(96, 128), (129, 352), (34, 1056)])
def test_grouped(mx, dtype, name, N, K):
    say("grouped %s %s N=%d K=%d" % (dtype, name, N, K))
    rng = np.random.default_rng([N, K, len(name)])
    counts = RAGGED[name]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    codes, scales = experts(rng, len(counts), N, K)
    x = gpu(rng.standard_normal((offsets[-1] + 3, K)), dtype)     # three rows of no expert
    check_grouped(mx, x, codes, scales, offsets)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("name", list(RAGGED))
@pytest.mark.parametrize("F,K", [(48, 128), (33, 352), (1, 64), (130, 544)])
def test_grouped_swiglu_gathered(mx, dtype, name, F, K):
    say("swiglu %s %s F=%d K=%d" % (dtype, name, F, K))
    rng = np.random.default_rng([F, K, len(name)])
    counts = RAGGED[name]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    R = int(offsets[-1]) + 2
    codes, scales = experts(rng, len(counts), 2 * F, K, 112, 122)
    x = gpu(rng.standard_normal((37, K)), dtype)
    tokens = rng.integers(0, 37, R)
    tokens[rng.random(R) < 0.1] = rng.choice([-1, 37, 2 ** 31 - 1, -2 ** 31])
    check_grouped(mx, x, codes, scales, offsets, tokens=tokens, swiglu=True)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("per", [1, 20, 100, 400])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("low,high", [(90, 120), (118, 150), (0, 130)])
def test_grouped_scale_ranges(mx, dtype, per, swiglu, low, high):
    say("grouped scales %s per=%d %d..%d" % (dtype, per, low, high))
    rng = np.random.default_rng([per, low, high])
    offsets = np.array([0, per, per, 2 * per])
    codes, scales = experts(rng, 3, 70, 160, low, high)
    check_grouped(mx, gpu(rng.standard_normal((2 * per, 160)), dtype), codes, scales, offsets,
                  swiglu=swiglu)


@pytest.mark.parametrize("per", [2, 90])
def test_grouped_slice_of_experts(mx, per):
    """A slice of a plan's experts: rows before and after the slice are zero."""
    rng = np.random.default_rng(per)
    counts = [per, 3 * per, 0, per + 1, 2 * per]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    codes, scales = experts(rng, 3, 50, 96)
    x = gpu(rng.standard_normal((offsets[-1], 96)), torch.bfloat16)
    out = torch.full((len(x), 50), float("nan"), dtype=torch.bfloat16, device="cuda")
    y = check_grouped(mx, x, codes, scales, offsets[1:5], Y=out)
    assert (y[:per] == 0).all() and (y[offsets[4]:] == 0).all()


@pytest.mark.parametrize("per", [2, 90])
def test_grouped_not_finite(mx, per):
    """A row with an infinity or NaN, an expert with a NaN scale: nothing spreads."""
    rng = np.random.default_rng(per)
    offsets = np.array([0, per, 2 * per, 3 * per])
    codes, scales = experts(rng, 3, 40, 192)
    scales[1, 7, 2] = 255
    x = rng.standard_normal((3 * per, 192))
    x[0, 5], x[2 * per, 100] = np.nan, np.inf
    xt = gpu(x, torch.float16)
    y = mx.grouped_linear(xt, gpu(codes), gpu(scales), gpu(offsets, torch.int32))
    bad = ~np.isfinite(ref.f64(y))
    want = np.zeros_like(bad)
    want[0] = True
    want[per:2 * per, 7] = True
    rows = np.arange(3 * per) != 2 * per
    assert np.array_equal(bad[rows], want[rows]) and bad[2 * per].all()
    clean = x.copy()
    clean[0], clean[2 * per] = 0, 0
    z = mx.grouped_linear(gpu(clean, torch.float16), gpu(codes), gpu(scales),
                          gpu(offsets, torch.int32))
    ok = rows & (np.arange(3 * per) != 0)
    assert np.array_equal(ref.f64(y)[ok], ref.f64(z)[ok], equal_nan=True)


def test_grouped_writes_only_its_output(mx):
    rng = np.random.default_rng(2)
    for per in (3, 100):
        offsets = np.array([0, per, 2 * per + 1])
        R, N = 2 * per + 1, 61
        codes, scales = experts(rng, 2, N, 96)
        buf = torch.full((R * N + 64,), 7.0, dtype=torch.float16, device="cuda")
        mx.grouped_linear(gpu(rng.standard_normal((R, 96)), torch.float16), gpu(codes), gpu(scales),
                          gpu(offsets, torch.int32), Y=buf[32:32 + R * N].view(R, N))
        assert (buf[:32] == 7).all() and (buf[32 + R * N:] == 7).all()
        assert not (buf[32:32 + R * N] == 7).all()


@pytest.mark.parametrize("per", [1, 40])
def test_grouped_experts_past_32_bits(mx, per):
    """Code offsets of the last expert past 2^32 bytes."""
    E, N, K = 34, 16384, 16384
    codes = torch.zeros((E, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((E, N, K // 32), 127, dtype=torch.uint8, device="cuda")
    codes[-1, -1] = 0x22
    codes[3, 9] = 0x44
    offsets = torch.tensor([0] * 4 + [per] * (E - 4) + [2 * per], dtype=torch.int32, device="cuda")
    x = torch.ones((2 * per, K), dtype=torch.bfloat16, device="cuda")
    y = mx.grouped_linear(x, codes, scales, offsets)
    assert (y[per:, -1] == K).all() and (y[per:, :-1] == 0).all()
    assert (y[:per, 9] == 2 * K).all() and y[:per].count_nonzero() == per


def test_grouped_binding_refusals(mx):
    c = torch.zeros(2, 7, 32, dtype=torch.uint8, device="cuda")
    s = torch.zeros(2, 7, 2, dtype=torch.uint8, device="cuda")
    x = torch.zeros(5, 64, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    for call in (lambda: mx.grouped_linear(x, c, s, off[:2]),
                 lambda: mx.grouped_linear(x, c, s, off, swiglu=True),
                 lambda: mx.grouped_linear(x[:, :32], c, s, off),
                 lambda: mx.grouped_linear(x, c[0], s[0], off),
                 lambda: mx.grouped_linear(x, c, s, off.long()),
                 lambda: mx.grouped_linear(x, c, s, off, tokens=off[::2]),
                 lambda: mx.grouped_linear(x, c, s, off, Y=x),
                 lambda: mx.route(x, 65), lambda: mx.route(x, 0), lambda: mx.route(x, 33),
                 lambda: mx.plan(off[None], 0), lambda: mx.plan(off, 3),
                 lambda: mx.combine(x, off[None], torch.zeros(1, 2, device="cuda"))):
        with pytest.raises(ValueError):
            call()


# -------------------------------------------------------------------- combine

@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (3, 6, 64), (70, 2, 1001), (9, 32, 4096), (300, 8, 776), (0, 2, 8)])
def test_combine(mx, dtype, T, k, N):
    say("combine %s T=%d k=%d N=%d" % (dtype, T, k, N))
    rng = np.random.default_rng([T, k, N])
    R = T * k
    y = gpu(rng.standard_normal((R, N)), dtype)
    pos = rng.permutation(R).reshape(T, k)
    pos = np.where(rng.random((T, k)) < 0.15, rng.choice([-1, R, 2 ** 31 - 1, -2 ** 31]), pos)
    w = gpu(rng.random((T, k)), torch.float32)
    out = mx.combine(y, gpu(pos, torch.int32), w)
    yv, wv = ref.f64(y), ref.f64(w)
    want, mags = np.zeros((T, N)), np.zeros((T, N))
    for j in range(k):
        used = (pos[:, j] >= 0) & (pos[:, j] < R)
        term = wv[used, j:j + 1] * yv[pos[used, j]]
        want[used] += term
        mags[used] += np.abs(term)
    bound = (k + 1) * 2.0 ** -24 * mags
    ref.check(out, want, bound + ref.rounded(np.abs(want) + bound, dtype), dtype)


def test_combine_of_a_dropped_token_is_zero_and_drops_not_finite_rows(mx):
    y = torch.full((4, 16), float("nan"), dtype=torch.float16, device="cuda")
    y[1] = 2
    pos = torch.tensor([[-1, -1], [1, 9]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, 1.0], [0.5, float("inf")]], device="cuda")
    out = mx.combine(y, pos, w)
    assert (out[0] == 0).all() and (out[1] == 1).all()


# ------------------------------------------------------------------ the layer

def layer(mx, x, logits, k, w1, w2):
    ids, weights = mx.route(logits, k)
    p = mx.plan(ids, logits.shape[1])
    h = mx.grouped_linear(x, *w1, p.offsets, tokens=p.tokens, swiglu=True)
    return mx.combine(mx.grouped_linear(h, *w2, p.offsets), p.positions, weights)


@pytest.mark.parametrize("T", [1, 37, 500])
def test_layer_in_a_graph_and_on_another_stream(mx, T):
    rng = np.random.default_rng(T)
    E, k, K, F = 8, 3, 256, 96
    w1 = mx.quantize(gpu(rng.standard_normal((E, 2 * F, K)) * 0.05, torch.bfloat16))
    w2 = mx.quantize(gpu(rng.standard_normal((E, K, F)) * 0.05, torch.bfloat16))
    x = gpu(rng.standard_normal((T, K)), torch.bfloat16)
    logits = gpu(rng.standard_normal((T, E)), torch.float32)
    layer(mx, x, logits, k, w1, w2)
    torch.cuda.synchronize()
    say("layer graph T=%d" % T)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer(mx, x, logits, k, w1, w2)
    side = torch.cuda.Stream()
    for rep in range(4):
        r = np.random.default_rng([T, rep])
        x.copy_(gpu(r.standard_normal((T, K)), torch.bfloat16))
        logits.copy_(gpu(r.standard_normal((T, E)), torch.float32))
        if rep == 2:
            logits.fill_(-float("inf"))
        want = layer(mx, x, logits, k, w1, w2)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = layer(mx, x + 0, logits, k, w1, w2)
        torch.cuda.current_stream().wait_stream(side)
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(other, want), "replay %d" % rep
        if rep == 2:
            assert (out == 0).all()


@pytest.mark.parametrize("T,k", [(5, 2), (200, 4)])
def test_layer_equals_the_dense_sum(mx, T, k):
    """All experts chosen per token would be the dense layer: here the k chosen
    ones, each computed alone with linear()."""
    rng = np.random.default_rng([T, k])
    E, K, F = 6, 192, 64
    w1 = mx.quantize(gpu(rng.standard_normal((E, 2 * F, K)) * 0.05, torch.bfloat16))
    w2 = mx.quantize(gpu(rng.standard_normal((E, K, F)) * 0.05, torch.bfloat16))
    x = gpu(rng.standard_normal((T, K)), torch.bfloat16)
    logits = gpu(rng.standard_normal((T, E)), torch.float32)
    out = ref.f64(layer(mx, x, logits, k, w1, w2))
    ids, weights = ref.route(ref.f64(logits), k, True)
    want = np.zeros((T, K))
    for e in range(E):
        h, _ = ref.swiglu(ref.f64(x) @ ref.f64(mx.dequantize(w1[0][e], w1[1][e], torch.float32)).T,
                          np.zeros((T, 2 * F)))
        y = h @ ref.f64(mx.dequantize(w2[0][e], w2[1][e], torch.float32)).T
        want += (weights * (ids == e)).sum(axis=1)[:, None] * y
    # two 16-bit roundings on the way (h, y) and the last: bf16 2^-8 each, relative to values
    # of the order of the largest output
    assert np.abs(out - want).max() <= 4 * 2.0 ** -8 * np.abs(want).max()
