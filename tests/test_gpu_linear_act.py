"""Products with an epilogue, and the gradient through an activation, on the GPU against
plain 64-bit forms (bounds derived in mxfp4_reference and mxfp4_grad_reference)."""
import numpy as np
import pytest

import mxfp4_grad_reference as gref
import mxfp4_reference as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

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


def weights(rng, shape, low=118, high=126):
    """Random codes and scale bytes [..., K]."""
    *lead, K = shape
    codes = rng.integers(0, 256, (*lead, K // 2), dtype=np.uint8)
    scales = rng.integers(low, high + 1, (*lead, K // 32), dtype=np.uint8)
    return codes, scales


def check_linear(mx, rng, M, N, K, dtype, act, bias=True, residual=False, save=True, workspace=None,
                 x_pad=0, r_pad=0, low=118, high=126):
    F = N // 2 if act == "swiglu" else N
    codes, scales = weights(rng, (N, K), low, high)
    x = gpu(rng.standard_normal((M, K + x_pad)), dtype)[:, :K]
    b = gpu(rng.standard_normal(N), dtype) if bias else None
    r = gpu(rng.standard_normal((M, F + r_pad)) * 2, dtype)[:, :F] if residual else None
    got = mx.linear_act(x, gpu(codes), gpu(scales), bias=b, activation=act, residual=r, save=save,
                        workspace=workspace)
    z, mags = ref.product(ref.f64(x), ref.values(codes, scales))
    if bias:
        z, mags = z + ref.f64(b), mags + np.abs(ref.f64(b))
    bz = ref.sum_bound(K, mags)
    y, by = gref.epilogue(z, bz, act, None if r is None else ref.f64(r))
    if save:
        got, got_z = got
        ref.check(got_z, z, bz + ref.rounded(np.abs(z) + bz, dtype), dtype)
    ref.check(got, y, by + ref.rounded(np.abs(y) + by, dtype), dtype)


# Rows and columns reach the streaming kernel (up to 16 rows; one, two and four tiles a
# block), every tiling, and K slices.
SIZES = [(1, 1, 32), (1, 64, 4096), (3, 200, 128), (16, 12304, 64), (17, 96, 2048), (31, 258, 96),
         (33, 130, 160), (70, 264, 4096), (100, 2050, 64), (640, 6656, 64), (2049, 4096, 32)]


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("act", gref.ACTIVATIONS)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear_act(mx, dtype, act, M, N, K):
    if act == "swiglu":
        N += N % 2
    if M * N > 1 << 21 and act in ("gelu", "silu"):
        pytest.skip("the plain form of the other activations covers the size")
    say("linear_act %s %s M=%d N=%d K=%d" % (dtype, act, M, N, K))
    rng = np.random.default_rng([M, N, K])
    check_linear(mx, rng, M, N, K, dtype, act, bias=True, residual=M % 2 == 1, save=True)
    if M * N < 1 << 19:
        check_linear(mx, rng, M, N, K, dtype, act, bias=False, residual=M % 2 == 0, save=False)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("act,M,N,K,low", [("gelu_tanh", 150, 28501, 2048, 118), ("swiglu", 150, 28500, 2048, 100),
                                           ("relu", 187, 6200, 8192, 118)])
def test_linear_act_tiles_of_96_rows(mx, dtype, act, M, N, K, low):
    """Whole tiles and part-filled ones, with scales on both sides of fp16's range, and in K slices."""
    say("linear_act 96 rows %s %s M=%d N=%d K=%d" % (dtype, act, M, N, K))
    check_linear(mx, np.random.default_rng([M, N, K]), M, N, K, dtype, act, residual=act == "relu",
                 low=low)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("act", ["none", "gelu", "swiglu"])
@pytest.mark.parametrize("N,K", [(4096, 4096), (1198, 14336), (16390, 1056), (66000, 256), (3500, 14976)])
def test_linear_act_one_row_of_many_weights(mx, dtype, act, N, K):
    """The kernel along the rows: one to eight waves on a row, ends of rows and of K inside a wave."""
    say("linear_act one row %s %s N=%d K=%d" % (dtype, act, N, K))
    check_linear(mx, np.random.default_rng([N, K]), 1, N, K, dtype, act, residual=act == "none")


@pytest.mark.parametrize("dtype", HALVES)
def test_linear_act_one_row_specials(mx, dtype):
    """Every scale byte, x up to the type's ends, an infinity in the last block."""
    say("linear_act one row specials %s" % dtype)
    rng = np.random.default_rng(12)
    N, K = 8200, 2080
    for low, high in ((90, 120), (118, 150), (0, 3)):       # above 250 products of N(0, 1) pass fp32
        check_linear(mx, rng, 1, N, K, dtype, "none", low=low, high=high)
    codes, scales = weights(rng, (N, K), 60, 70)
    scales[7, 3], scales[8, 64], scales[9, 0] = 253, 254, 255
    top, low = (2.0 ** 15, 2.0 ** -24) if dtype == torch.float16 else (2.0 ** 127, 2.0 ** -133)
    x = rng.standard_normal((1, K))
    x[0, ::5], x[0, 1::7] = top, low
    x = gpu(x, dtype)
    y = mx.linear_act(x, gpu(codes), gpu(scales))
    w = ref.values(codes, scales)
    z, mags = ref.product(ref.f64(x), w)
    # weights of 2^126 and more meet 2^127 here: the sum's parts pass fp32, their sign is the sum's or not
    far = (scales >= 253).any(axis=1)
    ref.check(y[:, ~far], z[:, ~far], (ref.sum_bound(K, mags) + ref.rounded(np.abs(z), dtype))[:, ~far], dtype)
    assert y[0, 9].isnan()
    x[0, K - 1] = float("inf")
    y = mx.linear_act(x, gpu(codes), gpu(scales))
    assert not y.isfinite().any()
    x = gpu(rng.standard_normal((1, K)) * 2.0 ** -10, dtype)
    scales[9, 0] = 120
    z, mags = ref.product(ref.f64(x), ref.values(codes, scales))
    ref.check(mx.linear_act(x, gpu(codes), gpu(scales)), z,
              ref.sum_bound(K, mags) + ref.rounded(np.abs(z), dtype), dtype)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M", [5, 50])
def test_linear_act_strides_and_alignment(mx, dtype, M):
    """Rows of X and of the residual further apart, outputs off 16 bytes."""
    say("linear_act strides %s M=%d" % (dtype, M))
    rng = np.random.default_rng(M)
    for pad, r_pad in ((8, 0), (64, 8), (0, 3)):
        check_linear(mx, rng, M, 256, 128, dtype, "gelu_tanh", residual=True, x_pad=pad,
                     r_pad=r_pad)
    N, K = 96, 64
    codes, scales = weights(rng, (N, K))
    x, b = gpu(rng.standard_normal((M, K)), dtype), gpu(rng.standard_normal(N + 1), dtype)[1:]
    aligned = mx.linear_act(x, gpu(codes), gpu(scales), bias=b.clone(), activation="silu", save=True)
    room = torch.full((2, M * N + 2), 7.0, dtype=dtype, device="cuda")
    y, z = room[0, 1:-1].view(M, N), room[1, 1:-1].view(M, N)
    out = mx.linear_act(x, gpu(codes), gpu(scales), bias=b, activation="silu", Y=y, Z=z)
    assert out[0] is y and out[1] is z
    assert torch.equal(y, aligned[0]) and torch.equal(z, aligned[1])
    assert (room[:, 0] == 7).all() and (room[:, -1] == 7).all()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear_act_slices_and_workspaces(mx, dtype, act):
    """K slices through the caller's workspace, dirty and larger than asked for, and none."""
    M, N, K = 40, 256, 4096
    say("linear_act slices %s %s" % (dtype, act))
    need = mx.library().mxfp4_linear_act_workspace_bytes(M, N, K)
    assert need > 0
    ws = torch.full((need + 48,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        check_linear(mx, np.random.default_rng(5), M, N, K, dtype, act, residual=True, workspace=ws)
    codes, scales = weights(np.random.default_rng(6), (N, K))
    x = gpu(np.random.default_rng(7).standard_normal((M, K)), dtype)
    y = torch.empty((M, N // 2 if act == "swiglu" else N), dtype=dtype, device="cuda")
    c, s = gpu(codes), gpu(scales)
    lib = mx.library()
    status = lib.mxfp4_linear_act(x.data_ptr(), 0 if dtype == torch.float16 else 1, M, K,
                                  c.data_ptr(), s.data_ptr(), N, K, None,
                                  5 if act == "swiglu" else 0, None, 0, y.data_ptr(), None, None, 0,
                                  torch.cuda.current_stream().cuda_stream)
    assert status == 0
    z, mags = ref.product(ref.f64(x), ref.values(codes, scales))
    want, by = gref.epilogue(z, ref.sum_bound(K, mags), act)
    ref.check(y, want, by + ref.rounded(np.abs(want) + by, dtype), dtype)


def test_linear_act_without_anything_is_linear(mx):
    """Bit for bit where both sum in the same order (no other split of K)."""
    for M in (2, 16, 24):
        rng = np.random.default_rng(M)
        codes, scales = (gpu(t) for t in weights(rng, (512, 1024)))
        x = gpu(rng.standard_normal((M, 1024)), torch.bfloat16)
        assert torch.equal(mx.linear_act(x, codes, scales), mx.linear(x, codes, scales))


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M", [2, 40])
def test_linear_act_specials(mx, dtype, M):
    """K = 0 leaves the bias; NaN and infinities in x, bias and residual stay in their rows and
    columns; scales outside fp16's range."""
    say("linear_act specials %s M=%d" % (dtype, M))
    rng = np.random.default_rng(M)
    N, K = 72, 64
    empty = torch.empty((N, 0), dtype=torch.uint8, device="cuda")
    b = gpu(rng.standard_normal(N), dtype)
    y, z = mx.linear_act(torch.empty((M, 0), dtype=dtype, device="cuda"), empty, empty, bias=b,
                         activation="relu", save=True)
    assert torch.equal(z, b.expand(M, N)) and torch.equal(y, b.clamp(min=0).expand(M, N))
    codes, scales = weights(rng, (N, K))
    x, r = gpu(rng.standard_normal((M, K)), dtype), gpu(rng.standard_normal((M, N)), dtype)
    clean = mx.linear_act(x, gpu(codes), gpu(scales), bias=b, activation="gelu", residual=r)
    b[5], b[6], r[1, 9], r[1, 10] = float("nan"), float("inf"), float("inf"), float("nan")
    x[0, 3] = float("nan")
    y = mx.linear_act(x, gpu(codes), gpu(scales), bias=b, activation="gelu", residual=r)
    assert y[0].isnan().all() and y[1:, 5].isnan().all() and (y[1:, 6] == float("inf")).all()
    assert y[1, 9] == float("inf") and y[1, 10].isnan()
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[0], keep[:, 5:7], keep[1, 9:11] = False, False, False
    assert torch.equal(y[keep], clean[keep])
    for low, high in ((90, 120), (118, 150), (0, 60)):
        check_linear(mx, rng, M, N, 128, dtype, "none", low=low, high=high)


# -------------------------------------------------------------------- experts

RAGGED = {"even": [0, 20, 40, 60, 80], "empty": [0, 0, 7, 7, 80], "one": [3, 4, 5, 6, 7],
          "short": [2, 30, 31, 60, 71], "none": [80, 80, 80, 80, 80], "falling": [5, 3, 40, -1, 60]}


def ranges(offsets, R):
    """Rows of each expert: an offset counts as at least 0 and those before it, at most R."""
    top, out = 0, []
    for o in offsets:
        top = max(top, min(max(o, 0), R))
        out.append(top)
    return list(zip(out, out[1:]))


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("name", list(RAGGED))
@pytest.mark.parametrize("act,N,K", [("none", 40, 96), ("relu", 129, 64), ("gelu", 96, 128),
                                     ("swiglu", 66, 160), ("swiglu", 512, 64)])
def test_grouped_linear_act(mx, dtype, name, act, N, K):
    say("grouped_linear_act %s %s %s N=%d K=%d" % (dtype, name, act, N, K))
    for scale in (1, 12):                                   # 80 and 960 rows: three tilings
        offsets = [o * scale for o in RAGGED[name]]
        E, R, T = 4, 80 * scale, 50
        rng = np.random.default_rng([N, K, scale])
        codes, scales = weights(rng, (E, N, K))
        x, b = gpu(rng.standard_normal((T, K)), dtype), gpu(rng.standard_normal((E, N)), dtype)
        tokens = rng.integers(-1, T + 1, R).astype(np.int32)       # -1 and T: rows of zeros
        c, s, o, t = gpu(codes), gpu(scales), gpu(np.array(offsets, dtype=np.int32)), gpu(tokens)
        y, zs = mx.grouped_linear_act(x, c, s, o, tokens=t, bias=b, activation=act, save=True)
        y32 = mx.grouped_linear_act(x, c, s, o, tokens=t, bias=b, activation=act,
                                    dtype=torch.float32)
        assert y32.dtype == torch.float32
        z, bz = np.zeros((R, N)), np.zeros((R, N))
        rows = ref.f64(x)[np.clip(tokens, 0, T - 1)] * ((tokens >= 0) & (tokens < T))[:, None]
        for e, (lo, hi) in enumerate(ranges(offsets, R)):
            p, mags = ref.product(rows[lo:hi], ref.values(codes[e], scales[e]))
            z[lo:hi] = p + ref.f64(b)[e]
            bz[lo:hi] = ref.sum_bound(K, mags + np.abs(ref.f64(b)[e]))
        want, by = gref.epilogue(z, bz, act)
        ref.check(zs, z, bz + ref.rounded(np.abs(z) + bz, dtype), dtype)
        ref.check(y, want, by + ref.rounded(np.abs(want) + by, dtype), dtype)
        ref.check(y32, want, by + ref.rounded(np.abs(want) + by, torch.float32), torch.float32)


@pytest.mark.parametrize("per", [0, 3, 40, 250])
def test_grouped_linear_act_without_bias_is_grouped_linear(mx, per):
    E, N, K = 6, 128, 256
    R = max(2, per * E)
    rng = np.random.default_rng(per)
    codes, scales = (gpu(t) for t in weights(rng, (E, N, K)))
    x = gpu(rng.standard_normal((R, K)), torch.bfloat16)
    offsets = gpu(np.sort(rng.integers(0, R + 1, E + 1)).astype(np.int32))
    assert torch.equal(mx.grouped_linear_act(x, codes, scales, offsets),
                       mx.grouped_linear(x, codes, scales, offsets))


# ------------------------------------------------------------- activation_grad

def check_activation_grad(mx, dy, z, act, offsets=None, **more):
    dtype = dy.dtype
    got, dbias = mx.activation_grad(dy, z, act, offsets=offsets, **more)
    dz, own = gref.activation_grad(ref.f64(dy), ref.f64(z), act)
    ref.check(got, dz, own + ref.rounded(np.abs(dz) + own, dtype), dtype)
    R = len(dz)
    groups = [(0, R)] if offsets is None else ranges(offsets.tolist(), R)
    for e, (lo, hi) in enumerate(groups):
        part = dbias if offsets is None else dbias[e]
        with np.errstate(all="ignore"):
            want = dz[lo:hi].sum(axis=0)
            bound = own[lo:hi].sum(axis=0) + (hi - lo + 8) * 2.0 ** -24 * np.abs(dz[lo:hi]).sum(axis=0)
        ref.check(part, want, bound + ref.TINY[torch.float32], torch.float32)
    alone = mx.activation_grad(dy, z, act, bias=False)
    assert torch.equal(alone.nan_to_num(7), got.nan_to_num(7))
    return got, dbias


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("act", gref.ACTIVATIONS)
@pytest.mark.parametrize("M,N", [(0, 8), (1, 2), (1, 4096), (6, 1000), (64, 514), (65, 66), (700, 130)])
def test_activation_grad(mx, dtype, act, M, N):
    say("activation_grad %s %s M=%d N=%d" % (dtype, act, M, N))
    rng = np.random.default_rng([M, N])
    F = N // 2 if act == "swiglu" else N
    check_activation_grad(mx, gpu(rng.standard_normal((M, F)), dtype),
                          gpu(rng.standard_normal((M, N)) * 3, dtype), act)


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("act", gref.ACTIVATIONS)
def test_activation_grad_far_values(mx, dtype, act):
    """Every magnitude of the type, both signs, zeros and infinities: slopes stay between -0.2
    and 1.2, so that dZ is finite wherever dY (times the up value) is."""
    say("activation_grad far %s %s" % (dtype, act))
    top = 15 if dtype == torch.float16 else 126
    z = np.ldexp(1.0, np.arange(-top + 1, top + 1))
    z = np.concatenate([z, 1.37 * z[:-1], np.linspace(-20, 20, 401), [0.0, np.inf]])
    z = np.concatenate([z, -z])
    if act == "swiglu":
        finite = np.isfinite(z)
        rows = np.concatenate([z[finite], np.full(finite.sum(), 0.75)])[None]
        zs, dy = gpu(rows, dtype), gpu(np.full((1, finite.sum()), -0.5), dtype)
        check_activation_grad(mx, dy, zs, act)
        return
    zs, dy = gpu(z[None], dtype), gpu(np.full((1, z.size), -0.5), dtype)
    got, _ = check_activation_grad(mx, dy, zs, act)
    assert got.isfinite().all()


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("name", list(RAGGED))
@pytest.mark.parametrize("act,N", [("gelu", 72), ("swiglu", 130), ("swiglu", 1040)])
def test_activation_grad_by_expert(mx, dtype, name, act, N):
    say("activation_grad by expert %s %s %s N=%d" % (dtype, name, act, N))
    for scale in (1, 9):
        rng = np.random.default_rng([N, scale])
        R, F = 80 * scale, N // 2 if act == "swiglu" else N
        offsets = gpu((np.array(RAGGED[name]) * scale).astype(np.int32))
        check_activation_grad(mx, gpu(rng.standard_normal((R, F)), dtype),
                              gpu(rng.standard_normal((R, N)), dtype), act, offsets=offsets)


def test_activation_grad_many_experts_and_no_rows(mx):
    rng = np.random.default_rng(3)
    E, R = 1024, 500
    offsets = gpu(np.sort(rng.integers(0, R + 1, E + 1)).astype(np.int32))
    check_activation_grad(mx, gpu(rng.standard_normal((R, 24)), torch.bfloat16),
                          gpu(rng.standard_normal((R, 24)), torch.bfloat16), "silu",
                          offsets=offsets)
    empty = torch.empty((0, 24), dtype=torch.bfloat16, device="cuda")
    dz, dbias = mx.activation_grad(empty, empty, "silu", offsets=offsets)
    assert dz.shape == (0, 24) and dbias.shape == (E, 24) and (dbias == 0).all()


@pytest.mark.parametrize("dtype", HALVES)
def test_activation_grad_strides_workspace_and_repeats(mx, dtype):
    rng = np.random.default_rng(11)
    for pad in (8, 3):
        dy = gpu(rng.standard_normal((200, 64 + pad)), dtype)[:, :64]
        z = gpu(rng.standard_normal((200, 128 + pad)), dtype)[:, pad:]
        ws = torch.full((mx.library().mxfp4_activation_grad_workspace_bytes(200, 128, 0) + 12,), 255,
                        dtype=torch.uint8, device="cuda")
        first = check_activation_grad(mx, dy, z, "swiglu", workspace=ws)
        again = mx.activation_grad(dy, z, "swiglu")
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
