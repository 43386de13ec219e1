"""The balance loss, the router's gradient and the weighted sum's gradient on the GPU against
plain 64-bit forms (bounds derived in mxfp4_grad_reference)."""
import numpy as np
import pytest

import mxfp4_grad_reference as gref
import mxfp4_reference as ref
from test_gpu_linear_act import HALVES, gpu, mx, say  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

FLOATS = [torch.float16, torch.bfloat16, torch.float32]


def routing(rng, T, E, k, dtype, masked):
    x = gpu(rng.standard_normal((T, E)) * 2, dtype)
    if masked:
        x[gpu(rng.random((T, E)) < 0.3)] = float("-inf")
        x[3::5] = float("-inf")
    ids, _ = ref.route(ref.f64(x), k, True)
    return x, gpu(ids.astype(np.int32))


SIZES = [(1, 1, 1), (2, 3, 2), (5, 64, 6), (33, 65, 8), (70, 128, 32), (300, 200, 4), (9, 1024, 9),
         (4099, 60, 4)]


def check_balance(mx, x, ids):  # noqa: F811
    """The softmax's errors enter the loss as they are (all terms are positive); tokens are added
    in runs of T / 2048, then 4 waves, 512 blocks and a tree of 10 levels."""
    loss, counts = mx.balance(x, ids)
    xs = ref.f64(x)
    want, want_counts = gref.balance(xs, ids.cpu().numpy())
    assert np.array_equal(counts.cpu().numpy(), want_counts)
    rel = gref.softmax_error(xs, 0).max(initial=0) + (len(xs) / 2048 + 540) * 2.0 ** -24
    assert abs(float(loss) - want) <= rel * abs(want), (float(loss), want)
    return counts


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("masked", [False, True])
def test_balance(mx, dtype, T, E, k, masked):  # noqa: F811
    say("balance %s T=%d E=%d k=%d masked=%s" % (dtype, T, E, k, masked))
    x, ids = routing(np.random.default_rng([T, E, k]), T, E, k, dtype, masked)
    check_balance(mx, x, ids)


def test_balance_of_a_balanced_routing_is_one_and_of_none_zero(mx):  # noqa: F811
    E = 16
    x = torch.zeros((E, E), device="cuda")
    ids = torch.arange(E, dtype=torch.int32, device="cuda")[:, None]
    loss, counts = mx.balance(x, ids)
    assert float(loss) == 1.0 and counts.tolist() == [1] * E + [E]
    loss, counts = mx.balance(x, torch.full_like(ids, -1))
    assert float(loss) == 0.0 and counts.tolist() == [0] * E + [E]
    loss, counts = mx.balance(torch.full_like(x, float("-inf")), ids)
    assert float(loss) == 0.0 and counts.tolist() == [1] * E + [0]
    loss, counts = mx.balance(x[:0], ids[:0])
    assert float(loss) == 0.0 and counts.tolist() == [0] * (E + 1)


def test_balance_counts_any_ids(mx):  # noqa: F811
    """Ids out of range are no choice, one that a token repeats counts as often; strided
    logits; not finite logits."""
    rng = np.random.default_rng(2)
    wide = gpu(rng.standard_normal((40, 90)), torch.bfloat16)
    ids = gpu(rng.integers(-5, 80, (40, 7)).astype(np.int32))
    ids[:, 1] = ids[:, 0]
    check_balance(mx, wide[:, 5:75], ids)
    for bad in (float("nan"), float("inf")):
        x = wide[:, :70].clone()
        x[7, 3] = bad
        loss, counts = mx.balance(x, ids)
        assert torch.isnan(loss) and int(counts[70]) == 40


# -------------------------------------------------------------- router's gradient

def check_route_grad(mx, x, ids, dw, renormalize, counts, dloss):  # noqa: F811
    got = mx.route_grad(x, ids, dw, renormalize=renormalize, counts=counts, dloss=dloss)
    assert got.dtype == x.dtype and got.is_contiguous()
    xs = ref.f64(x)
    want, mags = gref.route_grad(xs, ids.cpu().numpy(), None if dw is None else ref.f64(dw),
                                 renormalize, None if counts is None else counts.cpu().numpy(),
                                 0.0 if dloss is None else float(dloss))
    rel = 2 * gref.softmax_error(xs, ids.shape[1]).max(axis=1, keepdims=True)
    with np.errstate(all="ignore"):
        own = rel * mags
    ref.check(got, want, own + ref.rounded(np.abs(want) + own, x.dtype), x.dtype)
    return got


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_grad(mx, dtype, T, E, k, renormalize):  # noqa: F811
    say("route_grad %s T=%d E=%d k=%d %s" % (dtype, T, E, k, renormalize))
    rng = np.random.default_rng([T, E, k])
    x, ids = routing(rng, T, E, k, dtype, masked=T % 2 == 1)
    dw = gpu(rng.standard_normal((T, k)), torch.float32)
    dloss = torch.full((), -3.5 * T, device="cuda")         # both parts count
    _, counts = mx.balance(x, ids)
    both = check_route_grad(mx, x, ids, dw, renormalize, counts, dloss)
    check_route_grad(mx, x, ids, dw, renormalize, None, None)
    check_route_grad(mx, x, ids, None, renormalize, counts, dloss)
    assert (both[x == float("-inf")] == 0).all()
    assert torch.equal(both, mx.route_grad(x, ids, dw, renormalize=renormalize, counts=counts,
                                           dloss=dloss))
    if T > 1:                                               # a slice with the whole batch's counts
        part = mx.route_grad(x[1:], ids[1:], dw[1:], renormalize=renormalize, counts=counts,
                             dloss=dloss)
        assert torch.equal(part, both[1:])


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_grad_any_ids_and_strides(mx, dtype, renormalize):  # noqa: F811
    """Ids out of range and of experts at -infinity have no gradient, a repeated id the sum of its
    slots'; rows of logits further apart."""
    rng = np.random.default_rng(8)
    T, E, k = 60, 40, 9
    wide = gpu(rng.standard_normal((T, E + 7)), dtype)
    x = wide[:, 3:3 + E]
    x[:, 5] = float("-inf")
    x[10] = float("-inf")
    ids = gpu(rng.integers(-3, E + 3, (T, k)).astype(np.int32))
    ids[:, 2], ids[:, 3] = 5, ids[:, 4]
    ids[11] = -1
    ids[12] = 5
    got = check_route_grad(mx, x, ids, gpu(rng.standard_normal((T, k)), torch.float32), renormalize,
                           None, None)
    assert (got[10:13] == 0).all()


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("E", [7, 100, 300, 600])
@pytest.mark.parametrize("renormalize", [True, False])
def test_masks_of_the_lowest_value(mx, dtype, E, renormalize):  # noqa: F811
    """The type's lowest value as a mask: an expert like another (a row of it is uniform), as small
    as it is; beside -infinity; and logits far apart."""
    rng = np.random.default_rng(E)
    low = torch.finfo(dtype).min
    x = gpu(rng.standard_normal((12, E)), dtype)
    x[0], x[1, 1:], x[2, ::2] = low, low, low
    x[3], x[3, 4] = float("-inf"), low
    x[4, :3], x[5, 3:] = low, torch.finfo(dtype).max / 4
    x[6], x[6, 1] = 0.0, -150.0
    ids, _ = mx.route(x, 3)
    counts = check_balance(mx, x, ids)
    assert int(counts[E]) == 12
    check_route_grad(mx, x, ids, gpu(rng.standard_normal((12, 3)), torch.float32), renormalize, counts,
                     torch.full((), 30.0, device="cuda"))


def test_route_grad_not_finite_rows_stay_rows(mx):  # noqa: F811
    rng = np.random.default_rng(1)
    x = gpu(rng.standard_normal((12, 20)), torch.float32)
    ids, _ = mx.route(x, 3)
    dw, counts = gpu(rng.standard_normal((12, 3)), torch.float32), mx.balance(x, ids)[1]
    one = torch.ones((), device="cuda")
    clean = mx.route_grad(x, ids, dw, counts=counts, dloss=one)
    x[2, 4], x[5, int(ids[5, 0])] = float("nan"), float("inf")
    dw[9, 0] = float("nan")
    got = mx.route_grad(x, ids, dw, counts=counts, dloss=one)
    assert got[2].isnan().all() and got[5].isnan().any() and got[9].isnan().any()
    rest = [r for r in range(12) if r not in (2, 5, 9)]
    assert torch.equal(got[rest], clean[rest])


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_grad_is_the_difference_of_route_and_balance(mx, renormalize):  # noqa: F811
    """Central differences in 64 bits of what route() and balance() compute, at fixed choices."""
    rng = np.random.default_rng(6)
    T, E, k = 7, 10, 3
    x = rng.standard_normal((T, E))
    ids, _ = ref.route(x, k, True)
    dw, dloss = rng.standard_normal((T, k)), 2.5

    def total(v):
        p = gref.softmax(v)
        w = np.take_along_axis(p, ids, 1)
        if renormalize:
            w = w / w.sum(axis=1, keepdims=True)
        return (w * dw).sum() + dloss * gref.balance(v, ids)[0]
    step = 2.0 ** -14
    diff = np.zeros((T, E))
    for t in range(T):
        for e in range(E):
            d = np.zeros((T, E))
            d[t, e] = step
            diff[t, e] = (total(x + d) - total(x - d)) / (2 * step)
    logits, ids_gpu = gpu(x, torch.float32), gpu(ids.astype(np.int32))
    counts = mx.balance(logits, ids_gpu)[1]
    got = mx.route_grad(logits, ids_gpu, gpu(dw, torch.float32), renormalize=renormalize,
                        counts=counts, dloss=torch.full((), dloss, device="cuda"))
    # third derivatives of sums of a few terms below 8: the difference is off by 8 step^2
    assert np.abs(ref.f64(got) - diff).max() <= 8 * step ** 2 + 64 * 2.0 ** -24 * 8


# ------------------------------------------------------- the weighted sum's gradient

def check_combine_grad(mx, dout, y, tokens, positions, w):  # noqa: F811
    dtype = dout.dtype
    dy, dw = mx.combine_grad(dout, y, tokens, positions, w)
    assert dy.dtype == dtype and dw.dtype == torch.float32
    want, want_w, mags = gref.combine_grad(ref.f64(dout), ref.f64(y), tokens.cpu().numpy(),
                                           positions.cpu().numpy(), ref.f64(w))
    # the weights of one row are added in fp32, then one product
    k = w.shape[1]
    own = (k + 2) * 2.0 ** -24 * np.abs(want) if k == 1 or _distinct(positions) else \
        (k + 2) * 2.0 ** -24 * np.abs(ref.f64(w)).max(initial=0) * k * np.abs(ref.f64(dout)).max(initial=0)
    ref.check(dy, want, own + ref.rounded(np.abs(want) + own, dtype), dtype)
    ref.check(dw, want_w, ref.sum_bound(dout.shape[1], mags) + ref.rounded(np.abs(want_w), torch.float32),
              torch.float32)
    return dy, dw


def _distinct(positions):
    p = positions.cpu().numpy()
    p = p[p >= 0]
    return len(np.unique(p)) == p.size


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("rows32", [False, True])
@pytest.mark.parametrize("T,E,k,N", [(1, 1, 1, 1), (3, 8, 6, 64), (70, 16, 2, 1001), (9, 40, 32, 4096),
                                     (300, 64, 8, 776), (5, 4, 4, 520)])
def test_combine_grad(mx, dtype, rows32, T, E, k, N):  # noqa: F811
    say("combine_grad %s %s T=%d E=%d k=%d N=%d" % (dtype, rows32, T, E, k, N))
    rng = np.random.default_rng([T, E, k, N])
    logits = gpu(rng.standard_normal((T, E)), torch.float32)
    if T > 3:
        logits[2::7] = float("-inf")                        # padding tokens: rows of no choice
    ids, w = mx.route(logits, k)
    p = mx.plan(ids, E)
    y = gpu(rng.standard_normal((T * k, N)), torch.float32 if rows32 else dtype)
    y[int(p.offsets[-1]):] = float("nan")                   # not data
    dy, dw = check_combine_grad(mx, gpu(rng.standard_normal((T, N)), dtype), y, p.tokens, p.positions, w)
    assert (dy[int(p.offsets[-1]):] == 0).all() and (dw[p.positions < 0] == 0).all()


@pytest.mark.parametrize("N", [64, 37])
def test_combine_grad_of_any_tensors(mx, N):  # noqa: F811
    """Tokens and positions that are no plan's: every row is written once, nothing else is."""
    rng = np.random.default_rng(N)
    T, k, R = 20, 5, 70
    dout, w = gpu(rng.standard_normal((T, N)), torch.bfloat16), gpu(rng.random((T, k)), torch.float32)
    y = gpu(rng.standard_normal((R, N)), torch.bfloat16)
    tokens = gpu(rng.integers(-2, T + 2, R).astype(np.int32))
    positions = gpu(rng.integers(-2, R + 2, (T, k)).astype(np.int32))
    positions[:, 3] = positions[:, 1]                       # the same row twice
    tokens[positions[4, 1].clamp(0, R - 1).item()] = 4
    check_combine_grad(mx, dout, y, tokens, positions, w)
    room = torch.full((R + 2, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    mx.combine_grad(dout, y, tokens, positions, w, dY=room[1:-1])
    assert room[0].isnan().all() and room[-1].isnan().all() and room[1:-1].isfinite().all()


def test_combine_grad_empty_sizes(mx):  # noqa: F811
    none = torch.empty((0,), dtype=torch.int32, device="cuda")
    dout, w = torch.ones((3, 8), dtype=torch.float16, device="cuda"), torch.ones((3, 2), device="cuda")
    pos = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    dy, dw = mx.combine_grad(dout, dout[:0], none, pos, w)          # no rows
    assert dy.shape == (0, 8) and (dw == 0).all()
    dy, dw = mx.combine_grad(dout[:0], dout, pos[:, 0].contiguous(), pos[:0], w[:0])   # no tokens
    assert (dy == 0).all() and dw.shape == (0, 2)
    dy, dw = mx.combine_grad(dout[:, :0].contiguous(), dout[:, :0].contiguous(), pos[:, 0].contiguous(),
                             pos, w)                                  # no columns
    assert dy.shape == (3, 0) and (dw == 0).all()
