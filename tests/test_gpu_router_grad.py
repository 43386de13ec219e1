"""The balance loss and the router's gradient on the GPU over more tokens than the launches have
lane groups, with masks of the type's lowest value under bounds that reject mistakes, and with
logits that are not finite (forms and bounds in mxfp4_router_reference)."""
import numpy as np
import pytest

import mxfp4_reference as ref
import mxfp4_router_reference as rref
from test_gpu_linear_act import gpu, mx, say  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

FLOATS = [torch.float16, torch.bfloat16, torch.float32]


def check_balance(mx, x, ids):  # noqa: F811
    loss, counts = mx.balance(x, ids)
    want, bound, n = rref.balance(ref.f64(x), ids.cpu().numpy())
    assert np.array_equal(counts.cpu().numpy(), n)
    assert abs(float(loss) - want) <= bound + 2.0 ** -24 * abs(want), (float(loss), want, bound)
    return counts


def check_route_grad(mx, x, ids, dw, renormalize, counts, dloss):  # noqa: F811
    got = mx.route_grad(x, ids, dw, renormalize=renormalize, counts=counts, dloss=dloss)
    want, bound = rref.route_grad(ref.f64(x), ids.cpu().numpy(), None if dw is None else ref.f64(dw),
                                  renormalize, None if counts is None else counts.cpu().numpy(),
                                  0.0 if dloss is None else float(dloss))
    with np.errstate(all="ignore"):
        ref.check(got, want, bound + ref.rounded(np.abs(want) + bound, x.dtype), x.dtype)
    return got


def many(rng, T, E, k, dtype):
    """Masked logits, every fifth row of -infinities, the k largest (ties to the lowest); in the
    second half every seventh token names its first expert twice."""
    x = gpu(rng.standard_normal((T, E)) * 2, torch.float32).to(dtype)
    x[gpu(rng.random((T, E)) < 0.3)] = float("-inf")
    x[3::5] = float("-inf")
    top, ids = torch.sort(x.float(), dim=1, descending=True, stable=True)
    ids = torch.where(top == float("-inf"), -1, ids)[:, :k].to(torch.int32).contiguous()
    ids[T // 2::7, 1] = ids[T // 2::7, 0]
    return x, ids


# A launch of the gradient has 1024 blocks of 256 threads, of the loss 256 blocks of 512; a token
# takes 8 lanes up to 64 experts, 16 up to 128, 32 up to 256, then 64: these walk three tokens or
# more a lane group, the last round part-filled inside a wave.
LONG = [(70001, 60, 4), (33001, 128, 8), (17003, 200, 3), (9001, 300, 5), (9001, 600, 3)]


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("T,E,k", LONG)
def test_several_tokens_a_lane_group(mx, dtype, T, E, k):  # noqa: F811
    say("router, many tokens %s T=%d E=%d k=%d" % (dtype, T, E, k))
    rng = np.random.default_rng([T, E, k])
    x, ids = many(rng, T, E, k, dtype)
    dw = gpu(rng.standard_normal((T, k)), torch.float32)
    dloss = torch.full((), -3.5 * T, device="cuda")
    counts = check_balance(mx, x, ids)
    for renormalize in (True, False):
        both = check_route_grad(mx, x, ids, dw, renormalize, counts, dloss)
        check_route_grad(mx, x, ids, dw, renormalize, None, None)
        assert (both[x == float("-inf")] == 0).all()
        # a token's gradient does not depend on which lane group takes it, or when
        for lo, hi in ((T - 1000, T), (T // 2 - 3, T // 2 + 500)):
            part = mx.route_grad(x[lo:hi], ids[lo:hi], dw[lo:hi], renormalize=renormalize, counts=counts,
                                 dloss=dloss)
            assert torch.equal(part, both[lo:hi])
    check_route_grad(mx, x, ids, None, True, counts, dloss)


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("E", [7, 100, 200, 300, 600])
@pytest.mark.parametrize("renormalize", [True, False])
def test_lowest_values_as_masks(mx, dtype, E, renormalize):  # noqa: F811
    say("router, lowest values %s E=%d %s" % (dtype, E, renormalize))
    rng = np.random.default_rng(E)
    info = torch.finfo(dtype)
    x = gpu(rref.far_rows(rng, E, info.min, info.max)).to(dtype)
    ids, _ = mx.route(x, 3)
    dw = gpu(rng.standard_normal((12, 3)), torch.float32)
    counts = check_balance(mx, x, ids)
    assert int(counts[E]) == 12
    one = torch.full((), 30.0, device="cuda")
    check_route_grad(mx, x, ids, dw, renormalize, counts, one)
    check_route_grad(mx, x, ids, dw, renormalize, None, None)
    check_route_grad(mx, x, ids, None, renormalize, counts, one)


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("E", [20, 100, 300])
def test_logits_that_are_not_finite(mx, dtype, bad, E):  # noqa: F811
    """With renormalized weights alone the chosen logits are all that counts: one that is not finite
    makes the chosen experts' gradients NaN, one that is not chosen changes nothing.  Without
    renormalize, and with the loss, every gradient of the row is NaN."""
    rng = np.random.default_rng(E)
    x = gpu(rng.standard_normal((12, E)), torch.float32).to(dtype)
    x[:, 7] = float("-inf")
    ids, _ = mx.route(x, 3)
    dw = gpu(rng.standard_normal((12, 3)), torch.float32)
    counts, one = mx.balance(x, ids)[1], torch.ones((), device="cuda")
    clean = {r: mx.route_grad(x, ids, dw, renormalize=r) for r in (True, False)}
    loss = mx.route_grad(x, ids, counts=counts, dloss=one)
    y = x.clone()
    chosen = ids[2].tolist()
    free = next(e for e in range(E) if e not in ids[5].tolist() and e != 7)
    y[2, chosen[1]], y[5, free] = bad, bad
    got = mx.route_grad(y, ids, dw)
    assert got[2, chosen].isnan().all() and int(got[2].isnan().sum()) == 3 and (got[2].nan_to_num(0) == 0).all()
    keep = [r for r in range(12) if r != 2]
    assert torch.equal(got[keep], clean[True][keep])
    rest = [r for r in range(12) if r not in (2, 5)]
    for other, want in ((mx.route_grad(y, ids, dw, renormalize=False), clean[False]),
                        (mx.route_grad(y, ids, counts=counts, dloss=one), loss)):
        assert other[2].isnan().all() and other[5].isnan().all()
        assert torch.equal(other[rest], want[rest])
    check_route_grad(mx, y, ids, dw, True, None, None)
    n = check_counts(mx, y, ids)
    assert n == 12


def check_counts(mx, y, ids):  # noqa: F811
    loss, counts = mx.balance(y, ids)
    assert loss.isnan()
    only = torch.full((1, y.shape[1]), float("-inf"), dtype=y.dtype, device="cuda")
    only[0, 1] = float("nan")                               # a NaN counts as a usable expert
    loss, one = mx.balance(only, torch.full((1, 1), 1, dtype=torch.int32, device="cuda"))
    assert loss.isnan() and int(one[-1]) == 1
    return int(counts[-1])
