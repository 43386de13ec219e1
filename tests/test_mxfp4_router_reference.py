"""The whole-row reference of the router's operators against the row-by-row one, and what its
bounds reject: planted mistakes in rows whose mask is the type's lowest value."""
import numpy as np
import pytest
import torch

import mxfp4_grad_reference as gref
import mxfp4_reference as ref
import mxfp4_router_reference as rref

FLOATS = [torch.float16, torch.bfloat16, torch.float32]


@pytest.mark.parametrize("renormalize", [True, False])
def test_whole_rows_are_row_by_row(renormalize):
    rng = np.random.default_rng(1)
    T, E, k = 40, 11, 5
    x = rng.standard_normal((T, E)) * 3
    x[rng.random((T, E)) < 0.3] = -np.inf
    x[7], x[9, 2], x[11, 3] = -np.inf, np.nan, np.inf
    ids, dw = rng.integers(-2, E + 2, (T, k)), rng.standard_normal((T, k))
    ids[:, 1] = ids[:, 0]
    clean = np.isfinite(np.where(x == -np.inf, 0, x)).all(axis=1)
    want, counts = gref.balance(x[clean], ids[clean])
    loss, bound, n = rref.balance(x[clean], ids[clean])
    assert np.array_equal(n, counts) and abs(loss - want) < 1e-12 and 0 < bound < 1e-4 * loss
    for w, c in ((dw, counts), (dw, None), (None, counts)):
        a, _ = gref.route_grad(x, ids, w, renormalize, c, -1.5)
        b, _ = rref.route_grad(x, ids, w, renormalize, c, -1.5)
        assert np.array_equal(np.isnan(a), np.isnan(b))
        assert np.nanmax(np.abs(a - b)) < 1e-12


@pytest.mark.parametrize("dtype", FLOATS)
@pytest.mark.parametrize("renormalize", [True, False])
def test_bounds_reject_mistakes_in_far_rows(dtype, renormalize):
    """A mask that counts as an ordinary logit, one that counts as -infinity in a row of nothing
    else, the loss of the first, and large logits that count as ordinary ones are outside."""
    rng = np.random.default_rng(7)
    E, info = 7, torch.finfo(dtype)
    x = rref.far_rows(rng, E, info.min, info.max)
    x = ref.f64(torch.from_numpy(x).to(dtype))
    ids, _ = ref.route(x, 3, True)
    dw = rng.standard_normal((12, 3))
    loss, loss_bound, counts = rref.balance(x, ids)
    assert loss_bound < 1e-4 * loss
    want, bound = rref.route_grad(x, ids, dw, renormalize, counts, 30.0)
    bound = bound + ref.rounded(np.abs(want) + bound, dtype)
    low = x == info.min
    for wrong in (np.where(low, 0.0, x), np.where(low & ~low.all(axis=1, keepdims=True), -3.0, x)):
        got, _ = rref.route_grad(wrong, ids, dw, renormalize, counts, 30.0)
        for r in (1, 2, 4):
            assert (np.abs(got[r] - want[r]) > bound[r]).any(), r
        assert abs(rref.balance(wrong, ids)[0] - loss) > loss_bound
    zeroed = np.where(low, -np.inf, x)                       # as if the value were -infinity
    got, _ = rref.route_grad(zeroed, ids, dw, renormalize, counts, 30.0)
    assert (np.abs(got[0] - want[0]) > bound[0]).any()
    wide = np.where(x[5] > 1, 0.5, x[5])                     # row 5's large values are ordinary
    got, _ = rref.route_grad(np.where((np.arange(12) == 5)[:, None], wide, x), ids, dw, renormalize,
                             counts, 30.0)
    assert (np.abs(got[5] - want[5]) > bound[5]).any()
