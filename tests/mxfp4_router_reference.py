"""Plain 64-bit forms of the balance loss and of the router's gradient over many tokens at once
(numpy, whole rows), and error bounds that stay useful where logits lie far apart.

A probability's relative error: the difference d to the row's peak is rounded once, which moves
exp(-d) by d 2^-24, its own error is a few units, then a sum of E terms and a reciprocal.  Below
exp(-104) < 2^-150 nothing is left in fp32, so d counts up to 104.  An exponential below fp32's
normal range, 2^-126, may count as 0: that is an absolute error of FLUSHED for a probability.
"""
import numpy as np

from mxfp4_grad_reference import softmax

FLUSHED = 2.0 ** -126
FARTHEST = 104.0


def share_error(x, extra):
    """Relative error of the probabilities of each row [T, 1]; `extra` roundings come with them."""
    with np.errstate(all="ignore"):
        d = np.abs(x - x.max(axis=1, keepdims=True))
        d = np.where(np.isfinite(x), np.minimum(d, FARTHEST), 0)
    d = np.where(np.isnan(d), 0, d).max(axis=1, keepdims=True)
    return (x.shape[1] + extra + 32 + 4 * d) * 2.0 ** -24


def balance(x, ids):
    """(loss, its bound, counts [E + 1]).  All terms are positive, so that the probabilities' errors
    enter as they are.  Sums: a lane group's tokens (T / 2048 of them at the most, or two), the
    groups of a wave, 8 waves, 256 blocks, then wave and block of the last sum and a few products."""
    T, E = x.shape
    counts = np.zeros(E + 1, dtype=np.int64)
    counts[:E] = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
    counts[E] = (~(x == -np.inf)).any(axis=1).sum()
    chosen, tokens = counts[:E].sum(), counts[E]
    if chosen == 0 or tokens == 0:
        return 0.0, 0.0, counts
    c, scale = counts[:E].astype(np.float64), E / (float(chosen) * tokens)
    rows = (softmax(x) * c).sum(axis=1)
    loss = scale * rows.sum()
    bound = scale * (rows * share_error(x, 0)[:, 0]).sum() + loss * (T / 2048 + 300) * 2.0 ** -24
    return loss, bound + scale * T * c.sum() * FLUSHED, counts


def route_grad(x, ids, dw, renormalize, counts, dloss):
    """(dlogits, bound before the rounding), [T, E] each.  dw or counts None: no such part."""
    T, E = x.shape
    k = ids.shape[1]
    p = softmax(x)
    grad, mags, tiny = np.zeros((T, E)), np.zeros((T, E)), 0.0
    with np.errstate(all="ignore"):
        if counts is not None:
            c = counts[:E].astype(np.float64)
            scale = dloss * E / (max(c.sum(), 1) * max(float(counts[E]), 1))
            mean = (p * c).sum(axis=1, keepdims=True)
            grad += scale * p * (c - mean)
            mags += np.abs(scale) * p * (c + mean)
            tiny += (np.abs(scale) * (E + 1) + 1) * c.max() * FLUSHED
        if dw is not None:
            used = (ids >= 0) & (ids < E)
            slot = np.where(used, ids, 0)
            l = np.take_along_axis(x, slot, 1)
            used &= ~(l == -np.inf)
            w = np.take_along_axis(p, slot, 1)
            if renormalize:
                l = np.where(used, l, -np.inf)
                w = softmax(l)
            w = np.where(used, w, 0)
            d = np.where(used, dw, 0)
            mean, size = (w * d).sum(axis=1, keepdims=True), (w * np.abs(d)).sum(axis=1, keepdims=True)
            rows = np.broadcast_to(np.arange(T)[:, None], ids.shape)
            if renormalize:
                part, part_size = w * (d - mean), w * (np.abs(d) + size)
            else:
                part, part_size = w * d, w * np.abs(d)
                grad -= p * mean
                mags += p * size
            np.add.at(grad, (rows[used], slot[used]), part[used])
            np.add.at(mags, (rows[used], slot[used]), part_size[used])
            tiny += 2 * (E + k + 2) * np.abs(d[np.isfinite(d)]).max(initial=0) * FLUSHED
    # twice: each term holds two probabilities (or weights), its own and the mean's
    return grad, 2 * share_error(x, k) * mags + tiny


def far_rows(rng, E, low, high):
    """12 rows of E logits: the type's lowest value as a mask of all, all but one and every other
    expert, beside -infinity, of three experts; a quarter of the largest value; -150 beside 0."""
    x = rng.standard_normal((12, E))
    x[0], x[1, 1:], x[2, ::2] = low, low, low
    x[3], x[3, 4] = -np.inf, low
    x[4, :3], x[5, 3:] = low, high / 4
    x[6], x[6, 1] = 0.0, -150.0
    return x
