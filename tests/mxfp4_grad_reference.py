"""Plain 64-bit implementations of the products with an epilogue and of the backward
operators (numpy, elementary operations), and their error bounds.

Conventions of mxfp4_reference: a rounding to t bits is finfo(t).eps / 2 relative, an fp32
sum of n products (n/8 + 64) 2^-24 of the sum of magnitudes.
"""
import math

import numpy as np

import mxfp4_reference as ref

ACTIVATIONS = ("none", "relu", "silu", "gelu", "gelu_tanh", "swiglu")
C = 2 * math.sqrt(2 / math.pi)
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def sigmoid(z):
    with np.errstate(all="ignore"):
        return 1 / (1 + np.exp(-z))


def _cube(z):
    return C * (z + 0.044715 * z ** 3)


def value(z, act):
    """The activation (none of swiglu) in 64 bits."""
    with np.errstate(all="ignore"):
        if act == "none":
            return z
        if act == "relu":
            return np.where(z < 0, 0.0, z)
        if act == "silu":
            return z / (1 + np.exp(-z))
        if act == "gelu":
            return 0.5 * z * _erfc(-z / math.sqrt(2))
        return z / (1 + np.exp(-_cube(z)))


def slope(z, act):
    """Its derivative; beyond 40 (silu 150) the limits 0 and 1, as they are in 64 bits too."""
    with np.errstate(all="ignore"):
        if act == "none":
            return np.ones_like(z)
        if act == "relu":
            return np.where(z <= 0, 0.0, 1.0)
        z = np.where(np.isnan(z), z, z.clip(-150, 150) if act == "silu" else z.clip(-40, 40))
        if act == "silu":
            s = sigmoid(z)
            return s * (1 + z * sigmoid(-z))
        if act == "gelu":
            return 0.5 * _erfc(-z / math.sqrt(2)) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        s, q = sigmoid(_cube(z)), sigmoid(-_cube(z))
        return s + z * s * q * C * (1 + 3 * 0.044715 * z * z)


def act_bound(z, act, y):
    """Error of the activation's own fp32 arithmetic: the argument of an exponential carries
    its relative rounding (2^-23 of it and of what is derived from it) into the result.  A factor
    below fp32's normal range, 2^-126, may count as 0: a sigmoid is that small where |z| > 87.3, and
    |z| times a smaller one falls from there on, 87.4 * 2^-126 < 2^-119 (erfc and the tanh form
    reach it where |z| < 14)."""
    with np.errstate(all="ignore"):
        a = np.abs(z)
        arg = {"none": 0 * a, "relu": 0 * a, "silu": a, "gelu": a * a,
               "gelu_tanh": C * (a + 0.05 * a ** 3)}[act]
        own = (arg + 16) * 2.0 ** -22 * np.abs(y) if act not in ("none", "relu") else 0 * a
        return np.where(np.isfinite(own), own, 0) + 2.0 ** -119


# Largest slopes: silu 1.0999, gelu and its tanh form 1.129.
STEEPEST = {"none": 1.0, "relu": 1.0, "silu": 1.1, "gelu": 1.13, "gelu_tanh": 1.13}


def epilogue(z, bz, act, residual=None):
    """(y, bound before the rounding) of z with bound bz."""
    if act == "swiglu":
        y, by = ref.swiglu(z, bz)
    else:
        y = value(z, act)
        by = STEEPEST[act] * bz + act_bound(z, act, y)
    if residual is not None:
        by = by + 2.0 ** -24 * (np.abs(y) + np.abs(residual))
        y = y + residual
    return y, by


def slope_bound(z, act):
    """Absolute error of a slope in fp32.  silu: 1 - s is off by 2^-24 and meets |z|.  gelu: terms
    of at most 1 each, z^3 phi(z) < 1.  tanh form: 1 - s is off by 2^-24 where |u| < 17 (|z| < 6)
    and meets at most 6 * 1.6 * 6 = 58."""
    a = np.minimum(np.abs(z), 150)
    if act in ("none", "relu"):
        return 0 * a
    return {"silu": a + 8, "gelu": 0 * a + 16, "gelu_tanh": 0 * a + 64}[act] * 2.0 ** -22


def activation_grad(dy, z, act):
    """(dz, bound before the rounding) in 64 bits."""
    with np.errstate(all="ignore"):
        if act != "swiglu":
            dz = dy * slope(z, act)
            return dz, np.abs(dy) * slope_bound(z, act) + 2.0 ** -23 * np.abs(dz)
        F = z.shape[1] // 2
        g, u = z[:, :F], z[:, F:]
        s = value(g, "silu")
        dz = np.concatenate([dy * u * slope(g, "silu"), dy * s], axis=1)
        own = np.concatenate([np.abs(dy * u) * slope_bound(g, "silu"),
                              np.abs(dy) * act_bound(g, "silu", s)], axis=1)
        return dz, own + 2.0 ** -22 * np.abs(dz)


def softmax(x):
    """Over the experts above -infinity; a row without one is 0."""
    with np.errstate(all="ignore"):
        peak = x.max(axis=1, keepdims=True)
        p = np.exp(x - np.where(peak == -np.inf, 0, peak))
        total = p.sum(axis=1, keepdims=True)
        return np.where(total == 0, 0, p / total)


def balance(x, ids):
    """(loss, counts [E + 1]) in 64 bits."""
    E = x.shape[1]
    counts = np.array([(ids == e).sum() for e in range(E)] + [(x > -np.inf).any(axis=1).sum()
                                                              + np.isnan(x).all(axis=1).sum()])
    chosen, tokens = counts[:E].sum(), counts[E]
    if chosen == 0 or tokens == 0:
        return 0.0, counts
    return E * float((counts[:E] / chosen * softmax(x).sum(axis=0)).sum()) / tokens, counts


def route_grad(x, ids, dw, renormalize, counts, dloss):
    """(dlogits, the sum of the magnitudes of its terms) in 64 bits, slot by slot."""
    T, E = x.shape
    p = softmax(x)
    grad, mags = np.zeros((T, E)), np.zeros((T, E))
    with np.errstate(all="ignore"):
        if counts is not None:
            c = counts[:E].astype(np.float64)
            scale = dloss * E / (max(c.sum(), 1) * max(counts[E], 1))
            mean = (p * c).sum(axis=1, keepdims=True)
            grad += scale * p * (c - mean)
            mags += abs(scale) * p * (c + mean)
        if dw is None:
            return grad, mags
        for t in range(T):
            used = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E
                    and not x[t, ids[t, j]] == -np.inf]
            if not used:
                continue
            e, d = ids[t, used], dw[t, used]
            if renormalize:
                w = np.exp(x[t, e] - x[t, e].max())
                w /= w.sum()
                m, am = (w * d).sum(), (w * np.abs(d)).sum()
                for i, ei in enumerate(e):
                    grad[t, ei] += w[i] * (d[i] - m)
                    mags[t, ei] += w[i] * (np.abs(d[i]) + am)
            else:
                w = p[t, e]
                m, am = (w * d).sum(), (w * np.abs(d)).sum()
                grad[t] -= p[t] * m
                mags[t] += p[t] * am
                for i, ei in enumerate(e):
                    grad[t, ei] += w[i] * d[i]
                    mags[t, ei] += w[i] * np.abs(d[i])
    return grad, mags


def softmax_error(x, k):
    """Relative error of a probability: the difference to the peak is rounded once and enters the
    exponential (its own error a few units), a sum of E terms, the division."""
    with np.errstate(all="ignore"):
        d = np.where(np.isfinite(x), np.abs(x - x.max(axis=1, keepdims=True)), 0)
    return (x.shape[1] + k + 32 + 4 * np.where(np.isfinite(d), d, 0)) * 2.0 ** -24


def combine_grad(dout, y, tokens, positions, weights):
    """(dY, dweights, sum of |dout y| per choice) in 64 bits, choice by choice."""
    R, N = y.shape
    dy, dw = np.zeros((R, N)), np.zeros(weights.shape)
    mags = np.zeros(weights.shape)
    with np.errstate(all="ignore"):
        for t in range(positions.shape[0]):
            for j in range(positions.shape[1]):
                r = positions[t, j]
                if not 0 <= r < R:
                    continue
                dw[t, j] = (dout[t] * y[r]).sum()
                mags[t, j] = np.abs(dout[t] * y[r]).sum()
                if tokens[r] == t:
                    total = sum(weights[t, i] for i in range(weights.shape[1])
                                if positions[t, i] == r)
                    dy[r] = total * dout[t]
    return dy, dw, mags
