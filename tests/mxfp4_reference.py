"""Plain 64-bit implementations of the MXFP4 and expert operators (numpy,
elementary operations) and the error bounds the kernels are held to.

Shares no code with the package.  Bounds count a rounding to t bits as
finfo(t).eps / 2 relative, half the smallest subnormal below the normal range,
and a sum of n products in fp32 as (K/8 + 64) 2^-24 of the sum of magnitudes
(the matrix cores add at least 8 products per rounding).
"""
import numpy as np
import torch

MAGNITUDES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
CODE_VALUES = np.concatenate([MAGNITUDES, -MAGNITUDES])
UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}
LARGEST = {t: torch.finfo(t).max for t in UNIT}


def f64(t):
    """A torch tensor's values in numpy float64 (exact for 16 and 32 bits)."""
    return t.detach().cpu().double().numpy()


def quantize(x):
    """x float64 [rows, K] -> (nibbles uint8 [rows, K], scale bytes uint8 [rows, K/32]):
    the scale from frexp, the code by search for the nearest of the eight magnitudes."""
    rows, K = x.shape
    b = x.reshape(rows, K // 32, 32)
    finite = np.isfinite(b).all(axis=2)
    a = np.abs(np.where(finite[:, :, None], b, 0.0))
    peak = a.max(axis=2)
    e = np.where(peak > 0, np.frexp(peak)[1] - 3, 0).clip(-127, 127)
    v = np.ldexp(a, -e[:, :, None])
    d = np.abs(v[..., None] - MAGNITUDES)
    low = d.argmin(axis=3)                                  # the lower of two equally near
    tie = np.take_along_axis(d, np.minimum(low + 1, 7)[..., None], 3)[..., 0] == \
        np.take_along_axis(d, low[..., None], 3)[..., 0]
    code = np.where(tie & (low < 7) & (low % 2 == 1), low + 1, low)
    code = np.where(np.signbit(b), code + 8, code)
    code = np.where(finite[:, :, None], code, 0).astype(np.uint8).reshape(rows, K)
    return code, np.where(finite, e + 127, 255).astype(np.uint8)


def pack(nibbles):
    return (nibbles[..., 0::2] | (nibbles[..., 1::2] << 4)).astype(np.uint8)


def values(codes, scales):
    """float64 values of packed codes [..., K/2] and scale bytes [..., K/32]."""
    c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(codes.shape[:-1] + (-1,))
    e = np.repeat(scales.astype(np.int64) - 127, 32, axis=-1)
    v = np.ldexp(CODE_VALUES[c], e)
    return np.where(e == 128, np.nan, v)


def product(x, w):
    """(x w^T, |x| |w|^T) in 64 bits."""
    with np.errstate(all="ignore"):
        return x @ w.T, np.abs(x) @ np.abs(w).T


def sum_bound(K, mags):
    return (K / 8 + 64) * 2.0 ** -24 * mags


def rounded(y, dtype):
    """Bound of one rounding of values up to |y|."""
    return UNIT[dtype] * np.abs(y) + TINY[dtype]


def check(got, want, bound, dtype):
    """got (torch, dtype) is within bound of want; NaN where want is NaN; where
    want +- bound passes the dtype's largest value an infinity of its sign will do."""
    g = f64(got)
    assert g.shape == want.shape
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(g), nan), "NaN in other places: got %d, want %d" % (
        np.isnan(g).sum(), nan.sum())
    with np.errstate(all="ignore"):
        over = (np.abs(want) + bound > LARGEST[dtype]) & (np.sign(g) == np.sign(want)) & \
            (np.isinf(g) | (np.abs(g - want) <= bound))
        ok = nan | over | (np.abs(g - want) <= bound)
    if not ok.all():
        i = np.unravel_index(np.argmax(~ok), ok.shape)
        raise AssertionError("%d of %d out of bound, first at %s: got %r want %r bound %r"
                             % ((~ok).sum(), ok.size, i, g[i], want[i], np.asarray(bound)[i]))


def swiglu(h, bound):
    """silu(gate) * up and its bound from the bounds of the halves: |silu'| < 1.1,
    and the exponential's argument carries |gate| 2^-23 of relative error into it."""
    F = h.shape[1] // 2
    g, u, bg, bu = h[:, :F], h[:, F:], bound[:, :F], bound[:, F:]
    with np.errstate(all="ignore"):
        s = g / (1 + np.exp(-g))
    y = s * u
    return y, 1.1 * bg * (np.abs(u) + bu) + np.abs(s) * bu + (np.abs(g) + 8) * 2.0 ** -22 * np.abs(y)


def route(logits, k, renormalize):
    """ids [T, k] and weights [T, k] in 64 bits."""
    T, E = logits.shape
    ids, weights = np.full((T, k), -1, dtype=np.int64), np.zeros((T, k))
    for t in range(T):
        row = logits[t]
        usable = [e for e in range(E) if not row[e] == -np.inf]
        order = sorted(usable, key=lambda e: (0, 0.0, e) if np.isnan(row[e]) else (1, -row[e], e))
        chosen = order[:k]
        if not chosen:
            continue
        with np.errstate(all="ignore"):
            p = np.exp(row - row[order[0]])
            total = p[chosen if renormalize else usable].sum()
            ids[t, :len(chosen)] = chosen
            weights[t, :len(chosen)] = p[chosen] / total
    return ids, weights


def plan(ids, E):
    flat = ids.reshape(-1)
    b = np.where((flat >= 0) & (flat < E), flat, E)
    order = np.argsort(b, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(b, minlength=E + 1))[:E]])
    used = np.arange(flat.size) < offsets[E]
    positions = np.empty(flat.size, dtype=np.int64)
    positions[order] = np.where(used, np.arange(flat.size), -1)
    return offsets, np.where(used, order // ids.shape[1], -1), positions.reshape(ids.shape)
