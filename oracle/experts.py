"""CPU oracle of an MLP of experts in 8 bits, in float64: tokens sorted by expert and back, the
e4m3 quantisers, the product with a scale for each block of 128, and the gradients.

TEST INFRASTRUCTURE ONLY (see ``oracle/lmhead.py``).  Formulas written out plainly, slot by slot,
block by block and expert by expert; no shared code with the CUDA path.  The quantisers' scales
and quotients are 32-bit by definition.
"""
from __future__ import annotations

import numpy as np

# e4m3's values by code: 8 subnormals of 2^-9, then 2^e (1 + m / 8) up to 448
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [2.0 ** (e - 7) * (1 + m / 8) for e in range(1, 16) for m in range(8)][:-1])


def _f64(x):
    return np.asarray(x, dtype=np.float64)


# ------------------------------------------------------------------------------- routing

def sort(ids, E):
    """rows [T, k], slots [n], offsets [E + 1]: by expert, then by t * k + j."""
    ids = np.asarray(ids)
    T, k = ids.shape
    rows = np.full((T, k), -1, dtype=np.int64)
    slots, offsets = [], [0]
    for e in range(E):
        for s in np.nonzero(ids.reshape(-1) == e)[0]:
            rows[s // k, s % k] = len(slots)
            slots.append(int(s))
        offsets.append(len(slots))
    return rows, np.array(slots, dtype=np.int64), np.array(offsets, dtype=np.int64)


def gather(X, slots, k):
    return np.asarray(X)[np.asarray(slots) // k]


def combine(Ys, rows, weights=None, residual=None):
    """Y, and per element the size of the terms that make it up."""
    rows = np.asarray(rows)
    T, k = rows.shape
    Ys = _f64(Ys)
    Y = np.zeros((T, Ys.shape[1])) if residual is None else _f64(residual).copy()
    terms = np.abs(Y)
    for t in range(T):
        for j in range(k):
            if 0 <= rows[t, j] < Ys.shape[0]:
                v = (1.0 if weights is None else float(weights[t, j])) * Ys[rows[t, j]]
                Y[t] += v
                terms[t] += np.abs(v)
    return Y, terms


def combine_backward(dY, Ys, rows, weights):
    """dYs (NaN where no slot came from), dweights, and the size of its terms."""
    rows = np.asarray(rows)
    dY, Ys = _f64(dY), _f64(Ys)
    dYs = np.full(Ys.shape, np.nan)
    dw, terms = np.zeros(rows.shape), np.zeros(rows.shape)
    for t in range(rows.shape[0]):
        for j in range(rows.shape[1]):
            r = rows[t, j]
            if 0 <= r < Ys.shape[0]:
                dYs[r] = float(weights[t, j]) * dY[t]
                dw[t, j] = dY[t] @ Ys[r]
                terms[t, j] = np.abs(dY[t]) @ np.abs(Ys[r])
    return dYs, dw, terms


# ---------------------------------------------------------------------------- quantisers

def round_e4m3(x):
    """x (any floats) to e4m3's values, to nearest, ties to the even code; beyond 448: 448."""
    x = np.asarray(x)
    a = np.abs(x)
    # steps of 2^-3 of the value's power of two, 2^-9 below 2^-6; rint takes ties to the even step
    step = np.ldexp(np.ones((), dtype=a.dtype), np.maximum(np.frexp(a)[1] - 1, -6) - 3)
    with np.errstate(invalid="ignore"):
        return np.copysign(np.minimum(np.rint(a / step) * step, 448), x).astype(np.float64)


def block(x):
    """(values in 8 bits, scale) of one block of float32 values."""
    x = np.asarray(x, dtype=np.float32)
    s = scale(np.max(np.abs(x)) if x.size else np.float32(0))
    return round_e4m3(x * (np.float32(1) / s)), s


def scale(m):
    """The scale of blocks whose largest magnitudes are m."""
    m = np.asarray(m, dtype=np.float32)
    s = np.maximum(m * (np.float32(1) / np.float32(448)), np.float32(2.0 ** -126))
    return np.where(m > 0, s, np.float32(1))


def quant(x, tall=1):
    """x [T, d]: blocks of `tall` rows x 128 columns -> values in 8 bits and scales."""
    x = np.asarray(x, dtype=np.float32)
    T, d = x.shape
    nr, nc = (T + tall - 1) // tall, (d + 127) // 128
    full = np.zeros((nr * tall, nc * 128), dtype=np.float32)
    full[:T, :d] = x
    full = full.reshape(nr, tall, nc, 128)
    s = scale(np.abs(full).max(axis=(1, 3), initial=0))
    q = round_e4m3(full * (np.float32(1) / s)[:, None, :, None])
    return q.reshape(nr * tall, nc * 128)[:T, :d], s


def columns(x, offsets):
    """x [T, d] -> [d, 128 blocks]: each expert's tokens from a multiple of 128 on, zeros behind."""
    x = np.asarray(x, dtype=np.float32)
    parts = [np.zeros((x.shape[1], 0), dtype=np.float32)]
    for a, b in zip(offsets[:-1], offsets[1:]):
        p = np.zeros((x.shape[1], (b - a + 127) // 128 * 128), dtype=np.float32)
        p[:, :b - a] = x[a:b].T
        parts.append(p)
    return np.concatenate(parts, axis=1)


def expand(q, s, tall=1):
    """What the 8-bit values stand for."""
    q = _f64(q)
    full = np.repeat(np.repeat(_f64(s), tall, axis=0)[:q.shape[0]], 128, axis=1)[:, :q.shape[1]]
    return q * full


# ------------------------------------------------------------------------------- product

def matmul(A, sa, B, sb, offsets=None):
    """C [T, N] (rows of no expert: NaN) and per element the size of its terms; B [E, N, K]."""
    a = expand(A, sa)
    T = a.shape[0]
    offsets = [0, T] if offsets is None else offsets
    C = np.full((T, np.asarray(B).shape[1]), np.nan)
    terms = np.zeros_like(C)
    for e in range(len(offsets) - 1):
        r = slice(offsets[e], offsets[e + 1])
        b = expand(B[e], sb[e], 128)
        C[r] = a[r] @ b.T
        terms[r] = np.abs(a[r]) @ np.abs(b).T
    return C, terms


def matmul_columns(At, sat, Bt, sbt, offsets):
    """dW [E, N, K] and the size of its terms; At, Bt as ``columns`` and ``quant`` leave them."""
    a, b = expand(At, sat), expand(Bt, sbt, 128)
    dW, terms, at = [], [], 0
    for lo, hi in zip(offsets[:-1], offsets[1:]):
        n = (hi - lo + 127) // 128 * 128
        x, y = a[:, at:at + n], b[:, at:at + n]
        dW.append(x @ y.T)
        terms.append(np.abs(x) @ np.abs(y).T)
        at += n
    return np.stack(dW), np.stack(terms)
