"""CPU oracle of the attention sublayer's operators in float64: RMS norm with the
residual's addition, rotary positions with several axes, attention over packed documents.

TEST INFRASTRUCTURE ONLY (see ``oracle/lmhead.py``).  Formulas written out plainly, one
document and one head at a time; no shared code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


# ------------------------------------------------------------------------------- norm

def rmsnorm(R, gamma, eps):
    """Y and rstd [T] of the rows of R."""
    R, gamma = _f64(R), _f64(gamma)
    rstd = 1.0 / np.sqrt((R * R).mean(axis=1) + eps)
    return R * rstd[:, None] * gamma, rstd


def rmsnorm_backward(dY, R, gamma, eps, dR=None):
    """dX, dgamma, and per element the size of the terms that make dX up."""
    dY, R, gamma = _f64(dY), _f64(R), _f64(gamma)
    _, rstd = rmsnorm(R, gamma, eps)
    r = rstd[:, None]
    g = dY * gamma
    mean = (g * R).mean(axis=1)[:, None]
    dX = r * (g - R * r * r * mean)
    terms = r * (np.abs(g) + np.abs(R) * r * r * np.abs(g * R).mean(axis=1)[:, None])
    if dR is not None:
        dX = dX + _f64(dR)
        terms = terms + np.abs(_f64(dR))
    return dict(dX=dX, terms=terms, dgamma=(dY * R * r).sum(axis=0), dgamma_terms=np.abs(dY * R * r).sum(axis=0))


# ------------------------------------------------------------------------------- rope

def rope_angles(positions, sections, inv_freq):
    """[T, pairs]: position of the pair's axis times its frequency."""
    axis = np.repeat(np.arange(len(sections)), sections)
    return _f64(positions)[axis].T * _f64(inv_freq)


def rope(x, angles, interleaved, inverse=False):
    """x [heads, T, hd]; the first 2 * pairs elements of a row turn."""
    x = _f64(x)
    n = angles.shape[1]
    c, s = np.cos(angles), np.sin(angles) * (-1.0 if inverse else 1.0)
    y = x.copy()
    for p in range(n):
        a, b = (2 * p, 2 * p + 1) if interleaved else (p, p + n)
        y[..., a] = x[..., a] * c[:, p] - x[..., b] * s[:, p]
        y[..., b] = x[..., b] * c[:, p] + x[..., a] * s[:, p]
    return y


# -------------------------------------------------------------------------- attention

def visible(T, cu=None, prefix=None):
    """[T, T] bool: query i sees key j."""
    cu = [0, T] if cu is None else [int(c) for c in cu]
    see = np.zeros((T, T), dtype=bool)
    for s in range(len(cu) - 1):
        a, b = cu[s], cu[s + 1]
        p = 0 if prefix is None else int(prefix[s])
        for i in range(a, b):
            for j in range(a, b):
                see[i, j] = j <= i or j - a < p
    return see


def _scores(q, k, scale, softcap, slope):
    t = scale * (q @ k.T)
    d = np.ones_like(t)
    if softcap > 0:
        th = np.tanh(t / softcap)
        t, d = softcap * th, 1.0 - th * th
    if slope:
        n = np.arange(len(q))
        t = t - slope * np.abs(n[:, None] - n[None, :])
    return t, d


def attention(Q, K, V, see, scale, softcap=0.0, slopes=None):
    """O, lse (-inf where a query sees nothing), and sum_j P |V| per element."""
    Q, K, V = _f64(Q), _f64(K), _f64(V)
    H, T, _ = Q.shape
    grp = H // K.shape[0]
    O, size, lse = np.zeros_like(Q), np.zeros_like(Q), np.full((H, T), -np.inf)
    some = see.any(axis=1)
    for h in range(H):
        x, _ = _scores(Q[h], K[h // grp], scale, softcap, 0.0 if slopes is None else float(slopes[h]))
        x = np.where(see, x, -np.inf)
        m = np.where(some, x.max(axis=1, initial=-np.inf), 0.0)
        e = np.exp(x - m[:, None])
        l = e.sum(axis=1)
        lse[h, some] = (m + np.log(np.where(some, l, 1.0)))[some]
        P = e / np.where(some, l, 1.0)[:, None]
        O[h], size[h] = P @ V[h // grp], P @ np.abs(V[h // grp])
    return dict(O=O, lse=lse, size=size)


def attention_backward(Q, K, V, O, dO, lse, see, scale, softcap=0.0, slopes=None, errO=None):
    """dQ, dK, dV at the given O and lse, and bounds of what rounding P and dS to bf16 (2^-8 of
    each) and fp32 sums (2^-11 of the terms of dS; 2^-11 of P, from the scores' and the
    exponential's error) can do to them: bQ, bK, bV.  errO: what the O that D = dO . O is taken
    from may be off by (per element; default 0)."""
    Q, K, V, O, dO, lse = (_f64(a) for a in (Q, K, V, O, dO, lse))
    grp = Q.shape[0] // K.shape[0]
    out = dict(dQ=np.zeros_like(Q), dK=np.zeros_like(K), dV=np.zeros_like(V),
               bQ=np.zeros_like(Q), bK=np.zeros_like(K), bV=np.zeros_like(V))
    for h in range(Q.shape[0]):
        z = h // grp
        x, d = _scores(Q[h], K[z], scale, softcap, 0.0 if slopes is None else float(slopes[h]))
        P = np.where(see, np.exp(np.where(see, x, 0.0) - np.where(np.isfinite(lse[h]), lse[h], 0.0)[:, None]), 0.0)
        D = (dO[h] * O[h]).sum(axis=1)
        dP = dO[h] @ V[z].T
        dS = P * (dP - D[:, None]) * d
        terms = P * (np.abs(dO[h]) @ np.abs(V[z]).T + np.abs(dO[h] * O[h]).sum(axis=1)[:, None])
        err = 2.0 ** -8 * np.abs(dS) + 2.0 ** -11 * terms
        if errO is not None:
            err += P * d * (np.abs(dO[h]) * errO[h]).sum(axis=1)[:, None]
        out["dQ"][h] = scale * dS @ K[z]
        out["bQ"][h] = scale * err @ np.abs(K[z])
        out["dK"][z] += scale * dS.T @ Q[h]
        out["bK"][z] += scale * err.T @ np.abs(Q[h])
        out["dV"][z] += P.T @ dO[h]
        out["bV"][z] += (2.0 ** -8 + 2.0 ** -11) * P.T @ np.abs(dO[h])
    return out
