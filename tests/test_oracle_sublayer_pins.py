"""Pins of the sublayer oracle: gradients against central differences, closed forms, and the
invariances the operators have by definition."""
import numpy as np
import pytest

from oracle import attention as A
from oracle import sublayer as S


def _diff(f, x, w, h=1e-6):
    """Gradient of sum(w * f(x)) by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (w * (f(a) - f(b))).sum() / (2 * h)
    return g


def test_norm_gradient_by_differences():
    g = np.random.default_rng(1)
    R, dY, gamma = g.standard_normal((3, 8)), g.standard_normal((3, 8)), 1 + 0.3 * g.standard_normal(8)
    b = S.rmsnorm_backward(dY, R, gamma, 1e-3)
    assert np.allclose(b["dX"], _diff(lambda r: S.rmsnorm(r, gamma, 1e-3)[0], R, dY), atol=1e-8)
    assert np.allclose(b["dgamma"], _diff(lambda c: S.rmsnorm(R, c, 1e-3)[0], gamma, dY), atol=1e-8)
    assert np.allclose(S.rmsnorm_backward(dY, R, gamma, 1e-3, dR=R)["dX"], b["dX"] + R)


def test_norm_closed_forms():
    Y, rstd = S.rmsnorm(np.full((1, 16), -3.0), np.ones(16), 0.0)
    assert np.allclose(Y, -1.0) and np.allclose(rstd, 1 / 3)
    # without eps the norm does not see the row's scale: the gradient is orthogonal to R
    g = np.random.default_rng(2)
    R, dY = g.standard_normal((2, 8)), g.standard_normal((2, 8))
    assert np.allclose((S.rmsnorm_backward(dY, R, np.ones(8), 0.0)["dX"] * R).sum(axis=1), 0.0, atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_turns_and_returns(interleaved):
    g = np.random.default_rng(3)
    x = g.standard_normal((2, 5, 8))
    pos = g.integers(0, 10**6, (2, 5))
    inv = 100.0 ** (-np.arange(3) / 3)
    a = S.rope_angles(pos, [1, 2], inv)
    assert np.allclose(a[:, 0], pos[0]) and np.allclose(a[:, 2], pos[1] * inv[2])
    y = S.rope(x, a, interleaved)
    assert np.allclose(S.rope(y, a, interleaved, inverse=True), x)
    assert np.array_equal(y[..., 6:], x[..., 6:])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    # q . k depends on the distance alone (one axis)
    one = np.arange(5)[None]
    q = S.rope(np.repeat(x[:1, :1], 5, 1), S.rope_angles(one, [3], inv), interleaved)[0]
    k = S.rope(np.repeat(x[1:, :1], 5, 1), S.rope_angles(one, [3], inv), interleaved)[0]
    assert np.allclose(q[1] @ k[0], q[4] @ k[3]) and np.allclose(q[3] @ k[1], q[4] @ k[2])


def test_visible():
    see = S.visible(9, [0, 3, 3, 8], [2, 0, 0])
    want = np.zeros((9, 9), bool)
    want[0, :2] = want[1, :2] = want[2, :3] = True
    for i in range(3, 8):
        want[i, 3:i + 1] = True
    assert np.array_equal(see, want)


def test_attention_matches_the_causal_oracle():
    g = np.random.default_rng(4)
    Q, K, V, dO = g.standard_normal((4, 7, 4)), *g.standard_normal((2, 2, 7, 4)), g.standard_normal((4, 7, 4))
    see = S.visible(7)
    f, r = S.attention(Q, K, V, see, 0.5), A.forward(Q, K, V, 0.5)
    assert np.allclose(f["O"], r["O"]) and np.allclose(f["lse"], r["lse"])
    b = S.attention_backward(Q, K, V, f["O"], dO, f["lse"], see, 0.5)
    rb = A.backward(Q, K, V, r["O"], dO, r["lse"], 0.5)
    assert all(np.allclose(b[k], rb[k]) for k in ("dQ", "dK", "dV"))


@pytest.mark.parametrize("softcap,alibi,prefix", [(0.0, False, None), (1.5, False, None), (0.0, True, [2, 0]),
                                                  (0.7, True, [9, 1])])
def test_attention_gradient_by_differences(softcap, alibi, prefix):
    g = np.random.default_rng(5)
    T, see = 6, S.visible(6, [0, 3, 5], prefix)
    Q, K, V = g.standard_normal((2, T, 3)), g.standard_normal((1, T, 3)), g.standard_normal((1, T, 3))
    dO = g.standard_normal((2, T, 3))
    sl = [0.5, 0.25] if alibi else None
    fwd = lambda q, k, v: S.attention(q, k, v, see, 0.8, softcap, sl)
    f = fwd(Q, K, V)
    assert np.all(f["O"][:, 5] == 0) and np.all(np.isneginf(f["lse"][:, 5]))
    b = S.attention_backward(Q, K, V, f["O"], dO, f["lse"], see, 0.8, softcap, sl)
    assert np.allclose(b["dQ"], _diff(lambda q: fwd(q, K, V)["O"], Q, dO), atol=1e-7)
    assert np.allclose(b["dK"], _diff(lambda k: fwd(Q, k, V)["O"], K, dO), atol=1e-7)
    assert np.allclose(b["dV"], _diff(lambda v: fwd(Q, K, v)["O"], V, dO), atol=1e-7)
    assert np.all(b["dK"][:, 5] == 0) and np.all(b["dV"][:, 5] == 0)
