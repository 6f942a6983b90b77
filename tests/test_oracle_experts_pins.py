"""Pins of the experts' oracle: torch's own e4m3 conversion and sort, closed forms, finite
differences, and planted mistakes (CPU only)."""
import numpy as np
import pytest

from oracle import experts as X

torch = pytest.importorskip("torch")


def test_e4m3_values_and_rounding():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(X.E4M3, codes)
    g = np.random.default_rng(0)
    x = np.concatenate([g.uniform(-460, 460, 20000), g.standard_normal(20000) * 0.01, X.E4M3, -X.E4M3,
                        (X.E4M3[:-1] + X.E4M3[1:]) / 2]).astype(np.float32)
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(X.round_e4m3(x), want)
    assert X.round_e4m3(1e9) == 448 and X.round_e4m3(-500.0) == -448 and np.isnan(X.round_e4m3(np.nan))


def test_block_scale():
    q, s = X.block(np.array([448.0, -1.0, 0.5], dtype=np.float32))
    assert s == 1 and q.tolist() == [448.0, -1.0, 0.5]
    q, s = X.block(np.zeros(5, dtype=np.float32))
    assert s == 1 and not q.any()
    q, s = X.block(np.array([1e-45], dtype=np.float32))      # the scale keeps an inverse
    assert s == np.float32(2.0 ** -126)


def test_quant_is_block_by_block():
    g = np.random.default_rng(1)
    for T, d, tall in ((1, 5, 1), (7, 300, 1), (130, 140, 128), (0, 8, 1)):
        x = (g.standard_normal((T, d)) * np.exp(3 * g.standard_normal((T, d)))).astype(np.float32)
        q, s = X.quant(x, tall)
        for i in range(s.shape[0]):
            for j in range(s.shape[1]):
                r, c = slice(tall * i, tall * i + tall), slice(128 * j, 128 * j + 128)
                bq, bs = X.block(x[r, c])
                assert np.array_equal(q[r, c], bq) and s[i, j] == bs


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (7, 2, 3), (40, 8, 16), (33, 3, 200)])
def test_sort(T, k, E):
    g = np.random.default_rng(T)
    ids = g.integers(-1, E, (T, k))
    rows, slots, off = X.sort(ids, E)
    flat = torch.from_numpy(np.where(ids < 0, E, ids)).reshape(-1)
    order = torch.sort(flat, stable=True)[1].numpy()
    assert np.array_equal(slots, order[:slots.size]) and off[-1] == (ids >= 0).sum()
    assert np.array_equal(np.diff(off), np.bincount(ids[ids >= 0], minlength=E))
    assert np.array_equal(rows.reshape(-1)[slots], np.arange(slots.size)) and (rows[ids < 0] == -1).all()


def test_combine_gradients_by_differences():
    g = np.random.default_rng(3)
    T, k, E, d = 5, 3, 4, 6
    ids = g.integers(-1, E, (T, k))
    rows, slots, _ = X.sort(ids, E)
    Ys, w, dY = g.standard_normal((slots.size, d)), g.standard_normal((T, k)), g.standard_normal((T, d))
    loss = lambda Ys, w: float((X.combine(Ys, rows, w)[0] * dY).sum())
    dYs, dw, _ = X.combine_backward(dY, Ys, rows, w)
    h = 1e-6
    for i in np.ndindex(Ys.shape):
        a, b = Ys.copy(), Ys.copy()
        a[i] += h
        b[i] -= h
        assert abs((loss(a, w) - loss(b, w)) / (2 * h) - dYs[i]) < 1e-8
    for i in np.ndindex(w.shape):
        a, b = w.copy(), w.copy()
        a[i] += h
        b[i] -= h
        assert abs((loss(Ys, a) - loss(Ys, b)) / (2 * h) - dw[i]) < 1e-8
    # the gather's gradient: the combine without weights
    x = g.standard_normal((T, d))
    dXs = g.standard_normal((slots.size, d))
    dX, _ = X.combine(dXs, rows)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        diff = ((X.gather(a, slots, k) - X.gather(b, slots, k)) * dXs).sum() / (2 * h)
        assert abs(diff - dX[i]) < 1e-8


def test_product_and_its_gradients():
    """Unit scales and whole numbers: the product and both gradients are those of the dense layers."""
    g = np.random.default_rng(4)
    N, K, off = 24, 40, [0, 3, 3, 140, 141]
    T, E = off[-1], len(off) - 1
    A, B = g.integers(-8, 9, (T, K)).astype(float), g.integers(-8, 9, (E, N, K)).astype(float)
    dY = g.integers(-8, 9, (T, N)).astype(float)
    C, terms = X.matmul(A, np.ones((T, 1)), B, np.ones((E, 1, 1)), off)
    nb = sum((b - a + 127) // 128 for a, b in zip(off, off[1:]))
    dW, _ = X.matmul_columns(X.columns(dY, off), np.ones((N, nb)), X.columns(A, off), np.ones((1, nb)), off)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        assert np.array_equal(C[r], A[r] @ B[e].T) and np.array_equal(dW[e], dY[r].T @ A[r])
    assert (terms >= np.abs(C)).all()


def test_quantised_layer_near_the_exact_one():
    """A layer in 8 bits: each product's relative error is at most (1 + 2^-4)^2 - 1 of its size but
    for what the subnormals lose, 2^-10 of the scale an element."""
    g = np.random.default_rng(5)
    T, N, K = 9, 140, 300
    x, w = g.standard_normal((T, K)).astype(np.float32), g.standard_normal((N, K)).astype(np.float32)
    (a, sa), (b, sb) = X.quant(x), X.quant(w, 128)
    C, _ = X.matmul(a, sa, b[None], sb[None])
    xa, wa = np.abs(x).astype(float), np.abs(w).astype(float)
    ea = xa * 2.0 ** -4 + np.repeat(sa, 128, 1)[:, :K] * 2.0 ** -10
    eb = wa * 2.0 ** -4 + np.repeat(np.repeat(sb, 128, 0)[:N], 128, 1)[:, :K] * 2.0 ** -10
    bound = ea @ wa.T + xa @ eb.T + ea @ eb.T
    assert (np.abs(C - x.astype(float) @ w.T.astype(float)) <= bound * (1 + 1e-5)).all()


def test_planted_mistakes_are_seen():
    g = np.random.default_rng(6)
    x = g.standard_normal((130, 260)).astype(np.float32)
    q, s = X.quant(x)
    # a scale taken from the neighbouring block, tokens of two experts in one block
    assert np.abs(X.expand(q, np.roll(s, 1, axis=1)) - x).max() > 4 * np.abs(X.expand(q, s) - x).max()
    one, two = X.columns(x, [0, 130]), X.columns(x, [0, 5, 130])
    assert one.shape == two.shape and not np.array_equal(one, two)
