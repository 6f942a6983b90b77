"""GPU parity of the expert routing, the e4m3 quantisers and the block-scaled 8-bit products against
the float64 oracle, and a run of them as an MLP of experts is trained.

Tolerances are element by element.  u: half a step of the output's type (bf16 2^-8, fp32 2^-24).
Sorted places, gathered rows, quantised values and scales are equal: copies, or single 32-bit
operations rounded to nearest.  Sums over k slots: at most k + 1 roundings of 2^-24 of the terms.
Dot products over d columns: d + 16.  Products: a block of 128 terms and the blocks' sum, each
operation within 2^-23 of the terms' size (the tensor cores' sums may be cut off instead of
rounded), so 128 + blocks + 16 of them.
"""
import numpy as np
import pytest

from oracle import experts as X
from memory_efficient_exact_gb300 import inputs as I

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TY = {"bf16": (BF, 2.0 ** -8), "fp32": (F32, 2.0 ** -24)}


@pytest.fixture(scope="module")
def sbp():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from memory_efficient_exact_gb300 import _build
    _build.build_library()
    from memory_efficient_exact_gb300 import sbp as mod
    return mod


def dev(x, dt):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(dt).contiguous()


def host(t):
    return t.detach().double().cpu().numpy()


def near(name, got, want, bound):
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), (name, float((err / np.maximum(bound, 1e-300)).max()), np.argwhere(bad)[:4].tolist())


def ok(*results):
    torch.cuda.synchronize()
    for r in results:
        assert int(r["status"].item()) == 0


def normal(g, shape, dtype, std=1.0):
    x = (g.standard_normal(shape) * std).astype(np.float32)
    return I.round_bf16(x) if dtype == "bf16" else x


# ------------------------------------------------------------------------------- routing

def draw_ids(g, T, k, E, drop):
    """Distinct experts a token where there are enough, some much loaded, some slots dropped."""
    p = g.exponential(size=E) + 1e-3
    p /= p.sum()
    ids = np.stack([g.choice(E, k, replace=k > E, p=None if k == E else p) for _ in range(T)]) if T else \
        np.zeros((0, k), dtype=np.int64)
    ids[g.random((T, k)) < drop] = -1
    return ids


ROUTES = [(0, 2, 4, 0.0), (1, 1, 1, 0.0), (1, 8, 64, 0.0), (5, 2, 3, 0.3), (7, 3, 2, 0.0), (300, 8, 64, 0.1), (1000, 4, 1024, 0.0),
          (2048, 2, 7, 0.5), (2049, 2, 33, 0.0), (4099, 3, 100, 0.2), (33, 1, 5, 1.0)]


@pytest.mark.parametrize("T,k,E,drop", ROUTES)
def test_sort(sbp, T, k, E, drop):
    ids = draw_ids(np.random.default_rng(T + E), T, k, E, drop)
    rows, slots, off = X.sort(ids, E)
    place = torch.full((T * k,), 77, dtype=torch.int32, device="cuda")
    r = sbp.expert_sort(dev(ids, torch.int32), E, slots=place)
    ok(r)
    assert np.array_equal(host(r["rows"]), rows) and np.array_equal(host(r["offsets"]), off)
    got = host(place)
    assert np.array_equal(got[:slots.size], slots) and (got[slots.size:] == 77).all()


def test_sort_one_expert_for_all_and_many_blocks(sbp):
    T, k, E = 30000, 8, 16
    for fill in (None, 3):
        ids = np.random.default_rng(1).integers(-1, E, (T, k)) if fill is None else np.full((T, k), fill)
        r = sbp.expert_sort(dev(ids, torch.int32), E)
        ok(r)
        order = np.argsort(np.where(ids < 0, E, ids).reshape(-1), kind="stable")
        n = int((ids >= 0).sum())
        assert np.array_equal(host(r["slots"])[:n], order[:n])
        assert np.array_equal(host(r["offsets"]), np.concatenate([[0], np.cumsum(np.bincount(ids[ids >= 0], minlength=E))]))
        rows = np.full(T * k, -1)
        rows[order[:n]] = np.arange(n)
        assert np.array_equal(host(r["rows"]).reshape(-1), rows)


@pytest.mark.parametrize("T,E", [(63 * 2048, 40), (63 * 2048 + 1, 40), (64 * 2048 + 77, 1024), ((1 << 20) + 7, 33), ((1 << 22) + 1, 5)])
def test_sort_blocks_whose_counts_are_summed_once(sbp, T, E):
    ids = np.random.default_rng(T).integers(-1, E, (T, 1))
    r = sbp.expert_sort(dev(ids, torch.int32), E)
    ok(r)
    flat = ids.reshape(-1)
    n = int((flat >= 0).sum())
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable")[:n]
    assert np.array_equal(host(r["slots"])[:n], order)
    assert np.array_equal(host(r["offsets"]), np.concatenate([[0], np.cumsum(np.bincount(flat[flat >= 0], minlength=E))]))
    rows = np.full(T, -1)
    rows[order] = np.arange(n)
    assert np.array_equal(host(r["rows"]).reshape(-1), rows)


def test_sort_id_past_the_last_expert(sbp):
    for T in (3, 5000):
        ids = np.random.default_rng(2).integers(0, 4, (T, 2))
        ids[T - 1, 1] = 4
        r = sbp.expert_sort(dev(ids, torch.int32), 4)
        torch.cuda.synchronize()
        assert int(r["status"].item()) == sbp.ERR_EXPERT_RANGE
        assert host(r["rows"])[T - 1, 1] == -1 and host(r["offsets"])[4] == 2 * T - 1
        ok(sbp.expert_sort(dev(np.minimum(ids, 3), torch.int32), 4, status=r["status"]))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [8, 72, 136, 2048, 5128])
@pytest.mark.parametrize("T,k,E,drop", [(1, 8, 64, 0.0), (5, 2, 3, 0.3), (37, 1, 4, 0.0), (70, 3, 5, 0.1), (66, 8, 16, 0.2), (19, 11, 12, 0.0)])
def test_gather_combine_and_gradients(sbp, T, k, E, drop, d, dtype):
    ty, u = TY[dtype]
    g = np.random.default_rng(T * k + d)
    ids = draw_ids(g, T, k, E, drop)
    rows, slots, _ = X.sort(ids, E)
    n, dr = slots.size, dev(rows, torch.int32)
    x, ys, res, dy, dxs = (normal(g, (m, d), dtype) for m in (T, T * k, T, T, T * k))
    w = g.standard_normal((T, k)).astype(np.float32)
    pad = lambda: torch.full((T * k, d), 7.0, dtype=ty, device="cuda")
    xs = sbp.expert_gather(dev(x, ty), dr, Xs=pad())["Xs"]
    assert np.array_equal(host(xs)[:n], X.gather(x, slots, k)) and (host(xs)[n:] == 7).all()
    ysd = dev(ys, ty)
    ysd[n:] = float("nan")                       # rows of no slot are not read
    for weights, residual in ((w, res), (w, None), (None, res)):
        got = sbp.expert_combine(ysd, dr, None if weights is None else dev(weights, F32),
                                 residual=None if residual is None else dev(residual, ty))["Y"]
        want, terms = X.combine(ys[:n], rows, weights, residual)
        near("Y", host(got), want, u * np.abs(want) + (k + 1) * 2.0 ** -24 * terms + 1e-38)
    inplace = dev(res, ty)
    assert torch.equal(sbp.expert_combine(ysd, dr, dev(w, F32), residual=inplace, Y=inplace)["Y"],
                       sbp.expert_combine(ysd, dr, dev(w, F32), residual=dev(res, ty))["Y"])
    dx = sbp.expert_gather_backward(dev(dxs, ty), dr)["dX"]
    want, terms = X.combine(dxs[:n], rows)
    near("dX", host(dx), want, u * np.abs(want) + (k + 1) * 2.0 ** -24 * terms + 1e-38)
    b = sbp.expert_combine_backward(dev(dy, ty), ysd, dr, dev(w, F32), dYs=pad())
    dys, dw, terms = X.combine_backward(dy, ys[:n], rows, w)
    near("dYs", host(b["dYs"])[:n], dys, (u + 2.0 ** -24) * np.abs(dys) + 1e-38)
    assert (host(b["dYs"])[n:] == 7).all()
    near("dweights", host(b["dweights"]), dw, (d + 16) * 2.0 ** -24 * terms)
    assert (host(b["dweights"])[ids < 0] == 0).all()


def test_gather_8_bits_and_fewer_rows(sbp):
    g = np.random.default_rng(9)
    for T, k, d in ((1, 8, 16), (50, 2, 144), (130, 4, 2576)):
        rows, slots, _ = X.sort(draw_ids(g, T, k, 9, 0.1), 9)
        q = sbp.quant_e4m3(dev(normal(g, (T, d), "bf16"), BF))
        n = slots.size
        for cap in (T * k, max(n - 3, 0)):        # places past the rows there are: left out
            r = sbp.expert_gather(q["Y8"], dev(rows, torch.int32), scales=q["scales"], n_rows=cap)
            m = min(n, cap)
            assert np.array_equal(host(r["Xs"])[:m], X.gather(host(q["Y8"]), slots, k)[:m])
            assert np.array_equal(host(r["scales"])[:m], X.gather(host(q["scales"]), slots, k)[:m])


# ---------------------------------------------------------------------------- quantisers

def table(g, T, E):
    cuts = np.sort(g.integers(0, T + 1, E - 1))
    return np.concatenate([[0], cuts, [T]]).astype(np.int64)


def wide(g, shape, dtype):
    x = normal(g, shape, "fp32") * np.exp(g.standard_normal(shape)).astype(np.float32)
    x[:, :: 7] *= 30
    if shape[0] > 2:
        x[2] = 0
    return I.round_bf16(x) if dtype == "bf16" else x


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(0, 64), (1, 8), (3, 128), (9, 136), (130, 264), (301, 2560), (5, 16392)])
def test_quant_rows(sbp, T, d, dtype):
    x = wide(np.random.default_rng(T + d), (T, d), dtype)
    r = sbp.quant_e4m3(dev(x, TY[dtype][0]))
    q, s = X.quant(x)
    assert np.array_equal(host(r["Y8"]), q) and np.array_equal(host(r["scales"]), s.astype(np.float64))


def test_quant_rows_as_the_norm_leaves_them(sbp):
    """With gamma and R such that the norm's Y is exact, both give the same 8 bits."""
    x = dev(np.random.default_rng(3).choice([-1.0, 1.0], (9, 256)), BF)
    a, b = sbp.rmsnorm_e4m3(x, torch.ones(256, dtype=BF, device="cuda"), 0.0), sbp.quant_e4m3(x)
    assert torch.equal(a["Y8"].view(torch.uint8), b["Y8"].view(torch.uint8)) and torch.equal(a["scales"], b["scales"])


def test_quant_extremes(sbp):
    x = np.zeros((7, 256), dtype=np.float32)
    x[0, 0], x[1, 3], x[2, 130], x[3, 0] = 1e-45, 3e38, np.inf, np.nan
    x[3, 1], x[4, :] = 2.0, -448.0
    x[5, :128] = np.arange(128) * 2.0 ** -9        # subnormals of the 8-bit values, scale 1
    x[5, 0] = 448
    r = sbp.quant_e4m3(dev(x, F32))
    q, s = host(r["Y8"]), host(r["scales"])
    for i in (0, 1, 4, 5, 6):
        wq, ws = X.quant(x[i:i + 1])
        assert np.array_equal(q[i:i + 1], wq) and np.array_equal(s[i:i + 1], ws.astype(np.float64)), i
    assert np.isinf(s[2, 1]) and s[2, 0] == 1 and np.isnan(q[2, 130] * s[2, 1]) and np.isnan(q[3, 0])
    assert s[3, 0] == np.float32(2.0) * (np.float32(1.0) / np.float32(448.0)) and q[3, 1] == 448


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d,E", [(1, 8, 1), (127, 128, 1), (129, 136, 1), (300, 264, 3), (513, 72, 7), (40, 128, 33), (700, 520, 2)])
def test_quant_columns(sbp, T, d, E, dtype):
    g = np.random.default_rng(T + d + E)
    x = wide(g, (T, d), dtype)
    off = table(g, T, E)
    xt = X.columns(x, off)
    W = xt.shape[1]
    kw = dict(offsets=None if E == 1 else dev(off, torch.int32))
    nb = sbp.token_blocks(T, E)
    for tiles in (False, True):
        for rows in (False, True):
            yt = torch.full((d, 128 * nb), 1.0, device="cuda").to(F8)
            r = sbp.quant_e4m3_columns(dev(x, TY[dtype][0]), tiles=tiles, rows=rows, Yt8=yt, **kw)
            ok(r)
            q, s = X.quant(xt, 128 if tiles else 1)
            assert np.array_equal(host(yt)[:, :W], q) and (host(yt)[:, W:] == 1).all()
            assert np.array_equal(host(r["scales_t"])[:, :W // 128], s.astype(np.float64))
            if rows:
                q, s = X.quant(x)
                assert np.array_equal(host(r["Y8"]), q) and np.array_equal(host(r["scales"]), s.astype(np.float64))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("E,N,K", [(0, 16, 16), (0, 144, 272), (3, 128, 400), (2, 272, 128)])
def test_quant_weight(sbp, E, N, K, dtype):
    g = np.random.default_rng(N + K)
    w = np.stack([wide(g, (N, K), dtype) for _ in range(max(E, 1))])
    r = sbp.quant_e4m3_weight(dev(w if E else w[0], TY[dtype][0]))
    for e in range(max(E, 1)):
        q, s = X.quant(w[e], 128)
        at = (lambda t: host(t)[e]) if E else host
        assert np.array_equal(at(r["W8"]), q) and np.array_equal(at(r["scales"]), s.astype(np.float64))
        assert np.array_equal(at(r["Wt8"]), q.T) and np.array_equal(at(r["scales_t"]), s.T.astype(np.float64))


@pytest.mark.parametrize("T,d,tiles", [(1, 8, False), (5, 136, False), (9, 24, True), (130, 264, True), (300, 2568, False), (2, 20480, False),
                                       (257, 20488, True)])
def test_expand(sbp, T, d, tiles):
    g = np.random.default_rng(T + d)
    q, s = X.quant(wide(g, (T, d), "fp32"), 128 if tiles else 1)
    v = (q.astype(np.float32) * X.expand(np.ones_like(q), s, 128 if tiles else 1).astype(np.float32))
    for ty in (F32, BF):
        y = sbp.quant_e4m3_expand(dev(q, F8), dev(s, F32), ty, tiles=tiles)["Y"]
        assert torch.equal(y, torch.from_numpy(v).cuda().to(ty))


# ------------------------------------------------------------------------------ products

def operands(g, T, N, K, E):
    a, sa = X.quant(wide(g, (T, K), "fp32"))
    b, sb = zip(*[X.quant(normal(g, (N, K), "fp32", K ** -0.5), 128) for _ in range(E)])
    return a, sa, np.stack(b), np.stack(sb)


def check_product(sbp, off, N, K, dtype, seed, **kw):
    g = np.random.default_rng(seed)
    E, T = len(off) - 1, kw.pop("T", off[-1])
    a, sa, b, sb = operands(g, T, N, K, E)
    C = torch.full((T, N), 5.0, dtype=TY[dtype][0], device="cuda")
    one = E == 1 and off[-1] == T
    r = sbp.matmul_e4m3(dev(a, F8), dev(sa, F32), dev(b[0] if one else b, F8), dev(sb[0] if one else sb, F32),
                        offsets=None if one else dev(np.array(off), torch.int32), C=C)
    ok(r)
    want, terms = X.matmul(a, sa, b, sb, off)
    n = off[-1]
    got = host(C)
    assert (got[n:] == 5).all()
    steps = 128 + (K + 127) // 128 + 16
    near("C", got[:n], want[:n], TY[dtype][1] * np.abs(want[:n]) + steps * 2.0 ** -23 * terms[:n])
    return r


DENSE = [(1, 8, 16), (1, 256, 128), (2, 520, 2560), (7, 1024, 144), (9, 264, 1040), (16, 128, 4096), (17, 4096, 272), (31, 136, 384),
         (33, 512, 512), (64, 1000, 640), (127, 256, 256), (128, 128, 128), (129, 264, 400), (255, 512, 128), (256, 256, 1024),
         (257, 776, 656), (501, 1032, 2064), (640, 3000, 384), (1025, 520, 528)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,N,K", DENSE)
def test_product(sbp, T, N, K, dtype):
    check_product(sbp, [0, T], N, K, dtype, T + N + K)


# sizes that go to the tensor cores' tiles (of 256 and of 128 columns), ragged in every way: blocks
# of the sum from one to more than the operands' ring holds, odd numbers of them, last ones cut off
MANY = [(1500, 4104, 128), (1025, 4096, 144), (2049, 2056, 400), (700, 2568, 1040), (513, 4096, 2576), (300, 5128, 4112),
        (5000, 4104, 272), (3001, 8200, 656), (70, 8192, 4096)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,N,K", MANY)
def test_product_of_many_rows(sbp, T, N, K, dtype):
    check_product(sbp, [0, T], N, K, dtype, T + N + K)


@pytest.mark.parametrize("lens,N,K,behind", [
    ([1000, 0, 1, 255, 256, 257, 0, 900], 2056, 656, 0), ([1500, 1500], 4104, 528, 70), ([0, 3000, 0], 2056, 1168, 5),
    ([40] * 60, 2568, 400, 11), ([600, 0, 1300, 513, 7], 2056, 2064, 0)])
def test_product_of_experts_with_many_rows(sbp, lens, N, K, behind):
    off = np.concatenate([[0], np.cumsum(lens)]).tolist()
    check_product(sbp, off, N, K, "bf16", N + K + len(lens), T=off[-1] + behind)


# few rows of several wide matrices: the kernel with the operands exchanged
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,N,K,behind", [
    ([10, 0, 1, 33, 32, 31, 64, 9, 0, 17, 5, 3], 4096, 2064, 0), ([3] * 24, 2056, 2576, 7), ([20, 41, 7, 16], 8200, 1040, 0),
    ([65, 0, 100, 2, 30, 8, 8, 70], 4104, 4112, 3), ([32], 24584, 1168, 0)])
def test_product_of_experts_with_few_rows(sbp, lens, N, K, behind, dtype):
    off = np.concatenate([[0], np.cumsum(lens)]).tolist()
    check_product(sbp, off, N, K, dtype, N + K + len(lens), T=off[-1] + behind)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,N,K,behind", [
    ([1, 0, 2], 264, 272, 0), ([0, 0, 5, 0], 128, 128, 3), ([3] * 40, 136, 400, 0), ([0, 9, 17, 33, 1, 0], 512, 2064, 1),
    ([300, 0, 1, 255, 256, 257, 0], 520, 656, 0), ([128, 128], 256, 512, 70), ([0], 256, 128, 4), ([1000, 3, 1200], 1032, 384, 5),
    ([2] * 300, 128, 144, 0), ([700], 264, 128, 9)])
def test_product_of_experts(sbp, lens, N, K, behind, dtype):
    off = np.concatenate([[0], np.cumsum(lens)]).tolist()
    check_product(sbp, off, N, K, dtype, N + K + len(lens), T=off[-1] + behind)


@pytest.mark.parametrize("lens,N,K", [
    ([1], 8, 8), ([5], 128, 128), ([128], 264, 136), ([129], 520, 72), ([1000], 256, 512), ([0, 3, 0], 136, 264),
    ([300, 0, 1, 127, 128, 129, 0], 264, 392), ([2000, 70], 512, 776), ([1] * 70, 72, 128),
    # the tensor cores' tiles
    ([3000], 1032, 1800), ([1000, 0, 1700, 1, 128], 1544, 1032), ([5000, 70], 520, 776)])
def test_product_of_columns(sbp, lens, N, K):
    g = np.random.default_rng(N + K + len(lens))
    off = np.concatenate([[0], np.cumsum(lens)])
    T, E = int(off[-1]), len(lens)
    dy, x = wide(g, (T, N), "bf16") * 1e-4, wide(g, (T, K), "bf16")
    kw = dict(offsets=None if E == 1 else dev(off, torch.int32))
    # what lies behind the last expert's blocks is not read
    nb = sbp.token_blocks(T, E)
    junk = lambda rows: torch.full((rows, 128 * nb), float("nan"), device="cuda").to(F8)
    a = sbp.quant_e4m3_columns(dev(dy, BF), Yt8=junk(N), **kw)
    b = sbp.quant_e4m3_columns(dev(x, BF), tiles=True, Yt8=junk(K), **kw)
    r = sbp.matmul_e4m3_columns(a["Yt8"], a["scales_t"], b["Yt8"], b["scales_t"], T, **kw)
    ok(a, b, r)
    dyr = host(dev(dy, BF)).astype(np.float32)
    (qa, sa), (qb, sb) = X.quant(X.columns(dyr, off)), X.quant(X.columns(x, off), 128)
    want, terms = X.matmul_columns(qa, sa, qb, sb, off)
    got = host(r["dW"]).reshape(want.shape)
    steps = 128 + max((n + 127) // 128 for n in lens) + 16
    near("dW", got, want, steps * 2.0 ** -23 * terms)
    again = r["dW"].clone()
    r2 = sbp.matmul_e4m3_columns(a["Yt8"], a["scales_t"], b["Yt8"], b["scales_t"], T, dW=again, accumulate=True, **kw)
    ok(r2)
    near("twice", host(again).reshape(want.shape), 2 * want, 2 * (steps + 1) * 2.0 ** -23 * terms)


# tables that are longer than a warp, with empty experts at both ends and in between
@pytest.mark.parametrize("T,E", [(1500, 33), (700, 64), (2100, 300), (900, 1023), (3000, 1024)])
def test_long_tables(sbp, T, E):
    g = np.random.default_rng(E)
    cuts = np.sort(np.concatenate([np.zeros(E // 5, dtype=np.int64), g.integers(0, T + 1, E - 1 - 2 * (E // 5)),
                                   np.full(E // 5, T)]))
    off = np.concatenate([[0], cuts, [T]])
    check_product(sbp, list(off), 136, 144, "fp32", E)
    d, nb = 136, sbp.token_blocks(T, E)
    x = wide(g, (T, d), "bf16")
    xt = X.columns(x, off)
    W = xt.shape[1]
    out = {}
    for tiles in (False, True):
        yt = torch.full((d, 128 * nb), 1.0, device="cuda").to(F8)
        out[tiles] = sbp.quant_e4m3_columns(dev(x, BF), offsets=dev(off, torch.int32), tiles=tiles, Yt8=yt)
        ok(out[tiles])
        q, s = X.quant(xt, 128 if tiles else 1)
        assert np.array_equal(host(yt)[:, :W], q) and (host(yt)[:, W:] == 1).all()
        assert np.array_equal(host(out[tiles]["scales_t"])[:, :W // 128], s.astype(np.float64))
    a, b = out[False], out[True]
    r = sbp.matmul_e4m3_columns(a["Yt8"], a["scales_t"], b["Yt8"], b["scales_t"], T, offsets=dev(off, torch.int32))
    ok(r)
    (qa, sa), (qb, sb) = X.quant(xt), X.quant(xt, 128)
    want, terms = X.matmul_columns(qa, sa, qb, sb, off)
    steps = 128 + (int(np.diff(off).max()) + 127) // 128 + 16
    near("dW", host(r["dW"]), want, steps * 2.0 ** -23 * terms)


def test_long_tables_many_rows(sbp):
    lens = np.random.default_rng(5).integers(0, 130, 130)
    check_product(sbp, [0] + list(np.cumsum(lens)), 1024, 512, "bf16", 6)


@pytest.mark.parametrize("at", [0, 1, 31, 32, 33, 64, 255, 256, 299, 300])
def test_long_tables_that_are_bad(sbp, at):
    off = torch.arange(301, dtype=torch.int32, device="cuda")
    x = torch.randn(300, 128, device="cuda")
    w = sbp.quant_e4m3_weight(torch.randn(300, 16, 128, device="cuda"))
    q = sbp.quant_e4m3(x)
    for value in (-1, 301):
        off[at] = value
        C = torch.full((300, 16), 5.0, device="cuda")
        yt = torch.zeros((128, 128 * sbp.token_blocks(300, 300)), device="cuda").to(F8)
        r = sbp.matmul_e4m3(q["Y8"], q["scales"], w["W8"], w["scales"], offsets=off, C=C)
        c = sbp.quant_e4m3_columns(x, offsets=off, Yt8=yt)
        torch.cuda.synchronize()
        assert int(r["status"].item()) == int(c["status"].item()) == sbp.ERR_SEQLENS
        assert (host(C) == 5).all() and (host(yt) == 0).all()


def test_nothing_to_do(sbp):
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    w = sbp.quant_e4m3_weight(torch.randn(4, 64, 128, device="cuda"))
    x = sbp.quant_e4m3(torch.empty(0, 128, device="cuda"))
    r = sbp.matmul_e4m3(x["Y8"], x["scales"], w["W8"], w["scales"], offsets=off)
    t = sbp.quant_e4m3_columns(torch.empty(0, 64, device="cuda"), offsets=off)
    s = sbp.quant_e4m3_columns(torch.empty(0, 128, device="cuda"), offsets=off, tiles=True)
    dW = sbp.matmul_e4m3_columns(t["Yt8"], t["scales_t"], s["Yt8"], s["scales_t"], 0, offsets=off)
    ok(r, t, s, dW)
    assert r["C"].shape == (0, 64) and (host(dW["dW"]) == 0).all()
    keep = torch.full((4, 64, 128), 3.0, device="cuda")
    ok(sbp.matmul_e4m3_columns(t["Yt8"], t["scales_t"], s["Yt8"], s["scales_t"], 0, offsets=off, dW=keep, accumulate=True))
    assert (host(keep) == 3).all()


@pytest.mark.parametrize("T,N,K", [(6, 256, 128), (2000, 4096, 128), (60, 8192, 2048)])
@pytest.mark.parametrize("bad", [[1, 2, 4], [0, 5, 4], [0, 2, 100000], [0, -1, 4], [-2, 2, 4]])
def test_bad_tables(sbp, bad, T, N, K):
    """A status, and nothing is read or written by a bad table."""
    off = torch.tensor(bad, dtype=torch.int32, device="cuda")
    x = torch.randn(T, K, device="cuda")
    w = sbp.quant_e4m3_weight(torch.randn(2, N, K, device="cuda"))
    q = sbp.quant_e4m3(x)
    C = torch.full((T, N), 5.0, device="cuda")
    r = sbp.matmul_e4m3(q["Y8"], q["scales"], w["W8"], w["scales"], offsets=off, C=C)
    nb = sbp.token_blocks(T, 2)
    yt = torch.zeros((K, 128 * nb), device="cuda").to(F8)
    c = sbp.quant_e4m3_columns(x, offsets=off, Yt8=yt)
    d = sbp.quant_e4m3_columns(x, offsets=off, tiles=True)
    dW = torch.full((2, K, K), 5.0, device="cuda")
    m = sbp.matmul_e4m3_columns(c["Yt8"], c["scales_t"], d["Yt8"], d["scales_t"], T, offsets=off, dW=dW)
    torch.cuda.synchronize()
    for v in (r, c, d, m):
        assert int(v["status"].item()) == sbp.ERR_SEQLENS
    assert (host(C) == 5).all() and (host(dW) == 5).all() and (host(yt) == 0).all()


def test_values_that_are_not_finite(sbp):
    """A NaN reaches its own row and column of the product, and no other."""
    g = np.random.default_rng(8)
    for T, N, K in ((5, 264, 256), (300, 264, 256), (1100, 4104, 256), (30, 24584, 1040)):
        a, sa, b, sb = operands(g, T, N, K, 1)
        A, B = dev(a, F8), dev(b[0], F8)
        clean = host(sbp.matmul_e4m3(A, dev(sa, F32), B, dev(sb[0], F32))["C"])
        A.view(torch.uint8)[3, 200] = 0x7f
        B.view(torch.uint8)[10, 5] = 0xff
        C = host(sbp.matmul_e4m3(A, dev(sa, F32), B, dev(sb[0], F32))["C"])
        nan = np.zeros(C.shape, dtype=bool)
        nan[3], nan[:, 10] = True, True
        assert np.isnan(C[nan]).all() and np.array_equal(C[~nan], clean[~nan])


def test_same_bits_and_neighbours(sbp):
    """The same call gives the same bits; a row's result does not depend on the other rows."""
    g = np.random.default_rng(11)
    a, sa, b, sb = operands(g, 1700, 4104, 656, 1)
    args = [dev(a, F8), dev(sa, F32), dev(b[0], F8), dev(sb[0], F32)]
    one, two = (sbp.matmul_e4m3(*args)["C"] for _ in range(2))
    assert torch.equal(one, two)
    split = [0, 700, 1700]
    bb = torch.stack([args[2].view(torch.uint8)] * 2).view(F8)
    part = sbp.matmul_e4m3(args[0], args[1], bb, torch.stack([args[3]] * 2),
                           offsets=torch.tensor(split, dtype=torch.int32, device="cuda"))["C"]
    assert torch.equal(part, one)


def test_elements_past_2_31(sbp):
    """Rows of arrays of more than 2^31 elements: the same bits as the same rows alone."""
    T, d, K = 524800, 4104, 128
    gen = torch.Generator(device="cuda").manual_seed(5)
    last = slice(T - 384, T)
    A, W = torch.randn(T, K, generator=gen, device="cuda").to(BF), torch.randn(d, K, generator=gen, device="cuda")
    a, w = sbp.quant_e4m3(A), sbp.quant_e4m3_weight(torch.cat([W, W[:8]]))     # (weights in sixteens)
    B8, sb = w["W8"][:d].contiguous(), w["scales"][:(d + 127) // 128].contiguous()
    r = sbp.matmul_e4m3(a["Y8"], a["scales"], B8, sb)
    ok(r)
    few = sbp.matmul_e4m3(a["Y8"][last].contiguous(), a["scales"][last].contiguous(), B8, sb, dtype=F32)["C"]
    C = r["C"]
    assert T * d > 2 ** 31
    near("C", host(C[last]), host(few), 2.0 ** -8 * np.abs(host(few)) + 1e-6)
    q, p = sbp.quant_e4m3(C), sbp.quant_e4m3(C[last].contiguous())
    assert torch.equal(q["Y8"][last].view(torch.uint8), p["Y8"].view(torch.uint8))
    assert torch.equal(q["scales"][last], p["scales"])
    del q
    for tiles in (False, True):
        t, u = sbp.quant_e4m3_columns(C, tiles=tiles), sbp.quant_e4m3_columns(C[last].contiguous(), tiles=tiles)
        assert torch.equal(t["Yt8"][:, -384:].contiguous().view(torch.uint8), u["Yt8"].view(torch.uint8))
        assert torch.equal(t["scales_t"][:, -3:], u["scales_t"])
        del t
    rows = torch.arange(T, device="cuda", dtype=torch.int32).flip(0).view(T // 2, 2).contiguous()
    X = C[:T // 2].contiguous()
    xs = sbp.expert_gather(X, rows)["Xs"]
    assert torch.equal(xs[:2], X[-1:].expand(2, d)) and torch.equal(xs[-2:], X[:1].expand(2, d))
    wt = torch.full((T // 2, 2), 0.5, device="cuda")
    assert torch.equal(sbp.expert_combine(xs, rows, wt)["Y"], X)
    dys = sbp.expert_combine_backward(X, xs, rows, wt)["dYs"]
    assert torch.equal(dys[-2:], (0.5 * X[:1].float()).to(BF).expand(2, d))


# ---------------------------------------------------------------- streams, graphs, a run

def test_other_stream_and_graph_follows_its_table(sbp):
    """The whole path captured once; replays follow new ids, inputs and weights."""
    T, k, E, d, f = 96, 2, 6, 256, 384
    torch.manual_seed(0)
    ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    x, dy = torch.zeros(T, d, device="cuda", dtype=BF), torch.zeros(T, f, device="cuda", dtype=BF)
    w = torch.zeros(E, f, d, device="cuda", dtype=BF)
    wt = torch.zeros(T, k, device="cuda")

    def step():
        o = sbp.expert_sort(ids, E)
        q = sbp.quant_e4m3(x)
        # unused rows are zeros, so that whole buffers compare
        s = sbp.expert_gather(q["Y8"], o["rows"], scales=q["scales"], Xs=torch.zeros(T * k, d, device="cuda").to(F8),
                              scales_s=torch.zeros(T * k, 2, device="cuda"))
        W = sbp.quant_e4m3_weight(w)
        C = sbp.matmul_e4m3(s["Xs"], s["scales"], W["W8"], W["scales"], offsets=o["offsets"],
                            C=torch.zeros(T * k, f, device="cuda", dtype=BF))
        y = sbp.expert_combine(C["C"], o["rows"], wt)
        b = sbp.expert_combine_backward(dy, C["C"], o["rows"], wt, dYs=torch.zeros(T * k, f, device="cuda", dtype=BF))
        g = sbp.quant_e4m3_columns(b["dYs"], offsets=o["offsets"], rows=True)
        dX = sbp.matmul_e4m3(g["Y8"], g["scales"], W["Wt8"], W["scales_t"], offsets=o["offsets"],
                             C=torch.zeros(T * k, d, device="cuda", dtype=BF))
        xs = sbp.expert_gather(x, o["rows"], Xs=torch.zeros(T * k, d, device="cuda", dtype=BF))["Xs"]
        xt = sbp.quant_e4m3_columns(xs, offsets=o["offsets"], tiles=True)
        dW = sbp.matmul_e4m3_columns(g["Yt8"], g["scales_t"], xt["Yt8"], xt["scales_t"], T * k, offsets=o["offsets"])
        dx = sbp.expert_gather_backward(dX["C"], o["rows"])["dX"]
        return [o["offsets"], o["rows"], y["Y"], b["dweights"], dW["dW"], dx], [r["status"] for r in (o, C, g, dX, xt, dW)]

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        ids.copy_(torch.randint(-1, E if seed % 2 else 2, (T, k), generator=g, device="cuda"))
        for t in (x, dy, w, wt):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        fill(1)
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, st = step()
    for seed in (2, 3, 4):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        assert all(int(s.item()) == 0 for s in st)
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.current_stream())
            want, _ = step()
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_streams_at_once(sbp):
    """Calls on streams given by name, each product's kernels among another's: the same bits."""
    T, E, k = 3000, 8, 2
    torch.manual_seed(3)
    ids = torch.randint(0, E, (T, k), device="cuda", dtype=torch.int32)
    x = torch.randn(T, 1024, device="cuda").to(BF)
    w = sbp.quant_e4m3_weight(torch.randn(E, 4096, 1024, device="cuda").to(BF))
    few = sbp.quant_e4m3(torch.randn(40, 1024, device="cuda").to(BF))
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda") * 5
    ones = torch.ones(T, k, device="cuda")

    def step(stream):
        o = sbp.expert_sort(ids, E, stream=stream)
        xs = sbp.expert_gather(x, o["rows"], stream=stream)["Xs"]
        q = sbp.quant_e4m3_columns(xs, offsets=o["offsets"], rows=True, stream=stream)
        t = sbp.quant_e4m3_columns(xs, offsets=o["offsets"], tiles=True, stream=stream)
        C = sbp.matmul_e4m3(q["Y8"], q["scales"], w["W8"], w["scales"], offsets=o["offsets"], stream=stream)
        c = sbp.matmul_e4m3(few["Y8"], few["scales"], w["W8"], w["scales"], offsets=off, dtype=F32, stream=stream)
        W = sbp.matmul_e4m3_columns(q["Yt8"], q["scales_t"], t["Yt8"], t["scales_t"], T * k, offsets=o["offsets"], stream=stream)
        y = sbp.expert_combine(C["C"], o["rows"], stream=stream)["Y"]
        e = sbp.quant_e4m3_expand(q["Y8"], q["scales"], stream=stream)["Y"]
        b = sbp.expert_combine_backward(y, C["C"], o["rows"], ones, stream=stream)
        return [o["rows"], C["C"], c["C"], W["dW"], y, e, b["dYs"], b["dweights"]], [v["status"] for v in (o, q, t, C, c, W)]

    want, _ = step(None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for s in streams:
            got.append(step(s))
    torch.cuda.synchronize()
    for out, status in got:
        assert all(int(v.item()) == 0 for v in status)
        for g, v in zip(out, want):
            assert torch.equal(g, v)


def test_run_of_an_expert_mlp(sbp):
    """Norm in 8 bits, sort, gather, both products around a gated activation, combine; then the
    gradients: every stage against the oracle on what the stage before it left."""
    T, k, E, d, f = 150, 2, 5, 256, 144
    g = np.random.default_rng(21)
    x = dev(normal(g, (T, d), "bf16"), BF)
    res = dev(normal(g, (T, d), "bf16"), BF)
    gamma = dev(1 + 0.2 * normal(g, (d,), "bf16"), BF)
    wu, wd = dev(normal(g, (E, 2 * f, d), "bf16", d ** -0.5), BF), dev(normal(g, (E, d, f), "bf16", f ** -0.5), BF)
    ids = draw_ids(g, T, k, E, 0.1)
    rows, slots, off = X.sort(ids, E)
    n = slots.size
    w = dev(g.random((T, k)), F32)

    nrm = sbp.rmsnorm_e4m3(x, gamma, 1e-6, residual=res)
    o = sbp.expert_sort(dev(ids, torch.int32), E)
    xs = sbp.expert_gather(nrm["Y8"], o["rows"], scales=nrm["scales"], n_rows=n)
    U, D = sbp.quant_e4m3_weight(wu), sbp.quant_e4m3_weight(wd)
    gu = sbp.matmul_e4m3(xs["Xs"], xs["scales"], U["W8"], U["scales"], offsets=o["offsets"])
    a, b = gu["C"].float().chunk(2, dim=1)
    h = (torch.nn.functional.silu(a) * b).to(BF)
    h8 = sbp.quant_e4m3(h)
    y = sbp.matmul_e4m3(h8["Y8"], h8["scales"], D["W8"], D["scales"], offsets=o["offsets"])
    out = sbp.expert_combine(y["C"], o["rows"], w, residual=nrm["R"])["Y"]
    ok(o, gu, y)

    steps = lambda K: (128 + (K + 127) // 128 + 16) * 2.0 ** -23
    us = [X.quant(host(wu)[e], 128) for e in range(E)]
    want, terms = X.matmul(X.gather(host(nrm["Y8"]), slots, k), X.gather(host(nrm["scales"]), slots, k),
                           np.stack([q for q, _ in us]), np.stack([s for _, s in us]), off)
    near("gate and up", host(gu["C"]), want, 2.0 ** -8 * np.abs(want) + steps(d) * terms)
    ds = [X.quant(host(wd)[e], 128) for e in range(E)]
    hq, hs = X.quant(host(h))
    want, terms = X.matmul(hq, hs, np.stack([q for q, _ in ds]), np.stack([s for _, s in ds]), off)
    near("down", host(y["C"]), want, 2.0 ** -8 * np.abs(want) + steps(f) * terms)
    want, terms = X.combine(host(y["C"]), rows, host(w), host(nrm["R"]))
    near("out", host(out), want, 2.0 ** -8 * np.abs(want) + (k + 1) * 2.0 ** -24 * terms)

    # gradients of the down projection and the routing weights
    dout = dev(normal(g, (T, d), "bf16"), BF)
    cb = sbp.expert_combine_backward(dout, y["C"], o["rows"], w)
    dys, dw, terms = X.combine_backward(host(dout), host(y["C"]), rows, host(w))
    near("dweights", host(cb["dweights"]), dw, (d + 16) * 2.0 ** -24 * terms)
    gq = sbp.quant_e4m3_columns(cb["dYs"], offsets=o["offsets"], rows=True)
    dh = sbp.matmul_e4m3(gq["Y8"], gq["scales"], D["Wt8"], D["scales_t"], offsets=o["offsets"])
    ht = sbp.quant_e4m3_columns(h, offsets=o["offsets"], tiles=True)
    dWd = sbp.matmul_e4m3_columns(gq["Yt8"], gq["scales_t"], ht["Yt8"], ht["scales_t"], n, offsets=o["offsets"])
    ok(gq, dh, ht, dWd)
    near("dYs", host(cb["dYs"]), dys, (2.0 ** -8 + 2.0 ** -24) * np.abs(dys))
    q, s = X.quant(host(cb["dYs"]))
    want, terms = X.matmul(q, s, np.stack([q.T for q, _ in ds]), np.stack([s.T for _, s in ds]), off)
    near("dH", host(dh["C"]), want, 2.0 ** -8 * np.abs(want) + steps(d) * terms)
    (qa, sa), (qb, sb) = X.quant(X.columns(host(cb["dYs"]), off)), X.quant(X.columns(host(h), off), 128)
    want, terms = X.matmul_columns(qa, sa, qb, sb, off)
    near("dWd", host(dWd["dW"]), want, steps(T) * terms)
