"""GPU tests of the expert calls where their rules change: no rows at all, the sizes at which one
kernel takes over from another, and what each of them does with values that are not finite."""
import numpy as np
import pytest

from oracle import experts as X

torch = pytest.importorskip("torch")
from test_gpu_experts import check_product, dev, host, near, wide  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def sbp():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from memory_efficient_exact_gb300 import _build
    _build.build_library()
    from memory_efficient_exact_gb300 import sbp as mod
    return mod


def status(r):
    torch.cuda.synchronize()
    return int(r["status"].item())


# ------------------------------------------------------------------------- no rows at all

def without_rows(sbp, off, E):
    """Every call that takes a table, with T = 0; dW [E, 24, 40] of sevens, written and added to."""
    f8 = lambda *s: torch.zeros(s, device="cuda").to(F8)
    f32 = lambda *s: torch.zeros(s, device="cuda")
    dW = torch.full((E, 24, 40), 7.0, device="cuda")
    added = dW.clone()
    nb = sbp.token_blocks(0, E)
    cols = [f8(24, 128 * nb), f32(24, nb), f8(40, 128 * nb), f32(1, nb)]
    results = [sbp.matmul_e4m3(f8(0, 32), f32(0, 1), f8(E, 64, 32), f32(E, 1, 1), offsets=off),
               sbp.quant_e4m3_columns(torch.zeros(0, 64, device="cuda"), offsets=off),
               sbp.quant_e4m3_columns(torch.zeros(0, 64, device="cuda"), offsets=off, tiles=True, rows=True),
               sbp.matmul_e4m3_columns(*cols, 0, offsets=off, dW=dW),
               sbp.matmul_e4m3_columns(*cols, 0, offsets=off, dW=added, accumulate=True)]
    return [status(r) for r in results], dW, added


@pytest.mark.parametrize("E,at,value", [(1, 0, 1), (1, 1, 5), (2, 1, -1), (2, 1, 5), (33, 33, 1), (40, 32, -7), (1024, 700, 3)])
def test_bad_table_without_rows(sbp, E, at, value):
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[at] = value
    got, dW, added = without_rows(sbp, off, E)
    assert got == [sbp.ERR_SEQLENS] * 5
    assert (dW == 7).all() and (added == 7).all()          # nothing is computed


@pytest.mark.parametrize("E", [1, 3, 32, 33, 1024])
def test_good_table_without_rows(sbp, E):
    got, dW, added = without_rows(sbp, torch.zeros(E + 1, dtype=torch.int32, device="cuda"), E)
    assert got == [sbp.OK] * 5
    assert (dW == 0).all() and (added == 7).all()


def test_captured_call_without_rows_follows_its_table(sbp):
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x = torch.zeros((8, 0), device="cuda").to(F8)
    s, t = torch.zeros((8, 0), device="cuda"), torch.zeros((1, 0), device="cuda")
    dW = torch.full((3, 8, 8), 7.0, device="cuda")
    st = torch.full((), 3, dtype=torch.int32, device="cuda")
    call = lambda: sbp.matmul_e4m3_columns(x, s, x, t, 0, offsets=off, dW=dW, status=st)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for bad in (True, False, True):
        off[2] = 1 if bad else 0
        dW.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == (sbp.ERR_SEQLENS if bad else sbp.OK) and (dW == (7 if bad else 0)).all()


# ------------------------------------------------------- every product kernel, known by name

FEW, SWAP, NARROW, WIDE = "few", "swap", "many_128", "many_256"


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kernel,lens,N,K", [
    (FEW, [5], 264, 272), (FEW, [1, 0, 2, 0], 136, 144), (FEW, [31], 2048, 4112),
    (SWAP, [20, 41, 7, 16], 8200, 1040), (SWAP, [20, 0, 64], 8200, 1040), (SWAP, [65, 0, 100, 2, 30, 8, 8, 70], 4104, 2064),
    (NARROW, [600], 2056, 272), (NARROW, [700], 2568, 1040), (NARROW, [501, 529], 1544, 400), (NARROW, [1500], 4104, 128),
    (WIDE, [600], 4104, 272), (WIDE, [300], 5128, 1040), (WIDE, [257, 0, 643, 300], 2568, 400), (WIDE, [1300], 1800, 144)])
def test_each_kernel(sbp, kernel, lens, N, K, dtype):
    off = np.concatenate([[0], np.cumsum(lens)]).tolist()
    check_product(sbp, off, N, K, dtype, N + K + len(lens))
    assert sbp.last_product_kernel() == kernel


@pytest.mark.parametrize("kernel,lens,N,K", [
    (FEW, [5], 128, 128), (FEW, [300, 0, 200, 400], 72, 136),
    (NARROW, [700], 520, 1544), (NARROW, [900, 0, 400], 264, 1032), (NARROW, [1500], 520, 1032),
    (WIDE, [300], 1032, 2568), (WIDE, [130, 0, 570], 520, 1544), (WIDE, [1], 1032, 2568)])
def test_each_kernel_of_columns(sbp, kernel, lens, N, K):
    """dW against the oracle; accumulate adds it to what is there, in one rounding to fp32."""
    g = np.random.default_rng(N + K)
    off = np.concatenate([[0], np.cumsum(lens)])
    T = int(off[-1])
    dy, x = wide(g, (T, N), "bf16") * 2.0 ** -14, wide(g, (T, K), "bf16")
    kw = dict(offsets=None if len(lens) == 1 else dev(off, torch.int32))
    a, b = sbp.quant_e4m3_columns(dev(dy, BF), **kw), sbp.quant_e4m3_columns(dev(x, BF), tiles=True, **kw)
    args = [a["Yt8"], a["scales_t"], b["Yt8"], b["scales_t"], T]
    r = sbp.matmul_e4m3_columns(*args, **kw)
    assert sbp.last_product_kernel() == kernel and status(r) == sbp.OK
    (qa, sa), (qb, sb) = X.quant(X.columns(dy, off)), X.quant(X.columns(x, off), 128)
    want, terms = X.matmul_columns(qa, sa, qb, sb, off)
    steps = 128 + max((n + 127) // 128 for n in lens) + 16
    near("dW", host(r["dW"]).reshape(want.shape), want, steps * 2.0 ** -23 * terms)
    before = torch.randn(r["dW"].shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    dW = before.clone()
    assert status(sbp.matmul_e4m3_columns(*args, dW=dW, accumulate=True, **kw)) == sbp.OK
    assert sbp.last_product_kernel() == kernel and torch.equal(dW, before + r["dW"])


def test_kernel_of_a_call_without_rows(sbp):
    f8 = lambda *s: torch.zeros(s, device="cuda").to(F8)
    f32 = lambda *s: torch.zeros(s, device="cuda")
    sbp.matmul_e4m3(f8(1, 32), f32(1, 1), f8(64, 32), f32(1, 1))
    assert sbp.last_product_kernel() == FEW
    sbp.matmul_e4m3(f8(0, 32), f32(0, 1), f8(64, 32), f32(1, 1))
    assert sbp.last_product_kernel() == "none"


# ----------------------------------------------------- where one kernel takes over from another

@pytest.mark.parametrize("rows,E,N,K", [(1, 8, 4096, 4096), (2, 8, 4096, 4096), (1, 64, 4096, 2560), (2, 64, 4096, 2560),
                                        (4, 64, 4096, 2560), (1, 256, 2048, 2048), (4, 256, 2048, 2048)])
def test_fewer_rows_than_experts(sbp, rows, E, N, K):
    """A token's rows make no more units than there are rows, however long the table is."""
    lens = np.zeros(E, dtype=np.int64)
    lens[np.arange(rows) * 37 % E] += 1
    off = np.concatenate([[0], np.cumsum(lens)])
    byte = lambda *s: torch.full(s, 0x38, dtype=torch.uint8, device="cuda").view(F8)      # ones
    f32 = lambda *s: torch.ones(s, device="cuda")
    r = sbp.matmul_e4m3(byte(rows, K), f32(rows, K // 128), byte(E, N, K), f32(E, N // 128, K // 128), offsets=dev(off, torch.int32))
    assert sbp.last_product_kernel() == FEW and status(r) == sbp.OK and (host(r["C"]) == K).all()


@pytest.mark.parametrize("kernel,lens,N,K", [
    (NARROW, [48], 4096, 4096), (NARROW, [64], 4096, 4096), (NARROW, [128], 4096, 4096), (FEW, [32], 4096, 4096),
    (FEW, [1] * 4 + [0] * 4, 4096, 4096), (FEW, [1] * 8, 4096, 4096), (SWAP, [16] * 8, 4096, 4096), (SWAP, [32], 24576, 4096),
    (SWAP, [2000], 256, 256)])
def test_kernel_that_measures_least(sbp, kernel, lens, N, K):
    T, E = sum(lens), len(lens)
    lead, off = ((), None) if E == 1 else ((E,), dev(np.concatenate([[0], np.cumsum(lens)]), torch.int32))
    byte = lambda *s: torch.full(s, 0x38, dtype=torch.uint8, device="cuda").view(F8)
    f32 = lambda *s: torch.ones(s, device="cuda")
    r = sbp.matmul_e4m3(byte(T, K), f32(T, K // 128), byte(*lead, N, K), f32(*lead, N // 128, K // 128), offsets=off)
    assert sbp.last_product_kernel() == kernel and status(r) == sbp.OK and (host(r["C"]) == K).all()


@pytest.mark.parametrize("kernel,lens,N,K", [(NARROW, [128], 1024, 1024), (FEW, [1000], 512, 512), (NARROW, [30] * 32, 128, 256)])
def test_kernel_of_columns_that_measures_least(sbp, kernel, lens, N, K):
    T, E = sum(lens), len(lens)
    off = None if E == 1 else dev(np.concatenate([[0], np.cumsum(lens)]), torch.int32)
    a = sbp.quant_e4m3_columns(torch.ones(T, N, device="cuda"), offsets=off)
    b = sbp.quant_e4m3_columns(torch.ones(T, K, device="cuda"), offsets=off, tiles=True)
    r = sbp.matmul_e4m3_columns(a["Yt8"], a["scales_t"], b["Yt8"], b["scales_t"], T, offsets=off)
    assert sbp.last_product_kernel() == kernel and status(r) == sbp.OK
    # the scale fl(1 / 448) and its inverse are off by half a step of fp32 each, twice; sums of 448^2 n are exact
    near("dW", host(r["dW"]).reshape(E, -1), np.array(lens, dtype=np.float64)[:, None], 2.0 ** -20 * np.array(lens)[:, None])


@pytest.mark.parametrize("E,blocks,launches", [(64, 1, 1), (64, 2, 2), (64, 64, 2), (8, 96, 2), (300, 127, 2), (64, 128, 3), (384, 128, 3),
                                               (512, 95, 2), (512, 96, 3), (1024, 47, 2), (1024, 48, 3)])
def test_sort_sums_counts_once_where_that_is_shorter(sbp, E, blocks, launches):
    ids = np.random.default_rng(E + blocks).integers(-1, E, (2048 * blocks - 5, 1))
    r = sbp.expert_sort(dev(ids, torch.int32), E)
    assert sbp.last_launch_count() == launches and status(r) == sbp.OK
    n = int((ids >= 0).sum())
    assert np.array_equal(host(r["slots"])[:n], np.argsort(np.where(ids < 0, E, ids).reshape(-1), kind="stable")[:n])
    assert np.array_equal(host(r["offsets"]), np.concatenate([[0], np.cumsum(np.bincount(ids[ids >= 0], minlength=E))]))
    rows = np.full(ids.size, -1)
    rows[host(r["slots"])[:n].astype(np.int64)] = np.arange(n)
    assert np.array_equal(host(r["rows"]).reshape(-1), rows)


# -------------------------------------------------------------- values that are not ordinary

def strange(dtype):
    """[300, 264] values: a NaN, an infinity, subnormals, the type's largest and a column of NaN, each
    in a tile of its own and several of them apart; the places of the NaNs and the infinities."""
    big, tiny = (3.3895314e38, 2.0 ** -133) if dtype == BF else (3.4028235e38, 2.0 ** -149)
    x = np.random.default_rng(4).standard_normal((300, 264)).astype(np.float32)
    x = torch.from_numpy(x).to(dtype).float().numpy()
    nan, inf = np.zeros(x.shape, dtype=bool), np.zeros(x.shape, dtype=bool)
    nan[5, 7] = nan[5, 8] = nan[127, 127] = True       # in the first tile
    nan[:128, 140] = True                              # a column's whole block
    nan[200, 128:256] = True                           # a row's whole block
    inf[130, 3] = inf[299, 263] = True
    x[256:300, 0:128] = tiny                           # a tile of subnormals
    x[256:300, 128:256] = 0
    x[299, 130] = -tiny * 3
    x[140, 260] = -big
    x[inf] = np.inf
    x[130, 3] = -np.inf
    return x, nan, inf


def same_but_for(q, s, nan, inf, rows, cols, want_q, want_s):
    """Scales and values of blocks of rows x cols: those of the array with its NaNs as zeros; NaNs where
    they were; blocks with an infinity stand for NaN."""
    for i in range(0, nan.shape[0], rows):
        for j in range(0, nan.shape[1], cols):
            at = np.s_[i:i + rows, j:j + cols]
            sq = s[i // rows, j // cols]
            if inf[at].any():
                with np.errstate(invalid="ignore"):
                    assert np.isinf(sq) and np.isnan(q[at] * sq).all()
                continue
            assert sq == want_s[i // rows, j // cols], (i, j)
            assert np.isnan(q[at][nan[at]]).all() and np.array_equal(q[at][~nan[at]], want_q[at][~nan[at]]), (i, j)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantisers_with_strange_values(sbp, dtype):
    x, nan, inf = strange(dtype)
    plain = np.where(nan | inf, np.float32(0), x)
    t = dev(np.where(nan, np.float32(np.nan), x), dtype)
    assert torch.equal(t[~torch.from_numpy(nan).cuda()], dev(x, dtype)[~torch.from_numpy(nan).cuda()])
    r = sbp.quant_e4m3(t)
    same_but_for(host(r["Y8"]), host(r["scales"]), nan, inf, 1, 128, *X.quant(plain))
    off = [0, 300]
    xt = lambda a: X.columns(a, off)
    pad = lambda m: np.pad(m, ((0, 84), (0, 0))).T
    for tiles in (False, True):
        for rows in (False, True):
            c = sbp.quant_e4m3_columns(t, tiles=tiles, rows=rows)
            assert status(c) == sbp.OK
            same_but_for(host(c["Yt8"]), host(c["scales_t"]), pad(nan), pad(inf), 128 if tiles else 1, 128,
                         *X.quant(xt(plain), 128 if tiles else 1))
            if rows:
                same_but_for(host(c["Y8"]), host(c["scales"]), nan, inf, 1, 128, *X.quant(plain))
    w = sbp.quant_e4m3_weight(t[:288, :256].contiguous())
    at = np.s_[:288, :256]
    want_q, want_s = X.quant(plain[at], 128)
    same_but_for(host(w["W8"]), host(w["scales"]), nan[at], inf[at], 128, 128, want_q, want_s)
    same_but_for(host(w["Wt8"]), host(w["scales_t"]), nan[at].T, inf[at].T, 128, 128, want_q.T, want_s.T)
    e = host(sbp.quant_e4m3_expand(w["W8"], w["scales"], F32, tiles=True)["Y"])
    with np.errstate(invalid="ignore"):
        v = host(w["W8"]) * np.repeat(np.repeat(host(w["scales"]), 128, 0)[:288], 128, 1)
    assert np.array_equal(np.isnan(e), np.isnan(v))
    near("expand", e[~np.isnan(v)], v[~np.isnan(v)], 2.0 ** -24 * np.abs(v[~np.isnan(v)]) + 2.0 ** -150)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_weights_of_dropped_slots_are_not_read(sbp, dtype):
    g = torch.Generator(device="cuda").manual_seed(2)
    T, k, E, d = 33, 3, 5, 136
    ids = torch.randint(-1, E, (T, k), generator=g, device="cuda").int()
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    o = sbp.expert_sort(ids, E)
    ys, dy, w = n(T * k, d).to(dtype), n(T, d).to(dtype), n(T, k)
    junk = torch.where(ids < 0, torch.full_like(w, float("nan")), w)
    zero = torch.where(ids < 0, torch.zeros_like(w), w)
    assert torch.equal(sbp.expert_combine(ys, o["rows"], junk)["Y"], sbp.expert_combine(ys, o["rows"], zero)["Y"])
    back = [sbp.expert_combine_backward(dy, ys, o["rows"], v, dYs=torch.zeros_like(ys)) for v in (junk, zero)]
    assert all(torch.equal(back[0][key], back[1][key]) for key in ("dYs", "dweights"))
    assert (back[0]["dweights"][ids < 0] == 0).all() and torch.isfinite(back[0]["dYs"].float()).all()


@pytest.mark.parametrize("kernel,lens,N,K", [(FEW, [300, 0, 200, 400], 72, 136), (NARROW, [900, 0, 400], 264, 1032), (WIDE, [130, 0, 570], 520, 1544)])
def test_nan_in_columns(sbp, kernel, lens, N, K):
    """A NaN among an expert's tokens reaches its own row or column of that expert's dW, and no other."""
    g = np.random.default_rng(N)
    off, T = dev(np.concatenate([[0], np.cumsum(lens)]), torch.int32), sum(lens)
    dy, x = dev(g.standard_normal((T, N)), BF), dev(g.standard_normal((T, K)), BF)
    def run():
        a, b = sbp.quant_e4m3_columns(dy, offsets=off), sbp.quant_e4m3_columns(x, offsets=off, tiles=True)
        r = sbp.matmul_e4m3_columns(a["Yt8"], a["scales_t"], b["Yt8"], b["scales_t"], T, offsets=off)
        assert sbp.last_product_kernel() == kernel and status(r) == sbp.OK
        return r["dW"]
    for t in (dy[0, 3], dy[lens[0], N - 1], x[lens[0] + 1, 9]):     # (one must not be its block's largest)
        t.zero_()
    clean = run()
    dy[0, 3], dy[lens[0], N - 1], x[lens[0] + 1, 9] = (float("nan"),) * 3
    got = run()
    nan = torch.zeros(clean.shape, dtype=torch.bool, device="cuda")
    e = [i for i, n in enumerate(lens) if n][1]
    nan[0, 3] = nan[e, N - 1] = True
    nan[e, :, 9] = True
    assert torch.isnan(got[nan]).all() and torch.equal(got[~nan], clean[~nan])
