"""GPU parity of the attention over packed documents against the float64 oracle.

Tolerances are element by element, from the rounding the kernels do (u = 2^-8 is bf16's
largest relative rounding error, half a step):
  O     u |O| for its own rounding, u sum_j P |V| for P's, and 2^-11 of that sum for the fp32
        scores and exponentials (score errors below 2^-12 at these sizes);
  lse   2^-12 (the scores' fp32 sums) and 2^-20 of its value;
  dQ, dK, dV  u of the value, and the oracle's bounds for P and dS in bf16 (see there).
The backward is compared at the exact O and the lse it was given.  Its D = dO . O is that of the O
it was given, off by O's bound, but for units of 256 queries that see up to three blocks of 128
keys, which have it from P and dP.
"""
import numpy as np
import pytest

from oracle import sublayer as S
from memory_efficient_exact_gb300 import inputs as I

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(scope="module")
def sbp():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from memory_efficient_exact_gb300 import _build
    _build.build_library()
    from memory_efficient_exact_gb300 import sbp as mod
    return mod


def dev(x, dt=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(dt).contiguous()


def host(t):
    return t.detach().double().cpu().numpy()


def make(H, Hkv, T, hd, seed, gain=1.0):
    g = np.random.default_rng(seed)
    r = lambda n, k=1.0: I.round_bf16((k * g.standard_normal((n, T, hd))).astype(np.float32))
    return dict(Q=r(H, gain), K=r(Hkv), V=r(Hkv), dO=r(H))


def options(H, lens, prefix, softcap, alibi):
    cu = None if lens is None else np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    sl = None
    if alibi:
        sl = (2.0 ** (-8.0 * np.arange(1, H + 1) / H)).astype(np.float32)
    kw = dict(softcap=softcap)
    if cu is not None:
        kw["cu_seqlens"] = dev(cu, torch.int32)
    if prefix is not None:
        kw["prefix_lens"] = dev(np.asarray(prefix, np.int32), torch.int32)
    if sl is not None:
        kw["slopes"] = dev(sl, torch.float32)
    return cu, sl, kw


def near(name, got, want, bound):
    err = np.abs(got - want)
    assert np.all(err <= bound), (name, float((err / bound).max()), np.argwhere(err > bound)[:4].tolist())


def check(sbp, x, kw, cu, prefix, sl, scale):
    H, T, hd = x["Q"].shape
    see = S.visible(T, cu, prefix)
    a = {k: dev(v) for k, v in x.items()}
    f = sbp.attn_packed(a["Q"], a["K"], a["V"], scale, **kw)
    b = sbp.attn_packed_backward(a["Q"], a["K"], a["V"], f["O"], a["dO"], f["lse"], scale, **kw)
    torch.cuda.synchronize()
    sbp.check_status(f["status"])
    sbp.check_status(b["status"])
    cap = kw["softcap"]
    want = S.attention(x["Q"], x["K"], x["V"], see, scale, cap, sl)
    O, lse = host(f["O"]), host(f["lse"])
    near("O", O, want["O"], U * np.abs(want["O"]) + (U + 2.0 ** -11) * want["size"])
    some = see.any(axis=1)
    assert np.all(np.isneginf(lse[:, ~some])) and np.all(O[:, ~some] == 0)
    near("lse", lse[:, some], want["lse"][:, some], 2.0 ** -12 + 2.0 ** -20 * np.abs(want["lse"][:, some]))
    errO = U * np.abs(want["O"]) + (U + 2.0 ** -11) * want["size"]
    for q in range(0, T, 256):
        keys = np.flatnonzero(see[q:q + 256].any(axis=0))
        if len(keys) == 0 or keys[-1] // 128 - keys[0] // 128 < 3:
            errO[:, q:q + 256] = 0.0
    g = S.attention_backward(x["Q"], x["K"], x["V"], want["O"], x["dO"], lse, see, scale, cap, sl, errO)
    for k in "QKV":
        near("d" + k, host(b["d" + k]), g["d" + k], U * np.abs(g["d" + k]) + g["b" + k])
    seen = see.any(axis=0)
    assert np.all(host(b["dQ"])[:, ~some] == 0)
    assert np.all(host(b["dK"])[:, ~seen] == 0) and np.all(host(b["dV"])[:, ~seen] == 0)


# one token; lengths around the 64-key, 128-row and 256-row tiles; one document
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 400])
def test_one_document(sbp, T):
    x = make(2, 1, T, 128, seed=T)
    cu, sl, kw = options(2, None, None, 0.0, False)
    check(sbp, x, kw, cu, None, sl, 128 ** -0.5)


# documents that begin and end inside tiles, empty ones first, between and last, single
# tokens, padding behind them, grouped heads
@pytest.mark.parametrize("T,lens", [(300, [100, 0, 1, 150, 49]), (520, [0, 130, 126, 1, 1, 200]), (384, [128, 128, 128]),
                                    (300, [300, 0]), (257, [1]), (260, [0]), (700, [5] * 100), (513, [256, 257])])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (6, 2)])
def test_documents(sbp, T, lens, H, Hkv):
    x = make(H, Hkv, T, 64, seed=T + H)
    cu, sl, kw = options(H, lens, None, 0.0, False)
    check(sbp, x, kw, cu, None, sl, 0.125)


# a prefix of none, part, all and more than its document; with and without documents
@pytest.mark.parametrize("T,lens,prefix", [(300, None, [140]), (300, [100, 120, 60], [0, 70, 500]), (200, None, [0]),
                                           (640, [600, 40], [600, 1])])
def test_prefix(sbp, T, lens, prefix):
    x = make(2, 1, T, 128, seed=T)
    cu, sl, kw = options(2, lens, prefix, 0.0, False)
    check(sbp, x, kw, cu, prefix, sl, 128 ** -0.5)


# caps that bind (scores of some 4 x the cap) and hardly bind; distance bias; both
@pytest.mark.parametrize("softcap,alibi,gain", [(50.0, False, 4.0), (2.0, False, 8.0), (0.0, True, 1.0), (15.0, True, 4.0)])
@pytest.mark.parametrize("prefix", [None, [20, 130, 0]])
def test_cap_and_bias(sbp, softcap, alibi, gain, prefix):
    x = make(4, 2, 330, 128, seed=9, gain=gain)
    cu, sl, kw = options(4, [90, 140, 80], prefix, softcap, alibi)
    check(sbp, x, kw, cu, prefix, sl, 128 ** -0.5)


# slopes below 0 favour far keys: by more than 2^127 for the first head
@pytest.mark.parametrize("softcap", [0.0, 15.0, 100.0])
@pytest.mark.parametrize("prefix", [None, [200, 0]])
def test_slopes_of_either_sign(sbp, softcap, prefix):
    x = make(4, 2, 420, 128, seed=10)
    cu, _, kw = options(4, [300, 100], prefix, softcap, False)
    sl = np.array([-0.5, 0.25, -0.03125, 0.0], np.float32)
    check(sbp, x, {**kw, "slopes": dev(sl, torch.float32)}, cu, prefix, sl, 128 ** -0.5)


@pytest.mark.parametrize("hd", [8, 16, 40, 64, 72, 80, 96, 120, 128])
def test_head_widths(sbp, hd):
    x = make(3, 1, 200, hd, seed=hd)
    cu, sl, kw = options(3, [120, 70], None, 0.0, False)
    check(sbp, x, kw, cu, None, sl, hd ** -0.5)


def test_more_units_than_pairs(sbp):
    # 48 heads of 3 units: every barrier crosses unit boundaries
    x = make(48, 8, 600, 128, seed=1)
    cu, sl, kw = options(48, [300, 290], None, 0.0, False)
    check(sbp, x, kw, cu, None, sl, 128 ** -0.5)


@pytest.mark.parametrize("softcap,alibi", [(30.0, False), (30.0, True), (0.0, True), (100.0, False)])
def test_more_units_than_pairs_of_every_kernel(sbp, softcap, alibi):
    # units of one, two, three and more blocks behind one another: score buffers and barriers
    # start a unit at any of their phases
    x = make(48, 8, 900, 64, seed=14, gain=2.0)
    cu, sl, kw = options(48, [40, 90, 300, 20, 400], None, softcap, alibi)
    check(sbp, x, kw, cu, None, sl, 0.125)


@pytest.mark.parametrize("docs,softcap", [([16] * 20, 30.0), ([16] * 20, 0.0), ([3, 1, 7, 40, 2, 90], 50.0), ([400], 30.0)])
def test_peaked_rows_keep_their_gradients(sbp, docs, softcap):
    # rows whose probability lies on few keys: P (dP - D) is far smaller than dP and D, so D has to
    # be better than bf16.  What is left are the roundings of dS and of the result to bf16, each
    # 2^-8 / sqrt(3) of the norm if all were as large as can be: less than 2^-8 together
    T, sc = sum(docs), 128 ** -0.5
    x = make(4, 2, T, 128, seed=12, gain=4.0)
    cu, _, kw = options(4, docs, None, softcap, False)
    see = S.visible(T, cu, None)
    a = {k: dev(v) for k, v in x.items()}
    f = sbp.attn_packed(a["Q"], a["K"], a["V"], sc, **kw)
    b = sbp.attn_packed_backward(a["Q"], a["K"], a["V"], f["O"], a["dO"], f["lse"], sc, **kw)
    want = S.attention(x["Q"], x["K"], x["V"], see, sc, softcap, None)
    g = S.attention_backward(x["Q"], x["K"], x["V"], want["O"], x["dO"], want["lse"], see, sc, softcap, None)
    for k in "QKV":
        e = np.linalg.norm(host(b["d" + k]) - g["d" + k]) / np.linalg.norm(g["d" + k])
        assert e < 2.0 ** -8, (k, e)

def _document(x, a, b):
    """The operands of the document [a, b) alone."""
    return {k: v[:, a:b] for k, v in x.items()}


@pytest.mark.parametrize("lens,prefix,short", [
    ([2000] + [16] * 16, None, range(1, 4)),                        # behind a long one, in its last unit
    ([16] * 10 + [1500], [0] * 10 + [1500], range(10)),             # before one whose prefix reaches far ahead
    ([700, 128, 300, 120, 900], [0, 128, 0, 120, 900], [1, 3]),     # between, over the ends of the units of 256 rows
    ([1300, 40, 7, 1, 90, 128, 1200], None, [1, 2, 3, 4, 5])])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
def test_short_documents_beside_long_ones_keep_their_gradients(sbp, lens, prefix, short, softcap):
    # as test_peaked_rows_keep_their_gradients, whatever shares the unit with a short document
    T, sc = sum(lens) + 30, 128 ** -0.5
    x = make(4, 2, T, 128, seed=15, gain=4.0)
    cu, _, kw = options(4, lens, prefix, softcap, False)
    a = {k: dev(v) for k, v in x.items()}
    f = sbp.attn_packed(a["Q"], a["K"], a["V"], sc, **kw)
    b = sbp.attn_packed_backward(a["Q"], a["K"], a["V"], f["O"], a["dO"], f["lse"], sc, **kw)
    torch.cuda.synchronize()
    sbp.check_status(b["status"])
    err, size = dict.fromkeys("QKV", 0.0), dict.fromkeys("QKV", 0.0)
    for s in short:
        d = _document(x, cu[s], cu[s + 1])
        see = S.visible(lens[s], None, None if prefix is None else [prefix[s]])
        w = S.attention(d["Q"], d["K"], d["V"], see, sc, softcap, None)
        g = S.attention_backward(d["Q"], d["K"], d["V"], w["O"], d["dO"], w["lse"], see, sc, softcap, None)
        for k in "QKV":
            got = host(b["d" + k])[:, cu[s]:cu[s + 1]]
            err[k] += np.sum((got - g["d" + k]) ** 2)
            size[k] += np.sum(g["d" + k] ** 2)
    for k in "QKV":
        e = np.sqrt(err[k] / size[k])
        assert e < 2.0 ** -8, (k, e)


@pytest.mark.parametrize("gain,shift,softcap,alibi", [(4.0, 0.0, 50.0, False), (4.0, 0.0, 0.0, True), (3.0, 0.0, 30.0, True),
                                                      (1.0, 4.0, 0.0, False), (1.0, 0.0, 0.0, False)])
@pytest.mark.parametrize("hd", [64, 128])
def test_rows_of_long_documents_keep_their_gradients(sbp, gain, shift, softcap, alibi, hd):
    # rows that few of many keys hold, and values with a common part, which the O they leave shows and
    # dP - D does not: D is not that of the rounded O there.  Then dQ and dK have the roundings of dS
    # and of the result to bf16, 2^-8 / sqrt(3) of the norm each if all were as large as can be
    H, Hkv, T, sc = 4, 2, 1900, hd ** -0.5
    x = make(H, Hkv, T, hd, seed=22, gain=gain)
    x["V"] = I.round_bf16((x["V"] + shift).astype(np.float32))
    cu, sl, kw = options(H, [1100, 760], None, softcap, alibi)
    if alibi:
        sl = np.array([0.7, 0.25, 0.05, 0.001], np.float32)
        kw["slopes"] = dev(sl, torch.float32)
    a = {k: dev(v) for k, v in x.items()}
    f = sbp.attn_packed(a["Q"], a["K"], a["V"], sc, **kw)
    b = sbp.attn_packed_backward(a["Q"], a["K"], a["V"], f["O"], a["dO"], f["lse"], sc, **kw)
    torch.cuda.synchronize()
    sbp.check_status(b["status"])
    for s in range(2):
        d, see = _document(x, cu[s], cu[s + 1]), np.tril(np.ones((cu[s + 1] - cu[s],) * 2, dtype=bool))
        w = S.attention(d["Q"], d["K"], d["V"], see, sc, softcap, sl)
        g = S.attention_backward(d["Q"], d["K"], d["V"], w["O"], d["dO"], w["lse"], see, sc, softcap, sl)
        for k in "QK":
            for h in range(H if k == "Q" else Hkv):
                got, want = host(b["d" + k])[h, cu[s]:cu[s + 1]], g["d" + k][h]
                e = np.linalg.norm(got - want) / np.linalg.norm(want)
                assert e < 2.0 ** -8 * np.sqrt(2.0 / 3.0), (s, k, h, e)


@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_distances_of_far_rows(sbp, softcap):
    # rows past 2^24, which fp32 no longer tells from their neighbours: the bias goes by i - j
    n, base = 300, 2 ** 24 + 1
    T = base + n
    cu = np.concatenate([np.arange(0, 2 ** 24 + 1, 256), [base, T]]).astype(np.int32)
    x = make(1, 1, n, 8, seed=16)
    sl = np.array([1.0], np.float32)
    a = {k: torch.zeros((1, T, 8), dtype=torch.bfloat16, device="cuda") for k in x}
    for k in x:
        a[k][:, base:] = dev(x[k])
    kw = dict(cu_seqlens=dev(cu, torch.int32), slopes=dev(sl, torch.float32), softcap=softcap)
    f = sbp.attn_packed(a["Q"], a["K"], a["V"], 0.3, **kw)
    b = sbp.attn_packed_backward(a["Q"], a["K"], a["V"], f["O"], a["dO"], f["lse"], 0.3, **kw)
    torch.cuda.synchronize()
    sbp.check_status(f["status"])
    sbp.check_status(b["status"])
    see = S.visible(n)
    want = S.attention(x["Q"], x["K"], x["V"], see, 0.3, softcap, sl)
    lse = host(f["lse"][:, base:])
    near("O", host(f["O"][:, base:]), want["O"], U * np.abs(want["O"]) + (U + 2.0 ** -11) * want["size"])
    near("lse", lse, want["lse"], 2.0 ** -12 + 2.0 ** -20 * np.abs(want["lse"]))
    errO = U * np.abs(want["O"]) + (U + 2.0 ** -11) * want["size"]
    g = S.attention_backward(x["Q"], x["K"], x["V"], want["O"], x["dO"], lse, see, 0.3, softcap, sl, errO)
    for k in "QKV":
        near("d" + k, host(b["d" + k][:, base:]), g["d" + k], U * np.abs(g["d" + k]) + g["b" + k])


def test_units_without_a_token(sbp):
    # most units are padding alone: their rows are cleared between and behind the others
    x = make(48, 8, 1100, 64, seed=11)
    cu, sl, kw = options(48, [130, 170], None, 0.0, False)
    check(sbp, x, kw, cu, None, sl, 0.125)


def test_running_maximum_is_raised(sbp):
    # scores that grow along the keys by far more than the 2^8 the maximum may lag behind
    x = make(1, 1, 600, 128, seed=2)
    x["K"] = I.round_bf16((x["K"] * np.linspace(0.05, 6.0, 600)[None, :, None]).astype(np.float32))
    cu, sl, kw = options(1, None, None, 0.0, False)
    check(sbp, x, kw, cu, None, sl, 0.25)


@pytest.mark.parametrize("softcap,alibi", [(50.0, False), (50.0, True), (30.0, False), (51.0, False), (0.0, False)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_values_at_the_ends_of_their_range(sbp, softcap, alibi, sign):
    # rows whose scores are all at the cap, or all at its negative (without one: all at +-60), and V as
    # large and as small as the header allows (2^54 / T, 2^111 / T; 2^-30: the sums lose 2^-53)
    T, fixed = 512, 0.0 < softcap <= 50.0
    x = make(2, 1, T, 64, seed=18)
    x["Q"] = np.full_like(x["Q"], sign)
    x["K"] = np.full_like(x["K"], 60.0 if softcap == 0 else 4096.0)     # scale 1/64: scores of +-60, +-4096
    for k in (2.0 ** (45 if fixed else 102), 2.0 ** -30):
        y = dict(x, V=I.round_bf16((np.clip(x["V"], -1, 1) * k).astype(np.float32)))
        cu, sl, kw = options(2, [300, 212], None, softcap, alibi)
        a = {n: dev(v) for n, v in y.items()}
        f = sbp.attn_packed(a["Q"], a["K"], a["V"], 1.0 / 64, **kw)
        torch.cuda.synchronize()
        sbp.check_status(f["status"])
        want = S.attention(y["Q"], y["K"], y["V"], S.visible(T, cu), 1.0 / 64, softcap, sl)
        near("O", host(f["O"]), want["O"], U * np.abs(want["O"]) + (U + 2.0 ** -11) * want["size"] + 2.0 ** -53)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_padding_may_hold_anything(sbp, bad):
    H, Hkv, T, n = 4, 2, 400, 333
    x = make(H, Hkv, T, 64, seed=3)
    a = {k: dev(v) for k, v in x.items()}
    cu = dev(np.array([0, 200, n], np.int32), torch.int32)

    def run():
        f = sbp.attn_packed(a["Q"], a["K"], a["V"], 0.125, cu_seqlens=cu, softcap=20.0)
        O, lse = f["O"].clone(), f["lse"].clone()
        O[:, n:] = bad
        lse[:, n:] = bad
        b = sbp.attn_packed_backward(a["Q"], a["K"], a["V"], O, a["dO"], lse, 0.125, cu_seqlens=cu, softcap=20.0)
        return [f["O"], f["lse"], b["dQ"], b["dK"], b["dV"]]

    clean = run()
    for k in a:
        a[k][:, n:] = bad
    dirty = run()
    torch.cuda.synchronize()
    for c, d in zip(clean, dirty):
        assert torch.equal(c, d)
    assert torch.all(dirty[1][:, n:] == -float("inf")) and all(torch.all(t[:, n:] == 0) for t in dirty[:1] + dirty[2:])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("softcap,alibi", [(0.0, False), (0.0, True), (30.0, True), (90.0, True)])
@pytest.mark.parametrize("hd,lens", [(128, [130, 3, 480]), (72, [77])])
def test_padding_of_every_kernel_may_hold_anything(sbp, bad, softcap, alibi, hd, lens):
    # an odd end inside a block of 128, long and short units, padding that fills whole units
    H, Hkv, T, n = 4, 2, 1000, sum(lens)
    a = {k: dev(v) for k, v in make(H, Hkv, T, hd, seed=13).items()}
    _, _, kw = options(H, lens, None, softcap, alibi)

    def run():
        f = sbp.attn_packed(a["Q"], a["K"], a["V"], 0.1, **kw)
        b = sbp.attn_packed_backward(a["Q"], a["K"], a["V"], f["O"], a["dO"], f["lse"], 0.1, **kw)
        return [f["O"], f["lse"], b["dQ"], b["dK"], b["dV"]]

    clean = run()
    for k in a:
        a[k][:, n:] = bad
    dirty = run()
    torch.cuda.synchronize()
    for c, d in zip(clean, dirty):
        assert torch.equal(c, d)
    assert all(torch.isfinite(t[:, :n]).all() for t in dirty)


def test_infinite_keys_of_another_document_stay_masked(sbp):
    # an infinite K makes infinite scores for other documents' queries in the same tile; they
    # are masked before the exponential (V, Q and dO are summed over, so they must be finite)
    x = make(1, 1, 100, 64, seed=4)
    a = {k: dev(v) for k, v in x.items()}
    cu = dev(np.array([0, 60, 100], np.int32), torch.int32)
    want = sbp.attn_packed(a["Q"], a["K"], a["V"], 0.125, cu_seqlens=cu)["O"][:, :60].clone()
    a["K"][:, 80] = float("inf")
    got = sbp.attn_packed(a["Q"], a["K"], a["V"], 0.125, cu_seqlens=cu)["O"][:, :60]
    assert torch.equal(want, got)


def _call(sbp, a, out, **kw):
    f = sbp.attn_packed(a["Q"], a["K"], a["V"], 0.125, O=out["O"], lse=out["lse"], **kw)
    b = sbp.attn_packed_backward(a["Q"], a["K"], a["V"], f["O"], a["dO"], f["lse"], 0.125, dQ=out["dQ"], dK=out["dK"],
                                 dV=out["dV"], **kw)
    return f["status"], b["status"]


def _outputs(a):
    n = lambda t: torch.full_like(t, 7.0)
    return dict(O=n(a["Q"]), lse=torch.full(a["Q"].shape[:2], 7.0, device="cuda"), dQ=n(a["Q"]), dK=n(a["K"]), dV=n(a["V"]))


def test_same_bits_on_a_stream_and_in_graphs(sbp):
    H, Hkv, T = 6, 2, 500
    a = {k: dev(v) for k, v in make(H, Hkv, T, 64, seed=5).items()}
    cu = dev(np.array([0, 210, 460], np.int32), torch.int32)
    ref = _outputs(a)
    _call(sbp, a, ref, cu_seqlens=cu)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = _outputs(a)
    side.wait_stream(torch.cuda.current_stream())
    _call(sbp, a, got, cu_seqlens=cu, stream=side)
    side.synchronize()
    assert all(torch.equal(ref[k], got[k]) for k in ref)

    # two captured graphs that share a workspace; the second follows a changed table
    ws = torch.empty(sbp.attn_packed_workspace_bytes(H, Hkv, T, 64), dtype=torch.uint8, device="cuda")
    outs, graphs = [_outputs(a), _outputs(a)], []
    tables = [cu.clone(), cu.clone()]
    for o, c in zip(outs, tables):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            st = _call(sbp, a, o, cu_seqlens=c, workspace=ws)
        graphs.append((g, st))
    tables[1].copy_(dev(np.array([0, 64, 500], np.int32), torch.int32))
    other = _outputs(a)
    _call(sbp, a, other, cu_seqlens=tables[1])
    for _ in range(2):
        for g, _st in graphs:
            g.replay()
    torch.cuda.synchronize()
    for want, got in ((ref, outs[0]), (other, outs[1])):
        assert all(torch.equal(want[k], got[k]) for k in want)
    for _, st in graphs:
        for s in st:
            sbp.check_status(s)


@pytest.mark.parametrize("softcap,alibi", [(0.0, False), (30.0, True)])
def test_smaller_workspaces(sbp, softcap, alibi):
    # a group's query heads shared out to one, some or as many sums of dK and dV as the workspace
    # holds, the change of head inside a unit with its slope among them; guard bytes behind it
    H, Hkv, T, hd = 16, 2, 600, 64
    x = make(H, Hkv, T, hd, seed=17)
    cu, sl, kw = options(H, [300, 5, 280], None, softcap, alibi)
    full, lean = sbp.attn_packed_workspace_bytes(H, Hkv, T, hd), sbp.attn_packed_workspace_bytes_lean(H, Hkv, T, hd)
    part = 2 * Hkv * T * hd * 4
    assert full == lean + 8 * part              # (T hd is a multiple of the regions' 256 bytes)
    see = S.visible(T, cu)
    a = {k: dev(v) for k, v in x.items()}
    want = S.attention(x["Q"], x["K"], x["V"], see, 0.125, softcap, sl)
    errO = U * np.abs(want["O"]) + (U + 2.0 ** -11) * want["size"]
    few = torch.full((sbp.attn_packed_forward_workspace_bytes(H, Hkv, T, hd) + 64,), 9, dtype=torch.uint8, device="cuda")
    f = sbp.attn_packed(a["Q"], a["K"], a["V"], 0.125, workspace=few[:-64], **kw)
    near("O", host(f["O"]), want["O"], U * np.abs(want["O"]) + (U + 2.0 ** -11) * want["size"])
    assert torch.all(few[-64:] == 9)
    for n in (full, full - 1, lean + 2 * part, lean + 2 * part - 1, lean, sbp.attn_packed_workspace_bytes(H, Hkv, 4 * T, hd)):
        ws = torch.full((n + 64,), 9, dtype=torch.uint8, device="cuda")
        b = sbp.attn_packed_backward(a["Q"], a["K"], a["V"], f["O"], a["dO"], f["lse"], 0.125, workspace=ws[:n], **kw)
        torch.cuda.synchronize()
        sbp.check_status(b["status"])
        assert torch.all(ws[n:] == 9)
        g = S.attention_backward(x["Q"], x["K"], x["V"], want["O"], x["dO"], host(f["lse"]), see, 0.125, softcap, sl, errO)
        for k in "QKV":
            near(f"d{k} in {n}", host(b["d" + k]), g["d" + k], U * np.abs(g["d" + k]) + g["b" + k])
    with pytest.raises(sbp.SbpError):
        sbp.attn_packed_backward(a["Q"], a["K"], a["V"], f["O"], a["dO"], f["lse"], 0.125, workspace=ws[:lean - 1], **kw)


def test_one_workspace_for_shorter_batches(sbp):
    # sized for the longest, where a unit takes a group's heads together, used where it would not
    H, Hkv, hd = 32, 8, 64
    ws = torch.empty(sbp.attn_packed_workspace_bytes(H, Hkv, 5120, hd), dtype=torch.uint8, device="cuda")
    for T in (5120, 700, 40):
        assert T == 5120 or ws.numel() < sbp.attn_packed_workspace_bytes(H, Hkv, 2560, hd)
        x = make(H, Hkv, T, hd, seed=T) if T < 5120 else {k: np.zeros((H if k in "QdO" else Hkv, T, hd), np.float32) for k in ("Q", "K", "V", "dO")}
        a = {k: dev(v) for k, v in x.items()}
        f = sbp.attn_packed(a["Q"], a["K"], a["V"], 0.125, workspace=ws)
        b = sbp.attn_packed_backward(a["Q"], a["K"], a["V"], f["O"], a["dO"], f["lse"], 0.125, workspace=ws)
        torch.cuda.synchronize()
        sbp.check_status(b["status"])
        c = sbp.attn_packed_backward(a["Q"], a["K"], a["V"], f["O"], a["dO"], f["lse"], 0.125)
        # the same sums, in fp32 in another order, each rounded to bf16 once
        for k in ("dQ", "dK", "dV"):
            d = (b[k].double() - c[k].double()).abs()
            assert torch.all(d <= 2 * U * c[k].double().abs() + 2.0 ** -16 * c[k].double().abs().max()), (T, k)


def test_calls_on_two_streams_at_once(sbp):
    a = {k: dev(v) for k, v in make(16, 4, 900, 128, seed=6).items()}
    ref = _outputs(a)
    _call(sbp, a, ref)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], [_outputs(a) for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for s, o in zip(streams, outs):
            _call(sbp, a, o, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(ref[k], o[k]) for k in ref)


@pytest.mark.parametrize("cu", [[1, 50, 100], [0, 60, 50], [0, 50, 101], [0, -3, 100], [0, 1 << 30, 100]])
def test_bad_tables_set_the_status(sbp, cu):
    a = {k: dev(v) for k, v in make(2, 1, 100, 64, seed=7).items()}
    for st in _call(sbp, a, _outputs(a), cu_seqlens=dev(np.array(cu, np.int32), torch.int32)):
        torch.cuda.synchronize()
        with pytest.raises(sbp.SbpError) as e:
            sbp.check_status(st)
        assert e.value.code == sbp.ERR_SEQLENS
    good = dev(np.array([0, 50, 100], np.int32), torch.int32)
    for st in _call(sbp, a, _outputs(a), cu_seqlens=good, prefix_lens=dev(np.array([3, -1], np.int32), torch.int32)):
        torch.cuda.synchronize()
        assert int(st) == sbp.ERR_SEQLENS
    for st in _call(sbp, a, _outputs(a), cu_seqlens=good):
        sbp.check_status(st)


def test_python_refusals(sbp):
    a = {k: dev(v) for k, v in make(2, 1, 64, 64, seed=8).items()}
    Q, K, V = a["Q"], a["K"], a["V"]
    with pytest.raises(ValueError):
        sbp.attn_packed(Q.transpose(0, 1), K, V, 0.1)
    with pytest.raises(ValueError):
        sbp.attn_packed(Q, K, V[:, :32].contiguous(), 0.1)
    with pytest.raises(TypeError):
        sbp.attn_packed(Q.float(), K.float(), V.float(), 0.1)
    with pytest.raises(ValueError):
        sbp.attn_packed(Q, K, V, 0.1, cu_seqlens=torch.tensor([0, 64], device="cuda"))
    with pytest.raises(ValueError):
        sbp.attn_packed(Q, K, V, 0.1, slopes=torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError):
        sbp.attn_packed(Q.cpu(), K, V, 0.1)
    with pytest.raises(sbp.SbpError):
        sbp.attn_packed(Q, K, V, 0.0)
    f = sbp.attn_packed(Q, K, V, 0.1)
    with pytest.raises(ValueError):
        sbp.attn_packed_backward(Q, K, V, f["O"], a["dO"], f["lse"].double(), 0.1)


def test_no_tokens(sbp):
    e = lambda n: torch.empty((n, 0, 64), dtype=torch.bfloat16, device="cuda")
    f = sbp.attn_packed(e(4), e(2), e(2), 0.1)
    b = sbp.attn_packed_backward(e(4), e(2), e(2), f["O"], e(4), f["lse"], 0.1)
    sbp.check_status(f["status"])
    sbp.check_status(b["status"])
    assert f["O"].shape == (4, 0, 64) and b["dK"].shape == (2, 0, 64)


def _check_document(name, x, f, b, rows, heads, z, scale, softcap, sl):
    """Outputs of the document `rows` and the query heads that share key / value head z."""
    a, e = rows
    cut = lambda t, h: host(t[h, a:e])
    kv = slice(z, z + 1)
    q, dO = cut(x["Q"], heads), cut(x["dO"], heads)
    k, v = cut(x["K"], kv), cut(x["V"], kv)
    see = np.tril(np.ones((e - a, e - a), dtype=bool))
    w = S.attention(q, k, v, see, scale, softcap, None if sl is None else sl[heads])
    near(name + " O", cut(f["O"], heads), w["O"], U * np.abs(w["O"]) + (U + 2.0 ** -11) * w["size"])
    lse = cut(f["lse"], heads)
    near(name + " lse", lse, w["lse"], 2.0 ** -12 + 2.0 ** -20 * np.abs(w["lse"]))
    errO = U * np.abs(w["O"]) + (U + 2.0 ** -11) * w["size"]
    g = S.attention_backward(q, k, v, w["O"], dO, lse, see, scale, softcap, None if sl is None else sl[heads], errO)
    near(name + " dQ", cut(b["dQ"], heads), g["dQ"], U * np.abs(g["dQ"]) + g["bQ"])
    for t in "KV":
        near(f"{name} d{t}", cut(b["d" + t], kv), g["d" + t], U * np.abs(g["d" + t]) + g["b" + t])


@pytest.mark.parametrize("softcap,alibi", [(0.0, False), (30.0, True)])
def test_a_training_step_of_8192_tokens(sbp, softcap, alibi):
    # enough units that one of them walks all four query heads of a group, each with its slope, and
    # dK and dV are summed on chip; documents are independent, so some of them stand for all
    H, Hkv, T, hd, lens = 32, 8, 8192, 128, [1024, 2048, 777, 1, 2500, 1800]
    assert sbp.attn_packed_workspace_bytes(H, Hkv, T, hd) == sbp.attn_packed_workspace_bytes_lean(H, Hkv, T, hd)
    cu, sl, kw = options(H, lens, None, softcap, alibi)
    x = {k: dev(v) for k, v in make(H, Hkv, T, hd, seed=19, gain=2.0).items()}
    f = sbp.attn_packed(x["Q"], x["K"], x["V"], hd ** -0.5, **kw)
    b = sbp.attn_packed_backward(x["Q"], x["K"], x["V"], f["O"], x["dO"], f["lse"], hd ** -0.5, **kw)
    torch.cuda.synchronize()
    sbp.check_status(f["status"])
    sbp.check_status(b["status"])
    for z, docs in ((0, (0, 2)), (5, (3, 4)), (7, (2, 5))):
        for d in docs:
            _check_document(f"head {z} document {d}", x, f, b, (cu[d], cu[d + 1]), slice(4 * z, 4 * z + 4), z, hd ** -0.5,
                            softcap, sl)
    end = cu[-1]
    assert torch.all(f["O"][:, end:] == 0) and torch.all(b["dQ"][:, end:] == 0) and torch.all(b["dK"][:, end:] == 0)


def test_elements_past_2_31(sbp):
    H, Hkv, hd, n = 16, 2, 128, 512
    T = 2 ** 20 + 300
    assert (H - 1) * T * hd < 2 ** 31 < H * T * hd
    g = torch.Generator(device="cuda").manual_seed(20)
    r = lambda h: torch.randn((h, T, hd), generator=g, device="cuda", dtype=torch.bfloat16)
    x = dict(Q=r(H), K=r(Hkv), V=r(Hkv), dO=r(H))
    cu, sl, kw = options(H, [n] * (T // n) + [T % n], None, 0.0, True)
    f = sbp.attn_packed(x["Q"], x["K"], x["V"], hd ** -0.5, **kw)
    b = sbp.attn_packed_backward(x["Q"], x["K"], x["V"], f["O"], x["dO"], f["lse"], hd ** -0.5, **kw)
    torch.cuda.synchronize()
    sbp.check_status(f["status"])
    sbp.check_status(b["status"])
    for z, d in ((0, 0), (1, 1000), (1, len(cu) - 3), (1, len(cu) - 2)):
        _check_document(f"head {z} document {d}", x, f, b, (cu[d], cu[d + 1]), slice(8 * z, 8 * z + 8), z, hd ** -0.5, 0.0, sl)


def test_forward_of_the_causal_backward(sbp):
    # attn_causal_backward takes O and lse as a forward saves them: this one, of one document
    H, Hkv, T, hd = 4, 2, 600, 128
    x = make(H, Hkv, T, hd, seed=21)
    a = {k: dev(v) for k, v in x.items()}
    f = sbp.attn_packed(a["Q"], a["K"], a["V"], hd ** -0.5)
    b = sbp.attn_causal_backward(a["Q"], a["K"], a["V"], f["O"], a["dO"], f["lse"], hd ** -0.5, 256)
    torch.cuda.synchronize()
    sbp.check_status(b["status"])
    see = S.visible(T)
    w = S.attention(x["Q"], x["K"], x["V"], see, hd ** -0.5)
    errO = U * np.abs(w["O"]) + (U + 2.0 ** -11) * w["size"]
    g = S.attention_backward(x["Q"], x["K"], x["V"], w["O"], x["dO"], host(f["lse"]), see, hd ** -0.5, errO=errO)
    for k in "QKV":
        near("d" + k, host(b["d" + k]), g["d" + k], U * np.abs(g["d" + k]) + g["b" + k])
