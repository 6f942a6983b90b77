"""GPU parity of the RMS norm (with the residual's addition and the 8-bit output) and of the
rotary positions against the float64 oracle, and a run of them around the packed attention.

Tolerances are element by element.  u: half a step of the output's type (bf16 2^-8, fp32
2^-24, e4m3 2^-4).  The norm's fp32 arithmetic: fewer than 64 roundings of 2^-24 on any path
(16 products a thread, 10 steps of the sums over lanes and warps, the root and the division,
four products), so 2^-18 of the terms; twice that in the gradient, which has two sums.
"""
import numpy as np
import pytest

from oracle import sublayer as S
from memory_efficient_exact_gb300 import inputs as I

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TY = {"bf16": (torch.bfloat16, 2.0 ** -8), "fp32": (torch.float32, 2.0 ** -24)}


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


def near(name, got, want, bound):
    err = np.abs(got - want)
    assert np.all(err <= bound), (name, float((err / np.maximum(bound, 1e-300)).max()), np.argwhere(err > bound)[:4].tolist())


def rows(T, d, seed, dtype, n):
    g = np.random.default_rng(seed)
    x = [g.standard_normal((T, d)).astype(np.float32) for _ in range(n)]
    gamma = (1 + 0.3 * g.standard_normal(d)).astype(np.float32)
    if dtype == "bf16":
        x, gamma = [I.round_bf16(v) for v in x], I.round_bf16(gamma)
    return x, gamma


SHAPES = [(1, 8), (1, 4096), (3, 16), (9, 128), (5, 136), (17, 248), (70, 264), (33, 1000), (300, 2560), (7, 5120),
          (2, 8192), (3, 8200), (2, 16384), (2000, 64),
          # more rows than blocks and ring places
          (1000, 2056), (1700, 4096), (900, 5120), (430, 8536), (400, 16384)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,d", SHAPES)
def test_norm(sbp, T, d, residual, dtype):
    dt, u = TY[dtype]
    (X, res, dY, dR), gamma = rows(T, d, T + d, dtype, 4)
    res = 3 * res
    if dtype == "bf16":
        res = I.round_bf16(res)
    f = sbp.rmsnorm(dev(X, dt), dev(gamma, dt), 1e-6, residual=dev(res, dt) if residual else None)
    R = X.astype(np.float64) + (res if residual else 0.0)
    Y, _ = S.rmsnorm(R, gamma, 1e-6)
    near("R", host(f["R"]), R, u * np.abs(R))
    near("Y", host(f["Y"]), Y, (u + 2.0 ** -18) * np.abs(Y))
    # the gradient is taken at the stored sum
    Rs = host(f["R"])
    b = sbp.rmsnorm_backward(dev(dY, dt), f["R"], dev(gamma, dt), 1e-6, dR=dev(dR, dt) if residual else None)
    torch.cuda.synchronize()
    sbp.check_status(b["status"])
    g = S.rmsnorm_backward(dY, Rs, gamma, 1e-6, dR if residual else None)
    near("dX", host(b["dX"]), g["dX"], u * np.abs(g["dX"]) + 2.0 ** -17 * g["terms"])
    # sums over T rows in blocks: at most T + 64 roundings
    near("dgamma", host(b["dgamma"]), g["dgamma"], (T + 128) * 2.0 ** -24 * g["dgamma_terms"])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(1, 8), (1, 256), (3, 16), (5, 136), (33, 1000), (70, 264), (1001, 512), (3, 2048), (9, 4096)])
def test_norm_gradients_without_eps(sbp, T, d, dtype):
    # rows of a block past the last one are rows of zeros, whose 1 / sqrt(0 + eps) is infinite at
    # eps = 0: nothing of them may reach dgamma
    dt, u = TY[dtype]
    (R, dY), gamma = rows(T, d, T + d, dtype, 2)
    b = sbp.rmsnorm_backward(dev(dY, dt), dev(R, dt), dev(gamma, dt), 0.0)
    torch.cuda.synchronize()
    sbp.check_status(b["status"])
    g = S.rmsnorm_backward(dY, R, gamma, 0.0)
    near("dX", host(b["dX"]), g["dX"], u * np.abs(g["dX"]) + 2.0 ** -17 * g["terms"])
    near("dgamma", host(b["dgamma"]), g["dgamma"], (T + 128) * 2.0 ** -24 * g["dgamma_terms"])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,d", [(1, 8), (5, 136), (33, 1000), (9, 5120), (3, 16384)])
def test_norm_in_8_bits(sbp, T, d, dtype):
    dt, _ = TY[dtype]
    (X, res), gamma = rows(T, d, d, dtype, 2)
    X[:, : min(d, 128)] *= 100.0 if dtype == "fp32" else 128.0   # blocks of very different size
    f = sbp.rmsnorm_e4m3(dev(X, dt), dev(gamma, dt), 1e-6, residual=dev(res, dt))
    for out, u in ((torch.bfloat16, 2.0 ** -8), (torch.float32, 2.0 ** -24)):
        e = host(sbp.e4m3_expand(f["Y8"], f["scales"], out)["Y"])
        Y, _ = S.rmsnorm(X.astype(np.float64) + res, gamma, 1e-6)
        nb = (d + 127) // 128
        amax = np.stack([np.abs(Y[:, 128 * i:128 * i + 128]).max(axis=1) for i in range(nb)], 1)
        near("scales", host(f["scales"]), amax / 448, 2.0 ** -17 * amax / 448)
        s = np.repeat(amax / 448, 128, axis=1)[:, :d]
        # half a step of e4m3 (subnormal steps are 2^-9), then the output's rounding
        near("Y", e, Y, (np.maximum(2.0 ** -4 * np.abs(Y), 2.0 ** -10 * s)) * (1 + 2 * u + 2.0 ** -16) + u * np.abs(Y))


def test_norm_in_8_bits_of_zeros(sbp):
    X = torch.zeros((3, 256), dtype=torch.bfloat16, device="cuda")
    X[1, 5] = 2.0
    f = sbp.rmsnorm_e4m3(X, torch.ones(256, dtype=torch.bfloat16, device="cuda"), 1e-6)
    assert torch.all(f["scales"][[0, 2]] == 1) and f["scales"][1, 1] == 1 and f["scales"][1, 0] > 0
    y = sbp.e4m3_expand(f["Y8"], f["scales"])["Y"]
    assert torch.isfinite(y).all() and (y != 0).sum() == 1


@pytest.mark.parametrize("tiny", [2.0 ** -120, 2.0 ** -126, 2.0 ** -130, 2.0 ** -133])
def test_norm_in_8_bits_of_tiny_values(sbp, tiny):
    # the scale of a block stays a normal number: off by half of e4m3's smallest step of it
    X = torch.ones((2, 256), device="cuda") * torch.tensor([1.0, -1.0], device="cuda")[:, None]
    X[:, ::3] = 0.0
    g = torch.full((256,), tiny, device="cuda")
    want = host(sbp.rmsnorm(X, g, 0.0)["Y"])
    f = sbp.rmsnorm_e4m3(X, g, 0.0)
    got = host(sbp.e4m3_expand(f["Y8"], f["scales"], torch.float32)["Y"])
    near("Y", got, want, np.maximum(2.0 ** -4 * np.abs(want) * (1 + 2.0 ** -16), 2.0 ** -10 * 2.0 ** -126) + 2.0 ** -149)


def test_norm_nan_stays_in_its_row(sbp):
    X = torch.ones((4, 512), dtype=torch.bfloat16, device="cuda")
    X[2, 100] = float("nan")
    gamma = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    y = sbp.rmsnorm(X, gamma, 1e-6)["Y"]
    q = sbp.rmsnorm_e4m3(X, gamma, 1e-6)
    z = sbp.e4m3_expand(q["Y8"], q["scales"])["Y"]
    for t in (y, z):
        assert torch.isnan(t[2]).all() and torch.isfinite(t[[0, 1, 3]]).all()


def test_norm_in_place_accumulate_and_repeat(sbp):
    (X, res, dY, dR), gamma = rows(700, 1000, 1, "bf16", 4)
    X, res, dY, dR, gamma = (dev(t) for t in (X, res, dY, dR, gamma))
    a = sbp.rmsnorm(X, gamma, 1e-6, residual=res)
    r = res.clone()
    b = sbp.rmsnorm(X, gamma, 1e-6, residual=r, R=r)
    assert b["R"].data_ptr() == r.data_ptr() and torch.equal(a["R"], r) and torch.equal(a["Y"], b["Y"])
    g = sbp.rmsnorm_backward(dY, a["R"], gamma, 1e-6, dR=dR)
    for kw in (dict(dR=dR.clone()), dict(dR=dR, dX="dY")):
        d = dY.clone()
        kw["dX"] = d if kw.get("dX") else kw["dR"]
        acc = torch.full((1000,), 2.0, device="cuda")
        h = sbp.rmsnorm_backward(d, a["R"], gamma, 1e-6, dgamma=acc, accumulate=True, **kw)
        assert torch.equal(g["dX"], h["dX"]) and torch.equal(acc, 2.0 + g["dgamma"])
    torch.cuda.synchronize()
    sbp.check_status(g["status"])


def test_norm_of_elements_past_2_31(sbp):
    T, d = 2 ** 17 + 5, 16384
    g = torch.Generator(device="cuda").manual_seed(4)
    n = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)
    X, res, gamma, dY = n(T, d), n(T, d), n(d), n(T, d)
    f = sbp.rmsnorm(X, gamma, 1e-6, residual=res)
    q = sbp.rmsnorm_e4m3(X, gamma, 1e-6, residual=res)
    e = sbp.e4m3_expand(q["Y8"], q["scales"])["Y"]
    b = sbp.rmsnorm_backward(dY, f["R"], gamma, 1e-6)
    torch.cuda.synchronize()
    sbp.check_status(b["status"])
    for s in (slice(0, 4), slice(2 ** 17 - 2, T)):
        R = host(X[s]) + host(res[s])
        Y, _ = S.rmsnorm(R, host(gamma), 1e-6)
        near("R", host(f["R"][s]), R, 2.0 ** -8 * np.abs(R))
        near("Y", host(f["Y"][s]), Y, (2.0 ** -8 + 2.0 ** -18) * np.abs(Y))
        amax = np.abs(Y).reshape(len(Y), -1, 128).max(axis=2).repeat(128, axis=1)
        near("Y8", host(e[s]), Y, np.maximum(2.0 ** -4 * np.abs(Y), 2.0 ** -10 * amax / 448) * (1 + 2.0 ** -7 + 2.0 ** -16) + 2.0 ** -8 * np.abs(Y))
        w = S.rmsnorm_backward(host(dY[s]), host(f["R"][s]), host(gamma), 1e-6)
        near("dX", host(b["dX"][s]), w["dX"], 2.0 ** -8 * np.abs(w["dX"]) + 2.0 ** -17 * w["terms"])


ROPE = [(1, 1, 1, 16, 16, (8,), 0), (7, 8, 2, 128, 128, (64,), 0), (5, 3, 1, 64, 32, (16,), 1), (9, 4, 2, 128, 128, (16, 24, 24), 1),
        (33, 2, 2, 96, 48, (0, 24), 0), (3, 2, 1, 256, 256, (64, 32, 0, 32), 0), (130, 5, 1, 80, 80, (40,), 1),
        (4, 2, 0, 64, 64, (32,), 0), (6, 2, 1, 48, 0, (0,), 0)]


@pytest.mark.parametrize("T,H,Hkv,hd,rot,sections,il", ROPE)
def test_rope(sbp, T, H, Hkv, hd, rot, sections, il):
    g = np.random.default_rng(T + hd)
    heads = H + 2 * Hkv
    x = I.round_bf16(g.standard_normal((T, heads * hd)).astype(np.float32))
    # near and far positions, negative ones, the ends of int32
    pos = g.integers(-1000, 10 ** 6, (len(sections), T)).astype(np.int32)
    pos[0, 0] = 2 ** 31 - 1
    pos[-1, -1] = -(2 ** 31)
    kw = dict(sections=sections, rot_dim=rot, theta=5e5, interleaved=bool(il))
    f = sbp.rope_qkv(dev(x), dev(pos, torch.int32), H, Hkv, hd, **kw)
    inv = 5e5 ** (-2.0 * np.arange(rot // 2) / rot) if rot else np.zeros(0)
    ang = S.rope_angles(pos, sections, inv) if rot else np.zeros((T, 0))
    xh = x.reshape(T, heads, hd).transpose(1, 0, 2)

    # angles: positions below 2^31 times frequencies of 53 bits, 2^-22; the cosine and sine 2^-22
    def bound(y, x):
        n = rot // 2
        size = np.abs(x)
        if n:
            a, b = (slice(0, rot, 2), slice(1, rot, 2)) if il else (slice(0, n), slice(n, rot))
            size = size.copy()
            size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
        return 2.0 ** -8 * np.abs(y) + 2.0 ** -20 * size

    want = S.rope(xh[:H + Hkv], ang, il)
    got = np.concatenate([host(f["Q"]), host(f["K"])])
    near("QK", got, want, bound(want, xh[:H + Hkv]))
    assert np.array_equal(host(f["V"]), xh[H + Hkv:])
    assert np.array_equal(got[..., rot:], xh[:H + Hkv, :, rot:])
    # the gradient, from bf16 and from fp32 dK, dV
    d = g.standard_normal((heads, T, hd)).astype(np.float32)
    for kvt in (torch.bfloat16, torch.float32):
        dd = I.round_bf16(d)
        if kvt == torch.float32:
            dd[H:] = d[H:]
        b = sbp.rope_qkv_backward(dev(dd[:H]), dev(dd[H:H + Hkv], kvt), dev(dd[H + Hkv:], kvt), dev(pos, torch.int32), **kw)
        back = S.rope(dd[:H + Hkv], ang, il, inverse=True)
        got = host(b["dqkv"]).reshape(T, heads, hd).transpose(1, 0, 2)
        near("dqkv", got[:H + Hkv], back, bound(back, dd[:H + Hkv].astype(np.float64)))
        near("dv", got[H + Hkv:], dd[H + Hkv:], 2.0 ** -8 * np.abs(dd[H + Hkv:]))

def _turns(positions, freqs):
    """position * frequency / (2 pi) less its whole part, [T, pairs]: in integers, 1 / (2 pi) to
    300 bits from pi = 16 atan(1 / 5) - 4 atan(1 / 239)."""
    bits = 320

    def atan_inv(n):
        t, s, k, sign = (1 << bits) // n, 0, 1, 1
        while t:
            s += sign * (t // k)
            t //= n * n
            k += 2
            sign = -sign
        return s

    two_pi = 8 * (4 * atan_inv(5) - atan_inv(239))          # scaled by 2^bits
    out = np.zeros((len(positions), len(freqs)))
    for j, f in enumerate(freqs):
        num, den = float(f).as_integer_ratio()
        for i, p in enumerate(positions):
            turn = ((int(p) * num) << (2 * bits)) // (den * two_pi)      # scaled by 2^bits
            out[i, j] = ((turn % (1 << bits)) >> (bits - 64)) * 2.0 ** -64
    return out


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_of_fast_frequencies_at_far_positions(sbp, interleaved):
    # the angle keeps its precision however many turns it has made: within 2^-24 of a turn, 2^-21
    # in radians, and the cosine and sine 2^-22
    freqs = [1.0, 0.7310585786300049, 1e3, 12345.678, 1e6, -98765.4321, 2.0 ** 31 + 0.3, 2.0 ** 39]
    pos = [0, 1, 2, 77777, 2 ** 24 + 1, 2 ** 31 - 1, -(2 ** 31), -123456789]
    T, H, Hkv, hd = len(pos), 2, 1, 32
    x = I.round_bf16(np.random.default_rng(5).standard_normal((T, 4 * hd)).astype(np.float32))
    kw = dict(rot_dim=16, inv_freq=freqs, interleaved=interleaved)
    p = dev(np.array([pos], np.int32), torch.int32)
    f = sbp.rope_qkv(dev(x), p, H, Hkv, hd, **kw)
    xh = x.reshape(T, 4, hd).transpose(1, 0, 2)[:3]
    ang = 2 * np.pi * _turns(pos, freqs)
    size = np.abs(xh).max(axis=2, keepdims=True) * 2
    want = S.rope(xh, ang, interleaved)
    got = np.concatenate([host(f["Q"]), host(f["K"])])
    near("QK", got, want, 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * size)
    b = sbp.rope_qkv_backward(f["Q"], f["K"], f["V"], p, **kw)
    want = S.rope(got, ang, interleaved, inverse=True)
    near("dqkv", host(b["dqkv"]).reshape(T, 4, hd).transpose(1, 0, 2)[:3], want, 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * size)


def test_rope_rows_of_a_wider_buffer_and_own_frequencies(sbp):
    g = np.random.default_rng(0)
    T, H, Hkv, hd = 11, 2, 1, 64
    wide = dev(I.round_bf16(g.standard_normal((T, 4 * 64 + 40)).astype(np.float32)))
    pos = dev(np.arange(T)[None], torch.int32)
    inv = (1.0 / (1.0 + np.arange(32))).tolist()
    f = sbp.rope_qkv(wide[:, :256], pos, H, Hkv, hd, inv_freq=inv)
    c = sbp.rope_qkv(wide[:, :256].contiguous(), pos, H, Hkv, hd, inv_freq=inv)
    assert all(torch.equal(f[k], c[k]) for k in f)
    x = host(wide[:, :256]).reshape(T, 4, hd).transpose(1, 0, 2)
    want = S.rope(x[:3], S.rope_angles(np.arange(T)[None], [32], inv), False)
    near("QK", np.concatenate([host(f["Q"]), host(f["K"])]), want, 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * 8)
    # columns behind the heads are left as they are
    out = torch.full_like(wide, 3.0)
    sbp.rope_qkv_backward(f["Q"], f["K"], f["V"], pos, inv_freq=inv, dqkv=out[:, :256])
    torch.cuda.synchronize()
    assert torch.all(out[:, 256:] == 3.0)
    near("there and back", host(out[:, :256]), host(wide[:, :256]), 2.0 ** -5)


def test_rope_of_elements_past_2_31(sbp):
    T, H, Hkv, hd = 2 ** 18 + 3, 96, 16, 64
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((T, (H + 2 * Hkv) * hd), generator=g, device="cuda", dtype=torch.bfloat16)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")[None]
    f = sbp.rope_qkv(x, pos, H, Hkv, hd)
    b = sbp.rope_qkv_backward(f["Q"], f["K"], f["V"], pos)
    for s in (slice(0, 3), slice(T - 5, T)):
        xh = host(x[s]).reshape(-1, H + 2 * Hkv, hd).transpose(1, 0, 2)
        ang = S.rope_angles(host(pos[:, s]), [hd // 2], 10000.0 ** (-2.0 * np.arange(hd // 2) / hd))
        want = S.rope(xh[:H + Hkv], ang, False)
        got = np.concatenate([host(f["Q"][:, s]), host(f["K"][:, s])])
        near("QK", got, want, 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * 16)
        assert np.array_equal(host(f["V"][:, s]), xh[H + Hkv:])
        back = S.rope(got, ang, False, inverse=True)
        near("dqkv", host(b["dqkv"][s]).reshape(-1, H + 2 * Hkv, hd).transpose(1, 0, 2)[:H + Hkv], back,
             2.0 ** -8 * np.abs(back) + 2.0 ** -20 * 16)


def test_streams_and_graphs(sbp):
    (X, res, dY), gamma = rows(300, 512, 2, "bf16", 3)
    X, res, dY, gamma = (dev(t) for t in (X, res, dY, gamma))
    pos = dev(np.arange(300)[None], torch.int32)

    def run(stream=None):
        f = sbp.rmsnorm(X, gamma, 1e-6, residual=res, stream=stream)
        q = sbp.rmsnorm_e4m3(X, gamma, 1e-6, residual=res, stream=stream)
        e = sbp.e4m3_expand(q["Y8"], q["scales"], stream=stream)
        b = sbp.rmsnorm_backward(dY, f["R"], gamma, 1e-6, stream=stream)
        r = sbp.rope_qkv(f["Y"], pos, 4, 2, 64, stream=stream)
        g = sbp.rope_qkv_backward(r["Q"], r["K"], r["V"], pos, stream=stream)
        return [f["R"], f["Y"], e["Y"], b["dX"], b["dgamma"], r["Q"], r["K"], r["V"], g["dqkv"]]

    ref = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = run()
    X.add_(1.0)
    graph.replay()
    want = run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, cap))


def test_python_refusals(sbp):
    X = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    gamma = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    for f in (lambda: sbp.rmsnorm(X.t(), gamma, 1e-6), lambda: sbp.rmsnorm(X, gamma.float(), 1e-6),
              lambda: sbp.rmsnorm(X, gamma, 1e-6, residual=X[:2]), lambda: sbp.rmsnorm(X, gamma, 1e-6, R=X),
              lambda: sbp.rmsnorm_backward(X, X[:2], gamma, 1e-6), lambda: sbp.rmsnorm(X.cpu(), gamma, 1e-6),
              lambda: sbp.e4m3_expand(X, X), lambda: sbp.rope_qkv(X, pos, 2, 1, 16, sections=[4, 4]),
              lambda: sbp.rope_qkv(X, pos.long(), 2, 1, 16), lambda: sbp.rope_qkv(X, pos, 4, 1, 16),
              lambda: sbp.rope_qkv(X, pos, 2, 1, 16, inv_freq=[1.0])):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: sbp.rmsnorm(X.half(), gamma.half(), 1e-6), lambda: sbp.rmsnorm(X.half(), gamma, 1e-6)):
        with pytest.raises((TypeError, ValueError)):
            f()
    with pytest.raises(sbp.SbpError):
        sbp.rope_qkv(X, pos, 2, 1, 16, sections=[9])
    with pytest.raises(sbp.SbpError):
        sbp.rmsnorm(X[:, :60].contiguous(), gamma[:60].contiguous(), 1e-6)


def test_sublayer_forward_and_gradients(sbp):
    """norm -> projection -> rotary positions -> packed attention -> output projection, and
    back, against the same sublayer in float64 differentiated by autograd.  Every operator's
    output is rounded to bf16 (2^-8 at most, about 2^-9.3 in norm), some ten of them in a
    row on the longest path: 2e-2 in norm, the tolerance of the other bf16 gradients."""
    T, d, H, Hkv, hd, eps, cap = 300, 256, 4, 2, 64, 1e-6, 30.0
    g = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s, k=1.0: (k * torch.randn(s, generator=g, device="cuda")).bfloat16()
    X, res, gamma = n(T, d), n(T, d), (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).bfloat16()
    Wi, Wo = n((H + 2 * Hkv) * hd, d, k=d ** -0.5), n(d, H * hd, k=(H * hd) ** -0.5)
    dOut, dRes = n(T, d), n(T, d)
    cu = torch.tensor([0, 120, 121, 290], dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(k) for k in (120, 1, 169, 10)]).to(torch.int32).cuda()[None]
    kw = dict(cu_seqlens=cu, softcap=cap)

    f = sbp.rmsnorm(X, gamma, eps, residual=res)
    r = sbp.rope_qkv(f["Y"] @ Wi.t(), pos, H, Hkv, hd)
    a = sbp.attn_packed(r["Q"], r["K"], r["V"], hd ** -0.5, **kw)
    ctx = a["O"].transpose(0, 1).reshape(T, H * hd)
    out = ctx @ Wo.t()
    dctx = (dOut @ Wo).view(T, H, hd).transpose(0, 1).contiguous()
    b = sbp.attn_packed_backward(r["Q"], r["K"], r["V"], a["O"], dctx, a["lse"], hd ** -0.5, **kw)
    q = sbp.rope_qkv_backward(b["dQ"], b["dK"], b["dV"], pos)["dqkv"]
    m = sbp.rmsnorm_backward(q @ Wi, f["R"], gamma, eps, dR=dRes)
    got = dict(out=out, dX=m["dX"], dgamma=m["dgamma"], dWi=q.t() @ f["Y"], dWo=dOut.t() @ ctx)
    torch.cuda.synchronize()
    for s in (a["status"], b["status"], m["status"]):
        sbp.check_status(s)

    x, gm, wi, wo = (t.double().requires_grad_() for t in (X, gamma, Wi, Wo))
    R = x + res.double()
    y = R / torch.sqrt((R * R).mean(1, keepdim=True) + eps) * gm
    p = (y @ wi.t()).view(T, H + 2 * Hkv, hd).transpose(0, 1)
    ang = pos[0].double()[:, None] * 10000.0 ** (-torch.arange(0, hd, 2, device="cuda").double() / hd)
    c, s = torch.cos(ang), torch.sin(ang)
    x1, x2 = p[:H + Hkv, :, :hd // 2], p[:H + Hkv, :, hd // 2:]
    qk = torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1)
    kk, vv = (t.repeat_interleave(H // Hkv, 0) for t in (qk[H:], p[H + Hkv:]))
    t = cap * torch.tanh(qk[:H] @ kk.transpose(1, 2) * hd ** -0.5 / cap)
    see = torch.from_numpy(S.visible(T, cu.tolist())).cuda()
    pr = torch.softmax(t.masked_fill(~see, -1e300), -1) * see
    o = (pr @ vv).transpose(0, 1).reshape(T, H * hd) @ wo.t()
    gr = torch.autograd.grad((o * dOut.double()).sum() + (R * dRes.double()).sum(), (x, gm, wi, wo))
    want = dict(out=o, dX=gr[0], dgamma=gr[1], dWi=gr[2], dWo=gr[3])
    for k in want:
        e = ((got[k].double() - want[k]).norm() / want[k].norm()).item()
        assert e <= 2e-2, (k, e)
