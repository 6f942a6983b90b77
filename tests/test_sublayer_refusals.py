"""Host-side refusals of the norm, rotary and packed-attention calls (CPU only: every case
fails its checks before any CUDA call, so the fake device addresses are never touched)."""
import ctypes

import pytest

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def sbp():
    from memory_efficient_exact_gb300 import _build
    _build.build_library()
    from memory_efficient_exact_gb300 import sbp as mod
    return mod


def attn(sbp, backward=False, **kw):
    a = dict(Q=0x1000, K=0x2000, V=0x3000, O=0x4000, dO=0x5000, lse=0x6000, cu=0x7000, pre=None, n=1, sl=None, H=4,
             Hkv=2, T=16, hd=64, scale=0.125, cap=0.0, dQ=0x8000, dK=0x9000, dV=0xa000, ws=0x100000, wsb=1 << 30,
             st=0xb000)
    a.update(kw)
    head = [P(a["Q"]), P(a["K"]), P(a["V"])]
    mid = [P(a["cu"]), P(a["pre"]), a["n"], P(a["sl"]), a["H"], a["Hkv"], a["T"], a["hd"], a["scale"], a["cap"]]
    tail = [P(a["ws"]), a["wsb"], P(a["st"]), None]
    if backward:
        return sbp._lib.sbp_attn_packed_backward(*head, P(a["O"]), P(a["dO"]), P(a["lse"]), *mid, P(a["dQ"]),
                                                 P(a["dK"]), P(a["dV"]), *tail)
    return sbp._lib.sbp_attn_packed_forward(*head, *mid, P(a["O"]), P(a["lse"]), *tail)


@pytest.mark.parametrize("backward", [False, True])
def test_attention(sbp, backward):
    I, U, L, W = sbp.ERR_INVALID_ARG, sbp.ERR_UNSUPPORTED, sbp.ERR_ALIGNMENT, sbp.ERR_WORKSPACE
    cases = [(I, dict(Q=None)), (I, dict(lse=None)), (I, dict(st=None)), (I, dict(T=-1)), (I, dict(H=0)), (I, dict(Hkv=3)),
             (I, dict(Hkv=8)), (I, dict(hd=0)), (I, dict(n=0)), (I, dict(cu=None)), (I, dict(scale=0.0)),
             (I, dict(scale=-1.0)), (I, dict(scale=float("nan"))), (I, dict(scale=float("inf"))), (I, dict(cap=-1.0)),
             (I, dict(cap=float("nan"))), (I, dict(cap=float("inf"))), (U, dict(cap=1e-7)), (U, dict(cap=1e7)), (U, dict(hd=60)), (U, dict(hd=136)),
             (U, dict(T=1 << 31)), (L, dict(K=0x2008)), (L, dict(cu=0x7002)), (L, dict(sl=0x7001)),
             (W, dict(ws=0x100010)), (W, dict(wsb=16)), (W, dict(ws=None))]
    if backward:
        cases += [(I, dict(dO=None)), (I, dict(dV=None)), (L, dict(dQ=0x8004))]
    for code, kw in cases:
        assert attn(sbp, backward, **kw) == code, kw


@pytest.mark.parametrize("backward", [False, True])
def test_attention_scores_out_of_range(sbp, backward):
    # caps whose scores would lose accuracy, and scales that are infinite in fp32 log2 units
    for kw in [dict(cap=257.0), dict(scale=3e38), dict(scale=1e33, cap=1e-6)]:
        assert attn(sbp, backward, **kw) == sbp.ERR_UNSUPPORTED, kw


def test_attention_workspace(sbp):
    f = sbp.attn_packed_workspace_bytes
    assert f(4, 3, 16, 64) == 0 and f(4, 2, 16, 60) == 0 and f(4, 2, -1, 64) == 0
    assert f(4, 2, 0, 64) > 0
    # nothing of size T x T, and per token no more than the four interval ends and D
    assert f(32, 8, 65536, 128) - f(32, 8, 32768, 128) <= 32768 * (16 + 4 * 32 + 1)


@pytest.mark.parametrize("H,Hkv,hd", [(32, 8, 128), (32, 8, 64), (20, 4, 128), (16, 1, 128), (7, 7, 72), (48, 8, 8)])
def test_attention_workspace_of_the_longest_serves_all(sbp, H, Hkv, hd):
    # lengths on both sides of every change in how a group's heads are shared out
    full, lean, fwd = (getattr(sbp, f"attn_packed_{n}") for n in ("workspace_bytes", "workspace_bytes_lean",
                                                                  "forward_workspace_bytes"))
    Ts = sorted({0, 1, 127, 128, 255, 256, 257} | {256 * n + r for n in range(1, 200, 3) for r in (0, 1, 255)} | {1 << 20})
    for a, b in zip(Ts, Ts[1:]):
        assert 0 < fwd(H, Hkv, a, hd) <= lean(H, Hkv, a, hd) <= full(H, Hkv, a, hd)
        assert fwd(H, Hkv, a, hd) <= fwd(H, Hkv, b, hd) and lean(H, Hkv, a, hd) <= lean(H, Hkv, b, hd)
        for f, backward in ((fwd, False), (lean, True)):
            assert attn(sbp, backward, H=H, Hkv=Hkv, T=a, hd=hd, wsb=f(H, Hkv, a, hd) - 1) == sbp.ERR_WORKSPACE
    # the forward: four interval ends, two unit lists (one entry for 256 tokens) and a block a head
    assert fwd(H, Hkv, 8192, hd) <= 8192 * 16 + 64 * 32 + Hkv * 128 * hd * 2 + 9 * 256
    for f in (full, lean, fwd):
        assert f(H, Hkv, 16, hd + 4) == 0 and f(H, H + 1, 16, hd) == 0


def norm(sbp, which, **kw):
    a = dict(X=0x1000, res=0x2000, g=0x3000, T=4, d=64, eps=1e-6, dt=0, R=0x4000, Y=0x5000, s=0x6000, dR=0x7000, dX=0x8000,
             dg=0x9000, ws=0x100000, wsb=1 << 30, st=0xb000)
    a.update(kw)
    l = sbp._lib
    if which == "fwd":
        return l.sbp_rmsnorm_forward(P(a["X"]), P(a["res"]), P(a["g"]), a["T"], a["d"], a["eps"], a["dt"], P(a["R"]),
                                     P(a["Y"]), None)
    if which == "e4m3":
        return l.sbp_rmsnorm_forward_e4m3(P(a["X"]), P(a["res"]), P(a["g"]), a["T"], a["d"], a["eps"], a["dt"], P(a["R"]),
                                          P(a["Y"]), P(a["s"]), None)
    if which == "expand":
        return l.sbp_e4m3_expand(P(a["X"]), P(a["s"]), a["T"], a["d"], a["dt"], P(a["Y"]), None)
    return l.sbp_rmsnorm_backward(P(a["X"]), P(a["R"]), P(a["g"]), P(a["dR"]), a["T"], a["d"], a["eps"], a["dt"],
                                  P(a["dX"]), P(a["dg"]), 0, P(a["ws"]), a["wsb"], P(a["st"]), None)


def test_norm(sbp):
    I, U, L, W = sbp.ERR_INVALID_ARG, sbp.ERR_UNSUPPORTED, sbp.ERR_ALIGNMENT, sbp.ERR_WORKSPACE
    for which in ("fwd", "e4m3", "expand", "bwd"):
        for code, kw in [(I, dict(T=-1)), (I, dict(d=0)), (I, dict(dt=7)), (U, dict(d=60)), (U, dict(d=16392)),
                         (I, dict(X=None)), (L, dict(X=0x1004))]:
            assert norm(sbp, which, **kw) == code, (which, kw)
    for which in ("fwd", "e4m3"):
        for code, kw in [(I, dict(g=None)), (I, dict(Y=None)), (I, dict(res=None)), (I, dict(eps=-1.0)),
                         (I, dict(eps=float("nan"))), (I, dict(eps=float("inf"))), (L, dict(res=0x2002))]:
            assert norm(sbp, which, **kw) == code, (which, kw)
    assert norm(sbp, "e4m3", s=None) == I and norm(sbp, "e4m3", s=0x6001) == L and norm(sbp, "expand", s=None) == I
    for code, kw in [(I, dict(dX=None)), (I, dict(dg=None)), (I, dict(st=None)), (L, dict(dR=0x7008)), (W, dict(ws=None)),
                     (W, dict(wsb=8)), (W, dict(ws=0x100008))]:
        assert norm(sbp, "bwd", **kw) == code, kw
    assert sbp._lib.sbp_rmsnorm_backward_workspace_bytes(4, 60, 0) == 0
    # a workspace for the blocks of one wave: it does not grow with T
    assert sbp._lib.sbp_rmsnorm_backward_workspace_bytes(1 << 20, 4096, 0) == \
        sbp._lib.sbp_rmsnorm_backward_workspace_bytes(1 << 24, 4096, 0)


def rope(sbp, backward=False, **kw):
    a = dict(x=0x1000, ld=8 * 64, pos=0x2000, n=1, sec=(32,), inv=None, theta=1e4, rot=64, il=0, T=4, H=4, Hkv=2, hd=64,
             Q=0x3000, K=0x4000, V=0x5000, kvdt=0)
    a.update(kw)
    sec = None if a["sec"] is None else (ctypes.c_int32 * len(a["sec"]))(*a["sec"])
    inv = None if a["inv"] is None else (ctypes.c_double * len(a["inv"]))(*a["inv"])
    t = [P(a["pos"]), a["n"], sec, inv, a["theta"], a["rot"], a["il"], a["T"], a["H"], a["Hkv"], a["hd"]]
    if backward:
        return sbp._lib.sbp_rope_qkv_backward(P(a["Q"]), P(a["K"]), P(a["V"]), a["kvdt"], *t, P(a["x"]), a["ld"], None)
    return sbp._lib.sbp_rope_qkv_forward(P(a["x"]), a["ld"], *t, P(a["Q"]), P(a["K"]), P(a["V"]), None)


@pytest.mark.parametrize("backward", [False, True])
def test_rope(sbp, backward):
    I, U, L = sbp.ERR_INVALID_ARG, sbp.ERR_UNSUPPORTED, sbp.ERR_ALIGNMENT
    for code, kw in [(I, dict(x=None)), (I, dict(pos=None)), (I, dict(K=None)), (I, dict(T=-1)), (I, dict(H=0)),
                     (I, dict(Hkv=-1)), (I, dict(rot=80)), (I, dict(ld=500)), (I, dict(sec=(31,))), (I, dict(sec=(33,))),
                     (I, dict(n=2, sec=(40, -8))), (I, dict(sec=None)), (I, dict(n=0)), (I, dict(il=2)),
                     (I, dict(theta=0.0)), (I, dict(theta=float("nan"))), (I, dict(theta=float("inf"))),
                     (I, dict(inv=[float("nan")] * 32)), (I, dict(inv=[float("inf")] * 32)), (U, dict(hd=40, rot=32)),
                     (U, dict(hd=272, ld=8 * 272)), (U, dict(rot=24)), (U, dict(ld=516)),
                     (U, dict(n=5, sec=(8, 8, 8, 4, 4))), (L, dict(x=0x1008)), (L, dict(Q=0x3004)), (L, dict(pos=0x2001))]:
        assert rope(sbp, backward, **kw) == code, kw
    if backward:
        assert rope(sbp, True, kvdt=5) == I


@pytest.mark.parametrize("backward", [False, True])
def test_rope_frequencies_past_the_angles_precision(sbp, backward):
    # (a call without tokens reads its frequencies and enqueues nothing)
    for f, code in ((2.0 ** 40, sbp.OK), (-(2.0 ** 40), sbp.OK), (2.0 ** 41, sbp.ERR_UNSUPPORTED), (-1e300, sbp.ERR_UNSUPPORTED)):
        assert rope(sbp, backward, inv=[f] + [1.0] * 31, T=0) == code, f
    assert rope(sbp, backward, theta=1e-300, T=0) == sbp.ERR_UNSUPPORTED


def test_empty_calls_are_accepted_without_a_gpu(sbp):
    # T = 0 enqueues nothing where there is no status word to clear
    assert norm(sbp, "fwd", T=0) == sbp.OK and norm(sbp, "e4m3", T=0) == sbp.OK and norm(sbp, "expand", T=0) == sbp.OK
    assert rope(sbp, False, T=0) == sbp.OK and rope(sbp, True, T=0) == sbp.OK
    assert sbp.last_launch_count() == 0


def test_seqlens_status_has_a_name(sbp):
    assert sbp.status_string(sbp.ERR_SEQLENS) == "SBP_ERR_SEQLENS"
