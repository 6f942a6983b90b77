"""Host-side refusals of the expert-routing, quantiser and 8-bit product calls (CPU only: every case
fails its checks before any CUDA call, so the fake device addresses are never touched)."""
import ctypes

import pytest

P = ctypes.c_void_p
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sbp():
    from memory_efficient_exact_gb300 import _build
    _build.build_library()
    from memory_efficient_exact_gb300 import sbp as mod
    return mod


def call(f, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a)
    a.update(kw)
    args = [P(v) if k[0].isupper() else v for k, v in a.items() if k != "stream"]
    return f(*args, None)


SORT = dict(Ids=0x1000, t=4, k=2, e=8, Rows=0x2000, Slots=0x3000, Off=0x4000, Ws=0x100000, wsb=1 << 20, St=0x5000)
GATHER = dict(X=0x1000, S=None, Rows=0x2000, t=4, k=2, n=8, d=64, dt=0, Xs=0x3000, Ss=None)
COMB = dict(Ys=0x1000, Rows=0x2000, W=0x3000, Res=None, t=4, k=2, n=8, d=64, dt=0, Y=0x4000)
CBWD = dict(DY=0x1000, Ys=0x2000, Rows=0x3000, W=0x4000, t=4, k=2, n=8, d=64, dt=0, DYs=0x5000, DW=0x6000)
QROWS = dict(X=0x1000, t=4, d=64, dt=0, Y=0x2000, S=0x3000)
QCOLS = dict(X=0x1000, Off=0x2000, e=2, t=4, d=64, dt=0, tiles=0, Y=None, S=None, Yt=0x3000, St=0x4000, Status=0x5000)
QEXP = dict(Y8=0x1000, S=0x2000, t=4, d=64, tiles=0, dt=0, Y=0x3000)
QWEI = dict(W=0x1000, e=2, n=32, k=64, dt=0, W8=0x2000, S=0x3000, Wt=0x4000, St=0x5000)
MM = dict(A=0x1000, Sa=0x2000, B=0x3000, Sb=0x4000, Off=0x5000, e=2, t=4, n=32, k=64, dt=0, C=0x6000, Status=0x7000)
MMC = dict(A=0x1000, Sa=0x2000, B=0x3000, Sb=0x4000, Off=0x5000, e=2, t=4, n=32, k=64, DW=0x6000, acc=0,
           Status=0x7000)
BIG = (1 << 30) + 1


def test_calls(sbp):
    I, U, L, W = sbp.ERR_INVALID_ARG, sbp.ERR_UNSUPPORTED, sbp.ERR_ALIGNMENT, sbp.ERR_WORKSPACE
    table = [
        (sbp._lib.sbp_expert_sort, SORT,
         [(I, dict(t=-1)), (I, dict(k=0)), (I, dict(e=0)), (U, dict(e=1025)), (U, dict(t=BIG)), (U, dict(t=1 << 20, k=1 << 12)),
          (I, dict(Ids=None)), (I, dict(Rows=None)), (I, dict(Slots=None)), (I, dict(Off=None)), (I, dict(St=None)),
          (L, dict(Ids=0x1002)), (W, dict(t=2000, Ws=None)), (W, dict(t=2000, Ws=0x100010)), (W, dict(t=2000, wsb=16))]),
        (sbp._lib.sbp_expert_gather, GATHER,
         [(I, dict(t=-1)), (I, dict(k=0)), (I, dict(n=-1)), (I, dict(d=0)), (I, dict(dt=3)), (U, dict(d=60)), (U, dict(d=16392)),
          (U, dict(dt=2, d=72, S=0x4000, Ss=0x5000)), (U, dict(t=BIG)), (I, dict(X=None)), (I, dict(Rows=None)),
          (I, dict(Xs=None)), (I, dict(S=0x4000)), (I, dict(dt=2, S=0x4000)), (I, dict(dt=2, Ss=0x4000)), (L, dict(X=0x1008)),
          (L, dict(Rows=0x2001)), (L, dict(dt=2, S=0x4002, Ss=0x5000))]),
        (sbp._lib.sbp_expert_combine, COMB,
         [(I, dict(t=-1)), (I, dict(k=0)), (I, dict(d=0)), (I, dict(dt=2)), (U, dict(d=20)), (U, dict(n=1 << 32)), (I, dict(Ys=None)),
          (I, dict(Rows=None)), (I, dict(Y=None)), (L, dict(Ys=0x1004)), (L, dict(Res=0x1008)), (L, dict(W=0x3002))]),
        (sbp._lib.sbp_expert_combine_backward, CBWD,
         [(I, dict(t=-1)), (I, dict(k=0)), (I, dict(d=0)), (I, dict(dt=2)), (U, dict(d=20)), (I, dict(DY=None)), (I, dict(Ys=None)),
          (I, dict(Rows=None)), (I, dict(W=None)), (I, dict(DYs=None)), (I, dict(DW=None)), (L, dict(DYs=0x5004)),
          (L, dict(DW=0x6001))]),
        (sbp._lib.sbp_quant_e4m3_rows, QROWS,
         [(I, dict(t=-1)), (I, dict(d=0)), (I, dict(dt=2)), (U, dict(d=12)), (U, dict(t=BIG)), (U, dict(t=1 << 29, d=1024)),
          (I, dict(X=None)), (I, dict(Y=None)), (I, dict(S=None)), (L, dict(X=0x1008)), (L, dict(Y=0x2008)), (L, dict(S=0x3002))]),
        (sbp._lib.sbp_quant_e4m3_columns, QCOLS,
         [(I, dict(t=-1)), (I, dict(d=0)), (I, dict(dt=2)), (I, dict(e=0)), (U, dict(e=1025)), (I, dict(Off=None)), (I, dict(tiles=2)),
          (U, dict(d=12)), (I, dict(X=None)), (I, dict(Yt=None)), (I, dict(St=None)), (I, dict(Status=None)), (I, dict(Y=0x8000)),
          (I, dict(S=0x8000)), (L, dict(Yt=0x3008)), (L, dict(Off=0x2001))]),
        (sbp._lib.sbp_quant_e4m3_expand, QEXP,
         [(I, dict(t=-1)), (I, dict(d=0)), (I, dict(dt=2)), (I, dict(tiles=2)), (U, dict(d=12)), (U, dict(d=(1 << 20) + 8)),
          (I, dict(Y8=None)), (I, dict(S=None)), (I, dict(Y=None)), (L, dict(Y8=0x1004)), (L, dict(Y=0x3008)), (L, dict(S=0x2002))]),
        (sbp._lib.sbp_quant_e4m3_weight, QWEI,
         [(I, dict(e=0)), (I, dict(n=0)), (I, dict(k=0)), (I, dict(dt=2)), (U, dict(e=1025)), (U, dict(n=24)), (U, dict(k=72)),
          (I, dict(W=None)), (I, dict(W8=None)), (I, dict(Wt=None)), (I, dict(S=None)), (I, dict(St=None)), (L, dict(Wt=0x4008))]),
        (sbp._lib.sbp_matmul_e4m3, MM,
         [(I, dict(e=0)), (I, dict(t=-1)), (I, dict(n=0)), (I, dict(k=0)), (I, dict(Off=None)), (I, dict(dt=2)), (U, dict(e=1025)),
          (U, dict(k=72)), (U, dict(n=12)), (U, dict(t=BIG)), (U, dict(n=1 << 21)), (I, dict(A=None)), (I, dict(Sa=None)),
          (I, dict(B=None)), (I, dict(Sb=None)), (I, dict(C=None)), (I, dict(Status=None)), (L, dict(A=0x1008)), (L, dict(C=0x6004)),
          (L, dict(Sb=0x4002))]),
        (sbp._lib.sbp_matmul_e4m3_columns, MMC,
         [(I, dict(e=0)), (I, dict(t=-1)), (I, dict(n=0)), (I, dict(k=0)), (I, dict(Off=None)), (U, dict(e=1025)), (U, dict(k=12)),
          (U, dict(n=12)), (I, dict(A=None)), (I, dict(Sa=None)), (I, dict(B=None)), (I, dict(Sb=None)), (I, dict(DW=None)),
          (I, dict(Status=None)), (L, dict(B=0x3008)), (L, dict(DW=0x6008))]),
    ]
    for f, defaults, cases in table:
        for code, kw in cases:
            assert call(f, defaults, kw) == code, (f.__name__, kw)


def test_queries(sbp):
    f = sbp._lib.sbp_expert_sort_workspace_bytes
    assert f(-1, 2, 8) == 0 and f(4, 0, 8) == 0 and f(4, 2, 0) == 0 and f(4, 2, 1025) == 0 and f(1 << 30, 2, 8) == 0
    assert f(0, 2, 8) > 0 and f(1 << 20, 8, 256) <= (1 << 23) // 2048 * 256 * 4 + 1024
    assert sbp.token_blocks(0, 3) == 0 and sbp.token_blocks(1, 1) == 1 and sbp.token_blocks(129, 1) == 2
    assert sbp.token_blocks(5, 8) == 5 and sbp.token_blocks(256, 3) == (256 + 3 * 127) // 128
    assert sbp.token_blocks(-1, 1) == -1 and sbp.token_blocks(4, 0) == -1 and sbp.token_blocks(4, 1025) == -1
    # the most blocks: tables of a few rows, exhaustively
    for T in range(0, 9):
        for E in (1, 2, 3):
            def tables(left, e):
                if e == 1:
                    yield (left,)
                    return
                for n in range(left + 1):
                    for rest in tables(left - n, e - 1):
                        yield (n,) + rest
            most = max(sum((128 * n + 127) // 128 for n in t) for t in tables(T, E))
            assert most <= sbp.token_blocks(128 * T, E)


def test_binding_refuses_host_tensors_and_shapes(sbp):
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    ids = torch.zeros((4, 2), dtype=torch.int32)
    x, r = torch.zeros((4, 64), dtype=bf), torch.zeros((4, 2), dtype=torch.int32)
    for f in [lambda: sbp.expert_sort(ids, 4), lambda: sbp.expert_gather(x, r), lambda: sbp.expert_combine(x, r),
              lambda: sbp.expert_combine_backward(x, x, r, torch.zeros(4, 2)), lambda: sbp.quant_e4m3(x),
              lambda: sbp.quant_e4m3_columns(x), lambda: sbp.quant_e4m3_weight(x), lambda: sbp.quant_e4m3_expand(x.to(f8), torch.zeros(4, 1)),
              lambda: sbp.matmul_e4m3(x.to(f8), torch.zeros(4, 1), x.to(f8), torch.zeros(1, 1)),
              lambda: sbp.matmul_e4m3_columns(x.to(f8), torch.zeros(4, 1), x.to(f8), torch.zeros(1, 1), 4)]:
        with pytest.raises(ValueError):
            f()
