"""GPU tests of the expert calls where their rules change: no rows at all, the sizes at which one
kernel takes over from another, and what each of them does with values that are not finite."""
import pytest

torch = pytest.importorskip("torch")
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
