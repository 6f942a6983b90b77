"""The expert-routing, quantiser and 8-bit product calls in the checked build (a child process): a
guard zone behind the sort's workspace, outputs with guard elements behind them, the same bits as
the release build, a planted overrun that the sort has to report; and products whose operands
never come, which have to leave with a status and the context usable."""
import json
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import hashlib, json, os, sys
sys.path.insert(0, sys.argv[1])
import torch
from memory_efficient_exact_gb300 import _build
_build.build_library()
from memory_efficient_exact_gb300 import sbp
res = {"lib": os.path.basename(sbp.LIB_PATH)}
gen = torch.Generator().manual_seed(7)
bf, f32, i32, f8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn
def rnd(*shape, dtype=bf): return torch.randn(*shape, generator=gen).to(dtype).cuda()
def out(*shape, dtype=bf):
    n = 1
    for s in shape: n *= s
    buf = torch.full((n + 64,), 7.0, device="cuda").to(dtype)
    return buf, buf[:n].view(*shape)
def done(name, outs, *status):
    torch.cuda.synchronize()
    h = hashlib.sha256()
    for buf, t in outs: h.update(t.contiguous().view(torch.uint8).cpu().numpy().tobytes())
    res[name] = [max([int(s.item()) for s in status] or [0]),
                 all(bool(torch.all(b[-64:].float() == 7.0).item()) for b, _ in outs), h.hexdigest()]

def sort(tag, T, k, E):
    ids = torch.randint(-1, E, (T, k), generator=gen, dtype=i32).cuda()
    rows, slots, off = out(T, k, dtype=i32), out(T * k, dtype=i32), out(E + 1, dtype=i32)
    slots[1].fill_(-5)
    r = sbp.expert_sort(ids, E, rows=rows[1], slots=slots[1], offsets=off[1])
    done(tag, [rows, slots, off], r["status"])
    return rows[1], off[1]
for i, (T, k, E) in enumerate([(1, 8, 64), (700, 3, 1000), (3000, 8, 33)]):
    rows, off = sort(f"sort{i}", T, k, E)
    d = 264
    X, w, dY = rnd(T, d), rnd(T, k, dtype=f32), rnd(T, d)
    Xs, Y, dYs, dw = out(T * k, d), out(T, d), out(T * k, d), out(T, k, dtype=f32)
    Xs[1].fill_(0); dYs[1].fill_(0)
    sbp.expert_gather(X, rows, Xs=Xs[1])
    sbp.expert_combine(Xs[1], rows, w, Y=Y[1])
    sbp.expert_combine_backward(dY, Xs[1], rows, w, dYs=dYs[1], dweights=dw[1])
    done(f"route{i}", [Xs, Y, dYs, dw])

for i, (lens, N, K) in enumerate([([1], 272, 272), ([0, 3, 9], 144, 400), ([40, 0, 300, 257], 528, 656), ([1700], 2064, 1168),
                                  ([900, 0, 3, 1100], 1040, 1296),
                                  ([10, 0, 1, 33, 32, 31, 9, 17, 5], 4096, 2064)]):
    T, E = sum(lens), len(lens)
    off = None if E == 1 else torch.tensor([sum(lens[:j]) for j in range(E + 1)], dtype=i32).cuda()
    lead = () if E == 1 else (E,)
    nb, nn, nk = sbp.token_blocks(T, E), (N + 127) // 128, (K + 127) // 128
    x, W, dy = rnd(T, K), rnd(*lead, N, K), rnd(T, N)
    q = [out(T, K, dtype=f8), out(T, nk, dtype=f32)]
    sbp.quant_e4m3(x, Y8=q[0][1], scales=q[1][1])
    w = [out(*lead, N, K, dtype=f8), out(*lead, nn, nk, dtype=f32), out(*lead, K, N, dtype=f8), out(*lead, nk, nn, dtype=f32)]
    sbp.quant_e4m3_weight(W, W8=w[0][1], scales=w[1][1], Wt8=w[2][1], scales_t=w[3][1])
    g = [out(N, 128 * nb, dtype=f8), out(N, nb, dtype=f32), out(T, N, dtype=f8), out(T, nn, dtype=f32)]
    for _, t in g: t.view(torch.uint8).fill_(0)
    a = sbp.quant_e4m3_columns(dy, offsets=off, rows=True, Yt8=g[0][1], scales_t=g[1][1], Y8=g[2][1], scales=g[3][1])
    h = [out(K, 128 * nb, dtype=f8), out(nk, nb, dtype=f32)]
    for _, t in h: t.view(torch.uint8).fill_(0)
    b = sbp.quant_e4m3_columns(x, offsets=off, tiles=True, Yt8=h[0][1], scales_t=h[1][1])
    e = out(K, 128 * nb)
    sbp.quant_e4m3_expand(h[0][1], h[1][1], tiles=True, Y=e[1])
    done(f"quant{i}", q + w + g + h + [e], a["status"], b["status"])
    c = [out(T, N), out(T, N, dtype=f32), out(T, K), out(*lead, N, K, dtype=f32)]
    st = [sbp.matmul_e4m3(q[0][1], q[1][1], w[0][1], w[1][1], offsets=off, C=c[0][1]),
          sbp.matmul_e4m3(q[0][1], q[1][1], w[0][1], w[1][1], offsets=off, C=c[1][1]),
          sbp.matmul_e4m3(g[2][1], g[3][1], w[2][1], w[3][1], offsets=off, C=c[2][1]),
          sbp.matmul_e4m3_columns(g[0][1], g[1][1], h[0][1], h[1][1], T, offsets=off, dW=c[3][1])]
    done(f"product{i}", c, *[r["status"] for r in st])

if "checked" in res["lib"]:
    os.environ["SBP_FAULT_GUARD"] = "1"
    sort("planted", 3000, 8, 33)
    os.environ["SBP_FAULT_GUARD"] = "0"
    sort("after", 3000, 8, 33)
    res["overrun"] = sbp.ERR_WORKSPACE_OVERRUN
print(json.dumps(res))
"""


def _run(variant):
    env = dict(os.environ, SBP_LIBRARY_VARIANT=variant)
    env.pop("SBP_FAULT_GUARD", None)
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True, env=env, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


def test_guard_zones_and_output_padding():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    plain, checked = _run(""), _run("checked")
    assert plain.pop("lib") == "libsbp.so" and checked.pop("lib") == "libsbp_checked.so"
    over = checked.pop("overrun")
    assert checked.pop("planted")[0] == over and checked.pop("after")[0] == 0
    assert set(plain) == set(checked) and len(plain) == 18
    for k, (status, padding, bits) in plain.items():
        assert status == 0 and padding, k
        assert checked[k] == [0, True, bits], k


STALL = r"""
import json, os, sys
sys.path.insert(0, sys.argv[1])
import torch
from memory_efficient_exact_gb300 import _build
_build.build_library()
from memory_efficient_exact_gb300 import sbp
g = torch.Generator(device="cuda").manual_seed(1)
res = []
for T, N, K, dt in [(600, 4096, 1024, torch.bfloat16), (4096, 4096, 1024, torch.float32), (32, 24576, 4096, torch.bfloat16)]:
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    q, w = sbp.quant_e4m3(n(T, K)), sbp.quant_e4m3_weight(n(N, K))
    x, y = sbp.quant_e4m3_columns(n(T, N)), sbp.quant_e4m3_columns(n(T, K), tiles=True)
    def both():
        a = sbp.matmul_e4m3(q["Y8"], q["scales"], w["W8"], w["scales"], dtype=dt)
        b = sbp.matmul_e4m3_columns(x["Yt8"], x["scales_t"], y["Yt8"], y["scales_t"], T)
        torch.cuda.synchronize()
        return a, b
    want = both()
    os.environ["SBP_FAULT_STALL"] = "1"
    stalled = both()
    os.environ["SBP_FAULT_STALL"] = "0"
    again = both()
    res.append([[int(r["status"].item()) for r in stalled], [int(r["status"].item()) for r in again],
                torch.equal(want[0]["C"], again[0]["C"]) and torch.equal(want[1]["dW"], again[1]["dW"])])
print(json.dumps(res))
"""


def test_products_that_never_come():
    # a wait of the issuing warps runs out: every role of both CTAs leaves, tensor memory is freed,
    # and the next call is right
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    env = dict(os.environ, SBP_WAIT_LIMIT_MS="100")
    r = subprocess.run([sys.executable, "-c", STALL, ROOT], env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    from memory_efficient_exact_gb300 import sbp
    for stalled, again, same in json.loads(r.stdout.strip().splitlines()[-1]):
        assert stalled == [sbp.ERR_TIMEOUT] * 2 and again == [sbp.OK] * 2 and same
