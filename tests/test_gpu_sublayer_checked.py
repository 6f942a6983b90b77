"""The norm, rotary and packed-attention calls in the checked build (a child process): a guard zone
behind every workspace region, outputs with guard elements behind them, the same bits as the
release build, and a planted overrun that each call with a workspace has to report."""
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
bf = torch.bfloat16
def rnd(*shape, dtype=bf): return torch.randn(*shape, generator=gen).to(dtype).cuda()
def out(*shape, dtype=bf):
    n = 1
    for s in shape: n *= s
    buf = torch.full((n + 64,), 7.0, dtype=dtype, device="cuda")
    return buf, buf[:n].view(*shape)
def done(name, outs, *status):
    torch.cuda.synchronize()
    h = hashlib.sha256()
    for buf, t in outs: h.update(t.contiguous().view(torch.uint8).cpu().numpy().tobytes())
    res[name] = [max([int(s.item()) for s in status] or [0]),
                 all(bool(torch.all(b[-64:].float() == 7.0).item()) for b, _ in outs), h.hexdigest()]

CASES = [(4, 4, 300, 128, None, 0.0, False), (8, 2, 700, 64, [0, 130, 131, 500], 30.0, True), (2, 1, 33, 72, [0, 20], 0.0, True),
         (48, 8, 520, 128, [0, 256, 520], 90.0, False), (1, 1, 1, 8, None, 0.0, False)]
def attn(tag, H, Hkv, T, hd, cu, cap, alibi):
    Q, K, V, dO = rnd(H, T, hd), rnd(Hkv, T, hd), rnd(Hkv, T, hd), rnd(H, T, hd)
    kw = dict(softcap=cap, cu_seqlens=None if cu is None else torch.tensor(cu, dtype=torch.int32).cuda(),
              slopes=torch.linspace(0.5, 0.01, H).cuda() if alibi else None)
    O, lse = out(H, T, hd), out(H, T, dtype=torch.float32)
    f = sbp.attn_packed(Q, K, V, hd ** -0.5, O=O[1], lse=lse[1], **kw)
    g = [out(H, T, hd), out(Hkv, T, hd), out(Hkv, T, hd)]
    b = sbp.attn_packed_backward(Q, K, V, O[1], dO, lse[1], hd ** -0.5, dQ=g[0][1], dK=g[1][1], dV=g[2][1], **kw)
    done(tag, [O, lse] + g, f["status"], b["status"])
for i, c in enumerate(CASES): attn(f"attn{i}", *c)

def norm(tag, T, d, dtype):
    X, r, dY, g = rnd(T, d, dtype=dtype), rnd(T, d, dtype=dtype), rnd(T, d, dtype=dtype), rnd(d, dtype=dtype)
    R, Y, dX = out(T, d, dtype=dtype), out(T, d, dtype=dtype), out(T, d, dtype=dtype)
    dg = out(d, dtype=torch.float32)
    sbp.rmsnorm(X, g, 1e-5, residual=r, R=R[1], Y=Y[1])
    b = sbp.rmsnorm_backward(dY, R[1], g, 1e-5, dR=r, dX=dX[1], dgamma=dg[1])
    done(tag, [R, Y, dX, dg], b["status"])
for i, (T, d) in enumerate([(5, 136), (1000, 2056), (400, 5120), (3, 16384)]):
    norm(f"norm{i}", T, d, bf)
    norm(f"norm32_{i}", T, d, torch.float32)

qkv, pos = rnd(70, 8 * 96), torch.arange(140, dtype=torch.int32).view(2, 70).cuda()
Q, K, V = out(4, 70, 96), out(2, 70, 96), out(2, 70, 96)
sbp.rope_qkv(qkv, pos, 4, 2, 96, sections=[20, 28], Q=Q[1], K=K[1], V=V[1])
dq = out(70, 8 * 96)
sbp.rope_qkv_backward(Q[1], K[1], V[1], pos, sections=[20, 28], dqkv=dq[1])
done("rope", [Q, K, V, dq])

if "checked" in res["lib"]:
    os.environ["SBP_FAULT_GUARD"] = "1"
    c = CASES[1]
    attn("planted_attn", *c)
    norm("planted_norm", 400, 5120, bf)
    os.environ["SBP_FAULT_GUARD"] = "0"
    attn("after", *c)
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
    assert checked.pop("planted_attn")[0] == over and checked.pop("planted_norm")[0] == over
    assert checked.pop("after")[0] == 0
    assert set(plain) == set(checked) and len(plain) == 14
    for k, (status, padding, bits) in plain.items():
        assert status == 0 and padding, k
        assert checked[k] == [0, True, bits], k
