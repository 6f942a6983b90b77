"""Cases of the attention sublayer's operators: the norm before it, the rotary positions,
and the attention over packed documents, forward and backward.

norm  residual addition and root-mean-square norm:  R = X + residual,
      Y = R / sqrt(mean(R^2) + eps) * gamma; with its gradient ("step"), or with Y in
      8 bits (e4m3) and one scale for each 128 columns of a row, kept like that and
      expanded again ("e4m3").
rope  rotary positions with one to three axes on a token-major projection
      [T, (H + 2 Hkv) hd], given out as head-major Q, K, V; its gradient goes back.
attn  attention over packed documents (causal, with an optional bidirectional prefix),
      scores capped by a tanh and / or biased by the distance, grouped heads; forward
      ("fwd") or forward and gradients ("step").

``run`` computes the plain form with elementary torch operations in fp32, or (``own``)
calls the library.  ``exact`` gives the same outputs from the definition in fp64.
"""
import math

import torch

own = False

BF16, FP32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------------------ cases

def _docs(lens):
    return ",".join(str(n) for n in lens)


def _ints(text):
    return [int(x) for x in text.split(",")] if text else []


def _norm(name, T, d, mode, dtype="bf16", residual=True):
    return dict(name=name, op="norm", mode=mode, T=T, d=d, dtype=dtype, residual=residual)


def _rope(name, T, H, Hkv, hd, sections, mode, rot=None, interleaved=False, theta=1e6, far=0):
    return dict(name=name, op="rope", mode=mode, T=T, H=H, Hkv=Hkv, hd=hd, rot=hd if rot is None else rot,
                sections=_docs(sections), interleaved=interleaved, theta=theta, far=far)


def _attn(name, T, H, Hkv, hd, lens, mode, prefix=(), softcap=0.0, alibi=False, gain=1.0):
    """lens: the documents' lengths (tokens behind them are padding); gain widens the scores."""
    return dict(name=name, op="attn", mode=mode, T=T, H=H, Hkv=Hkv, hd=hd, docs=_docs(lens), prefix=_docs(prefix),
                softcap=softcap, alibi=alibi, gain=gain)


def listed():
    return [
        # one token through the norm: the smallest call, all latency
        _norm("norm_fwd_T1_d4096", 1, 4096, "fwd"),
        # the norm of a long training sequence at the headline width, both directions
        _norm("norm_step_T16384_d4096", 16384, 4096, "step"),
        # a wide model's norm that keeps its output in 8 bits, a ragged number of rows
        _norm("norm_e4m3_T8190_d5120", 8190, 5120, "e4m3"),
        # a handful of tokens: latency
        _rope("rope_fwd_T7_H8", 7, 8, 2, 128, (64,), "fwd"),
        # text positions of a long sequence, 32 query heads on 8, both directions
        _rope("rope_step_T16384_H32", 16384, 32, 8, 128, (64,), "step"),
        # video positions (time, height, width), odd length, neighbouring elements paired
        _rope("rope3_step_T8191_H32", 8191, 32, 8, 128, (16, 24, 24), "step", interleaved=True),
        # one short prompt: the smallest attention call
        _attn("attn_fwd_T33_H4", 33, 4, 2, 128, (33,), "fwd"),
        # logits of a packed batch of ragged documents, scores capped at 50
        _attn("attn_fwd_cap_T8192_H32", 8192, 32, 8, 128, (3001, 17, 1, 2048, 640, 0, 1500, 985), "fwd",
              softcap=50.0, gain=4.0),
        # a training step on the same kind of batch, without modifiers
        _attn("attn_step_docs_T8192_H32", 8192, 32, 8, 128, (1024, 2048, 777, 1, 2500, 1842), "step"),
        # prompts read in both directions before causal answers, distance bias, narrow heads
        _attn("attn_step_prefix_T4096_H16_hd64", 4096, 16, 16, 64, (1500, 1000, 1596), "step",
              prefix=(700, 0, 1596), alibi=True),
        # an odd batch with padding behind the documents, cap and distance bias together
        _attn("attn_step_cap_T4099_H20", 4099, 20, 4, 128, (2000, 3, 1700, 200), "step", softcap=30.0,
              alibi=True, gain=3.0),
        # one long document: the largest call
        _attn("attn_step_T16384_H32", 16384, 32, 8, 128, (16384,), "step"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "rope", "attn", "attn"])
    if op == "norm":
        d = 8 * _log(rng, 16, 1024)
        T = _log(rng, 1, min(32768, (16384 * 4096) // d))
        c = _norm("", T, d, rng.choice(["fwd", "step", "e4m3"]), rng.choice(["bf16", "bf16", "fp32"]),
                  rng.random() < 0.75)
    elif op == "rope":
        hd = rng.choice([64, 96, 128, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        H = Hkv * rng.choice([1, 2, 4, 5, 8])
        T = _log(rng, 1, max(1, min(32768, 16384 * 48 * 128 // ((H + 2 * Hkv) * hd))))
        rot = rng.choice([hd, hd, hd // 2])
        n = rng.choice([1, 1, 2, 3])
        cuts = sorted(rng.randint(0, rot // 2) for _ in range(n - 1))
        sec = [b - a for a, b in zip([0] + cuts, cuts + [rot // 2])]
        c = _rope("", T, H, Hkv, hd, sec, rng.choice(["fwd", "step"]), rot, rng.random() < 0.4,
                  rng.choice([1e4, 5e5, 1e6]), rng.choice([0, 0, 100000, 1000000]))
    else:
        hd = rng.choice([64, 80, 96, 128, 128, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        H = Hkv * rng.choice([1, 2, 4, 5, 8])
        mode = rng.choice(["fwd", "step", "step"])
        # documents of one token alone have no gradient but rounding: steps are longer
        T = _log(rng, 1 if mode == "fwd" else 16, min(16384, int(math.sqrt(16384.0 * 16384.0 * 32 / H))))
        if rng.random() < 0.25:
            lens = [T]
        else:
            lens, left = [], T
            while left > 0 and len(lens) < 24:
                n = min(left, 0 if rng.random() < 0.05 else _log(rng, 1, max(1, T // 2)))
                lens.append(n)
                left -= n
            if rng.random() < 0.5 and left > 0:
                lens.append(left)
        prefix = [rng.randint(0, n) for n in lens] if rng.random() < 0.3 else []
        cap = rng.choice([0.0, 0.0, 15.0, 30.0, 50.0])
        c = _attn("", T, H, Hkv, hd, lens, mode, prefix, cap,
                  rng.random() < 0.35, 1.0 if cap == 0.0 else rng.choice([1.0, 4.0]))
    del c["name"]
    return c


# ----------------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, dtype, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    s = dict(case=case)
    if case["op"] == "norm":
        T, d, dt = case["T"], case["d"], BF16 if case["dtype"] == "bf16" else FP32
        s["X"] = normal((T, d), dt)
        s["residual"] = normal((T, d), dt, 3.0) if case["residual"] else None
        s["gamma"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
        s["eps"] = 1e-6
        if case["mode"] == "step":
            s["dY"] = normal((T, d), dt)
            s["dR"] = normal((T, d), dt) if case["residual"] else None
    elif case["op"] == "rope":
        T, H, Hkv, hd = case["T"], case["H"], case["Hkv"], case["hd"]
        sec = _ints(case["sections"])
        s["qkv"] = normal((T, (H + 2 * Hkv) * hd), BF16)
        s["sections"] = sec
        t = torch.arange(T, device="cuda", dtype=torch.int32)
        rows = [t]                                # time (or the text position)
        if len(sec) > 1:                          # a video of 24 x 32 patches a frame
            rows = [t // 768, (t % 768) // 32, t % 32][3 - len(sec):]
        off = torch.randint(0, 1000, (1,), generator=g, device="cuda", dtype=torch.int32)
        s["positions"] = (torch.stack(rows) + off + case["far"]).contiguous()
        if case["mode"] == "step":
            s["dQ"] = normal((H, T, hd), BF16)
            s["dK"] = normal((Hkv, T, hd), BF16)
            s["dV"] = normal((Hkv, T, hd), BF16)
    else:
        T, H, Hkv, hd = case["T"], case["H"], case["Hkv"], case["hd"]
        lens = _ints(case["docs"])
        ends = [0]
        for n in lens:
            ends.append(ends[-1] + n)
        s["cu"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        pre = _ints(case["prefix"])
        s["prefix"] = torch.tensor(pre, dtype=torch.int32, device="cuda") if pre else None
        s["slopes"] = (torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float64) / H).float()
                       if case["alibi"] else None)
        s["scale"] = hd ** -0.5
        s["Q"] = normal((H, T, hd), BF16, case["gain"])
        s["K"] = normal((Hkv, T, hd), BF16)
        s["V"] = normal((Hkv, T, hd), BF16)
        if case["mode"] == "step":
            s["dO"] = normal((H, T, hd), BF16)
    return s


# -------------------------------------------------------------------------- operators

def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    return {"norm": _plain_norm, "rope": _plain_rope, "attn": _plain_attn}[case["op"]](s, case)


def _own(s, case):
    from memory_efficient_exact_gb300 import sbp
    if case["op"] == "norm":
        if case["mode"] == "e4m3":
            f = sbp.rmsnorm_e4m3(s["X"], s["gamma"], s["eps"], residual=s["residual"])
            y = sbp.e4m3_expand(f["Y8"], f["scales"], BF16)
            return [f["R"], y["Y"], f["scales"]]
        f = sbp.rmsnorm(s["X"], s["gamma"], s["eps"], residual=s["residual"])
        out = [f["R"], f["Y"]]
        if case["mode"] == "step":
            b = sbp.rmsnorm_backward(s["dY"], f["R"], s["gamma"], s["eps"], dR=s["dR"])
            out += [b["dX"], b["dgamma"]]
        return out
    if case["op"] == "rope":
        kw = dict(sections=s["sections"], rot_dim=case["rot"], theta=case["theta"], interleaved=case["interleaved"])
        f = sbp.rope_qkv(s["qkv"], s["positions"], case["H"], case["Hkv"], case["hd"], **kw)
        out = [f["Q"], f["K"], f["V"]]
        if case["mode"] == "step":
            out.append(sbp.rope_qkv_backward(s["dQ"], s["dK"], s["dV"], s["positions"], **kw)["dqkv"])
        return out
    kw = dict(cu_seqlens=s["cu"], prefix_lens=s["prefix"], slopes=s["slopes"], softcap=case["softcap"])
    f = sbp.attn_packed(s["Q"], s["K"], s["V"], s["scale"], **kw)
    out = [f["O"], f["lse"]]
    if case["mode"] == "step":
        b = sbp.attn_packed_backward(s["Q"], s["K"], s["V"], f["O"], s["dO"], f["lse"], s["scale"], **kw)
        out += [b["dQ"], b["dK"], b["dV"]]
    return out


def _plain_norm(s, case):
    dt = s["X"].dtype
    r = s["X"].float()
    if s["residual"] is not None:
        r = r + s["residual"].float()
    rstd = torch.rsqrt((r * r).mean(dim=1, keepdim=True) + s["eps"])
    gamma = s["gamma"].float()
    y = r * rstd * gamma
    R = r.to(dt) if s["residual"] is not None else s["X"]
    if case["mode"] == "e4m3":
        T, d = y.shape
        nb = (d + 127) // 128
        full = torch.zeros((T, nb * 128), device=y.device)
        full[:, :d] = y
        blk = full.view(T, nb, 128)
        amax = blk.abs().amax(dim=2)
        scales = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
        q = (blk / scales[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
        return [R, (q * scales[:, :, None]).view(T, nb * 128)[:, :d].to(BF16), scales]
    out = [R, y.to(dt)]
    if case["mode"] == "step":
        # the gradient's formula is on R as it was stored
        r = R.float()
        rstd = torch.rsqrt((r * r).mean(dim=1, keepdim=True) + s["eps"])
        xhat = r * rstd
        dy = s["dY"].float()
        g = dy * gamma
        dx = rstd * (g - xhat * (g * xhat).mean(dim=1, keepdim=True))
        if s["dR"] is not None:
            dx = dx + s["dR"].float()
        out += [dx.to(dt), (dy * xhat).sum(dim=0)]
    return out


def _angles(positions, sections, rot, theta):
    """cos and sin [T, rot / 2]: pair p turns by position[axis of p] * theta^(-2p / rot)."""
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).to(positions.device)
    inv = theta ** (-torch.arange(0, rot, 2, device=positions.device, dtype=torch.float64) / rot)
    a = positions.double()[axis, :].t() * inv
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(x, cos, sin, rot, interleaved):
    """x [heads, T, hd] fp32; the first rot elements turn, the others pass."""
    a = x[..., :rot]
    if interleaved:
        x1, x2 = a[..., 0::2], a[..., 1::2]
        y = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], dim=-1).flatten(-2)
    else:
        x1, x2 = a[..., :rot // 2], a[..., rot // 2:]
        y = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _plain_rope(s, case):
    T, H, Hkv, hd, rot, il = (case[k] for k in ("T", "H", "Hkv", "hd", "rot", "interleaved"))
    cos, sin = _angles(s["positions"], s["sections"], rot, case["theta"])
    x = s["qkv"].view(T, H + 2 * Hkv, hd).transpose(0, 1)
    qk = _rotate(x[:H + Hkv].float(), cos, sin, rot, il).to(BF16)
    out = [qk[:H], qk[H:], x[H + Hkv:].contiguous()]
    if case["mode"] == "step":
        d = torch.cat([s["dQ"], s["dK"]]).float()
        d = _rotate(d, cos, -sin, rot, il).to(BF16)
        out.append(torch.cat([d, s["dV"]]).transpose(0, 1).reshape(T, -1))
    return out


def _visible(cu, prefix, T):
    """[T, T]: query i (row) sees key j (column)."""
    t = torch.arange(T, device=cu.device)
    doc = torch.searchsorted(cu[1:].long(), t, right=True)
    last = cu.numel() - 2
    inside = doc <= last
    d = doc.clamp(max=last)
    see = (doc[:, None] == doc[None, :]) & inside[:, None]
    ahead = t[None, :] <= t[:, None]
    if prefix is not None:
        ahead = ahead | ((t - cu.long()[d]) < prefix.long()[d])[None, :]
    return see & ahead


def _plain_attn(s, case):
    T, H, Hkv, cap, scale = case["T"], case["H"], case["Hkv"], case["softcap"], s["scale"]
    grp = H // Hkv
    see = _visible(s["cu"], s["prefix"], T)
    t = torch.arange(T, device="cuda", dtype=torch.float32)
    dist = (t[:, None] - t[None, :]).abs()
    some = see.any(dim=1)
    O, lse = torch.empty_like(s["Q"]), torch.empty((H, T), device="cuda")
    step = case["mode"] == "step"
    if step:
        dQ, dK, dV = torch.empty_like(s["Q"]), torch.empty_like(s["K"]), torch.empty_like(s["V"])
    for h in range(Hkv):
        k, v = s["K"][h].float(), s["V"][h].float()
        dk, dv = torch.zeros_like(k), torch.zeros_like(v)
        for z in range(h * grp, (h + 1) * grp):
            q = s["Q"][z].float()
            x = q @ k.t() * scale
            th = None
            if cap > 0:
                th = torch.tanh(x / cap)
                x = cap * th
            if s["slopes"] is not None:
                x = x - s["slopes"][z] * dist
            x = torch.where(see, x, torch.full_like(x, -math.inf))
            m = torch.where(some, x.amax(dim=1), torch.zeros_like(t))
            e = torch.exp(x - m[:, None])
            l = e.sum(dim=1)
            lse[z] = m + torch.log(l)
            p = e / torch.where(some, l, torch.ones_like(l))[:, None]
            o = p @ v
            O[z] = o.to(BF16)
            if step:
                do = s["dO"][z].float()
                ds = p * (do @ v.t() - (do * o).sum(dim=1, keepdim=True))
                if cap > 0:
                    ds = ds * (1.0 - th * th)
                ds = ds * scale
                dQ[z] = (ds @ k).to(BF16)
                dk += ds.t() @ q
                dv += p.t() @ do
        if step:
            dK[h], dV[h] = dk.to(BF16), dv.to(BF16)
    return [O, lse, dQ, dK, dV] if step else [O, lse]


# ------------------------------------------------------------------------------- work

def _pairs(case):
    """(query, key) pairs that are seen, for one head."""
    lens, pre = _ints(case["docs"]), _ints(case["prefix"])
    n = 0
    for i, L in enumerate(lens):
        p = min(L, pre[i]) if pre else 0
        n += L * (L + 1) // 2 + p * (p - 1) // 2
    return n


def work(case):
    if case["op"] == "norm":
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["T"] * case["d"]
        res = 1 if case["residual"] else 0
        if case["mode"] == "e4m3":
            # Y goes out in 8 bits and comes back in bf16, as a sublayer's backward takes it
            b = n * (e * (1 + 2 * res) + 1 + 1 + 2) + 8 * case["T"] * ((case["d"] + 127) // 128)
        else:
            b = n * e * (2 + 2 * res)
        fl = 5 * n
        if case["mode"] == "step":
            b += n * e * (3 + res) + 4 * case["d"]
            fl += 10 * n
        return dict(bytes=b + e * case["d"], flops=fl)
    T, H, Hkv, hd = case["T"], case["H"], case["Hkv"], case["hd"]
    if case["op"] == "rope":
        n = T * (H + 2 * Hkv) * hd
        k = 2 if case["mode"] == "step" else 1
        return dict(bytes=k * 4 * n + 4 * T * len(_ints(case["sections"])), flops=k * 3 * T * (H + Hkv) * case["rot"])
    q, kv = T * H * hd * 2, T * Hkv * hd * 2
    b = 2 * q + 2 * kv + 4 * T * H
    f = 4 * H * hd * _pairs(case)
    if case["mode"] == "step":
        b += 4 * q + 4 * kv + 4 * T * H
        f += 10 * H * hd * _pairs(case)
    return dict(bytes=b, flops=f)


# -------------------------------------------------------------------- exact (64 bits)

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case)
    if case["op"] == "rope":
        return _exact_rope(s, case)
    cost = 2.0 * case["H"] * sum(n * n for n in _ints(case["docs"])) * case["hd"]
    if cost * (7 if case["mode"] == "step" else 2) > 6e12:
        return None
    return _exact_attn(s, case)


def _exact_norm(s, case):
    X = s["X"].double()
    gamma = s["gamma"].double().requires_grad_()
    R = X if s["residual"] is None else X + s["residual"].double()

    def norm(r):
        return r / torch.sqrt(r.pow(2).mean(-1, keepdim=True) + s["eps"]) * gamma

    with torch.no_grad():
        y = norm(R)
    if case["mode"] == "e4m3":
        T, d = y.shape
        scales = torch.stack([b.abs().amax(1) for b in y.split(128, dim=1)], 1) / 448.0
        return [R, None, torch.where(scales > 0, scales, torch.ones_like(scales))]
    if case["mode"] == "fwd":
        return [R, y]
    stored = (R.to(s["X"].dtype) if s["residual"] is not None else s["X"]).double().requires_grad_()
    dx, dg = torch.autograd.grad(norm(stored), (stored, gamma), s["dY"].double())
    if s["dR"] is not None:
        dx = dx + s["dR"].double()
    return [R, y, dx, dg]


def _exact_rope(s, case):
    T, H, Hkv, hd, rot = (case[k] for k in ("T", "H", "Hkv", "hd", "rot"))
    freq, which = [], []
    for axis, n in enumerate(s["sections"]):
        which += [axis] * n
    for p in range(rot // 2):
        freq.append(math.pow(case["theta"], -2.0 * p / rot))
    angle = torch.stack([s["positions"][a].double() * f for a, f in zip(which, freq)], 1)
    turn = torch.polar(torch.ones_like(angle), angle)

    def spin(x, w):                      # [T, rot] fp64, pairs as complex numbers
        if case["interleaved"]:
            z = torch.view_as_complex(x.reshape(T, rot // 2, 2).contiguous()) * w
            return torch.view_as_real(z).reshape(T, rot)
        z = torch.complex(x[:, :rot // 2], x[:, rot // 2:]) * w
        return torch.cat([z.real, z.imag], 1)

    def heads(x, w, n):                  # rotate heads 0 .. n-1 of [T, heads, hd]
        y = x.double().clone()
        for h in range(n):
            y[:, h, :rot] = spin(y[:, h, :rot], w)
        return y

    y = heads(s["qkv"].view(T, H + 2 * Hkv, hd), turn, H + Hkv).transpose(0, 1)
    out = [y[:H], y[H:H + Hkv], y[H + Hkv:]]
    if case["mode"] == "step":
        d = torch.cat([s["dQ"], s["dK"], s["dV"]]).transpose(0, 1)
        out.append(heads(d, turn.conj(), H + Hkv).reshape(T, -1))
    return out


def _exact_attn(s, case):
    """Document by document and head by head; the gradients by differentiating the forward."""
    T, H, Hkv, hd, cap = case["T"], case["H"], case["Hkv"], case["hd"], case["softcap"]
    lens, pre = _ints(case["docs"]), _ints(case["prefix"])
    step = case["mode"] == "step"
    O = torch.zeros((H, T, hd), dtype=torch.float64, device="cuda")
    lse = torch.full((H, T), -math.inf, dtype=torch.float64, device="cuda")
    dQ, dK, dV = (torch.zeros_like(x, dtype=torch.float64) for x in (s["Q"], s["K"], s["V"]))
    at = 0
    for i, L in enumerate(lens):
        if L == 0:
            continue
        r = slice(at, at + L)
        at += L
        n = torch.arange(L, device="cuda")
        hide = n[None, :] > n[:, None]
        if pre:
            hide = hide & (n[None, :] >= pre[i])
        for z in range(H):
            h = z * Hkv // H
            q, k, v = (x.double().requires_grad_(step) for x in (s["Q"][z, r], s["K"][h, r], s["V"][h, r]))
            x = torch.matmul(q, k.transpose(0, 1)) * s["scale"]
            if cap > 0:
                x = torch.tanh(x / cap) * cap
            if s["slopes"] is not None:
                x = x - s["slopes"][z].double() * (n[:, None] - n[None, :]).abs()
            x = x.masked_fill(hide, -math.inf)
            l = torch.logsumexp(x, 1)
            o = torch.matmul(torch.exp(x - l[:, None]), v)
            O[z, r], lse[z, r] = o.detach(), l.detach()
            if step:
                a, b, c = torch.autograd.grad(o, (q, k, v), s["dO"][z, r].double())
                dQ[z, r] = a
                dK[h, r] += b
                dV[h, r] += c
    return [O, lse, dQ, dK, dV] if step else [O, lse]
