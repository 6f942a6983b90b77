"""Cases of the operators around an MLP of experts in 8 bits, forward and backward.

route    tokens sorted by expert and back: for ids [T, k] the order of the slots (t, j) by
         expert (dropped slots: id -1), the tokens' rows in that order, and the sum of the
         experts' rows back in token order with a weight for each slot; with its gradients
         ("step").
quant    e4m3 with a scale for each block of 128: along the rows ("rows"), or what a backward
         takes: a gradient in rows and in columns, and the input's columns in 128 x 128 tiles,
         blocks of tokens starting anew with each expert ("columns").
product  C_i = A_i B_e^T for the rows i of each expert e (one expert: a linear layer), A with a
         scale for each 128 columns of a row, B with one for each 128 x 128 tile.
linear   what a training step does with such a layer in bf16: quantising, the product, and the
         gradients dX and dW, each a product in 8 bits.

``run`` computes the plain form with elementary torch operations in fp32, or (``own``) calls
the library.  ``exact`` gives the same outputs from the definition in fp64.
"""
import math
import random

import torch

own = False

BF16, FP32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


# ------------------------------------------------------------------------------ cases

def _text(ns):
    return ",".join(str(n) for n in ns)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _route(name, T, k, E, d, mode, dtype="bf16", drop=0.0, residual=False):
    return dict(name=name, op="route", mode=mode, T=T, k=k, E=E, d=d, dtype=dtype, drop=drop, residual=residual)


def _quant(name, lens, d, mode, dtype="bf16"):
    return dict(name=name, op="quant", mode=mode, lens=_text(lens), d=d, dtype=dtype)


def _product(name, lens, N, K, out="bf16"):
    """lens: the rows of each expert."""
    return dict(name=name, op="product", lens=_text(lens), N=N, K=K, out=out)


def _linear(name, lens, N, K):
    return dict(name=name, op="linear", lens=_text(lens), N=N, K=K)


def _shares(total, E, rng):
    """How a router shares `total` rows out to E experts: a few much loaded, some empty."""
    w = [0.0 if rng.random() < 0.1 else rng.lognormvariate(0.0, 0.8) for _ in range(E)]
    if sum(w) == 0:
        w[0] = 1.0
    s = sum(w)
    lens = [int(total * x / s) for x in w]
    for e in rng.choices(range(E), w, k=total - sum(lens)):
        lens[e] += 1
    return lens


def listed():
    r = random.Random(5)
    return [
        # one token to 8 of 64 experts and back, as a model answers: the smallest call, all latency
        _route("route_fwd_T1_k8_E64_d4096", 1, 8, 64, 4096, "fwd"),
        # a training step's tokens to 8 of 64 experts, both directions
        _route("route_step_T8192_k8_E64_d4096", 8192, 8, 64, 4096, "step"),
        # an odd batch in fp32, two experts a token, slots dropped at the experts' capacity, residual added
        _route("route_step_drop_T4099_k2_E8_d2560", 4099, 2, 8, 2560, "step", "fp32", 0.15, True),
        # activations before a product, a ragged number of rows
        _quant("quant_rows_T8190_d5120", [8190], 5120, "rows"),
        # what the gradient of the experts' weights takes
        _quant("quant_columns_T16384_E16_d4096", _shares(16384, 16, r), 4096, "columns"),
        # one token through a linear layer: the weights' bytes are the floor
        _product("product_T1_N4096_K4096", [1], 4096, 4096),
        # answering 24 requests at once, 8 experts a token of 64: a few rows each
        _product("product_T192_E64_N4096_K2560", _shares(192, 64, r), 4096, 2560),
        # a short prompt, odd length
        _product("product_T501_N4096_K12288", [501], 4096, 12288),
        # the experts' product of a long batch, ragged, some experts without a row
        _product("product_T32768_E32_N4096_K2560", _shares(32768, 32, r), 4096, 2560),
        # the MLP's first product at the headline width: the largest call
        _product("product_T16384_N24576_K4096", [16384], 24576, 4096),
        # a training step of a square projection
        _linear("linear_step_T8192_N4096_K4096", [8192], 4096, 4096),
        # a training step of the experts' layer
        _linear("linear_step_T16384_E16_N2560_K4096", _shares(16384, 16, r), 2560, 4096),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "quant", "product", "product", "linear"])
    if op == "route":
        k = rng.choice([1, 2, 3, 4, 8])
        E = max(k, _log(rng, 1, 256))
        d = 8 * _log(rng, 16, 1024)
        dt = rng.choice(["bf16", "bf16", "fp32"])
        T = _log(rng, 1, max(1, min(32768, 8192 * 8 * 4096 // (k * d * (2 if dt == "fp32" else 1)))))
        c = _route("", T, k, E, d, rng.choice(["fwd", "step"]), dt,
                   rng.choice([0.0, 0.0, 0.1, 0.5]), rng.random() < 0.4)
    else:
        E = rng.choice([1, 1, 2, 4, 8, 16, 33, 64])
        N = 16 * _log(rng, 8, 768)
        K = 16 * _log(rng, 8, 768)
        if op == "quant":
            T = _log(rng, 1, min(32768, 16384 * 4096 // K))
        else:
            most = 16384 * 24576 * 4096 if op == "product" else 16384 * 4096 * 4096
            T = _log(rng, 1, max(1, min(32768, most // (N * K))))
            while E * N * K > (64 * 4096 * 2560 if op == "product" else 16 * 4096 * 2560):
                E = max(1, E // 2)
        lens = [T] if E == 1 else _shares(T, E, rng)
        if op == "quant":
            c = _quant("", lens, K, rng.choice(["rows", "columns"]), rng.choice(["bf16", "bf16", "fp32"]))
        elif op == "product":
            c = _product("", lens, N, K, rng.choice(["bf16", "bf16", "fp32"]))
        else:
            c = _linear("", lens, N, K)
    del c["name"]
    return c


# ----------------------------------------------------------------------------- inputs

def _ends(lens):
    ends = [0]
    for n in lens:
        ends.append(ends[-1] + n)
    return ends


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, dtype, std=1.0):
        x = torch.randn(shape, generator=g, device="cuda")
        return (x * std if std != 1.0 else x).to(dtype)

    def activations(T, d, dtype=BF16, std=1.0):
        """Rows of different sizes, with a few wide columns."""
        x = torch.randn((T, d), generator=g, device="cuda")
        x *= torch.exp(0.5 * torch.randn((T, 1), generator=g, device="cuda")) * std
        wide = torch.rand((1, d), generator=g, device="cuda") < 0.01
        return torch.where(wide, 20.0 * x, x).to(dtype)

    s = dict(case=case)
    if case["op"] == "route":
        T, k, E, d, dt = case["T"], case["k"], case["E"], case["d"], BF16 if case["dtype"] == "bf16" else FP32
        logits = torch.randn((T, E), generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
        top, ids = torch.topk(logits, k, dim=1)
        dropped = int(T * k * case["drop"])
        ids.view(-1)[torch.randperm(T * k, generator=g, device="cuda")[:dropped]] = -1
        s["ids"] = ids.int().contiguous()
        s["weights"] = torch.softmax(top, dim=1)
        s["n"] = T * k - dropped
        s["X"] = activations(T, d, dt)
        s["Ys"] = normal((T * k, d), dt)
        s["residual"] = normal((T, d), dt, 3.0) if case["residual"] else None
        if case["mode"] == "step":
            s["dXs"] = normal((T * k, d), dt)
            s["dY"] = normal((T, d), dt)
        return s
    lens = _ints(case["lens"])
    T, E = sum(lens), len(lens)
    s["lens"] = lens
    s["offsets"] = torch.tensor(_ends(lens), dtype=torch.int32, device="cuda") if E > 1 else None
    if case["op"] == "quant":
        dt = BF16 if case["dtype"] == "bf16" else FP32
        s["X"] = activations(T, case["d"], dt)
        if case["mode"] == "columns":
            s["dY"] = normal((T, case["d"]), dt, 1e-4)
        return s
    N, K = case["N"], case["K"]
    lead = (E,) if E > 1 else ()
    if case["op"] == "product":
        s["A8"], s["sa"] = _rows8(activations(T, K).float())
        s["B8"] = torch.empty(lead + (N, K), dtype=E4M3, device="cuda")
        s["sb"] = torch.empty(lead + ((N + 127) // 128, (K + 127) // 128), device="cuda")
        for e in range(E):
            w = torch.randn((N, K), generator=g, device="cuda") * K ** -0.5
            s["B8"].view(-1, N, K)[e], s["sb"].view((-1,) + s["sb"].shape[-2:])[e] = _tiles8(w)
        return s
    s["X"] = activations(T, K)
    s["W"] = normal(lead + (N, K), BF16, K ** -0.5)
    s["dY"] = normal((T, N), BF16, 1e-4)
    return s


# -------------------------------------------------------------------------- operators

def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    return {"route": _plain_route, "quant": _plain_quant, "product": _plain_product,
            "linear": _plain_linear}[case["op"]](s, case)


def _own(s, case):
    from memory_efficient_exact_gb300 import sbp
    if case["op"] == "route":
        n = s["n"]
        o = sbp.expert_sort(s["ids"], case["E"])
        xs = sbp.expert_gather(s["X"], o["rows"])["Xs"]
        y = sbp.expert_combine(s["Ys"], o["rows"], s["weights"], residual=s["residual"])["Y"]
        out = [o["offsets"], o["rows"], o["slots"][:n], xs[:n], y]
        if case["mode"] == "step":
            out.append(sbp.expert_gather_backward(s["dXs"], o["rows"])["dX"])
            b = sbp.expert_combine_backward(s["dY"], s["Ys"], o["rows"], s["weights"])
            out += [b["dYs"][:n], b["dweights"]]
        return out
    if case["op"] == "quant":
        if case["mode"] == "rows":
            q = sbp.quant_e4m3(s["X"])
            return [sbp.e4m3_expand(q["Y8"], q["scales"], BF16)["Y"], q["scales"]]
        g = sbp.quant_e4m3_columns(s["dY"], offsets=s["offsets"], rows=True)
        x = sbp.quant_e4m3_columns(s["X"], offsets=s["offsets"], tiles=True)
        m = sum((n + 127) // 128 for n in s["lens"])     # blocks of tokens in use
        return [sbp.e4m3_expand(g["Y8"], g["scales"], BF16)["Y"], g["scales"],
                sbp.quant_e4m3_expand(g["Yt8"], g["scales_t"], BF16)["Y"][:, :128 * m], g["scales_t"][:, :m],
                sbp.quant_e4m3_expand(x["Yt8"], x["scales_t"], BF16, tiles=True)["Y"][:, :128 * m], x["scales_t"][:, :m]]
    if case["op"] == "product":
        return sbp.matmul_e4m3(s["A8"], s["sa"], s["B8"], s["sb"], offsets=s["offsets"],
                               dtype=BF16 if case["out"] == "bf16" else FP32)["C"]
    off, T = s["offsets"], s["X"].shape[0]
    w = sbp.quant_e4m3_weight(s["W"])
    x = sbp.quant_e4m3(s["X"])
    y = sbp.matmul_e4m3(x["Y8"], x["scales"], w["W8"], w["scales"], offsets=off)["C"]
    g = sbp.quant_e4m3_columns(s["dY"], offsets=off, rows=True)
    xt = sbp.quant_e4m3_columns(s["X"], offsets=off, tiles=True)
    dx = sbp.matmul_e4m3(g["Y8"], g["scales"], w["Wt8"], w["scales_t"], offsets=off)["C"]
    dw = sbp.matmul_e4m3_columns(g["Yt8"], g["scales_t"], xt["Yt8"], xt["scales_t"], T, offsets=off)["dW"]
    return [y, dx, dw]


def _plain_route(s, case):
    T, k, E, d, dt = case["T"], case["k"], case["E"], case["d"], s["X"].dtype
    n = s["n"]
    flat = s["ids"].reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    order = torch.sort(key, stable=True)[1]
    counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda").index_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts[:E], 0)
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device="cuda")
    rows = torch.where(flat < 0, torch.full_like(place, -1), place).int().view(T, k)
    slots = order[:n].int()
    xs = s["X"][order[:n] // k]
    keep = rows >= 0
    at = rows.clamp(min=0).long()
    w = torch.where(keep, s["weights"], torch.zeros_like(s["weights"]))
    y = torch.zeros((T, d), device="cuda") if s["residual"] is None else s["residual"].float()
    for j in range(k):
        y = y + w[:, j, None] * s["Ys"][at[:, j]].float()
    out = [offsets, rows, slots, xs, y.to(dt)]
    if case["mode"] == "step":
        dy = s["dY"].float()
        dx = torch.zeros((T, d), device="cuda")
        dys = torch.empty((T * k, d), dtype=dt, device="cuda")
        dw = torch.zeros((T, k), device="cuda")
        for j in range(k):
            dx = dx + torch.where(keep[:, j, None], s["dXs"][at[:, j]].float(), torch.zeros_like(dx))
            dw[:, j] = torch.where(keep[:, j], (dy * s["Ys"][at[:, j]].float()).sum(dim=1), dw[:, j])
        back = order[:n]
        dys = (s["weights"].reshape(-1)[back][:, None] * dy[back // k]).to(dt)
        out += [dx.to(dt), dys, dw]
    return out


def _scale(amax):
    s = torch.clamp(amax / 448.0, min=2.0 ** -126)
    return torch.where(amax > 0, s, torch.ones_like(s))


def _rows8(x):
    """x [T, d] fp32 -> e4m3 [T, d] and a scale for each 128 columns of a row."""
    T, d = x.shape
    nb = (d + 127) // 128
    full = torch.zeros((T, nb * 128), device=x.device)
    full[:, :d] = x
    blk = full.view(T, nb, 128)
    s = _scale(blk.abs().amax(dim=2))
    q = (blk * (torch.ones_like(s) / s)[:, :, None]).clamp(-448.0, 448.0).to(E4M3)
    return q.view(T, nb * 128)[:, :d].contiguous(), s


def _tiles8(x):
    """x [N, K] fp32 -> e4m3 [N, K] and a scale for each 128 x 128 tile."""
    N, K = x.shape
    nn, nk = (N + 127) // 128, (K + 127) // 128
    full = torch.zeros((nn * 128, nk * 128), device=x.device)
    full[:N, :K] = x
    t = full.view(nn, 128, nk, 128)
    s = _scale(t.abs().amax(dim=3).amax(dim=1))
    q = (t * (torch.ones_like(s) / s)[:, None, :, None]).clamp(-448.0, 448.0).to(E4M3)
    return q.view(nn * 128, nk * 128)[:N, :K].contiguous(), s


def _val_rows(q, s):
    T, d = q.shape
    x = torch.zeros((T, s.shape[1] * 128), device=q.device)
    x[:, :d] = q.float()
    return (x.view(T, -1, 128) * s[:, :, None]).view(T, -1)[:, :d]


def _val_tiles(q, s):
    N, K = q.shape
    x = torch.zeros((s.shape[0] * 128, s.shape[1] * 128), device=q.device)
    x[:N, :K] = q.float()
    return (x.view(s.shape[0], 128, s.shape[1], 128) * s[:, None, :, None]).view(x.shape)[:N, :K]


def _columns(x, lens):
    """x [T, d] -> [d, W]: the tokens along the rows, each expert's from a multiple of 128 on."""
    parts, at = [], 0
    for n in lens:
        p = torch.zeros((x.shape[1], (n + 127) // 128 * 128), device=x.device)
        p[:, :n] = x[at:at + n].t()
        parts.append(p)
        at += n
    return torch.cat(parts, dim=1)


def _plain_quant(s, case):
    x = s["X"].float()
    if case["mode"] == "rows":
        q, sc = _rows8(x)
        return [_val_rows(q, sc).to(BF16), sc]
    dy = s["dY"].float()
    q, sc = _rows8(dy)
    qt, st = _rows8(_columns(dy, s["lens"]))
    xt, sx = _tiles8(_columns(x, s["lens"]))
    return [_val_rows(q, sc).to(BF16), sc, _val_rows(qt, st).to(BF16), st, _val_tiles(xt, sx).to(BF16), sx]


def _plain_product(s, case):
    dt = BF16 if case["out"] == "bf16" else FP32
    N, K = case["N"], case["K"]
    a = _val_rows(s["A8"], s["sa"])
    B, sb = s["B8"].view(-1, N, K), s["sb"].view((-1,) + s["sb"].shape[-2:])
    C = torch.empty((a.shape[0], N), dtype=dt, device="cuda")
    at = 0
    for e, n in enumerate(s["lens"]):
        if n:
            C[at:at + n] = (a[at:at + n] @ _val_tiles(B[e], sb[e]).t()).to(dt)
        at += n
    return C


def _plain_linear(s, case):
    N, K, T = case["N"], case["K"], s["X"].shape[0]
    x, dy = s["X"].float(), s["dY"].float()
    W = s["W"].view(-1, N, K)
    a, g = _val_rows(*_rows8(x)), _val_rows(*_rows8(dy))
    gt = _val_rows(*_rows8(_columns(dy, s["lens"])))
    xt = _val_tiles(*_tiles8(_columns(x, s["lens"])))
    Y = torch.empty((T, N), dtype=BF16, device="cuda")
    dX = torch.empty((T, K), dtype=BF16, device="cuda")
    dW = torch.empty(W.shape, device="cuda")
    at = col = 0
    for e, n in enumerate(s["lens"]):
        w = _val_tiles(*_tiles8(W[e].float()))
        m = (n + 127) // 128 * 128
        Y[at:at + n] = (a[at:at + n] @ w.t()).to(BF16)
        dX[at:at + n] = (g[at:at + n] @ w).to(BF16)
        dW[e] = gt[:, col:col + m] @ xt[:, col:col + m].t()
        at += n
        col += m
    return [Y, dX, dW.view(s["W"].shape)]


# ------------------------------------------------------------------------------- work

def work(case):
    if case["op"] == "route":
        T, k, d, e = case["T"], case["k"], case["d"], 2 if case["dtype"] == "bf16" else 4
        row, n = d * e, T * k - int(T * k * case["drop"])
        b = 4 * (2 * T * k + n + case["E"] + 1) + (T + n) * row + 4 * T * k + (n + T) * row
        b += T * row if case["residual"] else 0
        f = 2 * n * d
        if case["mode"] == "step":
            b += (n + T) * row + (T + 2 * n) * row + 8 * T * k
            f += 4 * n * d
        return dict(bytes=b, flops=f)
    lens = _ints(case["lens"])
    T = sum(lens)
    blocks = sum((n + 127) // 128 for n in lens)
    if case["op"] == "quant":
        # the values go out in 8 bits and come back in bf16
        d, e = case["d"], 2 if case["dtype"] == "bf16" else 4
        nb = (d + 127) // 128
        b = T * d * (e + 4) + 8 * T * nb
        f = 3 * T * d
        if case["mode"] == "columns":
            b += T * d * e + 2 * blocks * 128 * d * 4 + 8 * blocks * (d + nb)
            f += 6 * T * d
        return dict(bytes=b, flops=f)
    N, K = case["N"], case["K"]
    used = sum(1 for n in lens if n)
    nn, nk = (N + 127) // 128, (K + 127) // 128
    if case["op"] == "product":
        out = 2 if case["out"] == "bf16" else 4
        return dict(bytes=T * (K + 4 * nk) + used * (N * K + 4 * nn * nk) + T * N * out, flops=2 * T * N * K)
    b = len(lens) * N * K * (2 + 4) + T * K * (2 + 2) + T * N * (2 + 2)
    return dict(bytes=b, flops=6 * T * N * K)


# -------------------------------------------------------------------- exact (64 bits)

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s, case)
    if case["op"] == "quant":
        return _exact_quant(s, case)
    flops = work(case)["flops"]
    if flops > 6e12:
        return None
    return _exact_product(s, case) if case["op"] == "product" else _exact_linear(s, case)


def _exact_route(s, case):
    """Expert by expert; the gradients by differentiating the forward."""
    T, k, E = case["T"], case["k"], case["E"]
    ids = s["ids"].view(-1)
    members = [torch.nonzero(ids == e).view(-1) for e in range(E)]
    slots = torch.cat(members)
    offsets = torch.tensor(_ends([m.numel() for m in members]), dtype=torch.int32, device="cuda")
    n = slots.numel()
    rows = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    rows[slots] = torch.arange(n, dtype=torch.int32, device="cuda")
    token = slots // k
    xs = s["X"].double()[token]
    Ys = s["Ys"][:n].double()
    w = s["weights"].double().view(-1)[slots]
    Y = torch.zeros((T, case["d"]), dtype=torch.float64, device="cuda")
    if s["residual"] is not None:
        Y += s["residual"].double()
    Y.index_add_(0, token, w[:, None] * Ys)
    out = [offsets, rows.view(T, k), slots.int(), xs, Y]
    if case["mode"] == "step":
        dX = torch.zeros((T, case["d"]), dtype=torch.float64, device="cuda")
        dX.index_add_(0, token, s["dXs"][:n].double())
        dy = s["dY"].double()[token]
        dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        dw[slots] = torch.einsum("nd,nd->n", dy, Ys)
        out += [dX, dy * w[:, None], dw.view(T, k)]
    return out


def _exact_quant(s, case):
    """The scales; which of two neighbours a value in 8 bits takes goes by the 32-bit product."""
    def peak(x, dims):
        m = x.double().abs().amax(dims) / 448.0
        return torch.where(m > 0, m.clamp(min=2.0 ** -126), torch.ones_like(m))

    def rowwise(x):
        return torch.stack([peak(b, (1,)) for b in x.split(128, dim=1)], 1)

    if case["mode"] == "rows":
        return [None, rowwise(s["X"])]
    by_token, by_tile = [], []
    at = 0
    for n in s["lens"]:
        for a in range(at, at + n, 128):
            b = min(a + 128, at + n)
            by_token.append(peak(s["dY"][a:b], (0,)))
            by_tile.append(torch.stack([peak(c, (0, 1)) for c in s["X"][a:b].split(128, dim=1)]))
        at += n
    return [None, rowwise(s["dY"]), None, torch.stack(by_token, 1), None, torch.stack(by_tile, 1)]


def _spread(s, rows, cols, tall):
    """One scale for every element: each entry of s over (tall rows, 128 columns)."""
    return s.double().repeat_interleave(tall, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def _exact_product(s, case):
    N, K = case["N"], case["K"]
    T = s["A8"].shape[0]
    A = s["A8"].double() * _spread(s["sa"], T, K, 1)
    nb = s["sb"].shape[-2:]
    out, at = [], 0
    for e, n in enumerate(s["lens"]):
        B = s["B8"].view(-1, N, K)[e].double() * _spread(s["sb"].reshape((-1,) + nb)[e], N, K, 128)
        out.append(torch.einsum("tk,nk->tn", A[at:at + n], B))
        at += n
    return torch.cat(out)


def _exact_linear(s, case):
    """What the 8-bit values stand for in fp64; the scales and the values are 32-bit by definition."""
    N, K, T = case["N"], case["K"], s["X"].shape[0]

    def stands_for(x, tall):
        r, c = x.shape
        s32 = torch.empty(((r + tall - 1) // tall, (c + 127) // 128), device="cuda")
        for j in range(s32.shape[1]):
            m = x[:, 128 * j:128 * j + 128].float().abs().amax(1)
            pad = torch.zeros(s32.shape[0] * tall - r, device="cuda")
            s32[:, j] = torch.cat([m, pad]).view(-1, tall).amax(1)
        s32 = torch.where(s32 > 0, (s32 / 448.0).clamp(min=2.0 ** -126), torch.ones_like(s32))
        inv = torch.ones_like(s32) / s32
        inv = inv.repeat_interleave(tall, 0)[:r].repeat_interleave(128, 1)[:, :c]
        q = (x.float() * inv).clamp(-448.0, 448.0).to(E4M3)
        return q.double() * _spread(s32, r, c, tall)

    Y, dX, dW, at = [], [], [], 0
    for e, n in enumerate(s["lens"]):
        x, g = s["X"][at:at + n], s["dY"][at:at + n]
        at += n
        w = stands_for(s["W"].view(-1, N, K)[e], 128)
        Y.append(torch.matmul(stands_for(x, 1), w.transpose(0, 1)))
        dX.append(torch.matmul(stands_for(g, 1), w))
        if n:
            dW.append(torch.matmul(stands_for(g.t().contiguous(), 1), stands_for(x.t().contiguous(), 128).t()))
        else:
            dW.append(torch.zeros((N, K), dtype=torch.float64, device="cuda"))
    return [torch.cat(Y), torch.cat(dX), torch.stack(dW).view(s["W"].shape)]
