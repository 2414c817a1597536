"""What the layer's training and 8-bit operators compute, at sizes of real use, for timing and comparison.

Operators: matrix products grouped by expert over ragged rows (forward, gradient of the rows, gradient of
the weights), the same product in 8-bit integers with a scale per token and per output channel, the SwiGLU
gate between the two products of an expert with its gradient, and the gradient of the weighted combine.

`run` computes them in plain torch operations in 32 bits, or, where `own` is true, through the package.
Sizes follow the repository's layers: H = 4096, I = 14336, E = 8, k = 2 (bf16 experts); H = I = 2880,
E = 128, k = 4 with a skewed expert popularity; H = 7168, I = 2048, E = 384, k = 8.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}

# the largest listed case, in multiply-adds and in weights
MAX_MACS = 8192 * 28672 * 4096
MAX_WEIGHTS = 8 * 28672 * 4096


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token through the gate/up matrices of its 4 experts: the smallest call
        dict(name="product-decode", op="product", dt="bf16", out="bf16", T=1, k=4, E=128, N=5760, K=2880, zipf=1.1,
             gather=True, spare=0),
        # a serving batch over 128 experts of very uneven popularity, the down matrices, fp32 results
        dict(name="product-ragged", op="product", dt="bf16", out="f32", T=509, k=4, E=128, N=2880, K=2880, zipf=1.1,
             gather=False, spare=0),
        # a long prompt or a training batch through wide gate/up matrices: the largest call
        dict(name="product-prefill", op="product", dt="bf16", out="bf16", T=4096, k=2, E=8, N=28672, K=4096, zipf=0.0,
             gather=True, spare=0),
        # one training step's backward products of the down matrices: both gradients, weights' in fp32
        dict(name="gradients-bf16", op="gradients", dt="bf16", out="bf16", dw="f32", T=3001, k=2, E=8, N=4096, K=14336,
             zipf=0.3, gather=False, spare=0),
        # the router's own gradients in fp32: one group of all tokens
        dict(name="gradients-router-f32", op="gradients", dt="f32", out="f32", dw="f32", T=4096, k=1, E=1, N=128,
             K=2880, zipf=0.0, gather=False, spare=0),
        # 8-bit products: one decoded token; a serving batch (the SwiGLU gate is quantized on the way); a long prompt
        dict(name="int8-decode", op="int8", dt="bf16", out="bf16", act="none", T=1, k=4, E=128, N=5760, K=2880,
             zipf=1.1, spare=0),
        dict(name="int8-ragged", op="int8", dt="bf16", out="bf16", act="swiglu", T=333, k=4, E=128, N=2880, K=2880,
             zipf=1.1, spare=0),
        dict(name="int8-prefill", op="int8", dt="bf16", out="bf16", act="none", T=4096, k=2, E=8, N=28672, K=4096,
             zipf=0.0, spare=0),
        # the gate between the products: a decode batch, and a training step's gradient (h again beside it)
        dict(name="swiglu-decode", op="swiglu", dt="bf16", rows=64, I=2880, grad=False),
        dict(name="swiglu-train", op="swiglu", dt="bf16", rows=6002, I=14336, grad=True),
        # the combine's gradient, gate weights and router logits included: a small and a long batch
        dict(name="combine-grad-small", op="combine_grad", dt="bf16", dy="bf16", T=16, k=8, E=384, H=7168, drop=0.0),
        dict(name="combine-grad-train", op="combine_grad", dt="bf16", dy="bf16", T=8192, k=8, E=384, H=7168, drop=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A matrix width: mostly a multiple of 32, sometimes of 8, sometimes odd."""
    n = _log(rng, lo, hi)
    r = rng.random()
    step = 32 if r < 0.6 else 8 if r < 0.8 else 1
    return max(step, n // step * step)


def draw(rng):
    op = rng.choice(["product", "product", "gradients", "gradients", "int8", "int8", "swiglu", "combine_grad"])
    if op == "swiglu":
        rows, I = _log(rng, 1, 6000), _width(rng, 32, 14336)
        return dict(op=op, dt=rng.choice(["bf16", "f32"]), rows=rows, I=I, grad=rng.random() < 0.6)
    if op == "combine_grad":
        E = _log(rng, 2, 384)
        return dict(op=op, dt=rng.choice(["bf16", "f32"]), dy=rng.choice(["bf16", "f32"]), T=_log(rng, 1, 4096),
                    k=rng.randint(1, min(8, E)), E=E, H=max(4, _width(rng, 32, 7168) // 4 * 4),
                    drop=rng.choice([0.0, 0.0, 0.1]))
    while True:
        E = _log(rng, 1, 256)
        k = rng.randint(1, min(8, E))
        case = dict(op=op, dt="bf16", out=rng.choice(["bf16", "f32"]), T=_log(rng, 1, 4096), k=k, E=E,
                    N=_width(rng, 32, 8192), K=_width(rng, 32, 8192), zipf=rng.choice([0.0, 0.5, 1.1]),
                    spare=rng.choice([0, 0, 7]))
        if op == "int8":
            case["act"] = rng.choice(["none", "swiglu"])
            case["dt"] = rng.choice(["bf16", "bf16", "f32"])
            if case["act"] == "swiglu":
                # a gate evaluated in 32 bits moves single integers: nobody keeps such sums in 32 bits
                case["out"] = "bf16"
        else:
            case["gather"] = rng.random() < 0.5
            case["dt"] = rng.choice(["bf16", "bf16", "bf16", "f32"])
            if case["dt"] == "f32":
                case["out"] = "f32"
            if op == "gradients":
                case["dw"] = rng.choice(["bf16", "f32"]) if case["dt"] == "bf16" else "f32"
        # fp32 products run at about a tenth of the rate of the bf16 ones; two products in a gradient pass
        macs = case["T"] * k * case["N"] * case["K"] * (10 if case["dt"] == "f32" and op != "int8" else 1)
        if macs * (2 if op == "gradients" else 1) <= MAX_MACS and E * case["N"] * case["K"] * 2 <= MAX_WEIGHTS:
            return case


# ------------------------------------------------------------------ inputs
def _route(T, k, E, zipf, seed):
    """Expert ids [T, k] (distinct per token, popularity rank^-zipf): the k largest of log popularity + Gumbel."""
    rng = np.random.default_rng(seed)
    logp = -zipf * np.log(1.0 + rng.permutation(E))
    u = rng.random((T, E))
    score = logp - np.log(-np.log(np.maximum(u, 1e-300)))
    if k < E:
        return np.argpartition(-score, k - 1, axis=1)[:, :k].astype(np.int32)
    return np.tile(np.arange(E, dtype=np.int32), (T, 1))


def _group(ids, E):
    """The stable grouping by expert: offsets [E + 1], perm_src (flat t * k + j of every grouped row)."""
    flat = ids.reshape(-1)
    perm = np.argsort(flat, kind="stable").astype(np.int32)
    offsets = np.zeros(E + 1, dtype=np.int32)
    offsets[1:] = np.cumsum(np.bincount(flat, minlength=E))
    return offsets, perm


def _normal(gen, shape, sigma, dt):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * sigma).to(dt)


def _weights(gen, E, N, K, sigma, dt):
    w = torch.empty((E, N, K), device="cuda", dtype=dt)
    for e in range(E):
        w[e] = _normal(gen, (N, K), sigma, dt)
    return w


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": case}
    op, dt = case["op"], DT[case["dt"]]
    if op == "swiglu":
        rows, I = case["rows"], case["I"]
        st["gu"] = _normal(gen, (rows, 2 * I), 1.5, dt)
        st["h"] = torch.empty((rows, I), device="cuda", dtype=dt)
        if case["grad"]:
            st["dh"] = _normal(gen, (rows, I), 0.02, dt)
            st["dgu"] = torch.empty((rows, 2 * I), device="cuda", dtype=dt)
        return st
    if op == "combine_grad":
        T, k, E, H = case["T"], case["k"], case["E"], case["H"]
        ids = _route(T, k, E, 0.5, seed)
        if case["drop"]:
            # pairs without an expert: not placed, and without a gradient
            ids = np.where(np.random.default_rng(seed + 1).random(ids.shape) < case["drop"], -1, ids)
        flat = ids.reshape(-1)
        order = np.argsort(np.where(flat < 0, E, flat), kind="stable")
        placed = int((flat >= 0).sum())
        inv = np.full(T * k, -1, dtype=np.int32)
        inv[order[:placed]] = np.arange(placed, dtype=np.int32)
        st["ids"] = torch.from_numpy(ids.astype(np.int32)).cuda()
        st["inv"] = torch.from_numpy(inv).cuda()
        st["dout"] = _normal(gen, (T, H), 0.02, dt)
        st["y"] = _normal(gen, (T * k, H), 1.0, torch.float32)
        st["w"] = torch.softmax(_normal(gen, (T, k), 1.0, torch.float32), dim=1)
        st["dy"] = torch.zeros((T * k, H), device="cuda", dtype=DT[case["dy"]])
        st["dw"] = torch.empty((T, k), device="cuda", dtype=torch.float32)
        st["dlogits"] = torch.empty((T, E), device="cuda", dtype=torch.float32)
        return st
    T, k, E, N, K = case["T"], case["k"], case["E"], case["N"], case["K"]
    offsets, perm = _group(_route(T, k, E, case["zipf"], seed), E)
    P = T * k
    rows = P + case["spare"]  # room for more rows than are placed
    st["bounds"] = [int(o) for o in offsets]
    st["offsets"] = torch.from_numpy(offsets).cuda()
    st["perm"] = torch.from_numpy(np.concatenate([perm, np.zeros(case["spare"], np.int32)])).cuda()
    if op == "int8":
        swiglu = case["act"] == "swiglu"
        # tokens are quantized before they are gathered; the gate's rows are already grouped
        st["x"] = _normal(gen, (rows if swiglu else T, 2 * K if swiglu else K), 1.0, dt)
        w = torch.empty((E, N, K), device="cuda", dtype=torch.int8)
        for e in range(E):
            w[e] = torch.clamp(torch.round(_normal(gen, (N, K), 32.0, torch.float32)), -127, 127).to(torch.int8)
        st["w"] = w
        st["w_scale"] = (torch.rand((E, N), generator=gen, device="cuda") * 0.5 + 0.75) * (0.02 / 32.0)
        st["y"] = torch.zeros((rows, N), device="cuda", dtype=DT[case["out"]])
        st["q"] = torch.empty((st["x"].shape[0], K), device="cuda", dtype=torch.int8)
        st["q_scale"] = torch.empty(st["x"].shape[0], device="cuda", dtype=torch.float32)
        return st
    st["x"] = _normal(gen, (T if case["gather"] else rows, K), 1.0, dt)
    if op == "product":
        st["w"] = _weights(gen, E, N, K, 0.02, dt)
        st["y"] = torch.zeros((rows, N), device="cuda", dtype=DT[case["out"]])
    else:
        st["w"] = _weights(gen, E, N, K, 0.02, dt)
        st["dy"] = _normal(gen, (rows, N), 0.02, dt)
        st["dx"] = torch.zeros((rows, K), device="cuda", dtype=DT[case["out"]])
        st["dw"] = torch.empty((E, N, K), device="cuda", dtype=DT[case["dw"]])
    if own:
        from mixture_experts_layer_token_amd import api

        need = api.moe_grouped_workspace(case["dt"], rows, N, K, E)
        st["ws"] = torch.empty(max(need, 256), device="cuda", dtype=torch.uint8)
    return st


# ------------------------------------------------------------------ one pass
def _run_own(st):
    from mixture_experts_layer_token_amd import api

    case = st["case"]
    op = case["op"]
    if op == "swiglu":
        if not case["grad"]:
            api.moe_swiglu(st["gu"], st["h"])
            return st["h"]
        api.moe_swiglu_grad(st["gu"], st["dh"], st["dgu"], h=st["h"])
        return [st["dgu"], st["h"]]
    if op == "combine_grad":
        api.moe_combine_grad(st["dout"], st["y"], st["w"], st["inv"], case["k"], st["dy"], st["dw"],
                             topk_ids=st["ids"], dlogits=st["dlogits"])
        return [st["dy"], st["dw"], st["dlogits"]]
    if op == "int8":
        if case["act"] == "swiglu":
            api.moe_quant_rows(st["x"], st["q"], st["q_scale"], act="swiglu", n_rows=st["offsets"][-1:])
            api.moe_grouped_gemm_i8(st["q"], st["q_scale"], st["w"], st["w_scale"], st["offsets"], st["y"])
        else:
            api.moe_quant_rows(st["x"], st["q"], st["q_scale"])
            api.moe_grouped_gemm_i8(st["q"], st["q_scale"], st["w"], st["w_scale"], st["offsets"], st["y"],
                                    perm_src=st["perm"], k=case["k"])
        return st["y"]
    gather = dict(perm_src=st["perm"], k=case["k"]) if case["gather"] else {}
    if op == "product":
        api.moe_grouped_gemm(st["x"], st["w"], st["offsets"], st["y"], ws=st["ws"], **gather)
        return st["y"]
    api.moe_grouped_gemm_dx(st["dy"], st["w"], st["offsets"], st["dx"], ws=st["ws"])
    api.moe_grouped_gemm_dw(st["dy"], st["x"], st["offsets"], st["dw"], ws=st["ws"], **gather)
    return [st["dx"], st["dw"]]


def _rows_of(st, key, e, div, ft):
    """Rows of expert e in type ft: the grouped rows themselves, or the tokens that perm_src names."""
    lo, hi = st["bounds"][e], st["bounds"][e + 1]
    if div:
        return st[key][torch.div(st["perm"][lo:hi], div, rounding_mode="floor").long()].to(ft)
    return st[key][lo:hi].to(ft)


def _silu(z):
    return z / (1 + torch.exp(-z))


def run(st):
    if own:
        return _run_own(st)
    case = st["case"]
    op = case["op"]
    f32 = torch.float32
    if op == "swiglu":
        I = case["I"]
        g, u = st["gu"][:, :I].to(f32), st["gu"][:, I:].to(f32)
        s = 1 / (1 + torch.exp(-g))
        h = g * s * u
        if not case["grad"]:
            return h.to(DT[case["dt"]])
        dh = st["dh"].to(f32)
        dg = dh * u * s * (1 + g * (1 - s))
        du = dh * g * s
        return [torch.cat([dg, du], dim=1).to(DT[case["dt"]]), h.to(DT[case["dt"]])]
    if op == "combine_grad":
        T, k, H, E = case["T"], case["k"], case["H"], case["E"]
        inv = st["inv"].long()
        dropped = (inv < 0).view(T, k)
        dout = st["dout"].to(f32)
        y = st["y"][inv.clamp(min=0)].view(T, k, H)
        dw = (y * dout[:, None, :]).sum(dim=2).masked_fill(dropped, 0.0)
        dy_tok = st["w"][:, :, None] * dout[:, None, :]
        dy = torch.zeros((T * k + 1, H), device="cuda", dtype=DT[case["dy"]])
        dy[torch.where(inv < 0, T * k, inv)] = dy_tok.view(T * k, H).to(DT[case["dy"]])
        dl = (st["w"] * (dw - (st["w"] * dw).sum(dim=1, keepdim=True))).masked_fill(dropped, 0.0)
        dlogits = torch.zeros((T, E + 1), device="cuda", dtype=f32)
        dlogits.scatter_(1, torch.where(st["ids"] < 0, E, st["ids"]).long(), dl)
        return [dy[:T * k], dw, dlogits[:, :E].contiguous()]
    E, N, K, b = case["E"], case["N"], case["K"], st["bounds"]
    if op == "int8":
        # in 64 bits: a quotient next to a half would round to the other integer
        x = st["x"].to(torch.float64)
        if case["act"] == "swiglu":
            x = _silu(x[:, :K]) * x[:, K:]
        amax = x.abs().amax(dim=1, keepdim=True)
        q = torch.round(torch.where(amax > 0, x * 127 / amax, 0.0)).to(f32)
        st = dict(st, q=q, s=(amax / 127).to(f32))
        div = 0 if case["act"] == "swiglu" else case["k"]
        y = torch.zeros_like(st["y"])
        for e in range(E):
            if b[e] < b[e + 1]:
                acc = _rows_of(st, "q", e, div, f32) @ st["w"][e].to(f32).t()
                y[b[e]:b[e + 1]] = (acc * _rows_of(st, "s", e, div, f32) * st["w_scale"][e]).to(y.dtype)
        return y
    div = case["k"] if case["gather"] else 0
    if op == "product":
        y = torch.zeros_like(st["y"])
        for e in range(E):
            if b[e] < b[e + 1]:
                y[b[e]:b[e + 1]] = (_rows_of(st, "x", e, div, f32) @ st["w"][e].to(f32).t()).to(y.dtype)
        return y
    dx, dw = torch.zeros_like(st["dx"]), torch.zeros_like(st["dw"])
    for e in range(E):
        if b[e] < b[e + 1]:
            dy = st["dy"][b[e]:b[e + 1]].to(f32)
            dx[b[e]:b[e + 1]] = (dy @ st["w"][e].to(f32)).to(dx.dtype)
            dw[e] = (dy.t() @ _rows_of(st, "x", e, div, f32)).to(dw.dtype)
    return [dx, dw]


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "swiglu":
        I = case["I"]
        outs = []
        # row blocks: the 64-bit temporaries of a long batch need not live together
        for r in range(0, case["rows"], 1024):
            gu = st["gu"][r:r + 1024].to(f64)
            g, u = gu[:, :I], gu[:, I:]
            sg = torch.sigmoid(g)
            if not case["grad"]:
                outs.append((g * sg * u,))
                continue
            dh = st["dh"][r:r + 1024].to(f64)
            dg = dh * u * (sg + g * sg * (1 - sg))
            outs.append((torch.cat([dg, dh * (g * sg)], dim=1), g * sg * u))
        cols = [torch.cat(c) for c in zip(*outs)]
        return cols if case["grad"] else cols[0]
    if op == "combine_grad":
        T, k, H, E = case["T"], case["k"], case["H"], case["E"]
        dy = torch.zeros((T * k, H), device="cuda", dtype=f64)
        dw = torch.zeros((T, k), device="cuda", dtype=f64)
        dlogits = torch.zeros((T, E), device="cuda", dtype=f64)
        inv = st["inv"].view(T, k).long()
        d, w = st["dout"].to(f64), st["w"].to(f64)
        for j in range(k):
            t = torch.nonzero(inv[:, j] >= 0)[:, 0]
            p = inv[t, j]
            dy[p] = w[t, j, None] * d[t]
            dw[t, j] = (st["y"][p].to(f64) * d[t]).sum(dim=1)
        mean = (w * dw).sum(dim=1)
        for j in range(k):
            t = torch.nonzero(inv[:, j] >= 0)[:, 0]
            dlogits[t, st["ids"][t, j].long()] = w[t, j] * (dw[t, j] - mean[t])
        return [dy, dw, dlogits]
    T, k, E, N, K = case["T"], case["k"], case["E"], case["N"], case["K"]
    token = st["perm"].long() // k
    if op == "int8":
        x = st["x"].to(f64)
        if case["act"] == "swiglu":
            x = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:]
        top = x.abs().max(dim=1).values
        # the integers nearest to 127 x / max |x| (halves to the even one), the scale max |x| / 127
        q = torch.where(top[:, None] > 0, torch.round(127 * x / top[:, None]), torch.zeros_like(x))
        if case["act"] == "none":
            q, top = q[token], top[token]
        y = torch.zeros(st["y"].shape, device="cuda", dtype=f64)
        for e in range(E):
            r = slice(st["bounds"][e], st["bounds"][e + 1])
            y[r] = torch.mm(q[r], st["w"][e].to(f64).t()) * (top[r, None] / 127) * st["w_scale"][e].to(f64)
        return y
    x = st["x"].to(f64)
    if case["gather"]:
        x = x[token]
    if op == "product":
        y = torch.zeros(st["y"].shape, device="cuda", dtype=f64)
        for e in range(E):
            r = slice(st["bounds"][e], st["bounds"][e + 1])
            y[r] = torch.mm(x[r], st["w"][e].to(f64).t())
        return y
    dx = torch.zeros(st["dx"].shape, device="cuda", dtype=f64)
    dw = torch.zeros(st["dw"].shape, device="cuda", dtype=f64)
    for e in range(E):
        r = slice(st["bounds"][e], st["bounds"][e + 1])
        dy = st["dy"][r].to(f64)
        dx[r] = torch.mm(dy, st["w"][e].to(f64))
        dw[e] = torch.mm(dy.t(), x[r])
    return [dx, dw]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "swiglu":
        n, b = case["rows"] * case["I"], BYTES[case["dt"]]
        # forward: g, u in, h out; gradient: g, u, dh in, dg, du, h out
        return {"bytes": n * b * (6 if case["grad"] else 3), "flops": n * (20 if case["grad"] else 8)}
    if op == "combine_grad":
        T, k, E, H = case["T"], case["k"], case["E"], case["H"]
        pairs = T * k * (1 - case["drop"])
        return {"bytes": int(T * H * BYTES[case["dt"]] + pairs * H * (4 + BYTES[case["dy"]]) + T * k * 16 + T * E * 4),
                "flops": int(3 * pairs * H)}
    T, k, E, N, K = case["T"], case["k"], case["E"], case["N"], case["K"]
    offsets, _ = _group(_route(T, k, E, case["zipf"], 0), E)
    touched, P = int((np.diff(offsets) > 0).sum()), T * k
    macs = P * N * K
    if op == "int8":
        x = T * K if case["act"] == "none" else P * 2 * K
        return {"bytes": x * BYTES[case["dt"]] + touched * N * (K + 4) + P * N * BYTES[case["out"]], "flops": 2 * macs}
    b = BYTES[case["dt"]]
    x = (T if case["gather"] else P) * K * b
    if op == "product":
        return {"bytes": x + touched * N * K * b + P * N * BYTES[case["out"]], "flops": 2 * macs}
    return {"bytes": x + P * N * b + touched * N * K * b + P * K * BYTES[case["out"]] + E * N * K * BYTES[case["dw"]],
            "flops": 4 * macs}
