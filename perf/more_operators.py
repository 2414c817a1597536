"""What the operators of a training step around the layer compute, at sizes of real use, for timing and comparison.

Operators: the gated feed-forward block grouped by expert (both projections, the activation and the product in one
call) and the gradient that reaches its projections from behind the down matrices; layer and RMS norm with their
gradients, the weight's and the bias' among them; the global norm of many gradients, and their clipping.

`run` computes them in plain torch operations in 32 bits, or, where `own` is true, through the package.
Sizes follow the repository's layers: H = 4096, I = 14336, E = 8, k = 2 (bf16 experts); H = I = 2880,
E = 128, k = 4 with a skewed expert popularity; H = 7168, I = 2048, E = 384, k = 8.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-5

# the largest listed cases: multiply-adds and weights of a block, elements of a norm
MAX_MACS = 8192 * 28672 * 4096
MAX_WEIGHTS = 8 * 28672 * 4096
MAX_NORM = 8192 * 7168


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token through the gate and up matrices of its 4 experts: the smallest call of the block
        dict(name="block-decode", op="block", dt="bf16", T=1, k=4, E=128, I=2880, K=2880, zipf=1.1, gather=True,
             keep=False, spare=0),
        # a serving batch over 128 experts of very uneven popularity
        dict(name="block-ragged", op="block", dt="bf16", T=509, k=4, E=128, I=2880, K=2880, zipf=1.1, gather=True,
             keep=False, spare=0),
        # a training batch through wide gate and up matrices, their results kept for the backward pass: the largest call
        dict(name="block-train", op="block", dt="bf16", T=4096, k=2, E=8, I=14336, K=4096, zipf=0.0, gather=True,
             keep=True, spare=0),
        # the block's backward pass from the rows behind the down matrices: a fine-tuning batch, and a training step
        dict(name="block-grad-small", op="block_grad", dt="bf16", T=131, k=8, E=32, I=2048, H=7168, zipf=0.5, spare=0),
        dict(name="block-grad-train", op="block_grad", dt="bf16", T=3001, k=2, E=8, I=14336, H=4096, zipf=0.3, spare=0),
        # the norm before the layer: one decoded token, and a training batch whose statistics are kept
        dict(name="norm-decode", op="norm", dt="bf16", rows=1, H=7168, rms=True, bias=False, stats=False),
        dict(name="norm-train", op="norm", dt="bf16", rows=8192, H=7168, rms=False, bias=True, stats=True),
        # its backward pass: a fine-tuning batch of odd length; a training step, with the residual's gradient added
        dict(name="norm-grad-small", op="norm_grad", dt="bf16", rows=517, H=2880, rms=True, bias=False, add=False),
        dict(name="norm-grad-train", op="norm_grad", dt="bf16", rows=8192, H=7168, rms=False, bias=True, add=True),
        # clipping: the gradients of a small fp32 layer; of a stack of layers, large and small tensors and both types; of
        # the expert matrices of a wide layer
        dict(name="clip-small", op="clip", dt="f32", tensors=5, total=1 << 17, spread=2.0, shapes=1, ratio=0.7),
        dict(name="clip-stack", op="clip", dt="mixed", tensors=193, total=150_000_001, spread=2.5, shapes=2, ratio=0.3),
        dict(name="clip-experts", op="clip", dt="bf16", tensors=3, total=1 << 30, spread=1.0, shapes=3, ratio=0.1),
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
    op = rng.choice(["block", "block", "block_grad", "block_grad", "norm", "norm_grad", "norm_grad", "clip"])
    if op in ("norm", "norm_grad"):
        while True:
            case = dict(op=op, dt=rng.choice(["bf16", "bf16", "f32"]), rows=_log(rng, 1, 16384), H=_width(rng, 32, 16384),
                        rms=rng.random() < 0.5)
            case["bias"] = not case["rms"] and rng.random() < 0.8
            case["stats" if op == "norm" else "add"] = rng.random() < 0.5
            if case["rows"] * case["H"] * BYTES[case["dt"]] <= MAX_NORM * 2:
                return case
    if op == "clip":
        return dict(op=op, dt=rng.choice(["bf16", "f32", "mixed"]), tensors=_log(rng, 1, 300), total=_log(rng, 1000, 1 << 28),
                    spread=rng.choice([0.5, 1.5, 2.5]), shapes=rng.randint(0, 1 << 30), ratio=rng.choice([0.1, 0.6, 2.0]))
    while True:
        E = _log(rng, 1, 256)
        case = dict(op=op, dt=rng.choice(["bf16", "bf16", "bf16", "f32"]), T=_log(rng, 1, 4096),
                    k=rng.randint(1, min(8, E)), E=E, I=_width(rng, 32, 8192), zipf=rng.choice([0.0, 0.5, 1.1]),
                    spare=rng.choice([0, 0, 7]))
        case["K" if op == "block" else "H"] = width = _width(rng, 32, 8192)
        if op == "block":
            case["gather"], case["keep"] = rng.random() < 0.6, rng.random() < 0.5
        # fp32 products run at about a tenth of the rate of the bf16 ones
        cells = (2 if op == "block" else 1) * case["I"] * width
        macs = case["T"] * case["k"] * cells * (10 if case["dt"] == "f32" else 1)
        if macs <= MAX_MACS and E * cells * 2 <= MAX_WEIGHTS:
            return case


def _sizes(case):
    """Elements of each gradient: log-normal shares of the total, at least one element each."""
    rng = random.Random(case["shapes"])
    share = [math.exp(rng.gauss(0.0, case["spread"])) for _ in range(case["tensors"])]
    scale = case["total"] / sum(share)
    return [max(1, int(s * scale)) for s in share]


def _types(case):
    """Types of the gradients: one for all, or every third in fp32 (norms, biases and routers among bf16 matrices)."""
    if case["dt"] == "mixed":
        return ["f32" if i % 3 == 0 else "bf16" for i in range(case["tensors"])]
    return [case["dt"]] * case["tensors"]


def _places(case):
    """Type, place in the flat buffer of that type (a multiple of 128 elements) and length of each gradient; and the
    buffers' lengths."""
    places, lengths = [], {}
    for n, t in zip(_sizes(case), _types(case)):
        at = lengths.get(t, 0)
        places.append((t, at, n))
        lengths[t] = at + (n + 127) // 128 * 128
    return places, lengths


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
    op = case["op"]
    if op == "clip":
        # the clipped gradients go into one flat buffer for each type, the way an optimizer's program may hold them
        places, lengths = _places(case)
        st["grads"] = [_normal(gen, (n,), 1e-3, DT[t]) for t, _, n in places]
        st["flat"] = {t: torch.zeros(n, device="cuda", dtype=DT[t]) for t, n in lengths.items()}
        st["outs"] = [st["flat"][t][at:at + n] for t, at, n in places]
        # ratio of the limit to the norm that is expected: below 1 the gradients are scaled
        st["max_norm"] = case["ratio"] * 1e-3 * math.sqrt(sum(_sizes(case)))
        st["norm"] = torch.empty(1, device="cuda", dtype=torch.float32)
        return st
    dt = DT[case["dt"]]
    if op in ("norm", "norm_grad"):
        rows, H = case["rows"], case["H"]
        # a residual stream: features of unequal size around an offset of their own, rows of unequal size
        size = torch.exp(_normal(gen, (rows, 1), 0.5, torch.float32))
        feature = _normal(gen, (H,), 0.5, torch.float32)
        st["x"] = (_normal(gen, (rows, H), 1.0, torch.float32).mul_(size).add_(feature + 0.5)).to(dt)
        st["weight"] = _normal(gen, (H,), 0.2, torch.float32).add_(1.0).to(dt)
        st["bias"] = _normal(gen, (H,), 0.2, dt) if case["bias"] else None
        if op == "norm":
            st["y"] = torch.empty((rows, H), device="cuda", dtype=dt)
            st["stats"] = torch.empty((rows, 2), device="cuda", dtype=torch.float32) if case["stats"] else None
            return st
        st["dy"] = _normal(gen, (rows, H), 0.02, dt)
        st["add"] = _normal(gen, (rows, H), 0.02, dt) if case["add"] else None
        # the statistics that the forward pass kept
        x = st["x"].to(torch.float64)
        mean = torch.zeros(rows, device="cuda", dtype=torch.float64) if case["rms"] else x.mean(dim=1)
        var = (x - mean[:, None]).square().mean(dim=1)
        st["stats"] = torch.stack([mean, (var + EPS).rsqrt()], dim=1).to(torch.float32)
        st["dx"] = torch.empty((rows, H), device="cuda", dtype=dt)
        st["dweight"] = torch.empty(H, device="cuda", dtype=dt)
        st["dbias"] = torch.empty(H, device="cuda", dtype=dt) if case["bias"] else None
        return st
    T, k, E, I = case["T"], case["k"], case["E"], case["I"]
    offsets, perm = _group(_route(T, k, E, case["zipf"], seed), E)
    rows = T * k + case["spare"]  # room for more rows than are placed
    st["bounds"] = [int(o) for o in offsets]
    st["offsets"] = torch.from_numpy(offsets).cuda()
    st["perm"] = torch.from_numpy(np.concatenate([perm, np.zeros(case["spare"], np.int32)])).cuda()
    if op == "block":
        K = case["K"]
        st["x"] = _normal(gen, (T if case["gather"] else rows, K), 1.0, dt)
        # projections of about unit size
        st["w"] = _weights(gen, E, 2 * I, K, 1.5 / math.sqrt(K), dt)
        st["h"] = torch.zeros((rows, I), device="cuda", dtype=dt)
        st["gu"] = torch.zeros((rows, 2 * I), device="cuda", dtype=dt) if case["keep"] else None
        return st
    H = case["H"]
    st["dy"] = _normal(gen, (rows, H), 0.02, dt)
    st["w"] = _weights(gen, E, H, I, 0.02, dt)
    st["gu"] = _normal(gen, (rows, 2 * I), 1.5, dt)
    st["dgu"] = torch.zeros((rows, 2 * I), device="cuda", dtype=dt)
    st["h"] = torch.zeros((rows, I), device="cuda", dtype=dt)
    return st


# ------------------------------------------------------------------ one pass
def _some(*tensors):
    return [t for t in tensors if t is not None]


def _run_own(st):
    from mixture_experts_layer_token_amd import api

    case = st["case"]
    op = case["op"]
    if op == "block":
        gather = dict(perm_src=st["perm"], k=case["k"]) if case["gather"] else {}
        api.moe_grouped_swiglu(st["x"], st["w"], st["offsets"], st["h"], gu=st["gu"], **gather)
        return _some(st["h"], st["gu"])
    if op == "block_grad":
        api.moe_grouped_swiglu_dx(st["dy"], st["w"], st["gu"], st["offsets"], st["dgu"], h=st["h"])
        return [st["dgu"], st["h"]]
    if op == "norm":
        api.moe_norm(st["x"], st["weight"], st["bias"], st["y"], eps=EPS, rms=case["rms"], stats=st["stats"])
        return _some(st["y"], st["stats"])
    if op == "norm_grad":
        api.moe_norm_grad(st["dy"], st["x"], st["weight"], st["stats"], st["dx"], dweight=st["dweight"],
                          dbias=st["dbias"], add=st["add"], rms=case["rms"])
        return _some(st["dx"], st["dweight"], st["dbias"])
    api.moe_clip_grad_norm(st["grads"], st["max_norm"], st["norm"], outs=st["outs"])
    return [st["norm"]] + list(st["flat"].values())


def _rows_of(st, key, e, div):
    """Rows of expert e in 32 bits: the grouped rows themselves, or the tokens that perm_src names."""
    lo, hi = st["bounds"][e], st["bounds"][e + 1]
    if div:
        return st[key][torch.div(st["perm"][lo:hi], div, rounding_mode="floor").long()].to(torch.float32)
    return st[key][lo:hi].to(torch.float32)


def run(st):
    if own:
        return _run_own(st)
    case = st["case"]
    op = case["op"]
    f32 = torch.float32
    if op == "clip":
        # the sum in 64 bits: there may be 10^9 terms
        total = torch.zeros((), device="cuda", dtype=torch.float64)
        for g in st["grads"]:
            v = g.to(f32)
            total = total + (v * v).sum(dtype=torch.float64)
        norm = torch.sqrt(total)
        scale = torch.clamp(st["max_norm"] / norm, max=1.0).to(f32)
        places, lengths = _places(case)
        flat = {t: torch.zeros(n, device="cuda", dtype=DT[t]) for t, n in lengths.items()}
        for g, (t, at, n) in zip(st["grads"], places):
            flat[t][at:at + n] = (g.to(f32) * scale).to(g.dtype)
        return [norm.to(f32).view(1)] + list(flat.values())
    if op == "norm":
        x = st["x"].to(f32)
        mean = torch.zeros_like(x[:, :1]) if case["rms"] else x.mean(dim=1, keepdim=True)
        d = x - mean
        rstd = 1 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + EPS)
        y = d * rstd * st["weight"].to(f32)
        if case["bias"]:
            y = y + st["bias"].to(f32)
        return _some(y.to(st["x"].dtype), torch.cat([mean, rstd], dim=1) if case["stats"] else None)
    if op == "norm_grad":
        x, dy = st["x"].to(f32), st["dy"].to(f32)
        mean, rstd = st["stats"][:, :1], st["stats"][:, 1:]
        xh = (x - mean) * rstd
        wdy = dy * st["weight"].to(f32)
        dx = wdy - xh * (wdy * xh).mean(dim=1, keepdim=True)
        if not case["rms"]:
            dx = dx - wdy.mean(dim=1, keepdim=True)
        dx = dx * rstd
        if case["add"]:
            dx = dx + st["add"].to(f32)
        dt = st["x"].dtype
        return _some(dx.to(dt), (dy * xh).sum(dim=0).to(dt), dy.sum(dim=0).to(dt) if case["bias"] else None)
    E, I, b = case["E"], case["I"], st["bounds"]
    if op == "block":
        div = case["k"] if case["gather"] else 0
        h = torch.zeros_like(st["h"])
        kept = torch.zeros_like(st["gu"]) if case["keep"] else None
        for e in range(E):
            if b[e] < b[e + 1]:
                gu = _rows_of(st, "x", e, div) @ st["w"][e].to(f32).t()
                g, u = gu[:, :I], gu[:, I:]
                h[b[e]:b[e + 1]] = (g / (1 + torch.exp(-g)) * u).to(h.dtype)
                if case["keep"]:
                    kept[b[e]:b[e + 1]] = gu.to(kept.dtype)
        return _some(h, kept)
    dgu, h = torch.zeros_like(st["dgu"]), torch.zeros_like(st["h"])
    for e in range(E):
        if b[e] < b[e + 1]:
            r = slice(b[e], b[e + 1])
            dh = st["dy"][r].to(f32) @ st["w"][e].to(f32)
            g, u = st["gu"][r, :I].to(f32), st["gu"][r, I:].to(f32)
            s = 1 / (1 + torch.exp(-g))
            h[r] = (g * s * u).to(h.dtype)
            dgu[r] = torch.cat([dh * u * s * (1 + g * (1 - s)), dh * g * s], dim=1).to(dgu.dtype)
    return [dgu, h]


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "clip":
        # blocks of elements: the 64-bit copies of the largest tensors need not live whole
        squares = sum(float(torch.linalg.vector_norm(part.to(f64)) ** 2) for g in st["grads"] for part in g.split(1 << 26))
        norm = math.sqrt(squares)
        scale = st["max_norm"] / norm if norm > st["max_norm"] else 1.0
        out = {t: torch.zeros(f.numel(), device="cuda", dtype=f64) for t, f in st["flat"].items()}
        for g, (t, at, n) in zip(st["grads"], _places(case)[0]):
            torch.mul(g.to(f64), scale, out=out[t][at:at + n])
        return [torch.tensor([norm], device="cuda", dtype=f64)] + list(out.values())
    if op == "norm":
        x = st["x"].to(f64)
        if case["rms"]:
            mean, var = torch.zeros(x.shape[0], device="cuda", dtype=f64), x.pow(2).mean(1)
        else:
            var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + EPS).pow(-0.5)
        y = torch.addcmul(st["bias"].to(f64) if case["bias"] else torch.zeros((), device="cuda", dtype=f64),
                          (x - mean[:, None]) * rstd[:, None], st["weight"].to(f64))
        return [y, torch.stack((mean, rstd), 1)] if case["stats"] else [y]
    if op == "norm_grad":
        # the row's Jacobian rstd (1 - [1 1^T / H] - xh xh^T / H) applied to w dy
        x, dy = st["x"].to(f64), st["dy"].to(f64)
        stats = st["stats"].to(f64)
        xh = (x - stats[:, :1]).mul_(stats[:, 1:])
        del x
        dweight = torch.linalg.vecdot(dy, xh, dim=0)
        dbias = torch.ones(dy.shape[0], device="cuda", dtype=f64) @ dy
        v = dy * st["weight"].to(f64)
        dx = v - xh * (torch.linalg.vecdot(v, xh)[:, None] / case["H"])
        if not case["rms"]:
            dx -= torch.mean(v, 1, keepdim=True)
        dx *= stats[:, 1:]
        if case["add"]:
            dx += st["add"].to(f64)
        return [dx, dweight, dbias] if case["bias"] else [dx, dweight]
    E, I, rows = case["E"], case["I"], st["h"].shape[0]
    h = torch.zeros((rows, I), device="cuda", dtype=f64)
    pair = torch.zeros((rows, 2 * I), device="cuda", dtype=f64)  # [g | u], or its gradient
    for e in range(E):
        r = slice(st["bounds"][e], st["bounds"][e + 1])
        if r.start == r.stop:
            continue
        w = st["w"][e].to(f64)
        if op == "block":
            x = st["x"][st["perm"][r].long() // case["k"]] if case["gather"] else st["x"][r]
            pair[r] = torch.mm(x.to(f64), w.t())
            h[r] = pair[r, :I] * torch.sigmoid(pair[r, :I]) * pair[r, I:]
            continue
        g, u = st["gu"][r].to(f64).split(I, dim=1)
        gate = torch.sigmoid(g)
        dh = torch.mm(st["dy"][r].to(f64), w)
        h[r] = gate * g * u
        pair[r, :I] = (gate + gate * (1 - gate) * g) * u * dh
        pair[r, I:] = gate * g * dh
    if op == "block":
        return [h, pair] if case["keep"] else [h]
    return [pair, h]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "clip":
        sizes = list(zip(_sizes(case), _types(case)))
        return {"bytes": sum(2 * n * BYTES[t] for n, t in sizes) + 4, "flops": sum(3 * n for n, _ in sizes)}
    b = BYTES[case["dt"]]
    if op in ("norm", "norm_grad"):
        n, H = case["rows"] * case["H"], case["H"]
        par = H * b * (1 + case["bias"])  # weight and bias, or their gradients
        if op == "norm":
            return {"bytes": 2 * n * b + par + (8 * case["rows"] if case["stats"] else 0), "flops": 8 * n}
        return {"bytes": (3 + case["add"]) * n * b + H * b + par + 8 * case["rows"], "flops": 14 * n}
    T, k, E, I = case["T"], case["k"], case["E"], case["I"]
    offsets, _ = _group(_route(T, k, E, case["zipf"], 0), E)
    touched, P = int((np.diff(offsets) > 0).sum()), T * k
    if op == "block":
        K = case["K"]
        rows = T if case["gather"] else P
        return {"bytes": b * (rows * K + touched * 2 * I * K + P * I * (3 if case["keep"] else 1)), "flops": 4 * P * I * K}
    H = case["H"]
    return {"bytes": b * (P * H + touched * I * H + 5 * P * I), "flops": 2 * P * I * H}
