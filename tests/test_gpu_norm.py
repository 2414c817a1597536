"""Layer and RMS norm of rows with their gradients, and the norm and clipping of gradients, against 64-bit references."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mixture_experts_layer_token_amd as moe  # noqa: E402

from grouped_ref import HALF_STEP, f64  # noqa: E402
from helpers import say  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


SENTINEL = 12345.0
DTS = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24  # half a step of fp32

SIZES = [(1, 1), (3, 7), (1, 8), (5, 9), (2, 64), (130, 65), (33, 512), (40, 513), (700, 768), (300, 1025), (257, 2048),
         (1, 2880), (517, 2880), (64, 4095), (64, 4096), (30, 4097), (1, 7168), (600, 7168), (9, 8192), (20, 8193), (300, 16384),
         (5, 16385), (3, 40000), (2, 70001)]


def adds(H):
    """Additions on the way of any element of a row into its sum: 8 per chunk of a lane, six in the wave, 16 waves."""
    return 8 * math.ceil(H / 8192) + 30


def strided(shape, dt, pad, off, gen, mean=0.0):
    full = (torch.randn((shape[0], shape[1] + pad), generator=gen, device="cuda") + mean).to(dt)
    return full[:, off:off + shape[1]]


def make(rows, H, dt, pdt, bias=True, weight=True, pad=0, off=0, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3000 + seed)
    x = strided((rows, H), dt, pad, off, gen, 0.7)
    dy = strided((rows, H), dt, pad, off, gen)
    add = torch.randn((rows, H), generator=gen, device="cuda").to(dt)
    w = (1 + 0.3 * torch.randn(H, generator=gen, device="cuda")).to(pdt) if weight else None
    b = torch.randn(H, generator=gen, device="cuda").to(pdt) if bias else None
    return x, dy, add, w, b


def within(got, value, bound, what):
    bad = ~((f64(got) - value).abs() <= bound)
    assert not bad.any(), "%s: %d of %d off, first at %s: got %r, want %r, bound %.3e" % (
        what, int(bad.sum()), bad.numel(), tuple(torch.nonzero(bad)[0].tolist()), float(f64(got)[bad][0]),
        float(value[bad][0]), float(bound[bad][0]))


def check_forward(x, w, b, eps, rms, y, stats, what=""):
    dt, H, n = y.dtype, x.shape[1], adds(x.shape[1])
    moe.moe_norm(x, w, b, y, eps=eps, rms=rms, stats=stats)
    torch.cuda.synchronize()
    X = f64(x)
    mean = torch.zeros_like(X[:, :1]) if rms else X.mean(1, keepdim=True)
    d = X - mean
    var = (d * d).mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    # the mean's error, then the deviations', the variance's and the root's
    em = torch.zeros_like(mean) if rms else (n + 2) * U * X.abs().mean(1, keepdim=True)
    ed = em + U * (d.abs() + em)
    ev = (2 * ed * d.abs() + ed * ed).mean(1, keepdim=True) + (n + 3) * U * var
    # (where eps is smaller than the variance's error, 1 / sqrt has no useful first order: such rows are constant ones)
    er = rstd * (0.5 * ev / (var + eps).clamp(min=1e-300) * (1 + ev / (var + eps).clamp(min=1e-300)) + 4 * U)
    W = torch.ones(H, dtype=torch.float64) if w is None else f64(w)
    B = torch.zeros(H, dtype=torch.float64) if b is None else f64(b)
    y_ref = d * rstd * W + B
    e = W.abs() * (ed * (rstd + er) + d.abs() * er) + 3 * U * ((d * rstd * W).abs() + B.abs())
    within(y, y_ref, e + HALF_STEP[dt] * (y_ref.abs() + e) + 1e-37, "y " + what)
    if stats is not None:
        within(stats[:, :1], mean, em + 2 * U * mean.abs() + 1e-37, "mean " + what)
        within(stats[:, 1:], rstd, er + U * rstd, "rstd " + what)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dt,pdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,H", SIZES)
def test_forward(rows, H, dt, pdt, rms):
    say("norm", rows, H, dt, pdt, "rms", rms)
    x, _, _, w, b = make(rows, H, DTS[dt], DTS[pdt], bias=not rms)
    full = torch.full((rows + 2, H), SENTINEL, device="cuda", dtype=DTS[dt])
    stats = torch.full((rows, 2), SENTINEL, device="cuda")
    check_forward(x, w, b, 1e-5, rms, full[1:-1], stats)
    assert (full[0] == full[-1]).all() and (full[0].float() == torch.tensor(SENTINEL, dtype=DTS[dt]).float().cuda()).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("pad,off", [(8, 0), (3, 1), (1, 0)])
@pytest.mark.parametrize("rows,H", [(7, 9), (130, 64), (41, 2880), (20, 4095), (6, 7168), (3, 16400)])
def test_forward_strides(rows, H, dt, pad, off):
    x, _, _, w, b = make(rows, H, DTS[dt], DTS[dt], pad=pad, off=off, seed=1)
    full = torch.full((rows, H + pad), SENTINEL, device="cuda", dtype=DTS[dt])
    y = full[:, off:off + H]
    check_forward(x, w, b, 1e-6, False, y, None)
    keep = torch.ones_like(full, dtype=torch.bool)
    keep[:, off:off + H] = False
    assert (full[keep].float() == torch.tensor(SENTINEL, dtype=DTS[dt]).float().cuda()).all()
    check_forward(x, None, b, 1e-6, False, y, None)
    check_forward(x, None, None, 1e-6, True, y, None)


def grad_reference(dy, x, w, stats, add, rms):
    X, D, S = f64(x), f64(dy), f64(stats)
    mean, rstd = S[:, :1] * (0 if rms else 1), S[:, 1:]
    H, n = X.shape[1], adds(X.shape[1])
    W = torch.ones(H, dtype=torch.float64) if w is None else f64(w)
    xh = (X - mean) * rstd
    v = D * W
    m1 = torch.zeros_like(mean) if rms else v.mean(1, keepdim=True)
    m2 = (v * xh).mean(1, keepdim=True)
    e1 = torch.zeros_like(mean) if rms else (n + 3) * U * v.abs().mean(1, keepdim=True)
    e2 = (n + 6) * U * (v * xh).abs().mean(1, keepdim=True)
    A = torch.zeros_like(X) if add is None else f64(add)
    dx = rstd * (v - m1 - xh * m2) + A
    ex = rstd * (e1 + xh.abs() * e2 + 6 * U * (v.abs() + m1.abs() + (xh * m2).abs())) + 2 * U * (dx.abs() + A.abs())
    rows = X.shape[0]
    dw, db = (D * xh).sum(0), D.sum(0)
    ew, eb = (rows + 40) * U * (D * xh).abs().sum(0), (rows + 40) * U * D.abs().sum(0)
    return (dx, ex), (dw, ew), (db, eb)


def check_gradient(x, dy, add, w, pdt, rms, ws=None, with_bias=True, with_weight=True, what=""):
    rows, H = x.shape
    dt = x.dtype
    X = f64(x)
    mean = X.mean(1) * (0 if rms else 1)
    stats = torch.stack([mean, ((X - mean[:, None]) ** 2).mean(1).add(1e-5) ** -0.5], 1).float().cuda()
    full = torch.full((rows + 2, H), SENTINEL, device="cuda", dtype=dt)
    dx = full[1:-1]
    dw = torch.full((H,), SENTINEL, device="cuda", dtype=pdt) if with_weight else None
    db = torch.full((H,), SENTINEL, device="cuda", dtype=pdt) if with_bias else None
    moe.moe_norm_grad(dy, x, w, stats, dx, dweight=dw, dbias=db, add=add, rms=rms, ws=ws)
    torch.cuda.synchronize()
    for got, (ref, e), name in zip((dx, dw, db), grad_reference(dy, x, w, stats, add, rms), ("dx", "dweight", "dbias")):
        if got is not None:
            within(got, ref, e + HALF_STEP[got.dtype] * (ref.abs() + e) + 1e-37, name + " " + what)
    assert (full[0].float() == torch.tensor(SENTINEL, dtype=dt).float().cuda()).all() and (full[0] == full[-1]).all()
    return dx.clone(), dw, db


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dt,pdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,H", SIZES)
def test_gradient(rows, H, dt, pdt, rms):
    say("norm gradient", rows, H, dt, pdt, "rms", rms)
    x, dy, add, w, _ = make(rows, H, DTS[dt], DTS[pdt], seed=2)
    check_gradient(x, dy, add if rows % 2 else None, w, DTS[pdt], rms, with_bias=not rms)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("pad,off", [(8, 0), (3, 1), (1, 0)])
@pytest.mark.parametrize("rows,H", [(7, 9), (130, 64), (41, 2880), (20, 4095), (6, 7168), (3, 16400)])
def test_gradient_strides_and_parts(rows, H, dt, pad, off):
    say("norm gradient strided", rows, H, dt, pad, off)
    x, dy, add, w, _ = make(rows, H, DTS[dt], torch.float32, pad=pad, off=off, seed=3)
    whole = check_gradient(x, dy, add, w, torch.float32, False)
    only_w = check_gradient(x, dy, add, w, torch.float32, False, with_bias=False)
    only_b = check_gradient(x, dy, add, w, torch.float32, False, with_weight=False)
    neither = check_gradient(x, dy, add, w, torch.float32, False, with_weight=False, with_bias=False)
    for other in (only_w, only_b, neither):
        for p, q in zip(whole, other):
            assert q is None or torch.equal(p, q)
    check_gradient(x, dy, None, None, torch.float32, False)


def test_gradient_of_no_rows_is_zero():
    for H in (64, 20000):
        x, dy, _, w, b = make(0, H, torch.bfloat16, torch.bfloat16)
        dw, db = torch.full_like(w, 5.0), torch.full_like(b, 5.0)
        moe.moe_norm_grad(dy, x, w, torch.empty((0, 2), device="cuda"), torch.empty_like(x), dweight=dw, dbias=db)
        moe.moe_norm(x, w, b, torch.empty_like(x))
        torch.cuda.synchronize()
        assert (dw == 0).all() and (db == 0).all()


def test_residual_gradient_added_in_place():
    x, dy, add, w, _ = make(200, 1000, torch.bfloat16, torch.bfloat16, seed=4)
    stats = torch.stack([x.float().mean(1), (x.float().var(1, correction=0) + 1e-5).rsqrt()], 1)
    dx = torch.empty_like(add)
    moe.moe_norm_grad(dy, x, w, stats, dx, add=add)
    moe.moe_norm_grad(dy, x, w, stats, add, add=add)
    torch.cuda.synchronize()
    assert torch.equal(dx, add)


def test_rows_that_are_not_finite_stay_alone():
    for H in (300, 7168, 17000):
        x, dy, _, w, b = make(40, H, torch.float32, torch.float32, seed=5)
        y, y2, dx, dx2 = (torch.empty_like(x) for _ in range(4))
        st, st2 = (torch.empty((40, 2), device="cuda") for _ in range(2))
        moe.moe_norm(x, w, b, y, stats=st)
        moe.moe_norm_grad(dy, x, w, st, dx)
        x[3, H - 1], x[17, 0], x[20] = float("nan"), float("inf"), float("-inf")
        moe.moe_norm(x, w, b, y2, stats=st2)
        moe.moe_norm_grad(dy, x, w, st2, dx2)
        torch.cuda.synchronize()
        keep = torch.ones(40, dtype=torch.bool, device="cuda")
        keep[[3, 17, 20]] = False
        for p, q in ((y, y2), (st, st2), (dx, dx2)):
            assert torch.equal(p[keep], q[keep])
        for r in (3, 17, 20):
            assert not torch.isfinite(y2[r]).any() or r == 17  # (an infinity of a row: its rstd is 0 or NaN)
            assert not torch.isfinite(dx2[r]).all()


def test_constant_rows_and_large_offsets():
    """A row of one value: its deviations are zeros (or the rounding of the mean), so y is the bias; a far mean does not spoil
    the variance, which a difference of squares would."""
    H = 4096
    x = torch.full((2, H), 3.0, device="cuda")
    x[1] = 1e4 + torch.linspace(-1, 1, H, device="cuda")
    w, b, y = torch.ones(H, device="cuda"), torch.randn(H, device="cuda"), torch.empty((2, H), device="cuda")
    moe.moe_norm(x, w, b, y, eps=1e-5)
    torch.cuda.synchronize()
    assert (y[0] - b).abs().max() <= 1e-3
    X = f64(x[1])
    want = (X - X.mean()) / (X.var(correction=0) + 1e-5).sqrt() + f64(b)
    # the mean of 1e4 is off by (n + 2) 2^-24 of it at most, against deviations of 0.58
    assert (f64(y[1]) - want).abs().max() <= (adds(H) + 3) * U * 1e4 / 0.5 * 2


def test_norm_refusals():
    x = torch.zeros((4, 32), device="cuda")
    w, y, st = torch.ones(32, device="cuda"), torch.empty_like(x), torch.zeros((4, 2), device="cuda")
    ok = dict(x=x, weight=w, bias=w, y=y, stats=st, eps=1e-5)
    for bad in (dict(x=x[0]), dict(y=y[:3]), dict(y=y.bfloat16()), dict(weight=w[:31]), dict(bias=w.bfloat16()), dict(stats=st[:3]),
                dict(stats=st.double()), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=x.t()), dict(x=x.cpu()),
                dict(x=x[:1].expand(4, 32)), dict(x=x.double(), y=y.double()), dict(weight=w.cpu())):
        a = dict(ok, **bad)
        with pytest.raises((ValueError, TypeError, AssertionError, moe.MoeError)):
            moe.moe_norm(a["x"], a["weight"], a["bias"], a["y"], eps=a["eps"], stats=a["stats"])
    ok = dict(dy=x, x=x, weight=w, stats=st, dx=y, dweight=w, dbias=w, add=None, ws=None)
    for bad in (dict(dy=x[:3]), dict(dx=y[:3]), dict(dx=y.bfloat16()), dict(dweight=w[:31]), dict(dbias=w.bfloat16()), dict(stats=None),
                dict(stats=st[:3]), dict(add=x[:3]), dict(add=x.bfloat16()), dict(ws=torch.empty(255, dtype=torch.uint8, device="cuda")),  # (256 = one part of 2 x 32 fp32)
                dict(dx=torch.empty((4, 40), device="cuda")[:, :32])):
        a = dict(ok, **bad)
        with pytest.raises((ValueError, TypeError, AssertionError, AttributeError, moe.MoeError)):
            moe.moe_norm_grad(a["dy"], a["x"], a["weight"], a["stats"], a["dx"], dweight=a["dweight"], dbias=a["dbias"],
                              add=a["add"], ws=a["ws"])


# ------------------------------------------------------------------ norm and clipping of gradients
LISTS = {
    "one": [1],
    "empty-among": [0, 5, 0, 8192, 3],
    "chunks": [8191, 8192, 8193, 16384, 16385, 1, 100000],
    "sixteen-chunks": [2048] * 10 + [2047, 4095, 1, 0, 7, 2048],
    "seventeen-chunks": [2048] * 15 + [2049],
    "many": [1 + (i * 7919) % 3000 for i in range(250)],
    "large": [30_000_001, 5, 7_000_000],
    "none": [],
    "all-empty": [0, 0],
}


def gradients(sizes, types, seed=0, shift=0, sigma=1e-2):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4000 + seed)
    out = []
    for i, n in enumerate(sizes):
        dt = DTS[types] if types in DTS else (torch.float32 if i % 3 == 0 else torch.bfloat16)
        out.append((torch.randn(n + shift, generator=gen, device="cuda") * sigma).to(dt)[shift:])
    return out


def expected(grads):
    return math.sqrt(sum(float((f64(g) ** 2).sum()) for g in grads))


def check_clipped(grads, outs, norm, max_norm, total):
    assert abs(float(norm) - total) <= U * total * 1.01
    scale = min(1.0, max_norm / total) if total > 0 else 1.0
    for g, o in zip(grads, outs):
        want = f64(g) * scale
        # the scale's rounding, the product's, and the result's
        e = 2.01 * U * want.abs()
        within(o, want, e + HALF_STEP[o.dtype] * (want.abs() + e) + 1e-37 if scale != 1.0 else torch.zeros_like(want), "clipped")


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("types", ["bf16", "f32", "mixed"])
@pytest.mark.parametrize("name", list(LISTS))
def test_clip(name, types, shift):
    say("clip", name, types, shift)
    grads = gradients(LISTS[name], types, shift=shift)
    total = expected(grads)
    norm = torch.full((1,), SENTINEL, device="cuda")
    moe.moe_grad_norm(grads, norm)
    torch.cuda.synchronize()
    assert abs(float(norm) - total) <= U * total * 1.01
    for max_norm in (0.3 * total if total else 1.0, 3.0 * total + 1.0):
        outs = [torch.full_like(g, SENTINEL) for g in grads]
        moe.moe_clip_grad_norm(grads, max_norm, norm, outs=outs)
        torch.cuda.synchronize()
        check_clipped(grads, outs, norm, max_norm, total)
        own = [g.clone() for g in grads]
        moe.moe_clip_grad_norm(own, max_norm, norm)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(own, outs))


def test_clip_into_views_leaves_the_gaps():
    grads = gradients([1000, 333, 9001], "bf16", seed=1)
    flat = torch.full((20000,), SENTINEL, device="cuda", dtype=torch.bfloat16)
    outs = [flat[5:1005], flat[2000:2333], flat[3000:12001]]
    norm = torch.empty(1, device="cuda")
    moe.moe_clip_grad_norm(grads, 0.01, norm, outs=outs)
    torch.cuda.synchronize()
    check_clipped(grads, outs, norm, 0.01, expected(grads))
    s = torch.tensor(SENTINEL, dtype=torch.bfloat16, device="cuda")
    for lo, hi in ((0, 5), (1005, 2000), (2333, 3000), (12001, 20000)):
        assert (flat[lo:hi] == s).all()


def test_only_some_results_and_dense_layouts():
    grads = gradients([600, 601, 602], "f32", seed=2)
    keep = grads[1].clone()
    out = torch.empty_like(grads[0])
    norm = torch.empty(1, device="cuda")
    moe.moe_clip_grad_norm(grads, 1e-3, norm, outs=[out, None, grads[2]])
    torch.cuda.synchronize()
    assert torch.equal(grads[1], keep)
    turned = torch.randn((30, 50), device="cuda").t()
    ref = f64(turned)
    moe.moe_clip_grad_norm([turned], 1.0, norm)
    torch.cuda.synchronize()
    total = float(ref.norm())
    assert abs(float(norm) - total) <= 1.01 * U * total
    assert torch.allclose(f64(turned), ref / total, rtol=3 * U, atol=0)


def test_extreme_values():
    """Squares past the fp32 range on both sides, and a norm that fp32 holds."""
    norm = torch.empty(1, device="cuda")
    for v in (1e30, 1e-30, 3e38):
        g = torch.full((10000,), v, device="cuda")
        moe.moe_grad_norm([g], norm)
        torch.cuda.synchronize()
        want = f64(g).norm()
        assert (abs(float(norm) - float(want)) <= 2 * U * float(want)) if want < 3.4e38 else math.isinf(float(norm))
    g = torch.full((10000,), 3e38, device="cuda")  # the norm passes the fp32 range, not the sum of squares
    moe.moe_clip_grad_norm([g], 1.0, norm)
    torch.cuda.synchronize()
    assert torch.allclose(g, torch.full_like(g, 0.01), rtol=4 * U, atol=0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_norm_that_is_not_finite_scales_nothing(bad):
    grads = gradients([5000, 70], "bf16", seed=3)
    grads[1][69] = bad
    keep = [g.clone() for g in grads]
    outs = [torch.zeros_like(g) for g in grads]
    norm = torch.empty(1, device="cuda")
    moe.moe_clip_grad_norm(grads, 1e-3, norm, outs=outs)
    moe.moe_clip_grad_norm(grads, 1e-3, norm)
    torch.cuda.synchronize()
    assert not math.isfinite(float(norm))
    for g, o, k in zip(grads, outs, keep):
        assert torch.equal(g.view(torch.int16), k.view(torch.int16)) and torch.equal(o.view(torch.int16), k.view(torch.int16))


def test_overlaps_and_other_refusals():
    g = torch.randn(1000, device="cuda")
    norm = torch.empty(1, device="cuda")
    for grads, outs in (([g, g], None), ([g[:600], g[500:]], None), ([g[:500]], [g[1:501]]), ([g[:400], g[400:800]], [g[400:800], g[:400]]),
                        ([g[:500], g[500:]], [torch.empty(500, device="cuda")] * 2)):
        with pytest.raises(moe.MoeError):
            moe.moe_clip_grad_norm(grads, 1.0, norm, outs=outs)
    moe.moe_grad_norm([g, g], norm)  # (nothing is written: counted twice)
    torch.cuda.synchronize()
    assert abs(float(norm) - float(f64(g).norm()) * 2 ** 0.5) <= 2 * U * float(norm)
    for m in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(moe.MoeError):
            moe.moe_clip_grad_norm([g], m, norm)
    for bad in (dict(norm=norm.double()), dict(norm=torch.empty(2, device="cuda")), dict(grads=[g.cpu()]), dict(grads=[g.half()]),
                dict(grads=[g[::2]]), dict(outs=[g.bfloat16()]), dict(outs=[g[:5]]), dict(outs=[]), dict(grads=[g.view(10, 100)[:, :50]]),
                dict(ws=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        a = dict(dict(grads=[g], outs=None, norm=norm, ws=None), **bad)
        with pytest.raises((ValueError, TypeError, AssertionError, moe.MoeError)):
            moe.moe_clip_grad_norm(a["grads"], 1.0, a["norm"], outs=a["outs"], ws=a["ws"])


def test_captured_norm_gradient_and_clip_replay():
    """The three of them in one graph, replayed with eager work between the replays."""
    x, dy, add, w, b = make(700, 1000, torch.bfloat16, torch.bfloat16, seed=6)

    def step():
        y, dx = torch.empty_like(x), torch.empty_like(x)
        stats = torch.empty((700, 2), device="cuda")
        dw, db = torch.empty_like(w), torch.empty_like(b)
        norm = torch.empty(1, device="cuda")
        moe.moe_norm(x, w, b, y, stats=stats)
        moe.moe_norm_grad(dy, x, w, stats, dx, dweight=dw, dbias=db, add=add)
        outs = [torch.empty_like(t) for t in (dx, dw, db)]
        moe.moe_clip_grad_norm([dx, dw, db], 0.5, norm, outs=outs)
        return [y, stats, norm] + outs

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for rep in range(4):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), rep
        step()
        torch.cuda.synchronize()


def test_side_stream():
    x, dy, _, w, b = make(300, 2880, torch.bfloat16, torch.bfloat16, seed=7)
    side = torch.cuda.Stream()
    res = []
    for stream in (None, side):
        y, dx, st = torch.empty_like(x), torch.empty_like(x), torch.empty((300, 2), device="cuda")
        dw, db, norm = torch.empty_like(w), torch.empty_like(b), torch.empty(1, device="cuda")
        torch.cuda.synchronize()
        moe.moe_norm(x, w, b, y, stats=st, stream=stream)
        moe.moe_norm_grad(dy, x, w, st, dx, dweight=dw, dbias=db, stream=stream)
        moe.moe_clip_grad_norm([dw, db, dx], 0.1, norm, stream=stream)
        torch.cuda.synchronize()
        res.append([y, dx, st, dw, db, norm])
    assert all(torch.equal(p, q) for p, q in zip(*res))
