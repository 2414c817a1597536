"""The gated block grouped by expert (forward, and the gradient that reaches its projections) against 64-bit references, over
ragged groups, odd sizes, strides, gathers, wrong index tables and values that are not finite."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mixture_experts_layer_token_amd as moe  # noqa: E402

import grouped_ref as R  # noqa: E402
from grouped_ref import HALF_STEP, f64  # noqa: E402
from helpers import say  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


SENTINEL = 12345.0
DTS = {"bf16": torch.bfloat16, "f32": torch.float32}

# rows per expert, I, K (the width on the other side: K of the projections, H of the down matrix)
GROUPS = {
    "one": ([1], 1, 1),
    "tiny-odd": ([0, 0, 3], 5, 7),
    "ragged": ([17, 0, 64, 1, 130], 96, 160),
    "odd": ([65, 300, 0, 1], 131, 77),
    "by8": ([33], 40, 264),
    "by4": ([29, 150], 36, 44),
    "tiles": ([513, 255, 256, 257], 264, 200),
    "large": ([700, 1100], 1160, 648),
    "decode": ([1, 0, 2, 1, 0, 3, 9], 352, 2880),
    "decode-odd": ([1, 0, 2, 1, 0, 3, 9], 77, 1111),
    "rows64": ([64, 33, 48, 17], 48, 512),
    "many": ([i % 5 for i in range(70)], 64, 96),
    "most": ([i % 3 for i in range(1024)], 16, 32),
    "deep": ([400, 600], 128, 2048),
    # (gradients of many tiles: the ones above are few, and have a kernel of their own)
    "deep-wide": ([400, 600], 1024, 2048),
    "odd-wide": ([900, 0, 700, 131], 1131, 77),
    "by4-wide": ([640, 1111], 1132, 44),
}


def rows_tensor(shape, dt, layout, gen, sigma=1.0):
    rows, n = shape
    pad, off = {"dense": (0, 0), "padded": ((-n) % 8 + 8, 0), "shifted": (3, 1)}[layout]
    full = (torch.randn((rows, n + pad), generator=gen, device="cuda") * sigma).to(dt)
    return full[:, off:off + n]


def out_tensor(shape, dt, layout="dense"):
    rows, n = shape
    pad, off = {"dense": (0, 0), "padded": ((-n) % 8 + 8, 0), "shifted": (3, 1)}[layout]
    full = torch.full((rows, n + pad), SENTINEL, device="cuda", dtype=dt)
    return full, full[:, off:off + n]


def flat_out(shape, dt, shift):
    """A contiguous tensor that starts `shift` elements into its memory, and that memory."""
    full = torch.full((shape[0] * shape[1] + shift + 8,), SENTINEL, device="cuda", dtype=dt)
    return full, full[shift:shift + shape[0] * shape[1]].view(shape)


def make(name, dt, layout="dense", gather=False, spare=0, seed=0):
    counts, I, K = GROUPS[name]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2000 + seed)
    E, placed = len(counts), int(sum(counts))
    rows = placed + spare
    off = R.offsets_of(counts)
    k = 3 if gather else 1
    T = (rows + k - 1) // k + 1
    x = rows_tensor((T if gather else rows, K), dt, layout, gen)
    w = rows_tensor((E * 2 * I, K), dt, layout, gen, 1.5 / K ** 0.5).unflatten(0, (E, 2 * I))
    down = rows_tensor((E * K, I), dt, layout, gen, 0.1).unflatten(0, (E, K))
    dy = rows_tensor((rows, K), dt, layout, gen)
    gu = rows_tensor((rows, 2 * I), dt, "dense", gen, 1.5)
    perm = torch.randint(0, T * k, (rows,), generator=gen, device="cuda", dtype=torch.int32) if gather else None
    return dict(x=x, w=w, down=down, dy=dy, gu=gu, perm=perm, k=k, off=off, offsets=torch.from_numpy(off).cuda(), I=I, K=K,
                E=E, rows=rows, placed=placed, gather=dict(perm_src=perm, k=k) if gather else {})


def within(got, value, bound, what):
    g = f64(got)
    placed = ~torch.isnan(value)
    bad = placed & ~((g - value).abs() <= bound)
    assert not bad.any(), "%s: %d of %d off, first at %s: got %r, want %r, bound %.3e" % (
        what, int(bad.sum()), int(placed.sum()), tuple(torch.nonzero(bad)[0].tolist()), float(g[bad][0]),
        float(value[bad][0]), float(bound[bad][0]))


# Steps of an fp32 sigmoid of g: the exponent g log2(e) is rounded (|g| 2^-24 of e^-g), then exponential, sum and reciprocal, at
# most two steps of 2^-23 each.
def gate_steps(g):
    return (g.abs() + 8) * 2.0 ** -23


def forward_reference(c):
    """(h, its bound before rounding, gu, its bound) in 64 bits; rows of no group NaN."""
    xg = R.gathered(c["x"], c["perm"], c["k"], c["rows"])
    gu, mag, n = R.product("y", xg, f64(c["w"]), None, c["off"])
    acc = (n + 1) * 2.0 ** -23 * mag  # as in grouped_ref.assert_product
    I = c["I"]
    g, u = gu[:, :I], gu[:, I:]
    silu = g * torch.sigmoid(g)
    h = silu * u
    # |SiLU'| <= 1.1; the two factors' errors, their product, and the gate's own steps
    eg, eu = acc[:, :I], acc[:, I:]
    bound = 1.1 * eg * (u.abs() + eu) + silu.abs() * eu + (gate_steps(g) + 2.0 ** -22) * h.abs()
    return h, bound, gu, acc


def check_forward(c, dt, layout="dense", keep=True, shift=0, what=""):
    full, h = out_tensor((c["rows"], c["I"]), dt, layout)
    gfull, gu = flat_out((c["rows"], 2 * c["I"]), dt, shift)
    moe.moe_grouped_swiglu(c["x"], c["w"], c["offsets"], h, gu=gu if keep else None, **c["gather"])
    torch.cuda.synchronize()
    ref, bound, gref, gbound = forward_reference(c)
    half = HALF_STEP[dt]
    within(h, ref, bound + half * (ref.abs() + bound) + 1e-37, "h " + what)
    n = c["placed"]
    keepmask = torch.ones_like(full, dtype=torch.bool)
    o = h.storage_offset() % full.shape[1] if full.shape[1] else 0
    keepmask[:n, o:o + c["I"]] = False
    s = torch.tensor(SENTINEL, dtype=dt, device="cuda")
    assert (full[keepmask] == s).all(), "h wrote outside " + what
    if keep:
        within(gu, gref, gbound + half * (gref.abs() + gbound) + 1e-37, "gu " + what)
        assert (gfull[:shift] == s).all() and (gfull[shift + n * 2 * c["I"]:] == s).all(), "gu wrote outside " + what
    else:
        assert (gfull == s).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("name", list(GROUPS))
def test_forward(name, dt, keep):
    say("block forward", name, dt, "keep", keep)
    check_forward(make(name, DTS[dt]), DTS[dt], keep=keep, what=name)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("layout,spare,shift", [("padded", 7, 0), ("shifted", 5, 1), ("dense", 3, 1), ("dense", 0, 4)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("name", ["ragged", "odd", "decode", "tiles", "rows64"])
def test_forward_strides_gather_spare_rows(name, dt, gather, layout, spare, shift):
    say("block forward strided", name, dt, layout, "gather", gather, "shift", shift)
    check_forward(make(name, DTS[dt], layout, gather, spare, seed=1), DTS[dt], layout, shift=shift, what="%s %s" % (name, layout))


def gradient_reference(c):
    """(dgu, bound before rounding, h, its bound) in 64 bits."""
    dh, mag, n = R.product("dx", None, f64(c["down"]), f64(c["dy"]), c["off"])
    acc = (n + 1) * 2.0 ** -23 * mag
    I = c["I"]
    gu = f64(c["gu"])
    g, u = gu[:, :I], gu[:, I:]
    s = torch.sigmoid(g)
    q = s * (1 + g * (1 - s))
    # s is off by gate_steps of itself, so q by s (1 + |g|) as much from its factor s and s |g| as much from 1 - s
    eq = 2 * s * (1 + g.abs()) * gate_steps(g)
    h = g * s * u
    eh = (gate_steps(g) + 2.0 ** -22) * h.abs()
    dg, du = dh * u * q, dh * g * s
    edg = u.abs() * (acc * (q.abs() + eq) + dh.abs() * (eq + 2.0 ** -21 * q.abs()))
    edu = acc * (g * s).abs() * 1.01 + (gate_steps(g) + 2.0 ** -22) * du.abs()
    nan = torch.isnan(dh)
    h[nan] = float("nan")
    return torch.cat([dg, du], 1), torch.cat([edg, edu], 1), h, eh


def check_gradient(c, dt, with_h=True, shift=0, what=""):
    gfull, dgu = flat_out((c["rows"], 2 * c["I"]), dt, shift)
    hfull, h = flat_out((c["rows"], c["I"]), dt, shift)
    moe.moe_grouped_swiglu_dx(c["dy"], c["down"], c["gu"], c["offsets"], dgu, h=h if with_h else None)
    torch.cuda.synchronize()
    ref, bound, href, hbound = gradient_reference(c)
    half, n = HALF_STEP[dt], c["placed"]
    within(dgu, ref, bound + half * (ref.abs() + bound) + 1e-37, "dgu " + what)
    s = torch.tensor(SENTINEL, dtype=dt, device="cuda")
    assert (gfull[:shift] == s).all() and (gfull[shift + n * 2 * c["I"]:] == s).all(), "dgu wrote outside " + what
    if with_h:
        within(h, href, hbound + half * (href.abs() + hbound) + 1e-37, "h " + what)
        assert (hfull[:shift] == s).all() and (hfull[shift + n * c["I"]:] == s).all(), "h wrote outside " + what
    else:
        assert (hfull == s).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("with_h", [False, True])
@pytest.mark.parametrize("name", list(GROUPS))
def test_gradient(name, dt, with_h):
    say("block gradient", name, dt, "h", with_h)
    check_gradient(make(name, DTS[dt], seed=2), DTS[dt], with_h, what=name)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("layout,spare,shift", [("padded", 7, 0), ("shifted", 5, 1), ("dense", 3, 1), ("dense", 0, 4)])
@pytest.mark.parametrize("name", ["ragged", "odd", "decode", "tiles", "odd-wide", "by4-wide"])
def test_gradient_strides_spare_rows(name, dt, layout, spare, shift):
    say("block gradient strided", name, dt, layout, "shift", shift)
    check_gradient(make(name, DTS[dt], layout, False, spare, seed=3), DTS[dt], shift=shift, what="%s %s" % (name, layout))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gradient_against_differences(dt):
    """du and dg as derivatives of sum(dh * SiLU(g) u) by central differences in 64 bits."""
    c = make("ragged", DTS[dt], seed=4)
    dgu = torch.empty((c["rows"], 2 * c["I"]), device="cuda", dtype=DTS[dt])
    moe.moe_grouped_swiglu_dx(c["dy"], c["down"], c["gu"], c["offsets"], dgu)
    torch.cuda.synchronize()
    dh, _, _ = R.product("dx", None, f64(c["down"]), f64(c["dy"]), c["off"])
    gu, I, eps = f64(c["gu"]), c["I"], 1e-6
    gen = torch.Generator().manual_seed(9)
    for _ in range(4):
        v = torch.randn(gu.shape, generator=gen, dtype=torch.float64)

        def loss(s):
            t = gu + s * eps * v
            return float((dh * torch.nn.functional.silu(t[:, :I]) * t[:, I:]).sum())

        num, got = (loss(1) - loss(-1)) / (2 * eps), f64(dgu) * v
        # every element of the gradient is off by half a step of its type and the sums' own error, the differences by eps^2
        assert abs(num - float(got.sum())) <= (HALF_STEP[DTS[dt]] + 2.0 ** -16) * float(got.abs().sum()) + 1e-6


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["ragged", "odd", "tiles", "decode", "decode-odd", "odd-wide"])
def test_values_that_are_not_finite_stay_in_their_rows(name, dt):
    a = make(name, DTS[dt], spare=9, seed=5)
    b = make(name, DTS[dt], spare=9, seed=5)
    e = int(np.argmax(np.diff(a["off"])))
    lo, hi = int(a["off"][e]), int(a["off"][e + 1])
    for t in ("x", "dy", "gu"):
        b[t][lo:hi:2] = float("nan")
        b[t][lo + 1:hi:2] = float("inf")
        b[t][b["placed"]:] = float("nan")
    outs = []
    for c in (a, b):
        h, h2 = (torch.zeros((c["rows"], c["I"]), device="cuda", dtype=DTS[dt]) for _ in range(2))
        gu, dgu = (torch.zeros((c["rows"], 2 * c["I"]), device="cuda", dtype=DTS[dt]) for _ in range(2))
        moe.moe_grouped_swiglu(c["x"], c["w"], c["offsets"], h, gu=gu)
        moe.moe_grouped_swiglu_dx(c["dy"], c["down"], c["gu"], c["offsets"], dgu, h=h2)
        torch.cuda.synchronize()
        outs.append([h, gu, dgu, h2])
    keep = torch.ones(a["rows"], dtype=torch.bool, device="cuda")
    keep[lo:hi] = False
    for p, q in zip(*outs):
        assert torch.equal(p[keep], q[keep])
        assert not torch.isfinite(q[lo:hi:2].float()).any()


def test_large_gates_do_not_overflow():
    """g far out on both sides: the exponential overflows or vanishes, h and the gradients stay what they are."""
    g = torch.tensor([-1e30, -500.0, -88.0, -20.0, -0.0, 0.0, 20.0, 88.0, 500.0, 1e30])
    I = len(g)
    for dt in (torch.float32, torch.bfloat16):
        gu = torch.cat([g, torch.full((I,), 2.0)]).to(dt).cuda()[None]
        off = torch.tensor([0, 1], dtype=torch.int32).cuda()
        x, w = torch.ones((1, 1), device="cuda", dtype=dt), gu.view(1, 2 * I, 1).contiguous()
        h, h2, dgu = torch.empty((1, I), device="cuda", dtype=dt), torch.empty((1, I), device="cuda", dtype=dt), torch.empty_like(gu)
        moe.moe_grouped_swiglu(x, w, off, h)
        moe.moe_grouped_swiglu_dx(x, torch.ones((1, 1, I), device="cuda", dtype=dt), gu, off, dgu, h=h2)
        torch.cuda.synchronize()
        gd = f64(gu)[0, :I]
        s = torch.sigmoid(gd)
        want_h = gd * s * 2
        q = s * (1 + gd * (1 - s))
        tol = HALF_STEP[dt] + 2.0 ** -14
        for got, want in ((h[0], want_h), (h2[0], want_h), (dgu[0, :I], 2 * q), (dgu[0, I:], gd * s)):
            assert ((f64(got) - want).abs() <= tol * want.abs() + 1e-30).all(), (dt, got, want)


def test_wrong_tables_reach_nothing_outside():
    """Offsets that run backwards or past the rows and gathers that name no row: clamped, empty, or zeros."""
    dt = torch.bfloat16
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    rows, I, K, E = 40, 64, 96, 4
    x = torch.randn((rows, K), generator=gen, device="cuda").to(dt)
    w = torch.randn((E, 2 * I, K), generator=gen, device="cuda").to(dt) * 0.1
    down = torch.randn((E, K, I), generator=gen, device="cuda").to(dt) * 0.1
    gu = torch.randn((rows, 2 * I), generator=gen, device="cuda").to(dt)
    off = torch.tensor([-5, 10, 7, 30, 1000], dtype=torch.int32, device="cuda")  # 0..10, none, 7..30, 30..40
    clean = [(0, 0, 10), (3, 30, 40)]
    hfull, h = flat_out((rows, I), dt, 4)
    gfull, dgu = flat_out((rows, 2 * I), dt, 4)
    moe.moe_grouped_swiglu(x, w, off, h)
    moe.moe_grouped_swiglu_dx(x, down, gu, off, dgu)
    torch.cuda.synchronize()
    for e, lo, hi in clean:
        lo = max(lo, 10) if e == 0 else lo  # (rows 7..9 belong to two groups here)
        g = f64(x[lo:hi]) @ f64(w[e]).T
        want = torch.nn.functional.silu(g[:, :I]) * g[:, I:]
        assert torch.allclose(f64(h[lo:hi]), want, rtol=2.0 ** -7, atol=1e-3)
    for full in (hfull, gfull):
        assert (full[:4] == SENTINEL).all() and (full[-4:] == SENTINEL).all()
    perm = torch.tensor([-1, 5, 1 << 30, 2, -7] * 8, dtype=torch.int32, device="cuda")
    ok = torch.tensor([0, E * 10], dtype=torch.int32, device="cuda")
    h1 = torch.full((rows, I), SENTINEL, device="cuda", dtype=dt)
    moe.moe_grouped_swiglu(x, w[:1].contiguous(), ok, h1, perm_src=perm, k=2)
    torch.cuda.synchronize()
    assert (h1[[0, 2, 4]] == 0).all() and torch.equal(h1[1], h1[6]) and (h1[1] != 0).any()
    # no rows of x at all
    moe.moe_grouped_swiglu(x[:0], w[:1].contiguous(), ok, h1, perm_src=perm, k=2)
    torch.cuda.synchronize()
    assert (h1 == 0).all()
    # no grouped rows at all: nothing to do
    moe.moe_grouped_swiglu(x[:0], w, torch.zeros(E + 1, dtype=torch.int32, device="cuda"), h1[:0])
    moe.moe_grouped_swiglu_dx(x[:0], down, gu[:0], torch.zeros(E + 1, dtype=torch.int32, device="cuda"), dgu[:0])


def test_results_repeat_bit_by_bit():
    c = make("large", torch.bfloat16, seed=7)
    runs = []
    for _ in range(3):
        h, gu, dgu = (torch.empty((c["rows"], n * c["I"]), device="cuda", dtype=torch.bfloat16) for n in (1, 2, 2))
        moe.moe_grouped_swiglu(c["x"], c["w"], c["offsets"], h, gu=gu)
        moe.moe_grouped_swiglu_dx(c["dy"], c["down"], c["gu"], c["offsets"], dgu)
        torch.cuda.synchronize()
        runs.append((h, gu, dgu))
    for r in runs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(r, runs[0]))


def test_expert_strides_and_another_stream():
    """Experts and rows of w with gaps, on a side stream."""
    dt = torch.bfloat16
    c = make("ragged", dt, seed=8)
    E, I, K = c["E"], c["I"], c["K"]
    wide = torch.full((E, 2 * I + 3, K + 8), float("nan"), device="cuda", dtype=dt)
    wide[:, :2 * I, :K] = c["w"]
    wdown = torch.full((E, K + 5, I + 8), float("nan"), device="cuda", dtype=dt)
    wdown[:, :K, :I] = c["down"]
    a, b = (torch.empty((c["rows"], I), device="cuda", dtype=dt) for _ in range(2))
    p, q = (torch.empty((c["rows"], 2 * I), device="cuda", dtype=dt) for _ in range(2))
    moe.moe_grouped_swiglu(c["x"], c["w"], c["offsets"], a)
    moe.moe_grouped_swiglu_dx(c["dy"], c["down"], c["gu"], c["offsets"], p)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    moe.moe_grouped_swiglu(c["x"], wide[:, :2 * I, :K], c["offsets"], b, stream=side)
    moe.moe_grouped_swiglu_dx(c["dy"], wdown[:, :K, :I], c["gu"], c["offsets"], q, stream=side)
    side.synchronize()
    assert torch.equal(a, b) and torch.equal(p, q)


def test_rows_of_results_and_operands_far_apart():
    """Offsets past 32 bits: rows of h, and of dy, 2^24 elements apart (more than 4 GiB in all)."""
    dt = torch.bfloat16
    rows, I, K, ld = 140, 64, 64, 1 << 24
    gen = torch.Generator(device="cuda")
    gen.manual_seed(10)
    x = torch.randn((rows, K), generator=gen, device="cuda").to(dt)
    w = (torch.randn((1, 2 * I, K), generator=gen, device="cuda") * 0.2).to(dt)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    near, far = torch.empty((rows, I), device="cuda", dtype=dt), torch.empty((rows, ld), device="cuda", dtype=dt)
    moe.moe_grouped_swiglu(x, w, off, near)
    moe.moe_grouped_swiglu(x, w, off, far[:, :I])
    torch.cuda.synchronize()
    assert torch.equal(near, far[:, :I])
    far[:, :K] = x
    down, gu = w[:, :K, :I].contiguous(), torch.randn((rows, 2 * I), generator=gen, device="cuda").to(dt)
    a, b = torch.empty_like(gu), torch.empty_like(gu)
    moe.moe_grouped_swiglu_dx(x, down, gu, off, a)
    moe.moe_grouped_swiglu_dx(far[:, :K], down, gu, off, b)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_refusals_of_the_python_names():
    dt = torch.bfloat16
    x, w, off = (torch.zeros(s, device="cuda", dtype=dt) for s in ((4, 32), (2, 128, 32), (3,)))
    off = off.int()
    h = torch.zeros((4, 64), device="cuda", dtype=dt)
    for bad in (dict(w=w[:, :127]), dict(h=h[:, :63]), dict(h=h.float()), dict(x=x.float()), dict(off=off[:2]), dict(off=off.float()),
                dict(gu=h), dict(gu=torch.zeros((4, 128), device="cuda")), dict(x=x[:3]), dict(w=w[0]), dict(w=w.cpu()),
                dict(w=w[:1].expand(2, 128, 32))):
        a = dict(dict(x=x, w=w, off=off, h=h, gu=None), **bad)
        with pytest.raises((ValueError, TypeError, AssertionError)):
            moe.moe_grouped_swiglu(a["x"], a["w"], a["off"], a["h"], gu=a["gu"])
    dy, down, gu, dgu = (torch.zeros(s, device="cuda", dtype=dt) for s in ((4, 32), (2, 32, 64), (4, 128), (4, 128)))
    for bad in (dict(dgu=dgu[:, :64]), dict(gu=gu.float()), dict(h=gu), dict(down=down[:, :31]), dict(down=down.float()),
                dict(off=off[:2]), dict(dy=dy.cpu()), dict(gu=torch.zeros((4, 136), device="cuda", dtype=dt)[:, :128])):
        a = dict(dict(dy=dy, down=down, gu=gu, off=off, dgu=dgu, h=None), **bad)
        with pytest.raises((ValueError, TypeError, AssertionError)):
            moe.moe_grouped_swiglu_dx(a["dy"], a["down"], a["gu"], a["off"], a["dgu"], h=a["h"])
