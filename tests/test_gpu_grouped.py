"""Grouped products over plain weights (forward, gradient of the rows, gradient of the weights; bf16, fp32 and
int8) against 64-bit references, over ragged groups, odd sizes, strides, gathers and wrong index tables."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mixture_experts_layer_token_amd as moe  # noqa: E402

import grouped_ref as R  # noqa: E402
from grouped_ref import f64  # noqa: E402
from helpers import say  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


SENTINEL = 12345.0

# rows per expert, N, K
GROUPS = {
    "one": ([1], 1, 1),
    "tiny-odd": ([0, 0, 3], 5, 7),
    "ragged": ([17, 0, 64, 1, 130], 96, 160),
    "odd": ([65, 300, 0, 1], 131, 77),
    "by8": ([33], 40, 264),
    "tiles": ([513, 255, 256, 257], 520, 200),
    "decode": ([1, 0, 2, 1, 0, 3, 9], 352, 2880),
    "decode-odd": ([1, 0, 2, 1, 0, 3, 9], 77, 1111),
    "many": ([i % 5 for i in range(70)], 64, 96),
    "most": ([i % 3 for i in range(1024)], 16, 32),
    "long-k": ([40, 20], 48, 4096),
    "wide": ([700, 12], 600, 1024),
    "skinny": ([2100], 24, 104),
}


def rows_tensor(shape, dt, layout, gen):
    """A [rows, n] device tensor: contiguous, a slice of wider rows that keeps 16-byte rows, or one that does not."""
    rows, n = shape
    pad, off = {"dense": (0, 0), "padded": ((-n) % 8 + 8, 0), "shifted": (3, 1)}[layout]
    full = torch.randn((rows, n + pad), generator=gen, device="cuda").to(dt)
    return full, full[:, off:off + n]


def out_tensor(shape, dt, layout):
    rows, n = shape
    pad, off = {"dense": (0, 0), "padded": ((-n) % 8 + 8, 0), "shifted": (3, 1)}[layout]
    full = torch.full((rows, n + pad), SENTINEL, device="cuda", dtype=dt)
    return full, full[:, off:off + n]


def untouched(full, view, rows_written):
    """Everything of `full` outside the written rows of `view` still holds the sentinel."""
    keep = torch.ones_like(full, dtype=torch.bool)
    off = view.storage_offset() % full.shape[1]
    keep[:rows_written, off:off + view.shape[1]] = False
    return bool((full[keep] == torch.tensor(SENTINEL, dtype=full.dtype, device="cuda")).all())


def make(name, dt, layout="dense", gather=False, spare=0, seed=0):
    counts, N, K = GROUPS[name]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000 + seed)
    E, placed = len(counts), int(sum(counts))
    rows = placed + spare
    off = R.offsets_of(counts)
    k = 3 if gather else 1
    T = (rows + k - 1) // k + 1
    _, x = rows_tensor((T if gather else rows, K), dt, layout, gen)
    _, w = rows_tensor((E * N, K), dt, layout, gen)
    w = w.unflatten(0, (E, N)) * 0.05
    if layout != "dense":
        full, v = rows_tensor((E * N, K), dt, layout, gen)
        v.copy_(w.reshape(E * N, K))
        w = v.unflatten(0, (E, N))
    _, dy = rows_tensor((rows, N), dt, layout, gen)
    perm = None
    if gather:
        perm = torch.randint(0, T * k, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    return dict(x=x, w=w, dy=dy, perm=perm, k=k, off=off, offsets=torch.from_numpy(off).cuda(), N=N, K=K, E=E,
                rows=rows, placed=placed, gather=dict(perm_src=perm, k=k) if gather else {})


def check_op(op, c, dt_out, layout="dense", what=""):
    """Run op into sentinel-filled outputs, compare with the reference, check what must be left alone."""
    xg = R.gathered(c["x"], c["perm"], c["k"], c["rows"])
    if op == "y":
        full, out = out_tensor((c["rows"], c["N"]), dt_out, layout)
        moe.moe_grouped_gemm(c["x"], c["w"], c["offsets"], out, **c["gather"])
        ref = R.product("y", xg, R.f64(c["w"]), None, c["off"])
    elif op == "dx":
        full, out = out_tensor((c["rows"], c["K"]), dt_out, layout)
        moe.moe_grouped_gemm_dx(c["dy"], c["w"], c["offsets"], out)
        ref = R.product("dx", None, R.f64(c["w"]), R.f64(c["dy"]), c["off"])
    else:
        full, o2 = out_tensor((c["E"] * c["N"], c["K"]), dt_out, layout)
        out = o2.unflatten(0, (c["E"], c["N"]))
        moe.moe_grouped_gemm_dw(c["dy"], c["x"], c["offsets"], out, **c["gather"])
        ref = R.product("dw", xg, None, R.f64(c["dy"]), c["off"])
    torch.cuda.synchronize()
    R.assert_product(out, *ref, what="%s %s" % (op, what))
    view = out if op != "dw" else o2
    assert untouched(full, view, c["E"] * c["N"] if op == "dw" else c["placed"]), "%s %s: wrote outside" % (op, what)


@pytest.mark.parametrize("op", ["y", "dx", "dw"])
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("name", list(GROUPS))
def test_product(name, dt, out, op):
    say("grouped", op, name, dt, out)
    check_op(op, make(name, R.TORCH_DT[dt]), R.TORCH_DT[out], what=name)


@pytest.mark.parametrize("op", ["y", "dx", "dw"])
@pytest.mark.parametrize("layout,spare", [("padded", 7), ("shifted", 5)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("name,dt", [("ragged", "bf16"), ("odd", "bf16"), ("by8", "bf16"), ("decode", "bf16"),
                                     ("tiles", "bf16"), ("ragged", "f32"), ("odd", "f32")])
def test_product_strides_gather_spare_rows(name, dt, gather, layout, spare, op):
    say("grouped strided", op, name, dt, layout, "gather", gather)
    c = make(name, R.TORCH_DT[dt], layout, gather, spare, seed=1)
    check_op(op, c, torch.float32, layout, what="%s %s" % (name, layout))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["ragged", "odd", "tiles", "decode"])
def test_nonfinite_rows_stay_where_they_are(name, dt):
    """NaN and infinite rows of one expert, and of the rows behind the last group, reach no other result."""
    c = make(name, R.TORCH_DT[dt], spare=9)
    e_bad = int(np.argmax(np.diff(c["off"])))
    lo, hi = int(c["off"][e_bad]), int(c["off"][e_bad + 1])
    for t in (c["x"], c["dy"]):
        t[lo:hi:2] = float("nan")
        t[lo + 1:hi:2] = float("inf")
        t[c["placed"]:] = float("nan")
    good = np.ones(c["rows"], bool)
    good[lo:hi] = False
    good[c["placed"]:] = False
    good = torch.from_numpy(good)
    y = torch.full((c["rows"], c["N"]), SENTINEL, device="cuda")
    dx = torch.full((c["rows"], c["K"]), SENTINEL, device="cuda")
    dw = torch.empty((c["E"], c["N"], c["K"]), device="cuda")
    moe.moe_grouped_gemm(c["x"], c["w"], c["offsets"], y)
    moe.moe_grouped_gemm_dx(c["dy"], c["w"], c["offsets"], dx)
    moe.moe_grouped_gemm_dw(c["dy"], c["x"], c["offsets"], dw)
    torch.cuda.synchronize()
    x, w, dy = R.f64(c["x"]), R.f64(c["w"]), R.f64(c["dy"])
    for got, ref in ((y, R.product("y", x, w, None, c["off"])), (dx, R.product("dx", None, w, dy, c["off"]))):
        v, m, n = ref
        v[~good] = float("nan")  # not compared
        R.assert_product(got, v, torch.nan_to_num(m, nan=0.0, posinf=0.0), n, name)
        assert not torch.isfinite(got[lo:hi]).any()
        assert (got[c["placed"]:] == SENTINEL).all()
    keep = [e for e in range(c["E"]) if e != e_bad]
    v, m, n = R.product("dw", x, None, dy, c["off"])
    R.assert_product(dw[keep], v[keep], m[keep], n, name + " dw")


def test_wrong_offsets_are_clamped():
    """Offsets outside [0, rows] or out of order: rows are cut to the ones that exist, nothing else is touched."""
    c = make("ragged", torch.bfloat16)
    rows, E = c["rows"], c["E"]
    offs = np.array([-5, 30, 30, 20, 60, 1 << 30], dtype=np.int32)  # groups 0..30, -, -, 20..60, 60..rows
    eff = [(0, 30), (30, 30), (30, 20), (20, 60), (60, rows)]
    o = torch.from_numpy(offs).cuda()
    dw = torch.empty((E, c["N"], c["K"]), device="cuda")
    moe.moe_grouped_gemm_dw(c["dy"], c["x"], o, dw)
    y = torch.full((rows, c["N"]), SENTINEL, device="cuda")
    moe.moe_grouped_gemm(c["x"], c["w"], o, y)
    torch.cuda.synchronize()
    x, dy, w = R.f64(c["x"]), R.f64(c["dy"]), R.f64(c["w"])
    for e, (lo, hi) in enumerate(eff):
        ref = R.product("dw", x[lo:hi], None, dy[lo:hi], np.array([0, max(hi - lo, 0)])) if lo < hi else None
        if ref is None:
            assert (dw[e] == 0).all()
        else:
            R.assert_product(dw[e:e + 1], *ref, what="expert %d" % e)
    for e, lo, hi in ((0, 0, 20), (3, 31, 60), (4, 60, rows)):  # rows that one group alone claims
        v = x[lo:hi] @ w[e].T
        R.assert_product(y[lo:hi], v, x[lo:hi].abs() @ w[e].abs().T, c["K"], "rows %d..%d" % (lo, hi))
    for bad in ([0] * 6, [1 << 30] * 6, [-7] * 6):  # no rows at all
        y.fill_(SENTINEL)
        ob = torch.tensor(bad, dtype=torch.int32, device="cuda")
        moe.moe_grouped_gemm(c["x"], c["w"], ob, y)
        moe.moe_grouped_gemm_dw(c["dy"], c["x"], ob, dw)
        torch.cuda.synchronize()
        assert (y == SENTINEL).all() and (dw == 0).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["ragged", "odd", "decode"])
def test_perm_src_outside_x_is_a_row_of_zeros(name, dt):
    c = make(name, R.TORCH_DT[dt], gather=True)
    p = c["perm"]
    p[::3] = -1
    p[1::5] = 1 << 30
    p[2::7] = c["x"].shape[0] * c["k"]  # one past the end
    p[4::11] = -(1 << 30)
    check_op("y", c, torch.float32, what=name)
    check_op("dw", c, torch.float32, what=name)


def test_no_rows():
    w = torch.randn((3, 8, 16), device="cuda").bfloat16()
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, y = torch.empty((0, 16), device="cuda").bfloat16(), torch.empty((0, 8), device="cuda").bfloat16()
    dw = torch.full((3, 8, 16), 7.0, device="cuda")
    moe.moe_grouped_gemm(x, w, off, y)
    moe.moe_grouped_gemm_dx(y, w, off, x)
    moe.moe_grouped_gemm_dw(y, x, off, dw)
    torch.cuda.synchronize()
    assert (dw == 0).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gradients_against_differences(dt):
    """d/dx and d/dw of sum(dy * y) by central differences along random directions (exact for a bilinear form, up
    to the rounding of the perturbed operands, which are chosen to be representable)."""
    counts, N, K = [7, 0, 20, 1], 24, 40
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    rows, E = sum(counts), len(counts)
    off = torch.from_numpy(R.offsets_of(counts)).cuda()

    def ints(shape):  # small integers: sums and differences stay exact in bf16 and in the fp32 sums
        return torch.randint(-4, 5, shape, generator=gen, device="cuda").to(R.TORCH_DT[dt])

    x, w, dy, vx, vw = ints((rows, K)), ints((E, N, K)), ints((rows, N)), ints((rows, K)), ints((E, N, K))
    dx, dw = torch.empty((rows, K), device="cuda"), torch.empty((E, N, K), device="cuda")
    moe.moe_grouped_gemm_dx(dy, w, off, dx)
    moe.moe_grouped_gemm_dw(dy, x, off, dw)

    def loss(xx, ww):
        y = torch.empty((rows, N), device="cuda")
        moe.moe_grouped_gemm(xx, ww, off, y)
        return float((y.double() * dy.double()).sum())

    assert loss(x + vx, w) - loss(x - vx, w) == 2 * float((dx.double() * vx.double()).sum())
    assert loss(x, w + vw) - loss(x, w - vw) == 2 * float((dw.double() * vw.double()).sum())


# ------------------------------------------------------------------ int8
def check_i8(name, out, layout="dense", gather=False, spare=0, mutate=None, extremes=False):
    counts, N, K = GROUPS[name]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(77)
    E, placed = len(counts), int(sum(counts))
    rows, k = placed + spare, 3 if gather else 1
    T = (rows + k - 1) // k + 1
    nx = T if gather else rows
    pad, o = {"dense": (0, 0), "padded": ((-K) % 16 + 16, 0), "shifted": (3, 1)}[layout]
    lo, hi = (-128, -127) if extremes else (-128, 128)
    qf = torch.randint(lo, hi, (nx, K + pad), generator=gen, device="cuda").to(torch.int8)
    wf = torch.randint(lo, hi, (E * N, K + pad), generator=gen, device="cuda").to(torch.int8)
    q, w = qf[:, o:o + K], wf[:, o:o + K].unflatten(0, (E, N))
    qs = torch.rand(nx, generator=gen, device="cuda") + 0.1
    ws = torch.rand((E, N), generator=gen, device="cuda") + 0.1
    perm = torch.randint(0, T * k, (rows,), generator=gen, device="cuda", dtype=torch.int32) if gather else None
    if mutate:
        mutate(perm, qs)
    off = R.offsets_of(counts)
    dt = R.TORCH_DT[out]
    full, y = out_tensor((rows, N), dt, layout)
    moe.moe_grouped_gemm_i8(q, qs, w, ws, torch.from_numpy(off).cuda(), y, **(dict(perm_src=perm, k=k) if gather else {}))
    torch.cuda.synchronize()
    qg, sg = R.gathered(q, perm, k, rows), R.gathered(qs[:, None], perm, k, rows)
    v, _, _ = R.product("y", qg, R.f64(w), None, off)
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        v[r] = v[r] * sg[r] * R.f64(ws)[e]
    # the sum is exact; its conversion to fp32 and two products round once each (2^-24), then the result's type
    bound = v.abs() * (1 + R.HALF_STEP[dt]) * 3.0001 * 2.0 ** -24 + v.abs() * R.HALF_STEP[dt] + 1e-37
    placed_rows = ~torch.isnan(v)
    bad = placed_rows & ~((R.f64(y) - v).abs() <= bound)
    assert not bad.any(), "%s: %d off, first at %s" % (name, int(bad.sum()), torch.nonzero(bad)[0].tolist())
    assert untouched(full, y, placed)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(GROUPS))
def test_int8_product(name, out):
    say("grouped int8", name, out)
    check_i8(name, out)


@pytest.mark.parametrize("layout,spare", [("padded", 7), ("shifted", 5)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("name", ["ragged", "odd", "by8", "decode", "tiles"])
def test_int8_product_strides_gather_spare_rows(name, gather, layout, spare):
    say("grouped int8 strided", name, layout, gather)
    check_i8(name, "f32", layout, gather, spare)


def test_int8_sums_do_not_overflow_or_round():
    """-128 times -128 everywhere: K = 4096 of them is 2^26, beyond what fp32 sums would keep exactly with odd parts."""
    check_i8("long-k", "f32", extremes=True)


def test_int8_perm_src_outside_is_zero():
    def mutate(perm, qs):
        perm[::3] = -1
        perm[1::4] = 1 << 30

    check_i8("ragged", "f32", gather=True, mutate=mutate)


# ------------------------------------------------------------------ streams, graphs, other launch conditions
@pytest.mark.parametrize("name", ["ragged", "decode", "tiles"])
def test_graph_replay_and_side_stream(name):
    c = make(name, torch.bfloat16)
    y = torch.zeros((c["rows"], c["N"]), device="cuda", dtype=torch.bfloat16)
    dx = torch.zeros((c["rows"], c["K"]), device="cuda", dtype=torch.bfloat16)
    dw = torch.zeros((c["E"], c["N"], c["K"]), device="cuda")
    need = moe.moe_grouped_workspace("bf16", c["rows"], c["N"], c["K"], c["E"])
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")

    def step():
        moe.moe_grouped_gemm(c["x"], c["w"], c["offsets"], y, ws=ws)
        moe.moe_grouped_gemm_dx(y, c["w"], c["offsets"], dx, ws=ws)
        moe.moe_grouped_gemm_dw(y, c["x"], c["offsets"], dw, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    ref = [t.clone() for t in (y, dx, dw)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    x0 = c["x"].clone()
    for rep in range(4):
        for t in (y, dx, dw):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for t, r in zip((y, dx, dw), ref):
            assert torch.equal(t, r), "replay %d" % rep
        c["x"].mul_(0.5)  # eager work between the replays, with other values
        step()
        torch.cuda.synchronize()
        assert not torch.equal(y, ref[0])
        c["x"].copy_(x0)


def test_two_calls_at_once():
    """Two streams with calls of their own in flight together (each with its own workspace)."""
    cs = [make("tiles", torch.bfloat16, seed=s) for s in (1, 2)]
    refs, outs = [], []
    for c in cs:
        dw = torch.zeros((c["E"], c["N"], c["K"]), device="cuda")
        moe.moe_grouped_gemm_dw(c["dy"], c["x"], c["offsets"], dw)
        refs.append(dw)
        outs.append(torch.zeros_like(dw))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(3):
        for c, o, s in zip(cs, outs, streams):
            with torch.cuda.stream(s):
                moe.moe_grouped_gemm_dw(c["dy"], c["x"], c["offsets"], o)
    torch.cuda.synchronize()
    for o, r in zip(outs, refs):
        assert torch.equal(o, r)


def test_rows_past_four_gigabytes():
    """x rows, results and weights whose byte offsets do not fit 32 bits."""
    K, N, rows = 4096, 64, 40
    T = (1 << 32) // (K * 2) + 1000
    x = torch.empty((T, K), device="cuda", dtype=torch.bfloat16)
    picks = torch.tensor([0, 1, T - 1, T - 2, T // 2, T - 999] * 7, dtype=torch.int32, device="cuda")[:rows]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    vals = torch.randn((rows, K), generator=gen, device="cuda").bfloat16()
    x[picks.long()] = vals
    named = x[picks.long()]  # (a row picked twice holds one of its values)
    w = torch.randn((2, N, K), generator=gen, device="cuda").bfloat16()
    dy = torch.randn((rows, N), generator=gen, device="cuda").bfloat16()
    off = np.array([0, 25, rows], np.int32)
    offsets = torch.from_numpy(off).cuda()
    y, dw = torch.empty((rows, N), device="cuda"), torch.empty((2, N, K), device="cuda")
    moe.moe_grouped_gemm(x, w, offsets, y, perm_src=picks * 2, k=2)
    moe.moe_grouped_gemm_dw(dy, x, offsets, dw, perm_src=picks * 2, k=2)
    torch.cuda.synchronize()
    R.assert_product(y, *R.product("y", f64(named), f64(w), None, off), what="y")
    R.assert_product(dw, *R.product("dw", f64(named), None, f64(dy), off), what="dw")
    # grouped rows in place: the last group lies past 4 GiB
    g2 = torch.tensor([0, 3, T - 30], dtype=torch.int32)
    offs = torch.cat([g2, torch.tensor([T], dtype=torch.int32)])
    w3 = torch.randn((3, N, K), generator=gen, device="cuda").bfloat16()
    x[:3], x[T - 30:] = vals[:3], vals[3:33]
    x[3:T - 30] = 0
    y2 = torch.full((T, N), SENTINEL, device="cuda", dtype=torch.bfloat16)
    moe.moe_grouped_gemm(x, w3, offs.cuda(), y2)
    torch.cuda.synchronize()
    assert (y2[3:T - 30] == 0).all()
    tail = f64(vals[3:33]) @ f64(w3[2]).T
    R.assert_product(y2[T - 30:], tail, f64(vals[3:33]).abs() @ f64(w3[2]).abs().T, K, "tail")


def test_explicit_stream_allocates_its_workspace_safely():
    counts, N, K = GROUPS["skinny"]
    c = make("skinny", torch.bfloat16)
    assert moe.moe_grouped_workspace("bf16", c["rows"], N, K, c["E"]) > 0  # few tiles, many rows: split sums
    dw, ref = (torch.empty((c["E"], N, K), device="cuda") for _ in range(2))
    moe.moe_grouped_gemm_dw(c["dy"], c["x"], c["offsets"], ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    moe.moe_grouped_gemm_dw(c["dy"], c["x"], c["offsets"], dw, stream=s)
    junk = torch.full((1 << 22,), 3.0, device="cuda")  # would take the freed workspace's place
    torch.cuda.synchronize()
    assert torch.equal(dw, ref) and float(junk[0]) == 3.0


def reference_on_gpu(op, x, w, y, off):
    """R.product with 64-bit products on the device (sizes for which the CPU would take minutes)."""
    E = len(off) - 1
    N, K = y.shape[1], x.shape[1]
    shape = {"y": y.shape, "dx": x.shape, "dw": (E, N, K)}[op]
    out, mag = (torch.zeros(shape, dtype=torch.float64, device="cuda") for _ in range(2))
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        a, b = {"y": lambda: (x[r].double(), w[e].double().T), "dx": lambda: (y[r].double(), w[e].double()),
                "dw": lambda: (y[r].double().T, x[r].double())}[op]()
        d = e if op == "dw" else r
        out[d], mag[d] = a @ b, a.abs() @ b.abs()
    return out.cpu(), mag.cpu(), {"y": K, "dx": N, "dw": max(1, int(np.diff(off).max()))}[op]


# several rounds of 256 x 256 tiles, odd ends everywhere: the shape of long calls
@pytest.mark.parametrize("op,N,K", [("y", 8200, 584), ("dx", 584, 8200), ("dw", 4104, 4136)])
@pytest.mark.parametrize("gather", [False, True])
def test_large_tiles(op, N, K, gather):
    say("grouped large", op, N, K, gather)
    counts = [3000, 0, 5101, 92]
    off = R.offsets_of(counts)
    rows, E, k = sum(counts), len(counts), 2 if gather else 1
    gen = torch.Generator(device="cuda")
    gen.manual_seed(21)
    x = torch.randn((rows, K), generator=gen, device="cuda").bfloat16()
    w = torch.randn((E, N, K), generator=gen, device="cuda").bfloat16()
    dy = torch.randn((rows, N), generator=gen, device="cuda").bfloat16()
    perm = torch.randint(0, rows * k, (rows,), generator=gen, device="cuda", dtype=torch.int32) if gather else None
    kw = dict(perm_src=perm, k=k) if gather else {}
    xg = x[(perm // k).long()] if gather else x
    offsets = torch.from_numpy(off).cuda()
    for dt in (torch.float32, torch.bfloat16):
        if op == "y":
            out = torch.empty((rows, N), device="cuda", dtype=dt)
            moe.moe_grouped_gemm(x, w, offsets, out, **kw)
        elif op == "dx":
            out = torch.empty((rows, K), device="cuda", dtype=dt)
            moe.moe_grouped_gemm_dx(dy, w, offsets, out)
        else:
            out = torch.empty((E, N, K), device="cuda", dtype=dt)
            moe.moe_grouped_gemm_dw(dy, x, offsets, out, **kw)
        torch.cuda.synchronize()
        R.assert_product(out, *reference_on_gpu(op, xg, w, dy, off), what=op)


def test_large_int8_tiles():
    counts, N, K = [3000, 0, 5101, 92], 8200, 592
    off = R.offsets_of(counts)
    rows, E = sum(counts), len(counts)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(22)
    q = torch.randint(-128, 128, (rows, K), generator=gen, device="cuda").to(torch.int8)
    w = torch.randint(-128, 128, (E, N, K), generator=gen, device="cuda").to(torch.int8)
    qs, ws = torch.rand(rows, generator=gen, device="cuda") + 0.1, torch.rand((E, N), generator=gen, device="cuda") + 0.1
    y = torch.empty((rows, N), device="cuda")
    moe.moe_grouped_gemm_i8(q, qs, w, ws, torch.from_numpy(off).cuda(), y)
    torch.cuda.synchronize()
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        v = (q[r].double() @ w[e].double().T) * qs[r, None].double() * ws[e].double()
        # the conversion of the exact sum and two products in fp32: 2^-24 each
        assert bool(((y[r].double() - v).abs() <= v.abs() * 3.0001 * 2.0 ** -24).all())


# weight gradients with few tiles: the rows in up to 32 parts, some parts without rows, a column of ones (a plain sum)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,N,K", [([9001], 16, 1), ([9001], 24, 40), ([4099, 2], 136, 200), ([1, 0, 6000], 8, 520),
                                        ([1025], 390, 1030)])
def test_weight_gradients_in_parts(counts, N, K, dt):
    say("grouped parts", counts, N, K, dt)
    off = R.offsets_of(counts)
    rows, E = sum(counts) + 5, len(counts)  # 5 rows behind the last group
    gen = torch.Generator(device="cuda")
    gen.manual_seed(31)
    x = torch.randn((rows, K), generator=gen, device="cuda").to(dt)
    dy = torch.randn((rows, N), generator=gen, device="cuda").to(dt)
    need = moe.moe_grouped_workspace("f32" if dt == torch.float32 else "bf16", rows, N, K, E)
    assert need >= 2 * E * N * K * 4
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN wherever a part is not written
    for out in (torch.float32, torch.bfloat16):
        dw = torch.empty((E, N, K), device="cuda", dtype=out)
        moe.moe_grouped_gemm_dw(dy, x, torch.from_numpy(off).cuda(), dw, ws=ws)
        torch.cuda.synchronize()
        R.assert_product(dw, *reference_on_gpu("dw", x, None, dy, off), what="dw")
