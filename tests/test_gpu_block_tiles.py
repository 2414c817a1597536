"""The gated block's tile kernels against 64-bit references where test_gpu_block.py's sizes take the kernels for few rows: tiles of
256 x 256 over several stages, far-out gates, wrong tables, matrices with gaps, and rows of weights past 32-bit offsets.

Which kernel a size takes is said beside it, for 256 compute units."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mixture_experts_layer_token_amd as moe  # noqa: E402

import grouped_ref as R  # noqa: E402
import test_gpu_block as B  # noqa: E402
from grouped_ref import HALF_STEP, f64  # noqa: E402
from helpers import say  # noqa: E402

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


@pytest.fixture(autouse=True)
def _groups(monkeypatch):
    # tiles of 256 x 256: of 128 x 128 there would be 18.4 x 31 = 570, a second round of 512; nine stages, the last of 8 elements,
    # tiles of fewer rows and columns at the edges, an expert without rows and one with a single one
    monkeypatch.setitem(B.GROUPS, "large-tiles", ([900, 0, 1, 1200], 1928, 520))
    monkeypatch.setitem(B.GROUPS, "large-tiles-grad", ([900, 0, 1, 1200], 3848, 520))


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("layout,spare,shift", [("dense", 0, 0), ("padded", 7, 8), ("dense", 3, 1)])
def test_large_tiles_forward(layout, spare, shift, gather, keep):
    say("block forward, large tiles", layout, "gather", gather, "keep", keep, "shift", shift)
    B.check_forward(B.make("large-tiles", BF16, layout, gather, spare, seed=30), BF16, layout, keep=keep, shift=shift)


@pytest.mark.parametrize("with_h", [False, True])
@pytest.mark.parametrize("layout,spare,shift", [("dense", 0, 0), ("padded", 7, 8), ("dense", 3, 1)])
def test_large_tiles_gradient(layout, spare, shift, with_h):
    say("block gradient, large tiles", layout, "h", with_h, "shift", shift)
    B.check_gradient(B.make("large-tiles-grad", BF16, layout, False, spare, seed=31), BF16, with_h, shift=shift)


# "tiles": direct 128 x 128 tiles; "odd": staged ones
@pytest.mark.parametrize("name,dt", [("large-tiles", "bf16"), ("tiles", "bf16"), ("odd", "bf16"), ("tiles", "f32"), ("odd", "f32")])
def test_large_gates_forward(name, dt):
    """g of some hundreds on both sides: e^-g overflows or vanishes.

    Beside the bounds of test_gpu_block.py: a reciprocal below 2^-126 may come back as zero, which takes |g u| 2^-126 from h: with g
    and u below 600, 5e-33."""
    c = B.make(name, B.DTS[dt], seed=32)
    c["w"] = c["w"] * 64
    h = torch.empty((c["rows"], c["I"]), device="cuda", dtype=B.DTS[dt])
    moe.moe_grouped_swiglu(c["x"], c["w"], c["offsets"], h)
    torch.cuda.synchronize()
    ref, bound, gu, _ = B.forward_reference(c)
    assert gu.nan_to_num().abs().max() < 600 and gu.nan_to_num().min() < -150
    B.within(h, ref, bound + HALF_STEP[B.DTS[dt]] * (ref.abs() + bound) + 1e-30, "h " + name)


# (direct: large-tiles-grad, deep-wide, by4-wide in fp32; staged: odd-wide)
@pytest.mark.parametrize("name,dt", [("large-tiles-grad", "bf16"), ("deep-wide", "bf16"), ("odd-wide", "bf16"), ("odd-wide", "f32"), ("by4-wide", "f32")])
def test_large_gates_gradient(name, dt):
    """As above; dgu loses at most |dh u| (1 + |g|) 2^-126: with dh below 100, 5e-31."""
    c = B.make(name, B.DTS[dt], seed=33)
    c["gu"] = c["gu"] * 64
    dgu, h = torch.empty_like(c["gu"]), torch.empty((c["rows"], c["I"]), device="cuda", dtype=B.DTS[dt])
    moe.moe_grouped_swiglu_dx(c["dy"], c["down"], c["gu"], c["offsets"], dgu, h=h)
    torch.cuda.synchronize()
    assert c["gu"].abs().max() < 600 and c["gu"].min() < -150
    ref, bound, href, hbound = B.gradient_reference(c)
    half = HALF_STEP[B.DTS[dt]]
    B.within(dgu, ref, bound + half * (ref.abs() + bound) + 1e-30, "dgu " + name)
    B.within(h, href, hbound + half * (href.abs() + hbound) + 1e-30, "h " + name)


@pytest.mark.parametrize("name,dt", [("deep-wide", "bf16"), ("odd-wide", "bf16"), ("odd-wide", "f32")])
def test_gradient_against_differences(name, dt):
    """As in test_gpu_block.py, where the kernel for few rows answers."""
    c = B.make(name, B.DTS[dt], seed=34)
    dgu = torch.empty_like(c["gu"])
    moe.moe_grouped_swiglu_dx(c["dy"], c["down"], c["gu"], c["offsets"], dgu)
    torch.cuda.synchronize()
    dh, _, _ = R.product("dx", None, f64(c["down"]), f64(c["dy"]), c["off"])
    gu, I, eps = f64(c["gu"]), c["I"], 1e-6
    v = torch.randn(gu.shape, generator=torch.Generator().manual_seed(10), dtype=torch.float64)

    def loss(s):
        t = gu + s * eps * v
        return float((dh * torch.nn.functional.silu(t[:, :I]) * t[:, I:]).sum())

    num, got = (loss(1) - loss(-1)) / (2 * eps), f64(dgu) * v
    # every element of the gradient is off by half a step of its type and the sums' own error; the losses, sums of n terms in 64
    # bits, by n 2^-53 of their magnitude at most, over 2 eps
    terms = float((dh * torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]).abs().sum())
    assert abs(num - float(got.sum())) <= (HALF_STEP[B.DTS[dt]] + 2.0 ** -16) * float(got.abs().sum()) + 2.0 ** -40 * terms / eps


def test_wrong_tables_reach_nothing_outside():
    """As in test_gpu_block.py, with I = 4096: 256 tiles forward, 4 x 32 small workgroups (sums over 96: at most 48) for the gradient."""
    rows, I, K, E = 40, 4096, 96, 4
    gen = torch.Generator(device="cuda")
    gen.manual_seed(35)
    x = torch.randn((rows, K), generator=gen, device="cuda").to(BF16)
    w = (torch.randn((E, 2 * I, K), generator=gen, device="cuda") * 0.1).to(BF16)
    down = (torch.randn((E, K, I), generator=gen, device="cuda") * 0.1).to(BF16)
    gu = torch.randn((rows, 2 * I), generator=gen, device="cuda").to(BF16)
    off = torch.tensor([-5, 10, 7, 30, 1000], dtype=torch.int32, device="cuda")  # 0..10, none, 7..30, 30..40
    hfull, h = B.flat_out((rows, I), BF16, 4)
    gfull, dgu = B.flat_out((rows, 2 * I), BF16, 4)
    moe.moe_grouped_swiglu(x, w, off, h)
    moe.moe_grouped_swiglu_dx(x, down, gu, off, dgu)
    torch.cuda.synchronize()
    for e, lo, hi in ((0, 0, 7), (2, 10, 30), (3, 30, 40)):  # (rows 7..9 belong to two groups)
        c = dict(x=x[lo:hi], w=w[e:e + 1], down=down[e:e + 1], dy=x[lo:hi], gu=gu[lo:hi], perm=None, k=1, off=R.offsets_of([hi - lo]), I=I,
                 K=K, rows=hi - lo)
        ref, bound, _, _ = B.forward_reference(c)
        B.within(h[lo:hi], ref, bound + HALF_STEP[BF16] * (ref.abs() + bound) + 1e-37, "h of expert %d" % e)
        ref, bound, _, _ = B.gradient_reference(c)
        B.within(dgu[lo:hi], ref, bound + HALF_STEP[BF16] * (ref.abs() + bound) + 1e-37, "dgu of expert %d" % e)
    for full in (hfull, gfull):
        assert (full[:4] == B.SENTINEL).all() and (full[-4:] == B.SENTINEL).all()


@pytest.mark.parametrize("name", ["large-tiles", "large-tiles-grad", "deep-wide"])
def test_matrices_with_gaps(name):
    c = B.make(name, BF16, seed=36)
    E, I, K = c["E"], c["I"], c["K"]
    wide = torch.full((E, 2 * I + 3, K + 8), float("nan"), device="cuda", dtype=BF16)
    wide[:, :2 * I, :K] = c["w"]
    wdown = torch.full((E, K + 5, I + 8), float("nan"), device="cuda", dtype=BF16)
    wdown[:, :K, :I] = c["down"]
    a, b = (torch.empty((c["rows"], I), device="cuda", dtype=BF16) for _ in range(2))
    p, q = (torch.empty((c["rows"], 2 * I), device="cuda", dtype=BF16) for _ in range(2))
    moe.moe_grouped_swiglu(c["x"], c["w"], c["offsets"], a)
    moe.moe_grouped_swiglu_dx(c["dy"], c["down"], c["gu"], c["offsets"], p)
    moe.moe_grouped_swiglu(c["x"], wide[:, :2 * I, :K], c["offsets"], b)
    moe.moe_grouped_swiglu_dx(c["dy"], wdown[:, :K, :I], c["gu"], c["offsets"], q)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(p, q)


# ------------------------------------------------------------------ rows past 32-bit offsets
def dense_case(rows, I, K, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def t(*shape, sigma=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(BF16)

    off = R.offsets_of([rows])
    return dict(x=t(rows, K), w=t(1, 2 * I, K, sigma=0.2), down=t(1, K, I, sigma=0.1), dy=t(rows, K), gu=t(rows, 2 * I, sigma=1.5), perm=None, k=1,
                off=off, offsets=torch.from_numpy(off).cuda(), I=I, K=K, E=1, rows=rows, placed=rows, gather={})


def stretched(w, ld):
    """The matrices of w with rows ld elements apart, among NaN."""
    E, n, k = w.shape
    far = torch.full((E, n, ld), float("nan"), device="cuda", dtype=w.dtype)[:, :, :k]
    far.copy_(w)
    return far


# ld 2^24: no tile of 256 rows has a descriptor; 4194232: 511 rows have one, so that of the gate's and up rows of 376 + 128 it still
# covers all, of 448 + 128 not
@pytest.mark.parametrize("I,ld", [(64, 1 << 24), (376, 4194232), (448, 4194232)])
def test_gate_and_up_rows_far_apart(I, ld):
    """w of more than 4 GiB; 5 rows: strips or halves of them, 100: tiles (direct for 376, else staged)."""
    say("block, far rows of w", I, ld)
    far = None
    for rows in (5, 100):
        c = dense_case(rows, I, 64, 37)
        if far is None:
            w, far = c["w"], stretched(c["w"], ld)
        c["w"] = far
        h, gu = torch.empty((rows, I), device="cuda", dtype=BF16), torch.empty((rows, 2 * I), device="cuda", dtype=BF16)
        moe.moe_grouped_swiglu(c["x"], far, c["offsets"], h, gu=gu)
        torch.cuda.synchronize()
        ref, bound, gref, gbound = B.forward_reference(dict(c, w=w))
        B.within(h, ref, bound + HALF_STEP[BF16] * (ref.abs() + bound) + 1e-37, "h")
        B.within(gu, gref, gbound + HALF_STEP[BF16] * (gref.abs() + gbound) + 1e-37, "gu")


@pytest.mark.parametrize("rows,I", [(5, 64), (140, 64), (140, 11008)])
def test_down_rows_and_dy_far_apart(rows, I):
    """Rows of dy, and 140 rows of w, 2^24 elements apart.  I = 64: small workgroups; 11008: 9 x 86 = 774 of them would be too many, and
    tiles run."""
    say("block gradient, far rows", rows, I)
    c = dense_case(rows, I, 140, 38)
    ref, bound, href, hbound = B.gradient_reference(c)
    far_w, far_dy = stretched(c["down"], 1 << 24), stretched(c["dy"][None], 1 << 24)[0]
    for w, dy in ((far_w, c["dy"]), (c["down"], far_dy)):
        dgu, h = torch.empty_like(c["gu"]), torch.empty((rows, I), device="cuda", dtype=BF16)
        moe.moe_grouped_swiglu_dx(dy, w, c["gu"], c["offsets"], dgu, h=h)
        torch.cuda.synchronize()
        B.within(dgu, ref, bound + HALF_STEP[BF16] * (ref.abs() + bound) + 1e-37, "dgu")
        B.within(h, href, hbound + HALF_STEP[BF16] * (href.abs() + hbound) + 1e-37, "h")
