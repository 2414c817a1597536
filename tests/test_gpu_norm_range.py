"""Norms of finite rows whose sums or squares leave the fp32 range on either side, against 64-bit references."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mixture_experts_layer_token_amd as moe  # noqa: E402

from grouped_ref import HALF_STEP, f64  # noqa: E402
from helpers import say  # noqa: E402
from test_gpu_norm import adds, grad_reference, make, within  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


DTS = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24
TINY = 2.0 ** -126

# a size of every kernel: 1 wave of one chunk or two, 4 of one or two, 16 of one, 8 of two, 16 of two, rows read again
SIZES = [(3, 5), (7, 512), (700, 1000), (9, 2047), (600, 2880), (2, 7168), (520, 7169), (3, 16384), (2, 16385)]
SCALES = [1e20, 2.0 ** 66, 1e30, 2.0 ** 124, 1e-14, 1e-16, 1e-24, 1e-30, 2.0 ** -126]


def reference(x, eps, rms):
    X = f64(x)
    mean = torch.zeros_like(X[:, :1]) if rms else X.mean(1, keepdim=True)
    d = X - mean
    var = (d * d).mean(1, keepdim=True)
    return X, mean, d, var, (var + eps) ** -0.5


def check(x, w, b, eps, rms, what):
    """y, mean and rstd within the error of fp32 sums (as for rows of any other size: the bounds are relative to the row)."""
    rows, H = x.shape
    n, dt = adds(H), x.dtype
    y, stats = torch.empty((rows, H), device="cuda", dtype=dt), torch.empty((rows, 2), device="cuda")
    moe.moe_norm(x, w, b, y, eps=eps, rms=rms, stats=stats)
    torch.cuda.synchronize()
    X, mean, d, var, rstd = reference(x, eps, rms)
    em = torch.zeros_like(mean) if rms else (n + 2) * U * X.abs().mean(1, keepdim=True)
    ed = em + U * (d.abs() + em)
    ev = (2 * ed * d.abs() + ed * ed).mean(1, keepdim=True) + (n + 3) * U * var
    er = rstd * (0.5 * ev / (var + eps) * (1 + ev / (var + eps)) + 4 * U)
    ref = d * rstd * f64(w) + f64(b)
    e = f64(w).abs() * (ed * (rstd + er) + d.abs() * er) + 3 * U * ((d * rstd * f64(w)).abs() + f64(b).abs())
    within(y, ref, e + HALF_STEP[dt] * (ref.abs() + e), "y " + what)
    # (statistics below the normal range are rounded to steps of 2^-149)
    within(stats[:, :1], mean, em + 2 * U * mean.abs() + 2.0 ** -149, "mean " + what)
    fits = rstd <= torch.finfo(torch.float32).max
    within(stats[:, 1:][fits], rstd[fits], (er + U * rstd)[fits] + 2.0 ** -149, "rstd " + what)
    assert (stats[:, 1:].cpu()[~fits] == float("inf")).all()
    return stats


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,H", SIZES)
def test_rows_of_any_size(rows, H, dt, rms):
    """Every scale among rows of ordinary ones, which stay what they are."""
    say("norm range", rows, H, dt, "rms", rms)
    x, _, _, w, b = make(rows, H, torch.float32, torch.float32, seed=20)
    for scale in SCALES:
        for eps in (0.0, 1e-5):
            z = x.clone()
            z[::2] *= scale
            check(z.to(DTS[dt]), w, b, eps, rms, "%g eps %g" % (scale, eps))


@pytest.mark.parametrize("rms", [False, True])
def test_far_ends_of_the_range(rms):
    """The largest elements, whose plain sum overflows, and the smallest, below the normal range; far from their mean and near."""
    top = torch.finfo(torch.float32).max
    for H in (64, 1000, 4096, 7168, 16384, 20000):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(21)
        x = torch.empty((6, H), device="cuda")
        x[0] = top
        x[0, ::3] = top / 2
        x[1] = torch.rand(H, generator=gen, device="cuda") * top
        x[2] = torch.randint(1, 1 << 20, (H,), generator=gen, device="cuda").double().mul(2.0 ** -149).float()
        x[3] = torch.randn(H, generator=gen, device="cuda") * 1e-20 + 1e-18
        x[4] = torch.randn(H, generator=gen, device="cuda") * 1e18 + 1e20
        x[5] = 0.5 * top * (1 - 2 * (torch.arange(H, device="cuda") % 2))
        w, b = torch.randn(H, generator=gen, device="cuda"), torch.randn(H, generator=gen, device="cuda")
        check(x, w, b, 0.0, rms, "%d" % H)


def test_constant_rows_of_any_size():
    """No deviations, also where the plain sum overflows (powers of two: their mean is exact): y is the bias."""
    for H in (64, 1024, 4096, 8192, 32768):
        x = torch.empty((3, H), device="cuda")
        x[0], x[1], x[2] = 2.0 ** 127, 2.0 ** -140, 2.0 ** 30
        w, b = torch.full((H,), 2.0, device="cuda"), torch.randn(H, device="cuda")
        y, stats = torch.empty_like(x), torch.empty((3, 2), device="cuda")
        for eps in (1e-5, 1e-36):
            moe.moe_norm(x, w, b, y, eps=eps, stats=stats)
            torch.cuda.synchronize()
            assert all(torch.equal(r, b) for r in y) and torch.equal(stats[:, 0], x[:, 0])
            want = float(torch.tensor(eps, dtype=torch.float32)) ** -0.5
            assert ((f64(stats[:, 1]) - want).abs() <= 4 * U * want).all()


def test_around_the_ends():
    """One element, whose square is just inside and just outside: y is its sign."""
    ends = [2.0 ** 64, 2.0 ** 54, 2.0 ** -50, 2.0 ** -63, 2.0 ** -75]
    x = torch.tensor([[v * (1 + s * 2.0 ** -23)] for v in ends for s in (-2, -1, -0.5, 0, 1, 2)], dtype=torch.float64).float().cuda()
    x[1::2] *= -1
    y, one = torch.empty_like(x), torch.ones(1, device="cuda")
    moe.moe_norm(x, one, None, y, eps=0.0, rms=True)
    torch.cuda.synchronize()
    assert ((f64(y) - f64(x.sign())).abs() <= 8 * U).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rms", [False, True])
def test_gradient_of_rows_of_any_size(dt, rms):
    """Forward, then the gradient from its statistics, while 1 / sqrt is within the normal range."""
    for rows, H in ((7, 512), (33, 2880), (5, 8192), (3, 16384), (3, 20000)):
        x, dy, add, w, b = make(rows, H, DTS[dt], torch.float32, seed=22)
        for scale in (1e20, 1e30, 1e-16, 1e-30):
            z = (x.float() * scale).to(DTS[dt])
            # (dx takes 1 / sqrt as a factor: dy of the row's size keeps it within the range)
            g = (dy.float() * scale).to(DTS[dt])
            y, dx = torch.empty_like(z), torch.empty((rows, H), device="cuda", dtype=DTS[dt])
            stats = torch.empty((rows, 2), device="cuda")
            dw, db = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
            moe.moe_norm(z, w, b, y, eps=0.0, rms=rms, stats=stats)
            moe.moe_norm_grad(g, z, w, stats, dx, dweight=dw, dbias=db, add=add, rms=rms)
            torch.cuda.synchronize()
            _, _, _, _, rstd = reference(z, 0.0, rms)
            assert ((f64(stats[:, 1:]) - rstd).abs() <= 1e-4 * rstd).all()
            for got, (ref, e), name in zip((dx, dw, db), grad_reference(g, z, w, stats, add, rms), ("dx", "dweight", "dbias")):
                within(got, ref, e + HALF_STEP[got.dtype] * (ref.abs() + e) + TINY * U, "%s %g" % (name, scale))
