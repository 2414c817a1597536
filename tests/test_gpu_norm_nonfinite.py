"""What rows that hold a NaN or an infinity give, element by element: their own results and the sums over rows."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mixture_experts_layer_token_amd as moe  # noqa: E402

from test_gpu_norm import DTS, make  # noqa: E402

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


def both(x, dy, w, b, rms):
    rows, H = x.shape
    y, dx, st = torch.empty_like(x), torch.empty_like(x), torch.empty((rows, 2), device="cuda")
    dw, db = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    moe.moe_norm(x, w, b, y, rms=rms, stats=st)
    moe.moe_norm_grad(dy, x, w, st, dx, dweight=dw, dbias=db, rms=rms)
    torch.cuda.synchronize()
    return y, st, dx, dw, db


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H", [300, 1000, 2880, 7168, 16384, 17000])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_layer_norm(value, H, dt):
    """The mean is not finite, and no element of y, dx or dweight is; the other rows and dbias do not know of it."""
    x, dy, _, w, b = make(40, H, DTS[dt], torch.float32, seed=50)
    clean = both(x, dy, w, b, False)
    x = x.clone()
    x[17, H - 1] = value
    y, st, dx, dw, db = both(x, dy, w, b, False)
    assert not torch.isfinite(y[17]).any() and not torch.isfinite(dx[17]).any() and not torch.isfinite(st[17]).any()
    assert not torch.isfinite(dw).any() and torch.equal(db, clean[4])
    keep = torch.arange(40, device="cuda") != 17
    for p, q in zip((y, st, dx), clean):
        assert torch.equal(p[keep], q[keep])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H", [300, 1000, 2880, 7168, 16384, 17000])
def test_rms_norm(H, dt):
    """An infinity: 1 / sqrt is 0, so its own element is NaN and the others are the bias; dx is not finite, dweight only where the
    infinity is.  A NaN: no element of the row or of dweight is finite."""
    x, dy, _, w, b = make(40, H, DTS[dt], torch.float32, seed=51)
    clean = both(x, dy, w, b, True)
    keep = torch.arange(40, device="cuda") != 17
    for value in (INF, -INF):
        z = x.clone()
        z[17, 5] = value
        y, st, dx, dw, db = both(z, dy, w, b, True)
        assert st[17].tolist() == [0.0, 0.0]
        other = torch.arange(H, device="cuda") != 5
        assert torch.isnan(y[17, 5]) and torch.equal(y[17][other], b.to(DTS[dt])[other])
        assert not torch.isfinite(dx[17]).any()
        assert torch.isnan(dw[5]) and torch.isfinite(dw[other]).all() and torch.equal(db, clean[4])
        for p, q in zip((y, st, dx), clean):
            assert torch.equal(p[keep], q[keep])
    z = x.clone()
    z[17, 5] = NAN
    y, st, dx, dw, db = both(z, dy, w, b, True)
    assert torch.isnan(y[17]).all() and torch.isnan(dx[17]).all() and torch.isnan(st[17, 1])
    assert torch.isnan(dw).all() and torch.equal(db, clean[4])
    for p, q in zip((y, st, dx), clean):
        assert torch.equal(p[keep], q[keep])
