"""8-bit row quantization, the SwiGLU gate with its gradient and the combine's gradient against 64-bit
references."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mixture_experts_layer_token_amd as moe  # noqa: E402

import grouped_ref as R  # noqa: E402
from helpers import say  # noqa: E402

F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def near(got, want, bound, what):
    err = (R.f64(got) - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), "%s: %d off, first at %s: %r, want %r" % (
        what, int(bad.sum()), torch.nonzero(bad)[0].tolist(), float(R.f64(got)[bad][0]), float(want[bad][0]))


# ------------------------------------------------------------------ quantization
SIZES = [(1, 1), (3, 7), (5, 32), (2, 511), (9, 512), (7, 520), (4, 2048), (3, 2049), (6, 2880), (2, 7168), (2, 14336),
         (1, 16391), (2, 20480)]


@pytest.mark.parametrize("rows,K", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quant_rows_exact(rows, K, dt):
    say("quant", rows, K, dt)
    x = (torch.randn((rows, K), generator=gen(K), device="cuda") * 3).to(R.TORCH_DT[dt])
    if K > 40:
        x[0, 5:37] = x[0].abs().max() / 2  # halves: 63.5
        x[0, 7:39:2] *= -1
    q = torch.full((rows, K), 99, dtype=torch.int8, device="cuda")
    s = torch.full((rows,), -1.0, device="cuda")
    moe.moe_quant_rows(x, q, s)
    torch.cuda.synchronize()
    v = R.f64(x)
    top = v.abs().amax(1, keepdim=True)
    # the product is exact in 64 bits and no ratio of two fp32 numbers comes closer to a half than 2^-33
    assert torch.equal(q.cpu().to(F64), torch.round(127 * v / top))
    near(s, top[:, 0] / 127, top[:, 0] / 127 * 2.0 ** -24 * 1.0001, "scale")


@pytest.mark.parametrize("scale", [1e-44, 1e-39, 1e-30, 1.0, 1e30, 3e38])
def test_quant_rows_range(scale):
    """Rows of any magnitude, fp32's smallest and largest included."""
    x = torch.rand((4, 100), generator=gen(1), device="cuda", dtype=torch.float64) * 2 - 1
    x = (x * scale).float()
    q = torch.empty((4, 100), dtype=torch.int8, device="cuda")
    s = torch.empty(4, device="cuda")
    moe.moe_quant_rows(x, q, s)
    torch.cuda.synchronize()
    v = R.f64(x)
    top = v.abs().amax(1, keepdim=True)
    assert torch.equal(q.cpu().to(F64), torch.round(127 * v / top))
    near(s, top[:, 0] / 127, top[:, 0] / 127 * 2.0 ** -24 + 2.0 ** -149, "scale")


def test_quant_rows_zero_and_nonfinite_rows():
    x = torch.randn((6, 300), generator=gen(2), device="cuda")
    x[1] = 0
    x[2, 17] = float("nan")
    x[3, 299] = float("inf")
    x[4, 0] = -float("inf")
    for t in (x, x.bfloat16()):
        q = torch.full((6, 300), 5, dtype=torch.int8, device="cuda")
        s = torch.empty(6, device="cuda")
        moe.moe_quant_rows(t, q, s)
        torch.cuda.synchronize()
        assert s[1] == 0 and (q[1:5] == 0).all()
        assert torch.isnan(s[2:5]).all()
        assert torch.isfinite(s[[0, 5]]).all() and (q[[0, 5]] != 0).any()


@pytest.mark.parametrize("rows,K", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quant_rows_swiglu(rows, K, dt):
    say("quant swiglu", rows, K, dt)
    x = (torch.randn((rows, 2 * K), generator=gen(K + 1), device="cuda") * 2).to(R.TORCH_DT[dt])
    q = torch.empty((rows, K), dtype=torch.int8, device="cuda")
    s = torch.empty(rows, device="cuda")
    moe.moe_quant_rows(x, q, s, act="swiglu")
    torch.cuda.synchronize()
    v = R.f64(x)
    v = v[:, :K] * torch.sigmoid(v[:, :K]) * v[:, K:]
    top = v.abs().amax(1, keepdim=True)
    # the gate in fp32: exp (2 steps of 2^-23), sum, quotient, product: below 8 * 2^-24 relative, the maximum alike;
    # 127 times both, and the integer is within half a step of that
    eps = 8 * 2.0 ** -24
    near(q, 127 * v / top.clamp(min=1e-300), 0.5 + 127 * 2 * eps, "q")
    near(s, top[:, 0] / 127, top[:, 0] / 127 * (eps + 2.0 ** -23), "scale")


def test_quant_rows_limit_and_misaligned():
    x = torch.randn((11 * 64 + 1,), generator=gen(3), device="cuda").bfloat16()
    for off in (0, 1):
        v = x[off:off + 11 * 64].view(11, 64)
        qb = torch.full((11 * 64 + 1,), 7, dtype=torch.int8, device="cuda")
        q = qb[off:off + 11 * 64].view(11, 64)
        s = torch.full((11,), 9.0, device="cuda")
        for n in (6, 0, -3, 100):
            q.fill_(7)
            s.fill_(9)
            moe.moe_quant_rows(v, q, s, n_rows=torch.tensor([n], dtype=torch.int32, device="cuda"))
            torch.cuda.synchronize()
            m = min(max(n, 0), 11)
            w = R.f64(v)[:m]
            if m:
                assert torch.equal(q[:m].cpu().to(F64), torch.round(127 * w / w.abs().amax(1, keepdim=True)))
            assert (q[m:] == 7).all() and (s[m:] == 9).all()
        assert qb[0 if off else -1] == 7


# ------------------------------------------------------------------ SwiGLU
def swiglu_ref(gu, dh):
    I = gu.shape[1] // 2
    g, u = gu[:, :I], gu[:, I:]
    s = torch.sigmoid(g)
    h = g * s * u
    if dh is None:
        return h, None, None
    # d SiLU / dg = s (1 + g (1 - s)): next to its zero at g = -1.28 the bracket cancels, so its error is bounded by
    # that of its two terms
    dg = dh * u * s * (1 + g * (1 - s))
    mag_dg = (dh * u * s).abs() * (1 + (g * (1 - s)).abs())
    return h, torch.cat([dg, dh * g * s], 1), torch.cat([mag_dg, (dh * g * s).abs()], 1)


# s: exp off by 2 steps (2^-23), 1 + e^-g and the quotient half a step each: 6 * 2^-24; 1 - s adds one rounding of a
# value up to 1 (absolute), three products more: 16 * 2^-24 covers all of them relative to the magnitudes
EPS_GATE = 16 * 2.0 ** -24


@pytest.mark.parametrize("rows,I", [(1, 1), (3, 5), (2, 8), (7, 40), (64, 2880), (5, 1111), (300, 96), (2, 14336),
                                    (70000, 8)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_swiglu_and_gradient(rows, I, dt):
    say("swiglu", rows, I, dt)
    t = R.TORCH_DT[dt]
    gu = (torch.randn((rows, 2 * I), generator=gen(I), device="cuda") * 4).to(t)
    dh = torch.randn((rows, I), generator=gen(I + 1), device="cuda").to(t)
    h, dgu, h2 = torch.empty_like(dh), torch.empty_like(gu), torch.empty_like(dh)
    dgu2 = torch.empty_like(gu)
    moe.moe_swiglu(gu, h)
    moe.moe_swiglu_grad(gu, dh, dgu, h=h2)
    moe.moe_swiglu_grad(gu, dh, dgu2)
    torch.cuda.synchronize()
    rh, rd, md = swiglu_ref(R.f64(gu), R.f64(dh))
    half = R.HALF_STEP[t]
    near(h, rh, rh.abs() * (half + EPS_GATE * (1 + half)) + 1e-37, "h")
    assert torch.equal(h, h2) and torch.equal(dgu, dgu2)
    near(dgu, rd, rd.abs() * half + md * EPS_GATE * (1 + half) + 1e-37, "dgu")


def test_swiglu_far_gates_limit_and_misaligned():
    g = torch.tensor([-1e30, -200.0, -88.0, -87.0, -20.0, 0.0, 20.0, 88.0, 200.0, 1e30], device="cuda")
    gu = torch.cat([g, torch.full_like(g, 0.5)]).repeat(4, 1)
    dh = torch.ones((4, 10), device="cuda")
    h, dgu = torch.full_like(dh, 77.0), torch.full_like(gu, 77.0)
    n = torch.tensor([3], dtype=torch.int32, device="cuda")
    moe.moe_swiglu(gu, h, n_rows=n)
    moe.moe_swiglu_grad(gu, dh, dgu, n_rows=n)
    torch.cuda.synchronize()
    rh, rd, md = swiglu_ref(R.f64(gu), R.f64(dh))
    # e^-g overflows fp32 from 88.7 on, where s is below 2^-127: the results are zeros then
    near(h[:3], rh[:3], rh[:3].abs() * 18 * 2.0 ** -24 + 1e-35, "h")
    near(dgu[:3], rd[:3], md[:3] * 18 * 2.0 ** -24 + 1e-35, "dgu")
    assert (h[3] == 77).all() and (dgu[3] == 77).all()
    base = torch.randn(1 + 3 * 48 * 2, generator=gen(9), device="cuda").bfloat16()
    a = base[1:].view(3, 96)  # rows that start on odd elements
    out = torch.zeros((3, 48), device="cuda", dtype=torch.bfloat16)
    ref = torch.zeros_like(out)
    moe.moe_swiglu(a, out)
    moe.moe_swiglu(a.clone(), ref)
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


def test_swiglu_gradient_against_differences():
    gu = torch.randn((6, 80), generator=gen(11), device="cuda")
    dh = torch.randn((6, 40), generator=gen(12), device="cuda")
    v = torch.randn((6, 80), generator=gen(13), device="cuda")
    dgu = torch.empty_like(gu)
    moe.moe_swiglu_grad(gu, dh, dgu)

    def loss(t):
        return float((swiglu_ref(t, None)[0] * R.f64(dh)).sum())

    eps = 1e-4  # the differences are taken in 64 bits: truncation O(eps^2), rounding 1e-16 / eps
    num = (loss(R.f64(gu) + eps * R.f64(v)) - loss(R.f64(gu) - eps * R.f64(v))) / (2 * eps)
    ana = float((R.f64(dgu) * R.f64(v)).sum())
    mag = float((R.f64(dgu).abs() * R.f64(v).abs()).sum())
    assert abs(num - ana) <= mag * 1e-6


# ------------------------------------------------------------------ gradient of the combine
@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 1), (1, 8, 8, 7168), (5, 2, 8, 77), (16, 4, 128, 2880), (40, 3, 16, 224),
                                     (9, 16, 1024, 100), (300, 5, 24, 256), (2, 8, 20, 9000)])
@pytest.mark.parametrize("odt,ydt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_combine_grad(T, k, E, H, odt, ydt, drop):
    say("combine grad", T, k, E, H, odt, ydt, drop)
    rng = np.random.default_rng(T * 1000 + H)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    dead = rng.random((T, k)) < drop
    ids[dead] = rng.choice([-1, E, 1 << 30])
    P = T * k
    flat = np.where(dead.reshape(-1), E, np.where(ids.reshape(-1) < 0, 0, ids.reshape(-1)))
    order = np.argsort(flat, kind="stable")
    placed = int((~dead).sum())
    inv = np.full(P, -1, np.int32)
    inv[order[:placed]] = np.arange(placed)
    dout = torch.randn((T, H), generator=gen(1), device="cuda").to(R.TORCH_DT[odt])
    y = torch.randn((P, H), generator=gen(2), device="cuda")
    w = torch.softmax(torch.randn((T, k), generator=gen(3), device="cuda"), 1)
    dy = torch.full((P, H), 77.0, device="cuda", dtype=R.TORCH_DT[ydt])
    dw = torch.full((T, k), 77.0, device="cuda")
    dl = torch.full((T, E), 77.0, device="cuda")
    tid, tinv = torch.from_numpy(ids).cuda(), torch.from_numpy(inv).cuda()
    moe.moe_combine_grad(dout, y, w, tinv, k, dy, dw, topk_ids=tid, dlogits=dl)
    dy2, dw2 = torch.full_like(dy, 77.0), torch.empty_like(dw)
    moe.moe_combine_grad(dout, y, w, tinv, k, dy2, dw2)
    torch.cuda.synchronize()
    assert torch.equal(dy, dy2) and torch.equal(dw, dw2)
    d, yy, ww = R.f64(dout), R.f64(y), R.f64(w)
    rdw, mag = torch.zeros((T, k), dtype=F64), torch.zeros((T, k), dtype=F64)
    half = R.HALF_STEP[R.TORCH_DT[ydt]]
    for t in range(T):
        for j in range(k):
            p = int(inv[t * k + j])
            if p < 0:
                continue
            want = ww[t, j] * d[t]
            near(dy[p], want, want.abs() * (half + 2.0 ** -24 * 1.01) + 1e-37, "dy")
            rdw[t, j] = (d[t] * yy[p]).sum()
            mag[t, j] = (d[t] * yy[p]).abs().sum()
    assert (dy[placed:] == 77).all()
    # a sum of H products: every addition (and product) off by 2^-24 of the magnitudes' sum at most
    bound = (H + 1) * 2.0 ** -24 * mag
    near(dw, rdw, bound + 1e-37, "dtopk_w")
    rl, lb = torch.zeros((T, E), dtype=F64), torch.zeros((T, E), dtype=F64)
    for t in range(T):
        mean = (ww[t] * rdw[t]).sum()
        # errors of the dot products, and k + 3 roundings of the magnitudes that are added up
        mb = (ww[t] * bound[t]).sum() + (k + 3) * 2.0 ** -24 * (ww[t] * (rdw[t].abs() + bound[t])).sum()
        for j in range(k):
            if inv[t * k + j] >= 0:
                rl[t, ids[t, j]] += ww[t, j] * (rdw[t, j] - mean)
                lb[t, ids[t, j]] += ww[t, j] * (bound[t, j] + mb + 4 * 2.0 ** -24 * (rdw[t, j].abs() + mean.abs()))
    near(dl, rl, lb + 1e-37, "dlogits")


def test_combine_grad_same_expert_twice_and_bad_positions():
    """A token that names one expert twice gets both parts in that logit; positions outside the rows are dropped."""
    T, k, E, H = 2, 3, 4, 64
    ids = torch.tensor([[1, 1, 2], [0, 3, 3]], dtype=torch.int32, device="cuda")
    inv = torch.tensor([0, 1, 2, 3, 1 << 30, -9], dtype=torch.int32, device="cuda")
    dout, y = torch.randn((T, H), generator=gen(4), device="cuda"), torch.randn((T * k, H), generator=gen(5), device="cuda")
    w = torch.softmax(torch.randn((T, k), generator=gen(6), device="cuda"), 1)
    dy, dw, dl = torch.full((T * k, H), 5.0, device="cuda"), torch.empty((T, k), device="cuda"), torch.empty((T, E), device="cuda")
    moe.moe_combine_grad(dout, y, w, inv, k, dy, dw, topk_ids=ids, dlogits=dl)
    torch.cuda.synchronize()
    assert (dy[4:] == 5).all() and (dw[1, 1:] == 0).all()
    d, yy, ww = R.f64(dout), R.f64(y), R.f64(w)
    r = torch.zeros((T, k), dtype=F64)
    for t, j, p in ((0, 0, 0), (0, 1, 1), (0, 2, 2), (1, 0, 3)):
        r[t, j] = (d[t] * yy[p]).sum()
    want = torch.zeros((T, E), dtype=F64)
    for t, j in ((0, 0), (0, 1), (0, 2), (1, 0)):
        want[t, ids[t, j].item()] += ww[t, j] * (r[t, j] - (ww[t] * r[t]).sum())
    near(dl, want, torch.full_like(want, 64 * 64 * 2.0 ** -24), "dlogits")
