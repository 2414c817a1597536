"""The training block whole: fused layer, shared expert, norm and clipping together against the same computation in 64 bits,
steps captured into graphs, parts that need no gradient, refusals."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mixture_experts_layer_token_amd as moe  # noqa: E402
from mixture_experts_layer_token_amd.train import GatedFFN, MoeTrainBlock, MoeTrainLayer, Norm, clip_grad_norm  # noqa: E402

from grouped_ref import f64  # noqa: E402
from helpers import say  # noqa: E402
from test_gpu_train import reference, rel, routed  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


# as in test_gpu_train: chains of fp32 sums; in bf16 up to eight tensors on the way are rounded (n, gu, h, out, sums; dy, dgu,
# dn), each by at most 2^-8 of its norm
TOL = {torch.float32: 2e-5, torch.bfloat16: 8 * 2.0 ** -8}


def norm64(x, w, b, rms, eps):
    d = x if rms else x - x.mean(1, keepdim=True)
    y = d / ((d * d).mean(1, keepdim=True) + eps).sqrt() * w
    return y if b is None else y + b


def gated64(x, wgu, wd):
    I = wd.shape[1]
    gu = x @ wgu.T
    return (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]) @ wd.T


def leaves64(module):
    return {n: f64(p).requires_grad_() for n, p in module.named_parameters()}


def block64(p, x, ids, rms, eps):
    n = norm64(x, p["norm.weight"], p.get("norm.bias"), rms, eps)
    out = x + reference(n, p["layer.w_router"], p.get("layer.bias"), p["layer.w_gate_up"], p["layer.w_down"], ids)
    return out + gated64(n, p["shared.w_gate_up"], p["shared.w_down"]) if "shared.w_gate_up" in p else out


def make(T, H, I, E, k, shared, rms, dtype, bias, seed=0):
    torch.manual_seed(seed)
    block = MoeTrainBlock(H, I, E, k, shared_I=shared, rms=rms, dtype=dtype, bias=bias, sigma=0.1)
    with torch.no_grad():
        block.norm.weight.add_(0.2 * torch.randn(H, device="cuda"))
        if block.norm.bias is not None:
            block.norm.bias.add_(0.2 * torch.randn(H, device="cuda"))
    x = (torch.randn((T, H), device="cuda") + 0.3).to(dtype).requires_grad_()
    dout = torch.randn((T, H), device="cuda").to(dtype)
    return block, x, dout


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,H,I,E,k,shared,rms,bias", [(1, 64, 32, 4, 2, 40, True, False), (40, 224, 352, 16, 4, None, False, True),
                                                       (333, 96, 72, 5, 2, 77, False, False), (7, 64, 64, 300, 8, 64, True, True),
                                                       (600, 256, 320, 3, 2, 512, True, False)])
def test_block_step_against_64_bits(T, H, I, E, k, shared, rms, bias, dtype):
    say("train block", T, H, I, E, k, shared, rms, bias, dtype)
    block, x, dout = make(T, H, I, E, k, shared, rms, dtype, bias)
    out = block(x)
    out.backward(dout)
    before = {n: f64(p.grad) for n, p in block.named_parameters()}
    norm = clip_grad_norm(block.parameters(), 0.05)
    torch.cuda.synchronize()
    ids = routed(block.layer, block.norm(x.detach()).detach())
    p, x64 = leaves64(block), f64(x).requires_grad_()
    ref = block64(p, x64, ids, rms, 1e-5)
    ref.backward(f64(dout))
    tol = TOL[dtype]
    assert rel(out, ref.detach()) <= tol
    assert rel(x.grad, x64.grad) <= tol
    total = math.sqrt(sum(float((g * g).sum()) for g in before.values()))
    assert abs(float(norm) - total) <= 2.0 ** -23 * total and total > 0.05
    for n, q in block.named_parameters():
        say("  d", n, rel(before[n], p[n].grad) if p[n].grad.norm() > 0 else 0)
        assert rel(before[n], p[n].grad) <= tol, n
        # the clipped gradient: scaled and rounded once
        want = before[n] * (0.05 / total)
        assert ((f64(q.grad) - want).abs() <= (torch.finfo(q.dtype).eps / 2 + 2.0 ** -22) * want.abs() + 1e-37).all(), n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_fused_layer_follows_the_unfused_one(dtype):
    """The same parameters: outputs and gradients of the two differ by the roundings of gu, h, dh and dgu alone."""
    torch.manual_seed(1)
    a = MoeTrainLayer(256, 192, 8, 2, dtype=dtype, sigma=0.1)
    b = MoeTrainLayer(256, 192, 8, 2, dtype=dtype, sigma=0.1, fused=True)
    b.load_state_dict(a.state_dict())
    res = []
    x0, dout = torch.randn((90, 256), device="cuda").to(dtype), torch.randn((90, 256), device="cuda").to(dtype)
    for layer in (a, b):
        x = x0.clone().requires_grad_()
        out = layer(x)
        res.append([out.detach()] + list(torch.autograd.grad(out, [x] + list(layer.parameters()), dout)))
    for p, q in zip(*res):
        assert rel(p, f64(q)) <= (4 * 2.0 ** -8 if dtype == torch.bfloat16 else 1e-5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,H,I", [(1, 8, 8), (5, 33, 17), (300, 256, 640), (2000, 128, 96)])
def test_gated_ffn(T, H, I, dtype):
    torch.manual_seed(2)
    ffn = GatedFFN(H, I, dtype=dtype, sigma=0.2)
    x = torch.randn((T, H), device="cuda").to(dtype).requires_grad_()
    dout = torch.randn((T, H), device="cuda").to(dtype)
    out = ffn(x)
    out.backward(dout)
    p, x64 = leaves64(ffn), f64(x).requires_grad_()
    ref = gated64(x64, p["w_gate_up"], p["w_down"])
    ref.backward(f64(dout))
    tol = 4 * 2.0 ** -8 if dtype == torch.bfloat16 else 1e-5
    assert rel(out, ref.detach()) <= tol and rel(x.grad, x64.grad) <= tol
    for n, q in ffn.named_parameters():
        assert rel(q.grad, p[n].grad) <= tol, n
    with torch.no_grad():
        assert torch.equal(ffn(x), out)


def test_gradients_against_differences():
    """Directional derivatives of the whole block in fp32 against central differences of the 64-bit block."""
    block, x, dout = make(21, 64, 48, 6, 2, 32, False, torch.float32, True, seed=3)
    block(x).backward(dout)
    ids = routed(block.layer, block.norm(x.detach()).detach())
    p = {n: f64(q) for n, q in block.named_parameters()}
    grads = dict({n: f64(q.grad) for n, q in block.named_parameters()}, x=f64(x.grad))
    p["x"] = f64(x)
    gen = torch.Generator().manual_seed(4)
    for name in p:
        v = torch.randn(p[name].shape, generator=gen, dtype=torch.float64) * p[name].abs().max().clamp(min=0.1)

        def loss(s):
            q = dict(p)
            q[name] = p[name] + s * 1e-5 * v
            xs = q.pop("x")
            return float((block64(q, xs, ids, False, 1e-5) * f64(dout)).sum())

        num, ana = (loss(1) - loss(-1)) / 2e-5, grads[name] * v
        assert abs(num - float(ana.sum())) <= 1e-5 * float(ana.abs().sum()) + 1e-8, name


def test_parts_that_need_no_gradient():
    block, x, dout = make(30, 64, 32, 4, 2, 32, False, torch.bfloat16, False, seed=5)
    block(x).backward(dout)
    full = {n: p.grad.clone() for n, p in block.named_parameters()}
    for name, p in block.named_parameters():
        for q in block.parameters():
            q.grad = None
            q.requires_grad_(False)
        p.requires_grad_(True)
        block(x.detach()).backward(dout)
        assert torch.equal(p.grad, full[name]), name
        assert all(q.grad is None for q in block.parameters() if q is not p)
    for q in block.parameters():
        q.grad = None
        q.requires_grad_(True)
    # only the residual leaves the norm; only the norm leaves it
    norm = Norm(64, dtype=torch.float32)
    y = torch.randn((9, 64), device="cuda", requires_grad=True)
    n, res = norm.with_residual(y)
    g, = torch.autograd.grad((res * 2).sum(), [y])
    assert torch.equal(g, torch.full_like(g, 2.0))
    (norm(y) * torch.randn((9, 64), device="cuda")).sum().backward()
    assert torch.isfinite(y.grad).all()
    empty = torch.empty((0, 64), device="cuda", dtype=torch.bfloat16, requires_grad=True)
    out = block(empty)
    out.sum().backward()
    assert out.shape == (0, 64) and all((q.grad == 0).all() for q in block.parameters())
    with torch.no_grad():
        assert torch.equal(block(x), block(x))


def test_training_steps_run():
    block, x, _ = make(200, 64, 96, 8, 2, 64, True, torch.bfloat16, True, seed=6)
    opt = torch.optim.SGD(block.parameters(), lr=0.05)
    for _ in range(3):
        loss = (block(x.detach()).float() - 1).square().mean()
        opt.zero_grad()
        loss.backward()
        norm = clip_grad_norm(block.parameters(), 1.0)
        opt.step()
        assert torch.isfinite(loss) and torch.isfinite(norm).all()
    assert all(torch.isfinite(p.float()).all() for p in block.parameters())


def test_captured_step_replays():
    block, x, dout = make(150, 96, 64, 8, 2, 48, False, torch.bfloat16, False, seed=7)
    params = list(block.parameters())

    def step():
        out = block(x)
        grads = torch.autograd.grad(out, [x] + params, dout)
        norm = torch.empty(1, device="cuda")
        outs = [torch.empty_like(g) for g in grads[1:]]
        moe.moe_clip_grad_norm(list(grads[1:]), 0.5, norm, outs=outs)
        return [out.detach(), grads[0], norm] + outs

    eager = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for rep in range(4):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for p, q in zip(got, eager):
            assert torch.equal(p, q), "replay %d" % rep
        with torch.no_grad():
            block(x * 0.5)
        torch.cuda.synchronize()


def test_shared_and_missing_gradients():
    a, b = (torch.nn.Parameter(torch.ones(10, device="cuda")) for _ in range(2))
    assert float(clip_grad_norm([a, b], 1.0)) == 0.0
    a.grad = torch.full((10,), 2.0, device="cuda")
    assert abs(float(clip_grad_norm([a, b, a], 1.0)) - 40 ** 0.5) <= 1e-6
    assert abs(float(a.grad.norm()) - 1) <= 1e-6
    b.grad = a.grad  # one tensor under two names counts once
    assert abs(float(clip_grad_norm([a, b], 2.0)) - 1) <= 1e-6
    assert abs(float(clip_grad_norm(a, 0.5)) - 1) <= 1e-6 and abs(float(b.grad.norm()) - 0.5) <= 1e-6


def test_refusals():
    block, x, _ = make(4, 64, 32, 4, 2, 32, True, torch.bfloat16, False)
    for bad in (x[:, :32], x[0], x.detach().cpu()):
        for m in (block, block.norm, block.shared):
            with pytest.raises(ValueError):
                m(bad)
    with pytest.raises(TypeError):
        block.shared(x.float())
    with pytest.raises(TypeError):
        Norm(64, dtype=torch.float16)(x)
    p = torch.nn.Parameter(torch.ones(4, device="cuda", dtype=torch.float16))
    p.grad = torch.ones_like(p)
    with pytest.raises(TypeError):
        clip_grad_norm([p], 1.0)
