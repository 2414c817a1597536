"""The training block's operators past 32-bit offsets, on two streams at once, and in graphs that run at the same time."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mixture_experts_layer_token_amd as moe  # noqa: E402

from grouped_ref import f64  # noqa: E402
from helpers import say  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


def test_norm_of_more_than_4_gib():
    """A row's results do not depend on where it lies; dweight of rows of which most have no gradient is that of the others."""
    rows, H = 1_100_000, 2048  # 4.5 GB
    say("norm, large")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x, y, dx = (torch.empty((rows, H), device="cuda", dtype=torch.bfloat16) for _ in range(3))
    dy = torch.zeros((rows, H), device="cuda", dtype=torch.bfloat16)
    for i in range(0, rows, 100_000):
        x[i:i + 100_000] = torch.randn((100_000, H), generator=gen, device="cuda")
    pick = [0, 1, 523_777, 1_048_575, 1_048_576, 1_048_577, 1_099_999]  # (rows 2^20 and on start past 4 GiB)
    dy[pick] = torch.randn((len(pick), H), generator=gen, device="cuda").bfloat16()
    w, b = (torch.randn(H, generator=gen, device="cuda").bfloat16() for _ in range(2))
    stats = torch.empty((rows, 2), device="cuda")
    dw, db = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    moe.moe_norm(x, w, b, y, stats=stats)
    moe.moe_norm_grad(dy, x, None, stats, dx, dweight=dw, dbias=db)
    xs, ys, dxs, ss = x[pick].contiguous(), torch.empty((7, H), device="cuda", dtype=torch.bfloat16), torch.empty(
        (7, H), device="cuda", dtype=torch.bfloat16), torch.empty((7, 2), device="cuda")
    dws, dbs = torch.empty_like(dw), torch.empty_like(db)
    moe.moe_norm(xs, w, b, ys, stats=ss)
    moe.moe_norm_grad(dy[pick].contiguous(), xs, None, ss, dxs, dweight=dws, dbias=dbs)
    torch.cuda.synchronize()
    # (few rows and many run with other shares of a row to a lane: sums in another order, one rounding apart)
    assert torch.allclose(stats[pick], ss, rtol=1e-5, atol=1e-6)
    for got, want in ((y[pick], ys), (dx[pick], dxs)):
        assert ((f64(got) - f64(want)).abs() <= 2.0 ** -7 * f64(want).abs() + 1e-3).all()
    assert torch.allclose(dw, dws, rtol=1e-4, atol=1e-4) and torch.allclose(db, dbs, rtol=1e-5, atol=1e-5)


def test_gradients_of_more_than_2_to_the_32_elements():
    n = (1 << 32) + 12345
    say("clip, large")
    g = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    for i in (0, 1, (1 << 31) - 1, 1 << 31, (1 << 32) - 1, 1 << 32, n - 1):
        g[i] = 3.0
    other = torch.full((1000,), 2.0, device="cuda")
    norm = torch.empty(1, device="cuda")
    moe.moe_clip_grad_norm([g, other], 1.0, norm)
    torch.cuda.synchronize()
    total = math.sqrt(7 * 9 + 4000)
    assert abs(float(norm) - total) <= 2.0 ** -23 * total
    want = torch.tensor(3.0 / total, dtype=torch.float64).bfloat16()
    for i in (0, 1, (1 << 31) - 1, 1 << 31, (1 << 32) - 1, 1 << 32, n - 1):
        assert abs(float(g[i]) - float(want)) <= 2.0 ** -8 * float(want)
    assert int(torch.count_nonzero(g[:1 << 31])) == 3 and int(torch.count_nonzero(g[1 << 31:])) == 4


def test_block_of_results_past_4_gib():
    """h and [g | u] past 4 GiB: the last rows are those of the same rows alone."""
    rows, I, K = 140_000, 8192, 64  # gu: 4.6 GB
    say("block, large")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    x = torch.randn((rows, K), generator=gen, device="cuda").bfloat16()
    w = (torch.randn((1, 2 * I, K), generator=gen, device="cuda") * 0.2).bfloat16()
    down = (torch.randn((1, K, I), generator=gen, device="cuda") * 0.1).bfloat16()
    h, gu = (torch.empty((rows, n * I), device="cuda", dtype=torch.bfloat16) for n in (1, 2))
    moe.moe_grouped_swiglu(x, w, torch.tensor([0, rows], dtype=torch.int32, device="cuda"), h, gu=gu)
    dgu, h2 = torch.empty_like(gu), torch.empty_like(h)
    moe.moe_grouped_swiglu_dx(x, down, gu, torch.tensor([0, rows], dtype=torch.int32, device="cuda"), dgu, h=h2)
    n = 512
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    hs, gus = (torch.empty((n, m * I), device="cuda", dtype=torch.bfloat16) for m in (1, 2))
    moe.moe_grouped_swiglu(x[-n:], w, off, hs, gu=gus)
    dgus, h2s = torch.empty_like(gus), torch.empty_like(hs)
    moe.moe_grouped_swiglu_dx(x[-n:], down, gus, off, dgus, h=h2s)
    torch.cuda.synchronize()
    # (K is one MFMA step pair: every tile shape adds up in the same order)
    for big, small in ((h, hs), (gu, gus), (dgu, dgus), (h2, h2s)):
        assert torch.equal(big[-n:], small)


def test_two_streams_at_once():
    """The same calls on two streams with tensors of their own, many times over: nothing is shared between them."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    x = torch.randn((3000, 2880), generator=gen, device="cuda").bfloat16()
    dy = torch.randn((3000, 2880), generator=gen, device="cuda").bfloat16()
    w = torch.randn(2880, generator=gen, device="cuda").bfloat16()

    def step():
        y, dx, st = torch.empty_like(x), torch.empty_like(x), torch.empty((3000, 2), device="cuda")
        dw, db, norm = torch.empty_like(w), torch.empty_like(w), torch.empty(1, device="cuda")
        moe.moe_norm(x, w, None, y, stats=st)
        moe.moe_norm_grad(dy, x, w, st, dx, dweight=dw, dbias=db)
        moe.moe_clip_grad_norm([dw, db, dx], 0.1, norm)
        return [y, dx, dw, db, norm]

    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(step())
    torch.cuda.synchronize()
    for res in got:
        assert all(torch.equal(p, q) for p, q in zip(res, want))


def test_two_graphs_at_once():
    """Two captured steps replayed together on two streams: their workspaces are their own."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    xs = [torch.randn((1500, 4096), generator=gen, device="cuda").bfloat16() for _ in range(2)]
    dy = torch.randn((1500, 4096), generator=gen, device="cuda").bfloat16()
    w = torch.randn(4096, generator=gen, device="cuda").bfloat16()

    def step(x):
        dx, st = torch.empty_like(x), torch.empty((1500, 2), device="cuda")
        y, dw, db, norm = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w), torch.empty(1, device="cuda")
        moe.moe_norm(x, w, None, y, stats=st)
        moe.moe_norm_grad(dy, x, w, st, dx, dweight=dw, dbias=db)
        outs = [torch.empty_like(t) for t in (dw, db)]
        moe.moe_clip_grad_norm([dw, db], 0.1, norm, outs=outs)
        return [y, dx, norm] + outs

    want = [[t.clone() for t in step(x)] for x in xs]
    torch.cuda.synchronize()
    graphs, got = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(step(x))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(4):
        for res in got:
            for t in res:
                t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for res, ref in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(res, ref)), rep
