"""Combinations of the grouped products' paths against 64-bit references: gathered rows in a weight gradient cut into parts,
expert strides larger than a matrix, calls with a workspace in flight together and in a graph, int8 sums of the full
length, and weights, results and weight gradients past 4 GiB."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mixture_experts_layer_token_amd as moe  # noqa: E402

import grouped_ref as R  # noqa: E402
from grouped_ref import f64  # noqa: E402
from helpers import say  # noqa: E402
from test_gpu_grouped import SENTINEL, make, reference_on_gpu, rows_tensor  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def nan_workspace(dt, rows, N, K, E):
    """Workspace whose every float is NaN: a part that is not written shows."""
    need = moe.moe_grouped_workspace("f32" if dt == torch.float32 else "bf16", rows, N, K, E)
    return need, torch.full((max(need, 256),), 0xFF, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ gathered rows, in parts
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("layout", ["dense", "padded", "shifted"])
@pytest.mark.parametrize("counts,N,K,k", [([9001], 24, 40, 4), ([4099, 2], 136, 200, 2), ([1, 0, 6000], 8, 520, 3),
                                          ([1025], 390, 1030, 1), ([2570, 2600], 256, 384, 16)])
def test_gathered_weight_gradient_in_parts(counts, N, K, k, layout, dt):
    say("grouped gathered parts", counts, N, K, k, layout, dt)
    off, E, rows = R.offsets_of(counts), len(counts), sum(counts) + 5
    T = rows // k + 3
    _, x = rows_tensor((T, K), dt, layout, gen(41))
    _, dy = rows_tensor((rows, N), dt, layout, gen(42))
    perm = torch.randint(0, T * k, (rows,), generator=gen(43), device="cuda", dtype=torch.int32)
    perm[::37] = -1
    perm[5::41] = T * k
    need, ws = nan_workspace(dt, rows, N, K, E)
    assert need >= 2 * E * N * K * 4
    src = torch.div(perm, k, rounding_mode="floor").long()
    named = (perm >= 0) & (src < T)
    xg = torch.where(named[:, None], x[src.clamp(0, T - 1)], torch.zeros((), dtype=dt, device="cuda"))
    for out in (torch.float32, torch.bfloat16):
        dw = torch.empty((E, N, K), device="cuda", dtype=out)
        moe.moe_grouped_gemm_dw(dy, x, torch.from_numpy(off).cuda(), dw, perm_src=perm, k=k, ws=ws)
        torch.cuda.synchronize()
        R.assert_product(dw, *reference_on_gpu("dw", xg, None, dy, off), what="dw")


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,N,K,aligned", [([1024] * 8, 640, 640, True), ([1024] * 8, 640, 640, False),
                                                ([8192], 1920, 1536, True)])
def test_weight_gradient_whose_tiles_fill_the_card_is_summed_in_one(counts, N, K, aligned, dt):
    """180 to 200 tiles: with one workgroup to a compute unit two parts each would take two rounds of half the length.  Rows
    on no 16-byte boundary go two to a unit, and bf16 ones are cut."""
    off, E, rows = R.offsets_of(counts), len(counts), sum(counts)
    _, x = rows_tensor((rows, K), dt, "dense" if aligned else "shifted", gen(44))
    _, dy = rows_tensor((rows, N), dt, "dense", gen(45))
    need, ws = nan_workspace(dt, rows, N, K, E)
    dw = torch.empty((E, N, K), device="cuda")
    moe.moe_grouped_gemm_dw(dy, x, torch.from_numpy(off).cuda(), dw, ws=ws)
    torch.cuda.synchronize()
    R.assert_product(dw, *reference_on_gpu("dw", x, None, dy, off), what="dw")
    assert bool((ws == 0xFF).all()) == (aligned or dt == torch.float32)


# ------------------------------------------------------------------ expert strides
def spread(E, N, K, pad, dt, fill):
    """[E, N, K] view of a buffer with `pad` elements between experts, and the buffer."""
    full = torch.full((E * (N * K + pad),), fill, dtype=dt, device="cuda")
    return full, full.as_strided((E, N, K), (N * K + pad, K, 1))


def gaps_hold(full, E, n, pad, value):
    return bool((full.view(E, n + pad)[:, n:] == torch.tensor(value, dtype=full.dtype, device="cuda")).all())


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad", [64, 7])
@pytest.mark.parametrize("name", ["ragged", "odd", "decode", "tiles", "many", "skinny"])
def test_expert_stride_larger_than_a_matrix(name, pad, dt):
    say("grouped expert stride", name, pad, dt)
    c = make(name, dt, spare=3)
    E, N, K, rows = c["E"], c["N"], c["K"], c["rows"]
    _, w = spread(E, N, K, pad, dt, float("nan"))
    w.copy_(c["w"])
    y, dx = torch.full((rows, N), SENTINEL, device="cuda"), torch.full((rows, K), SENTINEL, device="cuda")
    need, ws = nan_workspace(dt, rows, N, K, E)
    moe.moe_grouped_gemm(c["x"], w, c["offsets"], y, ws=ws)
    moe.moe_grouped_gemm_dx(c["dy"], w, c["offsets"], dx, ws=ws)
    full, dw = spread(E, N, K, pad, torch.float32, SENTINEL)
    moe.moe_grouped_gemm_dw(c["dy"], c["x"], c["offsets"], dw, ws=ws)
    torch.cuda.synchronize()
    x, ww, dy = f64(c["x"]), f64(c["w"]), f64(c["dy"])
    R.assert_product(y, *R.product("y", x, ww, None, c["off"]), what="y")
    R.assert_product(dx, *R.product("dx", None, ww, dy, c["off"]), what="dx")
    R.assert_product(dw, *R.product("dw", x, None, dy, c["off"]), what="dw")
    assert gaps_hold(full, E, N * K, pad, SENTINEL)
    assert (y[c["placed"]:] == SENTINEL).all() and (dx[c["placed"]:] == SENTINEL).all()


@pytest.mark.parametrize("pad", [64, 7])
@pytest.mark.parametrize("name", ["ragged", "odd", "decode", "tiles"])
def test_int8_expert_stride_larger_than_a_matrix(name, pad):
    c = make(name, torch.float32)
    E, N, K, rows = c["E"], c["N"], c["K"], c["rows"]
    q = torch.randint(-128, 128, (rows, K), generator=gen(1), device="cuda").to(torch.int8)
    _, w = spread(E, N, K, pad, torch.int8, 111)
    w.copy_(torch.randint(-128, 128, (E, N, K), generator=gen(2), device="cuda").to(torch.int8))
    y = torch.empty((rows, N), device="cuda")
    moe.moe_grouped_gemm_i8(q, torch.ones(rows, device="cuda"), w, torch.ones((E, N), device="cuda"), c["offsets"], y)
    torch.cuda.synchronize()
    v, _, _ = R.product("y", f64(q), f64(w), None, c["off"])
    assert float(v.abs().max()) < 1 << 24 and torch.equal(f64(y), v)  # exact in fp32, with scales of 1


# ------------------------------------------------------------------ int8 sums
@pytest.mark.parametrize("rows,N,K", [(2, 5, 131071), (40, 33, 131056), (200, 600, 131056), (200, 150, 131071),
                                      (2100, 2100, 131056)])
def test_int8_sums_of_the_full_length(rows, N, K):
    """Up to 131071 products of -128 with -128, 16 KiB below 2^31: sums held in fp32 would round, in fewer bits or past
    int32 wrap around.  With scales of 1 the result is the sum, rounded once to fp32."""
    say("int8 long sums", rows, N, K)
    q = torch.full((rows, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((1, N, K), -128, dtype=torch.int8, device="cuda")
    q[1::2] = torch.randint(-128, 128, (q[1::2].shape[0], K), generator=gen(3), device="cuda").to(torch.int8)
    q[::2, 7::11] = torch.randint(-128, -120, q[::2, 7::11].shape, generator=gen(4), device="cuda").to(torch.int8)
    w[0, 1::3] = torch.randint(-128, 128, (w[0, 1::3].shape[0], K), generator=gen(5), device="cuda").to(torch.int8)
    w[0, 2::3] = 127
    q[0] = -128
    y = torch.empty((rows, N), device="cuda")
    moe.moe_grouped_gemm_i8(q, torch.ones(rows, device="cuda"), w, torch.ones((1, N), device="cuda"),
                            torch.tensor([0, rows], dtype=torch.int32, device="cuda"), y)
    torch.cuda.synchronize()
    v = torch.zeros((rows, N), dtype=torch.float64, device="cuda")
    for k0 in range(0, K, 16384):
        v += q[:, k0:k0 + 16384].double() @ w[0, :, k0:k0 + 16384].double().T  # exact
    assert float(v[0, 0]) == 16384.0 * K
    assert torch.equal(y, v.float())


# ------------------------------------------------------------------ workspaces in flight and in graphs
def test_two_calls_with_workspaces_at_once():
    cs = [make("skinny", torch.bfloat16, seed=s) for s in (1, 2)]
    dims = [(c["rows"], c["N"], c["K"], c["E"]) for c in cs]
    refs = []
    for c in cs:
        dw = torch.zeros((c["E"], c["N"], c["K"]), device="cuda")
        moe.moe_grouped_gemm_dw(c["dy"], c["x"], c["offsets"], dw)
        refs.append(dw)
    assert not torch.equal(refs[0], refs[1])
    spaces = []
    for d in dims:
        need, ws = nan_workspace(torch.bfloat16, *d)
        assert need > 0
        spaces.append(ws)
    outs, streams = [torch.zeros_like(r) for r in refs], [torch.cuda.Stream() for _ in cs]
    busy = torch.ones((2048, 2048), device="cuda")
    torch.cuda.synchronize()
    for own in (True, False):  # workspaces of the caller's, and allocated in the call
        for _ in range(3):
            for c, o, s, ws in zip(cs, outs, streams, spaces):
                with torch.cuda.stream(s):
                    o.zero_()
                    busy @ busy
                    moe.moe_grouped_gemm_dw(c["dy"], c["x"], c["offsets"], o, ws=ws if own else None)
            torch.cuda.synchronize()
            for o, r in zip(outs, refs):
                assert torch.equal(o, r)


@pytest.mark.parametrize("own", [True, False])
def test_graphs_with_workspaces_replay(own):
    """Two graphs, each with a workspace of its own (the caller's, or allocated during capture), replayed in turn."""
    cs = [make("skinny", torch.bfloat16, seed=s) for s in (3, 4)]
    refs, outs, graphs, keep = [], [], [], []
    for c in cs:
        dims = (c["rows"], c["N"], c["K"], c["E"])
        ref, dw = torch.zeros(dims[3], dims[1], dims[2], device="cuda"), torch.zeros(dims[3], dims[1], dims[2], device="cuda")
        need, ws = nan_workspace(torch.bfloat16, *dims)
        assert need > 0
        kw = dict(ws=ws) if own else {}
        moe.moe_grouped_gemm_dw(c["dy"], c["x"], c["offsets"], ref, **kw)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_grouped_gemm_dw(c["dy"], c["x"], c["offsets"], dw, **kw)
        refs.append(ref), outs.append(dw), graphs.append(g), keep.append(ws)
    for rep in range(4):
        for g, o, r in zip(graphs, outs, refs):
            o.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, r), "replay %d" % rep
        eager = torch.empty_like(refs[0])  # eager work between the replays
        moe.moe_grouped_gemm_dw(cs[0]["dy"] * 2, cs[0]["x"], cs[0]["offsets"], eager)
        torch.cuda.synchronize()
        assert torch.equal(eager, refs[0] * 2)


# ------------------------------------------------------------------ past 4 GiB
@pytest.mark.parametrize("counts", [[3, 0, 30], [200, 1, 300]])
def test_weights_and_their_gradients_past_four_gigabytes(counts):
    """The last expert's matrix starts past 4 GiB: bf16 weights read by both products, an fp32 gradient, int8 weights."""
    N, K, E = 96, 512, 3
    off, rows = R.offsets_of(counts), sum(counts)
    stride = (1 << 31) + 64  # elements: 4 GiB and more even for int8, and 16-byte rows
    buf = torch.empty((E - 1) * stride * 2 + 4 * N * K, dtype=torch.uint8, device="cuda")
    w = buf.view(torch.bfloat16).as_strided((E, N, K), (stride, K, 1))
    x, dy = (torch.randn((rows, d), generator=gen(7), device="cuda").bfloat16() for d in (K, N))
    w.copy_(torch.randn((E, N, K), generator=gen(8), device="cuda"))
    offsets = torch.from_numpy(off).cuda()
    y, dx = torch.empty((rows, N), device="cuda"), torch.empty((rows, K), device="cuda")
    moe.moe_grouped_gemm(x, w, offsets, y)
    moe.moe_grouped_gemm_dx(dy, w, offsets, dx)
    torch.cuda.synchronize()
    R.assert_product(y, *R.product("y", f64(x), f64(w), None, off), what="y")
    R.assert_product(dx, *R.product("dx", None, f64(w), f64(dy), off), what="dx")
    q, w8 = (torch.randint(-128, 128, s, generator=gen(9), device="cuda").to(torch.int8) for s in ((rows, K), (E, N, K)))
    i8 = buf.view(torch.int8).as_strided((E, N, K), (stride, K, 1))
    i8.copy_(w8)
    moe.moe_grouped_gemm_i8(q, torch.ones(rows, device="cuda"), i8, torch.ones((E, N), device="cuda"), offsets, y)
    torch.cuda.synchronize()
    v = R.product("y", f64(q), f64(w8), None, off)[0]
    assert float(v.abs().max()) < 1 << 24 and torch.equal(f64(y), v)  # exact in fp32, with scales of 1
    dw = buf.view(torch.float32).as_strided((E, N, K), (stride // 2, K, 1))
    dw.fill_(SENTINEL)
    moe.moe_grouped_gemm_dw(dy, x, offsets, dw)
    torch.cuda.synchronize()
    R.assert_product(dw, *R.product("dw", f64(x), None, f64(dy), off), what="dw")


def test_rows_of_results_and_operands_past_four_gigabytes():
    """Rows 8 MB apart, 1100 of them: results of both products, and operands of the weight gradient, past 4 GiB."""
    N, K, E, ld = 64, 96, 2, (1 << 22) - 128
    off = np.array([0, 520, 1100], np.int32)
    rows, offsets = 1100, torch.from_numpy(off).cuda()
    buf = torch.empty((rows, ld), dtype=torch.bfloat16, device="cuda")
    x, dy = buf[:, :K], buf[:, 256:256 + N]
    x.copy_(torch.randn((rows, K), generator=gen(11), device="cuda"))
    dy.copy_(torch.randn((rows, N), generator=gen(12), device="cuda"))
    w = torch.randn((E, N, K), generator=gen(13), device="cuda").bfloat16()
    dw = torch.empty((E, N, K), device="cuda")
    y, dx = buf[:, 512:512 + N], buf[:, 1024:1024 + K]
    moe.moe_grouped_gemm(x, w, offsets, y)
    moe.moe_grouped_gemm_dx(dy, w, offsets, dx)
    moe.moe_grouped_gemm_dw(dy, x, offsets, dw)
    torch.cuda.synchronize()
    R.assert_product(y, *R.product("y", f64(x), f64(w), None, off), what="y")
    R.assert_product(dx, *R.product("dx", None, f64(w), f64(dy), off), what="dx")
    R.assert_product(dw, *R.product("dw", f64(x), None, f64(dy), off), what="dw")
    # the same rows, gathered: no descriptor covers all of them
    perm = torch.randint(0, 2 * rows, (rows,), generator=gen(14), device="cuda", dtype=torch.int32)
    xg = R.gathered(x, perm, 2, rows)
    moe.moe_grouped_gemm(x, w, offsets, y, perm_src=perm, k=2)
    moe.moe_grouped_gemm_dw(dy, x, offsets, dw, perm_src=perm, k=2)
    torch.cuda.synchronize()
    R.assert_product(y, *R.product("y", xg, f64(w), None, off), what="gathered y")
    R.assert_product(dw, *R.product("dw", xg, None, f64(dy), off), what="gathered dw")
