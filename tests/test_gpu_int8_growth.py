"""The buffers of the 8-bit layer as its batches grow: what it holds, what captured graphs keep, and a growth that fails."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mixture_experts_layer_token_amd as moe  # noqa: E402
from mixture_experts_layer_token_amd import api  # noqa: E402
from mixture_experts_layer_token_amd.int8 import MoeInt8Layer  # noqa: E402

E, H, I, k = 8, 256, 128, 2


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


def layer_of(max_T, seed=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def w(*shape):
        return (torch.randn(shape, generator=g, device="cuda") * 0.1).bfloat16()

    return MoeInt8Layer(w(E, H), None, w(E, 2 * I, H), w(E, H, I), k, max_T=max_T)


def tokens(T, seed=2):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((T, H), generator=g, device="cuda").bfloat16()


def held(make):
    """Device bytes that what make() returns holds."""
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    kept = make()
    torch.cuda.synchronize()
    return torch.cuda.memory_allocated() - before, kept


def buffers_for(T):
    """Bytes of the buffers of a layer made for T tokens, beyond those of one made for a single token."""
    one, a = held(lambda: layer_of(1))
    many, b = held(lambda: layer_of(T))
    return many - one


def test_a_layer_that_grows_step_by_step_holds_one_set(monkeypatch):
    n = 200
    calls = []
    sizes = api.moe_route_permute_workspace
    monkeypatch.setattr(api, "moe_route_permute_workspace", lambda *a: calls.append(a) or sizes(*a))
    x, ref = tokens(n), layer_of(n).forward(tokens(n))
    calls.clear()

    def grown():
        layer = layer_of(1)
        for T in range(1, n + 1):
            layer.forward(x[:T])
        return layer

    used, layer = held(grown)
    assert len(calls) <= 2 * n  # (one query per batch size)
    one, _ = held(lambda: layer_of(1))
    assert used - one <= 2.2 * buffers_for(n)
    assert torch.equal(layer.forward(x), ref)


def test_captured_sets_stay_and_add_up_to_no_more_than_the_last():
    n = 40
    x = tokens(n)
    outs = [torch.empty((T, H), device="cuda", dtype=torch.bfloat16) for T in range(1, n + 1)]
    refs = [layer_of(n).forward(x[:T]) for T in range(1, n + 1)]
    one, layer = held(lambda: layer_of(1))
    base = torch.cuda.memory_allocated()
    graphs = []
    for T in range(1, n + 1):
        layer.forward(x[:T], outs[T - 1])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.forward(x[:T], outs[T - 1])
        graphs.append(g)
    torch.cuda.synchronize()
    # (one set of at most twice the size, and smaller ones that add up to as much; 512-byte blocks)
    assert torch.cuda.memory_allocated() - base <= 4.2 * buffers_for(n) + 100 * 512
    fill = [torch.full((1 << b,), 7, dtype=torch.uint8, device="cuda") for b in range(9, 18) for _ in range(8)]
    for rep in range(3):
        for o in outs:
            o.zero_()
        for g, o, r in zip(graphs, outs, refs):
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, r), "replay %d" % rep
        layer.forward(x * 0.5)  # eager work between the replays
    assert all(bool((f == 7).all()) for f in fill)


def test_growth_while_the_last_forward_runs_on_another_stream():
    """Memory of the buffers that go is not given out before the forward that uses them has ended."""
    T = 512
    x, more = tokens(T), tokens(2 * T + 1)
    ref, more_ref = layer_of(T).forward(x), layer_of(2 * T + 1).forward(more)
    side, busy = torch.cuda.Stream(), torch.ones((4096, 4096), device="cuda")
    for _ in range(3):
        layer = layer_of(T)  # buffers of the current stream
        out, more_out = torch.empty_like(x), torch.empty_like(more)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(4):
                busy @ busy
            layer.forward(x, out)
            layer.forward(more, more_out)
        junk = [torch.full((256 << b,), 3, dtype=torch.uint8, device="cuda") for b in range(14) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(more_out, more_ref)
        assert all(bool((j == 3).all()) for j in junk)


@pytest.mark.parametrize("after", range(13))
def test_a_growth_that_fails_leaves_the_layer_as_it_was(monkeypatch, after):
    """Memory runs out at any of the buffers: the layer must not take itself for a larger one (its kernels would write
    past buffers of the old size), and serves batches of the old size, and larger ones once there is memory."""
    T, n = 6, 40
    x, ref, small = tokens(n), layer_of(n).forward(tokens(n)), layer_of(T).forward(tokens(n)[:T])
    layer, empty, made = layer_of(T), torch.empty, []
    out = torch.empty_like(x)

    def scarce(*a, **kw):
        if len(made) % 13 == after:
            made.clear()
            raise torch.cuda.OutOfMemoryError("out of memory")
        made.append(1)
        return empty(*a, **kw)

    monkeypatch.setattr(torch, "empty", scarce)
    with pytest.raises(torch.cuda.OutOfMemoryError):
        layer.forward(x, out)
    monkeypatch.undo()
    assert layer.max_T == T
    for name in ("ids", "gates", "q", "q_scale"):
        assert getattr(layer, name).shape[0] == T, name
    for name in ("perm", "inv", "gu", "h", "h_scale", "y"):
        assert getattr(layer, name).shape[0] == T * k, name
    assert torch.equal(layer.forward(x[:T]), small)
    assert torch.equal(layer.forward(x), ref)


def test_memory_for_the_batch_but_not_for_twice_the_old_size(monkeypatch):
    T = 6
    x, ref, empty = tokens(T + 1), layer_of(T + 1).forward(tokens(T + 1)), torch.empty
    layer = layer_of(T)

    def scarce(*a, **kw):
        if a[0] == (2 * T, k):
            raise torch.cuda.OutOfMemoryError("out of memory")
        return empty(*a, **kw)

    monkeypatch.setattr(torch, "empty", scarce)
    got = layer.forward(x)
    monkeypatch.undo()
    assert layer.max_T == T + 1 and torch.equal(got, ref)
