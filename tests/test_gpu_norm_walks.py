"""Norms of more rows than one round of workgroups takes, against 64-bit references: every kernel's walk over the rows, with a last
round that not all of its rows' teams have a row in."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mixture_experts_layer_token_amd as moe  # noqa: E402

from helpers import say  # noqa: E402
from test_gpu_norm import DTS, check_forward, check_gradient, make  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    moe.lib()


# rows of one round, of 256 compute units: 8192 up to H = 1024, 2048 up to 4096, 1024 up to 8192, 512 beyond
FORWARD = [(8203, 512), (16390, 77), (8195, 1000), (2051, 1500), (2051, 2880), (4100, 4095), (1029, 7168), (2050, 4100), (515, 16384),
           (1025, 8200), (521, 16385), (515, 40001)]
# 4096 up to 512, 2048 up to 1024, 1024 up to 2048, 512 up to 4096, 256 beyond; long rows: 512 for their sums, 113 and 51 for their columns
GRADIENT = [(4101, 512), (8203, 300), (2051, 1000), (4099, 777), (1027, 2000), (515, 2880), (1025, 4095), (259, 7168), (515, 8190), (259, 16384),
            (521, 16385), (130, 40001)]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,H", FORWARD)
def test_forward_walks(rows, H, dt, rms):
    say("norm walk", rows, H, dt, "rms", rms)
    x, _, _, w, b = make(rows, H, DTS[dt], DTS[dt], bias=not rms, seed=40)
    y, stats = torch.empty((rows, H), device="cuda", dtype=DTS[dt]), torch.empty((rows, 2), device="cuda")
    check_forward(x, w, b, 1e-5, rms, y, stats)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,H", GRADIENT)
def test_gradient_walks(rows, H, dt, rms):
    say("norm gradient walk", rows, H, dt, "rms", rms)
    x, dy, add, w, _ = make(rows, H, DTS[dt], torch.float32, seed=41)
    check_gradient(x, dy, add, w, torch.float32, rms)
