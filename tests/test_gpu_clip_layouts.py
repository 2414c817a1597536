"""Clipping into results whose strides differ from their gradients' only where there is one element."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import mixture_experts_layer_token_amd as moe  # noqa: E402

from grouped_ref import f64  # noqa: E402


def test_dimensions_of_one_element_have_any_stride():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.randn((1, 50, 40), device="cuda").transpose(1, 2)
    o = torch.full((50, 40), 12345.0, device="cuda").t()[None]
    assert g.stride() != o.stride()
    norm = torch.empty(1, device="cuda")
    moe.moe_clip_grad_norm([g], 1.0, norm, outs=[o])
    torch.cuda.synchronize()
    total = float(f64(g).norm())
    # the factor's rounding, the product's, and the result's
    assert ((f64(o) - f64(g) / total).abs() <= 3.01 * 2.0 ** -24 * f64(g).abs() / total).all()
    with pytest.raises(ValueError):  # another order in memory
        moe.moe_clip_grad_norm([g], 1.0, norm, outs=[torch.empty((1, 40, 50), device="cuda")])
