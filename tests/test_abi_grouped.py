"""Refusals of the grouped products over plain weights, the 8-bit operators, the SwiGLU gate and the combine's
gradient: every bad argument is turned away before a pointer is touched (no GPU needed)."""
import ctypes

import pytest

import mixture_experts_layer_token_amd as moe
from mixture_experts_layer_token_amd._lib import MoeGrouped

L = moe.lib()
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -6
F32, BF16 = 0, 1
P = ctypes.c_void_p(4096)  # never dereferenced: every call here is refused, or has nothing to do
ODD = ctypes.c_void_p(4097)


def desc(**kw):
    g = MoeGrouped()
    g.rows, g.E, g.N, g.K, g.k, g.x_rows = 16, 4, 64, 32, 2, 8
    g.offsets = 4096
    for k, v in kw.items():
        setattr(g, k, v)
    return g


def calls(g, dt=BF16, odt=BF16, a=P, b=P, c=P, ws=None, n=0):
    r = ctypes.byref(g)
    return [L.moe_grouped_gemm(r, dt, a, b, c, odt, ws, n, None),
            L.moe_grouped_gemm_dx(r, dt, a, b, c, odt, ws, n, None),
            L.moe_grouped_gemm_dw(r, dt, a, b, c, odt, ws, n, None)]


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(rows=(1 << 24) + 1), dict(E=0), dict(E=1025), dict(N=0),
                                 dict(K=0), dict(N=(1 << 20) + 1), dict(K=(1 << 20) + 1), dict(offsets=None),
                                 dict(offsets=4098), dict(ldx=31), dict(ldy=63), dict(ldw=31), dict(ldx=-40),
                                 dict(w_stride=64 * 32 - 1), dict(ldw=40, w_stride=64 * 32), dict(w_stride=-1)])
def test_bad_descriptors(bad):
    g = desc(**bad)
    assert calls(g) == [INVALID] * 3
    assert L.moe_grouped_gemm_i8(ctypes.byref(g), P, P, P, P, P, F32, None) == INVALID


def test_bad_gather():
    for bad in (dict(k=0), dict(k=17), dict(x_rows=-1), dict(x_rows=(1 << 24) + 1)):
        g = desc(perm_src=4096, **bad)
        assert [calls(g)[0], calls(g)[2]] == [INVALID] * 2
    assert calls(desc(perm_src=4097))[0] == INVALID


def test_null_and_misaligned_pointers():
    g = desc()
    assert L.moe_grouped_gemm(None, BF16, P, P, P, BF16, None, 0, None) == INVALID
    assert L.moe_grouped_gemm_dx(None, BF16, P, P, P, BF16, None, 0, None) == INVALID
    assert L.moe_grouped_gemm_dw(None, BF16, P, P, P, BF16, None, 0, None) == INVALID
    for which in ("a", "b", "c"):
        assert calls(g, **{which: None}) == [INVALID] * 3
        assert calls(g, **{which: ODD}) == [INVALID] * 3
        assert b"moe_grouped_gemm_dw" in L.moe_last_error()
    assert calls(g, dt=2) == [INVALID] * 3 and calls(g, odt=-1) == [INVALID] * 3
    r = ctypes.byref(g)
    for i in range(5):
        args = [P] * 5
        args[i] = None
        assert L.moe_grouped_gemm_i8(r, *args, F32, None) == INVALID
    assert L.moe_grouped_gemm_i8(r, P, ODD, P, P, P, F32, None) == INVALID
    assert L.moe_grouped_gemm_i8(r, P, P, P, P, P, 7, None) == INVALID


def test_int8_sums_that_could_overflow():
    g = desc(K=131072)
    assert L.moe_grouped_gemm_i8(ctypes.byref(g), P, P, P, P, P, F32, None) == UNSUPPORTED


def test_no_rows_is_nothing_to_do():
    g = desc(rows=0)
    assert calls(g, a=None, b=P, c=None)[0] == OK  # (the weights' gradient of no rows still writes zeros)
    assert calls(g, a=None, b=None, c=None)[:2] == [OK, OK]
    assert calls(g, a=None, b=None, c=None)[2] == INVALID
    assert L.moe_grouped_gemm_i8(ctypes.byref(g), None, None, None, None, None, F32, None) == OK


def test_workspace():
    assert L.moe_grouped_workspace(5, 16, 64, 32, 4) == 0
    assert L.moe_grouped_workspace(BF16, 16, 64, 32, 0) == 0
    for dt in (F32, BF16):
        for rows, N, K, E in ((4096, 128, 2880, 1), (8192, 64, 64, 2), (16, 64, 32, 4), (8192, 4096, 14336, 8)):
            need = L.moe_grouped_workspace(dt, rows, N, K, E)
            if need:
                g = desc(rows=rows, N=N, K=K, E=E)
                assert calls(g, dt=dt, ws=None, n=need) == [WORKSPACE] * 3
                assert calls(g, dt=dt, ws=P, n=need - 1) == [WORKSPACE] * 3
                assert calls(g, dt=dt, ws=ctypes.c_void_p(4096 + 16), n=need) == [WORKSPACE] * 3


def test_too_many_tiles():
    g = desc(rows=1, N=1 << 20, K=1 << 20, E=1024)
    assert calls(g, ws=P, n=1 << 62)[2] == UNSUPPORTED
    assert b"tiles" in L.moe_last_error()


def test_quant_and_gate_refusals():
    q = lambda x=P, dt=BF16, rows=4, K=8, act=0, n=None, qq=P, s=P: L.moe_quant_rows(x, dt, rows, K, act, n, qq, s, None)
    assert q(dt=3) == INVALID and q(act=2) == INVALID and q(rows=-1) == INVALID and q(K=0) == INVALID
    assert q(K=(1 << 20) + 1) == INVALID and q(x=None) == INVALID and q(qq=None) == INVALID and q(s=None) == INVALID
    assert q(x=ODD) == INVALID and q(s=ODD) == INVALID and q(n=ODD) == INVALID
    assert q(rows=0, x=None, qq=None, s=None) == OK
    f = lambda gu=P, dt=BF16, rows=4, I=8, n=None, h=P: L.moe_swiglu(gu, dt, rows, I, n, h, None)
    g = lambda gu=P, dh=P, dt=BF16, rows=4, I=8, n=None, d=P, h=None: L.moe_swiglu_grad(gu, dh, dt, rows, I, n, d, h, None)
    for c in (f, g):
        assert c(gu=None) == INVALID and c(dt=9) == INVALID and c(rows=-2) == INVALID and c(I=0) == INVALID
        assert c(gu=ODD) == INVALID and c(n=ODD) == INVALID and c(h=ODD) == INVALID and c(rows=0, gu=None) == OK
    assert f(h=None) == INVALID and g(dh=None) == INVALID and g(d=None) == INVALID and g(d=ODD) == INVALID


def test_combine_grad_refusals():
    def c(dout=P, odt=BF16, y=P, w=P, inv=P, T=4, k=2, H=64, dy=P, ydt=BF16, dw=P, ids=P, E=8, dl=P):
        return L.moe_combine_grad(dout, odt, y, w, inv, T, k, H, dy, ydt, dw, ids, E, dl, None)

    for name in ("dout", "y", "w", "inv", "dy", "dw", "ids"):
        assert c(**{name: None}) == INVALID, name
        assert c(**{name: ODD}) == INVALID, name
    assert c(dl=ODD) == INVALID
    assert c(odt=2) == INVALID and c(ydt=2) == INVALID and c(T=-1) == INVALID and c(k=0) == INVALID and c(k=17) == INVALID
    assert c(H=0) == INVALID and c(E=0) == INVALID and c(E=1025) == INVALID and c(T=1 << 22, k=16) == INVALID
    assert c(T=0, dout=None, y=None) == OK


def test_python_wrappers_refuse_mismatched_shapes():
    torch = pytest.importorskip("torch")
    x, w, y = torch.zeros(4, 8), torch.zeros(2, 6, 8), torch.zeros(4, 6)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, w, off, torch.zeros(4, 5))
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(torch.zeros(4, 7), w, off, y)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, w, off[:2], y)
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(torch.zeros(3, 8), w, off, y)  # rows differ and no perm_src
    with pytest.raises(ValueError):
        moe.moe_grouped_gemm(x, w, off, y, perm_src=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        moe.moe_quant_rows(x, torch.zeros(4, 8, dtype=torch.int8), torch.zeros(3))
    with pytest.raises(ValueError):
        moe.moe_swiglu(x, torch.zeros(4, 5))
