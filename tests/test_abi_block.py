"""Refusals of the gated block, the norm of rows and the norm and clipping of gradients: every bad argument is turned away
before a pointer is touched (no GPU needed)."""
import ctypes

import pytest

import mixture_experts_layer_token_amd as moe
from mixture_experts_layer_token_amd._lib import MoeGrouped, MoeNormDesc, MoeTensor

L = moe.lib()
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -6
F32, BF16 = 0, 1
P = ctypes.c_void_p(4096)  # never dereferenced: every call here is refused, or has nothing to do
ODD = ctypes.c_void_p(4097)


# ------------------------------------------------------------------ gated block
def desc(**kw):
    g = MoeGrouped()
    g.rows, g.E, g.N, g.K, g.k, g.x_rows = 16, 4, 64, 32, 2, 8
    g.offsets = 4096
    for k, v in kw.items():
        setattr(g, k, v)
    return g


def block(g, dt=BF16, x=P, w=P, h=P, gu=None):
    return L.moe_grouped_swiglu(ctypes.byref(g) if g else None, dt, x, w, h, gu, None)


def block_dx(g, dt=BF16, dy=P, w=P, gu=P, dgu=P, h=None):
    return L.moe_grouped_swiglu_dx(ctypes.byref(g) if g else None, dt, dy, w, gu, dgu, h, None)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(rows=(1 << 24) + 1), dict(E=0), dict(E=1025), dict(N=0), dict(K=0),
                                 dict(N=(1 << 20) + 1), dict(K=(1 << 20) + 1), dict(offsets=None), dict(offsets=4098), dict(ldy=63),
                                 dict(ldw=31), dict(w_stride=64 * 32 - 1), dict(w_stride=-1)])
def test_block_descriptors(bad):
    assert block(desc(**bad)) == INVALID and block_dx(desc(**bad)) == INVALID


def test_block_strides():
    # w has 2N rows in the block: an expert stride that fits N rows is too short
    for stride in (64 * 32, 2 * 64 * 32 - 1):
        assert block(desc(w_stride=stride)) == INVALID
    assert block(desc(ldx=31)) == INVALID
    assert block(desc(perm_src=4096, k=17)) == INVALID and block(desc(perm_src=4097)) == INVALID
    # the gradient has no x: its stride and gather are ignored
    assert block_dx(desc(rows=0, ldx=31, perm_src=4097)) == OK


def test_block_pointers_and_types():
    assert block(None) == INVALID and block_dx(None) == INVALID
    for name in ("x", "w", "h"):
        assert block(desc(), **{name: None}) == INVALID and block(desc(), **{name: ODD}) == INVALID
    assert block(desc(), gu=ODD) == INVALID
    for name in ("dy", "w", "gu", "dgu"):
        assert block_dx(desc(), **{name: None}) == INVALID and block_dx(desc(), **{name: ODD}) == INVALID
    assert block_dx(desc(), h=ODD) == INVALID
    assert b"moe_grouped_swiglu_dx" in L.moe_last_error()
    assert block(desc(), dt=2) == INVALID and block_dx(desc(), dt=-1) == INVALID
    assert block(desc(rows=0), x=None, w=None, h=None) == OK and block_dx(desc(rows=0), dy=None, w=None, gu=None, dgu=None) == OK


# ------------------------------------------------------------------ norm of rows
def norm(x=P, w=P, b=P, y=P, st=None, null=False, **kw):
    d = MoeNormDesc(8, 64, 0, BF16, BF16, 1e-5, 0, 0)
    for k, v in kw.items():
        setattr(d, k, v)
    return L.moe_norm(None if null else ctypes.byref(d), x, w, b, y, st, None)


def norm_grad(dy=P, x=P, w=P, st=P, add=None, dx=P, dw=P, db=P, ws=P, n=1 << 20, null=False, **kw):
    d = MoeNormDesc(8, 64, 0, BF16, BF16, 0.0, 0, 0)
    for k, v in kw.items():
        setattr(d, k, v)
    return L.moe_norm_grad(None if null else ctypes.byref(d), dy, x, w, st, add, dx, dw, db, ws, n, None)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(rows=(1 << 24) + 1), dict(H=0), dict(H=(1 << 20) + 1), dict(rms=2), dict(rms=-1),
                                 dict(dt=2), dict(pdt=-1), dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf")),
                                 dict(ldx=63), dict(ldy=63), dict(ldx=-64), dict(ldy=(1 << 40) + 1), dict(null=True)])
def test_norm_descriptors(bad):
    assert norm(**bad) == INVALID and norm_grad(**bad) == INVALID


def test_norm_pointers():
    for name in ("x", "y"):
        assert norm(**{name: None}) == INVALID
    for name in ("x", "y", "w", "b", "st"):
        assert norm(**{name: ODD}) == INVALID
    for name in ("dy", "x", "st", "dx"):
        assert norm_grad(**{name: None}) == INVALID
    for name in ("dy", "x", "w", "st", "add", "dx", "dw", "db"):
        assert norm_grad(**{name: ODD}) == INVALID
    assert norm(rows=0, x=None, y=None) == OK


def test_norm_workspace():
    for rows, H in ((1, 1), (8, 64), (5000, 7168), (100, 20000)):
        need = moe.moe_norm_workspace(rows, H)
        assert need >= 2 * H * 4 and need % 256 == 0
        for ws, n in ((None, need), (P, need - 1), (ctypes.c_void_p(4096 + 128), need)):
            assert norm_grad(ws=ws, n=n, rows=rows, H=H) == WORKSPACE
    for rows, H in ((0, 64), (-1, 64), (8, 0), ((1 << 24) + 1, 64), (8, (1 << 20) + 1)):
        assert moe.moe_norm_workspace(rows, H) == 0


# ------------------------------------------------------------------ norm and clipping of gradients
def entries(*spans):
    return (MoeTensor * max(len(spans), 1))(*[MoeTensor(*s) for s in spans])


def clip(t, n=None, max_norm=1.0, norm_out=P, ws=P, nws=1 << 20):
    return L.moe_clip_grad_norm(t, len(t) if n is None else n, max_norm, norm_out, ws, nws, None)


def only_norm(t, n=None, norm_out=P, ws=P, nws=1 << 20):
    return L.moe_grad_norm(t, len(t) if n is None else n, norm_out, ws, nws, None)


A, B, C = 1 << 20, 1 << 21, 1 << 22  # addresses


@pytest.mark.parametrize("bad", [(A, A, -1, F32), (A, A, 4, 2), (None, None, 4, F32), (A + 2, A + 2, 4, F32),
                                 (A + 1, None, 4, BF16), (A, B + 1, 4, BF16)])
def test_clip_entries(bad):
    good = (C, C, 16, F32)
    for t in (entries(bad), entries(good, bad)):
        assert clip(t) == INVALID and only_norm(t) == INVALID
        assert b"tensor %d" % (len(t) - 1) in L.moe_last_error()


@pytest.mark.parametrize("spans", [
    [(A, A, 100, F32), (A, A, 100, F32)],                      # the same gradient twice, in place
    [(A, A, 100, F32), (A + 396, A + 396, 100, F32)],          # the last element of one is the first of the next
    [(A, A, 100, F32), (B, B, 10, F32), (A + 8, None, 1, BF16)],
    [(A, A + 4, 100, F32)],                                    # its own result, shifted
    [(A, B, 100, F32), (C, B + 200, 100, F32)],                # two results
    [(A, B, 100, F32), (B, C, 100, F32)],                      # a result over another gradient
    [(A, B, 1000, F32), (B + 100, None, 5, F32), (C, C, 5, F32)],
    [(A, None, 1000, F32), (C, C, 5, F32), (B, A + 3996, 1, F32)],
])
def test_clip_overlaps(spans):
    assert clip(entries(*spans)) == INVALID
    assert b"overlap" in L.moe_last_error()
    assert clip(entries(*spans[::-1])) == INVALID


def test_clip_arguments():
    t = entries((A, A, 100, F32))
    for m in (0.0, -1.0, float("nan"), float("inf")):
        assert clip(t, max_norm=m) == INVALID
    for bad in (None, ODD):
        assert clip(t, norm_out=bad) == INVALID and only_norm(t, norm_out=bad) == INVALID
    for n in (-1, (1 << 16) + 1):
        assert clip(t, n=n) == INVALID and only_norm(t, n=n) == INVALID
    assert L.moe_clip_grad_norm(None, 1, 1.0, P, P, 1 << 20, None) == INVALID
    need = L.moe_grad_norm_workspace(1)
    assert need > 0
    for ws, n in ((None, need), (P, need - 1), (ctypes.c_void_p(4096 + 8), need)):
        assert clip(t, ws=ws, nws=n) == WORKSPACE and only_norm(t, ws=ws, nws=n) == WORKSPACE


def test_workspace_grows_with_the_list():
    sizes = [L.moe_grad_norm_workspace(n) for n in (0, 1, 400, 1 << 16)]
    assert sizes == sorted(sizes) and sizes[0] > 0 and sizes[3] > sizes[1] and all(n % 256 == 0 for n in sizes)
    assert L.moe_grad_norm_workspace(-1) == 0 and L.moe_grad_norm_workspace((1 << 16) + 1) == 0


def test_too_many_elements():
    t = entries((A, None, 1 << 39, F32), (A, None, 1 << 39, F32), (A, None, 1, F32))
    assert clip(t) == INVALID and only_norm(t) == INVALID
