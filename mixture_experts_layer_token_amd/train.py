"""A routed-expert MoE layer that trains, and what a training step needs around it: plain weights, forward and backward on the
library's kernels.

The layer is the one of ``layer.MoeLayer`` (router, stable grouping, SwiGLU experts, weighted combine) over plain
parameters instead of packed experts:

  w_router   [E, H]      router (bias [E] float32, optional)
  w_gate_up  [E, 2I, H]  gate rows, then up rows of every expert
  w_down     [E, H, I]

Forward: moe_route_permute, moe_grouped_gemm (gate/up, rows gathered), moe_swiglu, moe_grouped_gemm (down, fp32
results), moe_combine.  Backward: moe_combine_grad (down to the router's logits), moe_grouped_gemm_dx / _dw,
moe_swiglu_grad (which also recomputes the gated rows, so they are not kept), moe_combine with gate weights 1 for the
sum over a token's rows.  The choice of experts is not differentiated; the gate weights are the softmax of the chosen
logits.  The router's own products run in fp32.  With ``fused=True`` the gate is part of the products on both sides of it:
moe_grouped_swiglu forward, moe_grouped_swiglu_dx backward; h then comes from unrounded sums, so results differ from the
unfused layer's by its roundings of gu and dh.

Around it: ``GatedFFN``, the same gated block without experts (a shared expert); ``Norm``, layer or RMS norm;
``MoeTrainBlock``, x + layer(norm(x)) (+ shared(norm(x))); ``clip_grad_norm`` over all gradients of a step.

Capture into a graph like any autograd step: warm up on a side stream first, and drop every output of the warm-up
(its graph holds the parameters' gradient accumulators on that stream) before capturing.
"""
from __future__ import annotations

import torch

from . import api


class _MoeLayerFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_router, bias, w_gate_up, w_down, k, fused):
        T, H = x.shape
        E, I = w_gate_up.shape[0], w_down.shape[2]
        dev, n = x.device, T * k
        x, w_router = x.contiguous(), w_router.contiguous()
        i32 = dict(dtype=torch.int32, device=dev)
        ids, gates = torch.empty((T, k), **i32), torch.empty((T, k), dtype=torch.float32, device=dev)
        counts, offsets = torch.empty(E, **i32), torch.empty(E + 1, **i32)
        perm, inv = torch.empty(n, **i32), torch.empty(n, **i32)
        api.moe_route_permute(x, w_router, bias, k, ids, gates, counts, offsets, perm, inv)
        gu = torch.empty((n, 2 * I), dtype=x.dtype, device=dev)
        h = torch.empty((n, I), dtype=x.dtype, device=dev)
        if fused:
            api.moe_grouped_swiglu(x, w_gate_up, offsets, h, gu=gu, perm_src=perm, k=k)
        else:
            api.moe_grouped_gemm(x, w_gate_up, offsets, gu, perm_src=perm, k=k)
            api.moe_swiglu(gu, h)
        y = torch.empty((n, H), dtype=torch.float32, device=dev)
        api.moe_grouped_gemm(h, w_down, offsets, y)
        out = torch.empty_like(x)
        api.moe_combine(y, gates, inv, k, None, out)
        ctx.save_for_backward(x, w_router, w_gate_up, w_down, ids, gates, offsets, perm, inv, gu, y)
        ctx.k, ctx.has_bias, ctx.fused = k, bias is not None, fused
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        x, w_router, w_gate_up, w_down, ids, gates, offsets, perm, inv, gu, y = ctx.saved_tensors
        need_x, need_r, need_b, need_gu, need_dn, _, _ = ctx.needs_input_grad
        k, (T, H), (E, I) = ctx.k, x.shape, (w_gate_up.shape[0], w_down.shape[2])
        dev, n, f32 = x.device, T * k, torch.float32
        dout = dout.contiguous()
        dy = torch.empty((n, H), dtype=x.dtype, device=dev)
        dgates, dlogits = torch.empty((T, k), dtype=f32, device=dev), torch.empty((T, E), dtype=f32, device=dev)
        api.moe_combine_grad(dout, y, gates, inv, k, dy, dgates, topk_ids=ids, dlogits=dlogits)
        dx = dw_router = dbias = dw_gate_up = dw_down = None
        if need_x or need_gu or need_dn:
            dgu, h = torch.empty_like(gu), torch.empty((n, I), dtype=x.dtype, device=dev)
            if ctx.fused:
                api.moe_grouped_swiglu_dx(dy, w_down, gu, offsets, dgu, h=h if need_dn else None)
            else:
                dh = torch.empty_like(h)
                api.moe_grouped_gemm_dx(dy, w_down, offsets, dh)
                api.moe_swiglu_grad(gu, dh, dgu, h=h)
            if need_dn:
                dw_down = torch.empty_like(w_down, memory_format=torch.contiguous_format)
                api.moe_grouped_gemm_dw(dy, h, offsets, dw_down)
            if need_gu:
                dw_gate_up = torch.empty_like(w_gate_up, memory_format=torch.contiguous_format)
                api.moe_grouped_gemm_dw(dgu, x, offsets, dw_gate_up, perm_src=perm, k=k)
        # the router: one group of all tokens, in fp32
        if need_x or need_r or need_b:
            all_rows = _one_group(T, dev)
        if need_r:
            dwr = torch.empty((1, E, H), dtype=f32, device=dev)
            api.moe_grouped_gemm_dw(dlogits, x.to(f32), all_rows, dwr)
            dw_router = dwr[0].to(w_router.dtype)
        if need_b and ctx.has_bias:
            # the sum over the tokens as a product with ones: fixed order, and no memset node when captured
            column = torch.empty((1, E, 1), dtype=f32, device=dev)
            api.moe_grouped_gemm_dw(dlogits, torch.ones((T, 1), dtype=f32, device=dev), all_rows, column)
            dbias = column.view(E)
        if need_x:
            rows = torch.empty((n, H), dtype=f32, device=dev)
            api.moe_grouped_gemm_dx(dgu, w_gate_up, offsets, rows)
            by_router = torch.empty((T, H), dtype=f32, device=dev)
            api.moe_grouped_gemm_dx(dlogits, w_router.to(f32)[None], all_rows, by_router)
            dx = torch.empty_like(x)
            api.moe_combine(rows, torch.ones((T, k), dtype=f32, device=dev), inv, k, by_router, dx)
        return dx, dw_router, dbias, dw_gate_up, dw_down, None, None


def _one_group(rows, device):
    """offsets of one group that holds all rows, written on the device (nothing is copied from the host)."""
    return torch.arange(2, dtype=torch.int32, device=device) * rows


class MoeTrainLayer(torch.nn.Module):
    """Routed-expert SwiGLU layer with plain parameters; x and all weights in one type, bfloat16 or float32 (the
    router's bias is float32 with either).  `fused`: the gate in the same kernels as the products around it."""

    def __init__(self, H, I, E, k, dtype=torch.bfloat16, bias=False, device="cuda", sigma=0.02, fused=False):
        super().__init__()
        if not 1 <= k <= min(E, 16):
            raise ValueError("k=%d out of 1..min(E, 16)" % k)
        if H % (32 if dtype == torch.bfloat16 else 4):
            raise ValueError("H=%d must be a multiple of 32 (bfloat16: the router) or 4 (float32: the combine)" % H)
        self.k, self.fused = k, fused

        def par(*shape):
            return torch.nn.Parameter((torch.randn(shape, device=device) * sigma).to(dtype))

        self.w_router = par(E, H)
        self.bias = torch.nn.Parameter(torch.zeros(E, device=device)) if bias else None
        self.w_gate_up = par(E, 2 * I, H)
        self.w_down = par(E, H, I)

    def forward(self, x):
        if x.dim() != 2 or x.shape[1] != self.w_router.shape[1]:
            raise ValueError("x %s: [T, %d] expected" % (tuple(x.shape), self.w_router.shape[1]))
        if any(p.device != x.device for p in self.parameters()):
            raise ValueError("x is on %s, a parameter is not" % x.device)
        if any(p.dtype != x.dtype for p in (self.w_router, self.w_gate_up, self.w_down)):
            raise TypeError("x and the weights must have one type (x: %s)" % x.dtype)
        if self.bias is not None and self.bias.dtype != torch.float32:
            raise TypeError("the router's bias stays float32, got %s" % self.bias.dtype)
        with torch.cuda.device(x.device):
            return _MoeLayerFunction.apply(x, self.w_router, self.bias, self.w_gate_up, self.w_down, self.k,
                                           self.fused)


class _GatedFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate_up, w_down, keep):
        (T, H), I, dev = x.shape, w_down.shape[1], x.device
        x, rows = x.contiguous(), _one_group(T, dev)
        h = torch.empty((T, I), dtype=x.dtype, device=dev)
        gu = torch.empty((T, 2 * I), dtype=x.dtype, device=dev) if keep else None
        api.moe_grouped_swiglu(x, w_gate_up[None], rows, h, gu=gu)
        y = torch.empty((T, H), dtype=x.dtype, device=dev)
        api.moe_grouped_gemm(h, w_down[None], rows, y)
        if keep:
            ctx.save_for_backward(x, w_gate_up, w_down, gu)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w_gate_up, w_down, gu = ctx.saved_tensors
        need_x, need_gu, need_dn, _ = ctx.needs_input_grad
        (T, I2), dev = gu.shape, x.device
        dy, rows = dy.contiguous(), _one_group(T, dev)
        h = torch.empty((T, I2 // 2), dtype=x.dtype, device=dev) if need_dn else None
        dgu = torch.empty_like(gu)
        api.moe_grouped_swiglu_dx(dy, w_down[None], gu, rows, dgu, h=h)
        dx = dw_gate_up = dw_down = None
        if need_dn:
            dw_down = torch.empty_like(w_down, memory_format=torch.contiguous_format)
            api.moe_grouped_gemm_dw(dy, h, rows, dw_down[None])
        if need_gu:
            dw_gate_up = torch.empty_like(w_gate_up, memory_format=torch.contiguous_format)
            api.moe_grouped_gemm_dw(dgu, x, rows, dw_gate_up[None])
        if need_x:
            dx = torch.empty_like(x)
            api.moe_grouped_gemm_dx(dgu, w_gate_up[None], rows, dx)
        return dx, dw_gate_up, dw_down, None


def _keeps(*tensors):
    """Whether a backward pass can follow."""
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def _check_rows(x, H, *params):
    if x.dim() != 2 or x.shape[1] != H:
        raise ValueError("x %s: [T, %d] expected" % (tuple(x.shape), H))
    if any(p is not None and p.device != x.device for p in params):
        raise ValueError("x is on %s, a parameter is not" % x.device)


class GatedFFN(torch.nn.Module):
    """The gated feed-forward block of every token, y = w_down (SiLU(w_gate x) * (w_up x)): w_gate_up [2I, H] (gate rows, then up
    rows), w_down [H, I]; x and weights in one type, bfloat16 or float32."""

    def __init__(self, H, I, dtype=torch.bfloat16, device="cuda", sigma=0.02):
        super().__init__()
        self.w_gate_up = torch.nn.Parameter((torch.randn((2 * I, H), device=device) * sigma).to(dtype))
        self.w_down = torch.nn.Parameter((torch.randn((H, I), device=device) * sigma).to(dtype))

    def forward(self, x):
        _check_rows(x, self.w_down.shape[0], self.w_gate_up, self.w_down)
        if x.dtype != self.w_gate_up.dtype or x.dtype != self.w_down.dtype:
            raise TypeError("x and the weights must have one type (x: %s)" % x.dtype)
        with torch.cuda.device(x.device):
            return _GatedFunction.apply(x, self.w_gate_up, self.w_down, _keeps(x, self.w_gate_up, self.w_down))


class _NormFunction(torch.autograd.Function):
    """(norm(x), x): x again for the residual, so that its gradient joins the norm's in one kernel."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps, rms, keep):
        x = x.contiguous()
        y = torch.empty_like(x)
        stats = torch.empty((x.shape[0], 2), dtype=torch.float32, device=x.device) if keep else None
        api.moe_norm(x, weight, bias, y, eps=eps, rms=rms, stats=stats)
        if keep:
            ctx.save_for_backward(x, weight, stats)
        ctx.has_bias, ctx.rms = bias is not None, rms
        ctx.set_materialize_grads(False)
        return y, x.view_as(x)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dres):
        if dy is None:
            return dres, None, None, None, None, None
        x, weight, stats = ctx.saved_tensors
        _, need_w, need_b, _, _, _ = ctx.needs_input_grad
        dx = torch.empty_like(x)
        dweight = torch.empty_like(weight) if need_w else None
        dbias = torch.empty_like(weight) if need_b and ctx.has_bias else None
        api.moe_norm_grad(dy.contiguous(), x, weight, stats, dx, dweight=dweight, dbias=dbias,
                          add=None if dres is None else dres.contiguous(), rms=ctx.rms)
        return dx, dweight, dbias, None, None, None


class Norm(torch.nn.Module):
    """Layer norm (or RMS norm) of rows x [T, H], bfloat16 or float32, with a weight and (layer norm) a bias of `dtype`."""

    def __init__(self, H, rms=False, bias=None, eps=1e-5, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.rms, self.eps = rms, eps
        self.weight = torch.nn.Parameter(torch.ones(H, dtype=dtype, device=device))
        has_bias = not rms if bias is None else bias
        self.bias = torch.nn.Parameter(torch.zeros(H, dtype=dtype, device=device)) if has_bias else None

    def with_residual(self, x):
        """(norm(x), x): use the second for the residual, and the two gradients of x are added in the norm's own kernel.  (A view of
        x: not to be changed in place.)"""
        _check_rows(x, self.weight.shape[0], self.weight, self.bias)
        with torch.cuda.device(x.device):
            return _NormFunction.apply(x, self.weight, self.bias, self.eps, self.rms, _keeps(x, self.weight, self.bias))

    def forward(self, x):
        return self.with_residual(x)[0]


class MoeTrainBlock(torch.nn.Module):
    """x + layer(norm(x)) (+ shared(norm(x)) with `shared_I`): the pre-norm block around a routed-expert layer."""

    def __init__(self, H, I, E, k, shared_I=None, rms=True, eps=1e-5, dtype=torch.bfloat16, bias=False, device="cuda",
                 sigma=0.02):
        super().__init__()
        self.norm = Norm(H, rms=rms, eps=eps, dtype=dtype, device=device)
        self.layer = MoeTrainLayer(H, I, E, k, dtype=dtype, bias=bias, device=device, sigma=sigma, fused=True)
        self.shared = None if shared_I is None else GatedFFN(H, shared_I, dtype=dtype, device=device, sigma=sigma)

    def forward(self, x):
        n, res = self.norm.with_residual(x)
        out = res + self.layer(n)
        return out if self.shared is None else out + self.shared(n)


def clip_grad_norm(parameters, max_norm):
    """Scale the gradients of `parameters` in place by min(1, max_norm / norm), where norm is the 2-norm over all of them, and
    return norm (float32 [1], on the device: nothing waits for it).  `max_norm`: positive and finite.  A NaN or an infinity among
    the gradients scales nothing and makes norm one; a norm past fp32's range is an infinity there, and scales.  A gradient
    that several parameters share counts once."""
    parameters = [parameters] if isinstance(parameters, torch.Tensor) else list(parameters)
    grads = list({id(p.grad): p.grad for p in parameters if p.grad is not None}.values())
    if not grads:
        return torch.zeros(1, device=parameters[0].device if parameters else None)
    norm = torch.empty(1, dtype=torch.float32, device=grads[0].device)
    api.moe_clip_grad_norm(grads, max_norm, norm)
    return norm
