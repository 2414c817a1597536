"""A routed-expert MoE layer that trains: plain weights, forward and backward on the library's kernels.

The layer is the one of ``layer.MoeLayer`` (router, stable grouping, SwiGLU experts, weighted combine) over plain
parameters instead of packed experts:

  w_router   [E, H]      router (bias [E] float32, optional)
  w_gate_up  [E, 2I, H]  gate rows, then up rows of every expert
  w_down     [E, H, I]

Forward: moe_route_permute, moe_grouped_gemm (gate/up, rows gathered), moe_swiglu, moe_grouped_gemm (down, fp32
results), moe_combine.  Backward: moe_combine_grad (down to the router's logits), moe_grouped_gemm_dx / _dw,
moe_swiglu_grad (which also recomputes the gated rows, so they are not kept), moe_combine with gate weights 1 for the
sum over a token's rows.  The choice of experts is not differentiated; the gate weights are the softmax of the chosen
logits.  The router's own products run in fp32.

Capture into a graph like any autograd step: warm up on a side stream first, and drop every output of the warm-up
(its graph holds the parameters' gradient accumulators on that stream) before capturing.
"""
from __future__ import annotations

import torch

from . import api


class _MoeLayerFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_router, bias, w_gate_up, w_down, k):
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
        api.moe_grouped_gemm(x, w_gate_up, offsets, gu, perm_src=perm, k=k)
        h = torch.empty((n, I), dtype=x.dtype, device=dev)
        api.moe_swiglu(gu, h)
        y = torch.empty((n, H), dtype=torch.float32, device=dev)
        api.moe_grouped_gemm(h, w_down, offsets, y)
        out = torch.empty_like(x)
        api.moe_combine(y, gates, inv, k, None, out)
        ctx.save_for_backward(x, w_router, w_gate_up, w_down, ids, gates, offsets, perm, inv, gu, y)
        ctx.k, ctx.has_bias = k, bias is not None
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        x, w_router, w_gate_up, w_down, ids, gates, offsets, perm, inv, gu, y = ctx.saved_tensors
        need_x, need_r, need_b, need_gu, need_dn, _ = ctx.needs_input_grad
        k, (T, H), (E, I) = ctx.k, x.shape, (w_gate_up.shape[0], w_down.shape[2])
        dev, n, f32 = x.device, T * k, torch.float32
        dout = dout.contiguous()
        dy = torch.empty((n, H), dtype=x.dtype, device=dev)
        dgates, dlogits = torch.empty((T, k), dtype=f32, device=dev), torch.empty((T, E), dtype=f32, device=dev)
        api.moe_combine_grad(dout, y, gates, inv, k, dy, dgates, topk_ids=ids, dlogits=dlogits)
        dx = dw_router = dbias = dw_gate_up = dw_down = None
        if need_x or need_gu or need_dn:
            dh = torch.empty((n, I), dtype=x.dtype, device=dev)
            api.moe_grouped_gemm_dx(dy, w_down, offsets, dh)
            dgu, h = torch.empty_like(gu), torch.empty_like(dh)
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
        return dx, dw_router, dbias, dw_gate_up, dw_down, None


def _one_group(rows, device):
    """offsets of one group that holds all rows, written on the device (nothing is copied from the host)."""
    return torch.arange(2, dtype=torch.int32, device=device) * rows


class MoeTrainLayer(torch.nn.Module):
    """Routed-expert SwiGLU layer with plain parameters; x and all weights in one type, bfloat16 or float32 (the
    router's bias is float32 with either)."""

    def __init__(self, H, I, E, k, dtype=torch.bfloat16, bias=False, device="cuda", sigma=0.02):
        super().__init__()
        if not 1 <= k <= min(E, 16):
            raise ValueError("k=%d out of 1..min(E, 16)" % k)
        if H % (32 if dtype == torch.bfloat16 else 4):
            raise ValueError("H=%d must be a multiple of 32 (bfloat16: the router) or 4 (float32: the combine)" % H)
        self.k = k

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
            return _MoeLayerFunction.apply(x, self.w_router, self.bias, self.w_gate_up, self.w_down, self.k)
