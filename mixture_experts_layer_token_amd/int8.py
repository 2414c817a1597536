"""A routed-expert MoE layer with 8-bit integer experts (W8A8): int8 weights with a scale per output channel, and
activations quantized on the way with a scale per token.

The experts take half the bytes of bf16 ones.  Forward: moe_route_permute on the bf16 (or fp32) tokens, moe_quant_rows
(each token once, before it is gathered), moe_grouped_gemm_i8 (gate/up), moe_quant_rows with the SwiGLU gate (the
gated rows exist in 8 bits only), moe_grouped_gemm_i8 (down, fp32 results), moe_combine.  The gate/up results are kept in
bf16 whatever the tokens' type: that rounds each value by at most 2^-8 of it, the 8-bit rounding of the gated rows that
follows by 2^-8 of the row's largest.
"""
from __future__ import annotations

import torch

from . import api


def quantize_weights(w: torch.Tensor):
    """[E, N, K] bf16 / fp32 -> (int8 [E, N, K], scale [E, N]): one scale per output channel."""
    E, N, K = w.shape
    q = torch.empty((E, N, K), dtype=torch.int8, device=w.device)
    s = torch.empty((E, N), dtype=torch.float32, device=w.device)
    api.moe_quant_rows(w.contiguous().view(E * N, K), q.view(E * N, K), s.view(E * N))
    return q, s


class MoeInt8Layer:
    """`w_gate_up` [E, 2I, H] (gate rows, then up rows) and `w_down` [E, H, I] are quantized here; the router stays in
    its own type.  All buffers are allocated once for batches of up to max_T tokens, so one forward runs at a time.  A
    larger batch replaces them by ones of at least twice the size, or of its own size where memory does not suffice; the
    old ones go, unless a graph was captured with them (those that stay, together, are about as large as the last)."""

    def __init__(self, w_router, bias, w_gate_up, w_down, k, max_T=1):
        self.w_router, self.bias, self.k = w_router, bias, k
        self.E, self.H, self.I = w_gate_up.shape[0], w_gate_up.shape[2], w_down.shape[2]
        if tuple(w_gate_up.shape) != (self.E, 2 * self.I, self.H) or tuple(w_down.shape) != (self.E, self.H, self.I):
            raise ValueError("w_gate_up %s and w_down %s do not fit" % (tuple(w_gate_up.shape), tuple(w_down.shape)))
        if tuple(w_router.shape) != (self.E, self.H):
            raise ValueError("w_router %s: [%d, %d] expected" % (tuple(w_router.shape), self.E, self.H))
        if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (self.E,)):
            raise ValueError("bias %s %s: float32 [%d] expected" % (bias.dtype, tuple(bias.shape), self.E))
        self._outgrown = []  # buffers whose addresses captured graphs hold
        self._captured, self._stream = False, None  # of the present buffers: a graph holds them; the stream of the last forward
        self._sized_T, self._rws_bytes = 0, 256  # workspace that routes any batch of up to _sized_T tokens
        self.gate_up = quantize_weights(w_gate_up)
        self.down = quantize_weights(w_down)
        self._alloc(max_T)

    # the buffers, in the order _alloc makes them
    _BUFFERS = ("ids", "gates", "counts", "offsets", "perm", "inv", "q", "q_scale", "gu", "h", "h_scale", "y", "rws")

    def _alloc(self, T):
        """All buffers for T tokens, or, if one cannot be had, none of them: the layer stays as it was."""
        d, k, H, I, E = self.w_router.device, self.k, self.H, self.I, self.E
        n, sized_T, rws_bytes = max(T * k, 1), self._sized_T, self._rws_bytes
        xdt = "f32" if self.w_router.dtype == torch.float32 else "bf16"
        for t in range(sized_T + 1, T + 1):
            rws_bytes = max(rws_bytes, api.moe_route_permute_workspace(t, H, E, k, xdt))
        i8, i32, f32, u8 = torch.int8, torch.int32, torch.float32, torch.uint8
        sizes = (((T, k), i32), ((T, k), f32), ((E,), i32), ((E + 1,), i32), ((n,), i32), ((n,), i32), ((T, H), i8),
                 ((T,), f32), ((n, 2 * I), torch.bfloat16), ((n, I), i8), ((n,), f32), ((n, H), f32), ((rws_bytes,), u8))
        made = [torch.empty(shape, dtype=dtype, device=d) for shape, dtype in sizes]
        for name, t in zip(self._BUFFERS, made):
            setattr(self, name, t)
        self.max_T, self._sized_T, self._rws_bytes = T, max(sized_T, T), rws_bytes

    def _grow(self, T):
        old = [getattr(self, name) for name in self._BUFFERS]
        try:
            self._alloc(max(T, 2 * self.max_T))
        except torch.cuda.OutOfMemoryError:
            self._alloc(T)
        if self._captured:
            self._outgrown.append(old)
        elif self._stream is not None:
            for t in old:  # the last forward may still run, on another stream than the one they were allocated on
                t.record_stream(self._stream)
        self._captured, self._stream = False, None

    def forward(self, x, out=None):
        """One layer forward on the current stream (x [T, H] in the router's type)."""
        if x.dim() != 2 or x.shape[1] != self.H or x.dtype != self.w_router.dtype:
            raise ValueError("x %s %s: %s [T, %d] expected" % (x.dtype, tuple(x.shape), self.w_router.dtype, self.H))
        T = x.shape[0]
        if x.device != self.w_router.device:
            raise ValueError("x is on %s, the layer on %s" % (x.device, self.w_router.device))
        if out is None:
            out = torch.empty_like(x)
        elif out.shape != x.shape or out.device != x.device:
            raise ValueError("out %s on %s: that of x expected" % (tuple(out.shape), out.device))
        if T > self.max_T:
            self._grow(T)
        if T == 0:
            return out
        with torch.cuda.device(x.device):
            self._stream = torch.cuda.current_stream()
            self._captured = self._captured or torch.cuda.is_current_stream_capturing()
            self._run(x, out, T)
        return out

    def _run(self, x, out, T):
        k, n = self.k, T * self.k
        ids, gates, perm, inv = self.ids[:T], self.gates[:T], self.perm[:n], self.inv[:n]
        api.moe_route_permute(x, self.w_router, self.bias, k, ids, gates, self.counts, self.offsets, perm, inv,
                              ws=self.rws)
        api.moe_quant_rows(x, self.q[:T], self.q_scale[:T])
        api.moe_grouped_gemm_i8(self.q[:T], self.q_scale[:T], *self.gate_up, self.offsets, self.gu[:n], perm_src=perm, k=k)
        api.moe_quant_rows(self.gu[:n], self.h[:n], self.h_scale[:n], act="swiglu", n_rows=self.offsets[-1:])
        api.moe_grouped_gemm_i8(self.h[:n], self.h_scale[:n], *self.down, self.offsets, self.y[:n])
        api.moe_combine(self.y[:n], gates, inv, k, None, out)
