"""The MoE half of a transformer block on the libmpm kernels: residual
addition and RMSNorm, router, expert layer, and their gradients.

    h = x + residual;  y = rmsnorm(h) * w                    add_rmsnorm
    logits = y Wr^T                                          BF16 GEMM
    ids, prob, counts, loss = top-k of the logits            moe_route
    out = sum_j prob_j * expert_{ids_j}(y)                   MXFP8MoE

Training (forward, backward) quantises y inside the expert layer, which needs
the column-wise copies too; rollout (infer) takes the row-wise MXFP8 copy the
norm writes and gathers its bytes into the expert order, so that both run on
the same quantised operands.  Gradients:

    dprob = <dout, expert outputs>, dlogits, dWr = dlogits^T y
    dy = (expert layer's dX) + dlogits Wr;  dx, dw = norm's backward

Every step runs in the library's kernels on the current stream; this module
owns the buffers and sequences the calls.  No host synchronisation inside a
step.
"""
from __future__ import annotations

import torch

from . import _lib as L
from . import ops
from .moe import MXFP8MoE


class MoEBlock:
    """Buffers and launch sequence for a fixed (T, H, I, E, k).  T is a
    multiple of 128, H and I of 256 (the layer's GEMMs run on CTA pairs); E up to
    1024 (the router weight is kept padded to a multiple of 256 rows).

    norm_weight [H] bf16 or fp32, router_weight [E, H] bf16, w1 [E, 2I, H] and
    w2 [E, H, I] bf16.  score, normalize, scale, bias: as ops.moe_route."""

    def __init__(self, T, H, I, E, k, norm_weight, router_weight, w1, w2, eps=1e-6,
                 score="softmax", normalize=True, scale=1.0, bias=None):
        if T % 128 != 0 or H % 256 != 0 or I % 256 != 0:
            raise ValueError(f"T = {T} must be a multiple of 128, H = {H} and I = {I} of 256")
        if tuple(router_weight.shape) != (E, H) or router_weight.dtype != torch.bfloat16:
            raise ValueError(f"router_weight: expected bf16 {(E, H)}")
        self.T, self.H, self.I, self.E, self.k, self.eps = T, H, I, E, k, eps
        self.norm_weight, self.bias = norm_weight, bias
        self.kw = dict(score=score, normalize=normalize, scale=scale)
        dev = router_weight.device
        self.Ep = ops.pad_to(E, 256)
        self.wr = torch.zeros(self.Ep, H, dtype=torch.bfloat16, device=dev)
        self.experts = MXFP8MoE(T, H, I, E, k, device=dev)
        self.set_weights(router_weight, w1, w2)
        bf, f32 = torch.bfloat16, torch.float32
        e = lambda *s, dtype=bf: torch.empty(*s, dtype=dtype, device=dev)
        self.norm = {"y": e(T, H), "h": e(T, H), "rstd": e(T, dtype=f32)}
        self._h = None                               # what the last norm was taken of
        self._kept = False                           # whether the buffers are those of a whole forward
        self.logits_p = e(T, self.Ep, dtype=f32)
        self.logits = self.logits_p[:, :E]
        self.route = None
        self.route_ws = e(max(1, ops.moe_route_workspace_bytes(T, E)), dtype=torch.uint8)
        # the gradient of the padded logits: columns at or past E stay zero
        self.dlogits_p = torch.zeros(T, self.Ep, dtype=bf, device=dev)
        self.dprob = e(T, k, dtype=f32)
        self.dy_router = e(T, H)
        self.dwr = e(self.Ep, H, dtype=f32)
        self.dx = e(T, H)
        self.dw_norm = e(H, dtype=f32)
        self.norm_ws = e(ops.add_rmsnorm_backward_workspace_bytes(T, H), dtype=torch.uint8)
        self.one_segment = torch.tensor([0, T], dtype=torch.int32, device=dev)

    def set_weights(self, router_weight=None, w1=None, w2=None):
        """New router and / or expert weights (quantised here; w1 and w2
        together)."""
        if (w1 is None) != (w2 is None):
            raise ValueError("w1 and w2 are set together")
        if router_weight is not None:
            if tuple(router_weight.shape) != (self.E, self.H):
                raise ValueError(f"router_weight: expected {(self.E, self.H)}, got {tuple(router_weight.shape)}")
            self.wr[:self.E] = router_weight
        if w1 is not None:
            self.experts.quantize_weights(w1, w2)

    def _logits(self):
        ops.moe_grouped_gemm(L.KIND_BF16, L.GROUP_M, L.EPI_F32, 1, self.T, self.Ep, self.H, None,
                             self.norm["y"], self.wr, None, 0, None, 0, self.logits_p, tile_m=256)

    def _norm_and_route(self, x, residual, token_mask, quantize):
        self._kept = False
        ops.add_rmsnorm(x, self.norm_weight, residual=residual, eps=self.eps, quantize=quantize,
                        out=self.norm)
        self._h = x if residual is None else self.norm["h"]
        self._logits()
        self.route = ops.moe_route(self.logits, self.k, bias=self.bias, token_mask=token_mask,
                                   out=self.route, ws=self.route_ws, **self.kw)
        self._mask = token_mask

    def forward(self, x, residual=None, token_mask=None):
        """(out [T, H], h [T, H]) bf16: the expert layer's output and the
        residual stream h = x + residual (x itself without one).  The balance
        loss and the expert counts are in self.route.  The backward reads x or
        h and the mask again: they stay as they are until then."""
        self._norm_and_route(x, residual, token_mask, quantize=False)
        r = self.route
        out = self.experts.forward(self.norm["y"], r["ids"], r["prob"])
        self._kept = True
        return out, self._h

    def infer(self, x, residual=None, token_mask=None):
        """forward without what the gradient needs, on the norm's own MXFP8
        copy: the same bytes.  It overwrites what an earlier forward kept, and
        a backward after it is refused."""
        self._norm_and_route(x, residual, token_mask, quantize=True)
        r, n = self.route, self.norm
        out = self.experts.forward_quantized(n["row_q"], n["row_s"], r["ids"], r["prob"])
        return out, self._h

    def backward(self, dout, dh=None, dloss=None):
        """Gradients after forward, from dout [T, H] bf16, dh (nullable, bf16:
        the gradient that reaches h along the residual stream) and dloss
        (nullable, fp32 [1]: the gradient of the balance loss).

        Returns a dict: dx [T, H] bf16 (of x and of the residual), dw_norm [H],
        dw_router [E, H], dw1, dw2 fp32."""
        if not self._kept:
            raise RuntimeError("backward needs a forward: infer keeps nothing for it and overwrites "
                               "what an earlier forward kept")
        T, H, E = self.T, self.H, self.E
        r, n = self.route, self.norm
        dy, dw1, dw2 = self.experts.backward(dout)
        self.experts.prob_grad(dout, r["prob"], out=self.dprob)
        # fp32 logits, bf16 gradient: the GEMM operands' type
        ops.moe_route_backward(self.logits, r["ids"], r["counts"], r["n_tokens"], dprob=self.dprob,
                               dloss=dloss, bias=self.bias, token_mask=self._mask,
                               out=self.dlogits_p[:, :E], **self.kw)
        bf = L.KIND_BF16
        ops.moe_grouped_gemm(bf, L.GROUP_M, L.EPI_BF16, 1, T, H, self.Ep, None, self.dlogits_p,
                             self.wr, None, 0, None, 0, self.dy_router, b_k_per_expert=0,
                             tile_m=256, b_mn_major=True)
        ops.moe_grouped_gemm(bf, L.GROUP_K, L.EPI_F32, 1, self.Ep, H, 0, self.one_segment,
                             self.dlogits_p, n["y"], None, 0, None, 0, self.dwr, tile_m=256,
                             a_mn_major=True, b_mn_major=True)
        ops.add_rmsnorm_backward(dy, self._h, n["rstd"], self.norm_weight, dy2=self.dy_router, dh=dh,
                                 out=(self.dx, self.dw_norm), ws=self.norm_ws)
        return {"dx": self.dx, "dw_norm": self.dw_norm, "dw_router": self.dwr[:E], "dw1": dw1,
                "dw2": dw2}
