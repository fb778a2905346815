"""A MoE block of a residual network for fine-tuning: norms, router, experts.

``MoEBlock`` strings together what surrounds one ``MoELoRALayer`` in a
training step.  It takes the residual stream r and its normed copy n, which
the block before it made, and returns the next pair:

    logits = n W_r^T,  top-k of their softmax,  y = experts(n)
    r' = r + scale a(gate) norm(y; w_post),   n' = norm(r'; w_pre)

w_pre being the weight of the norm before the next block.  The backward takes
(dr', dn') to (dr, dn) and the gradients of the adapters, the norm weights, the
gate and the router's weight; the router's load-balancing and z losses enter
through ``aux_coef`` and ``z_coef``.  The products with W_r are plain matrix
products (torch.matmul); everything else runs in the CUDA library, all on the
current stream.  The block's gate is one value for each channel and its block side
bf16; gates for tokens or elements, weights kept around 0 and an fp32 block side are
arguments of ``lib.moe_block_norm_fwd`` / ``_bwd``.
"""
from __future__ import annotations

import torch

from . import _lib as L
from .ckpt import Packed8
from .layer import MoELoRALayer


class MoEBlock:
    """w: the layer's weights (W_gu, A_gu, B_gu, W_dn, A_dn, B_dn) and W_r [E,d]
    bf16; optionally w_post [d], w_pre [d] and gate [d] fp32 (left out: no such
    norm or gate).  residual: type of the residual stream (torch.bfloat16 or
    torch.float32); the block side is bf16.  checkpoint: a LayerScratch; the layer's
    pre-activations and output are then kept in 8 bits from forward to backward,
    and what lives within a call is shared by the blocks with the same scratch:
    the dr that backward returns holds until the next such call."""

    def __init__(self, T, d, f, E, k, r, alpha, w: dict, scale=1.0, gate_sigmoid=False, eps=1e-6,
                 aux_coef=0.0, z_coef=0.0, residual=torch.bfloat16, shared_expert=False,
                 train_norms=True, train_router=False, device="cuda", checkpoint=None):
        self.layer = MoELoRALayer(T, d, f, E, k, r, alpha, w, shared_expert=shared_expert,
                                  device=device, checkpoint=checkpoint)
        self.y8 = None if checkpoint is None else Packed8(T, d, device)

        def buf(name, *shape, dtype):
            if checkpoint is None:
                return torch.empty(*shape, dtype=dtype, device=device)
            return checkpoint.take(name, shape, dtype, device)
        self.T, self.E, self.k = T, E, k
        self.scale, self.sigmoid, self.eps = float(scale), bool(gate_sigmoid), float(eps)
        self.aux_coef, self.z_coef = float(aux_coef), float(z_coef)
        self.W_r = w["W_r"]
        self.w_post, self.w_pre, self.gate = w.get("w_post"), w.get("w_pre"), w.get("gate")
        f32, bf = dict(dtype=torch.float32, device=device), dict(dtype=torch.bfloat16, device=device)
        res = dict(dtype=residual, device=device)
        like = lambda t: None if t is None or not train_norms else torch.empty_like(t)  # noqa: E731
        self.ids = torch.empty(T, k, dtype=torch.int32, device=device)
        self.topk_w = torch.empty(T, k, **f32)
        self.losses, self.lse, self.pmean = torch.empty(2, **f32), torch.empty(T, **f32), torch.empty(
            E, **f32)
        self.loss_ws = buf("loss_ws", max(16, L.moe_router_loss_workspace_size(T, E)), dtype=torch.uint8)
        self.dlogits = buf("dlogits", T, E, dtype=torch.float32)
        self.r, self.n = torch.empty(T, d, **res), None if self.w_pre is None else torch.empty(T, d, **bf)
        self.rstd_y = None if self.w_post is None else torch.empty(T, **f32)
        self.rstd_r = None if self.w_pre is None else torch.empty(T, **f32)
        self.dr, self.dy = buf("dr", T, d, dtype=residual), buf("dy", T, d, dtype=torch.bfloat16)
        self.norm_ws = buf("norm_ws", max(16, L.moe_block_norm_workspace_size(T, d)), dtype=torch.uint8)
        self.norm_grads = {"dw_post": like(self.w_post), "dw_pre": like(self.w_pre),
                           "dgate": like(self.gate)}
        self.dW_r = torch.empty_like(self.W_r, dtype=torch.float32) if train_router else None

    def _gate(self):
        return dict(gate=self.gate, gate_kind="none" if self.gate is None else "channel",
                    gate_sigmoid=self.sigmoid, scale=self.scale, eps=self.eps)

    def forward(self, r, n):
        """(r', n') for r [T,d] and n [T,d] bf16; n' is None without w_pre.  The
        inputs are kept for the backward.  self.losses holds the router's two
        losses afterwards (without their coefficients)."""
        self._n = n
        self.logits = torch.matmul(n.float(), self.W_r.float().t())
        L.moe_router_topk(self.logits, self.k, self.ids, self.topk_w)
        y = self.layer.forward(n, self.ids, self.topk_w)
        L.moe_router_loss_fwd(self.logits, self.layer.counts, self.k, self.losses, self.lse,
                              self.pmean, self.loss_ws)
        L.moe_block_norm_fwd(r, y, self.r, self.n, w_post=self.w_post, w_pre=self.w_pre,
                             rstd_y=self.rstd_y, rstd_r=self.rstd_r, **self._gate())
        if self.y8 is not None:
            self.y8.pack(y)
        return self.r, self.n

    def backward(self, dr, dn=None):
        """(dr, dn, grads) for the gradients of r' (None: zero) and n'.  dn is a
        new bf16 tensor, the rest are the block's own buffers."""
        g = self.norm_grads
        if self.y8 is not None:
            self.y8.unpack(self.layer.Y)
        L.moe_block_norm_bwd(dr, dn, self.r, self.layer.Y, self.dr, self.dy, w_post=self.w_post,
                             w_pre=self.w_pre, rstd_y=self.rstd_y, rstd_r=self.rstd_r,
                             dgate=g["dgate"], dw_post=g["dw_post"], dw_pre=g["dw_pre"],
                             ws=self.norm_ws, **self._gate())
        lg = self.layer.backward(self.dy)
        L.moe_router_bwd(self.logits, self.lse, self.layer.counts, self.ids, self.topk_w, lg["dw"],
                         self.dlogits, aux_coef=self.aux_coef, z_coef=self.z_coef)
        dn_in = torch.addmm(lg["dX"].float(), self.dlogits, self.W_r.float()).to(torch.bfloat16)
        if self.dW_r is not None:
            torch.matmul(self.dlogits.t(), self._n.float(), out=self.dW_r)
        grads = {k: lg[k] for k in ("dA_gu", "dB_gu", "dA_dn", "dB_dn")}
        grads.update({k: v for k, v in g.items() if v is not None})
        if self.dW_r is not None:
            grads["dW_r"] = self.dW_r
        return self.dr, dn_in, grads
