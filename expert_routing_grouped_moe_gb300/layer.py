"""MoE-LoRA expert layer object: owns the device buffers, calls the C ABI.

``MoELoRALayer`` is a convenience wrapper over the library's calls for one
layer shape: it allocates every buffer once (torch device memory), then
``forward`` runs route -> grouped split-LoRA SwiGLU MLP -> combine and
``backward`` runs the grouped backward -> combine of dX and of the
routing-weight gradient.  With ``gather=False`` (default) the token rows are
first permuted into Xp / dYp by moe_permute and the GEMMs read them with TMA;
with ``gather=True`` the GEMMs copy token rows straight from X and dY
(sorted_src picks them), which saves the two [N, d] permuted buffers but is
slower on GB300.  With ``checkpoint`` (a ``LayerScratch``) the layer keeps its
pre-activations in 8 bits between forward and backward and shares the other
buffers with the layers that have the same scratch.  All arithmetic happens in
the CUDA library; this module only sequences calls and owns memory.
"""
from __future__ import annotations

import torch

from . import _lib as L
from .ckpt import Packed8

# Kernel launches issued by one forward / one backward in the default
# (permuted) mode: route 2 or 3 (L.moe_route_kernel_count), permute 1,
# forward GEMMs 4, combine 1; backward: permute 1, GEMMs 4 + weight-gradient
# GEMMs 4, partial-sum 1, combine 1.  The gather mode issues no permute.
LAUNCHES_FWD = 6   # besides the route's
LAUNCHES_BWD = 11


class MoELoRALayer:
    def __init__(self, T, d, f, E, k, r, alpha, weights: dict, shared_expert=False,
                 device="cuda", gather=False, full_grads=False, rank_r_tokens=False,
                 checkpoint=None):
        """full_grads: the backward also returns dW_gu [G,2f,d] and dW_dn
        [G,d,f] (fp32 gradients of the expert weights, for full fine-tuning;
        needs the permuted-row mode).  rank_r_tokens (permuted-row mode):
        the LoRA-A products xa_gu and u read the token rows of X / dY (small
        enough to stay in L2) instead of the permuted copies.  checkpoint: a
        LayerScratch; the forward then leaves h in 8 bits and the backward works on
        what these stand for (each h off by at most 1/254 of the largest of its
        chunk of 32); X is read again in the backward and must not change until
        then, and dX, dw and Y are the scratch's: they hold until the next call of
        a layer with the same scratch."""
        if full_grads and gather:
            raise ValueError("full weight gradients need the permuted-row mode (gather=False)")
        self.gather = bool(gather)
        self.rank_r_tokens = bool(rank_r_tokens) and not self.gather
        self.full_grads = bool(full_grads)
        self.dims = L.make_dims(T, d, f, E, k, r, alpha / r, shared_expert)
        self.T, self.d, self.f, self.E, self.k, self.r = T, d, f, E, k, r
        self.shared = bool(shared_expert)
        self.G = E + (1 if shared_expert else 0)
        self.K = k + (1 if shared_expert else 0)
        self.N = T * self.K          # permuted rows, in sorted order
        dev = torch.device(device)
        self.w = {n: weights[n].contiguous() for n in ("W_gu", "A_gu", "B_gu", "W_dn", "A_dn",
                                                          "B_dn")}
        i32 = dict(dtype=torch.int32, device=dev)
        bf = dict(dtype=torch.bfloat16, device=dev)
        f32 = dict(dtype=torch.float32, device=dev)
        P, G = self.N, self.G
        self.scratch = checkpoint

        def buf(name, *shape, dtype):   # lives within a call: the scratch's, if there is one
            if checkpoint is None:
                return torch.empty(*shape, dtype=dtype, device=dev)
            return checkpoint.take(name, shape, dtype, dev)
        self.counts = torch.zeros(G, **i32)
        self.offsets = torch.zeros(G + 1, **i32)
        self.tile_off = torch.zeros(G + 1, **i32)
        self.sorted_src = torch.zeros(self.N, **i32)
        self.dest_pos = torch.zeros(self.N, **i32)
        self.route_ws = torch.empty(max(16, L.moe_route_workspace_size(T, self.K, G)),
                                    dtype=torch.uint8, device=dev)
        b16, b32 = torch.bfloat16, torch.float32
        self.Xp = None if self.gather else buf("Xp", P, d, dtype=b16)
        self.Yp = buf("Yp", P, d, dtype=b16)
        # saved intermediates: h in fp32; act / xa_gu / xa_dn as hi+lo bf16 pairs
        hs = 32 * ((f + 15) // 16)
        self.h = buf("h", P, hs, dtype=b32)  # [gate 16 | up 16] chunks
        self.act = buf("act", 2, P, f, dtype=b16)
        self.h8 = None if checkpoint is None else Packed8(P, hs, dev)
        self.xa_gu = torch.empty(2, P, r, **bf)
        self.xa_dn = torch.empty(2, P, r, **bf)
        self.Y = buf("Y", T, d, dtype=b16)
        self.dYp = None if self.gather else buf("dYp", P, d, dtype=b16)
        self.dXp = buf("dXp", P, d, dtype=b16)
        self.dw_rows = buf("dw_rows", P, dtype=b32)
        self.dX = buf("dX", T, d, dtype=b16)
        self.dw = buf("dw", T, k, dtype=b32)
        self.grads = {
            "dA_gu": torch.empty(G, r, d, **f32), "dB_gu": torch.empty(G, 2 * f, r, **f32),
            "dA_dn": torch.empty(G, r, f, **f32), "dB_dn": torch.empty(G, d, r, **f32),
        }
        if self.full_grads:
            self.grads["dW_gu"] = torch.empty(G, 2 * f, d, **f32)
            self.grads["dW_dn"] = torch.empty(G, d, f, **f32)
        self.bwd_ws = buf("bwd_ws", L.moe_mlp_bwd_workspace_size(self.dims), dtype=torch.uint8)
        self._ids = None
        self._topk_w = None

    def launches_per_step(self):
        """Kernel launches of one forward + backward in this layer's mode."""
        ckpt = 0 if self.h8 is None else 2 if self.gather else 3   # pack, unpack, X permuted again
        return (L.moe_route_kernel_count(self.T, self.K, self.G) + LAUNCHES_FWD + LAUNCHES_BWD
                - (2 if self.gather else 0) + (2 if self.full_grads else 0) + ckpt)

    # ------------------------------------------------------------------ steps
    def route(self, ids, stream=None):
        L.moe_route(ids, self.E, self.shared, self.counts, self.offsets, self.tile_off,
                    self.sorted_src, self.dest_pos, self.route_ws, stream)

    def forward(self, X, ids, topk_w, stream=None):
        """Y [T,d] bf16 for token rows X [T,d], top-k ids [T,k], weights [T,k]."""
        self._ids, self._topk_w, self._X = ids, topk_w, X
        self.route(ids, stream)
        if not self.gather:
            L.moe_permute(X, self.K, self.dest_pos, self.Xp, stream)
        w = self.w
        X_tok = X if (self.Xp is None or self.rank_r_tokens) else None
        L.moe_lora_grouped_mlp_fwd(self.dims, self.Xp, X_tok,
                                   self.counts, self.offsets, self.tile_off,
                                   self.sorted_src, topk_w, w["W_gu"], w["A_gu"], w["B_gu"],
                                   w["W_dn"], w["A_dn"], w["B_dn"], self.Yp, self.h, self.act,
                                   self.xa_gu, self.xa_dn, stream)
        L.moe_unpermute_combine(self.Yp, self.dest_pos, self.k, self.shared, self.Y,
                                stream=stream)
        if self.h8 is not None:
            self.h8.pack(self.h, stream)
        return self.Y

    def backward(self, dY, stream=None):
        """dX [T,d] bf16, dw [T,k] fp32 and the four fp32 LoRA gradients."""
        if self._ids is None:
            raise RuntimeError("backward before forward")
        if self.h8 is not None:   # other layers have used the buffers since
            self.h8.unpack_swiglu(self.sorted_src, self._topk_w, self.shared, self.h, self.act, stream)
            if not self.gather:
                L.moe_permute(self._X, self.K, self.dest_pos, self.Xp, stream)
        if not self.gather:
            L.moe_permute(dY, self.K, self.dest_pos, self.dYp, stream)
        w, g = self.w, self.grads
        dY_tok = dY if (self.dYp is None or self.rank_r_tokens) else None
        L.moe_lora_grouped_mlp_bwd(self.dims, self.dYp, dY_tok,
                                   self.Xp, None if self.Xp is not None else self._X,
                                   self.counts, self.offsets,
                                   self.tile_off, self.sorted_src, self._topk_w, w["W_gu"],
                                   w["A_gu"], w["B_gu"], w["W_dn"], w["A_dn"], w["B_dn"], self.h,
                                   self.act, self.xa_gu, self.xa_dn, self.dXp, self.dw_rows,
                                   g["dA_gu"], g["dB_gu"], g["dA_dn"], g["dB_dn"], self.bwd_ws,
                                   stream, dW_gu=g.get("dW_gu"), dW_dn=g.get("dW_dn"))
        L.moe_unpermute_combine(self.dXp, self.dest_pos, self.k, self.shared, self.dX,
                                row_scalars=self.dw_rows, slot_out=self.dw, stream=stream)
        return {"dX": self.dX, "dw": self.dw, **g}

    def step(self, X, ids, topk_w, dY, stream=None):
        """One forward + backward pass of the layer (the hot path)."""
        self.forward(X, ids, topk_w, stream)
        return self.backward(dY, stream)

    def h_gate_up(self):
        """The saved pre-activations as a plain [N, 2f] (gate | up) fp32 tensor
        (un-interleaves the 16-feature chunks of the stored layout); of a
        checkpointed layer what its 8 bits stand for."""
        n, f = self.N, self.f
        h = self.h if self.h8 is None else self.h8.unpack(torch.empty_like(self.h))
        hc = h.view(n, -1, 2, 16)
        gate = hc[:, :, 0, :].reshape(n, -1)[:, :f]
        up = hc[:, :, 1, :].reshape(n, -1)[:, :f]
        return torch.cat([gate, up], dim=1)
