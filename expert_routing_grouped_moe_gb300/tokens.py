"""The two ends of a stack of blocks: token embedding and language-model head.

``MoEEmbedding`` and ``MoEHead`` own the buffers of ``lib.moe_embed_*`` and
``lib.moe_logprob_*`` for one batch size; ``MoEStack`` strings them together
with ``MoEBlock``s: tokens in, log probabilities out, and the gradients of one
training step.  The products with the head's weight are plain matrix products
(torch.mm); everything else runs in the CUDA library, on the current stream.
"""
from __future__ import annotations

import torch

from . import _lib as L
from .block import MoEBlock
from .ckpt import LayerScratch


class MoEEmbedding:
    """table [V,d], bf16 or fp32.  out: type of the rows (the residual stream's).
    train: backward() gives the table's gradient, in fp32, dense; grad: a tensor of its
    own that the gradient is added to instead (a tied head's, say)."""

    def __init__(self, table, tokens, out=torch.bfloat16, scale=1.0, pad_id=None, train=True,
                 grad=None):
        V, d = table.shape
        self.table, self.scale, self.pad_id = table, float(scale), pad_id
        self.out = torch.empty(tokens, d, dtype=out, device=table.device)
        self.shared = grad is not None
        self.grad = grad if self.shared else torch.empty(
            V, d, dtype=torch.float32, device=table.device) if train else None
        self.ws = (torch.empty(max(16, L.moe_embed_workspace_size(tokens, V, d)), dtype=torch.uint8,
                               device=table.device) if self.grad is not None else None)
        self._ids = None

    def forward(self, ids):
        """Rows [tokens, d] of ids [tokens] (int32 or int64), kept for the backward."""
        self._ids = ids
        L.moe_embed_fwd(ids, self.table, self.out, scale=self.scale)
        return self.out

    def backward(self, dout):
        """The table's gradient (None if it is not trained) from that of the rows."""
        if self._ids is None:
            raise RuntimeError("backward before forward")
        if self.grad is not None:
            L.moe_embed_bwd(self._ids, dout, self.grad, self.ws, scale=self.scale,
                            pad_id=self.pad_id, accumulate=self.shared)
        return self.grad


class MoEHead:
    """Logits = n W^T for rows n [tokens, d] bf16 and W [V,d] bf16, and what
    lib.moe_logprob_fwd makes of them.  targets: m tokens of each row.  After a call
    logp, lse and, where they were asked for, entropy, top_ids and top_logp hold its
    results.  The backward overwrites the logits with their gradient."""

    def __init__(self, W, tokens, targets=1, entropy=False, top=0, inv_temp=1.0, ignore_id=-100,
                 train=False):
        if W.dim() != 2 or W.dtype != torch.bfloat16:
            raise ValueError("W must be [V, d] torch.bfloat16")
        V = W.shape[0]
        dev, f32 = W.device, dict(dtype=torch.float32, device=W.device)
        self.W, self.inv_temp, self.ignore_id = W, float(inv_temp), int(ignore_id)
        shape = (tokens,) if targets == 1 else (tokens, targets)
        self.logits = torch.empty(tokens, V, dtype=torch.bfloat16, device=dev)
        self.logp, self.stats = torch.empty(shape, **f32), torch.empty(tokens, 2, **f32)
        self.lse = torch.empty(tokens, **f32)
        self.entropy = torch.empty(tokens, **f32) if entropy else None
        self.top_ids = torch.empty(tokens, top, dtype=torch.int32, device=dev) if top else None
        self.top_logp = torch.empty(tokens, top, **f32) if top else None
        self.dn = torch.empty(tokens, W.shape[1], dtype=torch.bfloat16, device=dev)
        self.dW = torch.empty(W.shape, **f32) if train else None
        self._n = None

    def _wanted(self):
        return dict(lse=self.lse, entropy=self.entropy, top_ids=self.top_ids,
                    top_logp=self.top_logp, inv_temp=self.inv_temp, ignore_id=self.ignore_id)

    def _logits(self, n):
        self._n = None     # of the call before; this one's once its logits have their values
        torch.mm(n, self.W.t(), out=self.logits)

    def forward(self, n, targets):
        """logp of targets [tokens] or [tokens, m] (int32 or int64)."""
        self._logits(n)
        L.moe_logprob_fwd(self.logits, targets, self.logp, self.stats, **self._wanted())
        self._n, self._targets = n, targets
        return self.logp

    def _back(self, n):
        self._n = None     # the logits are gone
        torch.mm(self.logits, self.W, out=self.dn)
        if self.dW is not None:
            torch.mm(self.logits.t(), n, out_dtype=torch.float32, out=self.dW)
        return self.dn, self.dW

    def backward(self, dlogp, dentropy=None, dlse=None):
        """(dn, dW or None) for the gradients of logp, entropy and lse."""
        if self._n is None:
            raise RuntimeError("backward before forward")
        L.moe_logprob_bwd(self.logits, self._targets, self.stats, dlogp, self.logits,
                          entropy=self.entropy, dentropy=dentropy, dlse=dlse,
                          inv_temp=self.inv_temp, ignore_id=self.ignore_id)
        return self._back(self._n)

    def step(self, n, targets, dlogp, dentropy=None, dlse=None):
        """forward and backward together, for gradients that are known ahead:
        (dn, dW or None)."""
        self._logits(n)
        L.moe_logprob_step(self.logits, targets, self.logp, self.stats, dlogp, self.logits,
                           dentropy=dentropy, dlse=dlse, **self._wanted())
        return self._back(n)


class MoEStack:
    """Embedding, first norm, blocks and head for ``tokens`` tokens.

        r = scale table[ids],  n = norm(r; w_first);  (r, n) through the blocks;
        logits = n W^T of the last normed stream

    cfg: f, E, k, r, alpha of the layers (a synth.LayerConfig will do).  blocks: one
    weight dict for each MoEBlock, all with w_pre.  head: W [V,d] bf16, or None: the
    table itself (bf16; with train_embedding its gradient gets both parts).
    checkpoint: the blocks keep their activations in 8 bits and share their buffers, which
    saves most of their memory and moves the gradients by about 1 % of their norm a block.
    train_norms (w_first among them) and the rest go to MoEBlock."""

    def __init__(self, tokens, cfg, table, blocks, w_first, head=None, scale=1.0, pad_id=None,
                 residual=torch.bfloat16, checkpoint=False, targets=1, entropy=False, top=0,
                 inv_temp=1.0, ignore_id=-100, train_embedding=True, train_head=False,
                 train_norms=True, eps=1e-6, **block):
        if not blocks or any(w.get("w_pre") is None for w in blocks):
            raise ValueError("a stack needs blocks, each with the weight w_pre of the norm after it")
        d, dev = table.shape[1], table.device
        self.tied = head is None
        self.head = MoEHead(table if self.tied else head, tokens, targets, entropy, top, inv_temp,
                            ignore_id, train=train_embedding if self.tied else train_head)
        self.embedding = MoEEmbedding(table, tokens, residual, scale, pad_id, train_embedding,
                                      grad=self.head.dW if self.tied else None)
        self.scratch = LayerScratch(dev) if checkpoint else None
        self.blocks = [MoEBlock(tokens, d, cfg.f, cfg.E, cfg.k, cfg.r, cfg.alpha, w, residual=residual,
                                eps=eps, train_norms=train_norms, checkpoint=self.scratch, device=dev,
                                **block)
                       for w in blocks]
        f32 = dict(dtype=torch.float32, device=dev)
        self.w_first, self.eps = w_first, float(eps)
        self.rstd = torch.empty(tokens, **f32)
        self.n = torch.empty(tokens, d, dtype=torch.bfloat16, device=dev)
        self.dx = torch.empty(tokens, d, dtype=residual, device=dev)
        self.dw_first = torch.empty_like(w_first) if train_norms else None
        self.ws = torch.empty(max(16, L.moe_block_norm_workspace_size(tokens, d)),
                              dtype=torch.uint8, device=dev) if train_norms else None

    def _through(self, ids):
        r = self.embedding.forward(ids)
        L.moe_block_norm_fwd(r, None, None, self.n, w_pre=self.w_first, rstd_r=self.rstd, eps=self.eps)
        n = self.n
        for b in self.blocks:
            r, n = b.forward(r, n)
        return n

    def _back(self, dn, dW):
        dr, grads = None, []
        for b in reversed(self.blocks):
            dr, dn, g = b.backward(dr, dn)
            grads.insert(0, g)
        L.moe_block_norm_bwd(dr, dn, self.embedding.out, None, self.dx, w_pre=self.w_first,
                             rstd_r=self.rstd, dw_pre=self.dw_first, ws=self.ws, eps=self.eps)
        return {"blocks": grads, "table": self.embedding.backward(self.dx),
                "head": None if self.tied else dW, "w_first": self.dw_first}

    def forward(self, ids, targets):
        """logp of targets [tokens] or [tokens, m] given the tokens ids [tokens]; lse,
        entropy and alternatives are in self.head."""
        return self.head.forward(self._through(ids), targets)

    def backward(self, dlogp, dentropy=None, dlse=None):
        """Gradients: "blocks" (each MoEBlock's), "table" (with a tied head's part),
        "head", "w_first"; None where one is not trained."""
        return self._back(*self.head.backward(dlogp, dentropy, dlse))

    def step(self, ids, targets, dlogp, dentropy=None, dlse=None):
        """forward and backward, the head's in one call; logp is in self.head."""
        return self._back(*self.head.step(self._through(ids), targets, dlogp, dentropy, dlse))
