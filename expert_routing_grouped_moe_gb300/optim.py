"""AdamW over many tensors at once: owns the moments, calls moe_adamw_step.

``MoEAdamW`` keeps what the step needs besides parameters and gradients: the
moments (fp32, or 8 bits with their scales), optional fp32 master copies of
bf16 parameters, the workspace of the gradient norm and the step count.  All
arithmetic happens in the CUDA library.
"""
from __future__ import annotations

import torch

from . import _lib as L


class MoEAdamW:
    """params: contiguous CUDA tensors, bf16 or fp32, or dicts with "param" and
    optionally "lr_mult", "weight_decay", "state_bits", "master".  grads: one
    tensor for each, bf16 or fp32, read at every step (the layer's gradient
    buffers, say); another list may be passed to step().

    state_bits 8: the moments take 2 bytes and 1/128 a value instead of 8.
    master: keep an fp32 copy of bf16 parameters, which receives the update and
    is rounded to the parameter.  max_norm > 0 clips by
    the global norm of all gradients; grad_norm holds it after each step (also
    with track_norm).  skip_nonfinite: a step whose norm is not finite changes
    nothing; step_count advances all the same."""

    def __init__(self, params, grads, lr=1e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0,
                 state_bits=32, master=True, max_norm=0.0, skip_nonfinite=False,
                 track_norm=False):
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        self.lr, self.betas, self.eps = lr, tuple(betas), eps
        self.max_norm, self.skip_nonfinite = float(max_norm), bool(skip_nonfinite)
        self.step_count = 0
        rows = []
        params, grads = list(params), list(grads)
        if len(params) != len(grads):
            raise ValueError("%d gradients for %d parameters" % (len(grads), len(params)))
        for p, g in zip(params, grads):
            q = dict(p) if isinstance(p, dict) else {"param": p}
            t, bits = q["param"], q.pop("state_bits", state_bits)
            if bits not in (8, 32):
                raise ValueError("state_bits must be 8 or 32")
            keep = q.pop("master", master) and t.dtype == torch.bfloat16
            n, dev = t.numel(), t.device
            sdtype = torch.float32 if bits == 32 else torch.float8_e4m3fn
            rows.append({
                "weight_decay": weight_decay, **q, "grad": g,
                "m": torch.zeros(n, dtype=sdtype, device=dev),
                "v": torch.zeros(n, dtype=sdtype, device=dev),
                "scales": None if bits == 32 else torch.zeros(
                    -(-n // L.MOE_ADAMW_BLOCK), 2, dtype=torch.uint8, device=dev),
                "master": t.detach().float().reshape(-1) if keep else None})
        self.table = L.AdamWTable(rows)
        needs_norm = self.max_norm > 0 or self.skip_nonfinite or track_norm
        dev = rows[0]["param"].device if rows else "cuda"
        self.grad_norm = torch.zeros(1, device=dev) if needs_norm else None
        self.ws = (torch.empty(max(16, L.moe_adamw_workspace_size(self.table)), dtype=torch.uint8,
                               device=dev) if needs_norm else None)

    def step(self, grads=None, lr=None, grad_scale=1.0, stream=None):
        """One step; lr overrides the constructor's for this step (a schedule).  A
        step that is refused does not count."""
        if grads is not None:
            self.table.set_grads(grads)
        # a parameter or a gradient may have been given other memory (3 us for 24 tensors)
        self.table.refresh(("param",) if grads is not None else ("param", "grad"))
        L.moe_adamw_step(self.table, self.step_count + 1, self.lr if lr is None else lr, self.betas,
                         self.eps, grad_scale, self.max_norm, self.skip_nonfinite, self.grad_norm,
                         self.ws, stream)
        self.step_count += 1

    def state_dict(self):
        """Step count and, for each tensor, its moments, scales and master copy."""
        keys = ("m", "v", "scales", "master")
        return {"step": self.step_count,
                "tensors": [{k: r[k] for k in keys if r[k] is not None} for r in self.table.rows]}

    def load_state_dict(self, state):
        if len(state["tensors"]) != self.table.n:
            raise ValueError("the state holds %d tensors, not %d" % (len(state["tensors"]),
                                                                     self.table.n))
        for r, s in zip(self.table.rows, state["tensors"]):
            for k in ("m", "v", "scales", "master"):
                if (r[k] is None) != (s.get(k) is None) or (
                        r[k] is not None and (r[k].shape != s[k].shape or r[k].dtype != s[k].dtype)):
                    raise ValueError("%s of the state does not fit" % k)
        step = int(state["step"])
        for r, s in zip(self.table.rows, state["tensors"]):
            for k in ("m", "v", "scales", "master"):
                if r[k] is not None:
                    r[k].copy_(s[k])
        self.step_count = step
