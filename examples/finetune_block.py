"""Fine-tunes the adapters, norm weights and gates of a few MoE blocks.

    python examples/finetune_block.py [--blocks 2] [--tokens 256] [--steps 60] [--state-bits 8]

A teacher (the same frozen weights, other adapters) gives the targets; the
loss is the mean squared error of the last normed stream, plus the router's
load-balancing and z losses.  Every step runs the whole path: norms, router,
expert layers, their backward passes, and one AdamW step over all tensors with
the gradient norm clipped.  Prints the loss and the norm.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from expert_routing_grouped_moe_gb300 import MoEAdamW, MoEBlock, lib, synth  # noqa: E402

ADAPTERS = ("A_gu", "B_gu", "A_dn", "B_dn")
AUX, ZED = 0.01, 0.001


def block_weights(cfg, seed, device):
    w = synth.layer_weights(cfg, seed, device=device)
    g = torch.Generator(device).manual_seed(seed * 31 + 7)
    w["W_r"] = (torch.randn(cfg.E, cfg.d, generator=g, device=device) / cfg.d ** 0.5).to(torch.bfloat16)
    w["w_post"] = torch.ones(cfg.d, device=device)
    w["w_pre"] = torch.ones(cfg.d, device=device)
    w["gate"] = torch.zeros(cfg.d, device=device)      # sigmoid(0) = 1/2
    return w


class Model:
    """Blocks one after the other; the first norm (of the input) is frozen."""

    def __init__(self, cfg, weights, device):
        self.blocks = [MoEBlock(cfg.T, cfg.d, cfg.f, cfg.E, cfg.k, cfg.r, cfg.alpha, w,
                                gate_sigmoid=True, aux_coef=AUX, z_coef=ZED, residual=torch.float32,
                                device=device) for w in weights]
        self.first = torch.ones(cfg.d, device=device)
        self.rstd = torch.empty(cfg.T, device=device)
        self.n0 = torch.empty(cfg.T, cfg.d, dtype=torch.bfloat16, device=device)

    def forward(self, x):
        lib.moe_block_norm_fwd(x, None, None, self.n0, w_pre=self.first, rstd_r=self.rstd)
        r, n = x, self.n0
        for b in self.blocks:
            r, n = b.forward(r, n)
        return n

    def backward(self, dn):
        """The blocks' gradients, from the gradient of the last normed stream."""
        dr, grads = None, []
        for b in reversed(self.blocks):
            dr, dn, g = b.backward(dr, dn)
            grads.insert(0, g)
        return grads

    def trained(self):
        """(parameter, name of its gradient) of every block."""
        out = []
        for b in self.blocks:
            w = dict(b.layer.w, w_post=b.w_post, w_pre=b.w_pre, gate=b.gate)
            out.append([(w[n], "d" + n) for n in ADAPTERS + ("w_post", "w_pre", "gate")])
        return out


def train(cfg, blocks=2, steps=60, state_bits=8, lr=2e-3, seed=1, device="cuda", log=print):
    """Losses of the steps."""
    weights = [block_weights(cfg, seed + i, device) for i in range(blocks)]
    teacher = []
    for i, w in enumerate(weights):
        other = synth.layer_weights(cfg, seed + 100 + i, device=device)
        teacher.append(dict(w, **{n: other[n] for n in ADAPTERS}))
        w["B_gu"], w["B_dn"] = torch.zeros_like(w["B_gu"]), torch.zeros_like(w["B_dn"])
    x = synth.hidden_rows(cfg.T, cfg.d, seed, device=device).float()
    target = Model(cfg, teacher, device).forward(x).float()
    model = Model(cfg, weights, device)
    grads = model.backward((model.forward(x).float() - target).to(torch.bfloat16))
    pairs = [(p, g[name]) for ps, g in zip(model.trained(), grads) for p, name in ps]
    # adapters: bf16 with fp32 master copies; norm weights and gates: fp32, never
    # decayed, their few moments in 32 bits
    opt = MoEAdamW([dict(param=p, weight_decay=0.01 if p.dim() > 1 else 0.0,
                         state_bits=state_bits if p.dim() > 1 else 32) for p, _ in pairs],
                   [g for _, g in pairs], lr=lr, max_norm=1.0, skip_nonfinite=True)
    losses = []
    for step in range(steps):
        n = model.forward(x).float()
        diff = n - target
        model.backward((diff * (2.0 / diff.numel())).to(torch.bfloat16))
        opt.step()
        router = sum(AUX * b.losses[0] + ZED * b.losses[1] for b in model.blocks)
        losses.append((diff.square().mean() + router).item())
        if log and (step % 10 == 0 or step == steps - 1):
            log("step %3d  loss %.5f  gradient norm %.4f" % (step, losses[-1], opt.grad_norm.item()))
    status = lib.moe_status()
    if status != lib.MOE_OK:
        raise RuntimeError("device status %d" % status)
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=256)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=8)
    ap.add_argument("--config", default="tiny", choices=sorted(synth.CONFIGS))
    a = ap.parse_args()
    cfg = synth.scaled(synth.CONFIGS[a.config], T=a.tokens, shared=False)
    train(cfg, a.blocks, a.steps, a.state_bits)


if __name__ == "__main__":
    main()
