"""Fine-tunes a small stack of MoE blocks on tokens: embedding, adapters, norms, head.

    python examples/finetune_tokens.py [--blocks 4] [--tokens 256] [--vocab 1000] [--steps 40] [--tied]

Sequences follow a fixed random successor for each token; the loss is the mean
negative log probability of the next token, of those that are asked for.  The
blocks keep their activations in 8 bits, the head's values and gradient come from
one call, and one AdamW step takes all gradients, clipped by their norm.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from expert_routing_grouped_moe_gb300 import MoEAdamW, MoEStack, lib, synth  # noqa: E402
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from finetune_block import ADAPTERS, block_weights  # noqa: E402

LENGTH = 32          # tokens of a sequence; its last one has no successor


def batches(tokens, vocab, seed, device):
    """Endless (ids, targets): -100 where nothing is asked."""
    g = torch.Generator(device).manual_seed(seed)
    follows = torch.randperm(vocab, generator=g, device=device)
    while True:
        ids = torch.randint(0, vocab, (tokens,), generator=g, device=device)
        for i in range(1, tokens):
            if i % LENGTH:
                ids[i] = follows[ids[i - 1]]
        targets = torch.roll(ids, -1)
        targets[LENGTH - 1::LENGTH] = -100
        targets[-1] = -100
        yield ids, targets


def train(cfg, vocab=1000, blocks=4, steps=40, tied=False, lr=2e-3, seed=1, device="cuda", log=print):
    """(losses of the steps, the last step's gradients)."""
    g = torch.Generator(device).manual_seed(seed)
    table = torch.randn(vocab, cfg.d, generator=g, device=device).to(torch.bfloat16)
    head = None if tied else (torch.randn(vocab, cfg.d, generator=g, device=device) / cfg.d ** 0.5).to(
        torch.bfloat16)
    weights = [block_weights(cfg, seed + i, device) for i in range(blocks)]
    model = MoEStack(cfg.T, cfg, table, weights, torch.ones(cfg.d, device=device), head=head,
                     residual=torch.float32, scale=0.1 if tied else 1.0, inv_temp=cfg.d ** -0.5 if tied else 1.0,
                     checkpoint=True, train_head=True, gate_sigmoid=True, aux_coef=0.01, z_coef=0.001)
    data = batches(cfg.T, vocab, seed, device)
    losses, opt = [], None
    for step in range(steps):
        ids, targets = next(data)
        asked = targets != -100
        weight = -1.0 / asked.sum().float()
        grads = model.step(ids, targets, weight.expand(cfg.T).contiguous())
        if opt is None:
            pairs = [(model.embedding.table, grads["table"]), (model.w_first, grads["w_first"])]
            if not tied:
                pairs.append((model.head.W, grads["head"]))
            for b, gb in zip(model.blocks, grads["blocks"]):
                w = dict(b.layer.w, w_post=b.w_post, w_pre=b.w_pre, gate=b.gate)
                pairs += [(w[n], gb["d" + n]) for n in ADAPTERS + ("w_post", "w_pre", "gate")]
            opt = MoEAdamW([dict(param=p, state_bits=8 if p.dim() > 1 else 32) for p, _ in pairs],
                           [q for _, q in pairs], lr=lr, max_norm=1.0, skip_nonfinite=True)
        opt.step()
        losses.append((model.head.logp.sum() * weight).item())
        if log and (step % 10 == 0 or step == steps - 1):
            log("step %3d  loss %.4f  gradient norm %.4f" % (step, losses[-1], opt.grad_norm.item()))
    status = lib.moe_status()
    if status != lib.MOE_OK:
        raise RuntimeError("device status %d" % status)
    return losses, [q for _, q in pairs]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--blocks", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=256)
    ap.add_argument("--vocab", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--tied", action="store_true")
    ap.add_argument("--config", default="tiny", choices=sorted(synth.CONFIGS))
    a = ap.parse_args()
    cfg = synth.scaled(synth.CONFIGS[a.config], T=a.tokens, shared=False)
    train(cfg, a.vocab, a.blocks, a.steps, a.tied)


if __name__ == "__main__":
    main()
