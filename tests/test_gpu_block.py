"""MoEBlock and MoEAdamW: a block's forward and backward against the oracles
strung together in 64 bits, the optimizer object's state, and the example's
training run."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle
from oracle import block_oracle as bo
from expert_routing_grouped_moe_gb300 import MoEAdamW, MoEBlock, lib as L, synth
from _util import assert_close_bf16, oracle_params, to64

pytestmark = pytest.mark.gpu
DEV = "cuda"
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routing_grouped_moe_gb300 import build
    build.build()
    L.load()


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("residual", [torch.bfloat16, torch.float32])
def test_block_forward_and_backward(residual, shared):
    import finetune_block as ex
    cfg = synth.scaled(synth.CONFIGS["tiny"], T=200, shared=shared)
    w = ex.block_weights(cfg, 3, DEV)
    g = torch.Generator(DEV).manual_seed(5)
    w["w_post"] = 1 + 0.2 * torch.randn(cfg.d, generator=g, device=DEV)
    w["w_pre"] = 1 + 0.2 * torch.randn(cfg.d, generator=g, device=DEV)
    w["gate"] = torch.randn(cfg.d, generator=g, device=DEV)
    aux, z, scale = 0.5, 0.25, 0.75
    b = MoEBlock(cfg.T, cfg.d, cfg.f, cfg.E, cfg.k, cfg.r, cfg.alpha, w, scale=scale,
                 gate_sigmoid=True, aux_coef=aux, z_coef=z, residual=residual,
                 shared_expert=shared, train_router=True)
    r = synth.hidden_rows(cfg.T, cfg.d, 1, device=DEV).to(residual)
    n = synth.hidden_rows(cfg.T, cfg.d, 2, device=DEV)
    dr = synth.hidden_rows(cfg.T, cfg.d, 3, device=DEV).to(residual)
    dn = synth.hidden_rows(cfg.T, cfg.d, 4, device=DEV)
    r1, n1 = b.forward(r, n)
    dr0, dn0, gr = b.backward(dr, dn)
    assert L.moe_status() == L.MOE_OK
    # the oracles in the same order; the layer's output enters as it is stored
    ids, tw = b.ids.cpu().numpy(), to64(b.topk_w)
    P = oracle_params({k: w[k] for k in ("W_gu", "A_gu", "B_gu", "W_dn", "A_dn", "B_dn")}, cfg)
    N = to64(n)
    assert_close_bf16(to64(b.layer.Y), oracle.layer_forward(N, ids, tw, P), "y")
    kw = dict(gate=to64(w["gate"]), kind="channel", sigmoid=True, scale=scale)
    f = bo.block_norm_forward(to64(r), to64(b.layer.Y), to64(w["w_post"]), to64(w["w_pre"]), **kw)
    assert_close_bf16(to64(r1), f["r"], "r")
    assert_close_bf16(to64(n1), f["n"], "n")
    counts = b.layer.counts.cpu().numpy()
    losses, _, _ = bo.router_losses(to64(b.logits), counts, cfg.k)
    np.testing.assert_allclose(to64(b.losses), losses, rtol=1e-5)
    q = bo.block_norm_backward(to64(dr), to64(dn), to64(r1), to64(b.layer.Y), to64(w["w_post"]),
                               to64(w["w_pre"]), to64(b.rstd_y), to64(b.rstd_r), **kw)
    assert_close_bf16(to64(dr0), q["dx"], "dr")
    for name in ("dgate", "dw_post", "dw_pre"):
        assert_close_bf16(to64(gr[name]), q[name], name)
    lo = oracle.layer_backward(N, ids, tw, to64(b.dy), P)
    for name in ("dA_gu", "dB_gu", "dA_dn", "dB_dn"):
        assert_close_bf16(to64(gr[name]), lo[name], name)
    dl, _ = bo.router_backward(to64(b.logits), counts, ids, tw, to64(b.layer.dw), aux, z, cfg.k)
    assert_close_bf16(to64(b.dlogits), dl, "dlogits")
    assert_close_bf16(to64(dn0), lo["dX"] + dl @ to64(w["W_r"]), "dn", rel_fro=1e-2)
    assert_close_bf16(to64(gr["dW_r"]), to64(b.dlogits).T @ N, "dW_r")


@pytest.mark.parametrize("bits", [8, 32])
def test_the_example_learns(bits):
    import finetune_block as ex
    cfg = synth.scaled(synth.CONFIGS["tiny"], T=256)
    losses = ex.train(cfg, blocks=2, steps=60, state_bits=bits, log=None)
    assert all(np.isfinite(losses)) and losses[-1] < 0.6 * losses[0], (losses[0], losses[-1])


def test_optimizer_state_saves_and_loads():
    g = torch.Generator(DEV).manual_seed(1)
    mk = lambda: [torch.randn(1000, generator=g, device=DEV).bfloat16(),  # noqa: E731
                  torch.randn(33, generator=g, device=DEV)]
    p, grads = mk(), [t.float() for t in mk()]
    opts = []
    for _ in range(2):
        q = [t.clone() for t in p]
        opts.append((q, MoEAdamW(q, grads, lr=1e-2, state_bits=8, max_norm=1.0)))
    (pa, a), (pb, b) = opts
    for _ in range(3):
        a.step()
    saved = {"step": a.state_dict()["step"],
             "tensors": [{k: v.clone() for k, v in t.items()} for t in a.state_dict()["tensors"]]}
    for t, s in zip(pb, pa):
        t.copy_(s)
    b.load_state_dict(saved)
    a.step()
    b.step([t.clone() for t in grads])
    assert b.step_count == 4
    for t, s in zip(pa, pb):
        assert torch.equal(t, s)
    with pytest.raises(ValueError, match="does not fit"):
        b.load_state_dict({"step": 1, "tensors": [{}, {}]})
    with pytest.raises(ValueError, match="gradients for"):
        b.step(grads[:1])


def test_a_refused_step_does_not_count():
    p, g = torch.randn(500, device=DEV), torch.randn(500, device=DEV)
    q = p.clone()
    a, b = MoEAdamW([p], [g], lr=1e-2), MoEAdamW([q], [g], lr=1e-2)
    for bad in (dict(lr=float("nan")), dict(lr=-1.0), dict(grad_scale=float("inf"))):
        with pytest.raises(L.MoeError):
            a.step(**bad)
    with pytest.raises(ValueError, match="as many values"):
        a.step(grads=[g[:100]])
    assert a.step_count == 0
    for _ in range(2):
        a.step()
        b.step()
    assert a.step_count == b.step_count == 2 and torch.equal(p, q)


@pytest.mark.parametrize("bits", [8, 32])
def test_parameters_and_gradients_that_were_given_other_memory(bits):
    """p.data = ... between two steps: the step goes to the new memory, and the old
    one, kept by whoever still has it, stays as it is."""
    g = torch.Generator(DEV).manual_seed(7)
    mk = lambda: [torch.randn(n, generator=g, device=DEV) for n in (700, 33)]  # noqa: E731
    p, grads, later, later_grads = mk(), mk(), mk(), mk()
    q = [t.clone() for t in p]
    a = MoEAdamW(p, grads, lr=1e-2, state_bits=bits, max_norm=1.0)
    b = MoEAdamW(q, [t.clone() for t in grads], lr=1e-2, state_bits=bits, max_norm=1.0)
    a.step()
    b.step()
    old, before = p[0].detach(), p[0].clone()
    p[0].data = later[0].clone()
    grads[1].data = later_grads[1].clone()
    q[0].copy_(later[0])
    b.table.rows[1]["grad"].copy_(later_grads[1])
    a.step()
    b.step()
    assert torch.equal(old, before)
    assert all(torch.equal(s, t) for s, t in zip(p, q))
    # a size that does not fit is refused and changes nothing
    p[1].data = torch.zeros(34, device=DEV)
    with pytest.raises(ValueError):
        a.step()
    assert a.step_count == 2 and torch.equal(p[0], q[0])


def test_the_optimizers_table_keeps_its_memory():
    """The memory that the table points to is not handed out again while it does."""
    ts = [torch.zeros(1 << 20, device=DEV) for _ in range(4)]
    row = dict(zip(("param", "grad", "m", "v"), ts))
    table = L.AdamWTable([row])
    ptrs = {t.data_ptr() for t in ts}
    for t in ts:
        t.data = torch.empty(0, device=DEV)
    again = [torch.ones(1 << 20, device=DEV) for _ in range(8)]
    assert not ptrs & {t.data_ptr() for t in again}
    with pytest.raises(ValueError):   # nothing of the row fits any more
        table.refresh()
    L.moe_adamw_step(table, 1, lr=0.1)
    assert all(bool((t == 1).all()) for t in again)


def test_a_state_that_is_refused_loads_nothing():
    p, g = torch.randn(500, device=DEV), torch.randn(500, device=DEV)
    a = MoEAdamW([p, p.clone()], [g, g], lr=1e-2, state_bits=8)
    a.step()
    held = [{k: t.clone() for k, t in s.items()} for s in a.state_dict()["tensors"]]
    other = [{k: torch.zeros_like(t) for k, t in s.items()} for s in held]
    with pytest.raises(KeyError):
        a.load_state_dict({"tensors": other})                     # no step
    with pytest.raises(ValueError, match="does not fit"):
        a.load_state_dict({"step": 3, "tensors": [other[0], dict(other[1], m=None)]})
    assert a.step_count == 1
    for s, h in zip(a.state_dict()["tensors"], held):
        assert all(torch.equal(s[k].view(torch.uint8), h[k].view(torch.uint8)) for k in h)
    a.load_state_dict({"step": 3, "tensors": [dict(s, note="kept elsewhere") for s in other]})
    assert a.step_count == 3 and not a.state_dict()["tensors"][1]["scales"].any()
