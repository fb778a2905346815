"""MoEEmbedding, MoEHead, checkpointed layers and MoEStack: the operators together
as a training step uses them."""
import os
import sys

import numpy as np
import pytest
import torch

from expert_routing_grouped_moe_gb300 import (LayerScratch, MoEEmbedding, MoEHead,
                                              MoELoRALayer, MoEStack, lib as L, synth)
from oracle import token_oracle as to
from _tokens import BF, DEV, F32, U, gen, np64

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routing_grouped_moe_gb300 import build
    build.build()
    L.load()


def layer_pair(cfg, scratch, seed, **kw):
    w = synth.layer_weights(cfg, seed, device=DEV)
    args = (cfg.T, cfg.d, cfg.f, cfg.E, cfg.k, cfg.r, cfg.alpha, w)
    a = synth.layer_activations(cfg, seed, device=DEV)
    ids = torch.empty(cfg.T, cfg.k, dtype=torch.int32, device=DEV)
    tw = torch.empty(cfg.T, cfg.k, device=DEV)
    L.moe_router_topk(a["logits"], cfg.k, ids, tw)
    return (MoELoRALayer(*args, shared_expert=cfg.shared, checkpoint=scratch, **kw),
            MoELoRALayer(*args, shared_expert=cfg.shared, **kw), a["X"], ids, tw, a["dY"])


CFGS = [synth.scaled(synth.CONFIGS["tiny"], T=200), synth.scaled(synth.CONFIGS["tiny"], T=133, shared=True, f=72)]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("cfg", CFGS)
def test_checkpointed_layer_works_on_what_its_codes_stand_for(cfg, gather):
    """The same bits as a layer whose h and act are replaced by their 8-bit values by hand."""
    c, p, X, ids, tw, dY = layer_pair(cfg, LayerScratch(DEV), 1, gather=gather)
    assert torch.equal(c.forward(X, ids, tw), p.forward(X, ids, tw))
    for b in (c.Yp, c.act, c.h, c.dXp):
        b.view(torch.uint8).fill_(0x7F)     # another layer's use of the scratch: NaN
    if not gather:
        c.Xp.view(torch.uint8).fill_(0x7F)
    codes = torch.empty(p.h.shape, dtype=torch.int8, device=DEV)
    scales = torch.empty(p.h.shape[0], p.h.shape[1] // 32, dtype=torch.uint8, device=DEV)
    L.moe_ckpt_pack(p.h, codes, scales)
    L.moe_ckpt_unpack_swiglu(codes, scales, p.sorted_src, tw, cfg.shared, p.h, p.act)
    got, want = c.backward(dY), p.backward(dY)
    assert sorted(got) == sorted(want)
    for n in got:
        assert torch.equal(got[n], want[n]), n
    assert L.moe_status() == L.MOE_OK


@pytest.mark.parametrize("kw", [dict(full_grads=True), dict(rank_r_tokens=True),
                                dict(full_grads=True, rank_r_tokens=True)])
def test_checkpointed_layer_with_the_layers_other_options(kw):
    """Full weight gradients read the activations and rows that came back; rank-r products
    read token rows."""
    c, p, X, ids, tw, dY = layer_pair(CFGS[1], LayerScratch(DEV), 7, **kw)
    assert torch.equal(c.forward(X, ids, tw), p.forward(X, ids, tw))
    for b in (c.Yp, c.act, c.h, c.dXp, c.Xp):
        b.view(torch.uint8).fill_(0x7F)
    L.moe_ckpt_unpack_swiglu(c.h8.codes, c.h8.scales, p.sorted_src, tw, True, p.h, p.act)
    got, want = c.backward(dY), p.backward(dY)
    assert sorted(got) == sorted(want)
    for n in got:
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("cfg", CFGS)
def test_checkpointed_gradients_are_near_the_exact_ones(cfg):
    """Each h is off by at most 1/254 of the largest of its 32, some 3 of their spread: 1.2 %
    of it at most and half of that on average.  A gradient is linear in two factors of
    h; 3 % of the gradients' norm bounds them."""
    c, p, X, ids, tw, dY = layer_pair(cfg, LayerScratch(DEV), 2)
    c.forward(X, ids, tw)
    p.forward(X, ids, tw)
    got, want = c.backward(dY), p.backward(dY)
    for n in want:
        off = (got[n].double() - want[n].double()).norm() / want[n].double().norm()
        assert off < 0.03, (n, float(off))


def wide_ups(cfg, seed, times=1000.0, **kw):
    """A layer whose first eight up features are large, and its inputs."""
    w = synth.layer_weights(cfg, seed, device=DEV)
    w["W_gu"][:, cfg.f:cfg.f + 8] *= times
    a = synth.layer_activations(cfg, seed, device=DEV)
    ids = torch.empty(cfg.T, cfg.k, dtype=torch.int32, device=DEV)
    tw = torch.empty(cfg.T, cfg.k, device=DEV)
    L.moe_router_topk(a["logits"], cfg.k, ids, tw)
    make = lambda **k2: MoELoRALayer(cfg.T, cfg.d, cfg.f, cfg.E, cfg.k, cfg.r, cfg.alpha, w,  # noqa: E731
                                     shared_expert=cfg.shared, **kw, **k2)
    return make, a["X"], ids, tw, a["dY"]


@pytest.mark.parametrize("f", [8, 72, 136])
@pytest.mark.parametrize("gather", [False, True])
def test_h_holds_zeros_where_there_is_no_feature(f, gather):
    """f = 8 mod 16: the last chunk has 8 gates and 8 ups, whichever tiles the product takes."""
    cfg = synth.scaled(CFGS[0], f=f)
    make, X, ids, tw, _ = wide_ups(cfg, 3, gather=gather)
    p = make()
    p.h.fill_(9)
    p.forward(X, ids, tw)
    last = p.h.view(p.N, -1, 2, 16)[:, -1]
    assert not last[:, :, 8:].any() and last[:, :, :8].any()


def test_the_last_chunk_is_scaled_by_its_own_features():
    """Codes and scales as those of h with zeros past f: eight large up features of another
    chunk do not cost the last one its bits."""
    make, X, ids, tw, _ = wide_ups(CFGS[1], 4)
    p, c = make(), make(checkpoint=LayerScratch(DEV))
    p.forward(X, ids, tw)
    c.forward(X, ids, tw)
    h = p.h.clone()
    h.view(p.N, -1, 2, 16)[:, -1, :, 8:] = 0
    codes, scales = to.ckpt_pack(h.cpu().numpy())
    assert np.array_equal(c.h8.codes.cpu().numpy(), codes) and np.array_equal(c.h8.scales.cpu().numpy(), scales)


def test_layers_that_share_a_scratch():
    """Forward one, forward the other, backward in reverse: the same as each alone."""
    s = LayerScratch(DEV)
    cfgs = [CFGS[0], synth.scaled(CFGS[0], f=136), CFGS[0]]
    shared = [layer_pair(c, s, 3 + i) for i, c in enumerate(cfgs)]
    alone = [layer_pair(c, LayerScratch(DEV), 3 + i) for i, c in enumerate(cfgs)]
    ys = [q[0].forward(*q[2:5]).clone() for q in shared]
    grads = [None] * 3
    for i in (2, 1, 0):
        grads[i] = {n: t.clone() for n, t in shared[i][0].backward(shared[i][5]).items()}
    for i, q in enumerate(alone):
        assert torch.equal(ys[i], q[0].forward(*q[2:5]))
        want = q[0].backward(q[5])
        for n in want:
            assert torch.equal(grads[i][n], want[n]), (i, n)
    kept = sum(t.numel() * t.element_size() for t in (shared[0][0].h8.codes, shared[0][0].h8.scales))
    assert s.bytes() > 4 * kept
    # whatever the layers' sizes, a view never reaches past its buffer
    assert shared[1][0].h.untyped_storage().nbytes() >= shared[1][0].h.numel() * 4


def test_h_gate_up_of_a_checkpointed_layer_is_its_own():
    """What its codes stand for, also after another layer of the same scratch ran."""
    s = LayerScratch(DEV)
    a, pa, *xa = layer_pair(CFGS[1], s, 5)
    b, _, *xb = layer_pair(CFGS[1], s, 6)
    a.forward(*xa[:3])
    pa.forward(*xa[:3])
    b.forward(*xb[:3])
    L.moe_ckpt_unpack(a.h8.codes, a.h8.scales, pa.h)
    assert torch.equal(a.h_gate_up(), pa.h_gate_up())
    assert not torch.equal(a.h_gate_up(), b.h_gate_up())


@pytest.mark.parametrize("m", [1, 3])
def test_head(m):
    """Its gradients against 64 bits from the logits as they were rounded: dn and dW are
    products of 8-bit-mantissa gradients summed in fp32 (or by the library) over up to
    V or T terms; half a step of bf16 for each gradient and for dn."""
    g = gen(7 + m)
    T, V, d = 90, 1003, 64
    W = (torch.randn(V, d, generator=g, device=DEV) / 8).to(BF)
    n = torch.randn(T, d, generator=g, device=DEV).to(BF)
    y = torch.randint(0, V, (T,) if m == 1 else (T, m), generator=g, device=DEV)
    dlogp = torch.randn(y.shape, generator=g, device=DEV)
    dh = torch.randn(T, generator=g, device=DEV)
    h = MoEHead(W, T, targets=m, entropy=True, top=5, inv_temp=0.8, train=True)
    h.forward(n, y)
    x = np64(h.logits)
    exact = np64(n) @ np64(W).T
    assert (np.abs(x - exact) <= 2.0 ** -8 * np.abs(exact) + 64 * U * (np.abs(np64(n)) @ np.abs(np64(W)).T)).all()
    inv = float(np.float32(0.8))
    r = to.logprob(x, y.view(T, m).cpu().numpy(), inv, top=5)
    assert np.allclose(np64(h.logp).reshape(T, m), r["logp"], rtol=1e-5, atol=1e-4)
    assert np.array_equal(h.top_ids.cpu().numpy(), r["top_ids"])
    d_x, mag = to.logprob_grad(x, y.view(T, m).cpu().numpy(), inv, dlogp=np64(dlogp).reshape(T, m), dentropy=np64(dh))
    dn, dW = (t.clone() for t in h.backward(dlogp, dentropy=dh))
    off = 2.0 ** -8 * np.abs(d_x) + 1e-4 * mag
    tol = off @ np.abs(np64(W)) + 2.0 ** -8 * np.abs(d_x @ np64(W)) + V * U * (np.abs(d_x) @ np.abs(np64(W)))
    assert (np.abs(np64(dn) - d_x @ np64(W)) <= tol).all()
    tol = off.T @ np.abs(np64(n)) + T * U * (np.abs(d_x).T @ np.abs(np64(n)))
    assert (np.abs(np64(dW) - d_x.T @ np64(n)) <= tol).all()
    dn2, dW2 = h.step(n, y, dlogp, dentropy=dh)
    # the two orders of a row's sums: the logits' gradients are the same up to a bf16 step
    assert (dn2.float() - dn.float()).norm() <= 0.01 * dn.float().norm()
    assert (dW2 - dW).norm() <= 0.01 * dW.norm()


def test_a_head_that_was_refused_has_nothing_to_go_back_from():
    g = gen(5)
    W = torch.randn(40, 16, generator=g, device=DEV).to(BF)
    n, y = torch.randn(6, 16, generator=g, device=DEV).to(BF), torch.zeros(6, dtype=torch.int64, device=DEV)
    dlogp = torch.ones(6, device=DEV)
    h = MoEHead(W, 6, train=True)
    h.forward(n, y)
    for call in (lambda: h.step(n, y, dlogp[:5]), lambda: h.forward(n, y[:5])):
        h.forward(n, y)
        with pytest.raises(ValueError):
            call()
        with pytest.raises(RuntimeError):
            h.backward(dlogp)
    h.forward(n, y)
    h.backward(dlogp)


def stack(cfg, V, blocks, checkpoint, tied, residual=BF, **kw):
    import finetune_block as ex
    g = gen(11)
    w = [ex.block_weights(cfg, 5 + i, DEV) for i in range(blocks)]
    table = torch.randn(V, cfg.d, generator=g, device=DEV).to(BF)
    head = None if tied else (torch.randn(V, cfg.d, generator=g, device=DEV) / 11).to(BF)
    first = 1 + 0.1 * torch.randn(cfg.d, generator=g, device=DEV)
    return MoEStack(cfg.T, cfg, table, w, first, head=head, scale=0.5, residual=residual, checkpoint=checkpoint,
                    gate_sigmoid=True, aux_coef=0.01, z_coef=0.001, **kw)


def batch(cfg, V, seed):
    g = gen(seed)
    ids = torch.randint(0, V, (cfg.T,), generator=g, device=DEV)
    y = torch.roll(ids, -1)
    y[::7] = -100
    return ids, y, torch.full((cfg.T,), -1.0 / cfg.T, device=DEV)


def flat(grads):
    out = {"table": grads["table"], "head": grads["head"], "w_first": grads["w_first"]}
    for i, g in enumerate(grads["blocks"]):
        out.update({"%d.%s" % (i, n): t for n, t in g.items()})
    return {n: t for n, t in out.items() if t is not None}


@pytest.mark.parametrize("tied", [False, True])
@pytest.mark.parametrize("residual", [BF, F32])
def test_stack_is_its_parts_in_turn(tied, residual):
    """A stack's step gives the bits of the same calls made one by one."""
    cfg, V = CFGS[0], 517
    a = stack(cfg, V, 2, False, tied, residual, train_head=True)
    ids, y, dlogp = batch(cfg, V, 1)
    a.forward(ids, y)
    got = {n: t.clone() for n, t in flat(a.backward(dlogp)).items()}
    b = stack(cfg, V, 2, False, tied, residual, train_head=True)
    r = b.embedding.forward(ids)
    assert torch.equal(r, (b.embedding.table[ids].float() * 0.5).to(residual))
    L.moe_block_norm_fwd(r, None, None, b.n, w_pre=b.w_first, rstd_r=b.rstd)
    n = b.n
    for blk in b.blocks:
        r, n = blk.forward(r, n)
    assert torch.equal(b.head.forward(n, y), a.head.logp)
    dn, dW = b.head.backward(dlogp)
    dW = None if dW is None else dW.clone()
    dr, gs = None, []
    for blk in reversed(b.blocks):
        dr, dn, g = blk.backward(dr, dn)
        gs.insert(0, g)
    dx, dw = torch.empty_like(dr), torch.empty_like(b.w_first)
    L.moe_block_norm_bwd(dr, dn, b.embedding.out, None, dx, w_pre=b.w_first, rstd_r=b.rstd, dw_pre=dw, ws=b.ws)
    ref, mag, count = to.embed_grad(ids.cpu().numpy(), np64(dx), V, 0.5, base=np64(dW) if tied else None)
    tol = (count[:, None] + 4) * U * mag + U * np.abs(ref)
    assert (np.abs(np64(got["table"]) - ref) <= tol).all()
    assert torch.equal(got["w_first"], dw)
    for i, g in enumerate(gs):
        for name, t in g.items():
            assert torch.equal(got["%d.%s" % (i, name)], t), name
    if not tied:
        assert torch.equal(got["head"], dW)


def test_checkpointed_stack():
    """The same loss; gradients near those without checkpoints (see the layer's bound; 3 %
    for each of three blocks that they pass); the buffers shared."""
    cfg, V = CFGS[0], 517
    a, b = (stack(cfg, V, 3, c, False, F32, train_head=True) for c in (True, False))
    ids, y, dlogp = batch(cfg, V, 2)
    assert torch.equal(a.forward(ids, y), b.forward(ids, y))
    ga, gb = flat(a.backward(dlogp)), flat(b.backward(dlogp))
    assert sorted(ga) == sorted(gb)
    for n in gb:
        off = (ga[n].double() - gb[n].double()).norm() / gb[n].double().norm()
        assert off < 0.09, (n, float(off))
    assert a.blocks[0].layer.h.data_ptr() == a.blocks[2].layer.h.data_ptr()
    assert a.blocks[0].r.data_ptr() != a.blocks[2].r.data_ptr()
    again = flat(a.step(ids, y, dlogp))
    for n in ga:
        off = (again[n].double() - gb[n].double()).norm() / gb[n].double().norm()
        assert off < 0.09, (n, float(off))
    assert L.moe_status() == L.MOE_OK


def test_a_stack_is_exact_unless_told_otherwise():
    cfg, V = CFGS[0], 517
    import finetune_block as ex
    g = gen(11)
    table = torch.randn(V, cfg.d, generator=g, device=DEV).to(BF)
    w = lambda: [ex.block_weights(cfg, 5 + i, DEV) for i in range(2)]  # noqa: E731
    args = (cfg.T, cfg, table)
    first = torch.ones(cfg.d, device=DEV)
    a, b = MoEStack(*args, w(), first), MoEStack(*args, w(), first, checkpoint=False)
    ids, y, dlogp = batch(cfg, V, 2)
    for m in (a, b):
        m.forward(ids, y)
    ga, gb = flat(a.backward(dlogp)), flat(b.backward(dlogp))
    for n in gb:
        assert torch.equal(ga[n], gb[n]), n


def test_gradient_of_a_token_that_is_not_there():
    """The loss asked of one position moves only the rows of the batch's tokens."""
    cfg, V = CFGS[0], 517
    a = stack(cfg, V, 1, True, False)
    ids, y, _ = batch(cfg, 100, 3)
    dlogp = torch.zeros(cfg.T, device=DEV)
    dlogp[5] = -1.0
    y[:] = 1
    a.forward(ids, y)
    g = a.backward(dlogp)
    assert not g["table"][100:].any() and g["table"][ids[5]].any() and g["head"] is None


def test_captured_step():
    """Forward, backward and their replay on other tokens, beside an eager stack."""
    cfg, V = CFGS[0], 517
    a, e = stack(cfg, V, 2, True, True), stack(cfg, V, 2, True, True)
    ids, y, dlogp = batch(cfg, V, 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a.step(ids, y, dlogp)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = flat(a.step(ids, y, dlogp))
    for seed in (5, 6):
        i2, y2, _ = batch(cfg, V, seed)
        ids.copy_(i2)
        y.copy_(y2)
        graph.replay()
        want = flat(e.step(i2, y2, dlogp))
        assert torch.equal(a.head.logp, e.head.logp)
        for n in want:
            assert torch.equal(grads[n], want[n]), n


def test_refusals():
    W = torch.zeros(7, 8, dtype=BF, device=DEV)
    with pytest.raises(RuntimeError):
        MoEEmbedding(W, 4).backward(torch.zeros(4, 8, dtype=BF, device=DEV))
    with pytest.raises(RuntimeError):
        MoEHead(W, 4).backward(torch.zeros(4, device=DEV))
    with pytest.raises(ValueError):
        MoEHead(W.float(), 4)
    with pytest.raises(ValueError):
        stack(CFGS[0], 50, 0, True, True)
    h = MoEHead(W, 4)
    h.forward(torch.zeros(4, 8, dtype=BF, device=DEV), torch.zeros(4, dtype=torch.int64, device=DEV))
    h.backward(torch.zeros(4, device=DEV))
    with pytest.raises(RuntimeError):   # the logits are gone
        h.backward(torch.zeros(4, device=DEV))
    with pytest.raises(ValueError):
        MoEEmbedding(W, 4).forward(torch.zeros(5, dtype=torch.int64, device=DEV))


@pytest.mark.parametrize("tied", [False, True])
def test_example_runs_and_trains_on_its_gradients(tied):
    import finetune_tokens as ex
    losses, grads = ex.train(CFGS[0], vocab=300, blocks=2, steps=3, tied=tied, log=None)
    assert len(losses) == 3 and all(np.isfinite(losses))
    assert all(torch.isfinite(g).all() and g.abs().max() > 0 for g in grads)
