"""Host-side argument checks of the norms around a block, the router's losses
and the AdamW step: error codes and messages before anything is launched (no
GPU needed; pointers are never dereferenced)."""
import ctypes

import pytest

P = ctypes.c_void_p
A = P(1 << 20)          # aligned
ODD = P((1 << 20) + 1)  # not even aligned for bf16


@pytest.fixture(scope="module")
def L():
    from expert_routing_grouped_moe_gb300 import build, _lib
    build.build()
    _lib.load()
    return _lib


def desc(L, **kw):
    base = dict(T=4, d=64, x_type=1, y_type=1, gate=0, gate_sigmoid=0, scale=1.0, eps=1e-6,
                w_offset=0.0)
    base.update(kw)
    return L.MoeNormDesc(**base)


def fwd(L, q, x=A, y=A, gate=None, w_post=A, w_pre=A, r=A, n=A, rstd_y=A, rstd_r=A):
    return L.load().moe_block_norm_fwd(ctypes.byref(q), x, y, gate, w_post, w_pre, r, n, rstd_y,
                                       rstd_r, None)


def bwd(L, q, dr=A, dn=A, r=A, y=A, gate=None, w_post=A, w_pre=A, rstd_y=A, rstd_r=A, dx=A, dy=A,
        dgate=None, dw_post=A, dw_pre=A, ws=A, ws_bytes=1 << 40):
    return L.load().moe_block_norm_bwd(ctypes.byref(q), dr, dn, r, y, gate, w_post, w_pre, rstd_y,
                                       rstd_r, dx, dy, dgate, dw_post, dw_pre, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(d=0), -1), (dict(d=16385), -2), (dict(x_type=2), -1),
    (dict(x_type=1, y_type=0), -2), (dict(gate=4), -1), (dict(gate_sigmoid=2), -1),
    (dict(eps=0.0), -1), (dict(eps=float("nan")), -1), (dict(scale=float("inf")), -1)])
def test_norm_descriptor(L, kw, code):
    assert fwd(L, desc(L, **kw)) == code
    assert bwd(L, desc(L, **kw)) == code


@pytest.mark.parametrize("kw", [
    dict(x=None, y=None), dict(y=None), dict(y=None, r=None), dict(r=None), dict(n=None),
    dict(w_pre=None), dict(rstd_y=None), dict(rstd_r=None), dict(gate=A), dict(x=ODD),
    dict(w_post=P((1 << 20) + 2)),
    dict(y=None, r=None, w_post=None, w_pre=None, n=None)])
def test_norm_forward_pointers(L, kw):
    assert fwd(L, desc(L), **kw) == L.MOE_ERR_INVALID_ARG
    assert L.load().moe_last_error()


@pytest.mark.parametrize("kw", [
    dict(dr=None, dn=None), dict(dn=None), dict(r=None), dict(w_pre=None), dict(y=None),
    dict(rstd_y=None), dict(dgate=A), dict(dy=ODD), dict(ws=None), dict(ws=P((1 << 20) + 8)),
    dict(w_post=None),
    dict(dx=None, dy=None, dw_post=None, dw_pre=None)])
def test_norm_backward_pointers(L, kw):
    assert bwd(L, desc(L), **kw) == L.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(gate=None), dict(gate=P((1 << 20) + 2)), dict(w_post=P((1 << 20) + 2)), dict(dgate=ODD)])
def test_norm_backward_without_tokens_checks_the_vectors_of_d_values(L, kw):
    """T = 0 leaves the gate of a channel kind and the weights as they are for T > 0."""
    kw = dict(dict(gate=A), **kw)
    assert bwd(L, desc(L, T=0, gate=2), **kw) == L.MOE_ERR_INVALID_ARG
    assert bwd(L, desc(L, gate=2), **kw) == L.MOE_ERR_INVALID_ARG


def test_norm_backward_without_tokens_and_a_gate_without_a_kind(L):
    assert bwd(L, desc(L, T=0, gate=0), gate=A) == L.MOE_ERR_INVALID_ARG
    # nothing is launched where no sum over the tokens is wanted
    for kind in (1, 3):
        assert bwd(L, desc(L, T=0, gate=kind), dw_post=None, dw_pre=None) == L.MOE_OK


def test_norm_workspace(L):
    lib = L.load()
    assert bwd(L, desc(L), ws_bytes=8) == L.MOE_ERR_WORKSPACE
    assert lib.moe_block_norm_workspace_size(0, 64) == 0
    assert lib.moe_block_norm_workspace_size(4, 16385) == 0
    # two column sums for each row of partials, at most as many rows as tokens
    # rounded up to a block's
    assert lib.moe_block_norm_workspace_size(1, 2048) == 2 * 2048 * 4
    assert lib.moe_block_norm_workspace_size(1 << 20, 2048) == \
        lib.moe_block_norm_workspace_size(1 << 30, 2048)


def test_router_arguments(L):
    lib = L.load()
    bad = L.MOE_ERR_INVALID_ARG

    def loss(T=4, E=8, k=2, p=(A, A, A, A, A, A), nbytes=1 << 30):
        return lib.moe_router_loss_fwd(p[0], T, E, k, *p[1:], nbytes, None)

    def grad(T=4, E=8, k=2, logits=A, lse=A, counts=A, ids=A, w=A, dw=A, aux=1.0, z=1.0, dl=A):
        return lib.moe_router_bwd(logits, lse, T, E, k, counts, ids, w, dw, aux, z, dl, None)
    for i in range(6):
        assert loss(p=[None if j == i else A for j in range(6)]) == bad
        assert loss(p=[ODD if j == i else A for j in range(6)]) == bad
    assert loss(T=0) == bad and loss(k=9) == bad and loss(E=0) == bad
    assert loss(E=1025) == L.MOE_ERR_UNSUPPORTED and loss(E=64, k=33) == L.MOE_ERR_UNSUPPORTED
    assert loss(nbytes=4) == L.MOE_ERR_WORKSPACE
    assert grad(T=0) == L.MOE_OK
    assert grad(T=-1) == bad and grad(k=9) == bad
    for kw in (dict(logits=None), dict(lse=None), dict(dl=None), dict(ids=None), dict(w=None),
               dict(counts=None), dict(dl=ODD), dict(dw=ODD)):
        assert grad(**kw) == bad, kw
    assert lib.moe_router_loss_workspace_size(4, 1025) == 0
    assert lib.moe_router_loss_workspace_size(1, 8) >= 9 * 4


def adam(L, n=1, h=None, ws=A, ws_bytes=1 << 30, norm=None, **kw):
    base = dict(param=1 << 20, master=None, grad=1 << 20, m=1 << 20, v=1 << 20, scales=None,
                n=100, param_type=1, grad_type=0, state_bits=32, lr_mult=1.0, weight_decay=0.0)
    base.update(kw)
    arr = (L.MoeAdamWTensor * 1)(L.MoeAdamWTensor(**base))
    hyper = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, grad_scale=1.0, max_norm=0.0,
                 skip_nonfinite=0)
    hyper.update(h or {})
    return L.load().moe_adamw_step(arr, n, ctypes.byref(L.MoeAdamWHyper(**hyper)), norm, ws,
                                   ws_bytes, None)


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(param=None), dict(grad=None), dict(m=None), dict(v=None),
    dict(scales=1 << 20), dict(state_bits=8), dict(state_bits=16), dict(param_type=3),
    dict(grad_type=2), dict(param_type=0, master=1 << 20), dict(param=(1 << 20) + 1),
    dict(m=(1 << 20) + 2), dict(lr_mult=-1.0), dict(weight_decay=float("nan")),
    dict(weight_decay=-0.1)])
def test_adamw_tensors(L, kw):
    kw = dict(kw)
    if kw.get("n") == -1:
        arr = (L.MoeAdamWTensor * 1)(L.MoeAdamWTensor(n=-1, state_bits=32))
        h = L.MoeAdamWHyper(1e-3, .9, .999, 1e-8, 1, 1.0, 0.0, 0)
        assert L.load().moe_adamw_step(arr, 1, ctypes.byref(h), None, None, 0, None) == \
            L.MOE_ERR_INVALID_ARG
        return
    assert adam(L, **kw) == L.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("h", [
    dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0),
    dict(step=0), dict(max_norm=-1.0), dict(max_norm=float("inf")), dict(grad_scale=float("nan")),
    dict(skip_nonfinite=2)])
def test_adamw_settings(L, h):
    assert adam(L, h=h) == L.MOE_ERR_INVALID_ARG


def test_adamw_workspace_and_counts(L):
    lib = L.load()
    assert adam(L, h=dict(max_norm=1.0), ws=None) == L.MOE_ERR_INVALID_ARG
    assert adam(L, h=dict(skip_nonfinite=1), ws_bytes=8) == L.MOE_ERR_WORKSPACE
    assert adam(L, n=-1) == L.MOE_ERR_INVALID_ARG
    h = L.MoeAdamWHyper(1e-3, .9, .999, 1e-8, 1, 1.0, 0.0, 0)
    assert lib.moe_adamw_step(None, 0, ctypes.byref(h), None, None, 0, None) == L.MOE_OK
    assert lib.moe_adamw_step(None, 2, ctypes.byref(h), None, None, 0, None) == \
        L.MOE_ERR_INVALID_ARG
    assert lib.moe_adamw_workspace_size(None, 3) == 0


def test_ring_selftest_arguments(L):
    f, bad = L.load().moe_selftest_ring_timeout, L.MOE_ERR_INVALID_ARG
    assert f(0, 0, A, None) == bad and f(2000001, 0, A, None) == bad
    assert f(1000, 2, A, None) == bad and f(1000, -2, A, None) == bad
    assert f(1000, 0, None, None) == bad and f(1000, 0, ODD, None) == bad


@pytest.mark.parametrize("bits", [16, 0, 4])
def test_state_bits_of_a_parameter(L, bits):
    """Refused before anything is made of them (the tensors' device is checked later)."""
    import torch
    from expert_routing_grouped_moe_gb300 import MoEAdamW
    with pytest.raises(ValueError, match="state_bits"):
        MoEAdamW([dict(param=torch.zeros(10), state_bits=bits)], [torch.zeros(10)])


def test_more_rows_than_the_c_interface_counts(L):
    """ctypes drops the upper bits of an int32: 2^32 + 2 rows would pass as 2."""
    import torch
    T = 2 ** 32 + 2
    x = torch.empty(T, 1, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="2\\^31"):
        L.moe_block_norm_fwd(x, None, None, x)
    with pytest.raises(ValueError, match="2\\^31"):
        L.moe_block_norm_bwd(x, x, x, None, x)
    l = torch.empty(T, 1, device="meta")
    with pytest.raises(ValueError, match="2\\^31"):
        L.moe_router_loss_fwd(l, None, 1, None, None, None, None)
    with pytest.raises(ValueError, match="2\\^31"):
        L.moe_router_bwd(l, None, None, None, None, None, l, k=1)
