"""8-bit checkpoints on the GPU against the 64-bit oracle.

Codes, scales and restored values are exact.  act, before any run: __expf is
off by 2 + 1.173 |g| steps of 2^-23, the quotient and its denominator by 3, the
two products by 1 each: (8 + 1.2 |g|) 2^-23, and the pair rounds twice by 2^-8:
2^-16 (values below 2^-120 aside)."""
import numpy as np
import pytest
import torch

from expert_routing_grouped_moe_gb300 import _lib as L
from oracle import token_oracle as to
from _tokens import BF, DEV, F32, gen, graph_of, np64, place

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routing_grouped_moe_gb300 import build
    build.build()
    L.load()


def make(R, C, dtype, off, g):
    x = torch.randn(R, C, generator=g, device=DEV) * torch.exp(6 * torch.randn(R, 1, generator=g, device=DEV))
    if R > 3:
        x[0] = 0
        x[1] = 127.0
        x[2] = 127.00001 if dtype == F32 else 128.0
        x[3, ::3] = 63.5       # ties: 63.5 / 0.5 is whole, 0.25 / 0.5 is not
        x[3, 1::3] = 0.25
    if R > 7:
        x[4, C // 2], x[5, 0], x[6, C - 1] = float("nan"), float("inf"), -float("inf")
        x[7] *= 1e-42
    return place((R, C), dtype, off, x)[0]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,C,off", [(1, 1, 0), (3, 31, 0), (9, 32, 0), (9, 33, 0), (64, 64, 0), (9, 40, 0),
                                     (9, 1001, 0), (700, 96, 1), (50, 2880, 0), (50, 2880, 4), (301, 264, 0),
                                     (20000, 8, 0), (9, 5000, 3)])
def test_pack_and_unpack(dtype, R, C, off):
    g = gen(R + C)
    x = make(R, C, dtype, off, g)
    codes, c_ok = place((R, C), torch.int8, off)
    scales, s_ok = place((R, -(-C // 32)), torch.uint8, off)
    L.moe_ckpt_pack(x, codes, scales)
    rc, rs = to.ckpt_pack(x.float().cpu().numpy())
    assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scales.cpu().numpy(), rs)
    assert c_ok() and s_ok()
    for out in (BF, F32):
        y, y_ok = place((R, C), out, off)
        L.moe_ckpt_unpack(codes, scales, y)
        assert np.array_equal(np64(y), to.ckpt_value(rc, rs), equal_nan=True) and y_ok()


def test_every_code_and_scale():
    """All codes under every exponent byte; beyond the type's range, infinities."""
    bytes_ = torch.arange(1, 250, dtype=torch.uint8, device=DEV)
    codes = torch.arange(-128, 128, device=DEV).to(torch.int8).repeat(249, 1)
    scales = bytes_[:, None].repeat(1, 8).contiguous()
    for out in (BF, F32):
        y = torch.empty(249, 256, dtype=out, device=DEV)
        L.moe_ckpt_unpack(codes, scales, y)
        with np.errstate(over="ignore"):
            want = to.ckpt_value(codes.cpu().numpy(), scales.cpu().numpy()).astype(np.float32)
        assert np.array_equal(np64(y), want)


@pytest.mark.parametrize("C", [256, 250])
def test_the_outermost_scale_bytes(C):
    """Byte 0 is 2^-127, byte 255 is NaN whatever the codes are."""
    codes = torch.arange(-128, 128, device=DEV).to(torch.int8)[:C].repeat(2, 1)
    scales = torch.tensor([0, 255], dtype=torch.uint8, device=DEV)[:, None].repeat(1, 8).contiguous()
    for out in (BF, F32):
        y = torch.empty(2, C, dtype=out, device=DEV)
        L.moe_ckpt_unpack(codes, scales, y)
        assert np.array_equal(np64(y), to.ckpt_value(codes.cpu().numpy(), scales.cpu().numpy()), equal_nan=True)


def test_the_outermost_scale_bytes_of_a_layer():
    codes = torch.full((2, 32), 3, dtype=torch.int8, device=DEV)
    scales = torch.tensor([[0], [255]], dtype=torch.uint8, device=DEV)
    h, act = torch.empty(2, 32, device=DEV), torch.empty(2, 2, 16, dtype=BF, device=DEV)
    L.moe_ckpt_unpack_swiglu(codes, scales, torch.arange(2, dtype=torch.int32, device=DEV),
                             torch.ones(2, 1, device=DEV), False, h, act)
    assert (h[0] == 3 * 2.0 ** -127).all() and torch.isnan(h[1]).all() and torch.isnan(act[0, 1]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("C", [64, 33])
def test_the_largest_values_stay_finite(C, dtype):
    top = torch.finfo(dtype).max
    x = torch.ones(5, C, dtype=dtype, device=DEV)
    x[0, 3], x[1, 32], x[2] = top, -top, -top
    x[3, 0] = 127 * 2.0 ** 121
    x[4, 1] = 126.5 * 2.0 ** 121
    codes = torch.empty(5, C, dtype=torch.int8, device=DEV)
    scales = torch.empty(5, -(-C // 32), dtype=torch.uint8, device=DEV)
    L.moe_ckpt_pack(x, codes, scales)
    rc, rs = to.ckpt_pack(x.float().cpu().numpy())
    assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scales.cpu().numpy(), rs)
    y = torch.empty_like(x)
    L.moe_ckpt_unpack(codes, scales, y)
    assert torch.isfinite(y).all()
    assert (np.abs(np64(y) - np64(x)) <= np.abs(np64(x)).max(1, keepdims=True) / 127).all()


@pytest.mark.parametrize("T,k,f,shared", [(1, 1, 8, False), (5, 2, 64, False), (33, 4, 1000, True),
                                          (130, 8, 768, False), (7, 3, 24, True), (3, 32, 40, True)])
def test_unpack_swiglu(T, k, f, shared):
    g = gen(T + f)
    K = k + shared
    P, hs = T * K, 32 * ((f + 15) // 16)
    h0 = 3 * torch.randn(P, hs, generator=g, device=DEV)
    codes = torch.empty(P, hs, dtype=torch.int8, device=DEV)
    scales = torch.empty(P, hs // 32, dtype=torch.uint8, device=DEV)
    L.moe_ckpt_pack(h0, codes, scales)
    order = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    gone = torch.rand(P, generator=g, device=DEV) < 0.1
    order[gone] = torch.tensor([-1, P, 2 ** 31 - 1], dtype=torch.int32, device=DEV)[
        torch.arange(int(gone.sum()), device=DEV) % 3]
    w = torch.rand(T, k, generator=g, device=DEV) + 0.01
    h, h_ok = place((P, hs), F32)
    act, a_ok = place((2, P, f), BF)
    h.fill_(5), act.fill_(6)
    L.moe_ckpt_unpack_swiglu(codes, scales, order, w, shared, h, act)
    assert h_ok() and a_ok()
    value = to.ckpt_value(codes.cpu().numpy(), scales.cpu().numpy())
    live = ~gone.cpu().numpy()
    assert np.array_equal(np64(h)[live], value[live])
    assert (h[gone] == 5).all() and (act[:, gone] == 6).all()       # left as they were
    src = np.where(live, order.cpu().numpy(), 0)
    t, j = src // K, src % K
    full = np.concatenate([np64(w), np.ones((T, 1))], 1)
    ref, gate = to.swiglu_from(value, f, full[t, j])
    got = np64(act[0]) + np64(act[1])
    tol = np.abs(ref) * (2.0 ** -16 + (8 + 1.2 * np.abs(gate)) * 2.0 ** -23) + 2.0 ** -120
    assert (np.abs(got - ref)[live] <= tol[live]).all()


def test_blocks_that_were_not_finite_spoil_their_features_only():
    f, P = 32, 4
    h0 = torch.ones(P, 64, device=DEV)
    h0[2, 40] = float("nan")            # chunk 1 of row 2: features 16 .. 31
    codes = torch.empty(P, 64, dtype=torch.int8, device=DEV)
    scales = torch.empty(P, 2, dtype=torch.uint8, device=DEV)
    L.moe_ckpt_pack(h0, codes, scales)
    h, act = torch.empty(P, 64, device=DEV), torch.empty(2, P, f, dtype=BF, device=DEV)
    order = torch.arange(P, dtype=torch.int32, device=DEV)
    L.moe_ckpt_unpack_swiglu(codes, scales, order, torch.ones(P, 1, device=DEV), False, h, act)
    bad = torch.zeros(P, f, dtype=torch.bool, device=DEV)
    bad[2, 16:] = True
    assert torch.equal(torch.isnan(act[0]), bad)
    spoilt = torch.zeros(P, 64, dtype=torch.bool, device=DEV)
    spoilt[2, 32:] = True               # the whole chunk, gates and ups
    assert torch.equal(torch.isnan(h), spoilt)


def test_no_rows():
    x, c = torch.empty(0, 40, device=DEV), torch.empty(0, 40, dtype=torch.int8, device=DEV)
    s = torch.empty(0, 2, dtype=torch.uint8, device=DEV)
    L.moe_ckpt_pack(x, c, s)
    L.moe_ckpt_unpack(c, s, x)
    L.moe_ckpt_unpack_swiglu(torch.empty(0, 64, dtype=torch.int8, device=DEV), s,
                             torch.empty(0, dtype=torch.int32, device=DEV), torch.empty(0, 2, device=DEV),
                             False, torch.empty(0, 64, device=DEV), torch.empty(2, 0, 32, dtype=BF, device=DEV))


def test_more_than_2_to_31_values():
    R, C = 1_100_000, 2048
    x = torch.zeros(R, C, dtype=BF, device=DEV)
    x[-1] = torch.randn(C, device=DEV).to(BF)
    codes = torch.empty(R, C, dtype=torch.int8, device=DEV)
    scales = torch.empty(R, C // 32, dtype=torch.uint8, device=DEV)
    L.moe_ckpt_pack(x, codes, scales)
    rc, rs = to.ckpt_pack(x[-2:].float().cpu().numpy())
    assert np.array_equal(codes[-2:].cpu().numpy(), rc) and np.array_equal(scales[-2:].cpu().numpy(), rs)
    assert not codes[:-1].any() and (scales[:-1] == 1).all()
    x.fill_(1)
    L.moe_ckpt_unpack(codes, scales, x)
    assert np.array_equal(np64(x[-2:]), to.ckpt_value(rc, rs)) and not x[:-1].any()


def test_streams_and_graphs():
    g = gen(4)
    x = torch.randn(77, 200, generator=g, device=DEV)
    codes = torch.empty(77, 200, dtype=torch.int8, device=DEV)
    scales = torch.empty(77, 7, dtype=torch.uint8, device=DEV)
    y = torch.empty_like(x)

    def both(stream=None):
        L.moe_ckpt_pack(x, codes, scales, stream=stream)
        L.moe_ckpt_unpack(codes, scales, y, stream=stream)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    both(s)
    torch.cuda.current_stream().wait_stream(s)
    want = to.ckpt_value(*to.ckpt_pack(x.cpu().numpy()))
    assert np.array_equal(np64(y), want)
    graph = graph_of(both)
    x.mul_(-3)
    y.zero_()
    graph.replay()
    assert np.array_equal(np64(y), to.ckpt_value(*to.ckpt_pack(x.cpu().numpy())))
