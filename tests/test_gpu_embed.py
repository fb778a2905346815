"""Embedding lookup and its gradient on the GPU against the 64-bit oracle.

Tolerances, before any run, with u = 2^-24 and r half a step of the output's
type: out is the product scale * value rounded to fp32 and to the type,
(u + r) |out|.  dtable is an fp32 sum of n rows in some order, a product with
the scale and at most one more sum: (n + 4) u times the sum of the terms'
sizes, and r |dtable|."""
import numpy as np
import pytest
import torch

from expert_routing_grouped_moe_gb300 import _lib as L
from oracle import token_oracle as to
from _tokens import BF, DEV, F32, HALF, U, gen, graph_of, np64, place

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routing_grouped_moe_gb300 import build
    build.build()
    L.load()


def workspace(T, V, d):
    return torch.empty(max(16, L.moe_embed_workspace_size(T, V, d)), dtype=torch.uint8, device=DEV)


def close(got, ref, tol):
    err = np.abs(np64(got) - ref)
    assert (err <= tol).all(), (float((err - tol).max()), float(err.max()))


@pytest.mark.parametrize("T,V,d,table,out,ids,scale,off", [
    (1, 10, 64, BF, BF, torch.int64, 1.0, 0), (1, 1, 1, F32, F32, torch.int32, -2.0, 0),
    (5, 7, 7, BF, F32, torch.int64, 3.7, 0), (513, 100, 520, F32, BF, torch.int32, 0.3, 0),
    (33, 50, 1001, BF, BF, torch.int64, 31.6, 0), (40, 50, 2880, BF, F32, torch.int32, 53.66, 0),
    (40, 50, 2048, F32, F32, torch.int64, 1.0, 1), (17, 9, 8200, BF, BF, torch.int32, 1.0, 3)])
def test_lookup(T, V, d, table, out, ids, scale, off):
    g = gen(T + d)
    w, _ = place((V, d), table, off, torch.randn(V, d, generator=g, device=DEV))
    i = torch.randint(0, V, (T,), generator=g, device=DEV).to(ids)
    o, untouched = place((T, d), out, off)
    L.moe_embed_fwd(i, w, o, scale=scale)
    s = float(np.float32(scale))
    ref = to.embed(i.cpu().numpy(), np64(w), s)
    close(o, ref, (U + HALF[out]) * np.abs(ref))
    assert untouched() and L.moe_status() == L.MOE_OK


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
def test_lookup_of_bad_ids_gives_zeros_and_the_status(ids):
    w = torch.randn(6, 40, device=DEV)
    i = torch.tensor([[0, -1, 5], [6, 3, 2 ** 31 - 1]], device=DEV).to(ids)
    o = torch.full((2, 3, 40), 9.0, device=DEV)
    L.moe_embed_fwd(i, w, o)
    assert L.moe_status() == L.MOE_ERR_BAD_IDS and L.moe_status() == L.MOE_OK
    assert torch.equal(o[0, 0], w[0]) and torch.equal(o[0, 2], w[5]) and torch.equal(o[1, 1], w[3])
    assert not o[0, 1].any() and not o[1, 0].any() and not o[1, 2].any()


def test_lookup_of_ids_past_32_bits():
    w = torch.randn(6, 40, device=DEV)
    o = torch.empty(2, 40, device=DEV)
    L.moe_embed_fwd(torch.tensor([2 ** 32 + 1, 1], device=DEV), w, o)
    assert L.moe_status() == L.MOE_ERR_BAD_IDS
    assert not o[0].any() and torch.equal(o[1], w[1])


def some_ids(kind, T, V, g):
    if kind == "one":
        return torch.full((T,), V // 2, device=DEV)
    if kind == "each":
        return torch.randperm(V, generator=g, device=DEV).repeat(-(-T // V))[:T]
    if kind == "runs":      # runs of 1, 2, ... tokens: every position against the chunks
        r = torch.repeat_interleave(torch.arange(V), torch.arange(V) % 90 + 1)[:T]
        r = torch.nn.functional.pad(r, (0, T - r.numel()), value=V - 1)
        return r.to(DEV)[torch.randperm(T, generator=g, device=DEV)]
    u = torch.rand(T, generator=g, device=DEV, dtype=torch.float64)
    return (torch.exp(u * np.log(V + 1)) - 1).long().clamp(0, V - 1)


CASES = [
    (1, 1, 1, BF, BF, "one", 1.0, False, 0), (1, 50, 2048, BF, F32, "zipf", 1.0, False, 0),
    (7, 5, 7, F32, F32, "zipf", -0.5, True, 0), (9, 300, 64, BF, F32, "one", 2.0, False, 0),
    (257, 511, 128, BF, F32, "zipf", 1.0, False, 0), (257, 512, 128, F32, BF, "each", 1.0, True, 0),
    (1037, 700, 1001, BF, BF, "zipf", 0.37, False, 0), (1037, 700, 1001, BF, F32, "runs", 0.37, True, 1),
    (3000, 90, 40, BF, F32, "runs", 1.0, False, 0), (3000, 90, 2880, BF, F32, "runs", 1.0, True, 0),
    (4100, 40, 72, F32, F32, "one", 1.0, False, 0), (8192, 1000, 16, BF, F32, "runs", 1.0, False, 0),
    (8193, 262143, 8, BF, BF, "zipf", 1.0, False, 0), (9001, 262144, 8, BF, F32, "zipf", 3.0, True, 0),
    (33000, 300, 24, F32, F32, "zipf", 1.0, False, 0), (70001, 3000, 8, BF, F32, "runs", 1.0, False, 0),
    (135000, 70000, 9, BF, F32, "zipf", 1.0, True, 0), (66000, 5, 8, BF, F32, "one", 1.0, False, 0)]


@pytest.mark.parametrize("T,V,d,rows,table,kind,scale,add,off", CASES)
def test_gradient(T, V, d, rows, table, kind, scale, add, off):
    g = gen(T + V + d)
    ids = some_ids(kind, T, V, g).to(torch.int64 if T % 2 else torch.int32)
    dout, _ = place((T, d), rows, off, torch.randn(T, d, generator=g, device=DEV))
    base = torch.randn(V, d, generator=g, device=DEV).to(table)
    dw, untouched = place((V, d), table, off, base if add else None)
    ws = workspace(T, V, d)
    ws.fill_(0xCC)
    L.moe_embed_bwd(ids, dout, dw, ws, scale=scale, accumulate=add)
    s = float(np.float32(scale))
    ref, mag, n = to.embed_grad(ids.cpu().numpy(), np64(dout), V, s, base=np64(base) if add else None)
    close(dw, ref, (n[:, None] + 4) * U * mag + HALF[table] * np.abs(ref))
    empty = n == 0
    if add:     # rows without a token keep their bits
        assert np.array_equal(np64(dw)[empty], np64(base)[empty])
    else:
        assert not np64(dw)[empty].any()
    assert untouched() and L.moe_status() == L.MOE_OK
    again = (base if add else torch.empty_like(base)).clone()
    L.moe_embed_bwd(ids, dout, again, ws, scale=scale, accumulate=add)
    assert torch.equal(again, dw)


@pytest.mark.parametrize("T", [40, 9000])
@pytest.mark.parametrize("table", [BF, F32])
@pytest.mark.parametrize("d", [1, 2, 3, 4, 5, 6, 7, 8, 9, 17])
def test_dense_gradient_of_narrow_tables(d, table, T):
    """Rows of which several fit a 16-byte word, from every place within one, over garbage: rows
    with and without a token in turn, alone and in pairs; a small batch (rows without a token
    are found one by one) and a larger one (all are zeroed ahead of the sums)."""
    g = gen(100 * d + T)
    V = 301
    rows = torch.arange(V, device=DEV)
    some = torch.cat([rows[:100:2], rows[100:200:4], rows[101:200:4], rows[200::7], rows[-1:]])
    ids = some[torch.randint(0, some.numel(), (T,), generator=g, device=DEV)]
    ids[:some.numel()] = some[:T]
    dout = torch.randn(T, d, generator=g, device=DEV)
    ref, mag, n = to.embed_grad(ids.cpu().numpy(), np64(dout), V)
    ws = workspace(T, V, d)
    for off in range(16 // (2 if table == BF else 4)):
        dw, untouched = place((V, d), table, off)
        dw.fill_(float("nan"))
        L.moe_embed_bwd(ids, dout, dw, ws)
        close(dw, ref, (n[:, None] + 4) * U * mag + HALF[table] * np.abs(ref))
        assert not np64(dw)[n == 0].any() and untouched(), off
    assert L.moe_status() == L.MOE_OK


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("add", [False, True])
def test_gradient_with_padding_and_bad_ids(ids, add):
    g = gen(3)
    T, V, d = 700, 40, 48
    i = torch.randint(0, V, (T,), generator=g, device=DEV)
    i[::5] = 7
    dout = torch.randn(T, d, generator=g, device=DEV)
    base = torch.randn(V, d, generator=g, device=DEV)
    ws = workspace(T, V, d)
    for bad in (False, True):
        if bad:
            i[3], i[100], i[699] = -1, V, 2 ** 31 - 1
        dw = base.clone()
        L.moe_embed_bwd(i.to(ids), dout, dw, ws, pad_id=7, accumulate=add)
        assert L.moe_status() == (L.MOE_ERR_BAD_IDS if bad else L.MOE_OK)
        ref, mag, n = to.embed_grad(i.cpu().numpy(), np64(dout), V, pad=7, base=np64(base) if add else None)
        close(dw, ref, (n[:, None] + 4) * U * mag + U * np.abs(ref))
        assert torch.equal(dw[7], base[7] if add else torch.zeros_like(base[7]))
    # a padding id that is no row of the table is no error
    i = i.clamp(0, V - 1)
    i[5] = V + 3
    L.moe_embed_bwd(i.to(ids), dout, dw, ws, pad_id=V + 3)
    assert L.moe_status() == L.MOE_OK


def test_padding_ids_past_64_bits_are_refused():
    ids, dout = torch.full((100,), 4, device=DEV), torch.randn(100, 24, device=DEV)
    dw, ws = torch.full((9, 24), 5.0, device=DEV), workspace(100, 9, 24)
    for bad in (2 ** 63, 2 ** 64 + 4):
        with pytest.raises(ValueError):
            L.moe_embed_bwd(ids, dout, dw, ws, pad_id=bad)
    assert (dw == 5.0).all()


def test_nothing_but_padding():
    dw = torch.full((9, 24), 5.0, device=DEV)
    ids, dout = torch.full((100,), 4, device=DEV), torch.randn(100, 24, device=DEV)
    L.moe_embed_bwd(ids, dout, dw, workspace(100, 9, 24), pad_id=4, accumulate=True)
    assert (dw == 5.0).all()
    L.moe_embed_bwd(ids, dout, dw, workspace(100, 9, 24), pad_id=4)
    assert not dw.any()


def test_no_tokens():
    ids, rows = torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, 24, device=DEV)
    dw, untouched = place((9, 24), F32, 1, torch.full((9, 24), 5.0))
    L.moe_embed_bwd(ids, rows, dw, None, accumulate=True)
    assert (dw == 5.0).all()
    L.moe_embed_bwd(ids, rows, dw, None)
    assert not dw.any() and untouched()
    L.moe_embed_fwd(ids, torch.randn(9, 24, device=DEV), rows)


def test_gradients_that_are_not_finite_stay_in_their_rows():
    ids = torch.arange(600, device=DEV) % 60
    dout = torch.ones(600, 32, device=DEV)
    dout[5, 3], dout[77, 0] = float("nan"), float("inf")
    dw = torch.empty(60, 32, device=DEV)
    L.moe_embed_bwd(ids, dout, dw, workspace(600, 60, 32))
    bad = torch.zeros(60, 32, dtype=torch.bool, device=DEV)
    bad[5, 3] = bad[17, 0] = True
    assert torch.equal(~torch.isfinite(dw), bad) and (dw[~bad] == 10).all()


def test_tables_past_2_to_31_values():
    V, d = 1_100_000, 2048
    w = torch.zeros(V, d, dtype=BF, device=DEV)
    ids = torch.tensor([0, V - 1, V - 2, 1_048_576, V - 1], device=DEV)
    w[ids] = torch.randn(5, d, device=DEV).to(BF)
    o = torch.empty(5, d, dtype=BF, device=DEV)
    L.moe_embed_fwd(ids, w, o)
    assert torch.equal(o, w[ids])
    keep = w[ids].float()
    dout = torch.randn(5, d, device=DEV)
    L.moe_embed_bwd(ids, dout, w, workspace(5, V, d), accumulate=True)
    two = dout[1] + dout[4]
    assert torch.equal(w[V - 1], (keep[1] + two).to(BF))
    assert torch.equal(w[1_048_576], (keep[3] + dout[3]).to(BF))
    assert not w[V // 2:1_048_576].any()
    L.moe_embed_bwd(ids, dout, w, workspace(5, V, d))
    assert torch.equal(w[V - 1], two.to(BF)) and not w[1:1_048_576].any() and not w[1_048_577:V - 2].any()


def test_streams_and_graphs():
    """Another stream; a captured call replayed on new data; two graphs with one workspace."""
    g = gen(9)
    T, V, d = 900, 333, 200
    ids = torch.randint(0, V, (T,), generator=g, device=DEV)
    dout = torch.randn(T, d, generator=g, device=DEV)
    want = torch.empty(V, d, device=DEV)
    ws = workspace(T, V, d)
    L.moe_embed_bwd(ids, dout, want, ws)
    a, b = torch.empty_like(want), torch.empty_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    L.moe_embed_bwd(ids, dout, a, ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, want)
    other = torch.randint(0, V, (T,), generator=g, device=DEV)
    one = graph_of(lambda: L.moe_embed_bwd(ids, dout, a, ws))
    two = graph_of(lambda: L.moe_embed_bwd(other, dout, b, ws))
    wb = torch.empty_like(want)
    L.moe_embed_bwd(other, dout, wb, ws)
    for _ in range(3):
        a.fill_(3), b.fill_(4)
        one.replay(), two.replay()
        assert torch.equal(a, want) and torch.equal(b, wb)
    ids.copy_(other)
    one.replay()
    assert torch.equal(a, wb)
