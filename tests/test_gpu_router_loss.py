"""The router's losses and the gradient of its logits on the GPU against the
64-bit oracle.

Tolerances, before any run, with u = 2^-24: exp of an argument a <= 0 in fp32
is off by (2 + |a|) u or so (the product with log2 e rounds at |a| u), so with
logits within about 16 of the maximum P is good to 32 u of itself, sums over E
terms add (32 + 5) u at most and sums over tokens their depth: 256 u of the sum
of the sizes of the terms covers dlogits and lse, 1024 u pmean and the losses.
A term whose P is below 2^-40 is covered by an absolute 2^-60."""
import numpy as np
import pytest
import torch

from expert_routing_grouped_moe_gb300 import _lib as L, synth
from oracle import block_oracle as bo
from _util import to64

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routing_grouped_moe_gb300 import build
    build.build()
    L.load()


def make(T, E, k, seed=0, blocked=0, skew=0.0, off=0):
    """off: begin every [T,E] buffer that many values past an aligned address."""
    g = torch.Generator(DEV).manual_seed(seed * 31 + T * 7 + E)

    def place(*shape, dtype=torch.float32):
        n = int(np.prod(shape))
        return torch.empty(n + off, dtype=dtype, device=DEV)[off:].view(*shape)
    logits = place(T, E)
    logits.copy_(torch.randn(T, E, generator=g, device=DEV) * 2)
    logits += skew * torch.arange(E, device=DEV)
    if blocked:
        logits[:, -blocked:] = -float("inf")
    ids = torch.empty(T, k, dtype=torch.int32, device=DEV)
    w = torch.empty(T, k, device=DEV)
    L.moe_router_topk(logits, k, ids, w) if off == 0 else None
    if off:
        v, i = torch.topk(logits, k, dim=1)
        ids.copy_(i)
        w.copy_(torch.softmax(v, 1))
    return {"logits": logits, "ids": ids, "w": w, "k": k,
            "counts": torch.bincount(ids.reshape(-1).long(), minlength=E).to(torch.int32),
            "dw": torch.randn(T, k, generator=g, device=DEV),
            "losses": torch.empty(2, device=DEV), "lse": torch.empty(T, device=DEV),
            "pmean": torch.empty(E, device=DEV), "dlogits": place(T, E),
            "ws": torch.empty(max(16, L.moe_router_loss_workspace_size(T, E)), dtype=torch.uint8,
                              device=DEV)}


def run(b, aux=0.3, z=0.2, dw=True, stream=None):
    L.moe_router_loss_fwd(b["logits"], b["counts"], b["k"], b["losses"], b["lse"], b["pmean"],
                          b["ws"], stream=stream)
    L.moe_router_bwd(b["logits"], b["lse"], b["counts"], b["ids"], b["w"],
                     b["dw"] if dw else None, b["dlogits"], aux_coef=aux, z_coef=z, stream=stream)


def check(b, aux=0.3, z=0.2, dw=True):
    l, c = to64(b["logits"]), b["counts"].cpu().numpy()
    aux, z = float(np.float32(aux)), float(np.float32(z))
    losses, lse, pm = bo.router_losses(l, c, b["k"])
    fin = np.isfinite(lse)
    np.testing.assert_array_equal(np.isneginf(to64(b["lse"])), ~fin)
    # |lse| near 0 comes from m + log s of opposite signs: sizes at most |m| + log E
    size = np.abs(l.max(1)) + np.log(l.shape[1]) + 1
    assert np.all(np.abs(to64(b["lse"])[fin] - lse[fin]) <= 256 * U * size[fin])
    assert np.all(np.abs(to64(b["pmean"]) - pm) <= 1024 * U * pm + 2.0 ** -60)
    zsize = np.mean(np.where(fin, size, 0) ** 2)
    assert abs(to64(b["losses"])[0] - losses[0]) <= 1024 * U * losses[0]
    assert abs(to64(b["losses"])[1] - losses[1]) <= 1024 * U * zsize
    d, mag = bo.router_backward(l, c, b["ids"].cpu().numpy(), to64(b["w"]),
                                to64(b["dw"]) if dw else None, aux, z, b["k"])
    err = np.abs(to64(b["dlogits"]) - d)
    # lse's error scales every P of its row
    bound = 256 * U * mag * (1 + np.where(fin, size, 0)[:, None] / 8) + 2.0 ** -60
    assert np.all(err <= bound), float(np.max(err / bound))


CASES = [(1, 1, 1), (1, 4, 2), (3, 2, 1), (5, 7, 3), (33, 8, 8), (100, 13, 4), (64, 16, 2),
         (257, 32, 4), (1000, 60, 4), (31, 64, 8), (4096, 128, 8), (77, 129, 8), (50, 256, 8),
         (40, 300, 16), (9, 509, 32), (20, 512, 6), (11, 1000, 8), (7, 1023, 5), (6, 1024, 32)]


@pytest.mark.parametrize("T,E,k", CASES)
def test_losses_and_gradient(T, E, k):
    b = make(T, E, k, blocked=E // 16, skew=0.02)
    run(b)
    check(b)
    run(b, dw=False)
    check(b, dw=False)
    run(b, aux=0.0, z=0.0)
    check(b, aux=0.0, z=0.0)
    assert L.moe_status() == L.MOE_OK


@pytest.mark.parametrize("E", [8, 60, 128, 512])
def test_pointers_that_no_vector_fits(E):
    b = make(70, E, 4, off=1)
    run(b)
    check(b)


@pytest.mark.parametrize("T,E,k,off", [
    (160_000, 5, 2, 0), (330_000, 8, 2, 0), (160_001, 13, 2, 0), (160_000, 16, 2, 0),
    (160_003, 19, 2, 0), (160_000, 30, 2, 0), (90_000, 32, 2, 0), (160_000, 32, 2, 1),
    (80_001, 60, 2, 0), (80_000, 61, 2, 0), (80_000, 64, 2, 1), (40_000, 100, 2, 0),
    (20_003, 130, 2, 0), (11_000, 260, 2, 0), (10_001, 515, 2, 0)])
def test_two_launches_and_two_turns_of_rows(T, E, k, off):
    """Every layout of a row, by vectors and by single logits, with more rows than the
    blocks take at once (608 blocks of 8 warps, 1 to 32 rows a warp), the last turn not
    full: the losses' two launches and the gradient."""
    b = make(T, E, k, off=off, skew=0.02)
    run(b)
    check(b)
    assert L.moe_status() == L.MOE_OK


@pytest.mark.parametrize("E", [17, 19, 29, 30, 31, 32])
@pytest.mark.parametrize("off", [0, 1])
def test_rows_of_17_to_32_experts(E, off):
    for T in (1, 7, 64, 1000):
        b = make(T, E, 4, blocked=E // 16, off=off)
        run(b)
        check(b)


def test_the_skewed_workload():
    cfg = synth.scaled(synth.CONFIGS["skewed_shared"], T=3000)
    act = synth.layer_activations(cfg, 1, device=DEV)
    b = make(cfg.T, cfg.E, cfg.k)
    b["logits"].copy_(act["logits"])
    L.moe_router_topk(b["logits"], cfg.k, b["ids"], b["w"])
    b["counts"] = torch.bincount(b["ids"].reshape(-1).long(), minlength=cfg.E + 1).to(torch.int32)
    run(b)
    check(b)


@pytest.mark.parametrize("E", [7, 8, 128, 300])
def test_rows_without_an_expert_and_lowest_values(E):
    b = make(20, E, 2)
    b["logits"][3] = -float("inf")
    b["logits"][19] = -float("inf")
    b["logits"][5] = torch.finfo(torch.float32).min      # finite: an even row
    b["logits"][6, 1:] = torch.finfo(torch.float32).min
    b["w"][3] = float("nan")                             # a softmax of nothing
    l = b["logits"].clone()
    run(b)
    assert torch.all(b["dlogits"][3] == 0) and torch.all(b["dlogits"][19] == 0)
    # the lowest value squared overflows the z loss: its rows out of the check
    assert torch.isneginf(b["lse"][3]) and torch.isfinite(b["lse"][5])
    b["logits"] = l.clone()
    b["logits"][5] = 0.0
    b["w"][5] = 0.5
    run(b)
    check(b)


def check_gradient(b, aux, z):
    """dlogits to 256 u of its terms whatever lse is.  Before any run: exp of an
    argument down to -45 is off by (2 + 1.2 * 45) 2 u, its subtraction by 45 u, the
    row's sum and the products by some 20 u: below 192 u of a P; the z term reads lse,
    4 u of |max| + log E off."""
    l, c = to64(b["logits"]), b["counts"].cpu().numpy()
    aux, z = float(np.float32(aux)), float(np.float32(z))
    d, mag = bo.router_backward(l, c, b["ids"].cpu().numpy(), to64(b["w"]), to64(b["dw"]), aux, z,
                                b["k"])
    size = np.abs(l.max(1, keepdims=True)) + np.log(l.shape[1])
    e = np.exp(l - l.max(1, keepdims=True))
    P = e / e.sum(1, keepdims=True)
    bound = 256 * U * mag + 4 * U * size * P * 2 * z / l.shape[0] + 2.0 ** -60
    err = np.abs(to64(b["dlogits"]) - d)
    assert np.all(err <= bound), float(np.max(err / bound))


@pytest.mark.parametrize("E", [7, 60, 64, 128, 300])
@pytest.mark.parametrize("mean", [0.0, 30.0, -1000.0, 1e4, 1e6])
def test_gradient_of_logits_that_are_not_centred(mean, E):
    """The rounding of lse, |lse| 2^-24, must not show in the probabilities."""
    b = make(500, E, 4)
    b["logits"].mul_(2.0).add_(mean)
    run(b, aux=0.7, z=0.0)
    check_gradient(b, 0.7, 0.0)
    b["dw"].zero_()                 # the balancing term alone
    run(b, aux=0.7, z=0.2)
    check_gradient(b, 0.7, 0.2)


@pytest.mark.parametrize("E", [7, 8, 128, 300])
def test_gradient_of_rows_of_the_lowest_value(E):
    """A row masked by the lowest value instead of -inf is an even row, 1/E each."""
    b = make(20, E, 2)
    low = torch.finfo(torch.float32).min
    b["logits"][5] = low
    b["logits"][6, 1:] = low
    b["w"][5] = 0.5
    for z in (0.0, 0.2):
        run(b, aux=0.3, z=z)
        check_gradient(b, 0.3, z)


def test_bad_ids_are_left_out_and_reported():
    b = make(16, 8, 2)
    run(b)
    assert L.moe_status() == L.MOE_OK
    b["ids"][4, 1] = 8
    b["ids"][5, 0] = -1
    run(b)
    assert L.moe_status() == L.MOE_ERR_BAD_IDS
    check(b)


def test_an_expert_named_twice_gets_both():
    b = make(16, 40, 3)
    b["ids"][:, 1] = b["ids"][:, 0]
    b["ids"][2] = b["ids"][2, 0]
    run(b)
    check(b)


def test_nan_stays_in_its_row():
    b = make(50, 128, 4)
    run(b)
    ref = b["dlogits"].clone()
    b["logits"][8, 5] = float("nan")
    run(b)
    assert torch.isnan(b["dlogits"][8]).all() and torch.isnan(b["losses"]).all()
    b["losses"].zero_()
    keep = [t for t in range(50) if t != 8]
    assert torch.equal(b["dlogits"][keep], ref[keep])


def test_equal_bits_on_another_stream_and_in_a_graph():
    b = make(20000, 64, 8)
    run(b)
    names = ("losses", "lse", "pmean", "dlogits")
    ref = {k: b[k].clone() for k in names}
    for k in names:
        b[k].zero_()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run(b, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for k in names:
        assert torch.equal(b[k], ref[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(b)
    for k in names:
        b[k].zero_()
    graph.replay()
    for k in names:
        assert torch.equal(b[k], ref[k]), k


def test_gradient_against_differences_of_the_kernel():
    """d/dh of sum(w dw) + aux + z along a random direction, from the kernels'
    own losses: weights by moe_router_topk, fp32 losses of size about 10 read
    to 2^-23 over 2h = 2^-5 gives 4e-5 absolute; curvature h^2 times third
    derivatives of order 1 adds 2.5e-4 of the sizes.  1e-3 of the size covers it."""
    T, E, k, aux, z, h = 64, 16, 4, 2.0, 0.5, 2.0 ** -6
    b = make(T, E, k)
    run(b, aux, z)
    grad, base = b["dlogits"].clone(), b["logits"].clone()
    v = 0.05 * torch.randn_like(base)           # too small to change the top k's order often
    ids = b["ids"].clone()
    vals = []
    for sign in (1, -1):
        b["logits"].copy_(base + sign * h * v)
        L.moe_router_topk(b["logits"], k, b["ids"], b["w"])
        assert torch.equal(b["ids"], ids)
        run(b, aux, z)
        vals.append(float((b["w"].double() * b["dw"].double()).sum()
                          + aux * b["losses"][0].double() + z * b["losses"][1].double()))
    num, ana = (vals[0] - vals[1]) / (2 * h), float((grad.double() * v.double()).sum())
    size = float((grad.double() * v.double()).abs().sum())
    assert abs(num - ana) <= 1e-3 * size + 4e-4, (num, ana, size)


def test_offsets_past_32_bits():
    T, E, k = (1 << 24) + 40, 132, 2
    assert T * E > 2 ** 31
    logits = torch.zeros(T, E, device=DEV)
    logits[-4:] = torch.randn(4, E, device=DEV)
    ids = torch.zeros(T, k, dtype=torch.int32, device=DEV)
    ids[:, 1] = 5
    w = torch.full((T, k), 0.5, device=DEV)
    dw = torch.zeros(T, k, device=DEV)
    dw[-4:] = torch.randn(4, k, device=DEV)
    counts = torch.full((E,), T * k // E, dtype=torch.int32, device=DEV)
    losses, lse, pm = torch.empty(2, device=DEV), torch.empty(T, device=DEV), torch.empty(E, device=DEV)
    ws = torch.empty(L.moe_router_loss_workspace_size(T, E), dtype=torch.uint8, device=DEV)
    L.moe_router_loss_fwd(logits, counts, k, losses, lse, pm, ws)
    dl = torch.empty_like(logits)
    L.moe_router_bwd(logits, lse, counts, ids, w, dw, dl, z_coef=1.0)
    d, mag = bo.router_backward(to64(logits[-4:]), None, ids[-4:].cpu().numpy(), to64(w[-4:]),
                                to64(dw[-4:]), 0.0, 4.0 / T, k)
    assert np.all(np.abs(to64(dl[-4:]) - d) <= 512 * U * mag)
    # near even rows: lse = log E, summed over 2^24 tokens in partial sums
    np.testing.assert_allclose(float(losses[1]), np.log(E) ** 2, rtol=1e-4)
    np.testing.assert_allclose(to64(pm), 1 / E, rtol=1e-4)


def test_refusals_of_tensors():
    b = make(8, 16, 2)
    with pytest.raises(ValueError, match="counts"):
        L.moe_router_loss_fwd(b["logits"], b["counts"][:8], 2, b["losses"], b["lse"], b["pmean"],
                              b["ws"])
    with pytest.raises(L.MoeError, match="workspace"):
        L.moe_router_loss_fwd(b["logits"], b["counts"], 2, b["losses"], b["lse"], b["pmean"],
                              torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(L.MoeError, match="needs ids"):
        L.moe_router_bwd(b["logits"], b["lse"], b["counts"], None, None, b["dw"], b["dlogits"], k=2)
    with pytest.raises(L.MoeError, match="counts"):
        L.moe_router_bwd(b["logits"], b["lse"], None, b["ids"], b["w"], b["dw"], b["dlogits"],
                         aux_coef=1.0)
    with pytest.raises(L.MoeError, match="positive"):
        L.moe_router_loss_fwd(b["logits"][:0], b["counts"], 2, b["losses"], b["lse"][:0],
                              b["pmean"], b["ws"])
