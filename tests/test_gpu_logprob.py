"""Log probabilities, entropy, alternatives and their gradient on the GPU against
the 64-bit oracle.

Tolerances, before any run, with u = 2^-24.  t = (x - M) c has three roundings
(difference, factor, product), so 2^t is off by 3 u |t| ln 2 + 4 u (the exponential);
what counts in S has |t| <= log2 V or so, and a row's sum of V / 512 terms a thread
and a tree adds (V / 512 + 20) u: S is good to s = (80 + V / 512) u.  Then
  logp   s + 2 u (|x - M| + |logp|)          (x, M scaled by inv_temp)
  lse    s + 2 u (|M| + |lse|)
  H      2 s (1 + ln V)                       (ln S, and sum 2^t t / S <= ln V + 1)
  dx     sum of the terms' sizes, each p (...) with p off by s + 8 u + 4 u |ln p|,
         twice that for the coefficients, and half a step of dx's type
Values below 2^-120 may be zeros."""
import numpy as np
import pytest
import torch

from expert_routing_grouped_moe_gb300 import _lib as L
from oracle import token_oracle as to
from _tokens import BF, DEV, F32, HALF, U, gen, graph_of, np64, place

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routing_grouped_moe_gb300 import build
    build.build()
    L.load()


class Case:
    def __init__(self, T, V, dtype, m=1, top=0, off=0, pad=0, seed=0, ids=torch.int64, x=None, inv=1.0,
                 entropy=True, y=None, grads=True):
        g = gen(seed * 977 + T * 31 + V)
        self.T, self.V, self.m, self.top, self.inv = T, V, m, top, inv
        self.guards = []
        if x is None:
            x = 3 * torch.randn(T, V, generator=g, device=DEV) + 5 * torch.randn(T, 1, generator=g, device=DEV)
        whole, _ = place((T, V + pad), dtype, off)
        whole.fill_(float("nan"))          # columns past V count for nothing
        self.logits = whole[:, :V]
        self.logits.copy_(x)
        dwhole, ok = place((T, V + pad), dtype, off)
        dwhole.fill_(11)
        self.dwhole, self.dlogits = dwhole, dwhole[:, :V]
        self.guards.append(ok)
        y = torch.randint(0, V, (T, m), generator=g, device=DEV) if y is None else y
        self.y = y.to(ids)
        self.targets = self.y[:, 0].contiguous() if m == 1 else self.y
        self.dlogp = torch.randn(T, m, generator=g, device=DEV).view(self.targets.shape)
        self.dh = torch.randn(T, generator=g, device=DEV) if grads and entropy else None
        self.dl = torch.randn(T, generator=g, device=DEV) if grads else None
        self.clear(entropy)

    def clear(self, entropy=True):
        def out(*shape, dtype=F32):
            t, ok = place(shape, dtype)
            self.guards.append(ok)
            return t
        T = self.T
        self.logp, self.stats, self.lse = out(*self.targets.shape), out(T, 2), out(T)
        self.entropy = out(T) if entropy else None
        self.top_ids = out(T, self.top, dtype=torch.int32) if self.top else None
        self.top_logp = out(T, self.top) if self.top else None

    def outs(self):
        return dict(lse=self.lse, entropy=self.entropy, top_ids=self.top_ids, top_logp=self.top_logp,
                    inv_temp=self.inv)

    def fwd(self, **kw):
        L.moe_logprob_fwd(self.logits, self.targets, self.logp, self.stats, **self.outs(), **kw)

    def bwd(self, into=None, **kw):
        L.moe_logprob_bwd(self.logits, self.targets, self.stats, self.dlogp,
                          self.dlogits if into is None else into, entropy=self.entropy, dentropy=self.dh,
                          dlse=self.dl, inv_temp=self.inv, **kw)

    def step(self, into=None, **kw):
        L.moe_logprob_step(self.logits, self.targets, self.logp, self.stats, self.dlogp,
                           self.dlogits if into is None else into, dentropy=self.dh, dlse=self.dl,
                           **self.outs(), **kw)

    def ref(self):
        x, y, inv = np64(self.logits), self.y.cpu().numpy(), float(np.float32(self.inv))
        f = lambda t: None if t is None else np64(t)  # noqa: E731
        with np.errstate(invalid="ignore", over="ignore"):
            r = to.logprob(x, y, inv, top=self.top)
            r["dx"], r["mag"] = to.logprob_grad(x, y, inv, dlogp=np64(self.dlogp).reshape(y.shape),
                                                dentropy=f(self.dh), dlse=f(self.dl))
        return r, x, inv

    def check_fwd(self, r=None):
        r, x, inv = r if r is not None else self.ref()
        y = self.y.cpu().numpy()
        s = (80 + self.V / 512) * U
        M = np.maximum(x.max(1), -3.4028234663852886e38)
        with np.errstate(invalid="ignore", over="ignore"):
            at = np.take_along_axis(x, np.where(r["ok"], y, 0), 1)
            tol = s + 2 * U * (inv * np.abs(at - M[:, None]) + np.abs(r["logp"]))
            near(np64(self.logp).reshape(y.shape), r["logp"], np.where(r["ok"], tol, 0))
            near(np64(self.lse), r["lse"], s + 2 * U * (inv * np.abs(M) + np.abs(r["lse"])))
            if self.entropy is not None:
                near(np64(self.entropy), r["entropy"], 2 * s * (1 + np.log(self.V)) + 0 * M)
            if self.top:
                assert np.array_equal(self.top_ids.cpu().numpy(), r["top_ids"])
                v = np.take_along_axis(x, np.maximum(r["top_ids"], 0), 1)
                near(np64(self.top_logp), r["top_logp"],
                     s + 2 * U * (inv * np.abs(v - M[:, None]) + np.abs(r["top_logp"])))

    def check_bwd(self, r=None, got=None):
        r, x, inv = r if r is not None else self.ref()
        s = (80 + self.V / 512) * U
        with np.errstate(invalid="ignore", over="ignore"):
            part = s + 8 * U + 4 * U * np.minimum(np.abs(r["logs"]), 100)
            if self.dh is not None:      # the entropy's own error, times p
                part = part + 2 * s
            tol = 2 * r["mag"] * part + HALF[self.logits.dtype] * np.abs(r["dx"]) + 2.0 ** -120
            if self.dh is not None:
                tol = tol + inv * r["p"] * np.abs(np64(self.dh))[:, None] * 4 * s * (1 + np.log(self.V))
        near(np64(self.dlogits if got is None else got), r["dx"], tol)
        if got is None:
            assert (self.dwhole[:, self.V:] == 11).all()
        assert all(ok() for ok in self.guards)


def near(got, ref, tol):
    with np.errstate(invalid="ignore"):
        same = (got == ref) | (np.isnan(got) & np.isnan(ref))
        fine = same | (np.abs(got - ref) <= tol)
    assert fine.all(), (np.argwhere(~fine)[:4].tolist(), got[~fine][:4], ref[~fine][:4])


SHAPES = [   # T, V, dtype, m, top, off, pad
    (1, 1, F32, 1, 1, 0, 0), (1, 1, BF, 2, 3, 1, 0), (3, 2, BF, 1, 2, 0, 5), (5, 7, F32, 1, 4, 1, 0),
    (4, 31, BF, 3, 32, 3, 1), (9, 257, BF, 1, 5, 0, 0), (9, 257, F32, 2, 5, 2, 3), (6, 1000, BF, 64, 20, 0, 24),
    (33, 4099, F32, 1, 0, 1, 0), (17, 16384, BF, 4, 8, 0, 0), (17, 16385, BF, 4, 8, 7, 0),
    (5, 50257, F32, 1, 32, 0, 0), (2, 50257, BF, 1, 1, 0, 0), (700, 18001, BF, 1, 3, 0, 0),
    (1, 151936, BF, 1, 20, 0, 0), (3, 151936, BF, 5, 0, 0, 64), (160, 20480, BF, 1, 2, 0, 0)]


@pytest.mark.parametrize("T,V,dtype,m,top,off,pad", SHAPES)
def test_values_and_gradient(T, V, dtype, m, top, off, pad):
    c = Case(T, V, dtype, m, top, off, pad, ids=torch.int64 if V % 2 else torch.int32)
    r = c.ref()
    c.fwd()
    c.check_fwd(r)
    c.bwd()
    c.check_bwd(r)
    c.clear()
    c.dwhole.fill_(11)
    c.step()
    c.check_fwd(r)
    c.check_bwd(r)
    assert L.moe_status() == L.MOE_OK


@pytest.mark.parametrize("T,V,dtype,top,off", [(761, 17000, BF, 0, 0), (1216, 9001, F32, 0, 1),
                                               (609, 16501, F32, 4, 3), (900, 20001, BF, 32, 5)])
def test_rows_just_above_the_places_for_blocks(T, V, dtype, top, off):
    c = Case(T, V, dtype, 1, top, off, 0)
    c.fwd()
    c.check_fwd()
    assert L.moe_status() == L.MOE_OK


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("inv", [0.25, 1.0, 1.7])
def test_temperature_in_place_and_without_entropy(dtype, inv):
    c = Case(7, 5000, dtype, 2, 4, inv=inv, entropy=False)
    r = c.ref()
    c.fwd()
    c.check_fwd(r)
    c.bwd()
    c.check_bwd(r)
    want = c.dlogits.clone()
    x = c.logits.clone()
    c.bwd(into=c.logits)
    assert torch.equal(c.logits, want)
    c.logits.copy_(x)
    c.dwhole.fill_(11)
    c.step()
    want = c.dlogits.clone()
    c.step(into=c.logits)
    assert torch.equal(c.logits, want)
    c.check_fwd(r)


@pytest.mark.parametrize("V", [1000, 18000])
@pytest.mark.parametrize("off_x,off_d", [(0, 1), (1, 0), (3, 5)])
def test_rows_of_another_alignment(V, off_x, off_d):
    c = Case(5, V, BF, 2, 2, off=off_x)
    r = c.ref()
    c.fwd()
    d, ok = place((5, V), BF, off_d)
    c.bwd(into=d)
    c.check_bwd(r, d)
    d.fill_(3)
    c.step(into=d)
    c.check_bwd(r, d)
    assert ok()


@pytest.mark.parametrize("V", [300, 40001])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_masked_rows(V, dtype):
    """-inf for some, for all but one, for all; the type's lowest value; few tokens left."""
    low = torch.finfo(dtype).min
    g = gen(V)
    x = torch.randn(8, V, generator=g, device=DEV)
    x[0, torch.rand(V, generator=g, device=DEV) < 0.5] = -INF
    x[1] = -INF
    x[2], x[2, V - 1] = -INF, 4.0
    x[3] = low
    x[4, ::2] = low
    x[5] = -INF
    x[5, 7], x[5, V // 2], x[5, V - 2] = 1.0, 1.0, 2.0
    x[6, 1:] = -INF
    x[7] = low
    x[7, 3] = -INF
    y = torch.tensor([[5], [0], [V - 1], [4], [1], [V // 2], [0], [9]], device=DEV)
    x[0, 5] = 0.5
    c = Case(8, V, dtype, 1, 6, x=x.to(dtype).float(), y=y)
    r = c.ref()
    c.fwd()
    c.check_fwd(r)
    c.bwd()
    c.check_bwd(r)
    assert not c.dlogits[1].any()
    c.dwhole.fill_(11)
    c.step()
    c.check_fwd(r)
    c.check_bwd(r)


def masked_rows(V, value, g):
    """Rows with `value` in whole words and threads' shares, scattered, everywhere, and all but
    one place; one more row is as large as the value is low."""
    x = torch.randn(8, V, generator=g, device=DEV)
    x[0, :3 * V // 4] = value
    x[1, V // 3:] = value
    x[2], x[2, V // 2] = value, 1.5
    x[3] = value
    x[4, torch.rand(V, generator=g, device=DEV) < 0.5] = value
    x[5], x[5, V // 3] = value, -INF
    x[6, V - 2] = 1e30
    x[7, :V // 2] = -INF
    y = torch.tensor([[V - 1], [0], [V // 2], [4], [1], [0], [V - 2], [V - 1]], device=DEV)
    x[4, 1] = 0.25
    return x, y


@pytest.mark.parametrize("V", [300, 40001])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [-1e4, -1e7, -1e10, -1e30, "lowest", -INF])
@pytest.mark.parametrize("inv", [1.0, 0.7])
def test_masks_of_any_value(V, dtype, value, inv):
    """Logits of any size count as far below the rest, in the words of a thread that sees
    nothing else too; a row of nothing else is uniform."""
    x, y = masked_rows(V, torch.finfo(dtype).min if value == "lowest" else value, gen(V))
    c = Case(8, V, dtype, 1, 6, x=x.to(dtype).float(), y=y, inv=inv)
    r = c.ref()
    c.fwd()
    c.check_fwd(r)
    c.bwd()
    c.check_bwd(r)
    c.clear()
    c.dwhole.fill_(11)
    c.step()
    c.check_fwd(r)
    c.check_bwd(r)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [-1e30, "lowest", -INF])
@pytest.mark.parametrize("inv", [1e-30, 1e-3, 0.01, 0.03, 0.045])
def test_masks_at_any_temperature(dtype, value, inv):
    x, y = masked_rows(5000, torch.finfo(dtype).min if value == "lowest" else value, gen(8))
    c = Case(8, 5000, dtype, 1, 6, x=x.to(dtype).float(), y=y, inv=inv)
    r = c.ref()
    c.fwd()
    c.check_fwd(r)
    c.bwd()
    c.check_bwd(r)
    c.clear()
    c.dwhole.fill_(11)
    c.step()
    c.check_fwd(r)
    c.check_bwd(r)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_lowest_temperature(dtype):
    """All of a row's probability on its best tokens, two of them in one row."""
    x, y = masked_rows(700, -INF, gen(9))
    x[6, 698], x[5] = 30.0, 2.0
    x[4, 9], x[4, 500] = 20.0, 20.0
    c = Case(8, 700, dtype, 1, 6, x=x.to(dtype).float(), y=y, inv=1e30)
    r = c.ref()
    c.fwd()
    c.check_fwd(r)
    c.bwd()
    c.check_bwd(r)


@pytest.mark.parametrize("V", [300, 40001])
@pytest.mark.parametrize("value", [-1e30, "lowest", -INF])
def test_large_gradients_of_the_entropy(V, value):
    """p = 0 has no gradient, however large its logarithm times the entropy's gradient is."""
    x, y = masked_rows(V, torch.finfo(BF).min if value == "lowest" else value, gen(V))
    c = Case(8, V, BF, 1, x=x.to(BF).float(), y=y)
    c.dh.mul_(1e6)
    r = c.ref()
    c.fwd()
    c.bwd()
    c.check_bwd(r)
    c.dwhole.fill_(11)
    c.step()
    c.check_bwd(r)


def test_a_target_that_is_masked():
    x = torch.zeros(2, 64, device=DEV)
    x[:, 5] = -INF
    c = Case(2, 64, F32, 1, x=x, y=torch.tensor([[5], [6]], device=DEV))
    r = c.ref()
    c.fwd()
    c.check_fwd(r)
    assert c.logp[0] == -INF
    c.bwd()
    c.check_bwd(r)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_target_of_the_lowest_value(dtype):
    """Its log probability is the type's lowest value too, and finite; listed last."""
    low = torch.finfo(dtype).min
    x = torch.full((2, 64), low, device=DEV)
    x[0, 3], x[1, :60] = 1.0, 0.5
    c = Case(2, 64, dtype, 2, 4, x=x, y=torch.tensor([[5, 3], [63, 0]], device=DEV))
    r = c.ref()
    c.fwd()
    c.check_fwd(r)
    assert torch.isfinite(c.logp).all() and torch.isfinite(c.top_logp).all()
    c.bwd()
    c.check_bwd(r)
    c.step()
    c.check_fwd(r)


@pytest.mark.parametrize("V", [90, 30000])
@pytest.mark.parametrize("what", [float("nan"), INF])
def test_rows_that_are_not_finite_spoil_themselves_only(V, what):
    c = Case(4, V, BF, 1, 3)
    c.logits[1, V // 3], c.logits[2, V - 1] = what, what
    clean = Case(4, V, BF, 1, 3)
    clean.fwd()
    clean.bwd()
    for run in ("two", "step"):
        if run == "two":
            c.fwd()
            c.bwd()
        else:
            c.step()
        for t in (1, 2):
            for o in (c.logp, c.lse, c.entropy, c.top_logp):
                assert torch.isnan(o[t]).all()
            assert torch.isnan(c.dlogits[t]).all()
            assert ((c.top_ids[t] >= 0) & (c.top_ids[t] < V)).all()
        for t in (0, 3):
            assert torch.isfinite(c.dlogits[t]).all() and torch.equal(c.top_ids[t], clean.top_ids[t])
    x = torch.full((1, V), float("nan"), device=DEV)
    c = Case(1, V, BF, 1, 3, x=x)
    c.fwd()
    assert torch.isnan(c.lse).all() and (c.top_ids == -1).all() and (c.top_logp == -INF).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [64, 700, 20011, 151936])
def test_equal_logits_go_by_the_lower_id(V, dtype):
    """All equal; two values; the best at both ends; negative and positive zeros."""
    g = gen(V)
    x = torch.zeros(5, V, device=DEV)
    x[1] = torch.randint(0, 2, (V,), generator=g, device=DEV).float()
    x[2, 0], x[2, V - 1], x[2, V // 2] = 3, 3, 3
    x[3] = torch.where(torch.rand(V, generator=g, device=DEV) < 0.5, 0.0, -0.0)
    x[4] = torch.randint(-3, 1, (V,), generator=g, device=DEV).float()
    c = Case(5, V, dtype, 1, 32, x=x)
    c.fwd()
    c.check_fwd()


@pytest.mark.parametrize("V", [5000, 16384, 40000])
def test_alternatives_of_ordered_and_clustered_rows(V):
    """Rising and falling rows, and rows whose best all lie in one thread's words."""
    x = torch.zeros(5, V, device=DEV)
    x[0] = torch.arange(V, device=DEV) / 64
    x[1] = -x[0]
    x[2, 8::4096] = 50.0 + torch.arange(len(range(8, V, 4096)), device=DEV)
    i = torch.arange(V, device=DEV)
    x[3] = torch.where(i // 4 % 512 == 5, 10.0 + i / 1000, 0.0)
    x[4] = torch.where(i // 8 % 512 < 40, 10.0 - i / 1e5, -i / 1e5)
    for top in (1, 31):
        c = Case(5, V, F32, 1, top, x=x)
        c.fwd()
        c.check_fwd()
        c = Case(5, V, BF, 1, top, x=x)
        c.fwd()
        c.check_fwd()


def test_more_equal_alternatives_than_are_sorted_at_once():
    """Thousands of tokens above the rest in the words of a few threads, all different."""
    V = 120000
    i = torch.arange(V, device=DEV)
    x = torch.where(i // 4 % 512 < 31, 100.0 + (i * 7919 % V) / 1000.0, -i / 1e3)
    c = Case(700, V, F32, 1, 32, x=x[None].repeat(700, 1), grads=False, entropy=False)
    c.fwd()
    one = Case(1, V, F32, 1, 32, x=x[None], entropy=False)
    one.fwd()
    one.check_fwd()
    assert (c.top_ids == one.top_ids).all()


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("V", [100, 20000])
def test_ignored_and_bad_targets(V, ids):
    y = torch.tensor([[-100, 3, 3, 99], [-100, -100, -100, -100], [0, 1, 0, 0], [7, -100, 7, 7]], device=DEV)
    c = Case(4, V, BF, 4, 0, y=y, ids=ids, entropy=False, grads=False)
    for run in (lambda: (c.fwd(), c.bwd()), c.step):
        c.dwhole.fill_(11)
        run()
        assert L.moe_status() == L.MOE_OK
        r = c.ref()
        c.check_fwd(r)
        c.check_bwd(r)
        assert not c.dlogits[1].any()
    y[0, 0], y[3, 1] = -1, V
    c = Case(4, V, BF, 4, 0, y=y, ids=ids, entropy=False, grads=False)
    for run in (c.fwd, c.step):
        run()
        assert L.moe_status() == L.MOE_ERR_BAD_IDS
        c.check_fwd()
    c.bwd()
    c.check_bwd()
    c = Case(4, V, BF, 1, 0, y=torch.tensor([[5], [7], [5], [1]], device=DEV), entropy=False, grads=False)
    c.fwd(ignore_id=5)
    assert L.moe_status() == L.MOE_OK
    assert c.logp[0] == 0 and c.logp[2] == 0 and c.logp[1] != 0
    c.bwd(ignore_id=5)
    assert not c.dlogits[0].any() and not c.dlogits[2].any() and c.dlogits[1].any()


def test_ids_past_64_bits_are_refused():
    """Their lower bits are tokens' ids."""
    c = Case(2, 50, F32, entropy=False, grads=False)
    for bad in (2 ** 63, 2 ** 64 + 3, -2 ** 63 - 1):
        for call in (c.fwd, c.bwd, c.step):
            with pytest.raises(ValueError):
                call(ignore_id=bad)
    c.fwd(ignore_id=2 ** 63 - 1)
    c.check_fwd()


def test_rows_that_get_no_gradient_are_not_read():
    """Zeros, whatever the logits hold; a NaN gradient is not nothing."""
    c = Case(3, 9000, F32, 2, entropy=False, grads=False)
    c.fwd()
    c.logits[1] = float("nan")
    c.dlogp[1] = 0
    c.bwd()
    assert not c.dlogits[1].any() and c.dlogits[0].any() and c.dlogits[2].any()
    c.dlogp[0, 1] = float("nan")
    c.bwd()
    assert torch.isnan(c.dlogits[0]).all()
    L.moe_logprob_bwd(c.logits, c.targets, c.stats, None, c.dlogits)
    assert not c.dlogits.any()


def test_offsets_past_2_to_31_values():
    T, V = 15000, 151936
    x = torch.zeros(T, V, dtype=BF, device=DEV)
    g = gen(2)
    x[-2:] = torch.randn(2, V, generator=g, device=DEV).to(BF)
    c = Case(2, V, BF, 1, 3, x=x[-2:].float())
    c.fwd()
    c.step()
    big = dict(logp=torch.empty(T, device=DEV), stats=torch.empty(T, 2, device=DEV))
    y = torch.zeros(T, dtype=torch.int64, device=DEV)
    y[-2:] = c.targets
    dlogp, dh, dl = (torch.zeros(T, device=DEV) for _ in range(3))
    dlogp[-2:], dh[-2:], dl[-2:] = c.dlogp, c.dh, c.dl
    dlogp[0] = 1
    ids, lp, ent = torch.empty(T, 3, dtype=torch.int32, device=DEV), torch.empty(T, 3, device=DEV), torch.empty(T, device=DEV)
    lse = torch.empty(T, device=DEV)
    L.moe_logprob_step(x, y, big["logp"], big["stats"], dlogp, x, dentropy=dh, dlse=dl, lse=lse, entropy=ent,
                       top_ids=ids, top_logp=lp)
    for to, got in ((c.logp, big["logp"]), (c.lse, lse), (c.entropy, ent), (c.top_ids, ids), (c.top_logp, lp)):
        to.copy_(got[-2:])
    c.check_fwd()
    c.check_bwd(got=x[-2:])
    assert torch.equal(ids[-2:], c.top_ids) and (ids[:-2] == torch.arange(3, device=DEV)).all()
    assert x[0, 0] > 0.9 and not x[1:-2].any()


def test_no_rows():
    z = torch.empty(0, device=DEV)
    x = torch.empty(0, 50, device=DEV)
    y = torch.empty(0, dtype=torch.int64, device=DEV)
    L.moe_logprob_fwd(x, y, z, torch.empty(0, 2, device=DEV))
    L.moe_logprob_bwd(x, y, torch.empty(0, 2, device=DEV), z, x)
    L.moe_logprob_step(x, y, z, torch.empty(0, 2, device=DEV), z, x)


@pytest.mark.parametrize("V", [3000, 70000])
def test_streams_and_graphs(V):
    c = Case(6, V, BF, 2, 4)
    c.fwd()
    c.bwd()
    keep = [t.clone() for t in (c.logp, c.lse, c.entropy, c.top_ids, c.dlogits)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.dlogits.zero_()
    c.fwd(stream=s)
    c.bwd(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(keep, (c.logp, c.lse, c.entropy, c.top_ids, c.dlogits)):
        assert torch.equal(a, b)
    graph = graph_of(lambda: (c.fwd(), c.bwd()))
    step = graph_of(c.step)
    c.logits.mul_(0.5)
    graph.replay()
    r = c.ref()
    c.check_fwd(r)
    c.check_bwd(r)
    c.dlogits.zero_()
    step.replay()
    c.check_fwd(r)
    c.check_bwd(r)
