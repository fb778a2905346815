"""The AdamW step on the GPU.  Its operations are rounded one by one, so every
result equals the oracle's fp32 restatement bit for bit, 8-bit states included
(the oracle finds those on the format's grid); the global norm is compared with
64 bits: the pair of floats it is summed in is good to about 2^-44, so its fp32
rounding is off by one unit at most (2^-23 used)."""
import math

import numpy as np
import pytest
import torch

from expert_routing_grouped_moe_gb300 import _lib as L
from oracle import block_oracle as bo
from _util import to64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HYPER = dict(lr=1e-2, betas=(0.9, 0.99), eps=1e-8)
KINDS = [(F32, F32, False), (F32, BF, False), (BF, F32, False), (BF, BF, False), (BF, F32, True),
         (BF, BF, True)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routing_grouped_moe_gb300 import build
    build.build()
    L.load()


def tensor(n, pt, gt, master, bits, seed, off=0, wd=0.0, lr_mult=1.0, fresh=False):
    """One row of the table; off: values that every buffer begins past an aligned address."""
    g = torch.Generator(DEV).manual_seed(seed)

    def place(x):
        raw = torch.empty(x.numel() + off, dtype=x.dtype, device=DEV)
        raw[off:].copy_(x)
        return raw[off:]
    p = torch.randn(n, generator=g, device=DEV)
    grad = torch.randn(n, generator=g, device=DEV) * torch.exp(
        2 * torch.randn(n, generator=g, device=DEV))
    grad[::17] = 0
    row = dict(param=place(p.to(pt)), grad=place(grad.to(gt)),
               master=place(p) if master else None, weight_decay=wd, lr_mult=lr_mult, scales=None)
    if bits == 32:
        row["m"] = place(torch.zeros(n, device=DEV) if fresh else
                         0.1 * torch.randn(n, generator=g, device=DEV))
        row["v"] = place(torch.zeros(n, device=DEV) if fresh else
                         torch.randn(n, generator=g, device=DEV).square())
    else:
        code = torch.randint(0, 0x78, (2, n), generator=g, device=DEV)
        code[0] += 128 * torch.randint(0, 2, (n,), generator=g, device=DEV)
        code *= 0 if fresh else 1
        row["m"], row["v"] = (place(c.to(torch.uint8)) for c in code)
        nb = -(-n // 256)
        row["scales"] = torch.randint(116, 122, (nb, 2), generator=g, device=DEV).to(torch.uint8)
        if fresh:
            row["scales"].zero_()
    return row


def expect(row, step, coef=1.0, **h):
    c = None
    if row["scales"] is not None:
        c = tuple(row[k].view(torch.uint8).cpu().numpy() for k in ("m", "v")) + (
            row["scales"].cpu().numpy(),)
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    return bo.adamw_step32(
        f(row["param"] if row["master"] is None else row["master"]), f(row["grad"]),
        None if c else f(row["m"]), None if c else f(row["v"]), c, step, h["lr"], *h["betas"],
        h["eps"], np.float32(row["weight_decay"]).astype(float), coef,
        np.float32(row["lr_mult"]).astype(float))


def check(row, exp):
    p = torch.from_numpy(exp[0]).to(DEV)
    assert torch.equal(row["param"], p.to(row["param"].dtype))
    if row["master"] is not None:
        assert torch.equal(row["master"], p)
    for k, e in zip(("m", "v"), exp[1:3]):
        assert torch.equal(row[k].view(torch.uint8) if row["scales"] is not None else row[k],
                           torch.from_numpy(e).to(DEV)), k
    if row["scales"] is not None:
        assert torch.equal(row["scales"], torch.from_numpy(exp[3]).to(DEV))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pt,gt,master", KINDS)
def test_every_kind_bit_for_bit(pt, gt, master, bits):
    sizes = [1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 10007, 70001]
    rows = [tensor(n, pt, gt, master, bits, seed=i, wd=0.1 * (i % 3), lr_mult=1.0 + (i % 2),
                   fresh=i == 3) for i, n in enumerate(sizes)]
    table = L.AdamWTable(rows)
    for step in (5, 6):
        exp = [expect(r, step, **HYPER) for r in rows]
        L.moe_adamw_step(table, step, **HYPER)
        for r, e in zip(rows, exp):
            check(r, e)


@pytest.mark.parametrize("seed", range(4))
def test_roots_and_quotients_over_the_exponents(seed):
    """Moments and gradients over some hundred binades: the step's own square root
    and division are the nearest fp32 values, as numpy's are."""
    n, g = 500_000, torch.Generator(DEV).manual_seed(seed)
    lo, hi, vlo, vhi = [(-40, 20, -80, 40), (-10, 10, -20, 20), (-60, -30, -126, -60),
                        (-45, 10, -126, 20)][seed]

    def mag(a, b):
        return torch.exp2(a + (b - a) * torch.rand(n, generator=g, device=DEV))
    sign = torch.where(torch.rand(n, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    row = dict(param=torch.zeros(n, device=DEV), grad=mag(lo, hi) * sign, m=mag(lo, hi) * sign.flip(0),
               v=mag(vlo, vhi), master=None, scales=None, weight_decay=0.0, lr_mult=1.0)
    if seed == 3:
        row["v"].zero_()
        row["grad"][::3] = 0
    h = dict(HYPER, lr=1.0)
    exp = expect(row, 3, **h)
    L.moe_adamw_step(L.AdamWTable([row]), 3, **h)
    check(row, exp)


@pytest.mark.parametrize("lo,hi", [(-90, -60), (-72, -40), (-75, 10), (-3, -3)])
def test_eight_bits_of_gradients_whose_squares_vanish(lo, hi):
    """Blocks whose values lie many binades apart, m above zero where v is not, and
    squares below the normal numbers: the codes are still the oracle's."""
    n, g = 100_003, torch.Generator(DEV).manual_seed(hi)
    grad = torch.exp2(lo + (hi - lo) * torch.rand(n, generator=g, device=DEV))
    grad = torch.where(torch.rand(n, generator=g, device=DEV) < 0.5, -grad, grad)
    grad[::7] = 0
    grad[5::256] *= 2.0 ** 20
    row = tensor(n, F32, F32, False, 8, seed=1, fresh=True)
    row["grad"] = grad
    for step in (1, 2, 3):
        exp = expect(row, step, **HYPER)
        L.moe_adamw_step(L.AdamWTable([row]), step, **HYPER)
        check(row, exp)


@pytest.mark.parametrize("bits", [32, 8])
def test_mixed_kinds_and_pointers_that_no_vector_fits(bits):
    rows = [tensor(300 + 11 * i, *KINDS[i % 6], 8 if (i % 5 == 0) else bits, seed=i, off=i % 4)
            for i in range(30)]
    exp = [expect(r, 1, **HYPER) for r in rows]
    L.moe_adamw_step(L.AdamWTable(rows), 1, **HYPER)
    for r, e in zip(rows, exp):
        check(r, e)


@pytest.mark.parametrize("off", [4, 8, 16])
@pytest.mark.parametrize("bits", [32, 8])
def test_pointers_on_16_and_32_byte_boundaries(bits, off):
    """Whole chunks and ragged ends, with the norm, whatever widths the pointers allow."""
    rows = [tensor(n, pt, gt, master, bits, seed=i, off=off)
            for i, ((pt, gt, master), n) in enumerate(zip(KINDS, [2048, 6144, 5000, 4097, 8192, 2056]))]
    norm = math.sqrt(sum(float(np.square(to64(r["grad"])).sum()) for r in rows))
    out, table = torch.zeros(1, device=DEV), L.AdamWTable(rows)
    ws = torch.empty(L.moe_adamw_workspace_size(table), dtype=torch.uint8, device=DEV)
    exp = [expect(r, 4, **HYPER) for r in rows]
    L.moe_adamw_step(table, 4, grad_norm=out, ws=ws, **HYPER)
    assert abs(out.item() - norm) <= 2 ** -23 * norm
    for r, e in zip(rows, exp):
        check(r, e)


def test_more_tensors_than_a_launch_takes():
    rows = [tensor(1 + (i * 37) % 600, *KINDS[4 * (i % 2)], 8 if i % 3 else 32, seed=i)
            for i in range(1700)]
    table = L.AdamWTable(rows)
    norm = torch.empty(1, device=DEV)
    ws = torch.empty(L.moe_adamw_workspace_size(table), dtype=torch.uint8, device=DEV)
    total = math.sqrt(sum(float(r["grad"].double().square().sum()) for r in rows))
    exp = [expect(r, 3, **HYPER) for r in rows]
    L.moe_adamw_step(table, 3, grad_norm=norm, ws=ws, **HYPER)
    assert abs(float(norm) - total) <= 2.0 ** -23 * total
    for r, e in zip(rows, exp):
        check(r, e)


@pytest.mark.parametrize("bits", [32, 8])
def test_clip_by_the_global_norm(bits):
    rows = [tensor(n, BF, F32, True, bits, seed=n) for n in (3, 5000, 300000)]
    rows.append(tensor(40000, F32, BF, False, 32, seed=9))
    table = L.AdamWTable(rows)
    ws = torch.empty(L.moe_adamw_workspace_size(table), dtype=torch.uint8, device=DEV)
    norm = torch.empty(1, device=DEV)
    total = math.sqrt(sum(float(r["grad"].double().square().sum()) for r in rows))
    for max_norm, scale in ((1.0, 1.0), (0.5, 0.25), (1e9, 2.0)):
        L.moe_adamw_step(table, 1, lr=0.0, grad_norm=norm, ws=ws, grad_scale=scale)
        assert abs(float(norm) - total * scale) <= 2.0 ** -23 * total * scale
        f = np.float32
        q = f(max_norm) / (f(norm.item()) + f(1e-6))
        coef = f(scale) * (f(1.0) if q >= 1 else q)
        exp = [expect(r, 2, coef=coef, **HYPER) for r in rows]
        L.moe_adamw_step(table, 2, max_norm=max_norm, grad_scale=scale, grad_norm=norm, ws=ws,
                         **HYPER)
        for r, e in zip(rows, exp):
            check(r, e)


def test_norm_of_one_value_among_many_small_ones():
    """What plain fp32 sums lose: 10^7 squares of 1e-4 beside one of 100."""
    n = 10_000_000
    row = tensor(n, F32, F32, False, 32, seed=1)
    row["grad"].fill_(1e-4)
    row["grad"][0] = 100.0
    table = L.AdamWTable([row])
    ws = torch.empty(L.moe_adamw_workspace_size(table), dtype=torch.uint8, device=DEV)
    norm = torch.empty(1, device=DEV)
    L.moe_adamw_step(table, 1, lr=0.0, grad_norm=norm, ws=ws)
    ref = math.sqrt(float(row["grad"].double().square().sum()))
    assert abs(float(norm) - ref) <= 2.0 ** -23 * ref


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_step_that_is_skipped_changes_nothing(value):
    rows = [tensor(700, BF, F32, True, 8, seed=1), tensor(3000, F32, F32, False, 32, seed=2)]
    rows[0]["grad"][600] = value
    table = L.AdamWTable(rows)
    ws = torch.empty(L.moe_adamw_workspace_size(table), dtype=torch.uint8, device=DEV)
    norm = torch.empty(1, device=DEV)
    before = [{k: t.clone() for k, t in r.items() if torch.is_tensor(t)} for r in rows]
    L.moe_adamw_step(table, 4, skip_nonfinite=True, grad_norm=norm, ws=ws, **HYPER)
    assert not torch.isfinite(norm).any()
    for r, b in zip(rows, before):
        for k in b:
            assert torch.equal(r[k].view(torch.uint8), b[k].view(torch.uint8)), k
    # without the switch it spoils its own block of 256 and no other
    exp = [expect(r, 4, **HYPER) for r in rows]
    L.moe_adamw_step(table, 4, **HYPER)
    check(rows[1], exp[1])
    keep = list(range(512)) 
    assert torch.equal(rows[0]["master"][keep], torch.from_numpy(exp[0][0][keep]).to(DEV))
    assert not torch.isfinite(rows[0]["master"][600])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("at", [0, 699, 250_000])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), 2e19, 1e20, 3e38])
def test_a_norm_that_overflows_clips_to_nothing(value, at, bits):
    """norm = inf gives a factor of 0: every gradient counts as zero, and only those
    that are themselves infinite spoil their values (0 inf)."""
    rows = [tensor(300_000, F32, F32, False, bits, seed=1), tensor(700, BF, F32, True, bits, seed=2),
            tensor(5000, BF, BF, False, 32, seed=3)]
    rows[0]["grad"][at] = value
    table = L.AdamWTable(rows)
    ws = torch.empty(L.moe_adamw_workspace_size(table), dtype=torch.uint8, device=DEV)
    norm = torch.empty(1, device=DEV)
    spoilt = not math.isfinite(value)
    rows[0]["grad"][at] = 0.0 if spoilt else value
    exp = [expect(r, 4, coef=0.0, **HYPER) for r in rows]
    rows[0]["grad"][at] = value
    L.moe_adamw_step(table, 4, max_norm=1.0, grad_norm=norm, ws=ws, **HYPER)
    assert float(norm) == float("inf")
    for r, e in zip(rows[1:], exp[1:]):
        check(r, e)
    if not spoilt:
        check(rows[0], exp[0])
        return
    keep = torch.ones(300_000, dtype=torch.bool, device=DEV)
    first = at // 256 * 256
    keep[first:first + 256] = False
    assert torch.equal(rows[0]["param"][keep], torch.from_numpy(exp[0][0]).to(DEV)[keep])
    assert not torch.isfinite(rows[0]["param"][at])


def test_a_norm_that_is_nan_stays_nan():
    rows = [tensor(300_000, F32, F32, False, 32, seed=1), tensor(700, BF, F32, True, 32, seed=2)]
    rows[0]["grad"][5] = float("inf")
    rows[0]["grad"][200_000] = float("nan")
    table = L.AdamWTable(rows)
    ws = torch.empty(L.moe_adamw_workspace_size(table), dtype=torch.uint8, device=DEV)
    norm = torch.empty(1, device=DEV)
    L.moe_adamw_step(table, 4, max_norm=1.0, grad_norm=norm, ws=ws, **HYPER)
    assert torch.isnan(norm).all() and torch.isnan(rows[1]["param"].float()).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value", [5e19, 1e21, -1e24])
def test_a_finite_gradient_whose_square_overflows(value, bits):
    """v = inf divides the update away, as the formula has it in fp32 (the kernel's
    largest denominator is 2^120: 1e24 / 2^120 is far below an ulp of the parameters),
    and spoils nothing."""
    row = tensor(3000, F32, F32, False, bits, seed=5, fresh=bits == 8)
    row["grad"][1000] = value
    row["grad"][2999] = value
    with np.errstate(all="ignore"):
        exp = expect(row, 4, **HYPER)
    assert np.isfinite(exp[0]).all()
    L.moe_adamw_step(L.AdamWTable([row]), 4, **HYPER)
    if bits == 32:
        check(row, exp)
    assert torch.equal(row["param"], torch.from_numpy(exp[0]).to(DEV))
    row["grad"].fill_(1.0)
    L.moe_adamw_step(L.AdamWTable([row]), 5, **HYPER)
    assert torch.isfinite(row["param"]).all()


def test_no_tensors_and_empty_tensors():
    norm = torch.full((1,), 3.0, device=DEV)
    ws = torch.empty(1 << 14, dtype=torch.uint8, device=DEV)
    L.moe_adamw_step(L.AdamWTable([]), 1, lr=0.1, grad_norm=norm, ws=ws)
    assert float(norm) == 0.0
    rows = [tensor(0, BF, F32, True, 8, seed=1), tensor(50, BF, F32, True, 8, seed=2),
            tensor(0, F32, F32, False, 32, seed=3)]
    exp = expect(rows[1], 1, **HYPER)
    L.moe_adamw_step(L.AdamWTable(rows), 1, **HYPER)
    check(rows[1], exp)


def test_eight_bit_states_follow_the_32_bit_ones():
    """200 steps on gradients of a fixed spread: the 8-bit run's parameters stay
    near the 32-bit run's.  A root's grid step is 12.5 %, dithered, so the
    denominators wander by some 20 % and updates by as much at random; over 200
    steps of alternating gradients the two end within a quarter of the distance
    travelled, where a root that never moved from its first value would be an
    order of magnitude off (the gradients shrink 30 times after 100 steps)."""
    n = 4096
    rows = [tensor(n, F32, F32, False, 32, seed=1, fresh=True),
            tensor(n, F32, F32, False, 8, seed=1, fresh=True)]
    table = L.AdamWTable(rows)
    start = rows[0]["param"].clone()
    g = torch.Generator(DEV).manual_seed(3)
    size = torch.exp(torch.randn(n, generator=g, device=DEV))
    for step in range(1, 201):
        grad = (torch.randn(n, generator=g, device=DEV) + 0.5) * size * (1.0 if step <= 100 else 0.03)
        for r in rows:
            r["grad"].copy_(grad)
        L.moe_adamw_step(table, step, lr=1e-3, betas=(0.9, 0.95), eps=1e-8)
    a, b = rows[0]["param"] - start, rows[1]["param"] - start
    assert float((a - b).norm() / a.norm()) < 0.25


def test_states_are_torchs_float8():
    """m and v may be held as torch.float8_e4m3fn; their values times the scales are
    the moments the step computed."""
    row = tensor(5000, F32, F32, False, 8, seed=4, fresh=True)
    row["m"], row["v"] = row["m"].view(E4), row["v"].view(E4)
    L.moe_adamw_step(L.AdamWTable([row]), 1, **HYPER)
    s = row["scales"].view(torch.float8_e8m0fnu).float().repeat_interleave(256, 0)[:5000]
    m, root = 0.1 * row["grad"], (0.01 * row["grad"].square()).sqrt()
    # one grid step: an eighth of the value, or the smallest step, 2^-9 of the scale
    for got, ref, sc in ((row["m"].float() * s[:, 0], m, s[:, 0]),
                         (row["v"].float() * s[:, 1], root, s[:, 1])):
        assert torch.all((got - ref).abs() <= ref.abs() / 8 + sc * 2.0 ** -9)


def test_equal_bits_on_another_stream_and_in_a_graph():
    def fresh():
        return [tensor(100_003, BF, F32, True, 8, seed=1), tensor(5001, F32, BF, False, 32, seed=2)]
    runs = []
    for how in ("plain", "stream", "graph"):
        rows = fresh()
        table = L.AdamWTable(rows)
        ws = torch.empty(L.moe_adamw_workspace_size(table), dtype=torch.uint8, device=DEV)
        step = lambda s=None: L.moe_adamw_step(table, 9, max_norm=1.0, ws=ws, stream=s,  # noqa: E731
                                               **HYPER)
        torch.cuda.synchronize()
        if how == "plain":
            step()
        elif how == "stream":
            s = torch.cuda.Stream()
            step(s)
            s.synchronize()
        else:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            graph.replay()
        torch.cuda.synchronize()
        runs.append(rows)
    for rows in runs[1:]:
        for r, q in zip(rows, runs[0]):
            for k in ("param", "master", "m", "v", "scales"):
                if r[k] is not None:
                    assert torch.equal(r[k], q[k]), k


def test_offsets_past_32_bits():
    """A tensor of more than 2^31 values: its last ones are right."""
    n = 2 ** 31 + 2 ** 20 + 13
    tail = 2 ** 20 + 13
    first = n - tail                     # a whole number of blocks
    assert first % 256 == 0
    p = torch.zeros(n, dtype=BF, device=DEV)
    g = torch.zeros(n, dtype=BF, device=DEV)
    gen = torch.Generator(DEV).manual_seed(5)
    p[first:] = torch.randn(tail, generator=gen, device=DEV).to(BF)
    g[first:] = torch.randn(tail, generator=gen, device=DEV).to(BF)
    m = torch.zeros(n, dtype=torch.uint8, device=DEV)
    v = torch.zeros(n, dtype=torch.uint8, device=DEV)
    sc = torch.zeros(-(-n // 256), 2, dtype=torch.uint8, device=DEV)
    p0, g0 = p[first:].clone(), g[first:].clone()
    L.moe_adamw_step(L.AdamWTable([dict(param=p, grad=g, m=m, v=v, scales=sc)]), 1, **HYPER)
    zero = np.zeros(tail, np.uint8)
    exp = bo.adamw_step32(p0.float().cpu().numpy(), g0.float().cpu().numpy(), None, None,
                          (zero, zero, np.zeros((-(-tail // 256), 2), np.uint8)), 1, HYPER["lr"],
                          *HYPER["betas"], HYPER["eps"], 0.0)
    assert torch.equal(p[first:], torch.from_numpy(exp[0]).to(DEV).to(BF))
    # the dither goes by the index in the tensor: compare the scales and signs
    assert torch.equal(sc[first // 256:], torch.from_numpy(exp[3]).to(DEV))
    assert torch.equal(m[first:] & 128, torch.from_numpy(exp[1]).to(DEV) & 128)
    assert not p[:4096].any()


def test_nothing_is_written_past_a_buffer():
    bands, rows = [], []
    for i, (kind, bits, n) in enumerate([(k, b, n) for k in KINDS for b in (8, 32)
                                         for n in (1, 300, 2049)]):
        row = tensor(n, *kind, bits, seed=i)
        for k, t in list(row.items()):
            if torch.is_tensor(t):
                nb = t.numel() * t.element_size()
                raw = torch.full((nb + 512,), 0xA5, dtype=torch.uint8, device=DEV)
                view = raw[256:256 + nb].view(t.dtype).view(t.shape)
                view.copy_(t)
                row[k] = view
                bands.append((raw, nb))
        rows.append(row)
    table = L.AdamWTable(rows)
    size = L.moe_adamw_workspace_size(table)
    raw = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    bands.append((raw, size))
    L.moe_adamw_step(table, 1, max_norm=1.0, ws=raw[256:256 + size], **HYPER)
    torch.cuda.synchronize()
    for raw, nb in bands:
        assert torch.all(raw[:256] == 0xA5) and torch.all(raw[256 + nb:] == 0xA5)


def test_refusals_of_tensors():
    row = tensor(64, BF, F32, False, 32, seed=1)
    bad = [(dict(m=row["m"][:8]), "as many values"), (dict(grad=row["grad"].half()), "float32 or"),
           (dict(scales=torch.zeros(1, 2, dtype=torch.uint8, device=DEV)), "go with 8-bit"),
           (dict(param=row["param"].cpu()), "CUDA"), (dict(v=row["v"].to(BF)), "both alike")]
    for change, match in bad:
        with pytest.raises(ValueError, match=match):
            L.AdamWTable([dict(row, **change)])
    table = L.AdamWTable([row])
    for kw, match in [(dict(step=0), "step"), (dict(betas=(1.0, 0.9)), "betas"),
                      (dict(lr=float("nan")), "lr"), (dict(eps=0.0), "eps"),
                      (dict(max_norm=1.0), "ws"), (dict(max_norm=-1.0), "max_norm")]:
        args = dict(HYPER, step=1)
        args.update(kw)
        with pytest.raises(L.MoeError, match=match):
            L.moe_adamw_step(table, args.pop("step"), **args)
    assert float(row["m"].abs().sum()) > 0


def test_refused_gradients_leave_the_table_as_it_was():
    rows = [tensor(n, BF, F32, False, 32, seed=i) for i, n in enumerate((64, 300, 1000))]
    table = L.AdamWTable(rows)
    new = [torch.randn_like(r["grad"]) for r in rows]
    bad = [(new[:2] + [new[2][:999]], ValueError, "as many values"),
           (new[:2] + [new[2].half()], ValueError, "float32 or"),
           ([new[0], new[1].cpu(), new[2]], ValueError, "CUDA"),
           ([new[0], new[1], torch.zeros(2000, device=DEV)[::2]], ValueError, "contiguous"),
           ([new[0], None, new[2]], TypeError, "Tensor"), (new[:2], ValueError, "gradients for")]
    for grads, error, match in bad:
        with pytest.raises(error, match=match):
            table.set_grads(grads)
    exp = [expect(r, 2, **HYPER) for r in rows]
    L.moe_adamw_step(table, 2, **HYPER)
    for r, e in zip(rows, exp):
        check(r, e)
    # and all of them where none is refused, of another type too
    new[1] = new[1].to(BF)
    table.set_grads(new)
    for r, g in zip(rows, new):
        r["grad"] = g
    exp = [expect(r, 3, **HYPER) for r in rows]
    L.moe_adamw_step(table, 3, **HYPER)
    for r, e in zip(rows, exp):
        check(r, e)
