"""The norms around a block on the GPU against the 64-bit oracle: types, gates,
widths from one column to the limit, pointers that no vector fits, rows of
zeros and NaN, in-place calls, streams, graphs and refusals.

Tolerances, before any run: with u = 2^-24, a row sum of d terms is at most
8 * 4 + 5 + 16 = 53 additions deep and each result meets a handful of such sums
and operations, so 256 u of the sum of the sizes of its terms covers an fp32
result; a sum over tokens is at most 512 additions deep here (768 u).  A bf16
result adds its rounding, 2^-9 of itself (2^-8 used)."""
import numpy as np
import pytest
import torch

from expert_routing_grouped_moe_gb300 import _lib as L
from oracle import block_oracle as bo
from _util import to64

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
GATES = [("none", False), ("token", False), ("token", True), ("channel", False),
         ("channel", True), ("element", False), ("element", True)]
NORMS = [(True, True), (True, False), (False, True), (False, False)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routing_grouped_moe_gb300 import build
    build.build()
    L.load()


def close(got, ref, mag, name, ulps=256):
    got64 = to64(got)
    bound = ulps * U * mag + 1e-37
    if got.dtype == BF:
        bound = bound + 2.0 ** -8 * np.abs(ref)
    bad = ~(np.abs(got64 - ref) <= bound)
    assert not bad.any(), "%s: %d of %d beyond the bound, worst %.3g times" % (
        name, bad.sum(), bad.size, np.nanmax(np.abs(got64 - ref) / bound))


def make(T, d, xt, yt, kind, post, pre, seed=0, place=None):
    """Inputs and output buffers; place(shape, type) may give views of its own."""
    g = torch.Generator(DEV).manual_seed(seed * 977 + 13 * T + d)
    place = place or (lambda *a: torch.empty(a[0], dtype=a[1], device=DEV))

    def rnd(shape, dtype, mul=1.0):
        t = place(shape, dtype)
        t.copy_((torch.randn(shape, generator=g, device=DEV) * mul).to(dtype))
        return t
    b = {"x": rnd((T, d), xt, 2.0), "y": rnd((T, d), yt, 0.5), "dr": rnd((T, d), xt),
         "dn": rnd((T, d), yt) if pre else None,
         "w_post": rnd((d,), F32) if post else None, "w_pre": rnd((d,), F32) if pre else None,
         "gate": {"none": lambda: None, "token": lambda: rnd((T,), F32),
                  "channel": lambda: rnd((d,), F32), "element": lambda: rnd((T, d), yt)}[kind]()}
    b["r"], b["n"] = place((T, d), xt), place((T, d), yt) if pre else None
    b["rstd_y"] = place((T,), F32) if post else None
    b["rstd_r"] = place((T,), F32) if pre else None
    b["dx"], b["dy"] = place((T, d), xt), place((T, d), yt)
    b["dgate"] = None if b["gate"] is None else place(b["gate"].shape, b["gate"].dtype)
    b["dw_post"] = place((d,), F32) if post else None
    b["dw_pre"] = place((d,), F32) if pre else None
    b["ws"] = torch.empty(max(16, L.moe_block_norm_workspace_size(T, d)), dtype=torch.uint8,
                          device=DEV)
    return b


def forward(b, kind, sigmoid, stream=None, **kw):
    L.moe_block_norm_fwd(b["x"], b["y"], b["r"], b["n"], w_post=b["w_post"], w_pre=b["w_pre"],
                         rstd_y=b["rstd_y"], rstd_r=b["rstd_r"], gate=b["gate"], gate_kind=kind,
                         gate_sigmoid=sigmoid, stream=stream, **kw)


def backward(b, kind, sigmoid, stream=None, **kw):
    L.moe_block_norm_bwd(b["dr"], b["dn"], b["r"], b["y"], b["dx"], b["dy"], w_post=b["w_post"],
                         w_pre=b["w_pre"], rstd_y=b["rstd_y"], rstd_r=b["rstd_r"], gate=b["gate"],
                         gate_kind=kind, gate_sigmoid=sigmoid, dgate=b["dgate"],
                         dw_post=b["dw_post"], dw_pre=b["dw_pre"], ws=b["ws"], stream=stream, **kw)


def n64(t):
    return None if t is None else to64(t)


def check(b, kind, sigmoid, scale=1.0, eps=1e-6, off=0.0, fwd=True, bwd=True):
    o = bo.block_norm_forward(n64(b["x"]), n64(b["y"]), n64(b["w_post"]), n64(b["w_pre"]),
                              n64(b["gate"]), kind, sigmoid, scale, eps, off)
    if fwd:
        close(b["r"], o["r"], o["mag_r"], "r")
        if b["n"] is not None:
            close(b["n"], o["n"], o["mag_n"], "n")
            close(b["rstd_r"], o["rstd_r"], o["rstd_r"], "rstd_r")
        if b["rstd_y"] is not None:
            close(b["rstd_y"], o["rstd_y"], o["rstd_y"], "rstd_y")
    if not bwd:
        return
    g = bo.block_norm_backward(n64(b["dr"]), n64(b["dn"]), n64(b["r"]), n64(b["y"]),
                               n64(b["w_post"]), n64(b["w_pre"]), n64(b["rstd_y"]),
                               n64(b["rstd_r"]), n64(b["gate"]), kind, sigmoid, scale, off)
    for k in ("dx", "dy", "dgate", "dw_post", "dw_pre"):
        if b[k] is not None:
            tok = k.startswith("dw") or (k == "dgate" and kind == "channel")
            close(b[k], g[k], g["mag_" + k], k, 768 if tok else 256)


SHAPES = [(1, 1), (1, 8), (3, 7), (5, 64), (33, 97), (700, 128), (7, 264), (65, 256), (41, 1001),
          (130, 2048), (9, 2880), (3, 4096), (2, 4104), (2, 5001), (3, 8192), (2, 16384),
          (2, 16383)]


@pytest.mark.parametrize("xt,yt", [(BF, BF), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("T,d", SHAPES)
def test_forward_and_backward(T, d, xt, yt):
    for i, (kind, sigmoid) in enumerate(GATES):
        post, pre = NORMS[(i + T) % 4] if i else (True, True)
        b = make(T, d, xt, yt, kind, post, pre, seed=i)
        kw = dict(scale=0.6, w_offset=0.5 if i % 2 else 0.0)
        forward(b, kind, sigmoid, eps=1e-5, **kw)
        backward(b, kind, sigmoid, **kw)
        check(b, kind, sigmoid, scale=np.float32(0.6).astype(float), eps=1e-5,
              off=kw["w_offset"])
    assert L.moe_status() == L.MOE_OK


@pytest.mark.parametrize("xt,yt", [(BF, BF), (F32, BF), (F32, F32)])
def test_pointers_that_no_vector_fits(xt, yt):
    """d is a multiple of 8, but every buffer begins one value off."""
    def place(shape, dtype):
        n = int(np.prod(shape))
        return torch.empty(n + 1, dtype=dtype, device=DEV)[1:].view(shape)
    for kind, sigmoid in GATES:
        b = make(13, 320, xt, yt, kind, True, True, place=place)
        forward(b, kind, sigmoid)
        backward(b, kind, sigmoid)
        check(b, kind, sigmoid)


def test_many_rows_for_each_block_and_ragged_groups():
    """More rows than blocks times groups, with a last turn that is not full."""
    for T, d in ((5003, 64), (2441, 520), (1217, 2048)):
        b = make(T, d, BF, BF, "channel", True, True)
        forward(b, "channel", True)
        backward(b, "channel", True)
        check(b, "channel", True)


@pytest.mark.parametrize("xt,yt", [(BF, BF), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("T,d,off", [
    (1300, 264, 0), (701, 1000, 0), (641, 2048, 0), (613, 2880, 0), (311, 4104, 0), (333, 8192, 0),
    (1301, 263, 0), (703, 1001, 0), (701, 1002, 0), (640, 2047, 0), (612, 2881, 0), (311, 4103, 0),
    (310, 8191, 0), (641, 2048, 1), (640, 1000, 3), (1217, 261, 5)])
def test_rows_through_the_ring(T, d, off, xt, yt):
    """Enough rows that they come by bulk copies, with a last tile that is not
    full; every gate with every choice of norms; widths and buffers (off values
    past an aligned address) that the copies' 16-byte words do not fit."""
    def place(shape, dtype):
        n = int(np.prod(shape))
        # NaN around each buffer: the words that come along must not matter
        raw = torch.full((n + 2 * off,), float("nan"), dtype=dtype, device=DEV)
        return raw[off:off + n].view(shape)
    for i, (kind, sigmoid) in enumerate(GATES):
        for post, pre in NORMS[:3]:
            b = make(T, d, xt, yt, kind, post, pre, seed=i, place=place)
            forward(b, kind, sigmoid, scale=0.5)
            if i % 2:     # frozen weights and gate
                b["dw_post"] = b["dw_pre"] = None
                b["dgate"] = b["dgate"] if kind in ("token", "element") else None
            backward(b, kind, sigmoid, scale=0.5)
            check(b, kind, sigmoid, scale=0.5)
    # without a residual's gradient, without some outputs
    b = make(T, d, xt, yt, "channel", True, True, place=place)
    forward(b, "channel", True)
    b["dr"] = None
    L.moe_block_norm_bwd(None, b["dn"], b["r"], b["y"], None, b["dy"], w_post=b["w_post"],
                         w_pre=b["w_pre"], rstd_y=b["rstd_y"], rstd_r=b["rstd_r"], gate=b["gate"],
                         gate_kind="channel", gate_sigmoid=True, dgate=b["dgate"], ws=b["ws"])
    b["dx"] = b["dw_post"] = b["dw_pre"] = None
    check(b, "channel", True, fwd=False)
    # the norm of x alone
    L.moe_block_norm_fwd(b["x"], None, None, b["n"], w_pre=b["w_pre"], rstd_r=b["rstd_r"])
    o = bo.block_norm_forward(n64(b["x"]), None, w_pre=n64(b["w_pre"]))
    close(b["n"], o["n"], o["mag_n"], "n")
    assert L.moe_status() == L.MOE_OK


@pytest.mark.parametrize("xt,yt", [(BF, BF), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("T,d,off", [(331, 8200, 0), (330, 12000, 0), (470, 12000, 1), (329, 16383, 0),
                                     (331, 16384, 0)])
def test_wide_rows_over_several_turns(T, d, off, xt, yt):
    """Above 8192 columns (four shares a thread, rows read directly): more rows than
    blocks, so that a block's loop turns, the next row is fetched ahead (or, with too
    many bytes a row, is not) and the column sums gather several rows."""
    def place(shape, dtype):
        n = int(np.prod(shape))
        raw = torch.full((n + 2 * off,), float("nan"), dtype=dtype, device=DEV)
        return raw[off:off + n].view(shape)
    for kind, sigmoid, (post, pre) in (("channel", True, (True, True)), ("element", False, (True, True)),
                                       ("token", True, (True, False)), ("none", False, (False, True))):
        b = make(T, d, xt, yt, kind, post, pre, seed=3, place=place)
        forward(b, kind, sigmoid, scale=0.5)
        backward(b, kind, sigmoid, scale=0.5)
        check(b, kind, sigmoid, scale=0.5)
    assert L.moe_status() == L.MOE_OK


@pytest.mark.parametrize("T,d,off", [(2500, 1001, 1), (3001, 520, 3), (2441, 2047, 0), (1601, 2881, 5)])
def test_the_place_of_the_first_rows_is_filled_again(T, d, off):
    """Rows that 16-byte words do not fit, and more tiles for a block than its ring
    holds: the first tile's first values are stored one by one where later tiles are
    copied to."""
    def place(shape, dtype):
        n = int(np.prod(shape))
        raw = torch.full((n + 2 * off + 8,), float("nan"), dtype=dtype, device=DEV)
        return raw[off:off + n].view(shape)
    for xt, yt in ((BF, BF), (F32, BF), (F32, F32)):
        b = make(T, d, xt, yt, "element", True, True, place=place)
        forward(b, "element", True)
        backward(b, "element", True)
        check(b, "element", True)
    assert L.moe_status() == L.MOE_OK


def test_norm_alone_and_gate_alone():
    # the norm of x alone (fp32 residual stream, bf16 block input), and its gradient
    b = make(50, 384, F32, BF, "none", False, True)
    L.moe_block_norm_fwd(b["x"], None, None, b["n"], w_pre=b["w_pre"], rstd_r=b["rstd_r"])
    o = bo.block_norm_forward(n64(b["x"]), None, w_pre=n64(b["w_pre"]))
    close(b["n"], o["n"], o["mag_n"], "n")
    L.moe_block_norm_bwd(b["dr"], b["dn"], b["x"], None, b["dx"], w_pre=b["w_pre"],
                         rstd_r=b["rstd_r"], dw_pre=b["dw_pre"], ws=b["ws"])
    g = bo.block_norm_backward(n64(b["dr"]), n64(b["dn"]), n64(b["x"]), None, w_pre=n64(b["w_pre"]),
                               rstd_r=n64(b["rstd_r"]))
    close(b["dx"], g["dx"], g["mag_dx"], "dx")
    close(b["dw_pre"], g["dw_pre"], g["mag_dw_pre"], "dw_pre", 768)
    # without the residual: r = scale sigmoid(gate) y, a shared expert's token gate
    b = make(50, 384, BF, BF, "token", False, False)
    L.moe_block_norm_fwd(None, b["y"], b["r"], gate=b["gate"], gate_kind="token",
                         gate_sigmoid=True)
    o = bo.block_norm_forward(None, n64(b["y"]), gate=n64(b["gate"]), kind="token", sigmoid=True)
    close(b["r"], o["r"], o["mag_r"], "r")
    # only dy and dgate are wanted; no dr comes back (dn alone)
    c = make(50, 384, BF, BF, "token", False, True)
    forward(c, "token", True)
    L.moe_block_norm_bwd(None, c["dn"], c["r"], c["y"], None, c["dy"], w_pre=c["w_pre"],
                         rstd_r=c["rstd_r"], gate=c["gate"], gate_kind="token", gate_sigmoid=True,
                         dgate=c["dgate"])
    g = bo.block_norm_backward(None, n64(c["dn"]), n64(c["r"]), n64(c["y"]), w_pre=n64(c["w_pre"]),
                               rstd_r=n64(c["rstd_r"]), gate=n64(c["gate"]), kind="token",
                               sigmoid=True)
    close(c["dy"], g["dy"], g["mag_dy"], "dy")
    close(c["dgate"], g["dgate"], g["mag_dgate"], "dgate")


def test_in_place_equals_out_of_place():
    for T, d in ((77, 2048), (77, 1001), (650, 2048), (330, 4096), (700, 1001)):
        b = make(T, d, BF, BF, "element", True, True)
        forward(b, "element", False)
        backward(b, "element", False)
        torch.cuda.synchronize()
        x, y, dr, dn = (b[k].clone() for k in ("x", "y", "dr", "dn"))
        L.moe_block_norm_fwd(x, y, x, y, w_post=b["w_post"], w_pre=b["w_pre"],
                             rstd_y=b["rstd_y"], rstd_r=b["rstd_r"], gate=b["gate"],
                             gate_kind="element")
        L.moe_block_norm_bwd(dr, dn, b["r"], b["y"], dr, dn, w_post=b["w_post"], w_pre=b["w_pre"],
                             rstd_y=b["rstd_y"], rstd_r=b["rstd_r"], gate=b["gate"],
                             gate_kind="element")
        assert torch.equal(x, b["r"]) and torch.equal(y, b["n"])
        assert torch.equal(dr, b["dx"]) and torch.equal(dn, b["dy"])


def test_rows_of_zeros_and_extreme_gates():
    b = make(6, 256, F32, F32, "channel", True, True)
    b["y"][2] = 0
    b["x"][2] = 0
    b["gate"][:4] = torch.tensor([100.0, -100.0, float("inf"), float("-inf")], device=DEV)
    forward(b, "channel", True)
    backward(b, "channel", True)
    for k in ("r", "n", "dx", "dy", "dgate", "dw_post", "dw_pre"):
        assert torch.isfinite(b[k]).all(), k
    assert torch.all(b["r"][2] == 0) and torch.all(b["n"][2] == 0)
    check(b, "channel", True)


@pytest.mark.parametrize("d", [512, 1001, 2048])
def test_a_row_with_nan_spoils_no_other_row(d):
    T = 40 if d < 1000 else 640
    b = make(T, d, BF, BF, "token", True, True)
    forward(b, "token", False)
    backward(b, "token", False)
    ref = {k: b[k].clone() for k in ("r", "n", "dx", "dy", "dgate")}
    b["y"][7, 3] = float("nan")
    b["x"][9, 300] = float("inf")
    forward(b, "token", False)
    backward(b, "token", False)
    keep = [t for t in range(T) if t not in (7, 9)]
    for k in ref:
        assert torch.equal(b[k][keep], ref[k][keep]), k
    assert torch.isnan(b["n"][7].float()).all()


def test_no_tokens():
    b = make(0, 64, BF, BF, "channel", True, True)
    for k in ("dgate", "dw_post", "dw_pre"):
        b[k].fill_(7.0)
    forward(b, "channel", False)
    backward(b, "channel", False)
    for k in ("dgate", "dw_post", "dw_pre"):
        assert torch.all(b[k] == 0), k


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_no_tokens_beside_gates_and_weights_that_are_not_finite(value):
    """The sums over no tokens are zeros whatever they would be multiplied with."""
    for sigmoid in (False, True):
        b = make(0, 64, BF, BF, "channel", True, True)
        b["gate"].fill_(value)
        b["w_post"].fill_(value)
        for k in ("dgate", "dw_post", "dw_pre"):
            b[k].fill_(7.0)
        backward(b, "channel", sigmoid)
        for k in ("dgate", "dw_post", "dw_pre"):
            assert torch.all(b[k] == 0), k


def test_equal_inputs_give_equal_bits_on_another_stream_and_in_a_graph():
    b = make(1500, 1024, BF, BF, "channel", True, True)
    forward(b, "channel", True)
    backward(b, "channel", True)
    names = ("r", "n", "dx", "dy", "dgate", "dw_post", "dw_pre")
    ref = {k: b[k].clone() for k in names}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for k in names:
        b[k].zero_()
    s.wait_stream(torch.cuda.current_stream())
    forward(b, "channel", True, stream=s)
    backward(b, "channel", True, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for k in names:
        assert torch.equal(b[k], ref[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward(b, "channel", True)
        backward(b, "channel", True)
    for k in names:
        b[k].zero_()
    graph.replay()
    for k in names:
        assert torch.equal(b[k], ref[k]), k


def test_gradient_against_differences_of_the_kernel():
    """Along a random direction in every input: (L(+h) - L(-h)) / 2h against the
    gradient, L summed in 64 bits from fp32 outputs.  With h = 2^-6 and entries
    near 1 the third-order term is about h^2 = 2.4e-4 of the curvature terms and
    the outputs' roundings give 2^-24 sqrt(T d) / h; 2e-3 of the sum of the
    directions' sizes covers both."""
    kind, h = "channel", 2.0 ** -6
    b = make(64, 192, F32, F32, kind, True, True)
    forward(b, kind, True)
    backward(b, kind, True)
    grads = {"x": b["dx"], "y": b["dy"], "gate": b["dgate"], "w_post": b["dw_post"],
             "w_pre": b["dw_pre"]}
    for name, grad in grads.items():
        base = b[name].clone()
        v = torch.randn_like(base) * 0.2
        vals = []
        for sign in (1, -1):
            b[name].copy_(base + sign * h * v)
            forward(b, kind, True)
            vals.append(float((b["r"].double() * b["dr"].double()).sum()
                              + (b["n"].double() * b["dn"].double()).sum()))
        b[name].copy_(base)
        num = (vals[0] - vals[1]) / (2 * h)
        ana = float((grad.double() * v.double()).sum())
        size = float((grad.double() * v.double()).square().sum().sqrt())
        assert abs(num - ana) <= 2e-3 * max(size, abs(ana)) * 8 ** 0.5, (name, num, ana, size)


def test_offsets_past_32_bits():
    """T d above 2^31: the last rows are right."""
    T, d = 1_050_000, 2056
    assert T * d > 2 ** 31
    x = torch.zeros(T, d, dtype=BF, device=DEV)
    n = torch.empty_like(x)
    w = torch.randn(d, device=DEV)
    rs = torch.empty(T, device=DEV)
    x[-5:] = torch.randn(5, d, device=DEV).to(BF)
    L.moe_block_norm_fwd(x, None, None, n, w_pre=w, rstd_r=rs)
    o = bo.block_norm_forward(to64(x[-5:]), None, w_pre=to64(w))
    close(n[-5:], o["n"], o["mag_n"], "n")
    dx = torch.full_like(x, 3.0)
    L.moe_block_norm_bwd(None, n, x, None, dx, w_pre=w, rstd_r=rs)
    g = bo.block_norm_backward(None, to64(n[-5:]), to64(x[-5:]), None, w_pre=to64(w),
                               rstd_r=to64(rs[-5:]))
    close(dx[-5:], g["dx"], g["mag_dx"], "dx")
    assert torch.all(dx[:100] == 0)


def test_nothing_is_written_past_a_buffer():
    bands = []

    def place(shape, dtype):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        raw = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=DEV)
        bands.append((raw, n))
        return raw[256:256 + n].view(dtype).view(shape)
    for T, d in ((9, 96), (311, 1001), (17, 2880), (5, 4104), (650, 2048), (320, 4104), (701, 1001), (311, 4103)):
        for kind in ("token", "channel", "element"):
            b = make(T, d, BF, BF, kind, True, True, place=place)
            raw = torch.full((b["ws"].numel() + 512,), 0xA5, dtype=torch.uint8, device=DEV)
            bands.append((raw, b["ws"].numel()))
            b["ws"] = raw[256:256 + b["ws"].numel()]
            forward(b, kind, True)
            backward(b, kind, True)
    torch.cuda.synchronize()
    for raw, n in bands:
        assert torch.all(raw[:256] == 0xA5) and torch.all(raw[256 + n:] == 0xA5)


def test_refusals_of_tensors():
    b = make(8, 64, BF, BF, "none", True, True)
    with pytest.raises(ValueError, match="contiguous"):
        L.moe_block_norm_fwd(b["x"].t().contiguous().t(), b["y"], b["r"])
    with pytest.raises(ValueError, match="shape"):
        L.moe_block_norm_fwd(b["x"], b["y"][:4], b["r"])
    with pytest.raises(ValueError, match="float32 or"):
        L.moe_block_norm_fwd(b["x"].half(), b["y"].half(), b["r"].half())
    with pytest.raises(ValueError, match="go together"):
        L.moe_block_norm_fwd(b["x"], b["y"], b["r"], gate_kind="token")
    with pytest.raises(L.MoeError, match="r is NULL"):
        L.moe_block_norm_fwd(b["x"], b["y"])
    with pytest.raises(L.MoeError, match="eps"):
        L.moe_block_norm_fwd(b["x"], b["y"], b["r"], eps=0.0)
    with pytest.raises(L.MoeError, match="needs a bf16"):
        L.moe_block_norm_fwd(b["x"], b["y"].float(), b["r"])
    with pytest.raises(L.MoeError, match="workspace"):
        forward(b, "none", False)
        b["ws"] = torch.empty(16, dtype=torch.uint8, device=DEV)
        backward(b, "none", False)
