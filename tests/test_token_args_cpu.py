"""Host-side argument checks of embedding, log probabilities and checkpoints:
error codes before anything is launched (no GPU needed; pointers are never
dereferenced)."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
A = P(1 << 20)          # aligned
ODD = P((1 << 20) + 1)  # aligned for nothing


@pytest.fixture(scope="module")
def L():
    from expert_routing_grouped_moe_gb300 import build, _lib
    build.build()
    _lib.load()
    return _lib


def embed(L, **kw):
    base = dict(T=4, V=10, d=64, id_type=3, table_type=1, row_type=1, scale=1.0)
    base.update(kw)
    return ctypes.byref(L.MoeEmbedDesc(**base))


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(V=0), -1), (dict(d=0), -1), (dict(d=(1 << 20) + 1), -2), (dict(id_type=0), -1),
    (dict(id_type=1), -1), (dict(table_type=2), -1), (dict(row_type=-1), -1), (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1)])
def test_embed_descriptor(L, kw, code):
    lib = L.load()
    assert lib.moe_embed_fwd(embed(L, **kw), A, A, A, None) == code
    assert lib.moe_embed_bwd(embed(L, **kw), A, A, A, -1, 0, A, 1 << 40, None) == code
    assert lib.moe_last_error()


@pytest.mark.parametrize("bad", [None, ODD])
def test_embed_pointers(L, bad):
    lib = L.load()
    for i in range(3):
        args = [A, A, A]
        args[i] = bad
        assert lib.moe_embed_fwd(embed(L), *args, None) == L.MOE_ERR_INVALID_ARG
        assert lib.moe_embed_bwd(embed(L), *args, -1, 0, A, 1 << 40, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_embed_bwd(embed(L), A, A, A, -1, 0, bad, 1 << 40, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_embed_bwd(embed(L), A, A, A, -1, 2, A, 1 << 40, None) == L.MOE_ERR_INVALID_ARG
    assert lib.moe_embed_bwd(None, A, A, A, -1, 0, A, 1 << 40, None) == L.MOE_ERR_INVALID_ARG
    # 32-bit ids on a 4-byte boundary are fine, 64-bit ones are not
    four = P((1 << 20) + 4)
    assert lib.moe_embed_fwd(embed(L), four, A, A, None) == L.MOE_ERR_INVALID_ARG


def test_embed_workspace(L):
    lib = L.load()
    n = L.moe_embed_workspace_size(5000, 1000, 64)
    assert n >= 5000 * 4
    assert lib.moe_embed_bwd(embed(L, T=5000, V=1000), A, A, A, -1, 0, A, n - 1, None) == L.MOE_ERR_WORKSPACE
    assert L.moe_embed_workspace_size(0, 1000, 64) == 0
    assert L.moe_embed_workspace_size(4, 0, 64) == 0 and L.moe_embed_workspace_size(4, 10, 1 << 21) == 0
    with pytest.raises(ValueError):
        L.moe_embed_workspace_size(1 << 31, 10, 64)


def logprob(L, **kw):
    base = dict(T=4, V=100, m=1, top=0, type=1, target_type=3, ld=100, dld=100, ignore_id=-100, inv_temp=1.0)
    base.update(kw)
    return ctypes.byref(L.MoeLogprobDesc(**base))


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(V=0), -1), (dict(V=0x7FFFFFFF, ld=1 << 40, dld=1 << 40), -2), (dict(type=2), -1),
    (dict(target_type=0), -1), (dict(m=0), -1), (dict(m=65), -1), (dict(top=-1), -1), (dict(top=33), -1),
    (dict(ld=99), -1), (dict(inv_temp=0.0), -1), (dict(inv_temp=-1.0), -1), (dict(inv_temp=float("inf")), -1),
    (dict(inv_temp=float("nan")), -1), (dict(T=1 << 29), -2)])
def test_logprob_descriptor(L, kw, code):
    lib = L.load()
    assert lib.moe_logprob_fwd(logprob(L, **kw), A, A, A, A, A, A, A, A, None) == code
    assert lib.moe_logprob_bwd(logprob(L, **kw), A, A, A, A, A, A, A, A, None) == code
    assert lib.moe_logprob_step(logprob(L, **kw), *[A] * 12, None) == code


def test_logprob_pointers(L):
    lib, bad = L.load(), L.MOE_ERR_INVALID_ARG
    q = logprob(L, top=3)
    for miss in (None, ODD):
        for i in range(8):
            args = [A] * 8
            args[i] = miss
            if miss is not None or i < 4:
                assert lib.moe_logprob_fwd(q, *args, None) == bad, (miss, i)
        for i in range(8):      # logits, targets, stats, entropy, dlogp, dentropy, dlse, dlogits
            args = [A] * 8
            args[i] = miss
            if miss is not None or i in (0, 1, 2, 3, 7):
                assert lib.moe_logprob_bwd(q, *args, None) == bad, (miss, i)
        for i in range(12):
            args = [A] * 12     # logits, targets, dlogp, dentropy, dlse, logp, stats, ..., dlogits
            args[i] = miss
            if miss is not None or i in (0, 1, 5, 6, 11):
                assert lib.moe_logprob_step(q, *args, None) == bad, (miss, i)
    # alternatives without a number of them; a row stride of the gradient below V
    assert lib.moe_logprob_fwd(logprob(L), A, A, A, A, None, None, A, None, None) == bad
    assert lib.moe_logprob_bwd(logprob(L, dld=99), A, A, A, A, A, A, A, P(1 << 30), None) == bad
    # in place needs the same row stride
    assert lib.moe_logprob_bwd(logprob(L, dld=104), A, A, A, A, A, A, A, A, None) == bad


def test_ckpt(L):
    lib, bad = L.load(), L.MOE_ERR_INVALID_ARG
    for x_type in (-1, 2):
        assert lib.moe_ckpt_pack(A, x_type, 4, 64, A, A, None) == bad
        assert lib.moe_ckpt_unpack(A, A, 4, 64, A, x_type, None) == bad
    for R, C in ((-1, 64), (4, 0), (4, -3)):
        assert lib.moe_ckpt_pack(A, 0, R, C, A, A, None) == bad
        assert lib.moe_ckpt_unpack(A, A, R, C, A, 0, None) == bad
    assert lib.moe_ckpt_pack(None, 0, 4, 64, A, A, None) == bad
    assert lib.moe_ckpt_pack(ODD, 1, 4, 64, A, A, None) == bad
    assert lib.moe_ckpt_pack(A, 0, 4, 64, None, A, None) == bad
    assert lib.moe_ckpt_unpack(A, None, 4, 64, A, 0, None) == bad
    for kw in (dict(P=-1), dict(f=0), dict(f=12), dict(k=0), dict(k=33), dict(shared=2)):
        a = dict(dict(P=4, f=64, k=2, shared=0), **kw)
        assert lib.moe_ckpt_unpack_swiglu(A, A, a["P"], a["f"], A, A, a["k"], a["shared"], A, A, None) == bad
    for i in range(6):
        for miss in (None, ODD):
            args = [A] * 6          # codes, scales, sorted_src, topk_w, h, act
            args[i] = miss
            if miss is ODD and i == 1:
                continue            # bytes
            assert lib.moe_ckpt_unpack_swiglu(args[0], args[1], 4, 64, args[2], args[3], 2, 0, args[4],
                                              args[5], None) == bad


@pytest.mark.parametrize("P,k,shared", [(5, 2, 0), (8, 2, 1), (1, 1, 1)])
def test_rows_that_are_not_whole_tokens(L, P, k, shared):
    """P rows are T tokens' k slots (and shared one): the last weight read is topk_w[T - 1]."""
    assert L.load().moe_ckpt_unpack_swiglu(A, A, P, 64, A, A, k, shared, A, A, None) == L.MOE_ERR_INVALID_ARG


def test_nothing_to_do_is_no_error(L):
    lib = L.load()
    assert lib.moe_embed_fwd(embed(L, T=0), None, None, None, None) == L.MOE_OK
    assert lib.moe_logprob_fwd(logprob(L, T=0), *[None] * 8, None) == L.MOE_OK
    assert lib.moe_logprob_bwd(logprob(L, T=0), *[None] * 8, None) == L.MOE_OK
    assert lib.moe_logprob_step(logprob(L, T=0), *[None] * 12, None) == L.MOE_OK
    assert lib.moe_ckpt_pack(None, 0, 0, 64, None, None, None) == L.MOE_OK
    assert lib.moe_ckpt_unpack(None, None, 0, 64, None, 0, None) == L.MOE_OK
    assert lib.moe_ckpt_unpack_swiglu(None, None, 0, 64, None, None, 2, 0, None, None, None) == L.MOE_OK


def test_bindings_refuse_before_the_library(L):
    """CPU tensors, missing tensors, other shapes and types."""
    i, w, o = torch.zeros(3, dtype=torch.int64), torch.zeros(5, 8), torch.zeros(3, 8)
    for args in ((i, w, o), (i.float(), w, o), (None, w, o), (i, None, o), (i, w, None), (i, w[0], o)):
        with pytest.raises((ValueError, TypeError)):
            L.moe_embed_fwd(*args)
        with pytest.raises((ValueError, TypeError)):
            L.moe_embed_bwd(args[0], args[2], args[1], torch.zeros(64, dtype=torch.uint8))
    with pytest.raises(ValueError):
        L.moe_embed_bwd(i, o, w, None, pad_id=-3)
    x, y, z = torch.zeros(3, 9), torch.zeros(3, dtype=torch.int64), torch.zeros(3)
    for args in ((x, y, z, torch.zeros(3, 2)), (None, y, z, z), (x, z, z, z), (x, None, z, z)):
        with pytest.raises((ValueError, TypeError)):
            L.moe_logprob_fwd(*args)
        with pytest.raises((ValueError, TypeError)):
            L.moe_logprob_bwd(args[0], args[1], args[3], z, x)
        with pytest.raises((ValueError, TypeError)):
            L.moe_logprob_step(*args, z, x)
    with pytest.raises(TypeError):
        L.moe_logprob_bwd(x, y, z, z, None)
    with pytest.raises(TypeError):
        L.moe_logprob_step(x, y, z, z, z, None)
    c, s = torch.zeros(3, 9, dtype=torch.int8), torch.zeros(3, 1, dtype=torch.uint8)
    for args in ((x, c, s), (None, c, s), (x[0], c, s), (x.half(), c, s)):
        with pytest.raises((ValueError, TypeError)):
            L.moe_ckpt_pack(*args)
        with pytest.raises((ValueError, TypeError)):
            L.moe_ckpt_unpack(args[1], args[2], args[0])


def test_scratch():
    """Views of one buffer a name; a larger user's replaces it, and both count; a user of another
    device is refused before anything is kept."""
    from expert_routing_grouped_moe_gb300 import LayerScratch
    s = LayerScratch("cpu")
    a, b = s.take("h", (3, 8), torch.float32, "cpu"), s.take("h", (5, 4), torch.bfloat16)
    assert a.shape == (3, 8) and b.shape == (5, 4) and a.data_ptr() == b.data_ptr() and s.bytes() == 96
    c, d = s.take("h", (100,), torch.float32), s.take("h", (2, 8), torch.float32)
    assert d.data_ptr() == c.data_ptr() != a.data_ptr() and s.bytes() == 96 + 400
    a.fill_(1)
    c.fill_(2)
    assert (a == 1).all()
    for name, n in (("h", 4), ("h", 1000), ("new", 4)):
        with pytest.raises(ValueError):
            s.take(name, (n,), torch.float32, "meta")
    assert s.bytes() == 96 + 400 and s.take("h", (100,), torch.float32).data_ptr() == c.data_ptr()
