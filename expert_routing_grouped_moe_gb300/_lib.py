"""ctypes binding of the C ABI in ``include/moe_gb300.h``.

Argument marshalling only: every function takes torch CUDA tensors (device
memory) and an optional ``torch.cuda.Stream`` and forwards raw pointers to
the library of the same name.  No arithmetic of the layer happens here.  If
the compiled library is missing the calls raise; there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libmoe_gb300.so")
TILE_M = 128

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_WORKSPACE = -3
MOE_ERR_CUDA = -4
MOE_ERR_BAD_IDS = -5
MOE_ERR_TIMEOUT = -6
MOE_PROBE_LINEAR = 0
MOE_PROBE_TILES = 1
MOE_F32 = 0
MOE_BF16 = 1
MOE_NORM_MAX_D = 16384
MOE_ADAMW_BLOCK = 256
GATE_KINDS = {"none": 0, "token": 1, "channel": 2, "element": 3}

EXPORTED = (
    "moe_router_topk", "moe_route_workspace_size", "moe_route",
    "moe_permute", "moe_unpermute_combine", "moe_lora_grouped_mlp_fwd",
    "moe_mlp_bwd_workspace_size", "moe_lora_grouped_mlp_bwd", "moe_status",
    "moe_last_error", "moe_abi_version", "moe_kernel_name", "moe_probe_arm", "moe_probe_count",
    "moe_route_noalloc", "moe_selftest_wait_timeout", "moe_probe_read_stream",
    "moe_route_kernel_count", "moe_ep_row_weights", "moe_ep_segment_ids", "moe_route_logits",
    "moe_block_norm_fwd", "moe_block_norm_workspace_size", "moe_block_norm_bwd",
    "moe_router_loss_workspace_size", "moe_router_loss_fwd", "moe_router_bwd",
    "moe_adamw_workspace_size", "moe_adamw_step", "moe_selftest_ring_timeout",
)


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str, msg: str):
        super().__init__("%s failed (%d): %s" % (where, code, msg))
        self.code = code


class MoeDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("f", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("r", ctypes.c_int32),
                ("lora_scale", ctypes.c_float), ("shared_expert", ctypes.c_int32)]

    @property
    def G(self):
        return self.E + self.shared_expert

    @property
    def K(self):
        return self.k + self.shared_expert


_lock = threading.Lock()
_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int32
_F = ctypes.c_float
_D = ctypes.c_double
_SZ = ctypes.c_size_t


class MoeNormDesc(ctypes.Structure):
    _fields_ = [("T", _I), ("d", _I), ("x_type", _I), ("y_type", _I), ("gate", _I),
                ("gate_sigmoid", _I), ("scale", _F), ("eps", _F), ("w_offset", _F)]


class MoeAdamWTensor(ctypes.Structure):
    _fields_ = [("param", _P), ("master", _P), ("grad", _P), ("m", _P), ("v", _P),
                ("scales", _P), ("n", ctypes.c_int64), ("param_type", _I), ("grad_type", _I),
                ("state_bits", _I), ("lr_mult", _F), ("weight_decay", _F)]


class MoeAdamWHyper(ctypes.Structure):
    _fields_ = [("lr", _D), ("beta1", _D), ("beta2", _D), ("eps", _D), ("step", ctypes.c_int64),
                ("grad_scale", _F), ("max_norm", _F), ("skip_nonfinite", _I)]


def load(path: str = LIB_PATH):
    """Load the compiled library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError("MoE CUDA library not built (%s); run "
                               "expert_routing_grouped_moe_gb300.build.build()" % path)
        lib = ctypes.CDLL(path)
        sig = {
            "moe_router_topk": (ctypes.c_int, [_P, _I, _I, _I, _P, _P, _P]),
            "moe_route_workspace_size": (_SZ, [_I, _I, _I]),
            "moe_route": (ctypes.c_int, [_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
            "moe_permute": (ctypes.c_int, [_P, _I, _I, _I, _P, _P, _P]),
            "moe_unpermute_combine": (ctypes.c_int, [_P, _P, _I, _I, _I, _I, _P, _P, _P, _P,
                                                     _P]),
            "moe_lora_grouped_mlp_fwd": (ctypes.c_int, [ctypes.POINTER(MoeDims)] + [_P] * 19),
            "moe_mlp_bwd_workspace_size": (_SZ, [ctypes.POINTER(MoeDims)]),
            "moe_lora_grouped_mlp_bwd": (ctypes.c_int, [ctypes.POINTER(MoeDims)] + [_P] * 28
                                         + [_SZ, _P]),
            "moe_status": (ctypes.c_int, [_P]),
            "moe_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_uint32, _P]),
            "moe_last_error": (ctypes.c_char_p, []),
            "moe_abi_version": (ctypes.c_int, []),
            "moe_kernel_name": (ctypes.c_char_p, [_I]),
            "moe_probe_arm": (ctypes.c_int, [ctypes.c_char_p, ctypes.POINTER(_P),
                                             ctypes.POINTER(_P), _I]),
            "moe_probe_count": (_I, [ctypes.c_char_p]),
            "moe_route_noalloc": (ctypes.c_int, [_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
            "moe_selftest_ring_timeout": (ctypes.c_int, [ctypes.c_uint32, _I, _P, _P]),
            "moe_probe_read_stream": (ctypes.c_int, [_P, _SZ, _I, _P]),
            "moe_route_kernel_count": (_I, [_I, _I, _I]),
            "moe_ep_row_weights": (ctypes.c_int, [_P, _P, _I, _I, _I, _P, _P]),
            "moe_route_logits": (ctypes.c_int, [_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P,
                                                _P, _SZ, _P]),
            "moe_ep_segment_ids": (ctypes.c_int, [_P, _I, _I, ctypes.c_int64, _P, _P]),
            "moe_block_norm_fwd": (ctypes.c_int, [ctypes.POINTER(MoeNormDesc)] + [_P] * 10),
            "moe_block_norm_workspace_size": (_SZ, [_I, _I]),
            "moe_block_norm_bwd": (ctypes.c_int, [ctypes.POINTER(MoeNormDesc)] + [_P] * 15
                                   + [_SZ, _P]),
            "moe_router_loss_workspace_size": (_SZ, [_I, _I]),
            "moe_router_loss_fwd": (ctypes.c_int, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P]),
            "moe_router_bwd": (ctypes.c_int, [_P, _P, _I, _I, _I, _P, _P, _P, _P, _F, _F, _P,
                                              _P]),
            "moe_adamw_workspace_size": (_SZ, [ctypes.POINTER(MoeAdamWTensor), _I]),
            "moe_adamw_step": (ctypes.c_int, [ctypes.POINTER(MoeAdamWTensor), _I,
                                              ctypes.POINTER(MoeAdamWHyper), _P, _P, _SZ, _P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _check(rc: int, where: str):
    if rc != MOE_OK:
        msg = load().moe_last_error().decode(errors="replace")
        raise MoeError(rc, where, msg)


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return t.data_ptr()


def _bf(t, name):
    return _ptr(t, torch.bfloat16, name)


def _i32(t, name):
    return _ptr(t, torch.int32, name)


def _f32(t, name):
    return _ptr(t, torch.float32, name)


try:   # the current stream's handle without building a Stream object (3 us a call)
    from torch._C import _cuda_getCurrentRawStream as _raw_stream, _cuda_getDevice as _device
except ImportError:
    _raw_stream = None


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and torch.cuda.is_initialized():
        return _raw_stream(_device())
    return torch.cuda.current_stream().cuda_stream


def make_dims(T, d, f, E, k, r, lora_scale, shared_expert=False) -> MoeDims:
    return MoeDims(int(T), int(d), int(f), int(E), int(k), int(r), float(lora_scale),
                   1 if shared_expert else 0)


# ---------------------------------------------------------------- C ABI calls

def moe_router_topk(logits, k, ids, weights, stream=None):
    T, E = logits.shape
    _check(load().moe_router_topk(_f32(logits, "logits"), T, E, int(k), _i32(ids, "ids"),
                                  _f32(weights, "weights"), _stream(stream)), "moe_router_topk")


def moe_probe_read_stream(buf, pattern=0, stream=None):
    """Stream the bytes of a device tensor into shared memory (measurement);
    pattern MOE_PROBE_LINEAR or MOE_PROBE_TILES."""
    _check(load().moe_probe_read_stream(_ptr(buf, name="buf"), buf.numel() * buf.element_size(),
                                        int(pattern), _stream(stream)), "moe_probe_read_stream")


def moe_route_kernel_count(T, K, G) -> int:
    """Kernels moe_route launches for this shape (2 or 3)."""
    n = int(load().moe_route_kernel_count(int(T), int(K), int(G)))
    _check(n if n < 0 else MOE_OK, "moe_route_kernel_count")
    return n


def moe_route_workspace_size(T, K, G) -> int:
    return int(load().moe_route_workspace_size(int(T), int(K), int(G)))


def moe_route(ids, E, shared_expert, counts, offsets, tile_off, sorted_src, dest_pos, ws,
              stream=None):
    T, k = ids.shape
    _check(load().moe_route(_i32(ids, "ids"), T, k, int(E), 1 if shared_expert else 0,
                            _i32(counts, "counts"), _i32(offsets, "offsets"),
                            _i32(tile_off, "tile_off"), _i32(sorted_src, "sorted_src"),
                            _i32(dest_pos, "dest_pos"), _ptr(ws, name="ws"),
                            ws.numel() * ws.element_size(), _stream(stream)), "moe_route")


def moe_route_logits(logits, k, shared_expert, ids, weights, counts, offsets, tile_off,
                     sorted_src, dest_pos, ws, stream=None):
    """moe_router_topk then moe_route in one call (ids, weights written)."""
    T, E = logits.shape
    _check(load().moe_route_logits(
        _f32(logits, "logits"), T, E, int(k), 1 if shared_expert else 0, _i32(ids, "ids"),
        _f32(weights, "weights"), _i32(counts, "counts"), _i32(offsets, "offsets"),
        _i32(tile_off, "tile_off"), _i32(sorted_src, "sorted_src"), _i32(dest_pos, "dest_pos"),
        _ptr(ws, name="ws"), ws.numel() * ws.element_size(), _stream(stream)),
        "moe_route_logits")


def moe_route_noalloc(ids, E, shared_expert, counts, offsets, tile_off, sorted_src, dest_pos,
                      stream=None):
    """moe_route with its scratch inside the library (no workspace argument)."""
    T, k = ids.shape
    _check(load().moe_route_noalloc(_i32(ids, "ids"), T, k, int(E), 1 if shared_expert else 0,
                                    _i32(counts, "counts"), _i32(offsets, "offsets"),
                                    _i32(tile_off, "tile_off"), _i32(sorted_src, "sorted_src"),
                                    _i32(dest_pos, "dest_pos"), _stream(stream)),
           "moe_route_noalloc")


def moe_permute(src, K, dest_pos, dst, stream=None):
    T, d = src.shape
    _check(load().moe_permute(_bf(src, "src"), T, d, int(K), _i32(dest_pos, "dest_pos"),
                              _bf(dst, "dst"), _stream(stream)), "moe_permute")


def moe_unpermute_combine(rows, dest_pos, k, shared_expert, out, weights=None, row_scalars=None,
                          slot_out=None, stream=None):
    T, d = out.shape
    _check(load().moe_unpermute_combine(
        _bf(rows, "rows"), _i32(dest_pos, "dest_pos"), T, d, int(k), 1 if shared_expert else 0,
        _f32(weights, "weights"), _f32(row_scalars, "row_scalars"), _f32(slot_out, "slot_out"),
        _bf(out, "out"), _stream(stream)), "moe_unpermute_combine")


def moe_lora_grouped_mlp_fwd(dims: MoeDims, Xp, X, counts, offsets, tile_off, sorted_src, topk_w,
                             W_gu, A_gu, B_gu, W_dn, A_dn, B_dn, Yp, h, act, xa_gu, xa_dn,
                             stream=None):
    """Pass the permuted rows Xp, or Xp=None and the token rows X (gathered)."""
    _check(load().moe_lora_grouped_mlp_fwd(
        ctypes.byref(dims), _bf(Xp, "Xp"), _bf(X, "X"), _i32(counts, "counts"),
        _i32(offsets, "offsets"),
        _i32(tile_off, "tile_off"), _i32(sorted_src, "sorted_src"), _f32(topk_w, "topk_w"),
        _bf(W_gu, "W_gu"), _bf(A_gu, "A_gu"), _bf(B_gu, "B_gu"), _bf(W_dn, "W_dn"),
        _bf(A_dn, "A_dn"), _bf(B_dn, "B_dn"), _bf(Yp, "Yp"), _f32(h, "h"), _bf(act, "act"),
        _bf(xa_gu, "xa_gu"), _bf(xa_dn, "xa_dn"), _stream(stream)), "moe_lora_grouped_mlp_fwd")


def moe_mlp_bwd_workspace_size(dims: MoeDims) -> int:
    return int(load().moe_mlp_bwd_workspace_size(ctypes.byref(dims)))


def moe_lora_grouped_mlp_bwd(dims: MoeDims, dYp, dY, Xp, X, counts, offsets, tile_off,
                             sorted_src, topk_w, W_gu, A_gu, B_gu, W_dn, A_dn, B_dn, h, act,
                             xa_gu, xa_dn, dXp, dw_rows, dA_gu, dB_gu, dA_dn, dB_dn, ws,
                             stream=None, dW_gu=None, dW_dn=None):
    """Pass permuted rows (dYp, Xp) or None and the token rows (dY, X).
    dW_gu [G,2f,d] / dW_dn [G,d,f] fp32: optional full weight gradients."""
    _check(load().moe_lora_grouped_mlp_bwd(
        ctypes.byref(dims), _bf(dYp, "dYp"), _bf(dY, "dY"), _bf(Xp, "Xp"), _bf(X, "X"),
        _i32(counts, "counts"),
        _i32(offsets, "offsets"), _i32(tile_off, "tile_off"), _i32(sorted_src, "sorted_src"),
        _f32(topk_w, "topk_w"), _bf(W_gu, "W_gu"), _bf(A_gu, "A_gu"), _bf(B_gu, "B_gu"),
        _bf(W_dn, "W_dn"), _bf(A_dn, "A_dn"), _bf(B_dn, "B_dn"), _f32(h, "h"), _bf(act, "act"),
        _bf(xa_gu, "xa_gu"), _bf(xa_dn, "xa_dn"), _bf(dXp, "dXp"), _f32(dw_rows, "dw_rows"),
        _f32(dA_gu, "dA_gu"), _f32(dB_gu, "dB_gu"), _f32(dA_dn, "dA_dn"), _f32(dB_dn, "dB_dn"),
        _f32(dW_gu, "dW_gu"), _f32(dW_dn, "dW_dn"),
        _ptr(ws, name="ws"), ws.numel() * ws.element_size(), _stream(stream)),
        "moe_lora_grouped_mlp_bwd")


def moe_ep_row_weights(topk_w, dest_pos, shared_expert, row_w, stream=None):
    """row_w[dest_pos[t*K + j]] = topk_w[t, j] (1 for the shared slot)."""
    T, k = topk_w.shape
    _check(load().moe_ep_row_weights(_f32(topk_w, "topk_w"), _i32(dest_pos, "dest_pos"), T, k,
                                     1 if shared_expert else 0, _f32(row_w, "row_w"),
                                     _stream(stream)), "moe_ep_row_weights")


def moe_ep_segment_ids(counts, ids, stream=None):
    """ids[i] = local expert of received row i, for counts [P, E_loc]."""
    P, E_loc = counts.shape
    _check(load().moe_ep_segment_ids(_i32(counts, "counts"), P, E_loc, ids.numel(),
                                     _i32(ids, "ids") if ids.numel() else None, _stream(stream)),
           "moe_ep_segment_ids")


# ------------------------------------------------- norms, router losses, optimizer

_TYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}


def _type(dtype, name):
    code = _TYPES.get(dtype)
    if code is None:
        raise ValueError("%s must be torch.float32 or torch.bfloat16, got %s" % (name, dtype))
    return code


def _shaped(t, shape, dtype, name):
    """Pointer of a contiguous CUDA tensor of this shape and type (None stays None)."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    p = _ptr(t, dtype, name)   # says what is wrong
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return p


def _rows(n):
    """A size that the C ABI takes as int32 (ctypes would drop its upper bits)."""
    if n > 0x7FFFFFFF:
        raise ValueError("%d rows or columns are more than 2^31 - 1" % n)
    return n


@functools.lru_cache(maxsize=256)
def _norm_setup(T, d, xt, yt, gate_kind, gate_sigmoid, scale, eps, w_offset):
    """Descriptor of a call with these settings, the gate's shape and its type."""
    if gate_kind not in GATE_KINDS:
        raise ValueError("gate_kind must be one of %s" % ", ".join(GATE_KINDS))
    _rows(T)
    _rows(d)
    desc = MoeNormDesc(T, d, _type(xt, "x"), _type(yt, "y"), GATE_KINDS[gate_kind],
                       1 if gate_sigmoid else 0, scale, eps, w_offset)
    gshape, gtype = {"none": ((0,), None), "token": ((T,), torch.float32),
                     "channel": ((d,), torch.float32), "element": ((T, d), yt)}[gate_kind]
    return ctypes.byref(desc), gshape, gtype


def _norm_desc(x, y, gate, gate_kind, gate_sigmoid, scale, eps, w_offset):
    """Descriptor, shape [T,d], types of the two sides, and the gate's shape and
    type, from the residual-side tensor x and the block-side tensor y."""
    if x is None:
        x = y
    elif y is None:
        y = x
    if x is None:
        raise ValueError("pass the residual-side tensor, the block-side tensor or both")
    sh = x.shape
    if len(sh) != 2:
        raise ValueError("rows must be [T, d], got %s" % (tuple(sh),))
    if (gate is None) != (gate_kind == "none"):
        raise ValueError("gate and gate_kind go together")
    xt, yt = x.dtype, y.dtype
    desc, gshape, gtype = _norm_setup(sh[0], sh[1], xt, yt, gate_kind, bool(gate_sigmoid),
                                      float(scale), float(eps), float(w_offset))
    return desc, sh, xt, yt, gshape, gtype


def moe_block_norm_fwd(x, y, r=None, n=None, w_post=None, w_pre=None, rstd_y=None, rstd_r=None,
                       gate=None, gate_kind="none", gate_sigmoid=False, scale=1.0, eps=1e-6,
                       w_offset=0.0, stream=None):
    """r = x + scale a(gate) norm(y; w_post), n = norm(r; w_pre).  x, r [T,d] of
    one type, y, n [T,d] of one type (x alone and n: two types as well); weights
    [d] fp32; rstd_y, rstd_r [T] fp32 (written).  gate: [T] ("token") or [d]
    ("channel") fp32, or [T,d] of y's type ("element")."""
    if y is None and n is not None:   # the norm of x alone: n has the block side's type
        desc, sh, xt, yt, gs, gt = _norm_desc(x, n, gate, gate_kind, gate_sigmoid, scale, eps,
                                              w_offset)
    else:
        # without a residual, r's own type is the residual side's
        desc, sh, xt, yt, gs, gt = _norm_desc(x if x is not None else r, y, gate, gate_kind,
                                              gate_sigmoid, scale, eps, w_offset)
    T, d = sh
    f32 = torch.float32
    _check(load().moe_block_norm_fwd(
        desc, _shaped(x, sh, xt, "x"), _shaped(y, sh, yt, "y"),
        _shaped(gate, gs, gt, "gate"), _shaped(w_post, (d,), f32, "w_post"),
        _shaped(w_pre, (d,), f32, "w_pre"), _shaped(r, sh, xt, "r"), _shaped(n, sh, yt, "n"),
        _shaped(rstd_y, (T,), f32, "rstd_y"), _shaped(rstd_r, (T,), f32, "rstd_r"),
        _stream(stream)), "moe_block_norm_fwd")


def moe_block_norm_workspace_size(T, d) -> int:
    return int(load().moe_block_norm_workspace_size(int(T), int(d)))


def moe_block_norm_bwd(dr, dn, r, y, dx=None, dy=None, w_post=None, w_pre=None, rstd_y=None,
                       rstd_r=None, gate=None, gate_kind="none", gate_sigmoid=False, dgate=None,
                       dw_post=None, dw_pre=None, ws=None, scale=1.0, eps=1e-6, w_offset=0.0,
                       stream=None):
    """Gradients of moe_block_norm_fwd from dr (of r; None: zero) and dn (of n);
    outputs left out are not computed.  dgate has the gate's shape and type,
    dw_post and dw_pre are [d] fp32."""
    x_side = dr if dr is not None else r if r is not None else dx
    y_side = y if y is not None else dn if dn is not None else dy
    desc, sh, xt, yt, gs, gt = _norm_desc(x_side, y_side, gate, gate_kind, gate_sigmoid, scale,
                                          eps, w_offset)
    T, d = sh
    f32 = torch.float32
    _check(load().moe_block_norm_bwd(
        desc, _shaped(dr, sh, xt, "dr"), _shaped(dn, sh, yt, "dn"),
        _shaped(r, sh, xt, "r"), _shaped(y, sh, yt, "y"), _shaped(gate, gs, gt, "gate"),
        _shaped(w_post, (d,), f32, "w_post"), _shaped(w_pre, (d,), f32, "w_pre"),
        _shaped(rstd_y, (T,), f32, "rstd_y"), _shaped(rstd_r, (T,), f32, "rstd_r"),
        _shaped(dx, sh, xt, "dx"), _shaped(dy, sh, yt, "dy"), _shaped(dgate, gs, gt, "dgate"),
        _shaped(dw_post, (d,), f32, "dw_post"), _shaped(dw_pre, (d,), f32, "dw_pre"),
        _ptr(ws, name="ws"), 0 if ws is None else ws.numel() * ws.element_size(),
        _stream(stream)), "moe_block_norm_bwd")


def moe_router_loss_workspace_size(T, E) -> int:
    return int(load().moe_router_loss_workspace_size(int(T), int(E)))


def _counts(counts, E):
    if counts is None:
        return None
    p = _i32(counts, "counts")
    if counts.dim() != 1 or counts.numel() < E:
        raise ValueError("counts must hold one count for each of the %d experts" % E)
    return p


def moe_router_loss_fwd(logits, counts, k, losses, lse, pmean, ws, stream=None):
    """losses [2] = (load-balancing loss, z loss), lse [T], pmean [E] of logits
    [T,E]; counts: moe_route's (its first E entries are read)."""
    T, E = logits.shape
    _rows(T)
    f32 = torch.float32
    _check(load().moe_router_loss_fwd(
        _f32(logits, "logits"), T, E, int(k), _counts(counts, E),
        _shaped(losses, (2,), f32, "losses"), _shaped(lse, (T,), f32, "lse"),
        _shaped(pmean, (E,), f32, "pmean"), _ptr(ws, name="ws"),
        ws.numel() * ws.element_size(), _stream(stream)), "moe_router_loss_fwd")


def moe_router_bwd(logits, lse, counts, ids, weights, dweights, dlogits, aux_coef=0.0,
                   z_coef=0.0, k=None, stream=None):
    """dlogits [T,E] through the top-k weights (dweights [T,k], or None) and
    through aux_coef losses[0] + z_coef losses[1].  k: needed without ids."""
    T, E = logits.shape
    _rows(T)
    f32 = torch.float32
    k = int(k) if k is not None else ids.shape[1]
    _check(load().moe_router_bwd(
        _f32(logits, "logits"), _shaped(lse, (T,), f32, "lse"), T, E, k, _counts(counts, E),
        _shaped(ids, (T, k), torch.int32, "ids"), _shaped(weights, (T, k), f32, "weights"),
        _shaped(dweights, (T, k), f32, "dweights"), aux_coef, z_coef,
        _shaped(dlogits, (T, E), f32, "dlogits"), _stream(stream)), "moe_router_bwd")


class AdamWTable:
    """The tensors of an AdamW step, checked once and kept as the array that
    moe_adamw_step reads.  rows: dicts with param, grad, m, v (same number of
    values each) and optionally master, scales, lr_mult (1), weight_decay (0).
    m and v in fp32, or in 8 bits (uint8 or torch.float8_e4m3fn) with scales
    [ceil(n / 256), 2] uint8.

    The array points to the memory that the tensors had when they were entered,
    which the table keeps alive.  A tensor that was given other memory since
    (t.data = ..., set_, resize_) is taken up by refresh()."""

    _NAMES = ("param", "grad", "m", "v", "master", "scales")

    def __init__(self, rows):
        self.rows = [dict(r) for r in rows]
        self.array = (MoeAdamWTensor * max(1, len(self.rows)))()
        self.n = len(self.rows)
        self._held = {}   # name -> rows that have one, the tensors, their pointers and storages
        for i, r in enumerate(self.rows):
            self.array[i] = self._entry(r)
        self._enter(self._NAMES)

    def _enter(self, names):
        """Notes where the tensors of these names are, and keeps that memory alive."""
        for name in names:
            at = [i for i, r in enumerate(self.rows) if r.get(name) is not None]
            ts = [self.rows[i][name] for i in at]
            self._held[name] = (at, ts, list(map(torch.Tensor.data_ptr, ts)),
                                [t.untyped_storage() for t in ts])

    def refresh(self, names=_NAMES):
        """Takes up the memory that the tensors of these names have now.  All that
        moved are checked before the first is taken."""
        moved = {}
        for name in names:
            at, ts, ptrs, _ = self._held[name]
            now = list(map(torch.Tensor.data_ptr, ts))
            if now != ptrs:
                moved.update((i, None) for i, a, b in zip(at, now, ptrs) if a != b)
        if not moved:
            return
        for i in moved:
            moved[i] = self._entry(self.rows[i])
            if moved[i].n != self.array[i].n:
                raise ValueError("tensor %d has %d values now, not %d" % (i, moved[i].n,
                                                                          self.array[i].n))
        for i, e in moved.items():
            self.array[i] = e
        self._enter(self._NAMES)

    @staticmethod
    def _entry(r):
        p, n = r["param"], r["param"].numel()
        eight = r["m"].element_size() == 1
        state = (torch.uint8, torch.float8_e4m3fn) if eight else (torch.float32,)
        for name in ("grad", "m", "v", "master"):
            if r.get(name) is not None and r[name].numel() != n:
                raise ValueError("%s must have as many values as param" % name)
        for name in ("m", "v"):
            if r[name].dtype not in state:
                raise ValueError("%s must be fp32, uint8 or float8_e4m3fn (both alike)" % name)
        sc = r.get("scales")
        if eight != (sc is not None):
            raise ValueError("scales go with 8-bit states")
        if eight and sc.shape != (-(-n // MOE_ADAMW_BLOCK), 2):
            raise ValueError("scales must have shape %s" % ((-(-n // MOE_ADAMW_BLOCK), 2),))
        return MoeAdamWTensor(
            _ptr(p, name="param"), _f32(r.get("master"), "master"), _ptr(r["grad"], name="grad"),
            _ptr(r["m"], name="m"), _ptr(r["v"], name="v"), _ptr(sc, torch.uint8, "scales"), n,
            _type(p.dtype, "param"), _type(r["grad"].dtype, "grad"), 8 if eight else 32,
            float(r.get("lr_mult", 1.0)), float(r.get("weight_decay", 0.0)))

    def set_grads(self, grads):
        """Other gradient tensors, in the order of the rows.  All are checked
        before the first is taken: a refusal leaves the table as it was."""
        grads = list(grads)
        if len(grads) != self.n:
            raise ValueError("%d gradients for %d tensors" % (len(grads), self.n))
        new = [self._grad(g, e.n) for g, e in zip(grads, self.array)]
        for r, e, g, (e_ptr, e_type) in zip(self.rows, self.array, grads, new):
            r["grad"], e.grad, e.grad_type = g, e_ptr, e_type
        self._enter(("grad",))

    @staticmethod
    def _grad(g, n):
        """Pointer and type of a gradient of n values."""
        if g is None:
            raise TypeError("grad must be a torch.Tensor")
        p = _ptr(g, name="grad")
        if g.numel() != n:
            raise ValueError("grad must have as many values as param")
        return p, _type(g.dtype, "grad")


def moe_adamw_workspace_size(table: AdamWTable) -> int:
    return int(load().moe_adamw_workspace_size(table.array, table.n))


def moe_adamw_step(table: AdamWTable, step, lr, betas=(0.9, 0.999), eps=1e-8, grad_scale=1.0,
                   max_norm=0.0, skip_nonfinite=False, grad_norm=None, ws=None, stream=None):
    """One AdamW step (step counts from 1) over the table's tensors, in place.
    max_norm > 0 clips by the global gradient norm, which grad_norm [1] fp32
    receives; ws is needed for the norm only."""
    h = MoeAdamWHyper(lr, betas[0], betas[1], eps, step, grad_scale, max_norm,
                      1 if skip_nonfinite else 0)
    _check(load().moe_adamw_step(
        table.array, table.n, ctypes.byref(h), _shaped(grad_norm, (1,), torch.float32, "grad_norm"),
        _ptr(ws, name="ws"), 0 if ws is None else ws.numel() * ws.element_size(),
        _stream(stream)), "moe_adamw_step")


def moe_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return int(load().moe_status(_stream(stream)))


def moe_selftest_wait_timeout(timeout_us: int, stream=None):
    """Enqueue the bounded-wait self-test: a GPU thread that waits on an
    mbarrier nothing arrives on for timeout_us, then records MOE_ERR_TIMEOUT
    (read it with moe_status)."""
    _check(load().moe_selftest_wait_timeout(int(timeout_us), _stream(stream)),
           "moe_selftest_wait_timeout")


def moe_selftest_ring_timeout(timeout_us: int, late: int, tiles, stream=None):
    """Enqueue the self-test of the norms' ring: warp `late` (0: the filling
    one, 1, or -1: none) misses a tile and gives up after timeout_us; tiles [1]
    int32 receives how many tiles were filled (-1: one was left in flight)."""
    _check(load().moe_selftest_ring_timeout(int(timeout_us), int(late), _i32(tiles, "tiles"),
                                            _stream(stream)), "moe_selftest_ring_timeout")


# ------------------------------------------------------------------ tracing

def kernel_names():
    lib, out, i = load(), [], 0
    while True:
        n = lib.moe_kernel_name(i)
        if n is None:
            return out
        out.append(n.decode())
        i += 1


class KernelProbe:
    """Device time of the next ``n`` launches of one kernel, from CUDA events
    the library records on the launch stream (see moe_probe_arm)."""

    def __init__(self, kernel: str, n: int):
        self.kernel = kernel
        self.start = [torch.cuda.Event(enable_timing=True) for _ in range(n)]
        self.stop = [torch.cuda.Event(enable_timing=True) for _ in range(n)]
        s = torch.cuda.current_stream()
        for e in self.start + self.stop:   # materialise the event handles
            e.record(s)
        torch.cuda.synchronize()
        arr = _P * n
        self._a = arr(*[e.cuda_event for e in self.start])
        self._b = arr(*[e.cuda_event for e in self.stop])
        _check(load().moe_probe_arm(kernel.encode(), self._a, self._b, n), "moe_probe_arm")

    def disarm(self):
        load().moe_probe_arm(self.kernel.encode(), None, None, 0)

    def times_ms(self):
        """Durations (ms) of the recorded launches (synchronises)."""
        n = int(load().moe_probe_count(self.kernel.encode()))
        torch.cuda.synchronize()
        return [self.start[i].elapsed_time(self.stop[i]) for i in range(n)]
