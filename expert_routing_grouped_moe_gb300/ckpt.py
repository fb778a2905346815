"""Buffers that a stack of layers shares when each keeps its activations in 8 bits.

A layer needs most of its device memory only while one of its calls runs: the
permuted rows, the pre-activations in fp32, the activations as pairs, the
gradients' rows.  With a ``LayerScratch`` those belong to all layers together,
and a layer keeps from its forward to its backward what 8 bits hold: the
pre-activations (``lib.moe_ckpt_pack``), from which the backward gets them and
the activations back (``lib.moe_ckpt_unpack_swiglu``).  At T = 4096, d = 2048,
f = 768, top-8, r = 64 a layer more then takes 0.07 GB instead of 1.1 (its
gradient buffers aside) and a step a tenth more time.
"""
from __future__ import annotations

import torch

from . import _lib as L


class LayerScratch:
    """Device buffers by name, each as large as its largest user asked for; users get
    views.  What one call leaves there the next call of any layer overwrites, so the
    layers of one scratch take turns: on one stream, or ordered by their caller.  A
    buffer stays where it is for the scratch's life: a layer larger than those before it
    gets another, which later layers share, so build the largest first."""

    def __init__(self, device="cuda"):
        self.device = torch.device(device)
        self._buf, self._made = {}, []

    def take(self, name, shape, dtype, device=None):
        """A tensor of this shape over the buffer of that name (made, or made larger,
        on first use; layers take theirs when they are built).  device: the user's, which
        has to be the scratch's."""
        n = 1
        for s in shape:
            n *= int(s)
        size = n * torch.empty(0, dtype=dtype).element_size()
        buf = self._buf.get(name)
        if buf is None or buf.numel() < size:
            # a larger buffer replaces the smaller one for later users; earlier ones keep theirs
            buf = torch.empty(max(16, size), dtype=torch.uint8, device=self.device)
        if device is not None and torch.empty(0, device=device).device != buf.device:
            raise ValueError("the scratch is on %s, its user on %s" % (buf.device, device))
        if self._buf.get(name) is not buf:
            self._buf[name] = buf
            self._made.append(buf)
        return buf[:size].view(dtype).view(*shape)

    def bytes(self):
        """Of all buffers, replaced ones among them."""
        return sum(b.numel() for b in self._made)


class Packed8:
    """Rows [R, C] kept in 8 bits: codes and scales, and the calls that fill and read them."""

    def __init__(self, R, C, device="cuda"):
        self.codes = torch.empty(R, C, dtype=torch.int8, device=device)
        self.scales = torch.empty(R, -(-C // L.MOE_CKPT_BLOCK), dtype=torch.uint8, device=device)

    def pack(self, x, stream=None):
        L.moe_ckpt_pack(x, self.codes, self.scales, stream=stream)

    def unpack(self, x, stream=None):
        L.moe_ckpt_unpack(self.codes, self.scales, x, stream=stream)
        return x

    def unpack_swiglu(self, sorted_src, topk_w, shared_expert, h, act, stream=None):
        L.moe_ckpt_unpack_swiglu(self.codes, self.scales, sorted_src, topk_w, shared_expert, h, act,
                                 stream=stream)
