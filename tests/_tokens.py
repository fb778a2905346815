"""Shared helpers of the tests of embedding, log probabilities and checkpoints."""
import numpy as np
import torch

DEV = "cuda"
U = 2.0 ** -24                       # half a step of fp32, relative
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
BF, F32 = torch.bfloat16, torch.float32


def place(shape, dtype, off=0, fill=None, guard=64):
    """(tensor, check): a tensor that begins `off` values past a 256-byte boundary inside
    a buffer of guard values; check() says whether anything around it was written."""
    n = int(np.prod(shape))
    pad = guard + off
    buf = torch.empty(256 + n + 2 * pad + 256, dtype=dtype, device=DEV)
    mark = 77 if not dtype.is_floating_point else 77.0
    buf.fill_(mark)
    start = 256 + off
    t = buf[start:start + n].view(shape)
    if fill is not None:
        t.copy_(fill)

    def check():
        return bool((buf[:start] == mark).all()) and bool((buf[start + n:] == mark).all())
    return t, check


def np64(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def graph_of(fn):
    """A captured graph of fn's launches (after one call outside of it)."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    return g
