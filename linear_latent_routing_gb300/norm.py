"""The norms before and after a block with its gate and residual scale, on torch CUDA tensors: a
binding over ``gma_norm_*`` (``include/gma_block.h``).

    a = o * silu(gate);  v = w_post * rms(a) per group;  r = residual + scale * v;  h = w_pre * rms(r)

``o`` is a mixer's output [B, H, N, d] (as ``gma.forward`` returns it, or any strides with contiguous
d) or rows [B, N, D]; everything else is token-major [B, N, D] with D = H * d.  Parameters are fp32 [D].
"""
import ctypes

import torch

from . import _marshal as m
from ._marshal import F32, NO_ROWS, dense, heads, rows

_vp, _sz = ctypes.c_void_p, ctypes.c_size_t
_norm_forward = m.declare("gma_norm_forward", _vp, _vp)
_norm_backward = m.declare("gma_norm_backward", _vp, _vp, _sz, _vp)
_norm_backward_workspace = m.declare("gma_norm_backward_workspace_size", _vp, restype=_sz)

_NORM = "7ifRqRR3QRR"
_norm_t = m.layout(_NORM)
_norm_grad_t = m.layout(_NORM + "RRRqRR3Q")
_empty = torch.empty


def _shape(o, residual, group):
    T, code, dev = m.first(o, "o")
    shape = o.shape
    if len(shape) == 4:
        B, H, N, d = shape
    elif len(shape) == 3:
        (B, N, d), H = shape, 1
    else:
        raise ValueError("o must be [B, H, N, d] or [B, N, D]")
    R = T
    if residual is not None:
        R = getattr(residual, "dtype", None)
        if R is not T and R is not F32:
            raise TypeError(f"residual must be {T} or {F32}")
    D = H * d
    return (B, N, H, d, group or D, code, m.CODES[R]), T, R, dev, (B, N, D), (D,)


def block_norm(o, w_post=None, gate=None, residual=None, scale=None, w_pre=None, eps=1e-6, group=0, out=None,
               out_h=None, stream=None):
    """Norm after a block (``w_post``) with its gate, residual scale and the next norm (``w_pre``).

    Returns (r, h): r [B, N, D] is the new residual stream, in the residual's dtype (the o dtype and v
    itself without a residual), and h [B, N, D] its norm, or None without ``w_pre``.  ``group`` is the
    number of channels that the first norm's mean runs over: 0 for all, or a power of two from 8 to 256
    that divides D (a head's d, for a norm per head).  ``out`` may be ``residual``.
    """
    if stream is not None:
        with m.on_stream(stream):
            return block_norm(o, w_post, gate, residual, scale, w_pre, eps, group, out, out_h)
    head, T, R, dev, full, vec = _shape(o, residual, group)
    if out is None:
        out = _empty(full, dtype=R, device=o.device)
    h = None
    if w_pre is not None:
        h = _empty(full, dtype=T, device=o.device) if out_h is None else out_h
    packed = _norm_t.pack(
        *head, eps, *heads(o, "o", o.shape, T, dev), *(rows(gate, "gate", full, T, dev) if gate is not None else NO_ROWS),
        *(rows(residual, "residual", full, R, dev) if residual is not None else NO_ROWS),
        dense(w_post, "w_post", vec, F32, dev), dense(scale, "scale", vec, F32, dev),
        dense(w_pre, "w_pre", vec, F32, dev), *rows(out, "out", full, R, dev),
        *(rows(h, "out_h", full, T, dev) if h is not None else NO_ROWS))
    r = _norm_forward(packed, m.handle(dev))
    if r:
        m.failed(r, "gma_norm_forward")
    return out, h


def block_norm_backward(dr, o, r, w_post=None, gate=None, scale=None, w_pre=None, dh=None, eps=1e-6, group=0,
                        residual=None, out=None, stream=None):
    """Gradients of sum(dr * r) + sum(dh * h) of ``block_norm`` with the same arguments.

    ``r`` is what the forward call returned (its dtype tells the residual stream's); ``residual`` says
    whether there was a residual; by default there was one if there is a ``scale`` or r's dtype is
    another than o's.  Either of dr and dh may be None.  Returns a dict: "o" (o's layout, contiguous, or
    ``out``), "gate", "residual" (None without one), "w_post", "scale", "w_pre" (None where the
    argument is).
    """
    if stream is not None:
        with m.on_stream(stream):
            return block_norm_backward(dr, o, r, w_post, gate, scale, w_pre, dh, eps, group, residual, out)
    if residual is None:
        residual = scale is not None or getattr(r, "dtype", None) is not getattr(o, "dtype", None)
    head, T, R, dev, full, vec = _shape(o, r if residual else None, group)
    device = o.device
    kept = rows(r, "r", full, R, dev)
    g = {"o": _empty(o.shape, dtype=T, device=device) if out is None else out,
         "gate": _empty(full, dtype=T, device=device) if gate is not None else None,
         "residual": _empty(full, dtype=R, device=device) if residual else None}
    for name, p in (("w_post", w_post), ("scale", scale), ("w_pre", w_pre)):
        g[name] = torch.empty_like(p) if p is not None else None
    packed = _norm_grad_t.pack(
        *head, eps, *heads(o, "o", o.shape, T, dev), *(rows(gate, "gate", full, T, dev) if gate is not None else NO_ROWS),
        *(kept if residual else NO_ROWS), dense(w_post, "w_post", vec, F32, dev),
        dense(scale, "scale", vec, F32, dev), dense(w_pre, "w_pre", vec, F32, dev), *kept, *NO_ROWS,
        *(rows(dr, "dr", full, R, dev) if dr is not None else NO_ROWS),
        *(rows(dh, "dh", full, T, dev) if dh is not None else NO_ROWS), *heads(g["o"], "out", o.shape, T, dev),
        *(rows(g["gate"], "gate", full, T, dev) if gate is not None else NO_ROWS),
        *(rows(g["residual"], "residual", full, R, dev) if residual else NO_ROWS),
        *(p.data_ptr() if p is not None else 0 for p in (g["w_post"], g["scale"], g["w_pre"])))
    n = _norm_backward_workspace(packed)
    ws = _empty(n, dtype=torch.uint8, device=device) if n else None
    q = _norm_backward(packed, ws.data_ptr() if n else 0, n, m.handle(dev))
    if q:
        m.failed(q, "gma_norm_backward")
    return g
