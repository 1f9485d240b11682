"""The norms before and after a block with its gate and residual scale, on torch CUDA tensors: a
binding over ``gma_norm_*`` (``include/gma_block.h``).

    a = o * silu(gate);  v = w_post * rms(a) per group;  r = residual + scale * v;  h = w_pre * rms(r)

``o`` is a mixer's output [B, H, N, d] (as ``gma.forward`` returns it, or any strides with contiguous
d) or rows [B, N, D]; everything else is token-major [B, N, D] with D = H * d.  Parameters are fp32 [D].
"""
import ctypes

import torch

from . import _marshal as m
from ._marshal import F32

_vp, _sz = ctypes.c_void_p, ctypes.c_size_t
_norm_forward = m.declare("gma_norm_forward", _vp, _vp)
_norm_backward = m.declare("gma_norm_backward", _vp, _vp, _sz, _vp)
_norm_backward_workspace = m.declare("gma_norm_backward_workspace_size", _vp, restype=_sz)

_NORM = "7ifRqRR3QRR"
_norm_t = m.layout(_NORM)
_norm_grad_t = m.layout(_NORM + "RRRqRR3Q")


def _heads(t, name, shape, dtype, like):
    """(pointer, batch stride, token stride, head stride) of [B, H, N, d] or [B, N, D]."""
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype != dtype or t.get_device() != like.get_device():
        m._fail(t, name, shape, dtype, like)
    s = t.stride()
    if s[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"{name}'s channels must be contiguous")
    return (t.data_ptr(), s[0], s[2], s[1]) if len(shape) == 4 else (t.data_ptr(), s[0], s[1], 0)


def _shape(o, residual, group):
    code = m.code(o, "o")
    if o.dim() == 4:
        B, H, N, d = o.shape
    elif o.dim() == 3:
        (B, N, d), H = o.shape, 1
    else:
        raise ValueError("o must be [B, H, N, d] or [B, N, D]")
    R = o.dtype
    if residual is not None:
        if not isinstance(residual, torch.Tensor) or residual.dtype not in (o.dtype, F32):
            raise TypeError(f"residual must be {o.dtype} or {F32}")
        R = residual.dtype
    D = H * d
    return B, N, H, d, D, group or D, code, R


def block_norm(o, w_post=None, gate=None, residual=None, scale=None, w_pre=None, eps=1e-6, group=0, out=None,
               out_h=None, stream=None):
    """Norm after a block (``w_post``) with its gate, residual scale and the next norm (``w_pre``).

    Returns (r, h): r [B, N, D] is the new residual stream, in the residual's dtype (the o dtype and v
    itself without a residual), and h [B, N, D] its norm, or None without ``w_pre``.  ``group`` is the
    number of channels that the first norm's mean runs over: 0 for all, or a power of two from 8 to 256
    that divides D (a head's d, for a norm per head).  ``out`` may be ``residual``.
    """
    B, N, H, d, D, group, code, R = _shape(o, residual, group)
    T, full, vec = o.dtype, (B, N, D), (D,)
    with m.on_stream(stream) as st:
        if out is None:
            out = torch.empty(full, dtype=R, device=o.device)
        h = None
        if w_pre is not None:
            h = torch.empty(full, dtype=T, device=o.device) if out_h is None else out_h
        packed = _norm_t.pack(
            B, N, H, d, group, code, m.CODES[R], eps, *_heads(o, "o", o.shape, T, o), *m.rows(gate, "gate", full, T, o),
            *m.rows(residual, "residual", full, R, o), m.dense(w_post, "w_post", vec, F32, o),
            m.dense(scale, "scale", vec, F32, o), m.dense(w_pre, "w_pre", vec, F32, o),
            *m.rows(out, "out", full, R, o), *m.rows(h, "out_h", full, T, o))
        m.call(_norm_forward, packed, st)
    return out, h


def block_norm_backward(dr, o, r, w_post=None, gate=None, scale=None, w_pre=None, dh=None, eps=1e-6, group=0,
                        residual=None, out=None, stream=None):
    """Gradients of sum(dr * r) + sum(dh * h) of ``block_norm`` with the same arguments.

    ``r`` is what the forward call returned (its dtype tells the residual stream's); ``residual`` says
    whether there was a residual, and defaults to whether ``scale``, or an r of another dtype than o's,
    shows one.  Either of dr and dh may be None.  Returns a dict: "o" (o's layout, contiguous, or
    ``out``), "gate", "residual" (None without one), "w_post", "scale", "w_pre" (None where the
    argument is).
    """
    if not isinstance(r, torch.Tensor):
        raise TypeError("r must be a CUDA tensor")
    if residual is None:
        residual = scale is not None or r.dtype != o.dtype
    B, N, H, d, D, group, code, R = _shape(o, r if residual else None, group)
    T, dev, full, vec = o.dtype, o.device, (B, N, D), (D,)
    with m.on_stream(stream) as st:
        kept = m.rows(r, "r", full, R, o)
        g = {"o": torch.empty(o.shape, dtype=T, device=dev) if out is None else out,
             "gate": torch.empty(full, dtype=T, device=dev) if gate is not None else None,
             "residual": torch.empty(full, dtype=R, device=dev) if residual else None}
        for name, p in (("w_post", w_post), ("scale", scale), ("w_pre", w_pre)):
            g[name] = torch.empty_like(p) if p is not None else None
        do = _heads(g["o"], "out", o.shape, T, o)
        packed = _norm_grad_t.pack(
            B, N, H, d, group, code, m.CODES[R], eps, *_heads(o, "o", o.shape, T, o), *m.rows(gate, "gate", full, T, o),
            *(kept if residual else m.NO_ROWS), m.dense(w_post, "w_post", vec, F32, o),
            m.dense(scale, "scale", vec, F32, o), m.dense(w_pre, "w_pre", vec, F32, o), *kept, *m.NO_ROWS,
            *m.rows(dr, "dr", full, R, o), *m.rows(dh, "dh", full, T, o), *do, *m.rows(g["gate"], "gate", full, T, o),
            *m.rows(g["residual"], "residual", full, R, o),
            *(p.data_ptr() if p is not None else 0 for p in (g["w_post"], g["scale"], g["w_pre"])))
        n = _norm_backward_workspace(packed)
        ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
        m.call(_norm_backward, packed, ws.data_ptr() if n else 0, n, st)
    return g
