"""The norms before and after a block with its gate and residual scale, on torch CUDA tensors: a
binding over ``gma_norm_*`` (``include/gma_block.h``).

    a = o * silu(gate);  v = w_post * rms(a) per group;  r = residual + scale * v;  h = w_pre * rms(r)

``o`` is a mixer's output [B, H, N, d] (as ``gma.forward`` returns it, or any strides with contiguous
d) or rows [B, N, D]; everything else is token-major [B, N, D] with D = H * d.  Parameters are fp32 [D].
Tensors that do not fit raise TypeError or ValueError, what the library refuses raises ``gma.GmaError``.
"""
import torch

from . import gma  # noqa: F401  (loads libgma.so, which _block is linked against)
from . import _block


def block_norm(o, w_post=None, gate=None, residual=None, scale=None, w_pre=None, eps=1e-6, group=0, out=None,
               out_h=None, stream=None):
    """Norm after a block (``w_post``) with its gate, residual scale and the next norm (``w_pre``).

    Returns (r, h): r [B, N, D] is the new residual stream, in the residual's dtype (the o dtype and v
    itself without a residual), and h [B, N, D] its norm, or None without ``w_pre``.  ``group`` is the
    number of channels that the first norm's mean runs over: 0 for all, or a power of two from 8 to 256
    that divides D (a head's d, for a norm per head).  ``out`` may be ``residual``; otherwise outputs do not
    overlap the inputs or one another.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return _block.block_norm(o, w_post, gate, scale, w_pre, eps, group, residual, out, out_h)
    return _block.block_norm(o, w_post, gate, scale, w_pre, eps, group, residual, out, out_h)


def block_norm_backward(dr, o, r, w_post=None, gate=None, scale=None, w_pre=None, dh=None, eps=1e-6, group=0,
                        residual=None, out=None, stream=None):
    """Gradients of sum(dr * r) + sum(dh * h) of ``block_norm`` with the same arguments.

    ``r`` is what the forward call returned (its dtype tells the residual stream's); ``residual`` says
    whether there was a residual: the forward call's tensor, whose values are not used, or a truth value.
    By default there was one if there is a ``scale`` or r's dtype is another than o's.  Either of dr and dh may be None.  Returns a dict: "o" (o's layout, contiguous, or
    ``out``), "gate", "residual" (None without one), "w_post", "scale", "w_pre" (None where the
    argument is).
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return _block.block_norm_backward(o, w_post, gate, scale, w_pre, eps, group, dr, r, dh, residual, out)
    return _block.block_norm_backward(o, w_post, gate, scale, w_pre, eps, group, dr, r, dh, residual, out)
