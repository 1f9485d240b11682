"""The selective state space scan and the short causal convolution in front of it, on torch CUDA
tensors: a binding over ``gma_scan_*`` and ``gma_conv_*`` (``include/gma_block.h``).

Activations are token-major, [B, N, channels], bf16 or fp32, with contiguous channels and any strides
between tokens and batch rows, so that they can be parts of a wider projection's rows.  Parameters
and scan states are contiguous fp32, ``a_log``, states and checkpoints on 16-byte boundaries.  Outputs given
by the caller must not overlap the inputs or one another.  ``lengths`` (int32 [B] on the device) gives each batch row's number
of tokens; the rows behind them are neither read nor written (in outputs allocated here they are zero).

``stream`` is the stream to run on (default: the current one).  Nothing here waits for the GPU.  Tensors
that do not fit raise TypeError or ValueError, what the library refuses raises ``gma.GmaError``.
"""
import torch

from . import gma  # noqa: F401  (loads libgma.so, which _block is linked against)
from . import _block


# ------------------------------------------------------------------ selective scan

def scan_checkpoints(u, S):
    """An uninitialised buffer for the states that ``scan`` keeps for ``scan_backward``."""
    return _block.scan_checkpoints(u, S)


def scan(u, dt, a_log, b, c, d_skip=None, dt_bias=None, z=None, state=None, state_out=None, lengths=None,
         checkpoints=None, out=None, stream=None):
    """Selective state space scan; returns y [B, N, D].

    u, dt and z [B, N, D], b and c [B, N, S] or [B, N, G, S] share one dtype; a_log [D, S], d_skip [D] and
    dt_bias [D] are fp32.  ``state`` [B, D, S] is the state before the first token (zeros if None);
    ``state_out`` takes the one after each row's last token and may be ``state``; ``checkpoints`` (from
    ``scan_checkpoints``) takes what ``scan_backward`` needs.  S is 8, 16, 32 or 64.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return _block.scan(u, dt, a_log, b, c, d_skip, dt_bias, z, state, state_out, lengths, checkpoints, out)
    return _block.scan(u, dt, a_log, b, c, d_skip, dt_bias, z, state, state_out, lengths, checkpoints, out)


def scan_step(u, dt, a_log, b, c, state, d_skip=None, dt_bias=None, z=None, out=None, stream=None):
    """One token for every sequence; returns y [B, D] and updates ``state`` [B, D, S] in place.

    u, dt and z [B, D], b and c [B, S] or [B, G, S]; parameters as in ``scan``.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return _block.scan_step(u, dt, a_log, b, c, d_skip, dt_bias, z, state, out)
    return _block.scan_step(u, dt, a_log, b, c, d_skip, dt_bias, z, state, out)


def scan_backward(dy, u, dt, a_log, b, c, checkpoints, d_skip=None, dt_bias=None, z=None, dstate_out=None,
                  lengths=None, out=None, stream=None):
    """Gradients of sum(dy * y) + sum(dstate_out * state_out) of ``scan`` with the same arguments.

    ``checkpoints`` are those that ``scan`` kept.  Returns a dict with the gradients "u", "dt", "z" (None
    without z), "b", "c" in the activations' dtype, "a_log", "d_skip", "dt_bias" (None where the parameter
    is) and "state" (of the state before the first token) in fp32.  ``out`` may hold tensors, under
    the names "u", "dt", "z", "b" and "c", that take those gradients (rows with strides).
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return scan_backward(dy, u, dt, a_log, b, c, checkpoints, d_skip, dt_bias, z, dstate_out, lengths, out)
    if out and not out.keys() <= {"u", "dt", "z", "b", "c"}:
        raise ValueError(f"out takes 'u', 'dt', 'z', 'b' and 'c', not {sorted(out.keys() - {'u', 'dt', 'z', 'b', 'c'})}")
    given = (out.get(k) for k in ("u", "dt", "z", "b", "c")) if out else (None,) * 5
    return _block.scan_backward(u, dt, a_log, b, c, d_skip, dt_bias, z, dy, checkpoints, dstate_out, lengths, *given)


# ------------------------------------------------------------------ short causal convolution

def conv(x, weight, bias=None, state=None, state_out=None, lengths=None, silu=True, out=None, stream=None):
    """Short causal convolution per channel, with silu unless ``silu`` is False; returns y [B, N, D].

    x [B, N, D]; weight [D, W] (W = 2, 3, 4, the last tap on the current token) and bias [D] fp32; ``state``
    [B, W - 1, D] holds the inputs before the first token, oldest first (zeros if None), and
    ``state_out`` takes the last W - 1 inputs of each row (not in place).
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return _block.conv(x, weight, bias, state, silu, state_out, lengths, out)
    return _block.conv(x, weight, bias, state, silu, state_out, lengths, out)


def conv_step(x, weight, bias, state, silu=True, out=None, stream=None):
    """One token for every sequence; returns y [B, D] and moves ``state`` [B, W - 1, D] on in place."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _block.conv_step(x, weight, bias, state, silu, out)
    return _block.conv_step(x, weight, bias, state, silu, out)


def conv_backward(dy, x, weight, bias=None, state=None, lengths=None, silu=True, out=None, stream=None):
    """Gradients of sum(dy * y) of ``conv`` with the same arguments; the state counts as a constant.

    Returns a dict: "x" in x's dtype (into ``out`` if given), "weight" and "bias" (None without one) in fp32.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return _block.conv_backward(x, weight, bias, state, silu, dy, lengths, out)
    return _block.conv_backward(x, weight, bias, state, silu, dy, lengths, out)
