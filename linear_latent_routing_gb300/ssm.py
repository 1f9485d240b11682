"""The selective state space scan and the short causal convolution in front of it, on torch CUDA
tensors: a binding over ``gma_scan_*`` and ``gma_conv_*`` (``include/gma_block.h``).

Activations are token-major, [B, N, channels], bf16 or fp32, with contiguous channels and any strides
between tokens and batch rows, so that they can be parts of a wider projection's rows.  Parameters
and scan states are contiguous fp32.  ``lengths`` (int32 [B] on the device) gives each batch row's number
of tokens; the rows behind them are neither read nor written (in outputs allocated here they are zero).

``stream`` is the stream to run on (default: the current one).  Nothing here waits for the GPU.
"""
import ctypes

import torch

from . import _marshal as m
from ._marshal import F32, NO_ROWS, dense, rows, rows4, token, token3

_vp, _sz = ctypes.c_void_p, ctypes.c_size_t
_scan_forward = m.declare("gma_scan_forward", _vp, _vp, _sz, _vp)
_scan_step = m.declare("gma_scan_step", _vp, _vp)
_scan_backward = m.declare("gma_scan_backward", _vp, _vp, _sz, _vp)
_scan_workspace = m.declare("gma_scan_workspace_size", _vp, restype=_sz)
_scan_backward_workspace = m.declare("gma_scan_backward_workspace_size", _vp, restype=_sz)
_conv_forward = m.declare("gma_conv_forward", _vp, _vp)
_conv_step = m.declare("gma_conv_step", _vp, _vp)
_conv_backward = m.declare("gma_conv_backward", _vp, _vp, _sz, _vp)
_conv_backward_workspace = m.declare("gma_conv_backward_workspace_size", _vp, restype=_sz)

_SCAN = "6iRRRRR6QRQ"
_scan_t = m.layout(_SCAN)
_scan_grad_t = m.layout(_SCAN + "RQRRRRR4Q")
_CONV = "5iIR5QR"
_conv_t = m.layout(_CONV)
_conv_grad_t = m.layout(_CONV + "RR2Q")

CHECKPOINT_TOKENS = 64
GMA_CONV_LINEAR = 0x1
_empty, _zeros, _int32 = torch.empty, torch.zeros, torch.int32


def _ptr(t):
    return 0 if t is None else t.data_ptr()


# ------------------------------------------------------------------ selective scan

def _scan_args(u, dt, a_log, b, c, d_skip, dt_bias, z):
    """The sizes, rows and parameters of a call on [B, N, D], in the header's order."""
    T, code, dev = m.first(u, "u")
    full = u.shape
    if len(full) != 3:
        raise ValueError("u must be [B, N, D]")
    B, N, D = full
    S = m.last_dim(a_log, "a_log", 2, "[D, S]")
    if b is not None and getattr(b, "dim", tuple)() == 4:
        G = b.shape[2]
        bc = (B, N, G, S)
        br, cr = rows4(b, "b", bc, T, dev), rows4(c, "c", bc, T, dev)
    else:
        G, bc = 1, (B, N, S)
        br, cr = rows(b, "b", bc, T, dev), rows(c, "c", bc, T, dev)
    head = (B, N, D, S, G, code, *rows(u, "u", full, T, dev), *rows(dt, "dt", full, T, dev),
            *(rows(z, "z", full, T, dev) if z is not None else NO_ROWS), *br, *cr,
            dense(m.need(a_log, "a_log"), "a_log", (D, S), F32, dev), dense(d_skip, "d_skip", (D,), F32, dev),
            dense(dt_bias, "dt_bias", (D,), F32, dev))
    return head, T, dev, full, bc


def scan_checkpoints(u, S):
    """An uninitialised buffer for the states that ``scan`` keeps for ``scan_backward``."""
    B, N, D = u.shape
    return _empty(B, -(-N // CHECKPOINT_TOKENS), D, S, dtype=F32, device=u.device)


def scan(u, dt, a_log, b, c, d_skip=None, dt_bias=None, z=None, state=None, state_out=None, lengths=None,
         checkpoints=None, out=None, stream=None):
    """Selective state space scan; returns y [B, N, D].

    u, dt and z [B, N, D], b and c [B, N, S] or [B, N, G, S] share one dtype; a_log [D, S], d_skip [D] and
    dt_bias [D] are fp32.  ``state`` [B, D, S] is the state before the first token (zeros if None);
    ``state_out`` takes the one after each row's last token and may be ``state``; ``checkpoints`` (from
    ``scan_checkpoints``) takes what ``scan_backward`` needs.  S is 8, 16, 32 or 64.
    """
    if stream is not None:
        with m.on_stream(stream):
            return scan(u, dt, a_log, b, c, d_skip, dt_bias, z, state, state_out, lengths, checkpoints, out)
    head, T, dev, full, _ = _scan_args(u, dt, a_log, b, c, d_skip, dt_bias, z)
    B, N, D, S = head[:4]
    if out is None:
        out = (_empty if lengths is None else _zeros)(full, dtype=T, device=u.device)
    packed = _scan_t.pack(
        *head, dense(state, "state", (B, D, S), F32, dev), dense(state_out, "state_out", (B, D, S), F32, dev),
        dense(lengths, "lengths", (B,), _int32, dev), *rows(out, "out", full, T, dev),
        dense(checkpoints, "checkpoints", (B, -(-N // CHECKPOINT_TOKENS), D, S), F32, dev))
    n = _scan_workspace(packed)
    ws = _empty(n, dtype=torch.uint8, device=u.device) if n else None
    r = _scan_forward(packed, _ptr(ws), n, m.handle(dev))
    if r:
        m.failed(r, "gma_scan_forward")
    return out


def scan_step(u, dt, a_log, b, c, state, d_skip=None, dt_bias=None, z=None, out=None, stream=None):
    """One token for every sequence; returns y [B, D] and updates ``state`` [B, D, S] in place.

    u, dt and z [B, D], b and c [B, S] or [B, G, S]; parameters as in ``scan``.
    """
    if stream is not None:
        with m.on_stream(stream):
            return scan_step(u, dt, a_log, b, c, state, d_skip, dt_bias, z, out)
    T, code, dev = m.first(u, "u")
    full = u.shape
    if len(full) != 2:
        raise ValueError("u must be [B, D]")
    B, D = full
    S = m.last_dim(a_log, "a_log", 2, "[D, S]")
    if b is not None and getattr(b, "dim", tuple)() == 3:
        G = b.shape[1]
        br, cr = token3(b, "b", (B, G, S), T, dev), token3(c, "c", (B, G, S), T, dev)
    else:
        G = 1
        br, cr = token(b, "b", (B, S), T, dev), token(c, "c", (B, S), T, dev)
    if out is None:
        out = _empty(full, dtype=T, device=u.device)
    h = dense(m.need(state, "state"), "state", (B, D, S), F32, dev)
    packed = _scan_t.pack(
        B, 1, D, S, G, code, *token(u, "u", full, T, dev), *token(dt, "dt", full, T, dev),
        *(token(z, "z", full, T, dev) if z is not None else NO_ROWS), *br, *cr,
        dense(a_log, "a_log", (D, S), F32, dev), dense(d_skip, "d_skip", (D,), F32, dev),
        dense(dt_bias, "dt_bias", (D,), F32, dev), h, h, 0, *token(out, "out", full, T, dev), 0)
    r = _scan_step(packed, m.handle(dev))
    if r:
        m.failed(r, "gma_scan_step")
    return out


def scan_backward(dy, u, dt, a_log, b, c, checkpoints, d_skip=None, dt_bias=None, z=None, dstate_out=None,
                  lengths=None, out=None, stream=None):
    """Gradients of sum(dy * y) + sum(dstate_out * state_out) of ``scan`` with the same arguments.

    ``checkpoints`` are those that ``scan`` kept.  Returns a dict with the gradients "u", "dt", "z" (None
    without z), "b", "c" in the activations' dtype, "a_log", "d_skip", "dt_bias" (None where the parameter
    is) and "state" (of the state before the first token) in fp32.  ``out`` may hold tensors, under
    the names "u", "dt", "z", "b" and "c", that take those gradients (rows with strides).
    """
    if stream is not None:
        with m.on_stream(stream):
            return scan_backward(dy, u, dt, a_log, b, c, checkpoints, d_skip, dt_bias, z, dstate_out, lengths, out)
    head, T, dev, full, bc = _scan_args(u, dt, a_log, b, c, d_skip, dt_bias, z)
    B, N, D, S = head[:4]
    device = u.device
    kept = dense(m.need(checkpoints, "checkpoints"), "checkpoints", (B, -(-N // CHECKPOINT_TOKENS), D, S), F32, dev)
    make = _empty if lengths is None else _zeros

    def new(shape):
        return make(shape, dtype=T, device=device)

    g = {"u": m.given(out, "u", lambda: new(full)), "dt": m.given(out, "dt", lambda: new(full)),
         "z": m.given(out, "z", lambda: new(full)) if z is not None else None,
         "b": m.given(out, "b", lambda: new(bc)), "c": m.given(out, "c", lambda: new(bc)),
         "a_log": torch.empty_like(a_log), "d_skip": torch.empty_like(d_skip) if d_skip is not None else None,
         "dt_bias": torch.empty_like(dt_bias) if dt_bias is not None else None,
         "state": _empty(B, D, S, dtype=F32, device=device)}
    of_bc = rows4 if len(bc) == 4 else rows
    packed = _scan_grad_t.pack(
        *head, 0, 0, dense(lengths, "lengths", (B,), _int32, dev), *NO_ROWS, kept, *rows(dy, "dy", full, T, dev),
        dense(dstate_out, "dstate_out", (B, D, S), F32, dev), *rows(g["u"], "out['u']", full, T, dev),
        *rows(g["dt"], "out['dt']", full, T, dev), *(rows(g["z"], "out['z']", full, T, dev) if z is not None else NO_ROWS),
        *of_bc(g["b"], "out['b']", bc, T, dev), *of_bc(g["c"], "out['c']", bc, T, dev), g["a_log"].data_ptr(),
        _ptr(g["d_skip"]), _ptr(g["dt_bias"]), g["state"].data_ptr())
    n = _scan_backward_workspace(packed)
    ws = _empty(n, dtype=torch.uint8, device=device) if n else None
    r = _scan_backward(packed, _ptr(ws), n, m.handle(dev))
    if r:
        m.failed(r, "gma_scan_backward")
    return g


# ------------------------------------------------------------------ short causal convolution

def conv(x, weight, bias=None, state=None, state_out=None, lengths=None, silu=True, out=None, stream=None):
    """Short causal convolution per channel, with silu unless ``silu`` is False; returns y [B, N, D].

    x [B, N, D]; weight [D, W] (W = 2, 3, 4, the last tap on the current token) and bias [D] fp32; ``state``
    [B, W - 1, D] holds the inputs before the first token, oldest first (zeros if None), and
    ``state_out`` takes the last W - 1 inputs of each row (not in place).
    """
    if stream is not None:
        with m.on_stream(stream):
            return conv(x, weight, bias, state, state_out, lengths, silu, out)
    T, code, dev = m.first(x, "x")
    full = x.shape
    if len(full) != 3:
        raise ValueError("x must be [B, N, D]")
    B, N, D = full
    W = m.last_dim(weight, "weight", 2, "[D, W]")
    past = (B, W - 1, D)
    if out is None:
        out = (_empty if lengths is None else _zeros)(full, dtype=T, device=x.device)
    packed = _conv_t.pack(
        B, N, D, W, code, 0 if silu else GMA_CONV_LINEAR, *rows(x, "x", full, T, dev),
        dense(weight, "weight", (D, W), F32, dev), dense(bias, "bias", (D,), F32, dev),
        dense(state, "state", past, T, dev), dense(state_out, "state_out", past, T, dev),
        dense(lengths, "lengths", (B,), _int32, dev), *rows(out, "out", full, T, dev))
    r = _conv_forward(packed, m.handle(dev))
    if r:
        m.failed(r, "gma_conv_forward")
    return out


def conv_step(x, weight, bias, state, silu=True, out=None, stream=None):
    """One token for every sequence; returns y [B, D] and moves ``state`` [B, W - 1, D] on in place."""
    if stream is not None:
        with m.on_stream(stream):
            return conv_step(x, weight, bias, state, silu, out)
    T, code, dev = m.first(x, "x")
    full = x.shape
    if len(full) != 2:
        raise ValueError("x must be [B, D]")
    B, D = full
    W = m.last_dim(weight, "weight", 2, "[D, W]")
    if out is None:
        out = _empty(full, dtype=T, device=x.device)
    h = dense(m.need(state, "state"), "state", (B, W - 1, D), T, dev)
    packed = _conv_t.pack(
        B, 1, D, W, code, 0 if silu else GMA_CONV_LINEAR, *token(x, "x", full, T, dev),
        dense(weight, "weight", (D, W), F32, dev), dense(bias, "bias", (D,), F32, dev), h, h, 0,
        *token(out, "out", full, T, dev))
    r = _conv_step(packed, m.handle(dev))
    if r:
        m.failed(r, "gma_conv_step")
    return out


def conv_backward(dy, x, weight, bias=None, state=None, lengths=None, silu=True, out=None, stream=None):
    """Gradients of sum(dy * y) of ``conv`` with the same arguments; the state counts as a constant.

    Returns a dict: "x" in x's dtype (into ``out`` if given), "weight" and "bias" (None without one) in fp32.
    """
    if stream is not None:
        with m.on_stream(stream):
            return conv_backward(dy, x, weight, bias, state, lengths, silu, out)
    T, code, dev = m.first(x, "x")
    full = x.shape
    if len(full) != 3:
        raise ValueError("x must be [B, N, D]")
    B, N, D = full
    W = m.last_dim(weight, "weight", 2, "[D, W]")
    if out is None:
        out = (_empty if lengths is None else _zeros)(full, dtype=T, device=x.device)
    g = {"x": out, "weight": torch.empty_like(weight), "bias": torch.empty_like(bias) if bias is not None else None}
    packed = _conv_grad_t.pack(
        B, N, D, W, code, 0 if silu else GMA_CONV_LINEAR, *rows(x, "x", full, T, dev),
        dense(weight, "weight", (D, W), F32, dev), dense(bias, "bias", (D,), F32, dev),
        dense(state, "state", (B, W - 1, D), T, dev), 0, dense(lengths, "lengths", (B,), _int32, dev), *NO_ROWS,
        *rows(dy, "dy", full, T, dev), *rows(out, "out", full, T, dev), g["weight"].data_ptr(), _ptr(g["bias"]))
    n = _conv_backward_workspace(packed)
    ws = _empty(n, dtype=torch.uint8, device=x.device) if n else None
    r = _conv_backward(packed, _ptr(ws), n, m.handle(dev))
    if r:
        m.failed(r, "gma_conv_backward")
    return g
