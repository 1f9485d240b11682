"""The selective state space scan and the short causal convolution in front of it, on torch CUDA
tensors: a binding over ``gma_scan_*`` and ``gma_conv_*`` (``include/gma_block.h``).

Activations are token-major, [B, N, channels], bf16 or fp32, with contiguous channels and any strides
between tokens and batch rows, so that they can be parts of a wider projection's rows.  Parameters
and scan states are contiguous fp32.  ``lengths`` (int32 [B] on the device) gives each batch row's number
of tokens; the rows behind them are neither read nor written (in outputs allocated here they are zero).
"""
import ctypes

import torch

from . import _marshal as m
from ._marshal import F32

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

CHECKPOINT_TOKENS = 128
GMA_CONV_LINEAR = 0x1


def _workspace(size, packed, device):
    n = size(packed)
    return (torch.empty(n, dtype=torch.uint8, device=device), n) if n else (None, 0)


def _ptr(t):
    return 0 if t is None else t.data_ptr()


# ------------------------------------------------------------------ selective scan

def _scan_args(u, dt, a_log, b, c, d_skip, dt_bias, z):
    """(sizes, packed rows of u, dt, z, b, c, packed parameters) of a call on [B, N, D]."""
    code = m.code(u, "u")
    T = u.dtype
    if u.dim() != 3:
        raise ValueError("u must be [B, N, D]")
    B, N, D = u.shape
    if not isinstance(a_log, torch.Tensor) or a_log.dim() != 2:
        raise ValueError("a_log must be [D, S]")
    S = a_log.shape[1]
    bc = (B, N, S)
    G = 1
    if isinstance(b, torch.Tensor) and b.dim() == 4:
        G = b.shape[2]
        bc = (B, N, G, S)
    rows = m.rows(u, "u", (B, N, D), T, u) + m.rows(m.need(dt, "dt"), "dt", (B, N, D), T, u) + \
        m.rows(z, "z", (B, N, D), T, u) + m.rows(m.need(b, "b"), "b", bc, T, u) + \
        m.rows(m.need(c, "c"), "c", bc, T, u)
    params = (m.dense(a_log, "a_log", (D, S), F32, u), m.dense(d_skip, "d_skip", (D,), F32, u),
              m.dense(dt_bias, "dt_bias", (D,), F32, u))
    return (B, N, D, S, G, code), rows, params, bc


def scan_checkpoints(u, S):
    """An uninitialised buffer for the states that ``scan`` keeps for ``scan_backward``."""
    B, N, D = u.shape
    return torch.empty(B, -(-N // CHECKPOINT_TOKENS), D, S, dtype=F32, device=u.device)


def scan(u, dt, a_log, b, c, d_skip=None, dt_bias=None, z=None, state=None, state_out=None, lengths=None,
         checkpoints=None, out=None, stream=None):
    """Selective state space scan; returns y [B, N, D].

    u, dt and z [B, N, D], b and c [B, N, S] or [B, N, G, S] share one dtype; a_log [D, S], d_skip [D] and
    dt_bias [D] are fp32.  ``state`` [B, D, S] is the state before the first token (zeros if None);
    ``state_out`` takes the one after each row's last token and may be ``state``; ``checkpoints`` (from
    ``scan_checkpoints``) takes what ``scan_backward`` needs.  S is 8, 16, 32 or 64.
    """
    sizes, rows, params, _ = _scan_args(u, dt, a_log, b, c, d_skip, dt_bias, z)
    B, N, D, S = sizes[:4]
    with m.on_stream(stream) as st:
        if out is None:
            make = torch.empty if lengths is None else torch.zeros
            out = make(B, N, D, dtype=u.dtype, device=u.device)
        packed = _scan_t.pack(
            *sizes, *rows, *params, m.dense(state, "state", (B, D, S), F32, u),
            m.dense(state_out, "state_out", (B, D, S), F32, u), m.dense(lengths, "lengths", (B,), torch.int32, u),
            *m.rows(out, "out", (B, N, D), u.dtype, u),
            m.dense(checkpoints, "checkpoints", (B, -(-N // CHECKPOINT_TOKENS), D, S), F32, u))
        ws, n = _workspace(_scan_workspace, packed, u.device)
        m.call(_scan_forward, packed, _ptr(ws), n, st)
    return out


def scan_step(u, dt, a_log, b, c, state, d_skip=None, dt_bias=None, z=None, out=None, stream=None):
    """One token for every sequence; returns y [B, D] and updates ``state`` [B, D, S] in place.

    u, dt and z [B, D], b and c [B, S] or [B, G, S]; parameters as in ``scan``.
    """
    code = m.code(u, "u")
    T = u.dtype
    if u.dim() != 2:
        raise ValueError("u must be [B, D]")
    B, D = u.shape
    if not isinstance(a_log, torch.Tensor) or a_log.dim() != 2:
        raise ValueError("a_log must be [D, S]")
    S = a_log.shape[1]
    G = b.shape[1] if isinstance(b, torch.Tensor) and b.dim() == 3 else 1
    bc = (B, 1, G, S) if isinstance(b, torch.Tensor) and b.dim() == 3 else (B, 1, S)
    with m.on_stream(stream) as st:
        if out is None:
            out = torch.empty(B, D, dtype=T, device=u.device)
        h = m.dense(m.need(state, "state"), "state", (B, D, S), F32, u)
        packed = _scan_t.pack(
            B, 1, D, S, G, code, *m.token(u, "u", (B, 1, D), T, u), *m.token(m.need(dt, "dt"), "dt", (B, 1, D), T, u),
            *m.token(z, "z", (B, 1, D), T, u), *m.token(m.need(b, "b"), "b", bc, T, u),
            *m.token(m.need(c, "c"), "c", bc, T, u), m.dense(a_log, "a_log", (D, S), F32, u),
            m.dense(d_skip, "d_skip", (D,), F32, u), m.dense(dt_bias, "dt_bias", (D,), F32, u), h, h, 0,
            *m.token(out, "out", (B, 1, D), T, u), 0)
        m.call(_scan_step, packed, st)
    return out


def scan_backward(dy, u, dt, a_log, b, c, checkpoints, d_skip=None, dt_bias=None, z=None, dstate_out=None,
                  lengths=None, out=None, stream=None):
    """Gradients of sum(dy * y) + sum(dstate_out * state_out) of ``scan`` with the same arguments.

    ``checkpoints`` are those that ``scan`` kept.  Returns a dict with the gradients "u", "dt", "z" (None
    without z), "b", "c" in the activations' dtype, "a_log", "d_skip", "dt_bias" (None where the parameter
    is) and "state" (of the state before the first token) in fp32.  ``out`` may hold tensors, under
    the names "u", "dt", "z", "b" and "c", that take those gradients (rows with strides).
    """
    sizes, rows, params, bc = _scan_args(u, dt, a_log, b, c, d_skip, dt_bias, z)
    B, N, D, S = sizes[:4]
    T, dev = u.dtype, u.device
    full = (B, N, D)
    kept = m.dense(m.need(checkpoints, "checkpoints"), "checkpoints", (B, -(-N // CHECKPOINT_TOKENS), D, S), F32, u)
    with m.on_stream(stream) as st:
        make = torch.empty if lengths is None else torch.zeros

        def new(shape):
            return make(shape, dtype=T, device=dev)

        g = {"u": m.given(out, "u", lambda: new(full)), "dt": m.given(out, "dt", lambda: new(full)),
             "z": m.given(out, "z", lambda: new(full)) if z is not None else None,
             "b": m.given(out, "b", lambda: new(bc)), "c": m.given(out, "c", lambda: new(bc)),
             "a_log": torch.empty_like(a_log), "d_skip": torch.empty_like(d_skip) if d_skip is not None else None,
             "dt_bias": torch.empty_like(dt_bias) if dt_bias is not None else None,
             "state": torch.empty(B, D, S, dtype=F32, device=dev)}
        packed = _scan_grad_t.pack(
            *sizes, *rows, *params, 0, 0, m.dense(lengths, "lengths", (B,), torch.int32, u), *m.NO_ROWS, kept,
            *m.rows(m.need(dy, "dy"), "dy", full, T, u), m.dense(dstate_out, "dstate_out", (B, D, S), F32, u),
            *m.rows(g["u"], "out['u']", full, T, u), *m.rows(g["dt"], "out['dt']", full, T, u),
            *m.rows(g["z"], "out['z']", full, T, u), *m.rows(g["b"], "out['b']", bc, T, u),
            *m.rows(g["c"], "out['c']", bc, T, u), g["a_log"].data_ptr(), _ptr(g["d_skip"]), _ptr(g["dt_bias"]),
            g["state"].data_ptr())
        ws, n = _workspace(_scan_backward_workspace, packed, dev)
        m.call(_scan_backward, packed, _ptr(ws), n, st)
    return g


# ------------------------------------------------------------------ short causal convolution

def _conv_shape(x, weight, dims):
    code = m.code(x, "x")
    if x.dim() != dims:
        raise ValueError("x must be [B, N, D]" if dims == 3 else "x must be [B, D]")
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [D, W]")
    return code, weight.shape[1]


def conv(x, weight, bias=None, state=None, state_out=None, lengths=None, silu=True, out=None, stream=None):
    """Short causal convolution per channel, with silu unless ``silu`` is False; returns y [B, N, D].

    x [B, N, D]; weight [D, W] (W = 2, 3, 4, the last tap on the current token) and bias [D] fp32; ``state``
    [B, W - 1, D] holds the inputs before the first token, oldest first (zeros if None), and
    ``state_out`` takes the last W - 1 inputs of each row.
    """
    code, W = _conv_shape(x, weight, 3)
    B, N, D = x.shape
    T, past = x.dtype, (B, W - 1, D)
    with m.on_stream(stream) as st:
        if out is None:
            out = (torch.empty if lengths is None else torch.zeros)(B, N, D, dtype=T, device=x.device)
        packed = _conv_t.pack(
            B, N, D, W, code, 0 if silu else GMA_CONV_LINEAR, *m.rows(x, "x", (B, N, D), T, x),
            m.dense(weight, "weight", (D, W), F32, x), m.dense(bias, "bias", (D,), F32, x),
            m.dense(state, "state", past, T, x), m.dense(state_out, "state_out", past, T, x),
            m.dense(lengths, "lengths", (B,), torch.int32, x), *m.rows(out, "out", (B, N, D), T, x))
        m.call(_conv_forward, packed, st)
    return out


def conv_step(x, weight, bias, state, silu=True, out=None, stream=None):
    """One token for every sequence; returns y [B, D] and moves ``state`` [B, W - 1, D] on in place."""
    code, W = _conv_shape(x, weight, 2)
    B, D = x.shape
    T = x.dtype
    with m.on_stream(stream) as st:
        if out is None:
            out = torch.empty(B, D, dtype=T, device=x.device)
        h = m.dense(m.need(state, "state"), "state", (B, W - 1, D), T, x)
        packed = _conv_t.pack(
            B, 1, D, W, code, 0 if silu else GMA_CONV_LINEAR, *m.token(x, "x", (B, 1, D), T, x),
            m.dense(weight, "weight", (D, W), F32, x), m.dense(bias, "bias", (D,), F32, x), h, h, 0,
            *m.token(out, "out", (B, 1, D), T, x))
        m.call(_conv_step, packed, st)
    return out


def conv_backward(dy, x, weight, bias=None, state=None, lengths=None, silu=True, out=None, stream=None):
    """Gradients of sum(dy * y) of ``conv`` with the same arguments; the state counts as a constant.

    Returns a dict: "x" in x's dtype (into ``out`` if given), "weight" and "bias" (None without one) in fp32.
    """
    code, W = _conv_shape(x, weight, 3)
    B, N, D = x.shape
    T = x.dtype
    with m.on_stream(stream) as st:
        if out is None:
            out = (torch.empty if lengths is None else torch.zeros)(B, N, D, dtype=T, device=x.device)
        g = {"x": out, "weight": torch.empty_like(weight), "bias": torch.empty_like(bias) if bias is not None else None}
        packed = _conv_grad_t.pack(
            B, N, D, W, code, 0 if silu else GMA_CONV_LINEAR, *m.rows(x, "x", (B, N, D), T, x),
            m.dense(weight, "weight", (D, W), F32, x), m.dense(bias, "bias", (D,), F32, x),
            m.dense(state, "state", (B, W - 1, D), T, x), 0, m.dense(lengths, "lengths", (B,), torch.int32, x),
            *m.NO_ROWS, *m.rows(m.need(dy, "dy"), "dy", (B, N, D), T, x), *m.rows(out, "out", (B, N, D), T, x),
            g["weight"].data_ptr(), _ptr(g["bias"]))
        ws, n = _workspace(_conv_backward_workspace, packed, x.device)
        m.call(_conv_backward, packed, _ptr(ws), n, st)
    return g
