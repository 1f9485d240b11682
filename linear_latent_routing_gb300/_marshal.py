"""What the bindings of ``include/gma_block.h`` share: checks of torch CUDA tensors and their
marshalling into that header's structs (packed bytes with the C layout, passed by pointer).

A call for one token takes a few microseconds on the GPU, so what runs per tensor here is kept to
one comparison of shape, dtype and device and one look at the strides; the words of an error are only
looked for once something does not fit.
"""
import ctypes
import struct

import torch

from .gma import GMA_BF16, GMA_F32, GmaError, lib

F32 = torch.float32
CODES = {torch.bfloat16: GMA_BF16, F32: GMA_F32}
NO_ROWS = (0, 0, 0)
_current_device = torch.cuda.current_device
_current_stream = torch._C._cuda_getCurrentRawStream


def declare(name, *argtypes, restype=ctypes.c_int):
    fn = getattr(lib, name)
    fn.argtypes = list(argtypes)
    fn.restype = restype
    return fn


def layout(fmt):
    """A struct of the header: fields in order, no padding (the header's structs have none)."""
    return struct.Struct("=" + fmt.replace("R", "Qqq"))


def first(t, name):
    """(dtype, its code, device) of an activation; they hold for the whole call."""
    try:
        dev, dtype = t.get_device(), t.dtype
    except AttributeError:
        raise TypeError(f"{name} must be a CUDA tensor") from None
    if dev < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    code = CODES.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be bf16 or fp32, got {dtype}")
    if dev != _current_device():
        raise ValueError(f"{name} must be on the current CUDA device")
    return dtype, code, dev


def _fail(t, name, shape, dtype, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the same device as the other tensors")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name}'s channels must be contiguous")


def rows(t, name, shape, dtype, dev):
    """(pointer, batch stride, token stride) of [B, N, channels] whose channels are contiguous."""
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == dev:
            s = t.stride()
            if s[2] == 1 or shape[2] == 1:
                return t.data_ptr(), s[0], s[1]
    except AttributeError:
        pass
    _fail(t, name, shape, dtype, dev)


def rows4(t, name, shape, dtype, dev):
    """As rows(), of [B, N, groups, values] with a token's values contiguous."""
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == dev:
            s = t.stride()
            if (s[3] == 1 or shape[3] == 1) and (s[2] == shape[3] or shape[2] == 1):
                return t.data_ptr(), s[0], s[1]
    except AttributeError:
        pass
    _fail(t, name, shape, dtype, dev)


def token(t, name, shape, dtype, dev):
    """As rows(), of [B, channels]: one token for every batch row."""
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == dev:
            s = t.stride()
            if s[1] == 1 or shape[1] == 1:
                return t.data_ptr(), s[0], 0
    except AttributeError:
        pass
    _fail(t, name, shape, dtype, dev)


def token3(t, name, shape, dtype, dev):
    """As token(), of [B, groups, values]."""
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == dev:
            s = t.stride()
            if (s[2] == 1 or shape[2] == 1) and (s[1] == shape[2] or shape[1] == 1):
                return t.data_ptr(), s[0], 0
    except AttributeError:
        pass
    _fail(t, name, shape, dtype, dev)


def heads(t, name, shape, dtype, dev):
    """(pointer, batch stride, token stride, head stride) of [B, H, N, d] or [B, N, D]."""
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == dev:
            s = t.stride()
            if s[-1] == 1 or shape[-1] == 1:
                return (t.data_ptr(), s[0], s[2], s[1]) if len(s) == 4 else (t.data_ptr(), s[0], s[1], 0)
    except AttributeError:
        pass
    _fail(t, name, shape, dtype, dev)


def dense(t, name, shape, dtype, dev):
    """The pointer of a contiguous tensor, or 0 for None."""
    if t is None:
        return 0
    try:
        if t.shape == shape and t.dtype is dtype and t.get_device() == dev:
            if t.is_contiguous():
                return t.data_ptr()
            raise ValueError(f"{name} must be contiguous")
    except AttributeError:
        pass
    _fail(t, name, shape, dtype, dev)


def need(t, name):
    if t is None:
        raise TypeError(f"{name} is required")
    return t


def last_dim(t, name, dims, what):
    """The size of the last of a parameter's `dims` dimensions."""
    shape = getattr(t, "shape", ())
    if len(shape) != dims:
        raise ValueError(f"{name} must be {what}")
    return shape[-1]


def given(out, name, make):
    """The caller's tensor for an output, or a new one."""
    t = out.get(name) if out else None
    return make() if t is None else t


class on_stream:
    """Makes `stream` the one that new tensors belong to, so that memory freed after the call is not
    handed out again before the call's kernels have run."""

    def __init__(self, stream):
        self._ctx = torch.cuda.stream(stream)

    def __enter__(self):
        self._ctx.__enter__()

    def __exit__(self, *exc):
        self._ctx.__exit__(*exc)


def handle(dev):
    """The current stream's handle (torch.cuda.current_stream().cuda_stream without its Stream object)."""
    return _current_stream(dev)


def failed(r, what):
    raise GmaError(r, what)
