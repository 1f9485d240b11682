"""What the bindings of ``include/gma_block.h`` share: checks of torch CUDA tensors and their
marshalling into that header's structs (packed bytes with the C layout, passed by pointer)."""
import ctypes
import struct

import torch

from .gma import GMA_BF16, GMA_F32, GmaError, lib

F32 = torch.float32
CODES = {torch.bfloat16: GMA_BF16, F32: GMA_F32}
NO_ROWS = (0, 0, 0)


def declare(name, *argtypes, restype=ctypes.c_int):
    fn = getattr(lib, name)
    fn.argtypes = list(argtypes)
    fn.restype = restype
    return fn


def layout(fmt):
    """A struct of the header: fields in order, no padding (the header's structs have none)."""
    return struct.Struct("=" + fmt.replace("R", "Qqq"))


def code(t, name):
    """The dtype code of an activation, which fixes the device of the whole call."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    c = CODES.get(t.dtype)
    if c is None:
        raise TypeError(f"{name} must be bf16 or fp32, got {t.dtype}")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} must be on the current CUDA device")
    return c


def _fail(t, name, shape, dtype, like):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != like.get_device():
        raise ValueError(f"{name} must be on the same device as the other tensors")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def rows(t, name, shape, dtype, like):
    """(pointer, batch stride, token stride) of [B, N, channels...] whose channels are contiguous."""
    if t is None:
        return NO_ROWS
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype != dtype or t.get_device() != like.get_device():
        _fail(t, name, shape, dtype, like)
    s = t.stride()
    width = 1
    for k in range(len(shape) - 1, 1, -1):
        if s[k] != width and shape[k] != 1:
            raise ValueError(f"{name}'s channels must be contiguous")
        width *= shape[k]
    return t.data_ptr(), s[0], s[1]


def token(t, name, shape, dtype, like):
    """As rows(), of [B, channels...]: one token for every batch row."""
    if t is None:
        return NO_ROWS
    return rows(t.unsqueeze(1) if isinstance(t, torch.Tensor) else t, name, shape, dtype, like)


def dense(t, name, shape, dtype, like):
    """The pointer of a contiguous tensor, or 0 for None."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype != dtype or t.get_device() != like.get_device():
        _fail(t, name, shape, dtype, like)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def need(t, name):
    if t is None:
        raise TypeError(f"{name} is required")
    return t


def given(out, name, make):
    """The caller's tensor for an output, or a new one."""
    t = out.get(name) if out else None
    return make() if t is None else t


class on_stream:
    """Makes `stream` (or the current stream) the one that new tensors belong to, so that memory
    freed after the call is not handed out again before the call's kernels have run."""

    def __init__(self, stream):
        self._ctx = torch.cuda.stream(stream) if stream is not None else None

    def __enter__(self):
        if self._ctx is not None:
            self._ctx.__enter__()
        return torch.cuda.current_stream().cuda_stream

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)


def call(fn, *args):
    r = fn(*args)
    if r:
        raise GmaError(r, fn.__name__)
