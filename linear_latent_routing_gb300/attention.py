"""Softmax attention on torch CUDA tensors, the exact layers of a hybrid stack beside the latent-routing mixer and the
selective scan: a binding over ``gma_attn_*`` (``include/gma_block.h``).

Whole sequences (``prompt``) with their backward pass, and new tokens over a cache of pages (``append``, ``paged``).
Tensors are bf16 or fp32, [B, N, heads, width] with any strides but contiguous heads (parts of a projection's rows,
or the mixers' [B, H, N, d] through ``transpose(1, 2)``); width is at most 128 and may differ between keys and values.  Query head h
of H reads key and value head h // (H // G) of G.

Sequences of different lengths are padded (``lengths``, int32 [B] on the device) or packed: [T, heads, width]
with ``offsets`` (int32 [B + 1] on the device, sequence b is rows offsets[b] to offsets[b + 1] - 1).  Rows of no sequence
are not written (in outputs allocated here they are zero), and nothing in them enters a result.  The elements of a sequence must be
finite; where they are not, that sequence's outputs are unspecified and other sequences' keep their bits.

``stream`` is the stream to run on (default: the current one).  Nothing here waits for the GPU, but with ``check=True``, which
raises on a time-out recorded on the device.  Tensors that do not fit raise TypeError or ValueError, what the library refuses
raises ``gma.GmaError``.
"""
import torch

from . import gma  # noqa: F401  (loads libgma.so, which _block is linked against)
from . import _block


# ------------------------------------------------------------------ whole sequences

def prompt_lse(q):
    """An uninitialised buffer for the log-sum-exp that ``prompt`` keeps for ``prompt_backward``: fp32 [B, H, N], or
    [H, T] for q [T, H, d]."""
    shape = (q.shape[0], q.shape[2], q.shape[1]) if q.dim() == 4 else (q.shape[1], q.shape[0])
    return torch.empty(shape, dtype=torch.float32, device=q.device)


def prompt(q, k, v, causal=True, scale=None, lengths=None, offsets=None, lse=None, out=None, stream=None, check=False):
    """Attention of every token over its sequence, or with ``causal`` over the tokens up to itself; returns o like q with v's width.

    q [B, N, H, d], k [B, N, G, d] and v [B, N, G, dv] share one dtype; or [T, ...] with ``offsets`` (without: one sequence).
    ``scale`` multiplies the scores (default d ** -0.5); ``lse`` (from ``prompt_lse``) takes every row's log-sum-exp.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return _block.attn_prompt(q, k, v, causal, scale, lengths, offsets, lse, out, check)
    return _block.attn_prompt(q, k, v, causal, scale, lengths, offsets, lse, out, check)


def prompt_backward(do, q, k, v, o, lse, causal=True, scale=None, lengths=None, offsets=None, out=None, stream=None, check=False):
    """Gradients of sum(do * o) of ``prompt`` with the same arguments; ``o`` and ``lse`` are what that call wrote.

    Returns a dict with "q", "k" and "v" in the activations' dtype, those of keys and values summed over the query heads that
    share them.  ``out`` may hold tensors under these names that take the gradients (any strides, contiguous heads).
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return prompt_backward(do, q, k, v, o, lse, causal, scale, lengths, offsets, out, None, check)
    if out and not out.keys() <= {"q", "k", "v"}:
        raise ValueError(f"out takes 'q', 'k' and 'v', not {sorted(out.keys() - {'q', 'k', 'v'})}")
    given = (out.get(x) for x in "qkv") if out else (None,) * 3
    return _block.attn_backward(q, k, v, causal, scale, lengths, offsets, do, o, lse, *given, check)


# ------------------------------------------------------------------ a cache of pages

def append(k, v, k_pages, v_pages, table, lengths, new_lengths=None, offsets=None, stream=None):
    """Writes the new tokens' keys and values to their places in the cache.

    k_pages [pages, page, G, d] and v_pages [pages, page, G, dv]; token t of sequence b lies in slot t % page of page
    table[b, t // page] (int32 [B, P], only entries of existing tokens are read).  ``lengths`` (int32 [B]) counts each
    sequence's tokens with the new ones, which are its last.  k [B, N, G, d] and v [B, N, G, dv] hold N new tokens a sequence, or
    ``new_lengths`` of them; with ``offsets`` they are packed [T, G, .]; [B, G, .] is one token each.  A table entry that names no
    page takes no writes and reads as zeros.
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return _block.attn_append(k, v, k_pages, v_pages, table, lengths, new_lengths, offsets)
    return _block.attn_append(k, v, k_pages, v_pages, table, lengths, new_lengths, offsets)


def paged(q, k_pages, v_pages, table, lengths, new_lengths=None, offsets=None, scale=None, lse=None, out=None, stream=None,
          check=False):
    """Attention of the new tokens over the cache, each over the tokens up to itself; returns o like q with v's width.

    q [B, N, H, d] (``new_lengths``, packed with ``offsets``, or [B, H, d], as in ``append``); the cache as ``append`` left it.  A token
    that sees none (a sequence with more new tokens than ``lengths``) gives zeros.  ``lse`` takes the rows' log-sum-exp, fp32
    [B, H, N] ([H, T] packed, [B, H] for one token each).
    """
    if stream is not None:
        with torch.cuda.stream(stream):
            return _block.attn_paged(q, k_pages, v_pages, table, lengths, new_lengths, offsets, scale, lse, out, check)
    return _block.attn_paged(q, k_pages, v_pages, table, lengths, new_lengths, offsets, scale, lse, out, check)
