"""Host-side checks of the softmax attention's entry points (no GPU needed): the structs' layout, workspace sizes, refusals before
anything is enqueued, and the reference that the GPU tests compare with."""
import ctypes
import os
import struct
import subprocess

import pytest
import torch

import attn_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20          # never dereferenced: validation fails first, or there is no device
HEADS = "Qqqq"
ATTN = "7iIfI" + HEADS * 4 + "QQQ"
PAGED = ATTN + HEADS * 2 + "3iIqQQ"


@pytest.fixture(scope="module")
def lib():
    from linear_latent_routing_gb300 import build
    build.build()
    from linear_latent_routing_gb300 import gma

    def fn(name, *argtypes, restype=ctypes.c_int):
        f = getattr(gma.lib, name)
        f.argtypes, f.restype = list(argtypes), restype
        return f
    vp, sz = ctypes.c_void_p, ctypes.c_size_t

    class L:
        forward = fn("gma_attn_forward", vp, vp, sz, vp)
        workspace = fn("gma_attn_workspace_size", vp, restype=sz)
        backward = fn("gma_attn_backward", vp, vp, sz, vp)
        backward_workspace = fn("gma_attn_backward_workspace_size", vp, restype=sz)
        append = fn("gma_attn_append", vp, vp)
        paged = fn("gma_attn_paged", vp, vp, sz, vp)
        paged_workspace = fn("gma_attn_paged_workspace_size", vp, restype=sz)
    return L


def _heads(B, N, heads, width, ptr=FAKE):
    return (ptr, N * heads * width, heads * width, width)


def _attn(**kw):
    d = dict(B=2, N=10, H=4, G=2, d=64, dv=32, dtype=1, flags=1, scale=0.125, reserved=0, lse=FAKE, lengths=0, offsets=0)
    B, N, H, G, w, wv = (kw.get(x, d[x]) for x in ("B", "N", "H", "G", "d", "dv"))
    d.update(q=_heads(B, N, H, w), k=_heads(B, N, G, w), v=_heads(B, N, G, wv), o=_heads(B, N, H, wv))
    d.update(kw)
    return (d["B"], d["N"], d["H"], d["G"], d["d"], d["dv"], d["dtype"], d["flags"], d["scale"], d["reserved"], *d["q"], *d["k"], *d["v"],
            *d["o"], d["lse"], d["lengths"], d["offsets"])


def _forward(**kw):
    return struct.pack("=" + ATTN, *_attn(**kw))


def _grad(**kw):
    g = dict(do=_heads(2, 10, 4, 32), dq=_heads(2, 10, 4, 64), dk=_heads(2, 10, 2, 64), dv_=_heads(2, 10, 2, 32))
    g.update({k: kw.pop(k) for k in list(kw) if k in g})
    return struct.pack("=" + ATTN + HEADS * 4, *_attn(**kw), *g["do"], *g["dq"], *g["dk"], *g["dv_"])


def _paged(**kw):
    p = dict(kp=_heads(0, 16, 2, 64), vp=_heads(0, 16, 2, 32), pages=9, page=16, table_pages=5, preserved=0, table_stride=5, table=FAKE,
             cached=FAKE)
    p.update({k: kw.pop(k) for k in list(kw) if k in p})
    kw.setdefault("flags", 0)
    return struct.pack("=" + PAGED, *_attn(**kw), *p["kp"], *p["vp"], p["pages"], p["page"], p["table_pages"], p["preserved"], p["table_stride"],
                       p["table"], p["cached"])


def test_structs_have_the_header_layout(tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gma_block.h"\nint main(void){printf("%zu %zu %zu %zu %zu %zu %zu %zu", '
                   "sizeof(gma_attn_t), sizeof(gma_attn_grad_t), sizeof(gma_attn_paged_t), offsetof(gma_attn_t, q), offsetof(gma_attn_t, lse), "
                   "offsetof(gma_attn_paged_t, k_pages), offsetof(gma_attn_paged_t, pages), offsetof(gma_attn_paged_t, table));return 0;}\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    one = struct.calcsize("=" + ATTN)
    assert got == [one, struct.calcsize("=" + ATTN + HEADS * 4), struct.calcsize("=" + PAGED), 40, 168, one, one + 64, one + 88]


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), 1), (dict(N=0), 1), (dict(H=3), 1), (dict(G=0), 1), (dict(d=0), 1), (dict(dtype=2), 1), (dict(flags=4), 1),
    (dict(reserved=1), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1),
    (dict(lengths=FAKE, offsets=FAKE), 1), (dict(lengths=FAKE + 2), 1), (dict(lse=FAKE + 1), 1), (dict(d=129), 2), (dict(dv=160), 2),
    (dict(B=65536), 2), (dict(N=1 << 28), 2), (dict(q=(0, 1, 1, 1)), 1), (dict(k=(FAKE + 1, 1280, 128, 64)), 1),
    (dict(v=(FAKE, -1, 64, 32)), 1), (dict(o=(FAKE, 1280, 128, 31)), 1), (dict(o=(FAKE, 0, 128, 32)), 1), (dict(o=(FAKE, 1280, 100, 32)), 1)])
def test_forward_refusals(lib, bad, status):
    assert lib.forward(_forward(**bad), FAKE, 1 << 40, None) == status
    assert lib.workspace(_forward(**bad)) == 0


@pytest.mark.parametrize("bad", [dict(lse=0), dict(do=(0, 0, 0, 0)), dict(dq=(FAKE, 2560, 256, 63)), dict(dk=(FAKE, 0, 128, 64)),
                                 dict(dv_=(FAKE + 1, 640, 64, 32)), dict(q=(0, 0, 0, 0))])
def test_backward_refusals(lib, bad):
    assert lib.backward(_grad(**bad), FAKE, 1 << 40, None) == 1


@pytest.mark.parametrize("bad,status", [
    (dict(pages=0), 1), (dict(page=0), 1), (dict(table_pages=0), 1), (dict(table_stride=-1), 1), (dict(table=0), 1), (dict(cached=0), 1),
    (dict(cached=FAKE + 2), 1), (dict(preserved=3), 1), (dict(flags=1), 1), (dict(kp=(0, 0, 0, 0)), 1), (dict(vp=(FAKE, -1, 64, 32)), 1),
    (dict(page=65537), 2), (dict(table_pages=1 << 25), 2)])
def test_paged_refusals(lib, bad, status):
    assert lib.paged(_paged(**bad), FAKE, 1 << 40, None) == status
    assert lib.append(_paged(**bad), None) == status


def test_append_writes_apart(lib):
    assert lib.append(_paged(kp=(FAKE, 0, 128, 64)), None) == 1            # pages on top of one another
    assert lib.append(_paged(k=(0, 0, 0, 0)), None) == 1
    assert lib.paged(_paged(q=(0, 0, 0, 0)), FAKE, 1 << 40, None) == 1


def test_workspaces(lib):
    for need, call, packed in ((lib.workspace, lib.forward, _forward()), (lib.backward_workspace, lib.backward, _grad()),
                               (lib.paged_workspace, lib.paged, _paged())):
        n = need(packed)
        assert n > 0 and n % 256 == 0
        assert call(packed, FAKE, n - 1, None) == 4 and call(packed, FAKE + 16, n, None) == 4 and call(packed, None, n, None) == 4


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("B,N,H,G", [(128, 1, 16, 2), (64, 1, 16, 4), (512, 1, 8, 8), (32, 6, 10, 2)])
def test_parts_take_a_tile_of_one_sequence(lib, dtype, B, N, H, G):
    """A part holds at most a sequence's rows, however many sequences there are: an SM's four parts and two more, dv sums and two numbers a row."""
    pages = dict(kp=(FAKE, 16 * G * 128, G * 128, 128), vp=(FAKE, 16 * G * 128, G * 128, 128), pages=9000, page=16, table_pages=600, table_stride=600)
    n = lib.paged_workspace(_paged(B=B, N=N, H=H, G=G, d=128, dv=128, dtype=dtype, **pages))
    parts = 4 * (152 // G + 1) + 2
    lists = 4096 + 128 * (B + 4 * 152)               # headers, an item of 64 bytes a sequence and part, a join of 32 a part
    assert 0 < n <= parts * H * N * (128 + 2) * 4 + lists


def test_copies_take_what_is_copied(lib):
    """bf16 rows off 16-byte boundaries are copied to dense ones of 64 here: q, k and v in the forward pass, do too in the backward pass."""
    B, N, H, G = 2, 1000, 4, 2
    size = dict(B=B, N=N, H=H, G=G)
    plain, odd = dict(size, d=64, dv=64), dict(size, d=63, dv=63)

    def grads(w):
        return dict(do=_heads(B, N, H, w), dq=_heads(B, N, H, w), dk=_heads(B, N, G, w), dv_=_heads(B, N, G, w))
    dense, slack = 2 * B * N * 64, 5 * 256
    more = lib.workspace(_forward(**odd)) - lib.workspace(_forward(**plain))
    assert dense * (H + 2 * G) <= more <= dense * (H + 2 * G) + slack
    more = lib.backward_workspace(_grad(**odd, **grads(63))) - lib.backward_workspace(_grad(**plain, **grads(64)))
    assert dense * (2 * H + 2 * G) <= more <= dense * (2 * H + 2 * G) + slack


def test_no_device(lib):
    if torch.cuda.is_available():
        pytest.skip("there is a device")
    assert lib.forward(_forward(), FAKE, 1 << 40, None) == 7
    assert lib.append(_paged(), None) == 7


def test_tensors_are_checked():
    from linear_latent_routing_gb300 import attention
    x = torch.zeros(2, 3, 4, 8)
    with pytest.raises(TypeError):
        attention.prompt(x, x, x)
    with pytest.raises(TypeError):
        attention.paged(x, x, x, None, None)
    with pytest.raises(ValueError):
        attention.prompt_backward(x, x, x, x, x, None, out={"o": x})
    assert attention.prompt_lse(x).shape == (2, 4, 3) and attention.prompt_lse(x[0]).shape == (4, 3)


@pytest.mark.parametrize("first,causal", [(0, True), (0, False), (4, True)])
def test_reference_against_autograd(first, causal):
    g = torch.Generator().manual_seed(0)
    n, L = 5, 9
    q, k, v, do = (torch.randn(*s, generator=g) for s in ((n, 4, 8), (L, 2, 8), (L, 2, 6), (n, 4, 6)))
    leaf = [t.double().requires_grad_() for t in (q, k, v)]
    s = torch.einsum("ihd,jhd->hij", leaf[0], leaf[1].repeat_interleave(2, 1)) * 0.3
    if causal:
        s = s.masked_fill(torch.arange(L) > first + torch.arange(n)[:, None], float("-inf"))
    o = torch.einsum("hij,jhd->ihd", s.softmax(-1), leaf[2].repeat_interleave(2, 1))
    o.backward(do.double())
    for got, want in zip(R.attend(q, k, v, 0.3, first, causal, do), (o, s.logsumexp(-1), *[t.grad for t in leaf])):
        assert torch.allclose(got[0], want, rtol=1e-12, atol=1e-12)
        assert (got[1] >= 0).all()
