"""Host-side checks of include/gma_block.h (no GPU needed): the packed structs have the header's layout,
workspace sizes, and refusals before anything is enqueued."""
import ctypes
import os
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20          # never dereferenced: validation fails first, or there is no device
NONE = (0, 0, 0)


def _layout(fmt):
    """A struct of the header: fields in order, no padding (the header's structs have none); R: gma_rows_t."""
    return struct.Struct("=" + fmt.replace("R", "Qqq"))


SCAN, CONV, NORM = "6i2IRRRRR6QRQ", "5iIR5QR", "7ifRqRR3QRR"


@pytest.fixture(scope="module")
def lib():
    from linear_latent_routing_gb300 import build
    build.build()
    from linear_latent_routing_gb300 import gma, norm, ssm

    def fn(name, *argtypes, restype=ctypes.c_int):
        f = getattr(gma.lib, name)
        f.argtypes, f.restype = list(argtypes), restype
        return f
    vp, sz = ctypes.c_void_p, ctypes.c_size_t

    class ssm_:
        scan, conv = ssm.scan, ssm.conv
        _scan_t, _scan_grad_t = _layout(SCAN), _layout(SCAN + "RQRRRRR4Q")
        _conv_t, _conv_grad_t = _layout(CONV), _layout(CONV + "RR2Q")
        _scan_forward = fn("gma_scan_forward", vp, vp, sz, vp)
        _scan_step = fn("gma_scan_step", vp, vp)
        _scan_backward = fn("gma_scan_backward", vp, vp, sz, vp)
        _scan_backward_workspace = fn("gma_scan_backward_workspace_size", vp, restype=sz)
        _conv_forward = fn("gma_conv_forward", vp, vp)
        _conv_step = fn("gma_conv_step", vp, vp)
        _conv_backward = fn("gma_conv_backward", vp, vp, sz, vp)
        _conv_backward_workspace = fn("gma_conv_backward_workspace_size", vp, restype=sz)

    class norm_:
        block_norm = norm.block_norm
        _norm_t, _norm_grad_t = _layout(NORM), _layout(NORM + "RRRqRR3Q")
        _norm_forward = fn("gma_norm_forward", vp, vp)
        _norm_backward = fn("gma_norm_backward", vp, vp, sz, vp)
        _norm_backward_workspace = fn("gma_norm_backward_workspace_size", vp, restype=sz)

    class L:
        ssm, norm = ssm_, norm_
    return L


def _rows(width, N=10, ptr=FAKE):
    return (ptr, N * width, width)


def _scan(lib, grad=False, **kw):
    d = dict(B=2, N=10, D=24, S=16, G=1, dtype=1, flags=0, reserved=0, a_log=FAKE, d_skip=FAKE, dt_bias=FAKE, state_in=0, state_out=0,
             lengths=0, ckpt=FAKE if grad else 0)
    width = kw.get("D", 24)
    gs = kw.get("G", 1) * kw.get("S", 16)
    d.update(u=_rows(width), dt=_rows(width), z=NONE, b=_rows(gs), c=_rows(gs), y=_rows(width))
    d.update(dy=_rows(width), dstate_out=0, du=_rows(width), ddt=_rows(width), dz=NONE, db=_rows(gs), dc=_rows(gs),
             da=FAKE, dd=FAKE, dbias=FAKE, dstate_in=0)
    d.update(kw)
    head = (d["B"], d["N"], d["D"], d["S"], d["G"], d["dtype"], d["flags"], d["reserved"], *d["u"], *d["dt"], *d["z"], *d["b"], *d["c"], d["a_log"],
            d["d_skip"], d["dt_bias"], d["state_in"], d["state_out"], d["lengths"], *d["y"], d["ckpt"])
    if not grad:
        return lib.ssm._scan_t.pack(*head)
    return lib.ssm._scan_grad_t.pack(*head, *d["dy"], d["dstate_out"], *d["du"], *d["ddt"], *d["dz"], *d["db"], *d["dc"],
                                     d["da"], d["dd"], d["dbias"], d["dstate_in"])


def _conv(lib, grad=False, **kw):
    d = dict(B=2, N=10, D=24, W=4, dtype=1, flags=0, x=_rows(24), weight=FAKE, bias=FAKE, state_in=0, state_out=0,
             lengths=0, y=_rows(24), dy=_rows(24), dx=_rows(24), dw=FAKE, db=FAKE)
    d.update(kw)
    head = (d["B"], d["N"], d["D"], d["W"], d["dtype"], d["flags"], *d["x"], d["weight"], d["bias"], d["state_in"],
            d["state_out"], d["lengths"], *d["y"])
    if not grad:
        return lib.ssm._conv_t.pack(*head)
    return lib.ssm._conv_grad_t.pack(*head, *d["dy"], *d["dx"], d["dw"], d["db"])


def _norm(lib, grad=False, **kw):
    d = dict(B=2, N=10, H=2, d=16, group=32, dtype=1, rdtype=0, eps=1e-6, o=(FAKE, 320, 16), o_head=160, gate=_rows(32),
             residual=_rows(32), w_post=FAKE, scale=FAKE, w_pre=FAKE, r=_rows(32), h=_rows(32), dr=_rows(32), dh=_rows(32),
             do=(FAKE, 320, 16), do_head=160, dgate=_rows(32), dres=_rows(32), dwpost=FAKE, dscale=FAKE, dwpre=FAKE)
    d.update(kw)
    head = (d["B"], d["N"], d["H"], d["d"], d["group"], d["dtype"], d["rdtype"], d["eps"], *d["o"], d["o_head"], *d["gate"],
            *d["residual"], d["w_post"], d["scale"], d["w_pre"], *d["r"], *d["h"])
    if not grad:
        return lib.norm._norm_t.pack(*head)
    return lib.norm._norm_grad_t.pack(*head, *d["dr"], *d["dh"], *d["do"], d["do_head"], *d["dgate"], *d["dres"],
                                      d["dwpost"], d["dscale"], d["dwpre"])


def test_packed_structs_have_the_header_layout(lib, tmp_path):
    src = tmp_path / "sizes.c"
    names = ("gma_scan_t", "gma_scan_grad_t", "gma_conv_t", "gma_conv_grad_t", "gma_norm_t", "gma_norm_grad_t")
    fields = {"gma_scan_t": ("u", "a_log", "y", "checkpoints"), "gma_scan_grad_t": ("dy", "dc", "dstate_in"),
              "gma_conv_t": ("x", "weight", "y"), "gma_conv_grad_t": ("dy", "dbias"),
              "gma_norm_t": ("eps", "o_head", "w_pre", "h"), "gma_norm_grad_t": ("d_o_head", "dresidual", "dw_pre")}
    body = "".join(f'printf("%zu ", sizeof({n}));' for n in names)
    body += "".join(f'printf("%zu ", offsetof({n}, {f}));' for n in names for f in fields[n])
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gma_block.h"\nint main(void){' + body + "return 0;}\n")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    s, n = lib.ssm, lib.norm
    sizes = [x.size for x in (s._scan_t, s._scan_grad_t, s._conv_t, s._conv_grad_t, n._norm_t, n._norm_grad_t)]
    assert got[:6] == sizes
    # field offsets, by the packed position of a marked value
    assert got[6:] == [32, 152, 200, 224, 232, 360, 408, 24, 48, 88, 112, 168, 28, 56, 128, 160, 256, 288, 328]


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), 1), (dict(N=0), 1), (dict(D=-1), 1), (dict(G=5), 1), (dict(dtype=2), 1), (dict(S=12), 2), (dict(S=128), 2),
    (dict(B=65536), 2), (dict(u=NONE), 1), (dict(dt=(FAKE + 1, 240, 24)), 1), (dict(b=(FAKE, -1, 16)), 1),
    (dict(a_log=0), 1), (dict(a_log=FAKE + 4), 1), (dict(state_in=FAKE + 8), 1), (dict(y=NONE), 1),
    (dict(y=(FAKE, 240, 23)), 1), (dict(y=(FAKE, 100, 24)), 1), (dict(lengths=FAKE + 2), 1), (dict(flags=1), 1), (dict(reserved=1), 1)])
def test_scan_refusals(lib, bad, status):
    assert lib.ssm._scan_forward(_scan(lib, **bad), None, 0, None) == status


def test_scan_step_refusals(lib):
    step = lib.ssm._scan_step
    one = dict(N=1, state_in=FAKE, state_out=FAKE)
    for bad in (dict(N=2), dict(state_in=0), dict(state_out=0), dict(lengths=FAKE), dict(ckpt=FAKE)):
        assert step(_scan(lib, **{**one, **bad}), None) == 1


@pytest.mark.parametrize("bad,status", [
    (dict(ckpt=0), 1), (dict(dy=NONE), 1), (dict(du=NONE), 1), (dict(db=(FAKE, 160, 8)), 1), (dict(da=0), 1),
    (dict(dd=0), 1), (dict(dbias=0), 1), (dict(z=(FAKE, 240, 24)), 1), (dict(S=24), 2)])
def test_scan_backward_refusals(lib, bad, status):
    assert lib.ssm._scan_backward(_scan(lib, True, **bad), FAKE, 1 << 30, None) == status


def test_scan_workspace(lib):
    g = _scan(lib, True)
    n = lib.ssm._scan_backward_workspace(g)
    assert n > 0 and n % 256 == 0
    assert lib.ssm._scan_backward_workspace(_scan(lib, True, S=12)) == 0
    f = lib.ssm._scan_backward
    assert f(g, FAKE, n - 1, None) == 4 and f(g, FAKE + 16, n, None) == 4 and f(g, None, n, None) == 4


@pytest.mark.parametrize("bad,status", [
    (dict(W=5), 2), (dict(W=1), 2), (dict(flags=4), 1), (dict(x=NONE), 1), (dict(weight=0), 1), (dict(y=(FAKE, 240, 8)), 1),
    (dict(state_in=FAKE + 1), 1), (dict(state_in=FAKE, state_out=FAKE), 1), (dict(D=0), 1), (dict(B=70000), 2)])
def test_conv_refusals(lib, bad, status):
    assert lib.ssm._conv_forward(_conv(lib, **bad), None) == status


def test_conv_step_and_backward_refusals(lib):
    step, back = lib.ssm._conv_step, lib.ssm._conv_backward
    one = dict(N=1, state_in=FAKE, state_out=FAKE)
    for bad in (dict(N=3), dict(state_in=0), dict(state_out=0), dict(lengths=FAKE)):
        assert step(_conv(lib, **{**one, **bad}), None) == 1
    for bad in (dict(dy=NONE), dict(dx=(FAKE, 240, 0)), dict(dw=0), dict(db=0)):
        assert back(_conv(lib, True, **bad), FAKE, 1 << 30, None) == 1
    n = lib.ssm._conv_backward_workspace(_conv(lib, True))
    assert n > 0 and back(_conv(lib, True), FAKE, n - 1, None) == 4


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(dtype=3), 1), (dict(rdtype=5), 1),
    (dict(dtype=0, rdtype=1), 1), (dict(group=0), 2), (dict(group=24), 2), (dict(group=64), 2), (dict(H=2048, d=16, group=8), 2),
    (dict(w_post=0, w_pre=0), 1), (dict(residual=NONE), 1), (dict(o=NONE), 1), (dict(o_head=-1), 1), (dict(r=NONE), 1),
    (dict(h=NONE), 1), (dict(r=(FAKE, 320, 31)), 1)])
def test_norm_refusals(lib, bad, status):
    assert lib.norm._norm_forward(_norm(lib, **bad), None) == status


@pytest.mark.parametrize("bad,status", [
    (dict(dr=NONE, dh=NONE), 1), (dict(w_pre=0), 1), (dict(r=NONE), 1), (dict(do=NONE), 1), (dict(do_head=8), 1),
    (dict(dgate=NONE), 1), (dict(dwpost=0), 1), (dict(dscale=0), 1), (dict(dwpre=0), 1), (dict(group=12), 2)])
def test_norm_backward_refusals(lib, bad, status):
    assert lib.norm._norm_backward(_norm(lib, True, **bad), FAKE, 1 << 30, None) == status


def test_norm_workspace(lib):
    n = lib.norm._norm_backward_workspace(_norm(lib, True))
    assert n > 0 and n % 256 == 0
    assert lib.norm._norm_backward(_norm(lib, True), FAKE, n - 1, None) == 4


def test_null_structs(lib):
    s, n = lib.ssm, lib.norm
    assert s._scan_forward(None, None, 0, None) == 1 and s._scan_step(None, None) == 1
    assert s._scan_backward(None, None, 0, None) == 1 and s._conv_forward(None, None) == 1
    assert s._conv_step(None, None) == 1 and s._conv_backward(None, None, 0, None) == 1
    assert n._norm_forward(None, None) == 1 and n._norm_backward(None, None, 0, None) == 1
    assert s._scan_backward_workspace(None) == 0 and s._conv_backward_workspace(None) == 0
    assert n._norm_backward_workspace(None) == 0


def test_valid_calls_find_no_device_without_a_gpu(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert lib.ssm._scan_forward(_scan(lib), None, 0, None) == 7
    assert lib.ssm._conv_forward(_conv(lib), None) == 7
    assert lib.norm._norm_forward(_norm(lib), None) == 7


def test_bindings_refuse_cpu_tensors(lib):
    import torch
    t = torch.zeros(1, 2, 8)
    with pytest.raises(TypeError):
        lib.ssm.scan(t, t, torch.zeros(8, 16), t, t)
    with pytest.raises(TypeError):
        lib.ssm.conv(t, torch.zeros(8, 4))
    with pytest.raises(TypeError):
        lib.norm.block_norm(t, torch.ones(8))


def test_norm_in_place_takes_the_same_rows_alone(lib):
    """r in place of a residual with other strides (a broadcast one) would be read and written by different threads."""
    import torch
    for bad in (dict(residual=(FAKE, 0, 32)), dict(residual=(FAKE, 320, 0)), dict(r=(FAKE, 640, 32))):
        assert lib.norm._norm_forward(_norm(lib, **bad), None) == 1
    for bad in (dict(dres=(FAKE, 640, 64)), dict(dr=(FAKE, 0, 32))):
        assert lib.norm._norm_backward(_norm(lib, True, **bad), FAKE, 1 << 30, None) == 1
    if not torch.cuda.is_available():      # strides that no row uses do not count
        assert lib.norm._norm_forward(_norm(lib, B=1, residual=(FAKE, 0, 32)), None) == 7
        assert lib.norm._norm_forward(_norm(lib, N=1, r=(FAKE, 320, 7)), None) == 7
        assert lib.norm._norm_backward(_norm(lib, True, B=1, dr=(FAKE, 0, 32)), FAKE, 1 << 30, None) == 7


def test_steps_ignore_token_strides(lib):
    """Strides that the header says are ignored refuse nothing: a call that is otherwise valid gets as far as the device."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    odd = {k: (FAKE, 24, -5) for k in ("u", "dt", "z", "y")}
    odd.update({k: (FAKE, 16, -7) for k in ("b", "c")})
    assert lib.ssm._scan_step(_scan(lib, N=1, state_in=FAKE, state_out=FAKE, **odd), None) == 7
    assert lib.ssm._conv_step(_conv(lib, N=1, state_in=FAKE, state_out=FAKE, x=(FAKE, 24, -1), y=(FAKE, 24, -1)), None) == 7


def test_scan_checkpoint_sizes(lib):
    """64 or 16 tokens, the buffer's bytes, and 0 where no call takes the sizes (2^31 - 1 tokens included)."""
    from linear_latent_routing_gb300 import gma
    tokens, size = gma.lib.gma_scan_checkpoint_tokens, gma.lib.gma_scan_checkpoint_size
    for f, t in ((tokens, ctypes.c_int), (size, ctypes.c_size_t)):
        f.argtypes, f.restype = [ctypes.c_void_p], t
    for B, N, D, S, n in ((2, 301, 384, 8, 16), (4, 2048, 1024, 16, 64), (1, 1, 1, 64, 16), (1, 2 ** 30, 8, 8, 64), (65535, 65, 8, 32, 64)):
        c = _scan(lib, B=B, N=N, D=D, S=S)
        assert tokens(c) == n and size(c) == B * -(-N // n) * D * S * 4
    for bad in (dict(N=2 ** 31 - 1), dict(N=2 ** 30 + 1), dict(S=12), dict(S=128), dict(B=0), dict(N=-1), dict(D=0), dict(B=65536),
                dict(D=2 ** 24 + 1)):
        c = _scan(lib, **bad)
        assert tokens(c) == 0 and size(c) == 0, bad
    assert tokens(None) == 0 and size(None) == 0
