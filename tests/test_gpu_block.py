"""The selective scan, the short convolution and the block norms on the GPU against the 64-bit
references of block_ref.py, with the error bounds derived there (a result may be off by what fp32
arithmetic of the same formulas can be off, and by half a step of its own type)."""
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF, "f32": F32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from linear_latent_routing_gb300 import build
    build.build()


def _ops():
    from linear_latent_routing_gb300 import norm, ssm
    return ssm, norm


def _draw(seed):
    g = torch.Generator()
    g.manual_seed(seed)

    def normal(*shape, dtype=F32, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(dtype)
    return normal


def _cuda(d):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


# ------------------------------------------------------------------ scan

def _scan_inputs(B, N, D, S, G, dtype, z=True, state=True, seed=0, pitch=0):
    """Inputs on the CPU; u, b, c as parts of one tensor's rows, `pitch` elements wider than needed."""
    r = _draw(seed)
    T = TYPES[dtype]
    x = r(B, N, D + 2 * G * S + pitch, dtype=T)
    t = {"u": x[:, :, :D], "b": x[:, :, D:D + G * S].unflatten(2, (G, S)),
         "c": x[:, :, D + G * S:D + 2 * G * S].unflatten(2, (G, S)), "dt": r(B, N, D, dtype=T),
         "a_log": torch.log(torch.arange(1, S + 1).float()) + r(D, S, std=0.2), "d_skip": r(D), "dt_bias": r(D) - 2,
         "z": r(B, N, D, dtype=T) if z else None, "state": r(B, D, S) if state else None}
    return t, r(B, N, D, dtype=T), r(B, D, S)


def _on_gpu(t):
    """To the GPU with the strides kept."""
    base = t["u"]._base.cuda() if t["u"]._base is not None else None
    out = {}
    for k, v in t.items():
        if isinstance(v, torch.Tensor) and v._base is not None and base is not None and k in "ubc":
            out[k] = base.as_strided(v.shape, v.stride(), v.storage_offset())
        else:
            out[k] = v.cuda() if isinstance(v, torch.Tensor) else v
    return out


def _run_scan(t, lengths=None, state_out=True, ckpt=False, out=None):
    ssm, _ = _ops()
    d = _on_gpu(t)
    h = torch.full((t["u"].shape[0], t["u"].shape[2], t["a_log"].shape[1]), float("nan"), device="cuda") if state_out else None
    ck = ssm.scan_checkpoints(d["u"], t["a_log"].shape[1]).fill_(float("nan")) if ckpt else None
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda") if lengths is not None else None
    y = ssm.scan(d["u"], d["dt"], d["a_log"], d["b"], d["c"], d["d_skip"], d["dt_bias"], d["z"], state=d["state"],
                 state_out=h, lengths=ln, checkpoints=ck, out=out)
    return d, y, h, ck, ln


SCANS = [  # B, N, D, S, G, dtype, z, state, lengths, pitch
    (1, 1, 1, 16, 1, "f32", True, True, None, 0),
    (1, 1, 8, 8, 1, "bf16", False, False, None, 0),
    (2, 5, 24, 16, 1, "bf16", True, True, None, 0),
    (3, 129, 40, 16, 2, "f32", True, False, [129, 0, 128], 0),
    (2, 300, 33, 32, 1, "f32", False, True, [300, 1], 3),
    (2, 130, 18, 64, 2, "bf16", True, True, [127, 130], 5),
    (1, 257, 72, 8, 3, "bf16", False, False, None, 8),
    (4, 64, 16, 16, 1, "f32", True, True, [64, 63, -3, 999], 0),
    (1, 640, 20, 16, 1, "bf16", True, False, None, 0),
]


def _id(c):
    return "-".join(str(x) for x in c[:6]) + ("-z" if c[6] else "") + ("-s" if c[7] else "") + ("-l" if c[8] else "")


@pytest.mark.parametrize("case", SCANS, ids=_id)
def test_scan_forward(case):
    B, N, D, S, G, dtype, z, state, lengths, pitch = case
    t, _, _ = _scan_inputs(B, N, D, S, G, dtype, z, state, pitch=pitch)
    _, y, h, _, _ = _run_scan(t, lengths)
    ry, rh = R.scan(**t, lengths=lengths)
    R.check(y, ry, "y")
    R.check(h, rh, "state")


@pytest.mark.parametrize("case", SCANS, ids=_id)
def test_scan_backward(case):
    B, N, D, S, G, dtype, z, state, lengths, pitch = case
    ssm, _ = _ops()
    t, dy, ds = _scan_inputs(B, N, D, S, G, dtype, z, state, seed=1, pitch=pitch)
    d, y, h, ck, ln = _run_scan(t, lengths, ckpt=True)
    ds = ds if state else None
    g = ssm.scan_backward(dy.cuda(), d["u"], d["dt"], d["a_log"], d["b"], d["c"], ck, d["d_skip"], d["dt_bias"], d["z"],
                          dstate_out=ds.cuda() if ds is not None else None, lengths=ln)
    _, _, ref = R.scan(**t, lengths=lengths, dy=dy, dstate_out=ds)
    for k in ("u", "dt", "z", "b", "c", "a_log", "d_skip", "dt_bias", "state"):
        assert (g[k] is None) == (ref[k] is None), k
        if g[k] is not None:
            R.check(g[k], ref[k], k)


BIG_SCANS = [  # calls with enough work for the forward pass in chunks: of 32 to 256 tokens, several and one
    (2, 700, 4096, 16, 1, "bf16", True, True, [700, 301], 0, False),      # 64
    (5, 33, 8192, 8, 2, "f32", False, True, [33, 0, 32, 1, 30], 0, True),   # 32, rows that end in each of the two
    (6, 27, 16384, 16, 1, "bf16", True, False, None, 0, False),           # one chunk
    (2, 900, 1100, 16, 1, "f32", True, False, [900, 513], 1, False),        # rows off 16-byte boundaries
    (1, 500, 4160, 32, 2, "bf16", True, True, None, 0, True),             # one channel a lane
    (2, 260, 2056, 64, 1, "f32", False, True, [260, 65], 0, False),         # two lanes a channel
    (1, 300, 4099, 64, 1, "bf16", True, True, None, 5, True),             # the same, odd
    (16, 1030, 1040, 16, 1, "bf16", False, False, None, 0, True),         # 128
    (16, 1500, 1536, 16, 1, "bf16", True, True, None, 0, False),          # 256
]


@pytest.mark.parametrize("case", BIG_SCANS, ids=_id)
def test_scan_forward_in_chunks(case, monkeypatch):
    monkeypatch.setattr(R, "DEVICE", "cuda")
    B, N, D, S, G, dtype, z, state, lengths, pitch, ckpt = case
    t, _, _ = _scan_inputs(B, N, D, S, G, dtype, z, state, seed=3, pitch=pitch)
    _, y, h, ck, _ = _run_scan(t, lengths, ckpt=ckpt, out=torch.zeros(B, N, D, dtype=TYPES[dtype], device="cuda"))
    ry, rh = R.scan(**t, lengths=lengths)
    R.check(y, ry, "y")
    R.check(h, rh, "state")
    if ckpt:      # the state before the second checkpoint's token
        n = 64 if ck.shape[1] == -(-N // 64) else 16
        assert ck.shape[1] == -(-N // n)
        short = {k: v[:, :n] if k in ("u", "dt", "b", "c", "z") and v is not None else v for k, v in t.items()}
        want = R.scan(**short, lengths=lengths)[1]
        if N > n and lengths is None:
            R.check(ck[:, 1], want, "checkpoint")
        first = t["state"] if state else torch.zeros(B, D, S)
        live = [i for i in range(B) if lengths is None or lengths[i] > 0]
        assert torch.equal(ck[live, 0].cpu(), first[live])


BIG_GRADS = [  # enough work for chunks of 64 tokens
    (2, 700, 1040, 16, 1, "bf16", True, True, [700, 301], 0),
    (3, 129, 8200, 8, 2, "f32", False, True, [128, 0, 129], 0),
    (2, 500, 1001, 32, 1, "f32", True, False, None, 3),
    (1, 450, 520, 64, 2, "bf16", True, True, None, 0),
]


@pytest.mark.parametrize("case", BIG_GRADS, ids=_id)
def test_scan_backward_in_long_chunks(case, monkeypatch):
    monkeypatch.setattr(R, "DEVICE", "cuda")
    B, N, D, S, G, dtype, z, state, lengths, pitch = case
    ssm, _ = _ops()
    t, dy, ds = _scan_inputs(B, N, D, S, G, dtype, z, state, seed=15, pitch=pitch)
    d, y, h, ck, ln = _run_scan(t, lengths, ckpt=True)
    assert ck.shape[1] == -(-N // 64)
    g = ssm.scan_backward(dy.cuda(), d["u"], d["dt"], d["a_log"], d["b"], d["c"], ck, d["d_skip"], d["dt_bias"], d["z"],
                          dstate_out=ds.cuda(), lengths=ln)
    _, _, ref = R.scan(**t, lengths=lengths, dy=dy, dstate_out=ds)
    for k in ("u", "dt", "z", "b", "c", "a_log", "d_skip", "dt_bias", "state"):
        assert (g[k] is None) == (ref[k] is None), k
        if g[k] is not None:
            R.check(g[k], ref[k], k)


def test_scan_without_optional_parameters():
    ssm, _ = _ops()
    t, dy, _ = _scan_inputs(2, 37, 24, 16, 1, "f32", False, False)
    t["d_skip"] = t["dt_bias"] = None
    d, y, h, ck, _ = _run_scan(t, ckpt=True)
    ry, rh, ref = R.scan(**t, dy=dy)
    R.check(y, ry, "y")
    g = ssm.scan_backward(dy.cuda(), d["u"], d["dt"], d["a_log"], d["b"], d["c"], ck)
    assert g["d_skip"] is None and g["dt_bias"] is None and g["z"] is None
    for k in ("u", "dt", "b", "c", "a_log"):
        R.check(g[k], ref[k], k)


def test_scan_rows_behind_the_last_token_are_left_alone():
    ssm, _ = _ops()
    lengths = [0, 7, 130]
    t, dy, _ = _scan_inputs(3, 140, 24, 16, 1, "bf16")
    poison = float("nan")
    for k in ("u", "dt", "z", "b", "c"):
        for i, n in enumerate(lengths):
            t[k][i, n:] = poison
    out = torch.full((3, 140, 24), 7.0, dtype=BF, device="cuda")
    d, y, h, ck, ln = _run_scan(t, lengths, ckpt=True, out=out)
    grads = {k: torch.full(t[k].shape, 5.0, dtype=BF, device="cuda") for k in ("u", "dt", "z", "b", "c")}
    g = ssm.scan_backward(dy.cuda(), d["u"], d["dt"], d["a_log"], d["b"], d["c"], ck, d["d_skip"], d["dt_bias"], d["z"],
                          lengths=ln, out=grads)
    assert torch.isfinite(h).all()
    for i, n in enumerate(lengths):
        assert (y[i, n:] == 7.0).all() and torch.isfinite(y[i, :n]).all()
        for k in grads:
            assert g[k] is grads[k]
            assert (g[k][i, n:] == 5.0).all() and torch.isfinite(g[k][i, :n].float()).all(), k
    for k in ("a_log", "d_skip", "dt_bias", "state"):
        assert torch.isfinite(g[k]).all(), k
    assert torch.equal(h[0], d["state"][0])


@pytest.mark.parametrize("B,N,D,S", [(3, 140, 24, 16), (4, 300, 8200, 8)])
def test_rows_behind_the_last_token_are_zero_in_new_buffers(B, N, D, S):
    """Without a caller's buffer the rows behind a sequence's end come out as zeros (memory that held NaN
    before), whatever kernel takes the call."""
    ssm, _ = _ops()
    lengths = [0, 7, N, 64][:B]
    t, dy, _ = _scan_inputs(B, N, D, S, 1, "bf16")
    d, _, _, ck, ln = _run_scan(t, lengths, ckpt=True)
    x, w, b = d["dt"], _draw(1)(D, 4).cuda(), _draw(2)(D).cuda()

    def dirty():
        for n in (1, 2, 3, 4, 5):
            torch.full((n, B, N, D), float("nan"), dtype=BF, device="cuda")
    dirty()
    y = ssm.scan(d["u"], d["dt"], d["a_log"], d["b"], d["c"], d["d_skip"], d["dt_bias"], d["z"], lengths=ln)
    dirty()
    g = ssm.scan_backward(dy.cuda(), d["u"], d["dt"], d["a_log"], d["b"], d["c"], ck, d["d_skip"], d["dt_bias"], d["z"],
                          lengths=ln)
    dirty()
    f = ssm.conv(x, w, b, lengths=ln)
    dirty()
    gc = ssm.conv_backward(dy.cuda(), x, w, b, lengths=ln)
    for v in (y, g["u"], g["dt"], g["z"], g["b"], g["c"], f, gc["x"]):
        assert torch.isfinite(v.float()).all()
        for i, n in enumerate(lengths):
            assert (v[i, n:] == 0).all()
            assert n == 0 or (v[i, :n] != 0).any()


def test_scan_state_in_place_and_pieces_of_a_sequence():
    """A sequence in pieces, the state updated in place, ends where the whole sequence does; the last
    piece is single tokens."""
    ssm, _ = _ops()
    t, _, _ = _scan_inputs(2, 150, 24, 16, 1, "f32", True, True, seed=4)
    ry, rh = R.scan(**t)
    d = _on_gpu(t)
    h = d["state"].clone()
    got = []
    for a, e in ((0, 1), (1, 130), (130, 147)):
        s = {k: d[k][:, a:e] for k in ("u", "dt", "b", "c", "z")}
        got.append(ssm.scan(s["u"], s["dt"], d["a_log"], s["b"], s["c"], d["d_skip"], d["dt_bias"], s["z"], state=h, state_out=h))
    for i in range(147, 150):
        s = {k: d[k][:, i] for k in ("u", "dt", "b", "c", "z")}
        got.append(ssm.scan_step(s["u"], s["dt"], d["a_log"], s["b"], s["c"], h, d["d_skip"], d["dt_bias"], s["z"])[:, None])
    R.check(torch.cat(got, 1), ry, "y")
    R.check(h, rh, "state")


@pytest.mark.parametrize("B,D,S,G,dtype,z", [(1, 1, 8, 1, "f32", False), (3, 70, 16, 2, "bf16", True),
                                            (130, 33, 32, 1, "bf16", False), (2, 512, 64, 1, "f32", True),
                                            (201, 600, 16, 1, "bf16", True), (201, 601, 16, 1, "f32", False),
                                            (67, 1000, 16, 1, "f32", True), (301, 520, 64, 2, "bf16", True)])
def test_scan_step(B, D, S, G, dtype, z):
    ssm, _ = _ops()
    t, _, _ = _scan_inputs(B, 1, D, S, G, dtype, z, True, seed=6)
    ry, rh = R.scan(**t)
    d = _on_gpu(t)
    s = {k: d[k][:, 0] if d[k] is not None else None for k in ("u", "dt", "b", "c", "z")}
    y = ssm.scan_step(s["u"], s["dt"], d["a_log"], s["b"], s["c"], d["state"], d["d_skip"], d["dt_bias"], s["z"])
    R.check(y, R.X(ry.v[:, 0], ry.e[:, 0]), "y")
    R.check(d["state"], rh, "state")


def test_scan_long_sequence_forgets_and_stays_bounded():
    """5000 tokens of a few channels; large step sizes (delta > 20, decays that underflow to zero) and
    tiny ones among them."""
    t, _, _ = _scan_inputs(1, 5000, 9, 8, 1, "f32", False, True, seed=8)
    t["dt"][:, ::37] = 40.0
    t["dt"][:, 5::41] = -30.0
    _, y, h, _, _ = _run_scan(t)
    ry, rh = R.scan(**t)
    R.check(y, ry, "y")
    R.check(h, rh, "state")


@pytest.mark.parametrize("D", [16, 8208])
def test_scan_of_rates_that_overflow_or_vanish(D):
    """a_log of 100 and of -100: decays of exactly zero and of one, in padded batches too."""
    ssm, _ = _ops()
    t, dy, _ = _scan_inputs(2, 300, D, 8, 1, "f32", True, True, seed=13)
    t["a_log"][:, ::3] = 100.0
    t["a_log"][:, 1::3] = -100.0
    lengths = [300, 37]
    d, y, h, ck, ln = _run_scan(t, lengths, ckpt=True)
    g = ssm.scan_backward(dy.cuda(), d["u"], d["dt"], d["a_log"], d["b"], d["c"], ck, d["d_skip"], d["dt_bias"], d["z"], lengths=ln)
    for v in [y, h] + list(g.values()):
        assert torch.isfinite(v).all()
    # h with a decay of zero is the last token's input, with a decay of one the sum of all
    delta = torch.nn.functional.softplus(t["dt"].double() + t["dt_bias"].double())
    x = (delta * t["u"].double())[..., None] * t["b"].double()
    for i, n in enumerate(lengths):
        assert torch.allclose(h[i, :, ::3].cpu().double(), x[i, n - 1, :, ::3], rtol=1e-5, atol=1e-30)
        # 300 additions and a few roundings of each term
        want = t["state"][i, :, 1::3].double() + x[i, :n, :, 1::3].sum(0)
        scale = (t["state"][i, :, 1::3].double().abs() + x[i, :n, :, 1::3].abs().sum(0))
        assert ((h[i, :, 1::3].cpu().double() - want).abs() <= 400 * 2.0 ** -24 * scale).all()


def test_calls_of_empty_sequences_alone():
    """Every sequence empty, on every path: states pass through, gradients are zero, and what follows on
    the stream sees it."""
    ssm, _ = _ops()
    for D in (16, 8208):
        t, dy, ds = _scan_inputs(2, 130, D, 16, 1, "bf16", True, True, seed=14)
        for _ in range(3):
            d, y, h, ck, ln = _run_scan(t, [0, 0], ckpt=True)
            assert torch.equal(h, d["state"])
            g = ssm.scan_backward(dy.cuda(), d["u"], d["dt"], d["a_log"], d["b"], d["c"], ck, d["d_skip"], d["dt_bias"], d["z"],
                                  dstate_out=ds.cuda(), lengths=ln)
            assert torch.equal(g["state"], ds.cuda())
            for k in ("a_log", "d_skip", "dt_bias", "u", "dt", "z", "b", "c"):
                assert (g[k] == 0).all(), k


def test_scan_strides_beyond_32_bits():
    """Batch rows more than 2^31 elements apart (only the rows themselves are touched)."""
    ssm, _ = _ops()
    t, _, _ = _scan_inputs(2, 9, 16, 16, 1, "bf16", True, False, seed=9)
    gap = 2 ** 31 + 64
    far = torch.empty(gap + 9 * 16, dtype=BF, device="cuda")
    d = _on_gpu(t)
    u = far.as_strided((2, 9, 16), (gap, 16, 1))
    u.copy_(d["u"])
    y = ssm.scan(u, d["dt"], d["a_log"], d["b"], d["c"], d["d_skip"], d["dt_bias"], d["z"], out=u.new_empty(2, 9, 16))
    R.check(y, R.scan(**t)[0], "y")
    ssm.scan(d["u"], d["dt"], d["a_log"], d["b"], d["c"], d["d_skip"], d["dt_bias"], d["z"], out=u)
    assert torch.equal(u.contiguous(), y)


# ------------------------------------------------------------------ convolution

CONVS = [  # B, N, D, W, dtype, silu, bias, state, lengths, pitch
    (1, 1, 1, 2, "f32", True, True, False, None, 0),
    (2, 3, 24, 4, "bf16", True, True, True, None, 0),
    (3, 100, 40, 4, "f32", True, False, True, [100, 0, 2], 0),
    (2, 33, 17, 3, "bf16", False, True, True, [33, 32], 1),
    (2, 64, 520, 4, "bf16", True, True, False, None, 24),
    (4, 47, 8, 2, "f32", True, True, True, [1, 47, 16, 48], 8),
    (2, 2000, 8208, 4, "bf16", True, True, True, [1937, 64], 0),         # runs of 64 tokens
    (1, 4100, 8200, 3, "f32", True, False, False, None, 0),
]


@pytest.mark.parametrize("case", CONVS, ids=lambda c: "-".join(str(x) for x in c[:5]))
def test_conv_forward_and_backward(case):
    B, N, D, W, dtype, silu, bias, state, lengths, pitch = case
    ssm, _ = _ops()
    r, T = _draw(2), TYPES[dtype]
    x = r(B, N, D + pitch, dtype=T)
    t = {"x": x[:, :, :D], "weight": r(D, W, std=0.6), "bias": r(D) if bias else None,
         "state": r(B, W - 1, D, dtype=T) if state else None}
    dy = r(B, N, D, dtype=T)
    ry, after, ref = R.conv(**t, lengths=lengths, silu_=silu, dy=dy)
    d = {k: v.cuda() if v is not None else None for k, v in t.items()}
    d["x"] = x.cuda()[:, :, :D]
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda") if lengths is not None else None
    so = torch.full((B, W - 1, D), float("nan"), dtype=T, device="cuda")
    y = ssm.conv(d["x"], d["weight"], d["bias"], state=d["state"], state_out=so, lengths=ln, silu=silu)
    R.check(y, ry, "y")
    assert torch.equal(so.cpu().double(), after)
    g = ssm.conv_backward(dy.cuda(), d["x"], d["weight"], d["bias"], state=d["state"], lengths=ln, silu=silu)
    for k in ("x", "weight", "bias"):
        assert (g[k] is None) == (ref[k] is None)
        if g[k] is not None:
            R.check(g[k], ref[k], k)


def test_conv_rows_behind_the_last_token_are_left_alone():
    ssm, _ = _ops()
    r = _draw(3)
    lengths = [0, 5, 40]
    x, w, b, dy = r(3, 40, 24, dtype=BF), r(24, 4), r(24), r(3, 40, 24, dtype=BF)
    for i, n in enumerate(lengths):
        x[i, n:] = float("nan")
        dy[i, n:] = float("nan")
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    y, dx = (torch.full((3, 40, 24), 3.0, dtype=BF, device="cuda") for _ in range(2))
    ssm.conv(x.cuda(), w.cuda(), b.cuda(), lengths=ln, out=y)
    g = ssm.conv_backward(dy.cuda(), x.cuda(), w.cuda(), b.cuda(), lengths=ln, out=dx)
    for i, n in enumerate(lengths):
        for v in (y, dx):
            assert (v[i, n:] == 3.0).all() and torch.isfinite(v[i, :n].float()).all()
    assert torch.isfinite(g["weight"]).all() and torch.isfinite(g["bias"]).all()


@pytest.mark.parametrize("B,D,W,dtype", [(1, 1, 2, "f32"), (5, 2080, 4, "bf16"), (3, 37, 3, "bf16")])
def test_conv_steps_continue_the_sequence(B, D, W, dtype):
    ssm, _ = _ops()
    r, T = _draw(5), TYPES[dtype]
    x, w, b = r(B, 9, D, dtype=T), r(D, W), r(D)
    ry, after, _ = R.conv(x, w, b)
    xd, wd, bd = x.cuda(), w.cuda(), b.cuda()
    h = torch.zeros(B, W - 1, D, dtype=T, device="cuda")
    got = [ssm.conv(xd[:, :4], wd, bd, state_out=h)]
    got += [ssm.conv_step(xd[:, i], wd, bd, h)[:, None] for i in range(4, 9)]
    R.check(torch.cat(got, 1), ry, "y")
    assert torch.equal(h.cpu().double(), after)


# ------------------------------------------------------------------ norms

NORMS = [  # B, H, N, d, dtype, group, gate, post, res, scale, pre
    (1, 1, 1, 1, "f32", 0, False, True, None, False, False),
    (2, 2, 3, 16, "bf16", 16, True, True, None, False, False),
    (2, 8, 5, 64, "bf16", 0, True, True, "f32", True, True),
    (1, 4, 7, 128, "bf16", 128, True, True, "bf16", True, True),
    (3, 1, 4, 37, "f32", 0, True, True, "f32", True, True),
    (2, 3, 5, 10, "bf16", 0, False, True, "bf16", False, True),
    (1, 1, 9, 2048, "f32", 256, False, False, "f32", True, True),
    (1, 1, 3, 8200, "bf16", 8, True, True, "f32", True, True),
    (1, 1, 2, 16384, "f32", 0, True, True, "f32", True, True),
    (1, 2, 700, 32, "f32", 32, True, True, None, False, False),
    (2, 1, 6, 333, "bf16", 0, False, False, None, False, True),
    (1, 16, 1301, 128, "bf16", 128, True, True, None, False, False),      # two rows a thread
    (1, 1, 1301, 2048, "f32", 0, True, True, "f32", True, True),
    (1, 32, 5, 128, "bf16", 0, True, True, "f32", True, True),            # 512 threads a row
    (2, 1, 3, 6000, "f32", 0, True, True, "f32", True, True),             # two pieces a thread
    (1, 1, 2, 3003, "bf16", 0, True, True, "bf16", True, True),
]


def _norm_inputs(case, seed=0):
    B, H, N, d, dtype, group, gate, post, res, scale, pre = case
    r, T, D = _draw(seed), TYPES[dtype], H * d
    t = {"o": r(B, H, N, d, dtype=T), "gate": r(B, N, D + 8, dtype=T)[:, :, 8:] if gate else None,
         "w_post": 1 + r(D, std=0.3) if post else None, "residual": r(B, N, D, dtype=TYPES[res], std=2.0) if res else None,
         "scale": r(D, std=0.5) if scale else None, "w_pre": 1 + r(D, std=0.3) if pre else None}
    return t, r(B, N, D, dtype=TYPES[res] if res else T), r(B, N, D, dtype=T) if pre else None


@pytest.mark.parametrize("case", NORMS, ids=lambda c: "-".join(str(x) for x in c))
def test_norm_forward_and_backward(case):
    _, norm = _ops()
    group = case[5]
    t, dr, dh = _norm_inputs(case)
    d = {k: v.cuda() if v is not None else None for k, v in t.items()}
    r, h = norm.block_norm(**d, group=group)
    kept = r.cpu()
    rr, rh, ref = R.norm(**t, group=group, r_stored=kept, dr=dr, dh=dh)
    R.check(r, rr, "r")
    assert (h is None) == (rh is None)
    if h is not None:
        R.check(h, rh, "h")
    g = norm.block_norm_backward(dr.cuda(), d["o"], r, d["w_post"], gate=d["gate"], scale=d["scale"], w_pre=d["w_pre"],
                                 dh=dh.cuda() if dh is not None else None, group=group, residual=t["residual"] is not None)
    for k in ("o", "gate", "residual", "w_post", "scale", "w_pre"):
        assert (g[k] is None) == (ref[k] is None), k
        if g[k] is not None:
            R.check(g[k], ref[k], k)


def test_norm_layouts_and_in_place():
    """The mixer layout by strides, token-major rows and an in-place residual give the same bits."""
    _, norm = _ops()
    t, dr, dh = _norm_inputs((2, 4, 6, 32, "bf16", 0, True, True, "f32", True, True))
    d = {k: v.cuda() if v is not None else None for k, v in t.items()}
    r, h = norm.block_norm(**d)
    rows = d["o"].transpose(1, 2).contiguous()
    for o in (rows.transpose(1, 2), rows.reshape(2, 6, 128)):
        r2, h2 = norm.block_norm(**{**d, "o": o})
        assert torch.equal(r, r2) and torch.equal(h, h2)
    same = d["residual"].clone()
    r3, h3 = norm.block_norm(**{**d, "residual": same}, out=same)
    assert r3 is same and torch.equal(r, r3) and torch.equal(h, h3)
    # gradients of one of the two outputs alone, and of a norm with no gradient for its second weight
    back = dict(w_post=d["w_post"], gate=d["gate"], scale=d["scale"], w_pre=d["w_pre"])
    for a, b in ((dr, None), (None, dh)):
        g = norm.block_norm_backward(a.cuda() if a is not None else None, d["o"], r, **back, dh=b.cuda() if b is not None else None)
        ref = R.norm(**t, r_stored=r.cpu(), dr=a, dh=b)[2]
        for k in ("o", "gate", "residual", "w_post", "scale", "w_pre"):
            R.check(g[k], ref[k], k)


# ------------------------------------------------------------------ together, streams, graphs, bits

def _block(seed=11, B=2, N=70, D=64, S=16, W=4):
    r = _draw(seed)
    return {"xbc": r(B, N, D + 2 * S, dtype=BF), "w": r(D + 2 * S, W, std=0.5), "wb": r(D + 2 * S, std=0.1),
            "dt": r(B, N, D, dtype=BF), "a_log": torch.log(torch.arange(1, S + 1).float()).repeat(D, 1),
            "d_skip": torch.ones(D), "dt_bias": r(D, std=0.3) - 3, "z": r(B, N, D, dtype=BF),
            "res": r(B, N, D), "w_post": torch.ones(D), "scale": r(D, std=0.1), "w_pre": torch.ones(D)}


def _block_forward(p, ckpt=None, out=None):
    ssm, norm = _ops()
    D, S = p["a_log"].shape
    f = ssm.conv(p["xbc"], p["w"], p["wb"])
    u, b, c = f[:, :, :D], f[:, :, D:D + S], f[:, :, D + S:]
    y = ssm.scan(u, p["dt"], p["a_log"], b, c, p["d_skip"], p["dt_bias"], checkpoints=ckpt)
    r, h = norm.block_norm(y, p["w_post"], gate=p["z"], residual=p["res"], scale=p["scale"], w_pre=p["w_pre"])
    return f, y, r, h


def test_block_forward_and_backward_together():
    """Convolution, scan and norms in a row, and their backward passes, each step against its reference on
    the tensors that the GPU handed over."""
    ssm, norm = _ops()
    p = _block()
    g = _cuda(p)
    D, S = p["a_log"].shape
    kept = ssm.scan_checkpoints(g["dt"], S)
    f, y, r, h = _block_forward(g, kept)
    R.check(f, R.conv(p["xbc"], p["w"], p["wb"])[0], "conv")
    fc = f.cpu()
    scan_in = dict(u=fc[:, :, :D], dt=p["dt"], a_log=p["a_log"], b=fc[:, :, D:D + S], c=fc[:, :, D + S:],
                   d_skip=p["d_skip"], dt_bias=p["dt_bias"])
    R.check(y, R.scan(**scan_in)[0], "scan")
    norm_in = dict(o=y.cpu(), w_post=p["w_post"], gate=p["z"], residual=p["res"], scale=p["scale"], w_pre=p["w_pre"])
    rn = _draw(12)
    dr, dh = rn(*r.shape), rn(*h.shape, dtype=BF)
    rr, rh, ref = R.norm(**norm_in, r_stored=r.cpu(), dr=dr, dh=dh)
    R.check(r, rr, "r")
    R.check(h, rh, "h")
    gn = norm.block_norm_backward(dr.cuda(), y, r, g["w_post"], gate=g["z"], scale=g["scale"], w_pre=g["w_pre"], dh=dh.cuda())
    for k in gn:
        R.check(gn[k], ref[k], "norm " + k)
    dy = gn["o"]
    dxbc = torch.empty_like(f)        # the scan's gradients go straight into the convolution's rows
    gs = ssm.scan_backward(dy, f[:, :, :D], g["dt"], g["a_log"], f[:, :, D:D + S], f[:, :, D + S:], kept, g["d_skip"],
                           g["dt_bias"], out={"u": dxbc[:, :, :D], "b": dxbc[:, :, D:D + S], "c": dxbc[:, :, D + S:]})
    ref = R.scan(**scan_in, dy=dy.cpu())[2]
    ref["b"], ref["c"] = (x.map(lambda v: v.squeeze(2)) for x in (ref["b"], ref["c"]))
    for k in ("u", "dt", "b", "c", "a_log", "d_skip", "dt_bias", "state"):
        R.check(gs[k], ref[k], "scan " + k)
    gc = ssm.conv_backward(dxbc, g["xbc"], g["w"], g["wb"])
    ref = R.conv(p["xbc"], p["w"], p["wb"], dy=dxbc.cpu())[2]
    for k in gc:
        R.check(gc[k], ref[k], "conv " + k)


def test_norm_after_the_latent_routing_mixer():
    """gma.forward's output goes into the gated per-head norm as it is."""
    from linear_latent_routing_gb300 import gma, inputs as W
    _, norm = _ops()
    w = W.scaled(W.LM_CAUSAL, B=1, H=3, N=90)
    host = W.make_inputs(w)
    dev = _cuda(host)
    o = gma.forward(dev["QX"], dev["KX"], dev["V"], dev["mu"], dev["raw"], dev["logits"], True, check=True)
    D = w.H * w.d_v
    gate, weight = _draw(1)(1, 90, D, dtype=BF), torch.ones(D)
    v, _ = norm.block_norm(o, weight.cuda(), gate=gate.cuda(), group=w.d_v)
    R.check(v, R.norm(o.cpu(), weight, gate=gate, group=w.d_v)[0], "v")


def test_other_streams_and_captured_graphs():
    """The same bits on another stream and from a captured graph that is replayed on new inputs, with two
    graphs alive."""
    ssm, norm = _ops()
    p = _cuda(_block())
    want = [t.clone() for t in _block_forward(p)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = _block_forward(p)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    y = ssm.conv(p["xbc"], p["w"], p["wb"], stream=s)
    s.synchronize()
    assert torch.equal(y, want[0])
    D, S = p["a_log"].shape
    other = _cuda(_block(seed=77))
    want2 = [t.clone() for t in _block_forward(other)]
    graphs = []
    for _ in range(2):
        kept = ssm.scan_checkpoints(p["dt"], S)
        _block_forward(p, kept)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = _block_forward(p, kept)
            f, yy, r, h = out
            gn = norm.block_norm_backward(r, yy, r, p["w_post"], gate=p["z"], scale=p["scale"], w_pre=p["w_pre"], dh=h)
            gs = ssm.scan_backward(gn["o"], f[:, :, :D], p["dt"], p["a_log"], f[:, :, D:D + S], f[:, :, D + S:], kept,
                                   p["d_skip"], p["dt_bias"])
            gc = ssm.conv_backward(f, p["xbc"], p["w"], p["wb"])
        graphs.append((graph, out, (gn["o"], gs["a_log"], gs["b"], gc["weight"])))
    saved = {k: v.clone() for k, v in p.items()}
    results = []
    for src, expect in ((saved, want), (other, want2)):
        for k in p:
            p[k].copy_(src[k])
        per_graph = []
        for graph, out, grads in graphs:
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, expect):
                assert torch.equal(a, b)
            per_graph.append([x.clone() for x in grads])
        for a, b in zip(*per_graph):
            assert torch.equal(a, b)
        results.append(per_graph[0])
    assert not torch.equal(results[0][0], results[1][0])


def test_repeated_calls_give_the_same_bits():
    ssm, norm = _ops()
    t, dy, ds = _scan_inputs(3, 300, 100, 16, 1, "bf16", seed=5)
    d, y, h, ck, _ = _run_scan(t, ckpt=True)
    runs = []
    for _ in range(2):
        g = ssm.scan_backward(dy.cuda(), d["u"], d["dt"], d["a_log"], d["b"], d["c"], ck, d["d_skip"], d["dt_bias"], d["z"],
                              dstate_out=ds.cuda())
        runs.append(g)
    for k in runs[0]:
        assert torch.equal(runs[0][k], runs[1][k]), k


def test_bindings_refuse_what_does_not_fit():
    ssm, norm = _ops()
    t, dy, _ = _scan_inputs(2, 6, 16, 16, 1, "bf16")
    d = _on_gpu(t)
    ok = dict(u=d["u"], dt=d["dt"], a_log=d["a_log"], b=d["b"], c=d["c"])
    bad = [("dt", d["dt"].float(), TypeError), ("dt", d["dt"][:, :5], ValueError), ("b", d["b"].cpu(), TypeError),
           ("a_log", d["a_log"].t(), ValueError), ("a_log", d["a_log"].double(), TypeError), ("u", d["u"].half(), TypeError),
           ("u", d["u"][0], ValueError), ("c", None, TypeError),
           ("dt", d["dt"].transpose(1, 2).contiguous().transpose(1, 2), ValueError)]
    for k, v, err in bad:
        with pytest.raises(err):
            ssm.scan(**{**ok, k: v})
    from linear_latent_routing_gb300.gma import GmaError
    with pytest.raises(GmaError):
        ssm.scan(**{**ok, "a_log": d["a_log"][:, :12].contiguous(), "b": d["b"][..., :12], "c": d["c"][..., :12]})
    with pytest.raises(TypeError):
        ssm.scan(**ok, lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(GmaError):
        ssm.conv(d["u"], torch.zeros(16, 5, device="cuda"))
    with pytest.raises(GmaError):
        norm.block_norm(d["u"], torch.ones(16, device="cuda"), group=12)
    with pytest.raises(ValueError):
        norm.block_norm(d["u"], torch.ones(15, device="cuda"))


def test_outputs_that_are_inputs_are_refused():
    ssm, norm = _ops()

    def bf(*shape):
        return torch.zeros(*shape, device="cuda", dtype=BF)
    u, dt, b, c, dy = bf(2, 20, 32), bf(2, 20, 32), bf(2, 20, 16), bf(2, 20, 16), bf(2, 20, 32)
    a_log = torch.zeros(32, 16, device="cuda")
    ck = ssm.scan_checkpoints(u, 16)
    ssm.scan(u, dt, a_log, b, c, checkpoints=ck)
    w, wn = torch.zeros(32, 4, device="cuda"), torch.ones(32, device="cuda")
    state = torch.zeros(2, 32, 16, device="cuda")
    same = bf(2, 20, 32)
    for call in (lambda: ssm.scan(u, dt, a_log, b, c, out=u), lambda: ssm.scan(u, dt, a_log, b, c, z=same, out=same),
                 lambda: ssm.scan_step(u[:, 0], dt[:, 0], a_log, b[:, 0], c[:, 0], state, out=dt[:, 0]),
                 lambda: ssm.scan_backward(dy, u, dt, a_log, b, c, ck, out={"u": dy}),
                 lambda: ssm.scan_backward(dy, u, dt, a_log, b, c, ck, out={"u": same, "dt": same}),
                 lambda: ssm.scan_backward(dy, u, dt, a_log, b, c, ck, out={"du": same}),
                 lambda: ssm.conv(u, w, out=u), lambda: ssm.conv_step(u[:, 0], w, None, bf(2, 3, 32), out=u[:, 0]),
                 lambda: ssm.conv_backward(dy, u, w, out=dy), lambda: ssm.conv_backward(dy, u, w, out=u),
                 lambda: norm.block_norm(u, wn, out=u), lambda: norm.block_norm(u, wn, w_pre=wn, out=same, out_h=same),
                 lambda: norm.block_norm_backward(dy, u, same, wn, out=dy)):
        with pytest.raises(ValueError):
            call()
    # parts of one wider buffer's rows are not the same tensor
    wide, want = bf(2, 20, 64), ssm.scan(u, dt, a_log, b, c)
    wide[..., :32] = u
    assert torch.equal(ssm.scan(wide[..., :32], dt, a_log, b, c, out=wide[..., 32:]), want)


def test_norm_backward_takes_the_forward_calls_residual():
    """`residual` may be what the forward call was given (or its in-place result), a truth value or None; what
    has no truth value raises its own error, and rows that are not r's are refused."""
    _, norm = _ops()
    for res, scale in (("bf16", True), ("bf16", False), ("f32", False)):
        t, dr, dh = _norm_inputs((2, 4, 6, 32, "bf16", 0, True, True, res, scale, True), seed=21)
        d = {k: v.cuda() if v is not None else None for k, v in t.items()}
        r, _ = norm.block_norm(**d)
        back = dict(w_post=d["w_post"], gate=d["gate"], scale=d["scale"], w_pre=d["w_pre"], dh=dh.cuda())
        ref = R.norm(**t, r_stored=r.cpu(), dr=dr, dh=dh)[2]
        for residual in (d["residual"], r, True):
            g = norm.block_norm_backward(dr.cuda(), d["o"], r, **back, residual=residual)
            for k in ("o", "gate", "residual", "w_post", "scale", "w_pre"):
                assert (g[k] is None) == (ref[k] is None), k
                if g[k] is not None:
                    R.check(g[k], ref[k], k)
        with pytest.raises(ValueError):
            norm.block_norm_backward(dr.cuda(), d["o"], r, **back, residual=d["residual"][:, :5])
        with pytest.raises(TypeError):
            norm.block_norm_backward(dr.cuda(), d["o"], r, **back, residual=d["residual"].double())

    class Neither:
        def __bool__(self):
            raise KeyError("neither")
    with pytest.raises(KeyError):
        norm.block_norm_backward(dr.cuda(), d["o"], r, **back, residual=Neither())


@pytest.mark.parametrize("D", [16, 8208])
def test_scan_of_a_rate_that_is_not_a_number(D):
    """A NaN in a_log comes out as NaN in what it enters and nowhere else, on every path: over lanes of tokens and
    in chunks, one token, and the backward pass with either spacing of checkpoints."""
    ssm, _ = _ops()
    t, dy, ds = _scan_inputs(2, 130, D, 16, 1, "f32", True, True, seed=22)
    bad, at, state = torch.tensor([5]), 5, 3
    others = torch.tensor([i for i in range(D) if i != at], device="cuda")

    def run():
        d, y, h, ck, _ = _run_scan(t, ckpt=True)
        _, y2, _, _, _ = _run_scan(t)
        g = ssm.scan_backward(dy.cuda(), d["u"], d["dt"], d["a_log"], d["b"], d["c"], ck, d["d_skip"], d["dt_bias"], d["z"],
                              dstate_out=ds.cuda())
        s = {k: d[k][:, 0] for k in ("u", "dt", "b", "c", "z")}
        h1 = d["state"].clone()
        y1 = ssm.scan_step(s["u"], s["dt"], d["a_log"], s["b"], s["c"], h1, d["d_skip"], d["dt_bias"], s["z"])
        return y, y2, h, g, y1, h1
    good = run()
    t["a_log"][bad, state] = float("nan")
    y, y2, h, g, y1, h1 = run()
    for v, w in ((y, good[0]), (y2, good[1]), (y1, good[4])):
        assert v[..., at].isnan().all()
        assert torch.equal(v[..., others], w[..., others])
    for v, w in ((h, good[2]), (h1, good[5])):
        assert v[:, at, state].isnan().all()
        assert torch.equal(v[:, others], w[:, others])
    assert g["a_log"][at, state].isnan()
    assert torch.equal(g["a_log"][others], good[3]["a_log"][others])
    for k in ("u", "dt"):
        assert g[k][..., at].isnan().all() and torch.equal(g[k][..., others], good[3][k][..., others]), k
    assert g["state"][:, at, state].isnan().all() and torch.equal(g["state"][:, others], good[3]["state"][:, others])


def test_scan_calls_from_two_host_threads():
    """Calls of one kernel with different amounts of shared memory from two host threads at once, on streams of their
    own: each gets the launch that it asked for."""
    import ctypes
    import threading

    from linear_latent_routing_gb300 import gma
    from test_block_abi import SCAN, _layout
    forward = gma.lib.gma_scan_forward
    forward.argtypes, forward.restype = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p], ctypes.c_int

    def job(B, N, D, S):
        t = {k: torch.zeros(B, N, n, device="cuda") for k, n in (("u", D), ("dt", D), ("b", S), ("c", S), ("y", D))}
        a_log = torch.zeros(D, S, device="cuda")
        rows = {k: (v.data_ptr(), v.stride(0), v.stride(1)) for k, v in t.items()}
        call = _layout(SCAN).pack(B, N, D, S, 1, 0, 0, 0, *rows["u"], *rows["dt"], 0, 0, 0, *rows["b"], *rows["c"], a_log.data_ptr(),
                                  0, 0, 0, 0, 0, *rows["y"], 0)
        return call, torch.cuda.Stream(), (t, a_log)
    for shapes in (((1, 8, 8, 8), (1, 8, 8, 64)),                  # tokens over lanes: 8 and 64 states
                   ((184, 32, 320, 16), (114, 32, 512, 16))):      # one chunk: blocks of five and of eight warps
        jobs = [job(*s) for s in shapes]
        torch.cuda.synchronize()
        ready, results = threading.Barrier(2), [[], []]

        def work(i):
            call, stream, _ = jobs[i]
            ready.wait()
            for _ in range(2000):
                results[i].append(forward(call, None, 0, stream.cuda_stream))
        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for th in threads:
            th.start()
        for th in threads:
            th.join()
        torch.cuda.synchronize()
        assert [set(r) for r in results] == [{0}, {0}], shapes


def test_scan_checkpoints_of_sizes_that_no_call_takes():
    ssm, _ = _ops()
    u = torch.zeros(1, 1, 8, dtype=BF, device="cuda")
    for tokens, S in ((10, 12), (10, 128), (2 ** 31 - 1, 16), (2 ** 30 + 1, 16)):
        with pytest.raises(ValueError):
            ssm.scan_checkpoints(u.expand(1, tokens, 8), S)
    assert ssm.scan_checkpoints(u.expand(1, 33, 8), 64).shape == (1, 3, 8, 64)


def test_memory_that_is_not_there_raises_torchs_error():
    """As every other call that allocates through torch does."""
    ssm, _ = _ops()
    u = torch.zeros(1, 1, 8, dtype=BF, device="cuda").expand(60000, 2 ** 20, 8)      # 2 TB of checkpoints
    with pytest.raises(torch.OutOfMemoryError):
        ssm.scan_checkpoints(u, 64)


# ------------------------------------------------------------------ long chunks and runs
#
# Calls that fill the GPU with chunks of 128 and 256 tokens have 10^8 elements.  Channels do not meet in the scan's output
# and state, nor in the convolution: a few distinct ones, repeated over the width, are compared with the
# reference, and every repetition has to give the same bits.

def _fake_rows(width, N):
    return 1 << 20, N * width, width


def _chunk_tokens(B, N, D, S, dtype):
    """The chunk that the forward pass without checkpoints takes, by what its workspace holds: the states and one sum per
    channel of each chunk."""
    import ctypes

    from linear_latent_routing_gb300 import gma
    from test_block_abi import SCAN, _layout
    size = gma.lib.gma_scan_workspace_size
    size.argtypes, size.restype = [ctypes.c_void_p], ctypes.c_size_t
    rows, pair = _fake_rows(D, N), _fake_rows(S, N)
    got = size(_layout(SCAN).pack(B, N, D, S, 1, int(dtype == "bf16"), 0, 0, *rows, *rows, 0, 0, 0, *pair, *pair, 1 << 20, 0, 0, 0, 0, 0, *rows, 0))

    def up(n):
        return -(-n // 256) * 256
    fits = [c for c in (32, 64, 128, 256) if up(B * -(-N // c) * D * S * 4) + up(B * -(-N // c) * D * 4) == got]
    return fits[0] if len(fits) == 1 else None


LONG_SCANS = [  # distinct channels, repetitions, S, dtype, z, chunk; 3 x 3000 tokens
    (46, 256, 16, "bf16", True, 256),
    (51, 231, 8, "f32", False, 256),          # an odd width: rows off every boundary
    (16, 256, 16, "f32", True, 128),
    (17, 241, 8, "bf16", False, 128),         # odd
    (32, 128, 32, "bf16", True, 128),         # one channel a lane
]


@pytest.mark.parametrize("case", LONG_SCANS, ids=lambda c: "-".join(str(x) for x in c))
def test_scan_forward_in_the_longest_chunks(case, monkeypatch):
    """Lengths that end inside a chunk, on its edge and at the sequence's end."""
    monkeypatch.setattr(R, "DEVICE", "cuda")
    few, times, S, dtype, z, chunk = case
    ssm, _ = _ops()
    B, N, lengths, D = 3, 3000, [3000, 2817, 512], few * times
    assert _chunk_tokens(B, N, D, S, dtype) == chunk
    t, _, _ = _scan_inputs(B, N, few, S, 1, dtype, z, True, seed=31)
    t["b"], t["c"] = t["b"].squeeze(2), t["c"].squeeze(2)
    ry, rh = R.scan(**t, lengths=lengths)
    d = {k: v.cuda() if v is not None else None for k, v in t.items()}
    for k in ("u", "dt", "z"):
        d[k] = d[k].repeat(1, 1, times) if d[k] is not None else None
    d["a_log"], d["state"] = d["a_log"].repeat(times, 1), d["state"].repeat(1, times, 1)
    d["d_skip"], d["dt_bias"] = d["d_skip"].repeat(times), d["dt_bias"].repeat(times)
    h = torch.full((B, D, S), float("nan"), device="cuda")
    y = ssm.scan(**d, state_out=h, lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    y, h = y.unflatten(2, (times, few)), h.unflatten(1, (times, few))
    R.check(y[:, :, 0], ry, "y")
    R.check(h[:, 0], rh, "state")
    assert (y == y[:, :, :1]).all() and (h == h[:, :1]).all()


def _run_tokens(B, N, D, W, dtype):
    """The tokens of a thread's run in the convolution, by the rows of partial sums in its backward workspace: one for
    every eight runs."""
    import ctypes

    from linear_latent_routing_gb300 import gma
    from test_block_abi import CONV, _layout
    size = gma.lib.gma_conv_backward_workspace_size
    size.argtypes, size.restype = [ctypes.c_void_p], ctypes.c_size_t
    rows = _fake_rows(D, N)
    got = size(_layout(CONV + "RR2Q").pack(B, N, D, W, int(dtype == "bf16"), 0, *rows, 1 << 20, 1 << 20, 0, 0, 0, *rows, *rows, *rows, 1 << 20, 1 << 20))
    fits = [r for r in (8, 16, 32, 64, 128, 256) if -(-B * -(-(-(-N // r)) // 8) * (W + 1) * (-(-D // 4) * 4) * 4 // 256) * 256 == got]
    return fits[0] if len(fits) == 1 else None


LONG_CONVS = [  # distinct channels, repetitions, W, dtype, tokens, lengths, run
    (24, 342, 4, "bf16", 7500, [7500, 5000], 256),
    (139, 59, 3, "f32", 7500, None, 256),              # an odd width
    (24, 342, 2, "f32", 4000, [4000, 2561], 128),
    (139, 59, 4, "bf16", 4000, [3968, 129], 128),       # odd
]


@pytest.mark.parametrize("case", LONG_CONVS, ids=lambda c: "-".join(str(x) for x in c[:5]))
def test_conv_in_the_longest_runs(case, monkeypatch):
    monkeypatch.setattr(R, "DEVICE", "cuda")
    few, times, W, dtype, N, lengths, run = case
    ssm, _ = _ops()
    B, D, r, T = 2, few * times, _draw(32), TYPES[dtype]
    assert _run_tokens(B, N, D, W, dtype) == run
    t = {"x": r(B, N, few, dtype=T), "weight": r(few, W, std=0.6), "bias": r(few), "state": r(B, W - 1, few, dtype=T)}
    dy = r(B, N, few, dtype=T)
    ry, after, ref = R.conv(**t, lengths=lengths, dy=dy)
    d = {k: v.cuda().repeat(1, 1, times) for k, v in (("x", t["x"]), ("state", t["state"]), ("dy", dy))}
    w, b = t["weight"].cuda().repeat(times, 1), t["bias"].cuda().repeat(times)
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda") if lengths is not None else None
    so = torch.full((B, W - 1, D), float("nan"), dtype=T, device="cuda")
    y = ssm.conv(d["x"], w, b, state=d["state"], state_out=so, lengths=ln)
    g = ssm.conv_backward(d["dy"], d["x"], w, b, state=d["state"], lengths=ln)
    assert torch.equal(so[..., :few].double(), after) and torch.equal(so, so[..., :few].repeat(1, 1, times))
    for got, want, name in ((y, ry, "y"), (g["x"], ref["x"], "x")):
        R.check(got[..., :few], want, name)
        assert torch.equal(got, got[..., :few].repeat(1, 1, times)), name
    for name in ("weight", "bias"):
        R.check(g[name][:few], ref[name], name)
        assert torch.equal(g[name], g[name][:few].repeat(*((times, 1) if name == "weight" else (times,)))), name


def test_scan_backward_into_some_of_the_callers_rows():
    """With lengths and a part of `out`: the caller's rows behind a sequence's end are left alone, the other gradients are
    zero there, and every one has the bits that it has without `out`."""
    ssm, _ = _ops()
    for D, lengths in ((24, [0, 7, 130]), (8200, [129, 0, 64])):
        t, dy, ds = _scan_inputs(3, 140, D, 16, 1, "bf16", seed=33)
        d, _, _, ck, ln = _run_scan(t, lengths, ckpt=True)
        args = (dy.cuda(), d["u"], d["dt"], d["a_log"], d["b"], d["c"], ck, d["d_skip"], d["dt_bias"], d["z"])
        want = ssm.scan_backward(*args, dstate_out=ds.cuda(), lengths=ln)
        for names in (("u",), ("dt", "b"), ("z", "c")):
            wide = {k: torch.full((*t[k].shape[:2], t[k][0, 0].numel() + 8), 5.0, dtype=BF, device="cuda") for k in names}
            mine = {k: (wide[k][..., 8:].unflatten(2, t[k].shape[2:]) if k in "bc" else wide[k][..., 8:]) for k in names}
            torch.full((5, 3, 140, D), float("nan"), dtype=BF, device="cuda")          # what a new buffer may hold
            g = ssm.scan_backward(*args, dstate_out=ds.cuda(), lengths=ln, out=mine)
            for k in g:
                if k not in names:
                    assert torch.equal(g[k], want[k]), k
                    continue
                assert g[k] is mine[k] and (wide[k][..., :8] == 5.0).all(), k
                for i, n in enumerate(lengths):
                    assert torch.equal(g[k][i, :n], want[k][i, :n]) and (g[k][i, n:] == 5.0).all(), k


@pytest.mark.parametrize("d", [32, 10])
def test_norm_backward_into_strided_rows(d):
    """`out` as heads of token-major rows with a gap beside them: the bits of a contiguous one, the gap left alone."""
    _, norm = _ops()
    B, H, N = 2, 4, 6
    t, dr, dh = _norm_inputs((B, H, N, d, "bf16", 0, True, True, "f32", True, True), seed=34)
    c = {k: v.cuda() if v is not None else None for k, v in t.items()}
    r, _ = norm.block_norm(**c)
    args = dict(w_post=c["w_post"], gate=c["gate"], scale=c["scale"], w_pre=c["w_pre"], dh=dh.cuda())
    want = norm.block_norm_backward(dr.cuda(), c["o"], r, **args)
    wide = torch.full((B, N, H * d + 8), 5.0, dtype=BF, device="cuda")
    out = wide[..., 8:].unflatten(2, (H, d)).transpose(1, 2)
    g = norm.block_norm_backward(dr.cuda(), c["o"], r, **args, out=out)
    assert g["o"] is out and (wide[..., :8] == 5.0).all()
    for k in want:
        assert torch.equal(g[k], want[k]), k


def test_strides_beyond_32_bits_on_every_path():
    """Batch rows more than 2^31 elements apart give the bits of neighbouring ones: the scan in chunks, its backward
    pass, the convolution and the norms, inputs and outputs."""
    ssm, norm = _ops()
    N, D = 300, 4096
    gap = 2 ** 31 + 64
    store = [torch.empty(gap + N * D, dtype=BF, device="cuda") for _ in range(2)]

    def far(i, t=None):
        v = store[i].as_strided((2, N, D), (gap, D, 1))
        return v if t is None else v.copy_(t)
    t, dy, _ = _scan_inputs(2, N, D, 16, 1, "bf16", True, False, seed=41)
    d, y, _, ck, _ = _run_scan(t, ckpt=True)
    rest = (d["dt"], d["a_log"], d["b"], d["c"])
    more = (d["d_skip"], d["dt_bias"], d["z"])
    assert torch.equal(ssm.scan(far(0, d["u"]), *rest, *more, out=far(1)), y)
    g = ssm.scan_backward(dy.cuda(), d["u"], *rest, ck, *more)
    f = ssm.scan_backward(dy.cuda(), far(0), *rest, ck, *more, out={"u": far(1)})
    for k in g:
        assert (g[k] is None and f[k] is None) or torch.equal(g[k], f[k]), k
    r = _draw(42)
    w, b, wn = r(D, 4).cuda(), r(D).cuda(), (1 + r(D, std=0.3)).cuda()
    assert torch.equal(ssm.conv(far(0), w, b, out=far(1)), ssm.conv(d["u"], w, b))
    g, f = ssm.conv_backward(dy.cuda(), d["u"], w, b), ssm.conv_backward(dy.cuda(), far(0), w, b, out=far(1))
    for k in g:
        assert torch.equal(g[k], f[k]), k
    v, vf = norm.block_norm(d["u"], wn, gate=d["z"])[0], norm.block_norm(far(0), wn, gate=d["z"], out=far(1))[0]
    assert torch.equal(v, vf)
    args = dict(w_post=wn, gate=d["z"])
    g, f = norm.block_norm_backward(dy.cuda(), d["u"], v, **args), norm.block_norm_backward(dy.cuda(), far(0), v, **args, out=far(1))
    for k in g:
        assert (g[k] is None and f[k] is None) or torch.equal(g[k], f[k]), k
