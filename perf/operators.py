"""Cases and plain forms of the operators that stand next to the latent-routing mixer in a block.

Three operators, all in token-major rows [B, N, channels] as a block's projections give and take them:

* scan: the selective state space scan, a second mixer with a fixed state.  Per channel c and state n
      delta_t = softplus(dt_t + dt_bias),   A = -exp(a_log),
      h_t[n] = exp(delta_t A[n]) h_{t-1}[n] + delta_t b_t[n] u_t,
      y_t = (sum_n c_t[n] h_t[n] + d_skip u_t) * silu(z_t);
* conv: the short causal convolution per channel before it, pre_t = sum_k w[k] x_{t-W+1+k} + bias,
      y = silu(pre), with the last W - 1 inputs as the state of a sequence that goes on;
* norm: the norms around a block, with its gate and residual scale,
      v = w_post * rms(o * silu(gate)) (in groups of channels),  r' = r + scale * v,  h = w_pre * rms(r'),
      where the block's output o comes in the mixers' layout [B, H, N, d] and h is taken of r' as stored.

Forms: "prompt" (a forward pass, with the state for what follows), "train" (forward and backward) and
"step" (one token for every sequence of a batch, states updated in place).
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------ cases

def listed():
    def scan(name, form, B, N, D, S, G, dtype, z, carry, ragged):
        return dict(name=name, op="scan", form=form, B=B, N=N, D=D, S=S, G=G, dtype=dtype, z=z, carry=carry,
                    ragged=ragged)

    def conv(name, form, B, N, D, W, dtype, carry, ragged):
        return dict(name=name, op="conv", form=form, B=B, N=N, D=D, W=W, dtype=dtype, carry=carry, ragged=ragged)

    def norm(name, form, B, H, N, d, dtype, group, gate, res):
        return dict(name=name, op="norm", form=form, B=B, H=H, N=N, d=d, dtype=dtype, group=group, gate=gate,
                    res=res)

    return [
        # one long prompt at the long-context layer's width (16 heads of 128): few rows, a long axis
        scan("scan_prompt_long", "prompt", 1, 65536, 2048, 16, 1, "bf16", True, False, False),
        # a padded batch of prompts that go on from kept states, odd sizes, two groups of b and c
        scan("scan_prompt_ragged", "prompt", 7, 513, 520, 32, 2, "f32", False, True, True),
        # a training step at the language-model-shaped layer's batch and length, expanded width
        scan("scan_train_lm", "train", 4, 2048, 1024, 16, 1, "bf16", True, False, False),
        # training in fp32 on a piece of a longer sequence: state in, state and its gradient out
        scan("scan_train_f32", "train", 2, 301, 384, 8, 1, "f32", False, True, False),
        # decoding at the decode workload's batch and width
        scan("scan_step_batch", "step", 128, 1, 2048, 16, 1, "bf16", True, True, False),
        # decoding for one user: latency
        scan("scan_step_one", "step", 1, 1, 1024, 16, 1, "bf16", True, True, False),
        # the convolution of two prompts at the width sweep's length
        conv("conv_prompt", "prompt", 2, 16384, 2080, 4, "bf16", False, False),
        # its training step over a padded classification-shaped batch
        conv("conv_train", "train", 32, 1024, 512, 4, "bf16", False, True),
        # its decoding step
        conv("conv_step_batch", "step", 128, 1, 2080, 4, "bf16", True, False),
        # both norms, gate and residual scale of a block in training, with an fp32 residual stream
        norm("norm_train", "train", 4, 16, 2048, 128, "bf16", 0, True, "f32"),
        # the gated per-head norm of a long prompt before the output projection
        norm("norm_prompt_heads", "prompt", 1, 16, 65536, 128, "bf16", 128, True, "none"),
        # one token for each of a few users, fp32
        norm("norm_token", "prompt", 4, 8, 1, 64, "f32", 0, True, "f32"),
    ]


def _log_int(rng, lo, hi, multiple=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = max(lo, min(hi, v))
    return max(multiple, v // multiple * multiple)


def draw(rng):
    op = rng.choice(["scan", "scan", "conv", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    form = rng.choice(["prompt", "train", "step"]) if op != "norm" else rng.choice(["prompt", "train"])
    wide = rng.choice([1, 8, 8, 16])          # widths that are odd, and ones that are not
    if op == "norm":
        H, d = rng.choice([1, 2, 8, 16]), rng.choice([16, 32, 64, 128])
        if rng.random() < 0.25:
            H, d = 1, _log_int(rng, 33, 4096)
        B, N = _log_int(rng, 1, 32), _log_int(rng, 1, 4096)
        # a stored bf16 residual stream in training is left out: whether a value next to a border rounds up or
        # down would decide the fp32 parameter gradients that are taken of it
        res = rng.choice(["none", "f32", dtype] if form == "prompt" else ["none", "f32"])
        group = d if H > 1 and rng.random() < 0.4 else 0
        return dict(op=op, form=form, B=B, H=H, N=N, d=d, dtype=dtype, group=group, gate=rng.random() < 0.7,
                    res=res)
    D = _log_int(rng, 64, 4096, wide)
    if form == "step":
        B, N = _log_int(rng, 1, 256), 1
    else:
        B = _log_int(rng, 1, 16)
        N = _log_int(rng, 1, min(32768, (1 << (25 if op == "conv" else 23)) // (B * D)))
    if op == "conv":
        return dict(op=op, form=form, B=B, N=N, D=D, W=rng.choice([2, 3, 4]), dtype=dtype,
                    carry=form == "step" or rng.random() < 0.3, ragged=form != "step" and rng.random() < 0.3)
    S = rng.choice([8, 16, 16, 32, 64]) if form != "train" else rng.choice([8, 16, 16, 32])
    G = 2 if D % 2 == 0 and rng.random() < 0.3 else 1
    return dict(op=op, form=form, B=B, N=N, D=D, S=S, G=G, dtype=dtype, z=rng.random() < 0.6,
                carry=form == "step" or rng.random() < 0.3, ragged=form != "step" and rng.random() < 0.3)


def work(case):
    """Inputs read once and outputs written once; flops of the recurrence itself."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm":
        rows, D = case["B"] * case["N"], case["H"] * case["d"]
        er = {"none": 0, "f32": 4, "bf16": 2}[case["res"]]
        gate = e if case["gate"] else 0
        per = e + gate + (2 * er + e if er else e)
        flops = 14
        if case["form"] == "train":   # dr, dh in; do, dgate, dresidual out
            per += (2 * er + e if er else e) + e + gate
            flops += 30
        return {"bytes": rows * D * per, "flops": rows * D * flops}
    B, N, D = case["B"], case["N"], case["D"]
    elems = B * N * D
    if case["op"] == "conv":
        W = case["W"]
        state = B * (W - 1) * D * e * (2 if case["carry"] else 1) if case["form"] != "train" else 0
        if case["form"] == "train":
            return {"bytes": elems * e * 4, "flops": elems * (2 * W + 8) * 3}
        return {"bytes": elems * e * 2 + state, "flops": elems * (2 * W + 8)}
    S, G = case["S"], case["G"]
    z = e if case["z"] else 0
    fwd = elems * (3 * e + z) + B * N * 2 * G * S * e + B * D * S * 4 * (2 if case["carry"] else 1)
    flops = elems * S * 7
    if case["form"] == "train":       # dy in; du, ddt, dz, db, dc out
        fwd += elems * (3 * e + z) + B * N * 2 * G * S * e
        flops += elems * S * 20
    return {"bytes": fwd, "flops": flops}


# ------------------------------------------------------------------------------------ inputs

def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    T = TYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32) * (hi - lo) + lo

    s = {}
    if case["op"] == "norm":
        B, H, N, d = case["B"], case["H"], case["N"], case["d"]
        D = H * d
        R = {"none": None, "f32": torch.float32, "bf16": torch.bfloat16}[case["res"]]
        s["o"] = normal(B, H, N, d).to(T)
        # the gate is a part of a wider projection's rows
        s["gate"] = normal(B, N, 2 * D).to(T)[:, :, D:] if case["gate"] else None
        s["w_post"] = 1 + normal(D, std=0.1)
        s["residual"] = normal(B, N, D, std=2.0).to(R) if R is not None else None
        s["scale"] = uniform(D, lo=0.05, hi=0.5) if R is not None else None
        s["w_pre"] = 1 + normal(D, std=0.1) if R is not None else None
        s["dr"] = normal(B, N, D).to(R if R is not None else T)
        s["dh"] = normal(B, N, D).to(T) if R is not None else None
        return s
    B, N, D = case["B"], case["N"], case["D"]
    if case["ragged"]:
        n = (uniform(B) * (N + 1)).long().clamp(0, N)
        n[0] = N
        s["lengths"] = n.to(torch.int32)
    else:
        s["lengths"] = None
    if case["op"] == "conv":
        W = case["W"]
        s["weight"] = uniform(D, W, lo=-1.0, hi=1.0) / math.sqrt(W)
        s["bias"] = normal(D, std=0.1)
        s["x"] = normal(B, N, D).to(T) if case["form"] != "step" else normal(B, D).to(T)
        s["state"] = normal(B, W - 1, D).to(T) if case["carry"] else None
        s["dy"] = normal(B, N, D).to(T)
        return s
    S, G = case["S"], case["G"]
    # u, b and c are parts of one convolution's rows
    xbc = normal(B, N, D + 2 * G * S).to(T)
    s["u"] = xbc[:, :, :D]
    s["b"] = xbc[:, :, D:D + G * S].unflatten(2, (G, S))
    s["c"] = xbc[:, :, D + G * S:].unflatten(2, (G, S))
    s["dt"] = normal(B, N, D, std=0.5).to(T)
    # step sizes between 0.001 and 0.1 at dt = 0, decay rates 1 to S
    d0 = torch.exp(uniform(D, lo=math.log(1e-3), hi=math.log(1e-1)))
    s["dt_bias"] = d0 + torch.log(-torch.expm1(-d0))
    s["a_log"] = torch.log(torch.arange(1, S + 1, device="cuda", dtype=torch.float32)) + normal(D, S, std=0.1)
    s["d_skip"] = 1 + normal(D, std=0.2)
    s["z"] = normal(B, N, 2 * D).to(T)[:, :, :D] if case["z"] else None
    s["state"] = normal(B, D, S) if case["carry"] else None
    s["dy"] = normal(B, N, D).to(T)
    s["dstate"] = normal(B, D, S) if case["carry"] else None
    if case["form"] == "step":
        for k in ("u", "b", "c", "dt", "z"):
            s[k] = s[k][:, 0] if s[k] is not None else None
    return s


def prepare(case, seed):
    return dict(_inputs(case, seed), case=dict(case))


# ------------------------------------------------------------------------------------ plain forms

def _softplus(x):
    return torch.where(x > 20, x, torch.log1p(torch.exp(x)))


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _mask(lengths, N):
    """1 for a sequence's tokens, 0 for the rows behind them, [B, N, 1]; or 1."""
    if lengths is None:
        return 1.0
    return (torch.arange(N, device=lengths.device) < lengths[:, None]).float()[:, :, None]


def _recurrence(a, b):
    """x_t = a_t x_{t-1} + b_t along dimension 1, by doubling."""
    k = 1
    while k < b.shape[1]:
        b = torch.cat([b[:, :k], a[:, k:] * b[:, :-k] + b[:, k:]], 1)
        a = torch.cat([a[:, :k], a[:, k:] * a[:, :-k]], 1)
        k *= 2
    return b


def _plain_scan(s, case):
    B, N, D, S, G = case["B"], case["N"], case["D"], case["S"], case["G"]
    T, step = TYPES[case["dtype"]], case["form"] == "step"
    u, dt, b, c, z = (s[k].float() if s[k] is not None else None for k in ("u", "dt", "b", "c", "z"))
    if step:
        u, dt, b, c, z = (t.unsqueeze(1) if t is not None else None for t in (u, dt, b, c, z))
    live = _mask(s["lengths"], N)
    A = -torch.exp(s["a_log"])
    raw = dt + s["dt_bias"]
    delta = _softplus(raw) * live
    u = u * live
    bd, cd = (t[:, :, :, None].expand(B, N, G, D // G, S).reshape(B, N, D, S) if G > 1 else t for t in (b, c))
    a = torch.exp(delta[..., None] * A)
    x = (delta * u)[..., None] * bd
    if s["state"] is not None:
        x[:, 0] += a[:, 0] * s["state"]
    h = _recurrence(a, x)
    del x
    state = h[:, -1].clone()
    pre = (h * cd).sum(-1) + s["d_skip"] * u
    y = pre * z * _sigmoid(z) if z is not None else pre
    y = (y * live).to(T)
    if step:
        s["state"].copy_(state)
        return y[:, 0], s["state"]
    if case["form"] == "prompt":
        return y, state
    dy = s["dy"].float() * live
    dyy, dz = dy, None
    if z is not None:
        sig = _sigmoid(z)
        dyy = dy * z * sig
        dz = (dy * pre * sig * (1 + z * (1 - sig))).to(T)
    first = s["state"] if s["state"] is not None else torch.zeros(B, D, S, device=h.device)
    g = dyy[..., None] * cd
    if s["dstate"] is not None:
        g[:, -1] += s["dstate"]
    a_next = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    g = _recurrence(a_next.flip(1), g.flip(1)).flip(1)
    del a_next
    dx = (g * bd).sum(-1)
    db = (g * (delta * u)[..., None]).reshape(B, N, G, D // G, S).sum(3)
    dc = (h * dyy[..., None]).reshape(B, N, G, D // G, S).sum(3)
    q = g * a * torch.cat([first[:, None], h[:, :-1]], 1)
    ddt = (dx * u + (q * A).sum(-1)) * _sigmoid(raw) * live
    da = (q * delta[..., None]).sum((0, 1)) * A
    du = (dx * delta + s["d_skip"] * dyy) * live
    out = [y, state, du.to(T), ddt.to(T), da, db.to(T), dc.to(T), (dyy * u).sum((0, 1)), ddt.sum((0, 1)), dz]
    if s["dstate"] is not None:
        out.append(g[:, 0] * a[:, 0])
    return out


def _plain_conv(s, case):
    B, N, D, W = case["B"], case["N"], case["D"], case["W"]
    T, step = TYPES[case["dtype"]], case["form"] == "step"
    x = (s["x"][:, None] if step else s["x"]).float()
    first = s["state"].float() if s["state"] is not None else torch.zeros(B, W - 1, D, device=x.device)
    live = _mask(s["lengths"], N)
    rows = torch.cat([first, x * live], 1)
    near = rows.unfold(1, W, 1)                                   # [B, N, D, W]
    pre = (near * s["weight"]).sum(-1) + s["bias"]
    sig = _sigmoid(pre)
    y = (pre * sig * live).to(T)
    if s["lengths"] is None:
        state = rows[:, N:].to(T)
    else:
        at = s["lengths"].long()[:, None] + torch.arange(W - 1, device=x.device)
        state = torch.gather(rows, 1, at[:, :, None].expand(B, W - 1, D)).to(T)
    if step:
        s["state"].copy_(state)
        return y[:, 0], s["state"]
    if case["form"] == "prompt":
        return y, state
    dpre = s["dy"].float() * live * sig * (1 + pre * (1 - sig))
    ahead = torch.cat([dpre, torch.zeros(B, W - 1, D, device=x.device)], 1).unfold(1, W, 1)
    dx = (ahead * s["weight"].flip(1)).sum(-1) * live
    dw = (near * dpre[..., None]).sum((0, 1))
    return y, dx.to(T), dw, dpre.sum((0, 1))


EPS = 1e-6


def _groups(x, group):
    return x.unflatten(-1, (-1, group)) if group else x.unsqueeze(-2)


def _plain_norm(s, case):
    B, H, N, d = case["B"], case["H"], case["N"], case["d"]
    T, D, group = TYPES[case["dtype"]], H * d, case["group"]
    o = s["o"].float().transpose(1, 2).reshape(B, N, D)
    gate = s["gate"].float() if s["gate"] is not None else None
    sig = _sigmoid(gate) if gate is not None else None
    u = o * gate * sig if gate is not None else o
    ug = _groups(u, group)
    rstd = torch.rsqrt((ug * ug).mean(-1, keepdim=True) + EPS)
    n = (ug * rstd).flatten(-2)
    v = n * s["w_post"]
    if s["residual"] is None:
        r, h = v.to(T), None
    else:
        r = (s["residual"].float() + s["scale"] * v).to(s["residual"].dtype)
        rf = r.float()                    # the second norm is that of the residual stream as stored
        rstd2 = torch.rsqrt((rf * rf).mean(-1, keepdim=True) + EPS)
        h = (rf * rstd2 * s["w_pre"]).to(T)
    if case["form"] == "prompt":
        return r, h
    dr = s["dr"].float()
    dscale = dw_pre = dres = None
    dv = dr
    if s["residual"] is not None:
        dh = s["dh"].float()
        m = dh * s["w_pre"]
        dr = dr + rstd2 * (m - rf * rstd2 * rstd2 * (m * rf).mean(-1, keepdim=True))
        dw_pre = (dh * rf * rstd2).sum((0, 1))
        dscale = (dr * v).sum((0, 1))
        dres = dr.to(s["residual"].dtype)
        dv = dr * s["scale"]
    dw_post = (dv * n).sum((0, 1))
    m = _groups(dv * s["w_post"], group)
    du = (rstd * (m - ug * rstd * rstd * (m * ug).mean(-1, keepdim=True))).flatten(-2)
    dgate = None
    do = du
    if gate is not None:
        do = du * gate * sig
        dgate = (du * o * sig * (1 + gate * (1 - sig))).to(T)
    do = do.reshape(B, N, H, d).transpose(1, 2).to(T)
    return r, h, do, dgate, dres, dw_post, dscale, dw_pre


# ------------------------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    op, form = case["op"], case["form"]
    if not own:
        return {"scan": _plain_scan, "conv": _plain_conv, "norm": _plain_norm}[op](s, case)
    if op == "norm":
        from linear_latent_routing_gb300 import norm
        r, h = norm.block_norm(s["o"], s["w_post"], gate=s["gate"], residual=s["residual"], scale=s["scale"],
                               w_pre=s["w_pre"], eps=EPS, group=case["group"])
        if form == "prompt":
            return r, h
        g = norm.block_norm_backward(s["dr"], s["o"], r, s["w_post"], gate=s["gate"], scale=s["scale"],
                                     w_pre=s["w_pre"], dh=s["dh"], eps=EPS, group=case["group"])
        return (r, h, g["o"], g["gate"], g["residual"], g["w_post"], g["scale"], g["w_pre"])
    from linear_latent_routing_gb300 import ssm
    if op == "conv":
        if form == "step":
            return ssm.conv_step(s["x"], s["weight"], s["bias"], s["state"]), s["state"]
        if form == "prompt":
            state = torch.empty(case["B"], case["W"] - 1, case["D"], dtype=s["x"].dtype, device="cuda")
            return ssm.conv(s["x"], s["weight"], s["bias"], state=s["state"], state_out=state,
                            lengths=s["lengths"]), state
        y = ssm.conv(s["x"], s["weight"], s["bias"], state=s["state"], lengths=s["lengths"])
        g = ssm.conv_backward(s["dy"], s["x"], s["weight"], s["bias"], state=s["state"], lengths=s["lengths"])
        return y, g["x"], g["weight"], g["bias"]
    args = (s["u"], s["dt"], s["a_log"], s["b"], s["c"])
    extra = dict(d_skip=s["d_skip"], dt_bias=s["dt_bias"], z=s["z"])
    if form == "step":
        return ssm.scan_step(*args, s["state"], **extra), s["state"]
    state = torch.empty(case["B"], case["D"], case["S"], device="cuda")
    if form == "prompt":
        return ssm.scan(*args, state=s["state"], state_out=state, lengths=s["lengths"], **extra), state
    kept = ssm.scan_checkpoints(s["u"], case["S"])
    y = ssm.scan(*args, state=s["state"], state_out=state, lengths=s["lengths"], checkpoints=kept, **extra)
    g = ssm.scan_backward(s["dy"], *args, kept, dstate_out=s["dstate"], lengths=s["lengths"], **extra)
    out = [y, state, g["u"], g["dt"], g["a_log"], g["b"], g["c"], g["d_skip"], g["dt_bias"], g["z"]]
    return out + [g["state"]] if s["dstate"] is not None else out


# ------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
         for k, v in _inputs(case, seed).items()}
    return {"scan": _exact_scan, "conv": _exact_conv, "norm": _exact_norm}[case["op"]](case, s)


def _exact_scan(case, s):
    """Token by token: the recurrence as it is defined, and its adjoint from the last token back."""
    B, N, D, S, G = (case[k] for k in "BNDSG")
    step = case["form"] == "step"
    rows = {k: (s[k][:, None] if step else s[k]) if s[k] is not None else None for k in ("u", "dt", "b", "c", "z")}
    A = -s["a_log"].exp()
    raw = rows["dt"] + s["dt_bias"]
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    count = s["lengths"].tolist() if s["lengths"] is not None else [N] * B
    alive = torch.tensor([[t < n for t in range(N)] for n in count], device="cuda")
    of_group = torch.arange(D, device="cuda") // (D // G)
    h = s["state"].clone() if s["state"] is not None else torch.zeros(B, D, S, device="cuda", dtype=torch.float64)
    first, train = h, case["form"] == "train"
    pre = torch.zeros(B, N, D, device="cuda", dtype=torch.float64)
    kept = []
    for t in range(N):
        new = (delta[:, t, :, None] * A).exp() * h
        new = new + (delta[:, t] * rows["u"][:, t])[..., None] * rows["b"][:, t, of_group]
        h = torch.where(alive[:, t, None, None], new, h) if s["lengths"] is not None else new
        if train:
            kept.append(h)
        pre[:, t] = (h * rows["c"][:, t, of_group]).sum(-1)
    pre = pre + s["d_skip"] * rows["u"]
    z = rows["z"]
    sig = torch.special.expit(z) if z is not None else None
    y = pre * z * sig if z is not None else pre
    y = torch.where(alive[..., None], y, torch.zeros_like(y))
    if step:
        return y[:, 0], h
    if not train:
        return y, h
    zero = torch.zeros(B, N, D, device="cuda", dtype=torch.float64)
    dy = torch.where(alive[..., None], s["dy"], zero)
    dpre = dy * z * sig if z is not None else dy
    dz = dy * pre * (sig + z * sig * (1 - sig)) if z is not None else None
    g = s["dstate"].clone() if s["dstate"] is not None else torch.zeros_like(first)
    du, ddt = torch.zeros_like(zero), torch.zeros_like(zero)
    db = torch.zeros(B, N, G, S, device="cuda", dtype=torch.float64)
    dc, da = torch.zeros_like(db), torch.zeros(D, S, device="cuda", dtype=torch.float64)
    dsoft = torch.special.expit(raw)
    for t in reversed(range(N)):
        on = alive[:, t, None]
        bt, ct = rows["b"][:, t, of_group], rows["c"][:, t, of_group]
        before = kept[t - 1] if t else first
        g = g + torch.where(on, dpre[:, t], zero[:, t])[..., None] * ct
        gl = torch.where(on[..., None], g, torch.zeros_like(g))
        dc[:, t] = (kept[t] * dpre[:, t, :, None]).view(B, G, D // G, S).sum(2)
        db[:, t] = (gl * (delta[:, t] * rows["u"][:, t])[..., None]).view(B, G, D // G, S).sum(2)
        decay = (delta[:, t, :, None] * A).exp()
        through = (gl * bt).sum(-1)
        rate = gl * decay * before
        du[:, t] = through * delta[:, t] + s["d_skip"] * dpre[:, t]
        ddt[:, t] = (through * rows["u"][:, t] + (rate * A).sum(-1)) * dsoft[:, t]
        da += (rate * delta[:, t, :, None]).sum(0)
        g = torch.where(on[..., None], g * decay, g)
    out = [y, h, du, ddt, da * A, db, dc, (dpre * rows["u"]).sum((0, 1)), ddt.sum((0, 1)), dz]
    return out + [g] if s["dstate"] is not None else out


def _exact_conv(case, s):
    """Tap by tap."""
    B, N, D, W = (case[k] for k in "BNDW")
    x = s["x"][:, None] if case["form"] == "step" else s["x"]
    state = s["state"] if s["state"] is not None else torch.zeros(B, W - 1, D, device="cuda", dtype=torch.float64)
    count = s["lengths"].tolist() if s["lengths"] is not None else [N] * B
    alive = torch.tensor([[t < n for t in range(N)] for n in count], device="cuda")[..., None]
    rows = torch.cat([state, x], 1)
    pre = s["bias"].expand(B, N, D).clone()
    for k in range(W):
        pre += rows[:, k:k + N] * s["weight"][:, k]
    sig = torch.special.expit(pre)
    y = torch.where(alive, pre * sig, torch.zeros_like(pre))
    after = torch.stack([rows[i, n:n + W - 1] for i, n in enumerate(count)])
    if case["form"] == "step":
        return y[:, 0], after
    if case["form"] == "prompt":
        return y, after
    dpre = torch.where(alive, s["dy"] * (sig + pre * sig * (1 - sig)), torch.zeros_like(pre))
    drows = torch.zeros_like(rows)
    dw = torch.zeros(D, W, device="cuda", dtype=torch.float64)
    for k in range(W):
        drows[:, k:k + N] += dpre * s["weight"][:, k]
        dw[:, k] = (dpre * rows[:, k:k + N]).sum((0, 1))
    dx = torch.where(alive, drows[:, W - 1:], torch.zeros_like(pre))
    return y, dx, dw, dpre.sum((0, 1))


def _exact_norm(case, s):
    """From the definition; the gradients by reverse differentiation of it in 64 bits."""
    B, H, N, d = (case[k] for k in "BHNd")
    D, group = H * d, case["group"] or H * d
    res = s["residual"]
    stored = {"none": TYPES[case["dtype"]], "f32": torch.float32, "bf16": torch.bfloat16}[case["res"]]
    want = case["form"] == "train"
    leaf = {k: s[k].detach().requires_grad_(want) if s[k] is not None else None
            for k in ("o", "gate", "residual", "w_post", "scale", "w_pre")}
    u = leaf["o"].permute(0, 2, 1, 3).reshape(B, N, D)
    if leaf["gate"] is not None:
        u = u * torch.nn.functional.silu(leaf["gate"])
    parts = u.view(B, N, D // group, group)
    v = (parts / (parts.pow(2).sum(-1, keepdim=True) / group + EPS).sqrt()).view(B, N, D) * leaf["w_post"]
    r = v if res is None else leaf["residual"] + leaf["scale"] * v
    if res is None:
        if not want:
            return r, None
        r.backward(s["dr"])
        return (r.detach(), None, leaf["o"].grad, leaf["gate"].grad if leaf["gate"] is not None else None, None,
                leaf["w_post"].grad, None, None)
    # the norm of the stored residual stream, whose rounding passes its gradient on
    kept = r + (r.detach().to(stored).double() - r.detach())
    h = kept / (kept.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * leaf["w_pre"]
    if not want:
        return r, h
    (r * s["dr"]).sum().add((h * s["dh"]).sum()).backward()
    return (r.detach(), h.detach(), leaf["o"].grad, leaf["gate"].grad if leaf["gate"] is not None else None,
            leaf["residual"].grad, leaf["w_post"].grad, leaf["scale"].grad, leaf["w_pre"].grad)
