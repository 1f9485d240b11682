"""The block operators in 64 bits on the CPU, with a running bound of the error that fp32 arithmetic
may make, for the tests of include/gma_block.h.

Every quantity is a pair (v, e): the value in 64 bits and a first-order bound of the error of the
same computation in fp32, U = 2^-24 an operation.  A product carries |x| e_y + |y| e_x + U |xy|, a
sum of n terms the terms' errors and (n - 1) U sum |x|, whatever its order; functions carry their
argument's error through their slope and their own error:
  ex2.approx      2^-22 = 4 U relative;
  expf            2 ulp = 4 U relative, with its argument's rounding |x| U for the fast form;
  log1pf, expm1f, rsqrtf, fast division: 2 ulp = 4 U relative each.
SLACK = 2 covers second-order terms and products taken in another order (decays multiplied together
before they meet the state, as a scan over time lanes does).
A rounding to bf16 adds half a step, 2^-8 relative, to fp32 2^-24.
"""
import torch

DEVICE = "cpu"       # where the references compute; long cases use the GPU's fp64 units
U = 2.0 ** -24
SLACK = 2.0
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


class X:
    def __init__(self, v, e=None):
        self.v = v
        self.e = torch.zeros_like(v) if e is None else e

    def __add__(self, o):
        v = self.v + o.v
        return X(v, self.e + o.e + U * v.abs())

    def __sub__(self, o):
        return self + (-o)

    def __neg__(self):
        return X(-self.v, self.e)

    def __mul__(self, o):
        if not isinstance(o, X):
            return X(self.v * o, self.e * abs(o))
        v = self.v * o.v
        return X(v, self.v.abs() * o.e + o.v.abs() * self.e + U * v.abs())

    def sum(self, dim, keepdim=False):
        dims = (dim,) if isinstance(dim, int) else tuple(dim)
        n = 1
        for d in dims:
            n *= self.v.shape[d]
        return X(self.v.sum(dims, keepdim), (self.e + (n - 1) * U * self.v.abs()).sum(dims, keepdim))

    def f(self, value, slope, rel):
        return X(value, slope.abs() * self.e + rel * U * value.abs())

    def map(self, fn):
        return X(fn(self.v), fn(self.e))

    def __getitem__(self, i):
        return X(self.v[i], self.e[i])


def lift(t):
    return None if t is None else X(t.detach().to(DEVICE).double())


def stack(xs, dim):
    return X(torch.stack([x.v for x in xs], dim), torch.stack([x.e for x in xs], dim))


def where(c, x, y):
    return X(torch.where(c, x.v, y.v), torch.where(c, x.e, y.e))


def zeros(*shape):
    return X(torch.zeros(*shape, dtype=torch.float64, device=DEVICE))


def live_of(count, N):
    """[B, N]: which tokens are a sequence's."""
    return torch.arange(N, device=DEVICE) < torch.tensor(count, device=DEVICE)[:, None]


def sigmoid(x):
    s = torch.special.expit(x.v)
    return X(s, s * (1 - s) * x.e + (x.v.abs() + 12) * U * s)


def silu(x):
    return x * sigmoid(x)


def dsilu(x):
    s = sigmoid(x)
    one = X(torch.ones_like(x.v))
    return s * (one + x * (one - s))


def softplus(x):
    v = torch.logaddexp(x.v, torch.zeros_like(x.v))
    return X(v, torch.special.expit(x.v) * x.e + (x.v.abs() + 10) * U * v)


def rate_of(a_log):
    """A = -exp(a_log), with the two constants that turn it to base 2 and back."""
    v = -a_log.v.exp()
    return X(v, 8 * U * v.abs())


def decay_of(delta, A):
    x = delta * A
    return x.f(x.v.exp(), x.v.exp(), 4)


def lengths_list(lengths, B, N):
    return [N] * B if lengths is None else [min(max(int(n), 0), N) for n in lengths]


# ------------------------------------------------------------------ selective scan

def scan(u, dt, a_log, b, c, d_skip=None, dt_bias=None, z=None, state=None, lengths=None, dy=None,
         dstate_out=None):
    """(y, state_out) of X, and the dict of gradients if dy is given; rows behind the last tokens
    are zero."""
    u, dt, a_log, b, c, d_skip, dt_bias, z, state, dy, dstate_out = map(
        lift, (u, dt, a_log, b, c, d_skip, dt_bias, z, state, dy, dstate_out))
    B, N, D = u.v.shape
    S = a_log.v.shape[1]
    if b.v.dim() == 3:
        b, c = b.map(lambda t: t.unsqueeze(2)), c.map(lambda t: t.unsqueeze(2))
    G = b.v.shape[2]
    of = torch.arange(D, device=DEVICE) // (D // G)
    count = lengths_list(lengths, B, N)
    live = live_of(count, N)
    A = rate_of(a_log)
    raw = dt + dt_bias if dt_bias is not None else dt
    delta = softplus(raw)
    xu = delta * u
    h = state if state is not None else zeros(B, D, S)
    first, hs, decays, pres = h, [], [], []
    for t in range(N):
        on = live[:, t, None, None]
        a = decay_of(delta[:, t].map(lambda v: v.unsqueeze(-1)), A)
        new = a * h + xu[:, t].map(lambda v: v.unsqueeze(-1)) * b[:, t].map(lambda v: v[:, of])
        h = where(on, new, h)
        p = (c[:, t].map(lambda v: v[:, of]) * h).sum(2)
        if d_skip is not None:
            p = p + d_skip * u[:, t]
        hs.append(h)
        decays.append(a)
        pres.append(p)
    pre = stack(pres, 1)
    y = pre * silu(z) if z is not None else pre
    y = where(live[..., None], y, zeros(B, N, D))
    if dy is None:
        return y, h
    nothing = zeros(B, N, D)
    dp = where(live[..., None], dy * silu(z) if z is not None else dy, nothing)
    r = dstate_out if dstate_out is not None else zeros(B, D, S)
    da, dus, ddts, dbs, dcs = zeros(D, S), [None] * N, [None] * N, [None] * N, [None] * N
    for t in reversed(range(N)):
        on = live[:, t, None, None]
        wide = (lambda v: v.unsqueeze(-1))
        bt, ct = b[:, t].map(lambda v: v[:, of]), c[:, t].map(lambda v: v[:, of])
        g = where(on, r + ct * dp[:, t].map(wide), zeros(B, D, S))

        def groups(x):
            return x.map(lambda v: v.view(B, G, D // G, S)).sum(2)
        dcs[t] = groups(hs[t] * dp[:, t].map(wide))
        dbs[t] = groups(g * xu[:, t].map(wide))
        x = (bt * g).sum(2)
        back = decays[t] * g
        q = back * (hs[t - 1] if t else first)
        du = x * delta[:, t]
        dus[t] = du + d_skip * dp[:, t] if d_skip is not None else du
        ddts[t] = (x * u[:, t] + (q * A).sum(2)) * sigmoid(raw[:, t])
        da = da + (q * delta[:, t].map(wide)).sum(0)
        r = where(on, back, r)
    ddt = where(live[..., None], stack(ddts, 1), nothing)
    grads = {"u": where(live[..., None], stack(dus, 1), nothing), "dt": ddt, "b": stack(dbs, 1),
             "c": stack(dcs, 1), "a_log": da * A, "state": r,
             "d_skip": (dp * u).sum((0, 1)) if d_skip is not None else None,
             "dt_bias": ddt.sum((0, 1)) if dt_bias is not None else None,
             "z": where(live[..., None], dy * pre * dsilu(z), nothing) if z is not None else None}
    return y, h, grads


# ------------------------------------------------------------------ convolution

def conv(x, weight, bias=None, state=None, lengths=None, silu_=True, dy=None):
    """(y, state_out tensor, gradients or None)."""
    x, weight, bias, state, dy = map(lift, (x, weight, bias, state, dy))
    B, N, D = x.v.shape
    W = weight.v.shape[1]
    past = state.v if state is not None else torch.zeros(B, W - 1, D, dtype=torch.float64, device=DEVICE)
    rows = torch.cat([past, x.v], 1)
    count = lengths_list(lengths, B, N)
    live = live_of(count, N)[..., None]
    near = X(rows.unfold(1, W, 1))
    pre = (near * weight).sum(3)
    if bias is not None:
        pre = pre + bias
    nothing = zeros(B, N, D)
    y = where(live, silu(pre) if silu_ else pre, nothing)
    after = torch.stack([rows[i, n:n + W - 1] for i, n in enumerate(count)])
    if dy is None:
        return y, after, None
    dp = where(live, dy * dsilu(pre) if silu_ else dy, nothing)
    pad = dp.map(lambda v: torch.cat([v, torch.zeros(B, W - 1, D, dtype=torch.float64, device=DEVICE)], 1).unfold(1, W, 1))
    dx = where(live, (pad * weight.map(lambda v: v.flip(1))).sum(3), nothing)
    return y, after, {"x": dx, "weight": (dp.map(lambda v: v.unsqueeze(-1)) * near).sum((0, 1)),
                      "bias": dp.sum((0, 1)) if bias is not None else None}


# ------------------------------------------------------------------ norms

def _rms(x, group, eps):
    """1 / sqrt(mean(x^2) + eps) per group, spread over the group's channels."""
    n = x.v.shape[-1]
    g = x.map(lambda v: v.unflatten(-1, (n // group, group)))
    m = (g * g).sum(g.v.dim() - 1, True) * (1.0 / group)
    s = m.v + eps
    r = X(s.rsqrt(), 0.5 * s ** -1.5 * (m.e + 2 * U * s) + 4 * U * s.rsqrt())
    return r.map(lambda v: v.expand(*v.shape[:-1], group).flatten(-2))


def _group_mean(x, group):
    n = x.v.shape[-1]
    g = x.map(lambda v: v.unflatten(-1, (n // group, group)))
    m = g.sum(g.v.dim() - 1, True) * (1.0 / group)
    return m.map(lambda v: v.expand(*v.shape[:-1], group).flatten(-2))


def norm(o, w_post=None, gate=None, residual=None, scale=None, w_pre=None, eps=1e-6, group=0, r_stored=None, dr=None,
         dh=None):
    """(r, h, gradients or None); h and the gradients are taken of `r_stored`, the r' that is kept."""
    o4 = o.dim() == 4
    o, w_post, gate, residual, scale, w_pre, kept, dr, dh = map(
        lift, (o, w_post, gate, residual, scale, w_pre, r_stored, dr, dh))
    if o4:
        B, H, N, d = o.v.shape
        o = o.map(lambda v: v.transpose(1, 2).reshape(B, N, H * d))
    D = o.v.shape[-1]
    group = group or D
    a = o * silu(gate) if gate is not None else o
    rstd = _rms(a, group, eps) if w_post is not None else None
    n = a * rstd if w_post is not None else a
    v = n * w_post if w_post is not None else n
    sv = v * scale if scale is not None else v
    r = residual + sv if residual is not None else sv
    h = None
    if w_pre is not None and kept is not None:
        rs2 = _rms(kept, D, eps)
        h = kept * rs2 * w_pre
    if dr is None and dh is None:
        return r, h, None
    t = dr if dr is not None else zeros(*a.v.shape)
    grads = {"w_pre": None, "scale": None, "w_post": None, "gate": None, "residual": None}
    if dh is not None:
        m = dh * w_pre
        t = t + rs2 * (m - kept * (rs2 * rs2 * _group_mean(m * kept, D)))
        grads["w_pre"] = (dh * kept * rs2).sum((0, 1))
    elif w_pre is not None:
        grads["w_pre"] = zeros(D)
    grads["residual"] = t if residual is not None else None
    dv = t * scale if scale is not None else t
    if scale is not None:
        grads["scale"] = (t * v).sum((0, 1))
    q = dv
    if w_post is not None:
        grads["w_post"] = (dv * n).sum((0, 1))
        q = dv * w_post
        q = rstd * (q - a * (rstd * rstd * _group_mean(q * a, group)))
    do = q
    if gate is not None:
        do = q * silu(gate)
        grads["gate"] = q * o * dsilu(gate)
    grads["o"] = do.map(lambda x: x.reshape(B, N, H, d).transpose(1, 2)) if o4 else do
    return r, h, grads


# ------------------------------------------------------------------ comparison

def worst(got, ref):
    """The largest error of a result as a share of what its type and the fp32 bound allow (<= 1 is
    right).  Values are finite."""
    g = got.detach().to(ref.v.device)
    assert tuple(g.shape) == tuple(ref.v.shape), (g.shape, ref.v.shape)
    half = HALF_STEP[g.dtype]
    g = g.double()
    assert torch.isfinite(g).all()
    allowed = SLACK * ref.e + half * (ref.v.abs() + SLACK * ref.e) + 1e-37
    return float(((g - ref.v).abs() / allowed).max()) if g.numel() else 0.0


def check(got, ref, what):
    w = worst(got, ref)
    assert w <= 1.0, f"{what}: {w:.3g} times the allowed error"
