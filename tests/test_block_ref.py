"""The 64-bit references of the block operators against differences of their own forward passes, and
against hand-worked values (CPU)."""
import math

import pytest
import torch

import block_ref as R


def _rng(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)


def _differences(f, tensors, grads, step=1e-5, tol=1e-7):
    """Central differences of f(tensors) along a random direction of each tensor."""
    rand = _rng(99)
    for name, t in tensors.items():
        if t is None or grads.get(name) is None:
            continue
        d = rand(*t.shape)
        up, down = f({**tensors, name: t + step * d}), f({**tensors, name: t - step * d})
        got = float((grads[name].v * d).sum())
        assert abs((up - down) / (2 * step) - got) <= tol * (1 + abs(got)), name


@pytest.mark.parametrize("z,G,lengths", [(True, 1, None), (False, 2, [5, 0, 3]), (True, 2, [7, 1, 4])])
def test_scan_gradients_are_those_of_differences(z, G, lengths):
    rand = _rng(1)
    B, N, D, S = 3, 7, 4, 8
    t = {"u": rand(B, N, D), "dt": rand(B, N, D), "a_log": rand(D, S) * 0.5, "b": rand(B, N, G, S),
         "c": rand(B, N, G, S), "d_skip": rand(D), "dt_bias": rand(D), "z": rand(B, N, D) if z else None,
         "state": rand(B, D, S)}
    dy, dstate = rand(B, N, D), rand(B, D, S)
    grads = R.scan(**t, lengths=lengths, dy=dy, dstate_out=dstate)[2]

    def f(s):
        y, h = R.scan(**s, lengths=lengths)
        return float((y.v * dy).sum() + (h.v * dstate).sum())
    _differences(f, t, grads)


@pytest.mark.parametrize("W,lengths", [(4, None), (2, [3, 0, 6]), (3, [1, 2, 6])])
def test_conv_gradients_are_those_of_differences(W, lengths):
    rand = _rng(2)
    B, N, D = 3, 6, 5
    t = {"x": rand(B, N, D), "weight": rand(D, W), "bias": rand(D)}
    state, dy = rand(B, W - 1, D), rand(B, N, D)
    grads = R.conv(**t, state=state, lengths=lengths, dy=dy)[2]
    _differences(lambda s: float((R.conv(**s, state=state, lengths=lengths)[0].v * dy).sum()), t, grads)


@pytest.mark.parametrize("group,gate,residual,w_pre", [(0, True, True, True), (8, True, False, False),
                                                       (8, False, True, True), (0, False, False, True)])
def test_norm_gradients_are_those_of_differences(group, gate, residual, w_pre):
    rand = _rng(3)
    B, H, N, d = 2, 2, 3, 8
    D = H * d
    t = {"o": rand(B, H, N, d), "w_post": rand(D), "gate": rand(B, N, D) if gate else None,
         "residual": rand(B, N, D) if residual else None, "scale": rand(D) if residual else None,
         "w_pre": rand(D) if w_pre else None}
    dr, dh = rand(B, N, D), rand(B, N, D) if w_pre else None
    kept = R.norm(**t, group=group)[0].v
    grads = R.norm(**t, group=group, r_stored=kept, dr=dr, dh=dh)[2]

    def f(s):
        r = R.norm(**s, group=group)[0].v
        out = float((r * dr).sum())
        if w_pre:
            out += float((R.norm(**s, group=group, r_stored=r)[1].v * dh).sum())
        return out
    _differences(f, t, grads)


def test_scan_by_hand():
    """Two tokens, one channel: h1 = d1 b1 u1, h2 = exp(-d2 e^a) h1 + d2 b2 u2 (eight equal states)."""
    u, dt = torch.tensor([[[2.0], [3.0]]]), torch.tensor([[[0.5], [-0.25]]])
    a_log = torch.full((1, 8), 0.3)
    b, c = torch.full((1, 2, 8), 0.7), torch.full((1, 2, 8), -1.5)
    y, h = R.scan(u, dt, a_log, b, c)
    d1, d2 = math.log1p(math.exp(0.5)), math.log1p(math.exp(-0.25))
    h1 = d1 * 0.7 * 2
    h2 = math.exp(-d2 * math.exp(0.3)) * h1 + d2 * 0.7 * 3
    assert torch.allclose(h.v, torch.full((1, 1, 8), h2, dtype=torch.float64), rtol=1e-6)
    assert torch.allclose(y.v[0, :, 0], torch.tensor([-12 * h1, -12 * h2], dtype=torch.float64), rtol=1e-6)


def test_norm_by_hand():
    """o = (3, 4) twice over eight channels in groups of eight: rms = sqrt(12.5)."""
    o = torch.tensor([3.0, 4.0] * 4).reshape(1, 1, 8)
    r, _, _ = R.norm(o, w_post=torch.full((8,), 2.0), eps=0.0, group=8)
    assert torch.allclose(r.v[0, 0, :2], torch.tensor([6.0, 8.0], dtype=torch.float64) / math.sqrt(12.5))
