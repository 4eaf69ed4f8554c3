"""The activations' values and derivatives, to bounds of a few roundings.

With D = 8, x = (g, 1, 0, ...), one gate row (1, 0, ...), and one other row
(0, 1, 0, ...), G is g and U is 1 to the last bit; with dh = 1 in that hidden
feature and 0 in the others, dx[:, 0] is act'(g) and dx[:, 1] is act(g), the
float32 results of the activation themselves.

Bounds, u = 2^-24.  s = 1 / (1 + E), E = exp(-v): the float32 exponential is
within 2 u of itself, 1 + E within u more, the reciprocal within 2 u, so s is
within 5 u; its complement c = E s within 2 + 5 + 1 = 8 u.  silu: v = g; the
value g s is within 6 u; the derivative s + s g c adds the terms' roundings:
7 u s + 16 u |s g c|.  gelu: v = 2 sqrt(2 / pi) g (1 + 0.044715 g^2) is within
7 u of itself, which moves E by 7 |v| u of itself, and s by c times that, c by s
times that.  Below v = -88.7 E is infinite and s, less than 2^-128, is zero."""

import math

import pytest
import torch

import adaln_fwd_amd as A

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _say(msg):
    print(f"[glu] {msg}", flush=True)


def _kernel(g, act):
    """act(g), act'(g) of float32, and the forward's h."""
    M = g.numel()
    x = torch.zeros(M, 8)
    x[:, 0], x[:, 1] = g, 1
    wg, wu, dh = torch.zeros(8, 8), torch.zeros(8, 8), torch.zeros(M, 8)
    wg[0, 0], wu[0, 1], dh[:, 0] = 1, 1, 1
    x, wg, wu, dh = [t.cuda() for t in (x, wg, wu, dh)]
    h, saved = A.glu_fwd(x, wg, wu, act=act, save=True)
    assert torch.equal(saved[0, :, 0].cpu(), g)
    dx = A.glu_bwd(dh, x, wg, wu, saved, act=act)[0]
    again = A.glu_bwd(dh, x, wg, wu, None, act=act)[0]
    assert torch.equal(dx, again)
    assert torch.equal(h[:, 0], dx[:, 1])
    return dx[:, 1].cpu().double(), dx[:, 0].cpu().double()


def _bounds(g, act):
    """a, da of float64 and their bounds."""
    g = g.double()
    if act == "silu":
        v, dv = g, torch.ones_like(g)
    else:
        k = 2 * math.sqrt(2 / math.pi)
        v, dv = k * (g + 0.044715 * g ** 3), k * (1 + 3 * 0.044715 * g * g)
    s, c = torch.sigmoid(v), torch.sigmoid(-v)
    move = 0 * v if act == "silu" else 7 * v.abs()
    t = g * s * c * dv
    a = g * s
    ea = U * a.abs() * (6 + c * move)
    eda = U * (s * (7 + c * move) + t.abs() * (16 + (1 - 2 * c).abs() * move))
    if act == "gelu":
        # the polynomial of the derivative: 5 more roundings
        eda = eda + 5 * U * t.abs()
    low = 2.0 ** -128 * (1 + g.abs() * (1 + dv)) + 2.0 ** -126
    return a, s + t, ea + low, eda + low


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M", [4, 64, 24001])
def test_activations_of_float32(act, M):
    """Over [-12, 12], where the tests on random numbers hardly go; by the
    kernels for few tokens and by those for many."""
    _say(f"activation {act} {M}")
    g = torch.linspace(-12, 12, M) if M > 100 else \
        torch.linspace(-5, 11.9, M)
    got, dgot = _kernel(g, act)
    a, da, ea, eda = _bounds(g, act)
    for x, ref, tol, n in ((got, a, ea, "act"), (dgot, da, eda, "act'")):
        err = (x - ref).abs()
        bad = ~(err <= tol)
        assert not bad.any(), (n, int(bad.sum()), float(g[(err / tol).argmax()]),
                               float((err / tol).max()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_derivatives_of_the_largest_numbers(act, dtype):
    """act' is 1 or 0 there, where g^2 and exp(-g) are infinite."""
    _say(f"largest numbers {act} {dtype}")
    g = torch.tensor([1e4, 1e12, 1e18, 2e19, 1e30, 3e38])
    g = torch.cat([g, -g]).to(dtype)
    for M in (12, 240):
        x = torch.zeros(M, 8, dtype=dtype)
        x[:, 0] = g.repeat(M // 12)
        x[:, 1] = 1
        wg, wu, dh = torch.zeros(8, 8), torch.zeros(8, 8), torch.zeros(M, 8)
        wg[0, 0], wu[0, 1], dh[:, 0] = 1, 1, 1
        x, wg, wu, dh = [t.to(dtype).cuda() for t in (x, wg, wu, dh)]
        h, saved = A.glu_fwd(x, wg, wu, act=act, save=True)
        want = x[:, 0].clamp_min(0)
        assert torch.equal(h[:, 0], want)
        for s in (saved, None):
            dx = A.glu_bwd(dh, x, wg, wu, s, act=act)[0]
            assert torch.equal(dx[:, 0], (want > 0).to(dtype))
            assert torch.equal(dx[:, 1], want)
