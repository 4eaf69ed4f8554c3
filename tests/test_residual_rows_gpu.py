"""The gated join with dropout, every element compared so that no missing number
passes: small calls, and calls past the caches' size, whose kernels access memory
with the streaming hint, also in place and packed.

Tolerances: those of test_residual_gpu.py.  y: 3 * 2^-24 of (|x| + |g h s|), then
half a step of the type.  dh: three roundings of itself and half a step.  dgate:
(n + 2) * 2^-24 of the sum of the terms' absolute values, n of them."""

import pytest
import torch

import adaln_fwd_amd as A
from tests import near
from tests import ref_residual as R
from tests.test_residual_gpu import HALF, RNG, SHAPES, U

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _make(rows, D, nmod, dt):
    g = torch.Generator(device="cuda").manual_seed(rows + D)
    return [torch.randn(n, D, generator=g, device="cuda").to(dt)
            for n in (rows, rows, rows, nmod)]


def _check(x, h, dy, gate, mod, p, y, dh, dgate):
    """On the GPU, in float64: rows [T, D], mod: each row's vector."""
    dt, (T, D) = h.dtype, h.shape
    keep, s = (torch.ones(1, 1, dtype=torch.bool), 1.0) if p == 0 else \
        R.keep_mask(T, D, p, RNG)
    keep = keep.cuda().expand(T, D)
    sums = torch.zeros(2, *gate.shape, dtype=torch.float64, device="cuda")
    count = torch.bincount(mod, minlength=gate.shape[0])
    for a in range(0, T, 4000):
        i = slice(a, a + 4000)
        g = gate.double()[mod[i]]
        branch = torch.where(keep[i], s * h[i].double(), 0.0)
        want = x[i].double() + g * branch
        slack = 3 * U * (x[i].double().abs() + (g * branch).abs())
        near.check(y[i], want, slack + HALF[dt] * (want.abs() + slack), "y")
        want = torch.where(keep[i], s * g * dy[i].double(), 0.0)
        slack = 3 * U * want.abs()
        near.check(dh[i], want, slack + HALF[dt] * (want.abs() + slack), "dh")
        terms = branch * dy[i].double()
        sums[0].index_add_(0, mod[i], terms)
        sums[1].index_add_(0, mod[i], terms.abs())
    near.check(dgate, sums[0], (count + 2)[:, None] * U * sums[1], "dgate")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_small_calls(shape, dt, p):
    B, N, D = shape
    if D > A.max_d(dt):
        D //= 2
    x, h, dy, gate = _make(B * N, D, B, dt)
    rng = torch.tensor(RNG, device="cuda") if p else None
    v = [t.view(B, N, D) for t in (x, h, dy)]
    y = A.residual_fwd(v[0], v[1], gate, p=p, rng=rng)
    dh, dgate = A.residual_bwd(v[2], v[1], gate, p=p, rng=rng)
    mod = torch.arange(B, device="cuda").repeat_interleave(N)
    _check(x, h, dy, gate, mod, p, y.view(-1, D), dh.view(-1, D), dgate)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("packed", [False, True], ids=["uniform", "packed"])
def test_past_the_caches(dt, p, packed):
    """A call moves more than 192 MiB; rows of an odd number of vectors."""
    T, D = 24000, 1544 if dt == BF16 else 772
    assert 3 * T * 3088 > 192 << 20
    print(f"[residual] {dt} {p} {'packed' if packed else ''}", flush=True)
    x, h, dy, gate = _make(T, D, 3, dt)
    rng = torch.tensor(RNG, device="cuda") if p else None
    kw = dict(p=p, rng=rng)
    if packed:
        off, mods = [0, 1, 7001, 7001, 20000, T], [2, 0, 1, 0, 2]
        tab = A.SegTable(off, mods)
        mod = torch.cat([torch.full((b - a,), m) for a, b, m in
                         zip(off, off[1:], mods)]).cuda()

        def fwd(x, h, **more):
            return A.residual_fwd_segments(x, h, gate, tab, **kw, **more)

        def bwd(dy, h, **more):
            return A.residual_bwd_segments(dy, h, gate, tab, **kw, **more)
    else:
        x, h, dy = (t.view(3, T // 3, D) for t in (x, h, dy))
        mod = torch.arange(3, device="cuda").repeat_interleave(T // 3)

        def fwd(x, h, **more):
            return A.residual_fwd(x, h, gate, **kw, **more)

        def bwd(dy, h, **more):
            return A.residual_bwd(dy, h, gate, **kw, **more)

    y = fwd(x, h)
    dh, dgate = bwd(dy, h)
    flat = [t.reshape(T, D) for t in (x, h, dy)]
    _check(*flat, gate, mod, p, y.view(T, D), dh.view(T, D), dgate)
    for i in range(2):
        c = [x.clone(), h.clone()]
        assert fwd(*c, y=c[i]) is c[i] and torch.equal(c[i], y)
        c = [dy.clone(), h.clone()]
        again, d2 = bwd(*c, dh=c[i])
        assert again is c[i] and torch.equal(again, dh)
        assert torch.equal(d2, dgate)
