"""The gated join with dropout on the GPU, against the 64-bit reference.

Tolerances.  y: gate * (h * s) has two roundings, the sum a third: 3 * 2^-24 of
(|x| + |g h s|), then half a step of the type, 2^-24 or 2^-8.  dh: three
roundings of itself and half a step.  dgate: n terms of two roundings each, in
some order of n - 1 additions: (n + 2) * 2^-24 of the sum of the terms'
absolute values."""

import pytest
import torch

import adaln_fwd_amd as A
from tests import ref_residual as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
RNG = (0x9876543210ABCDEF - 2 ** 64, 77)


def _make(B, N, D, dt, seed=0):
    g = torch.Generator().manual_seed(seed)
    x, h, dy = (torch.randn(B, N, D, generator=g).to(dt) for _ in range(3))
    return x, h, dy, torch.randn(B, D, generator=g).to(dt)


def _near(got, want, scale, dt, what):
    err = (got.double().cpu() - want).abs()
    allow = 3 * U * scale + HALF[dt] * (want.abs() + 3 * U * scale)
    bad = err > allow
    assert not bad.any(), (what, float((err - allow).max()))


def _check(x, h, dy, gate, p, got, rng=RNG, mod=None, nmod=0):
    """got: y, dh, dgate; rows flattened."""
    dt = h.dtype
    y, dh, dgate = got
    D = h.shape[-1]
    flat = [None if t is None else t.reshape(-1, D) for t in (x, h, dy)]
    want = R.forward(flat[0], flat[1], gate, p, rng, mod)
    xs = torch.zeros_like(want) if x is None else flat[0].double()
    _near(y.reshape(-1, D), want, xs.abs() + (want - xs).abs(), dt, "y")
    wdh, wdg, sums = R.backward(flat[2], flat[1], gate, p, rng, mod, nmod)
    _near(dh.reshape(-1, D), wdh, wdh.abs(), dt, "dh")
    if gate is None:
        assert dgate is None
        return
    n = flat[1].shape[0]
    err = (dgate.double().cpu() - wdg).abs()
    assert not (err > (n + 2) * U * sums).any(), float(err.max())


SHAPES = [(1, 1, 8), (2, 1, 64), (1, 7, 40), (3, 65, 136), (2, 300, 1536),
          (1, 1000, 64), (5, 33, 4104), (1, 90, 8192), (1, 5, 32768),
          (300, 2, 64), (2, 1, 16376)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("p", [0.0, 0.1])
def test_values_and_gradients(shape, dt, p):
    B, N, D = shape
    if dt == F32 and D > A.max_d(dt):
        D //= 2
    x, h, dy, gate = _make(B, N, D, dt)
    rng = torch.tensor(RNG, device="cuda") if p else None
    d = [t.cuda() for t in (x, h, dy, gate)]
    y = A.residual_fwd(d[0], d[1], d[3], p=p, rng=rng)
    dh, dgate = A.residual_bwd(d[2], d[1], d[3], p=p, rng=rng)
    mod = torch.arange(B).repeat_interleave(N)
    _check(x, h, dy, gate, p, (y, dh, dgate), mod=mod, nmod=B)


@pytest.mark.parametrize("D", [4, 12, 100, 1156])
def test_f32_rows_that_end_inside_a_block_of_numbers(D):
    x, h, dy, gate = _make(2, 37, D, F32, seed=D)
    rng = torch.tensor(RNG, device="cuda")
    d = [t.cuda() for t in (x, h, dy, gate)]
    y = A.residual_fwd(d[0], d[1], d[3], p=0.4, rng=rng)
    dh, dgate = A.residual_bwd(d[2], d[1], d[3], p=0.4, rng=rng)
    mod = torch.arange(2).repeat_interleave(37)
    _check(x, h, dy, gate, 0.4, (y, dh, dgate), mod=mod, nmod=2)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_dropout_alone_and_the_plain_sum(dt):
    x, h, dy, gate = _make(2, 50, 200, dt)
    rng = torch.tensor(RNG, device="cuda")
    d = [t.cuda() for t in (x, h, dy)]
    for xin, p in ((None, 0.5), (d[0], 0.5), (d[0], 0.0), (None, 0.0)):
        y = A.residual_fwd(xin, d[1], p=p, rng=rng)
        dh, dgate = A.residual_bwd(d[2], None, p=p, rng=rng)
        _check(None if xin is None else x, h, dy, None, p, (y, dh, dgate))


def test_rates_from_almost_none_to_almost_all():
    x, h, dy, gate = _make(1, 64, 512, F32)
    rng = torch.tensor(RNG, device="cuda")
    d = [t.cuda() for t in (x, h, dy, gate)]
    mod = torch.zeros(64, dtype=torch.int64)
    # the first is less than half of 2^-16: nothing is dropped
    for p in (2.0 ** -18, 2.0 ** -16, 0.999, 1 - 2.0 ** -16):
        y = A.residual_fwd(d[0], d[1], d[3], p=p, rng=rng)
        dh, dgate = A.residual_bwd(d[2], d[1], d[3], p=p, rng=rng)
        _check(x, h, dy, gate, p if p > 2.0 ** -17 else 0.0, (y, dh, dgate),
               mod=mod, nmod=1)


def test_what_is_dropped_leaves_nothing():
    """Infinities and NaN where the mask drops."""
    x, h, dy, gate = _make(1, 40, 256, F32)
    keep, _ = R.keep_mask(40, 256, 0.5, RNG)
    h[0][~keep] = float("nan")
    gate[:] = 2.0
    rng = torch.tensor(RNG, device="cuda")
    d = [t.cuda() for t in (x, h, dy, gate)]
    y = A.residual_fwd(d[0], d[1], d[3], p=0.5, rng=rng).cpu()
    assert torch.equal(y[0][~keep], x[0][~keep]) and y.isfinite().all()
    dh, dgate = A.residual_bwd(d[2], d[1], d[3], p=0.5, rng=rng)
    assert dgate.isfinite().all() and not dh.cpu()[0][~keep].any()
    d[2][0, ~keep] = float("inf")
    dh, dgate = A.residual_bwd(d[2], d[1], d[3], p=0.5, rng=rng)
    assert dgate.isfinite().all() and dh.isfinite().all()


def test_types_and_packing_share_the_mask():
    _, h, _, _ = _make(2, 31, 96, BF16)
    rng = torch.tensor(RNG, device="cuda")
    one = torch.ones(2, 31, 96)
    a = A.residual_fwd(None, one.to(BF16).cuda(), p=0.3, rng=rng) != 0
    b = A.residual_fwd(None, one.cuda(), p=0.3, rng=rng) != 0
    c = A.residual_fwd(None, one.reshape(1, 62, 96).cuda(), p=0.3, rng=rng) != 0
    assert torch.equal(a, b) and torch.equal(a.reshape(62, 96), c[0])


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_segments(dt, p):
    g = torch.Generator().manual_seed(5)
    off = [0, 0, 3, 3, 700, 701, 2000, 2000]
    mods = [4, 0, 1, 2, 0, 2, 2]  # vector 3 unused, 0 and 2 shared
    x, h, dy = (torch.randn(2000, 520, generator=g).to(dt) for _ in range(3))
    gate = torch.randn(5, 520, generator=g).to(dt)
    mod = torch.cat([torch.full((b - a,), m) for a, b, m in
                     zip(off, off[1:], mods)]).long()
    rng = torch.tensor(RNG, device="cuda")
    d = [t.cuda() for t in (x, h, dy, gate)]
    tab = A.SegTable(off, mods)
    y = A.residual_fwd_segments(d[0], d[1], d[3], tab, p=p, rng=rng)
    dh, dgate = A.residual_bwd_segments(d[2], d[1], d[3], tab, p=p, rng=rng)
    _check(x, h, dy, gate, p, (y, dh, dgate), mod=mod, nmod=5)
    assert not dgate[3].any() and not dgate[4].any()
    y2 = A.residual_fwd_segments(d[0], d[1], d[3], off, mods, p=p, rng=rng)
    assert torch.equal(y, y2)


def test_empty_calls():
    z = torch.zeros(3, 0, 64, device="cuda")
    gate = torch.ones(3, 64, device="cuda")
    assert A.residual_fwd(z, z, gate).shape == (3, 0, 64)
    dh, dgate = A.residual_bwd(z, z, gate, dgate=torch.ones_like(gate))
    assert not dgate.any()
    t = torch.zeros(0, 64, device="cuda")
    dh, dgate = A.residual_bwd_segments(t, t, gate, [0, 0, 0], [1, 1],
                                        dgate=torch.ones_like(gate))
    assert not dgate.any()
    e = torch.zeros(0, 4, 64, device="cuda")
    A.residual_bwd(e, e, gate[:0])


def test_in_place_streams_and_repeats():
    x, h, dy, gate = (t.cuda() for t in _make(2, 3000, 1544, BF16))
    rng = torch.tensor(RNG, device="cuda")
    y = A.residual_fwd(x, h, gate, p=0.1, rng=rng)
    dh, dgate = A.residual_bwd(dy, h, gate, p=0.1, rng=rng)
    for src in ("x", "h"):
        c = {"x": x.clone(), "h": h.clone()}
        out = A.residual_fwd(c["x"], c["h"], gate, p=0.1, rng=rng, y=c[src])
        assert out is c[src] and torch.equal(out, y)
    for src in ("dy", "h"):
        c = {"dy": dy.clone(), "h": h.clone()}
        a, b = A.residual_bwd(c["dy"], c["h"], gate, p=0.1, rng=rng, dh=c[src])
        assert torch.equal(a, dh) and torch.equal(b, dgate)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a, b = A.residual_bwd(dy, h, gate, p=0.1, rng=rng, stream=s)
    s.synchronize()
    assert torch.equal(a, dh) and torch.equal(b, dgate)


def test_captured_calls_draw_new_numbers():
    x, h, dy, gate = (t.cuda() for t in _make(1, 200, 256, BF16))
    rng = torch.tensor(RNG, device="cuda")
    ws = torch.empty(A.residual_bwd_workspace_bytes(1, 200, 256, BF16) + 16,
                     dtype=torch.uint8, device="cuda")
    A.residual_bwd(dy, h, gate, p=0.3, rng=rng)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rng[1] += 1
        y = A.residual_fwd(x, h, gate, p=0.3, rng=rng)
        dh, dgate = A.residual_bwd(dy, h, gate, p=0.3, rng=rng, workspace=ws)
    seen = []
    for i in range(1, 4):
        graph.replay()
        torch.cuda.synchronize()
        now = torch.tensor((RNG[0], RNG[1] + i), device="cuda")
        assert torch.equal(rng, now)
        assert torch.equal(y, A.residual_fwd(x, h, gate, p=0.3, rng=now))
        a, b = A.residual_bwd(dy, h, gate, p=0.3, rng=now)
        assert torch.equal(dh, a) and torch.equal(dgate, b)
        seen.append(y.clone())
    assert not torch.equal(seen[0], seen[1])


def test_refusals_of_the_binding_on_the_gpu():
    x, h, dy, gate = (t.cuda() for t in _make(2, 3, 64, BF16))
    rng = torch.tensor(RNG, device="cuda")
    for bad in (dict(p=-0.1), dict(p=1.0), dict(p=0.1)):
        with pytest.raises(ValueError):
            A.residual_fwd(x, h, gate, **bad)
    with pytest.raises(TypeError):
        A.residual_fwd(x, h, gate, p=0.1, rng=rng.int())
    with pytest.raises(ValueError):
        A.residual_fwd(x, h, gate, p=0.1, rng=rng.cpu())
    with pytest.raises(ValueError):
        A.residual_fwd(x, h, gate[:1])
    with pytest.raises(TypeError):
        A.residual_fwd(x, h, gate.float())
    with pytest.raises(ValueError):
        A.residual_fwd(x.transpose(0, 1), h.transpose(0, 1), gate)
    with pytest.raises(ValueError):
        A.residual_bwd(dy, h, dgate=gate.float())
    with pytest.raises(TypeError):
        A.residual_bwd(dy, None, gate)
    big = torch.zeros(2, 4000, 64, device="cuda", dtype=BF16)
    with pytest.raises(A.AdalnError):
        A.residual_bwd(big, big, gate,
                       workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


def test_rows_past_32_bit_offsets():
    """2^31 elements and more: the last rows are where they belong."""
    N, D = 262400, 8192
    h = torch.zeros(1, N, D, device="cuda", dtype=BF16)
    h[0, -3:] = 1
    rng = torch.tensor(RNG, device="cuda")
    y = A.residual_fwd(None, h, p=0.5, rng=rng, y=h)
    keep, s = R.keep_mask(3, D, 0.5, RNG, row0=N - 3)
    assert torch.equal(y[0, -3:].cpu().double(), keep.double() * s)
