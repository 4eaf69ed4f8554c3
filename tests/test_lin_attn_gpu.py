"""Linear attention on the GPU, against the 64-bit reference.

Tolerances, relative to the sum of the terms' absolute values, each term times
1 + |log_decay| * distance: a power of the decay has a relative error of a few
2^-24 for itself and one per unit of its exponent, the rounding of its argument;
float32 additions and products, at most N / 8 + 4 d + 64 in a row (a matrix
instruction adds 16 terms to a sum, chunks of 32 tokens pass the state on with a
product); of bf16, three numbers on a term's way that are given as the sum of two
bf16, 2^-16 each.  Then half a step of the output's type.  States and the
gradients of states are float32 whatever the type."""

import pytest
import torch

import adaln_fwd_amd as A
from tests import ref_lin_attn as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def _make(B, N, H, d, dt, seed=0):
    g = torch.Generator().manual_seed(seed)
    q, k, v, do = (torch.randn(B, N, H, d, generator=g).to(dt)
                   for _ in range(4))
    S0, dS = (torch.randn(B, H, d, d, generator=g) * 3 for _ in range(2))
    decay = -(2.0 ** -torch.linspace(0, 9, H))
    if H > 2:
        decay[0], decay[1] = 0.0, float("-inf")
    return q, k, v, do, S0, dS, decay


def _near(got, want, sums, N, d, dt, what, out=None):
    rel = (N / 8 + 4 * d + 64) * U + (3 * 2.0 ** -16 if dt == BF16 else 0)
    slack = rel * sums
    allow = slack + HALF[out or dt] * (want.abs() + slack)
    err = (got.double().cpu() - want).abs()
    bad = ~(err <= allow)
    assert not bad.any(), (what, bad.nonzero()[0].tolist(),
                           float((err / allow).max()))


def _check_all(ins, outs, grads, dt, seqs, scale):
    """seqs: (sample or None, first token, end) of each state."""
    q, k, v, do, S0, dS, decay = ins
    o, last = outs
    dq, dk, dv, d0 = grads
    d = q.shape[-1]
    for i, (b, a, e) in enumerate(seqs):
        pick = (lambda t: (t if b is None else t[b])[a:e])
        n = e - a
        s0, ds = (None if t is None else t[i] for t in (S0, dS))
        x = (pick(q), pick(k), pick(v), decay, scale, s0)
        want, wlast = R.forward(*x)
        sums, slast = R.forward(*x, sums=True)
        _near(pick(o), want, sums, n, d, dt, "o")
        if last is not None:
            _near(last[i], wlast, slast, n, d, dt, "state", F32)
        want = R.backward(pick(do), *x[:5], s0, ds)
        sums = R.backward(pick(do), *x[:5], s0, ds, sums=True)
        for got, w, s, what in zip((dq, dk, dv), want, sums,
                                   ("dq", "dk", "dv")):
            _near(pick(got), w, s, n, d, dt, what)
        if d0 is not None:
            _near(d0[i], want[3], sums[3], n, d, dt, "dstate", F32)


def _run(ins, scale=None, tab=None, save=True, views=None):
    q, k, v, do, S0, dS, decay = ins
    g = [t.cuda() for t in (q, k, v, do)] if views is None else views
    S0, dS = (None if t is None else t.cuda() for t in (S0, dS))
    decay = decay.cuda()
    o, last, saved = A.lin_attn_fwd(*g[:3], decay, scale=scale, state=S0,
                                    final=True, save=save, seg_offsets=tab)
    grads = A.lin_attn_bwd(g[3], *g[:3], decay, scale=scale, state=S0,
                           saved=saved, dstate_out=dS, seg_offsets=tab)
    return (o, last), grads


SHAPES = [(1, 1, 1, 8), (2, 3, 4, 16), (1, 31, 3, 32), (1, 32, 3, 40),
          (3, 33, 2, 64), (1, 64, 3, 72), (2, 65, 3, 96), (1, 127, 4, 104),
          (1, 128, 3, 128), (1, 129, 5, 128), (2, 300, 3, 128),
          (1, 1000, 4, 64), (1, 777, 3, 24), (40, 5, 3, 48), (1, 2200, 2, 128)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_values_and_gradients(shape, dt):
    B, N, H, d = shape
    ins = _make(B, N, H, d, dt)
    outs, grads = _run(ins)
    _check_all(ins, outs, grads, dt, [(b, 0, N) for b in range(B)], d ** -0.5)


@pytest.mark.parametrize("d", [4, 12, 20, 36, 44, 68, 100, 124])
def test_f32_heads_of_odd_vectors(d):
    ins = _make(1, 70, 3, d, F32)
    outs, grads = _run(ins, scale=-0.3)
    _check_all(ins, outs, grads, F32, [(0, 0, 70)], -0.3)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_without_states(dt):
    ins = list(_make(2, 400, 3, 64, dt))
    ins[4] = ins[5] = None
    outs, grads = _run(ins, save=False)
    assert grads[3] is None
    _check_all(ins, outs, grads, dt, [(b, 0, 400) for b in range(2)], 0.125)
    q, k, v = (t.cuda() for t in ins[:3])
    o, last, saved = A.lin_attn_fwd(q, k, v, ins[6].cuda())
    assert last is None and saved is None and torch.equal(o, outs[0])


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_packed_sequences(dt):
    off = [0, 0, 1, 40, 40, 640, 641, 1300, 1364]
    ins = list(_make(1, 1364, 4, 72, dt))
    for i in range(4):
        ins[i] = ins[i][0]
    g = torch.Generator().manual_seed(9)
    ins[4], ins[5] = (torch.randn(8, 4, 72, 72, generator=g) for _ in range(2))
    outs, grads = _run(ins, tab=off)
    _check_all(ins, outs, grads, dt, [(None, a, b) for a, b in
                                      zip(off, off[1:])], 72 ** -0.5)
    # sequences without tokens hand their states on
    assert torch.equal(outs[1][0].cpu(), ins[4][0])
    assert torch.equal(grads[3][3].cpu(), ins[5][3])
    again, _ = _run(ins, tab=A.SegTable(off))
    assert torch.equal(again[0], outs[0])


def test_whole_numbers_come_out_exactly():
    """Without decay, of small whole numbers: every sum is exact, so every
    element of every output is."""
    for dt in (BF16, F32):
        for N, d in ((700, 128), (333, 64), (95, 96), (200, 32)):
            g = torch.Generator().manual_seed(N)
            q, k, v, do = (torch.randint(-1, 2, (2, N, 3, d), generator=g)
                           .to(dt) for _ in range(4))
            S0, dS = (torch.randint(-3, 4, (2, 3, d, d), generator=g).float()
                      for _ in range(2))
            ins = (q, k, v, do, S0, dS, torch.zeros(3))
            (o, last), grads = _run(ins, scale=1.0)
            for b in range(2):
                x = (q[b], k[b], v[b], torch.zeros(3), 1.0, S0[b])
                want = R.forward(*x)
                assert torch.equal(o[b].cpu(), want[0].to(dt))
                assert torch.equal(last[b].cpu().double(), want[1])
                back = R.backward(do[b], *x, dS[b])
                for got, w in zip(grads[:3], back):
                    assert torch.equal(got[b].cpu(), w.to(dt))
                assert torch.equal(grads[3][b].cpu().double(), back[3])


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_views_of_a_projection_and_head_major(dt):
    B, N, H, d = 2, 150, 3, 64
    ins = _make(B, N, H, d, dt, seed=4)
    outs, grads = _run(ins)
    x = torch.stack([t.cuda() for t in ins[:3]], 2).reshape(B, N, 3 * H * d)
    views = [x[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d))
             for i in range(3)]
    # head-major do; gradients into slices of one tensor
    do = ins[3].cuda().transpose(1, 2).contiguous().transpose(1, 2)
    dx = torch.full_like(x, 7.0)
    dviews = [dx[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d))
              for i in range(3)]
    decay, S0, dS = (t.cuda() for t in (ins[6], ins[4], ins[5]))
    o = torch.empty(B, H, N, d, device="cuda", dtype=dt).transpose(1, 2)
    got, last, saved = A.lin_attn_fwd(*views, decay, state=S0, final=True,
                                      save=True, o=o)
    assert got is o and torch.equal(o, outs[0]) and torch.equal(last, outs[1])
    A.lin_attn_bwd(do, *views, decay, state=S0, saved=saved, dstate_out=dS,
                   dq=dviews[0], dk=dviews[1], dv=dviews[2])
    for a, b in zip(dviews, grads):
        assert torch.equal(a, b)


def test_shared_heads():
    """Keys and values of one head for all: a distance of 0 between heads."""
    ins = list(_make(1, 90, 4, 64, F32))
    one = [ins[i][:, :, :1].cuda() for i in (1, 2)]
    k, v = (t.expand(1, 90, 4, 64) for t in one)
    ins[1], ins[2] = k.cpu(), v.cpu()
    outs, grads = _run(ins, views=[ins[0].cuda(), k, v, ins[3].cuda()])
    _check_all(ins, outs, grads, F32, [(0, 0, 90)], 0.125)


def test_a_sequence_in_pieces():
    """Pieces from state to state, and the gradients back through them."""
    q, k, v, do, S0, dS, decay = (t.cuda() for t in
                                  _make(1, 500, 3, 64, F32))
    o, last, _ = A.lin_attn_fwd(q, k, v, decay, state=S0, final=True)
    want = A.lin_attn_bwd(do, q, k, v, decay, state=S0, dstate_out=dS)
    s, cuts, parts = S0, [0, 77, 300, 500], []
    states = []
    for a, b in zip(cuts, cuts[1:]):
        states.append(s)
        y, s, _ = A.lin_attn_fwd(q[:, a:b], k[:, a:b], v[:, a:b], decay,
                                 state=s, final=True)
        parts.append(y)
    tol = dict(rtol=1e-4, atol=1e-3)
    torch.testing.assert_close(torch.cat(parts, 1), o, **tol)
    torch.testing.assert_close(s, last, **tol)
    ds = dS
    for a, b, s in reversed(list(zip(cuts, cuts[1:], states))):
        dq, dk, dv, ds = A.lin_attn_bwd(do[:, a:b], q[:, a:b], k[:, a:b],
                                        v[:, a:b], decay, state=s,
                                        dstate_out=ds)
        for got, w in zip((dq, dk, dv), want):
            torch.testing.assert_close(got, w[:, a:b], **tol)
    torch.testing.assert_close(ds, want[3], **tol)


@pytest.mark.parametrize("shape", [(1, 1, 8), (1, 12, 128), (3, 4, 72),
                                   (70, 5, 96), (64, 24, 128), (2, 3, 40)],
                         ids=str)
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_steps(shape, dt):
    B, H, d = shape
    q, k, v, _, S0, _, decay = _make(B, 1, H, d, dt)
    g = [t[:, 0].cuda() for t in (q, k, v)]
    o, out = A.lin_attn_step(*g, decay.cuda(), S0.cuda(),
                             state_out=torch.empty_like(S0, device="cuda"))
    for b in range(B):
        x = (q[b], k[b], v[b], decay, d ** -0.5, S0[b])
        want, last = R.forward(*x)
        sums, slast = R.forward(*x, sums=True)
        # no product is split in two: the float32 tolerance for both types
        _near(o[b:b + 1], want, sums, 1, d, F32, "o", dt)
        _near(out[b], last, slast, 1, d, F32, "state")
    own = S0.cuda()
    o2, out2 = A.lin_attn_step(*g, decay.cuda(), own)
    assert out2 is own and torch.equal(own, out) and torch.equal(o2, o)


def test_steps_follow_a_prompt():
    q, k, v, _, S0, _, decay = (t.cuda() for t in _make(2, 45, 3, 64, F32))
    o, last, _ = A.lin_attn_fwd(q, k, v, decay, state=S0, final=True)
    y, s, _ = A.lin_attn_fwd(q[:, :40], k[:, :40], v[:, :40], decay, state=S0,
                             final=True)
    for t in range(40, 45):
        y, s = A.lin_attn_step(q[:, t], k[:, t], v[:, t], decay, s)
        torch.testing.assert_close(y, o[:, t], rtol=1e-4, atol=1e-3)
    torch.testing.assert_close(s, last, rtol=1e-4, atol=1e-3)


def test_what_lies_behind_a_sequence_is_not_read():
    """Tokens past a sequence's end in a longer buffer hold NaN."""
    q, k, v, do, S0, dS, decay = _make(1, 170, 3, 64, BF16)
    outs, grads = _run((q[:, :135], k[:, :135], v[:, :135], do[:, :135], S0,
                        dS, decay))
    for t in (q, k, v, do):
        t[:, 135:] = float("nan")
    views = [t.cuda()[:, :135] for t in (q, k, v, do)]
    more, mgrads = _run((q, k, v, do, S0, dS, decay), views=views)
    for a, b in zip(outs + grads, more + mgrads):
        assert torch.equal(a, b)
    # and what lies there is left as it is
    o = torch.full((1, 170, 3, 64), 5.0, device="cuda", dtype=BF16)
    A.lin_attn_fwd(*views[:3], decay.cuda(), state=S0.cuda(), o=o[:, :135])
    assert torch.equal(o[:, :135], outs[0]) and (o[:, 135:] == 5).all()


def test_empty_calls():
    z = torch.zeros(2, 0, 3, 64, device="cuda")
    S = torch.randn(2, 3, 64, 64, device="cuda")
    decay = torch.zeros(3, device="cuda")
    o, last, _ = A.lin_attn_fwd(z, z, z, decay, state=S, final=True)
    assert o.shape == z.shape and torch.equal(last, S)
    assert not A.lin_attn_fwd(z, z, z, decay, final=True)[1].any()
    *_, d0 = A.lin_attn_bwd(z, z, z, z, decay, state=S, dstate_out=S)
    assert torch.equal(d0, S)
    e = torch.zeros(0, 5, 3, 64, device="cuda")
    assert A.lin_attn_fwd(e, e, e, decay, final=True)[1].shape == (0, 3, 64, 64)
    h = torch.zeros(2, 5, 0, 64, device="cuda")
    A.lin_attn_bwd(h, h, h, h, decay[:0])
    A.lin_attn_step(e[:, 0], e[:, 0], e[:, 0], decay, S[:0])


def test_streams_graphs_and_repeats():
    ins = _make(1, 1500, 3, 128, BF16)
    q, k, v, do, S0, dS, decay = (t.cuda() for t in ins)

    def run(stream=None):
        o, last, saved = A.lin_attn_fwd(q, k, v, decay, state=S0, final=True,
                                        save=True, stream=stream)
        return (o, last) + A.lin_attn_bwd(do, q, k, v, decay, state=S0,
                                          saved=saved, dstate_out=dS,
                                          stream=stream)

    want = run()
    for got in (run(), ):
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    # without the saved states
    for a, b in zip(A.lin_attn_bwd(do, q, k, v, decay, state=S0,
                                   dstate_out=dS), want[2:]):
        assert torch.equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
        y, st = A.lin_attn_step(q[:, 0], k[:, 0], v[:, 0], decay, got[1])
    for i in range(3):
        q.copy_(q.flip(1))
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        y2, st2 = A.lin_attn_step(q[:, 0], k[:, 0], v[:, 0], decay, want[1])
        for a, b in zip(got + (y, ), want + (y2, )):
            assert torch.equal(a, b)


def test_refusals_of_the_binding_on_the_gpu():
    q, k, v, do, S0, dS, decay = (t.cuda() for t in _make(2, 3, 4, 64, BF16))
    with pytest.raises(ValueError):
        A.lin_attn_fwd(q, k[:, :2], v, decay)
    with pytest.raises(TypeError):
        A.lin_attn_fwd(q, k.float(), v, decay)
    with pytest.raises(TypeError):
        A.lin_attn_fwd(q, k, v, decay.double())
    with pytest.raises(ValueError):
        A.lin_attn_fwd(q, k, v, decay[:3])
    with pytest.raises(TypeError):
        A.lin_attn_fwd(q, k, v, decay, state=S0.to(BF16))
    with pytest.raises(ValueError):
        A.lin_attn_fwd(q, k, v, decay, state=S0[:1])
    with pytest.raises(ValueError):
        A.lin_attn_fwd(q.transpose(-1, -2), k, v, decay)
    with pytest.raises(ValueError):
        A.lin_attn_step(q, k, v, decay, S0)
    with pytest.raises(A.AdalnError):
        A.lin_attn_fwd(*[t[..., :60].contiguous() for t in (q, k, v)], decay)
    with pytest.raises(A.AdalnError):
        t = torch.zeros(1, 2, 1, 136, device="cuda")
        A.lin_attn_fwd(t, t, t, decay[:1])
    long = torch.zeros(1, 900, 1, 64, device="cuda")
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        A.lin_attn_bwd(long, long, long, long, decay[:1], saved=small)
    with pytest.raises(A.AdalnError):
        A.lin_attn_bwd(long, long, long, long, decay[:1], workspace=small)


def test_rows_past_32_bit_offsets():
    """A head's last tokens, 2^31 elements and more into the tensors."""
    N, H, d = 70000, 260, 128
    x = torch.zeros(1, N, H, d, device="cuda", dtype=BF16)
    g = torch.Generator().manual_seed(2)
    tail = torch.randn(40, 3, d, generator=g).to(BF16)
    x[0, -40:, -3:] = tail.cuda()
    decay = torch.full((H,), -0.05, device="cuda")
    o, last, _ = A.lin_attn_fwd(x, x, x, decay, final=True)
    want, wlast = R.forward(tail, tail, tail, decay[:3].cpu(), d ** -0.5)
    sums, slast = R.forward(tail, tail, tail, decay[:3].cpu(), d ** -0.5,
                            sums=True)
    _near(o[0, -40:, -3:], want, sums, 40, d, BF16, "o")
    _near(last[0, -3:], wlast, slast, 40, d, BF16, "state", F32)
    assert not o[0, :-40].any() and not o[0, -40:, :-3].any()
