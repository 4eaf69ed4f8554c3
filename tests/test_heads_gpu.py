"""Rotary positions and query/key norms on the GPU against the float64
reference.

Tolerances.  A kernel's value is a float32 result rounded once to its type, so
|err| <= eps_T / 2 * |ref| + C * scale: `scale` bounds the terms that are
added (the largest magnitudes of the head, after the norm's factors) and C
counts the float32 roundings on the way, each 2^-24 of such a term: cos and
sin are within 2^-22 (phase 2^-32 turns, polynomial and its roundings), the
products and the norm's factors another dozen roundings, the row sums of up to
512 terms at most 32 + 6 roundings deep; C = 64 * 2^-24 covers them.  The
reference's own angle, a float64 product, is off by up to 2^-53 of the angle
per axis, which adds `4 * 2^-53 * max angle`."""

import numpy as np
import pytest
import torch

import adaln_fwd_amd as A
from tests import ref_heads as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _say(msg):
    print(f"[heads] {msg}", flush=True)


def _tol(ref, scale, dtype, angle=0.0):
    return (torch.finfo(dtype).eps / 2 * ref.abs()
            + (64 * 2.0 ** -24 + 4 * 2.0 ** -53 * angle) * scale + 1e-37)


def _close(got, ref, scale, what, angle=0.0):
    got = got.detach()
    err = (got.double().cpu() - ref).abs()
    # tiny results: bfloat16 and float32 share the smallest normal, 2^-126
    bad = ~(err <= _tol(ref, scale, got.dtype, angle))
    assert not bad.any(), (what, int(bad.sum()), float(err[bad].max()))


def _rows_max(x):
    return x.abs().amax(-1, keepdim=True)


def _inputs(B, N, Hq, Hk, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]

    def n(*s, std=1.0):
        return (torch.randn(*s, generator=g) * std).to(dt)

    return dict(q=n(B, N, Hq, d) + 0.5, k=n(B, N, Hk, d, std=3.0),
                dq=n(B, N, Hq, d, std=1e-2), dk=n(B, N, Hk, d),
                wq=1 + n(d, std=0.1), wk=n(d))


def _freqs(pairs, axes):
    per = pairs // axes
    return A.rope_freqs([pairs - per * (axes - 1)] + [per] * (axes - 1))


CASES = [
    # B, N, Hq, Hk, d, pairs, axes, layout, dtype
    (1, 1, 12, 12, 128, 64, 3, "interleaved", "bf16"),
    (1, 1, 1, 1, 64, 32, 1, "half", "f32"),
    (2, 7, 3, 1, 64, 32, 2, "half", "bf16"),
    (3, 17, 5, 5, 128, 64, 3, "half", "bf16"),
    (2, 333, 12, 2, 128, 64, 3, "interleaved", "bf16"),
    (1, 1025, 4, 4, 96, 32, 2, "half", "bf16"),         # part rotated
    (1, 50, 3, 2, 72, 31, 3, "interleaved", "bf16"),    # 9 vectors, odd pairs
    (2, 19, 2, 3, 40, 20, 2, "interleaved", "bf16"),    # 5 vectors
    (1, 33, 7, 1, 8, 4, 1, "interleaved", "bf16"),      # one vector
    (1, 33, 7, 1, 16, 8, 2, "half", "bf16"),
    (1, 40, 2, 2, 256, 128, 3, "half", "bf16"),
    (1, 9, 2, 1, 512, 192, 2, "interleaved", "bf16"),
    (1, 9, 2, 1, 512, 96, 4, "half", "bf16"),
    (2, 65, 3, 2, 128, 64, 3, "interleaved", "f32"),
    (1, 65, 3, 2, 128, 64, 1, "half", "f32"),
    (2, 31, 2, 2, 4, 2, 1, "interleaved", "f32"),
    (2, 31, 2, 2, 12, 4, 1, "half", "f32"),             # 3 vectors
    (1, 21, 5, 3, 68, 34, 2, "interleaved", "f32"),     # 17 vectors
    (1, 5, 2, 1, 512, 96, 4, "half", "f32"),
    (1, 5, 2, 1, 260, 128, 3, "interleaved", "f32"),    # 65 vectors
    (4, 4100, 1, 1, 32, 16, 2, "interleaved", "f32"),   # blocks of 16 tokens
    (1, 20, 64, 16, 32, 16, 2, "half", "bf16"),
    (1, 16391, 2, 1, 64, 32, 3, "interleaved", "bf16"),  # many per workgroup
    # the widest heads in blocks as long as the LDS admits
    (1, 20001, 2, 1, 512, 192, 2, "interleaved", "bf16"),
    (1, 20001, 1, 1, 512, 96, 4, "half", "f32"),
    (500, 1, 3, 1, 32, 16, 1, "half", "bf16"),           # a batch of tokens
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_all_four_passes(case):
    B, N, Hq, Hk, d, pairs, axes, layout, dtype = CASES[case]
    _say(f"case {case}: {CASES[case]}")
    h = _inputs(B, N, Hq, Hk, d, dtype, seed=case)
    g = torch.Generator().manual_seed(case)
    pos = torch.randint(-1000, 100000, (N, axes), generator=g,
                        dtype=torch.int32)
    freqs = _freqs(pairs, axes)
    ang = R.angles(pos, freqs)
    top = float(ang.abs().max())
    x = {n: v.cuda() for n, v in h.items()}
    f = {n: v.double() for n, v in h.items()}
    p = pos.cuda()

    for got, n in zip(A.rope_fwd(x["q"], x["k"], p, freqs, layout=layout),
                      "qk"):
        _close(got, R.rotate(f[n], ang, layout), _rows_max(f[n]), "rope " + n,
               top)
    for got, n in zip(A.rope_bwd(x["dq"], x["dk"], p, freqs, layout=layout),
                      ("dq", "dk")):
        _close(got, R.rotate(f[n], ang, layout, -1.0), _rows_max(f[n]),
               "rope " + n, top)
    out = A.qk_norm_rope_fwd(x["q"], x["k"], x["wq"], x["wk"], p, freqs,
                             layout=layout)
    for got, n in zip(out, "qk"):
        ref = R.qk_fwd(f[n], f["w" + n], ang, layout)
        _close(got, ref, _rows_max(ref), "norm " + n, top)
    dq, dk, dwq, dwk = A.qk_norm_rope_bwd(
        x["dq"], x["dk"], x["q"], x["k"], x["wq"], x["wk"], p, freqs,
        layout=layout)
    for got, dw, n, H in ((dq, dwq, "q", Hq), (dk, dwk, "k", Hk)):
        dx, rw, terms = R.qk_bwd(f["d" + n], f[n], f["w" + n], ang, layout)
        r = 1 / torch.sqrt((f[n] ** 2).mean(-1, keepdim=True) + R.EPS)
        scale = r * _rows_max(f["d" + n]) * 2 * f["w" + n].abs().max() \
            * (1 + _rows_max(f[n] * r))
        _close(got, dx, scale, "norm d" + n, top)
        # a lane adds its own rows one after another (at most a quarter of
        # them), then at most 64 sums of sums
        depth = B * N * H / 4 + 64
        err = (dw.double().cpu() - rw).abs()
        tol = (depth + 64) * 2.0 ** -24 * terms + 8 * 2.0 ** -53 * top * terms
        assert (err <= tol + 1e-37).all(), ("dw" + n, float((err / terms).max()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_positions(dtype):
    _say(f"far positions {dtype}")
    ends = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30, 12345678, 999983]
    pos = torch.tensor([[a, b] for a in ends for b in ends[:4]],
                       dtype=torch.int32)
    # frequencies that float64 products of such positions hold exactly enough:
    # multiples of 2^-20, so the reference's angles are exact
    freqs = np.round(_freqs(32, 2) * 2 ** 20) / 2 ** 20
    h = _inputs(1, pos.shape[0], 2, 1, 64, dtype)
    q, k = A.rope_fwd(h["q"].cuda(), h["k"].cuda(), pos.cuda(), freqs)
    # the reference reduces the angle with the remainder of exact integers
    ang = R.angles(pos, freqs)
    ang = torch.fmod(ang, 2 * torch.pi)
    # 2^31 * 2^-53 of the rounding of 2 pi itself, over 2^31 / 6.3 turns
    for got, n in ((q, "q"), (k, "k")):
        f = h[n].double()
        _close(got, R.rotate(f, ang, "interleaved"), _rows_max(f), n,
               angle=2.0 ** 32)


def test_batched_positions_and_3d():
    _say("positions of each sample; packed tokens")
    h = _inputs(3, 50, 2, 1, 64, "f32")
    g = torch.Generator().manual_seed(1)
    pos = torch.randint(0, 500, (3, 50, 2), generator=g, dtype=torch.int32)
    freqs = _freqs(32, 2)
    q, k = A.rope_fwd(h["q"].cuda(), h["k"].cuda(), pos.cuda(), freqs)
    _close(q, R.rotate(h["q"].double(), R.angles(pos, freqs), "interleaved"),
           _rows_max(h["q"].double()), "batched", 1000)
    q3, k3 = A.rope_fwd(h["q"].cuda().flatten(0, 1),
                        h["k"].cuda().flatten(0, 1),
                        pos.cuda().flatten(0, 1), freqs)
    assert torch.equal(q3, q.flatten(0, 1)) and torch.equal(k3, k.flatten(0, 1))


def _everything(q, k, dq, dk, wq, wk, pos, freqs, layout, out=None, **kw):
    """The outputs of all four entry points."""
    a = A.rope_fwd(q, k, pos, freqs, layout=layout, **kw)
    b = A.rope_bwd(dq, dk, pos, freqs, layout=layout, **kw)
    c = A.qk_norm_rope_fwd(q, k, wq, wk, pos, freqs, layout=layout, **kw)
    e = A.qk_norm_rope_bwd(dq, dk, q, k, wq, wk, pos, freqs, layout=layout,
                           **kw)
    return [*a, *b, *c, *e]


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_views_equal_contiguous(layout):
    _say(f"views {layout}")
    B, N, Hq, Hk, d = 2, 75, 4, 2, 64
    h = _inputs(B, N, Hq, Hk, d, "bf16")
    x = {n: v.cuda() for n, v in h.items()}
    pos = torch.arange(2 * N, dtype=torch.int32).reshape(N, 2).cuda()
    freqs = _freqs(32, 2)
    args = [x[n] for n in ("q", "k", "dq", "dk", "wq", "wk")]
    want = _everything(*args, pos, freqs, layout)
    # slices of one projection's output, and head-major gradients
    qkv = torch.full((B, N, (Hq + 2 * Hk) * d), 9.0, dtype=torch.bfloat16,
                     device="cuda")
    q = qkv[..., :Hq * d].unflatten(-1, (Hq, d))
    k = qkv[..., Hq * d:(Hq + Hk) * d].unflatten(-1, (Hk, d))
    q.copy_(x["q"])
    k.copy_(x["k"])
    dq = x["dq"].transpose(1, 2).contiguous().transpose(1, 2)
    dk = x["dk"].transpose(1, 2).contiguous().transpose(1, 2)
    got = _everything(q, k, dq, dk, x["wq"], x["wk"], pos, freqs, layout)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # outputs into views: everything around them stays as it was
    room = torch.full((B, Hq + 1, N + 3, d + 8), 5.0, dtype=torch.bfloat16,
                      device="cuda")
    qo = room[:, :Hq, 1:N + 1, :d].transpose(1, 2)
    a, b = A.qk_norm_rope_fwd(q, k, x["wq"], x["wk"], pos, freqs,
                              layout=layout, q_out=qo)
    assert a is qo and torch.equal(a, want[4]) and torch.equal(b, want[5])
    qo.fill_(5.0)
    assert (room == 5.0).all()
    # in place, inside the projection's output
    A.rope_fwd(q, k, pos, freqs, layout=layout, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert (qkv[..., (Hq + Hk) * d:] == 9.0).all()


def test_repeated_input_and_single_tensors():
    _say("expanded heads; one tensor alone")
    h = _inputs(2, 30, 4, 1, 64, "f32")
    x = {n: v.cuda() for n, v in h.items()}
    pos = torch.arange(30, dtype=torch.int32).reshape(30, 1).cuda()
    freqs = _freqs(32, 1)
    shared = x["k"].expand(2, 30, 4, 64)
    a, _ = A.rope_fwd(shared, None, pos, freqs)
    _, b = A.rope_fwd(None, shared.contiguous(), pos, freqs)
    assert torch.equal(a, b)
    full = _everything(*[x[n] for n in ("q", "k", "dq", "dk", "wq", "wk")],
                       pos, freqs, "half")
    dq, none, dwq, none2 = A.qk_norm_rope_bwd(
        x["dq"], None, x["q"], None, x["wq"], None, pos, freqs, layout="half")
    assert none is None and none2 is None
    assert torch.equal(dq, full[6]) and torch.equal(dwq, full[8])
    none, dk, none2, dwk = A.qk_norm_rope_bwd(
        None, x["dk"], None, x["k"], None, x["wk"], pos, freqs, layout="half")
    # (dw's order of summation goes by the call's sizes, and these two calls
    # have different ones: each sum of 60 terms is within 60 * 2^-24 of the sum
    # of their magnitudes, plus the products' three roundings of each term)
    assert torch.equal(dk, full[7])
    _, _, terms = R.qk_bwd(h["dk"].double(), h["k"].double(),
                           h["wk"].double(), R.angles(pos.cpu(), freqs), "half")
    assert ((dwk - full[9]).double().cpu().abs()
            <= 2 * (60 + 3) * 2.0 ** -24 * terms).all()
    with pytest.raises(ValueError):
        A.rope_fwd(x["q"], None, pos, freqs, k_out=x["q"])


def test_output_that_overlaps_itself_is_refused():
    q = torch.zeros(2, 30, 4, 64, device="cuda")
    pos = torch.zeros(30, 1, dtype=torch.int32, device="cuda")
    room = torch.zeros(2, 30, 1, 64, device="cuda").expand(2, 30, 4, 64)
    with pytest.raises(A.AdalnError, match="overlap"):
        A.rope_fwd(q, None, pos, _freqs(32, 1), q_out=room)


def test_non_finite_rows_stay_in_their_heads():
    _say("zeros, infinities and NaN")
    h = _inputs(1, 40, 3, 2, 64, "f32")
    x = {n: v.cuda() for n, v in h.items()}
    pos = torch.arange(40, dtype=torch.int32).reshape(40, 1).cuda()
    freqs = _freqs(32, 1)
    args = [x[n] for n in ("dq", "dk", "wq", "wk")]
    clean = _everything(x["q"], x["k"], *args, pos, freqs, "interleaved")
    q = x["q"].clone()
    q[0, 3, 1] = float("inf")
    q[0, 5, 2, 7] = float("nan")
    q[0, 7, 0] = 0
    got = _everything(q, x["k"], *args, pos, freqs, "interleaved")
    keep = torch.ones(1, 40, 3, dtype=torch.bool, device="cuda")
    keep[0, 3, 1] = keep[0, 5, 2] = keep[0, 7, 0] = False
    for i in (0, 4, 6):
        assert torch.equal(got[i][keep], clean[i][keep])
        assert got[i][0, 5, 2].isnan().any()
    for i in (1, 5, 7, 9):
        assert torch.equal(got[i], clean[i])
    assert (got[4][0, 7, 0] == 0).all()
    dx, _, _ = R.qk_bwd(h["dq"].double(), q.double().cpu(), h["wq"].double(),
                        R.angles(pos.cpu(), freqs), "interleaved")
    # a head of zeros: r = 1 / sqrt(eps), dx = r * g
    np.testing.assert_allclose(got[6][0, 7, 0].cpu(), dx[0, 7, 0], rtol=1e-5,
                               atol=1e-5 * float(dx[0, 7, 0].abs().max()))


def test_no_heads():
    """A tensor without heads next to one with: its weight's gradient is 0."""
    h = _inputs(1, 20, 2, 1, 64, "f32")
    x = {n: v.cuda() for n, v in h.items()}
    pos = torch.arange(20, dtype=torch.int32).reshape(-1, 1).cuda()
    f = _freqs(32, 1)
    none = x["q"][:, :, :0]
    dq, dk, dwq, dwk = A.qk_norm_rope_bwd(none, x["dk"], none, x["k"],
                                          x["wq"], x["wk"], pos, f)
    assert dq.shape == none.shape and not dwq.any()
    want = A.qk_norm_rope_bwd(None, x["dk"], None, x["k"], None, x["wk"], pos,
                              f)
    assert torch.equal(dk, want[1]) and torch.equal(dwk, want[3])
    q, k = A.rope_fwd(none, none, pos, f)
    assert q.shape == none.shape


def test_empty():
    pos = torch.zeros(0, 1, dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 0, 3, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    f = _freqs(32, 1)
    assert A.rope_fwd(q, q, pos, f)[0].shape == q.shape
    dq, dk, dwq, dwk = A.qk_norm_rope_bwd(q, q, q, q, w, w, pos, f)
    assert dq.shape == q.shape and not dwq.any() and not dwk.any()


def test_offsets_past_32_bits():
    """Tokens 2^31 elements apart, and heads (4 GiB each way)."""
    _say("far strides")
    far = 2 ** 31 + 64
    room = torch.empty(far + 4096, dtype=torch.bfloat16, device="cuda")
    h = _inputs(1, 2, 2, 1, 64, "bf16")
    pos = torch.tensor([[3], [4]], dtype=torch.int32, device="cuda")
    f = _freqs(32, 1)
    want, _ = A.rope_fwd(h["q"].cuda(), None, pos, f)
    for strides in ((1, far, 64, 1), (1, 64, far, 1)):
        q = room.as_strided((1, 2, 2, 64), strides)
        q.copy_(h["q"])
        got, _ = A.rope_fwd(q, None, pos, f)
        assert torch.equal(got, want)
        A.rope_fwd(q, None, pos, f, q_out=q)
        assert torch.equal(q, want)


def test_stream_and_repeat():
    _say("another stream; bitwise repeatable")
    h = _inputs(4, 1001, 6, 3, 128, "bf16")
    x = [h[n].cuda() for n in ("q", "k", "dq", "dk", "wq", "wk")]
    pos = torch.arange(1001, dtype=torch.int32).reshape(-1, 1).cuda()
    f = _freqs(64, 1)
    want = _everything(*x, pos, f, "half")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = _everything(*x, pos, f, "half", stream=s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_in_a_graph():
    _say("captured and replayed")
    h = _inputs(2, 700, 4, 2, 128, "bf16")
    x = [h[n].cuda() for n in ("q", "k", "dq", "dk", "wq", "wk")]
    pos = torch.arange(700, dtype=torch.int32).reshape(-1, 1).cuda()
    f = _freqs(64, 1)
    want = [t.clone() for t in _everything(*x, pos, f, "half")]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = _everything(*x, pos, f, "half")
    keep = [t.clone() for t in x]
    for i in range(3):
        for t in outs:
            t.fill_(float("nan"))
        for t, v in zip(x, keep):       # eager work between replays
            t.copy_(v if i != 1 else v * 2)
        if i == 1:
            f[:] = f                    # the table is read at capture only
            other = [t.clone() for t in _everything(*x, pos, f, "half")]
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, other if i == 1 else want):
            assert torch.equal(a, b), i


def test_backward_in_place():
    """dq written over dq_out, dk over k."""
    _say("backward in place")
    h = _inputs(2, 501, 3, 2, 72, "bf16")
    x = {n: v.cuda() for n, v in h.items()}
    pos = torch.arange(501, dtype=torch.int32).reshape(-1, 1).cuda()
    f = _freqs(36, 1)
    args = [x[n] for n in ("dq", "dk", "q", "k", "wq", "wk")]
    want = A.qk_norm_rope_bwd(*args, pos, f)
    got = A.qk_norm_rope_bwd(*args, pos, f, dq=x["dq"], dk=x["k"])
    assert got[0] is x["dq"] and got[1] is x["k"]
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_more_frequencies_than_the_small_form_holds():
    """Pairs turned by several axes at once, and more than 64 pairs: the same
    angles whichever way the table travels."""
    _say("dense table")
    h = _inputs(1, 60, 2, 1, 128, "f32")
    q, k = h["q"].cuda(), h["k"].cuda()
    g = torch.Generator().manual_seed(8)
    pos = torch.randint(0, 64, (60, 3), generator=g, dtype=torch.int32)
    dense = torch.rand(3, 64, generator=g, dtype=torch.float64).numpy() - 0.5
    got = A.rope_fwd(q, k, pos.cuda(), dense)
    ang = R.angles(pos, dense)
    for a, n in zip(got, "qk"):
        f = h[n].double()
        _close(a, R.rotate(f, ang, "interleaved"), _rows_max(f), n, 200)
    # one axis split over two columns of positions: the sum is the same angle
    one = _freqs(64, 1)
    two = np.concatenate([one, one])
    a = A.rope_fwd(q, k, pos[:, :1].contiguous().cuda() * 2, one)
    b = A.rope_fwd(q, k, pos[:, :1].expand(60, 2).contiguous().cuda(), two)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_streams_at_once():
    """Calls on two streams share nothing."""
    _say("two streams")
    h = _inputs(1, 3000, 8, 8, 128, "bf16")
    x = [h[n].cuda() for n in ("q", "k", "dq", "dk", "wq", "wk")]
    y = [t.flip(0, 1).contiguous() if t.dim() == 4 else t for t in x]
    pos = torch.arange(3000, dtype=torch.int32).reshape(-1, 1).cuda()
    f = _freqs(64, 1)
    want = [_everything(*v, pos, f, "half") for v in (x, y)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for i, v in enumerate((x, y)):
            got[i].append(_everything(*v, pos, f, "half", stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            for a, b in zip(run, want[i]):
                assert torch.equal(a, b)
