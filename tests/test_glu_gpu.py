"""The gated feed-forward on the GPU against float64.

Two kinds of test.  Whole numbers: inputs chosen so that every G is at least
32, where both activations are the identity to the last bit (exp(-32) is
below 2^-24), and so that dG, dU fit bfloat16 exactly; then every sum is an
exact float32 and each output is the exact integer rounded once, compared bit
for bit, so that not one term may be missing.  Real numbers, with tolerances:
an output is rounded once (eps/2 = 2^-8 of the value); a float32 sum of K
terms is within K * 2^-24 of the sum of their magnitudes; dG and dU are
rounded to bfloat16 inside (at most 2^-8 of each, independent: 8 standard
deviations of their sum are at most 8 * 2^-8 times the root of the sum of the
squared terms), or, up to 64 tokens, split into two bfloat16 (the second one
rounds at most 2^-8 of each, within 2^-8 of itself)."""

import pytest
import torch

import adaln_fwd_amd as A
from tests import ref_glu as R

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"[glu] {msg}", flush=True)


def _whole(M, D, F, seed=0):
    """G = 64 + a few, U a few, dh in -1, 0, 1."""
    g = torch.Generator().manual_seed(seed)

    def sparse(r, c, p):
        v = torch.randint(0, 2, (r, c), generator=g) * 2 - 1
        return v * (torch.rand(r, c, generator=g) < p)

    # about 8 (at most some 30) terms of +-1 in each G and U
    p = min(1.0, (8 / max(D - 1, 1)) ** 0.5)
    x, wg, wu = sparse(M, D, p), sparse(F, D, p), sparse(F, D, p)
    x[:, 0], wg[:, 0], wu[:, 0] = 8, 8, 0
    dh = torch.randint(-1, 2, (M, F), generator=g)
    return [t.to(torch.bfloat16) for t in (dh, x, wg, wu)]


SIZES = [
    # M, D, F
    (1, 64, 64), (1, 8, 8), (1, 1536, 4096), (2, 72, 136), (5, 1000, 200),
    (16, 512, 520), (17, 264, 1032), (33, 64, 8), (63, 128, 72),
    (64, 1536, 264), (65, 320, 328), (127, 128, 256), (128, 256, 128),
    (129, 136, 264), (200, 1000, 1480), (255, 64, 64), (257, 72, 2056),
    (777, 1000, 1480), (1024, 512, 512), (1030, 264, 4104), (3001, 8, 16),
    (2500, 1536, 2048), (4097, 520, 1288), (300, 5120, 640),
    (2048, 2048, 4096), (4100, 512, 2064), (4097, 1032, 2056),
    (1000, 2048, 2048),
]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_whole_numbers_exact(case, dt):
    M, D, F = SIZES[case]
    act = "gelu" if case % 2 else "silu"
    _say(f"whole {SIZES[case]} {act} {dt}")
    dh, x, wg, wu = [t.to(dt) for t in _whole(M, D, F, case)]
    dev = [t.cuda() for t in (dh, x, wg, wu)]
    # float64 products of the same integers, on the GPU's general matrix path
    dhf, xf, wgf, wuf = [t.double() for t in dev]
    G, U = xf @ wgf.t(), xf @ wuf.t()
    assert G.min() >= 32 and G.max() < 256 and U.abs().max() < 256
    h = A.glu_fwd(*dev[1:], act=act)
    assert torch.equal(h, (G * U).to(dt))
    h2, saved = A.glu_fwd(*dev[1:], act=act, save=True)
    assert torch.equal(h2, h)
    assert torch.equal(saved[0].double(), G)
    assert torch.equal(saved[1].double(), U)
    dG, dU = dhf * U, dhf * G
    want = [(dG @ wgf + dU @ wuf), dG.t() @ xf, dU.t() @ xf]
    for s in (saved, None):
        got = A.glu_bwd(*dev, s, act=act)
        for a, b, n in zip(got, want, ("dx", "dwg", "dwu")):
            # the sums are exact in float32 below 2^24
            assert b.abs().max() < 2 ** 24
            b = b.float().to(dt)
            assert torch.equal(a, b), (n, s is None, int((a != b).sum()))


def _real(M, D, F, seed, dt=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)

    def n(*s, std=1.0):
        return (torch.randn(*s, generator=g) * std).to(dt)

    return n(M, F, std=1e-2), n(M, D), n(F, D, std=2 * D ** -0.5), \
        n(F, D, std=D ** -0.5)


def _within(got, ref, tol, what):
    err = (got.double().cpu() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()),
                           float((err / tol.clamp_min(1e-300)).max()))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("size", [(1, 256, 520), (7, 1536, 1024),
                                  (130, 200, 392), (513, 768, 1096)])
def test_real_numbers(size, act, dt):
    _check_real(size, act, dt, split=False)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("size", [(1, 64, 64), (1, 256, 520), (2, 72, 2056),
                                  (4, 1536, 1024), (5, 264, 8200),
                                  (16, 512, 520), (17, 1000, 264),
                                  (33, 136, 1032), (63, 328, 16),
                                  (64, 768, 4104)])
def test_gradients_of_few_tokens_are_rounded_once(size, act):
    """Up to 64 tokens dG and dU have two parts: within 2^-16 of each."""
    _check_real(size, act, torch.bfloat16, split=True)


def _check_real(size, act, dt, split):
    M, D, F = size
    _say(f"real {size} {act} {dt}")
    dh, x, wg, wu = _real(M, D, F, M, dt)
    f = [t.double() for t in (dh, x, wg, wu)]
    ref_h, G, U = R.fwd(*f[1:], act)
    dx, dwg, dwu, dG, dU = R.bwd(*f, act)
    a, da = R.act(G, act)
    e24, e8 = 2.0 ** -24, torch.finfo(dt).eps / 2
    # float32 errors of G and U; of the exponential, 2^-23 (1 + |2 v|) with
    # |2 v| <= 2 |g|^3; of the rest of the activation, 16 roundings
    eG = (D + 2) * e24 * (f[1].abs() @ f[2].abs().t())
    eU = (D + 2) * e24 * (f[1].abs() @ f[3].abs().t())
    slope = 1.2
    eact = 16 * e24 * (1 + G.abs()) + 2 ** -23 * (1 + G.abs() ** 3) * \
        (1 / (1 + torch.exp(G.abs()))) * (1 + G.abs() ** 3)
    ea = slope * eG + eact
    eda = 1.5 * eG + eact
    h = A.glu_fwd(x.cuda(), wg.cuda(), wu.cuda(), act=act)
    _within(h, ref_h, e8 * ref_h.abs() + U.abs() * ea + a.abs() * eU + 1e-37,
            "h")
    edG = f[0].abs() * (U.abs() * eda + da.abs() * eU)
    edU = f[0].abs() * ea
    h, saved = A.glu_fwd(x.cuda(), wg.cuda(), wu.cuda(), act=act, save=True)
    for s in (saved, None):
        got = A.glu_bwd(dh.cuda(), x.cuda(), wg.cuda(), wu.cuda(), s, act=act)

        def tol(ref, L, Lerr, W, K):
            t = e8 * ref.abs() + 1e-37
            for l, le, w in zip(L, Lerr, W):
                t = t + le @ w.abs() + (K + 2) * e24 * (l.abs() @ w.abs())
                if split:  # each part adds K terms
                    t = t + (2.0 ** -16 + K * e24) * (l.abs() @ w.abs())
            if split:
                return t
            sq = sum((l ** 2) @ (w ** 2) for l, w in zip(L, W))
            return t + 8 * e8 * sq.sqrt()

        _within(got[0], dx, tol(dx, (dG, dU), (edG, edU), f[2:], 2 * F), "dx")
        _within(got[1], dwg, tol(dwg, (dG.t(),), (edG.t(),), f[1:2], M), "dwg")
        _within(got[2], dwu, tol(dwu, (dU.t(),), (edU.t(),), f[1:2], M), "dwu")


def test_ends_of_the_activations():
    """Where the logistic function saturates, and around zero."""
    _say("activation ends")
    g = torch.tensor([0.0, -0.0, 1e-30, 1.0, -1.0, -5.0, -9.0, 30.0, -30.0,
                      -88.0, -200.0, 200.0, 1e4, -1e4, 3e38, -3e38])
    M = g.numel()
    x = torch.zeros(M, 8, dtype=torch.bfloat16)
    x[:, 0] = g
    x[:, 1] = 1
    wg = torch.zeros(8, 8, dtype=torch.bfloat16)
    wu = torch.zeros(8, 8, dtype=torch.bfloat16)
    wg[:, 0], wu[:, 1] = 1, 1
    dh = torch.ones(M, 8, dtype=torch.bfloat16)
    for act in ("silu", "gelu"):
        h, saved = A.glu_fwd(x.cuda(), wg.cuda(), wu.cuda(), act=act, save=True)
        gd = x[:, :1].double()
        a, da = R.act(gd.clamp(-1e6, 1e6), act)
        a = torch.where(gd > 1e5, gd, a)
        # exp(-x) of float32 is off by up to (1 + |x|) 2^-23 of itself
        small = a.abs() * 2 ** -8 + a.abs() * (1 + 2 * gd.abs() ** 3).clamp_max(
            300) * 2 ** -23 + 1e-37
        _within(h[:, :1], a, small, act)
        fine = gd[:, 0].abs() <= 1e4
        dx = A.glu_bwd(dh.cuda(), x.cuda(), wg.cuda(), wu.cuda(), saved,
                       act=act)[0]
        assert torch.isfinite(dx[fine.cuda()]).all()
        # dx[:, 0] = sum over 8 columns of act'(g), [:, 1] of act(g)
        _within(dx[fine.cuda()][:, 0], 8 * da[fine, 0],
                8 * (2 ** -6.9 * da[fine, 0].abs() + 2 ** -20), act + "'")


def test_rows_past_the_end_and_other_rows_are_left_alone():
    """Outputs inside larger buffers: only their own elements are written;
    a token of infinities spoils only its own rows of h and dx."""
    _say("guards")
    M, D, F = 130, 136, 200
    dh, x, wg, wu = [t.cuda() for t in _real(M, D, F, 3)]

    def room(*s):
        n = 1
        for v in s:
            n *= v
        r = torch.full((n + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
        return r, r[256:256 + n].view(*s)

    r1, h = room(M, F)
    r2, dx = room(M, D)
    r3, dwg = room(F, D)
    r4, dwu = room(F, D)
    need = A.glu_bwd_workspace_bytes(M, D, F)
    ws = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    A.glu_fwd(x, wg, wu, h=h)
    A.glu_bwd(dh, x, wg, wu, dx=dx, dwg=dwg, dwu=dwu,
              workspace=ws[256:256 + need])
    for r in (r1, r2, r3, r4):
        assert (r[:256] == 7).all() and (r[-256:] == 7).all()
    assert (ws[:256] == 77).all() and (ws[-256:] == 77).all()
    y = x.clone()
    y[40] = float("inf")
    y[99, 3] = float("nan")
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[40] = keep[99] = False
    h2 = A.glu_fwd(y, wg, wu)
    dx2 = A.glu_bwd(dh, y, wg, wu)[0]
    assert torch.equal(h2[keep], h[keep]) and h2[99].isnan().all()
    assert torch.equal(dx2[keep], dx[keep])


def test_3d_empty_stream_repeat():
    _say("shapes, empty, stream, repeat")
    dh, x, wg, wu = [t.cuda() for t in _real(600, 256, 264, 9)]
    h, saved = A.glu_fwd(x, wg, wu, save=True)
    h3 = A.glu_fwd(x.view(3, 200, 256), wg, wu)
    assert h3.shape == (3, 200, 264) and torch.equal(h3.view(600, 264), h)
    want = A.glu_bwd(dh, x, wg, wu, saved)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = A.glu_bwd(dh.view(3, 200, 264), x.view(3, 200, 256), wg, wu, saved,
                    stream=s)
    s.synchronize()
    assert torch.equal(got[0].view(600, 256), want[0])
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    empty = x[:0]
    assert A.glu_fwd(empty, wg, wu).shape == (0, 264)
    dx, dwg, dwu = A.glu_bwd(dh[:0], empty, wg, wu)
    assert dx.shape == (0, 256) and not dwg.any() and not dwu.any()


def test_in_a_graph():
    _say("captured and replayed")
    dh, x, wg, wu = [t.cuda() for t in _real(300, 512, 776, 4)]

    def run():
        h, saved = A.glu_fwd(x, wg, wu, save=True)
        return [h, *A.glu_bwd(dh, x, wg, wu, saved),
                *A.glu_bwd(dh, x, wg, wu)]

    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run()
    keep = x.clone()
    for i in range(3):
        for t in outs:
            t.fill_(float("nan"))
        x.copy_(keep * 2 if i == 1 else keep)
        other = [t.clone() for t in run()] if i == 1 else want
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, other):
            assert torch.equal(a, b), i


def test_two_streams_at_once():
    """Calls on two streams share nothing but their inputs."""
    _say("two streams")
    dh, x, wg, wu = [t.cuda() for t in _real(500, 512, 776, 6)]

    def run(x, **kw):
        h, saved = A.glu_fwd(x, wg, wu, save=True, **kw)
        return [h, *A.glu_bwd(dh, x, wg, wu, saved, **kw)]

    y = x.flip(0).contiguous()
    want = [run(x), run(y)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for i, v in enumerate((x, y)):
            got[i].append(run(v, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            for a, b in zip(r, want[i]):
                assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """More than 2^32 hidden elements: the last tokens' outputs, and the
    weights' gradients of the last hidden features, exactly."""
    M, D, F = 270000, 64, 16384
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of device memory")
    _say(f"M*F = {M * F}")
    _, x, wg, wu = [t.cuda() for t in _whole(1000, D, F, 5)]
    x = x.repeat(M // 1000, 1)
    # one in four is not zero: the largest sums, of dh * 64 * 8 over 1000
    # tokens 270 times, have a deviation of 2.2e6, an eighth of 2^24
    g = torch.Generator().manual_seed(6)
    dh = torch.randint(-1, 2, (1000, F), generator=g)
    dh = (dh * (torch.rand(1000, F, generator=g) < 0.375)).cuda()
    dh = dh.to(torch.bfloat16)
    dh = dh.repeat(M // 1000, 1)
    h = A.glu_fwd(x, wg, wu)
    dx, dwg, dwu = A.glu_bwd(dh, x, wg, wu)
    last = slice(M - 1000, M)
    xf, wgf, wuf, df = [t.double() for t in (x[last], wg, wu, dh[last])]
    G, U = xf @ wgf.t(), xf @ wuf.t()
    assert torch.equal(h[last], (G * U).to(torch.bfloat16))
    assert torch.equal(h[:1000], h[last])
    want = (df * U) @ wgf + (df * G) @ wuf
    assert torch.equal(dx[last], want.float().to(torch.bfloat16))
    assert torch.equal(dx[:1000], dx[last])
    # every thousand tokens are alike: 270 times the sums of one thousand
    for got, l in ((dwg, df * U), (dwu, df * G)):
        want = 270 * (l.t() @ xf)
        assert want.abs().max() < 2 ** 24
        assert torch.equal(got, want.float().to(torch.bfloat16))
