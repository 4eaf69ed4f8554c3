"""The way to the experts and back on the GPU, against the 64-bit reference.

Tolerances.  Orders and copies are exact.  Sums of k terms: (k + 1) * 2^-24 of
the terms' absolute values, then half a step of the type (2^-8 or 2^-24).  dys:
one rounding of the product, then that of the type.  dw: D products and
additions in some order, (D + 1) * 2^-24 of the absolute values."""

import pytest
import torch

import adaln_fwd_amd as A
from tests import ref_experts as R

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def _choices(T, k, E, lost=0.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    e = torch.randint(0, E, (T, k), generator=g)
    if lost:
        out = torch.tensor([-1, E, E + 7, -(2 ** 31), 2 ** 31 - 1])
        pick = out[torch.randint(0, 5, (T, k), generator=g)]
        e = torch.where(torch.rand(T, k, generator=g) < lost, pick, e)
    return e


PLANS = [(1, 1, 1), (1, 2, 16), (5, 3, 7), (64, 1, 2), (1000, 8, 60),
         (4096, 2, 512), (8191, 1, 3), (8193, 1, 3), (5000, 4, 64),
         (70001, 3, 37), (33, 64, 512), (300000, 4, 129), (6144, 1, 3),
         (6145, 1, 3)]


@pytest.mark.parametrize("size", PLANS, ids=str)
@pytest.mark.parametrize("lost", [0.0, 0.3])
def test_plan(size, lost):
    T, k, E = size
    e = _choices(T, k, E, lost)
    offsets, slot = A.experts_plan(e.to(torch.int32).cuda(), E)
    wide = A.experts_plan(e.cuda(), E)
    assert torch.equal(offsets, wide[0]) and torch.equal(slot, wide[1])
    want = R.plan(e, E)
    assert torch.equal(offsets.cpu(), want[0])
    assert torch.equal(slot.cpu(), want[1])


def test_plans_of_one_kind_of_expert_and_of_none():
    for T in (700, 20000):
        for value in (0, 5, -1):
            e = torch.full((T, 2), value, dtype=torch.int32)
            offsets, slot = A.experts_plan(e.cuda(), 6)
            want = R.plan(e, 6)
            assert torch.equal(offsets.cpu(), want[0])
            assert torch.equal(slot.cpu(), want[1])
    # wide numbers are not cut to 32 bits
    e = torch.tensor([[2 ** 32 + 1, 1]])
    assert A.experts_plan(e.cuda(), 4)[1].tolist() == [[-1, 0]]
    offsets, slot = A.experts_plan(
        torch.zeros(0, 3, dtype=torch.int32, device="cuda"), 4)
    assert offsets.tolist() == [0] * 5 and slot.shape == (0, 3)


def _near(got, want, scale, k, dt, what):
    err = (got.double().cpu() - want).abs()
    allow = k * U * scale + HALF[dt] * (want.abs() + k * U * scale)
    assert not (err > allow).any(), (what, float((err - allow).max()))


ROWS = [(1, 1, 3, 8), (1, 2, 16, 1536), (7, 3, 5, 40), (200, 2, 8, 2056),
        (64, 8, 60, 264), (33, 4, 9, 8192), (3, 64, 100, 16), (500, 1, 4, 64),
        (6, 2, 4, 32768)]


@pytest.mark.parametrize("size", ROWS, ids=str)
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lost", [0.0, 0.4])
def test_rows(size, dt, lost):
    T, k, E, D = size
    if D > A.max_d(dt):
        D //= 2
    g = torch.Generator().manual_seed(D)
    e = _choices(T, k, E, lost)
    x, dy = (torch.randn(T, D, generator=g).to(dt) for _ in range(2))
    ys, dxs = (torch.randn(T * k, D, generator=g).to(dt) for _ in range(2))
    w = torch.randn(T, k, generator=g)
    offsets, slot = A.experts_plan(e.cuda(), E)
    sl, n = slot.cpu(), int(offsets[-1])
    # rows that no choice has: never read, left as they are
    ys[n:], dxs[n:] = float("nan"), float("inf")
    rest = torch.full((T * k, D), 7.0, dtype=dt)
    xs = A.experts_sort_fwd(x.cuda(), slot, xs=rest.cuda())
    assert torch.equal(xs.cpu(), R.sort_fwd(x, sl, rest))
    dx = A.experts_sort_bwd(dxs.cuda(), slot)
    one = torch.ones(T, k)
    _near(dx, R.sort_bwd(dxs, sl), R.join_fwd(dxs.abs(), sl, one), k + 1, dt,
          "dx")
    y = A.experts_join_fwd(ys.cuda(), slot, w.cuda())
    _near(y, R.join_fwd(ys, sl, w), R.join_fwd(ys.abs(), sl, w.abs()), k + 1,
          dt, "y")
    dys, dw = A.experts_join_bwd(dy.cuda(), ys.cuda(), slot, w.cuda(),
                                 dys=rest.cuda())
    wdys, wdw = R.join_bwd(dy, ys, sl, w, rest)
    _near(dys, wdys, wdys.abs(), 1, dt, "dys")
    _, sums = R.join_bwd(dy.abs(), ys.abs(), sl, w, rest)
    assert not ((dw.double().cpu() - wdw).abs() > (D + 1) * U * sums).any()


def test_infinite_rows_stay_with_their_tokens():
    """A row's infinities reach its own token only, also where others of its
    token's choices are dropped."""
    e = torch.tensor([[0, 1], [1, -1], [-1, -1]])
    _, slot = A.experts_plan(e.cuda(), 2)
    ys = torch.ones(6, 64, device="cuda")
    ys[slot[0, 1]] = float("inf")
    w = torch.tensor([[0.5, 0.5], [2.0, float("nan")],
                      [float("nan"), 1.0]]).cuda()
    y = A.experts_join_fwd(ys, slot, w)
    assert y[0].isinf().all()
    assert (y[1] == 2).all() and (y[2] == 0).all()


def test_slots_out_of_range_count_as_dropped():
    slot = torch.tensor([[0, 5], [-3, 2 ** 31 - 1], [4, 100]],
                        dtype=torch.int32, device="cuda")
    x = torch.arange(1.0, 4, device="cuda")[:, None].expand(3, 16).contiguous()
    xs = A.experts_sort_fwd(x, slot, xs=torch.zeros(6, 16, device="cuda"))
    assert xs[:, 0].tolist() == [1, 0, 0, 0, 3, 1]
    assert A.experts_sort_bwd(xs, slot)[:, 0].tolist() == [2, 0, 3]
    w = torch.ones(3, 2, device="cuda")
    assert A.experts_join_fwd(xs, slot, w)[:, 0].tolist() == [2, 0, 3]
    dys, dw = A.experts_join_bwd(x, xs, slot, w, dys=xs.clone())
    assert dys[:, 0].tolist() == [1, 0, 0, 0, 3, 1]
    assert dw.tolist() == [[16, 16], [0, 0], [144, 0]]


def test_in_place_streams_and_graphs():
    T, k, E, D = 3000, 2, 8, 520
    g = torch.Generator().manual_seed(3)
    e = _choices(T, k, E, 0.1).to(torch.int32).cuda()
    x, dy = (torch.randn(T, D, generator=g).to(BF16).cuda() for _ in range(2))
    ys = torch.randn(T * k, D, generator=g).to(BF16).cuda()
    w = torch.rand(T, k, generator=g).cuda()

    def run():
        offsets, slot = A.experts_plan(e, E)
        xs = A.experts_sort_fwd(x, slot, xs=torch.zeros_like(ys))
        y = A.experts_join_fwd(ys, slot, w)
        dys, dw = A.experts_join_bwd(dy, ys, slot, w, dys=torch.zeros_like(ys))
        dx = A.experts_sort_bwd(dys, slot)
        return offsets, slot, xs, y, dys, dw, dx

    want = run()
    # dys in the place of ys
    own = ys.clone()
    dys, dw = A.experts_join_bwd(dy, own, want[1], w, dys=own)
    n = int(want[0][-1])
    assert torch.equal(dys[:n], want[4][:n]) and torch.equal(dw, want[5])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    slot = A.experts_plan(e, E, stream=s)[1]
    y = A.experts_join_fwd(ys, slot, w, stream=s)
    s.synchronize()
    assert torch.equal(slot, want[1]) and torch.equal(y, want[3])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for i in range(3):
        e.copy_(_choices(T, k, E, 0.1, seed=i))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, run()):
            assert torch.equal(a, b)


def test_rows_past_32_bit_offsets():
    T, k, D = 140000, 2, 8192
    e = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    e[-1] = 1
    offsets, slot = A.experts_plan(e, 2)
    assert slot[-1].tolist() == [2 * T - 2, 2 * T - 1]
    x = torch.zeros(T, D, dtype=BF16, device="cuda")
    x[-1] = 3
    xs = A.experts_sort_fwd(x, slot)
    assert (xs[-2:] == 3).all() and not xs[-4:-2].any()
    dx = A.experts_sort_bwd(xs, slot)
    assert (dx[-1] == 6).all() and not dx[-2].any()


def test_refusals_of_the_binding_on_the_gpu():
    e = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    x = torch.zeros(4, 8, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    for E in (0, 513):
        with pytest.raises(A.AdalnError):
            A.experts_plan(e, E)
    with pytest.raises(A.AdalnError):
        A.experts_plan(torch.zeros(4, 65, dtype=torch.int32, device="cuda"), 2)
    with pytest.raises(ValueError):
        A.experts_plan(e.t(), 2)
    with pytest.raises(TypeError):
        A.experts_sort_fwd(x, e.long())
    with pytest.raises(ValueError):
        A.experts_sort_fwd(x[:3], e)
    with pytest.raises(ValueError):
        A.experts_sort_bwd(x, e)
    with pytest.raises(TypeError):
        A.experts_join_fwd(x.repeat(2, 1), e, w.double())
    with pytest.raises(ValueError):
        A.experts_join_bwd(x, x, e, w)
    big = torch.zeros(100000, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(A.AdalnError):
        A.experts_plan(big, 4, workspace=torch.empty(16, dtype=torch.uint8,
                                                     device="cuda"))
