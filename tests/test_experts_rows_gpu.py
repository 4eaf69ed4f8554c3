"""The rows to the experts and back, every one compared so that no missing number
passes: small calls, whose unowned rows hold NaN, and calls past the caches'
size, whose kernels access memory with the streaming hint, also in place.

Tolerances: those of test_experts_gpu.py.  Copies are exact.  Sums of k terms:
(k + 1) * 2^-24 of the terms' absolute values (and one for the weight), then half
a step of the type.  dys: one rounding of the product, then that of the type.  dw:
(D + 1) * 2^-24 of the absolute values."""

import pytest
import torch

import adaln_fwd_amd as A
from tests import near
from tests.test_experts_gpu import HALF, ROWS, U, _choices

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _check(T, k, E, D, dt, lost, rows=2000):
    """Everything on the GPU, in float64, some tokens at a time."""
    g = torch.Generator(device="cuda").manual_seed(D + T)

    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda").to(dt)

    x, dy, ys, dxs = normal(T, D), normal(T, D), normal(T * k, D), \
        normal(T * k, D)
    w = torch.randn(T, k, generator=g, device="cuda")
    offsets, slot = A.experts_plan(_choices(T, k, E, lost).cuda(), E)
    n = int(offsets[-1])
    assert n == T * k if lost == 0 else n < T * k
    # rows that no choice has: never read, left as they are
    ys[n:], dxs[n:] = float("nan"), float("inf")
    rest = torch.full((T * k, D), 7.0, dtype=dt, device="cuda")
    xs = A.experts_sort_fwd(x, slot, xs=rest.clone())
    dx = A.experts_sort_bwd(dxs, slot)
    y = A.experts_join_fwd(ys, slot, w)
    dys, dw = A.experts_join_bwd(dy, ys, slot, w, dys=rest.clone())
    own = ys.clone()
    dys2, dw2 = A.experts_join_bwd(dy, own, slot, w, dys=own)
    assert dys2 is own and torch.equal(own[:n], dys[:n])
    assert torch.equal(dw2, dw) and own[n:].isnan().all()
    assert (xs[n:] == 7).all() and (dys[n:] == 7).all()
    for a in range(0, T, rows):
        pick = slice(a, min(T, a + rows))
        at = slot[pick].long()
        on = at >= 0
        at = at.clamp(min=0)
        wide = (lambda t: torch.where(on[..., None], t[at].double(), 0.0))
        ws, one = w[pick].double(), dy[pick].double()[:, None]
        assert torch.equal(xs[at][on], x[pick][:, None].expand(-1, k, -1)[on])
        for got, rows_of, f, what in ((y, wide(ys), ws[..., None], "y"),
                                      (dx, wide(dxs), 1.0, "dx")):
            terms = rows_of * f
            slack = (k + 2) * U * terms.abs().sum(1)
            want = terms.sum(1)
            near.check(got[pick], want, slack + HALF[dt] * (want.abs() + slack),
                       what)
        want = ws[..., None] * one
        slack = U * want.abs()
        near.check(dys[at][on], want[on],
                   (slack + HALF[dt] * (want.abs() + slack))[on], "dys")
        terms = wide(ys) * one
        near.check(dw[pick], terms.sum(-1),
                   (D + 1) * U * terms.abs().sum(-1), "dw")


@pytest.mark.parametrize("size", ROWS, ids=str)
@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lost", [0.0, 0.4])
def test_small_calls(size, dt, lost):
    T, k, E, D = size
    if D > A.max_d(dt):
        D //= 2
    e = _choices(T, k, E, lost)
    if lost and ((e >= 0) & (e < E)).all():
        lost = 0.0                   # (so few choices that none was dropped)
    _check(T, k, E, D, dt, lost)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,k,row", [(24000, 3, 4112), (60000, 1, 1808)])
def test_past_the_caches(T, k, row, dt):
    """Every call moves more than 192 MiB, by rows that end inside a tile."""
    assert T * (1 + k) * row > 192 << 20
    print(f"[experts] {T} x {k}, {row} bytes a row", flush=True)
    _check(T, k, 9, row // (2 if dt == BF16 else 4), dt, 0.2)
