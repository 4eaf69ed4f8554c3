"""The way to the experts without a GPU: the reference against a hand example
and differences, and the refusals of the C entry points and of the binding."""

import pytest
import torch

import adaln_fwd_amd as A
from adaln_fwd_amd import _lib
from tests import ref_experts as R

P = 0x1000


def test_plan_by_hand():
    expert = torch.tensor([[2, 0], [2, -1], [0, 2], [9, 1]])
    offsets, slot = R.plan(expert, 3)
    assert offsets.tolist() == [0, 2, 3, 6]
    assert slot.tolist() == [[3, 0], [4, -1], [1, 5], [-1, 2]]


def test_reference_gradients_against_differences():
    g = torch.Generator().manual_seed(1)
    expert = torch.tensor([[2, 0], [2, -1], [0, 2], [1, 1]])
    _, slot = R.plan(expert, 3)
    x, dy = (torch.randn(4, 3, generator=g, dtype=torch.float64)
             for _ in range(2))
    ys, dxs = (torch.randn(8, 3, generator=g, dtype=torch.float64)
               for _ in range(2))
    w = torch.randn(4, 2, generator=g, dtype=torch.float64)
    zero = torch.zeros(8, 3, dtype=torch.float64)
    dx = R.sort_bwd(dxs, slot)
    dys, dw = R.join_bwd(dy, ys, slot, w, zero)
    for t, grad, loss in (
            (x, dx, lambda v: (R.sort_fwd(v, slot, zero) * dxs).sum()),
            (ys, dys, lambda v: (R.join_fwd(v, slot, w) * dy).sum()),
            (w, dw, lambda v: (R.join_fwd(ys, slot, v) * dy).sum())):
        for i in range(t.numel()):
            d = torch.zeros(t.numel(), dtype=torch.float64)
            d[i] = 1e-4
            d = d.reshape(t.shape)
            diff = (loss(t + d) - loss(t - d)) / 2e-4
            assert float(diff) == pytest.approx(float(grad.flatten()[i]),
                                                abs=1e-8)


def _no_gpu():
    if torch.cuda.device_count() > 0:
        pytest.skip("host-validation tests run only without a GPU")


def test_refusals_of_the_plan():
    _no_gpu()
    lib = A.load()

    def plan(e=P, wide=0, off=P, slot=P, ws=P, wb=1 << 30, T=5, k=2, E=4):
        return lib.adaln_experts_plan(e, wide, off, slot, ws, wb, T, k, E, None)

    assert plan(T=-1) == plan(k=0) == plan(k=65) == plan(E=0) == plan(E=513) \
        == plan(T=1 << 30, k=2) == _lib.ERR_INVALID
    assert plan(e=None) == plan(off=None) == plan(slot=None) \
        == _lib.ERR_INVALID
    assert plan(e=P + 4, wide=1) == plan(e=P + 2) == plan(off=P + 2) \
        == plan(slot=P + 1) == _lib.ERR_ALIGN
    need = lib.adaln_experts_plan_workspace_bytes(100000, 2, 4)
    assert need > 0
    assert plan(T=100000, wb=need - 1) == plan(T=100000, ws=None) \
        == _lib.ERR_WORKSPACE
    for bad in ((5, 2, 4), (100000, 0, 4), (100000, 2, 513), (-1, 2, 4)):
        assert lib.adaln_experts_plan_workspace_bytes(*bad) == 0


def test_refusals_of_the_rows():
    _no_gpu()
    lib = A.load()
    E = _lib
    for f in (lib.adaln_experts_sort_fwd, lib.adaln_experts_sort_bwd):
        assert f(None, P, P, 5, 2, 64, 1, None) == E.ERR_INVALID
        assert f(P, None, P, 5, 2, 64, 1, None) == E.ERR_INVALID
        assert f(P, P, None, 5, 2, 64, 1, None) == E.ERR_INVALID
        assert f(P, P, P, 5, 2, 60, 1, None) == E.ERR_ALIGN
        assert f(P + 8, P, P, 5, 2, 64, 1, None) == E.ERR_ALIGN
        assert f(P, P + 2, P, 5, 2, 64, 1, None) == E.ERR_ALIGN
        assert f(P, P, P, 5, 2, 64, 5, None) == E.ERR_DTYPE
        assert f(P, P, P, 5, 2, 32776, 1, None) == E.ERR_UNSUPPORTED
        assert f(P, P, P, 5, 65, 64, 1, None) == E.ERR_INVALID
        assert f(P, P, P, -5, 2, 64, 1, None) == E.ERR_INVALID
        assert f(None, None, None, 0, 2, 64, 1, None) == E.OK
    f = lib.adaln_experts_join_fwd
    assert f(P, P, None, P, 5, 2, 64, 1, None) == E.ERR_INVALID
    assert f(P, P, P + 2, P, 5, 2, 64, 1, None) == E.ERR_ALIGN
    assert f(None, None, None, None, 0, 2, 64, 1, None) == E.OK
    f = lib.adaln_experts_join_bwd
    for i in range(6):
        args = [P] * 6
        args[i] = None
        assert f(*args, 5, 2, 64, 1, None) == E.ERR_INVALID
    assert f(*[P] * 4, P + 8, P, 5, 2, 64, 1, None) == E.ERR_ALIGN
    assert f(*[None] * 6, 0, 2, 64, 1, None) == E.OK


def test_refusals_of_the_binding():
    e = torch.zeros(4, 2, dtype=torch.int32)
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        A.experts_plan(e, 3)
    with pytest.raises(TypeError, match="int32 or int64"):
        A.experts_plan(e.float(), 3)
    with pytest.raises(ValueError, match="\\[T, k\\]"):
        A.experts_plan(e[0], 3)
    with pytest.raises(ValueError, match="GPU tensor"):
        A.experts_sort_fwd(x, e)
    with pytest.raises(ValueError, match="slot \\[T, k\\]"):
        A.experts_sort_fwd(x, e[0])
    with pytest.raises(TypeError, match="dtype"):
        A.experts_join_fwd(x.half(), e, x)
