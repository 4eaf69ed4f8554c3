"""The gated feed-forward without a GPU: the float64 reference against
differences, and the refusals of the C entry points and of the binding."""

import pytest
import torch

import adaln_fwd_amd as A
from adaln_fwd_amd import _lib
from tests import ref_glu as R


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_reference_gradient_against_differences(act):
    g = torch.Generator().manual_seed(5)
    x, wg, wu, dh = (torch.randn(*s, generator=g, dtype=torch.float64)
                     for s in ((3, 4), (5, 4), (5, 4), (3, 5)))
    grads = R.bwd(dh, x, wg, wu, act)[:3]
    h = 1e-6
    for which, grad in enumerate(grads):
        for i in range(grad.numel()):
            args = [x, wg, wu]
            d = torch.zeros(grad.numel(), dtype=torch.float64)
            d[i] = h
            d = d.reshape(grad.shape)
            lo, hi = list(args), list(args)
            lo[which], hi[which] = args[which] - d, args[which] + d
            num = float(((R.fwd(*hi, act)[0] - R.fwd(*lo, act)[0]) * dh).sum())
            assert num / (2 * h) == pytest.approx(float(grad.flatten()[i]),
                                                  abs=1e-7)


P = 0x1000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.device_count() > 0:
        pytest.skip("host-validation tests run only without a GPU")
    return A.load()


@pytest.mark.parametrize("M,D,F,act,dt,code", [
    (4, 64, 64, 0, 2, _lib.ERR_DTYPE),
    (4, 64, 64, 0, 9, _lib.ERR_DTYPE),
    (4, 64, 64, 2, 1, _lib.ERR_INVALID),
    (-1, 64, 64, 0, 1, _lib.ERR_INVALID),
    (4, 0, 64, 0, 1, _lib.ERR_INVALID),
    (4, 64, 0, 0, 1, _lib.ERR_INVALID),
    (4, 60, 64, 0, 1, _lib.ERR_ALIGN),
    (4, 64, 68, 0, 1, _lib.ERR_ALIGN),
    (4, 65544, 64, 0, 1, _lib.ERR_UNSUPPORTED),
    (4, 64, 262152, 0, 1, _lib.ERR_UNSUPPORTED),
    ((1 << 24) + 1, 64, 64, 0, 1, _lib.ERR_UNSUPPORTED),
])
def test_refused_sizes(lib, M, D, F, act, dt, code):
    assert lib.adaln_glu_fwd(P, P, P, P, None, M, D, F, act, dt, None) == code
    assert lib.adaln_glu_bwd(P, P, P, P, None, P, P, P, P, 1 << 50, M, D, F,
                             act, dt, None) == code
    assert lib.adaln_last_error()
    if code != _lib.ERR_INVALID or act == 0:
        assert lib.adaln_glu_bwd_workspace_bytes(M, D, F, dt) == 0


def test_refused_pointers(lib):
    size = (4, 64, 64, 0, 1, None)
    for bad, code in ((None, _lib.ERR_INVALID), (P + 8, _lib.ERR_ALIGN)):
        for i in range(4):
            a = [P] * 4
            a[i] = bad
            assert lib.adaln_glu_fwd(*a, None, *size) == code
        need = lib.adaln_glu_bwd_workspace_bytes(4, 64, 64, 1)
        for i in (0, 1, 2, 3, 5, 6, 7):
            a = [P] * 8
            a[i] = bad
            assert lib.adaln_glu_bwd(*a, P, need, *size) == code
    assert lib.adaln_glu_fwd(P, P, P, P, P + 4, *size) == _lib.ERR_ALIGN
    assert need >= 2 * 4 * 64 * 2
    for ws, n, code in ((None, need, _lib.ERR_WORKSPACE),
                        (P, need - 1, _lib.ERR_WORKSPACE),
                        (P + 8, need, _lib.ERR_ALIGN)):
        assert lib.adaln_glu_bwd(*[P] * 8, ws, n, *size) == code
    assert lib.adaln_glu_fwd(None, None, None, None, None, 0, 64, 64, 0, 1,
                             None) == _lib.OK
    assert lib.adaln_glu_bwd_workspace_bytes(0, 64, 64, 1) == 0


def test_workspace_holds_the_partial_sums(lib):
    """Few tiles: the sums are split, and the workspace has room for them."""
    for M, D, F in ((1, 64, 64), (100, 1536, 4096), (777, 1000, 1480),
                    (20000, 64, 8), (4096, 5120, 13824)):
        n = lib.adaln_glu_bwd_workspace_bytes(M, D, F, 1)
        assert n >= 4 * M * F
        assert n <= 4 * M * F + 256 + 4 * 1024 * 128 * 128
        assert lib.adaln_glu_bwd_workspace_bytes(M, D, F, 0) >= 8 * M * F


def test_binding_refuses():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(32, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        A.glu_fwd(x, w, w)
    with pytest.raises(TypeError):
        A.glu_fwd(x.half(), w.half(), w.half())
    with pytest.raises(ValueError, match="act"):
        A.glu_fwd(x, w, w, act="relu")
    with pytest.raises(ValueError):
        A.glu_fwd(x[0], w, w)
