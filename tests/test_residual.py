"""The gated join with dropout without a GPU: the reference's generator
against published vectors, its gradient against differences, and the refusals
of the C entry points and of the binding."""

import ctypes

import numpy as np
import pytest
import torch

import adaln_fwd_amd as A
from adaln_fwd_amd import _lib
from tests import ref_residual as R


def test_generator_against_published_vectors():
    # the test vectors published with the generator
    f = 0xFFFFFFFF
    for ctr, key, want in [
            ((0, 0, 0, 0), (0, 0),
             (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((f, f, f, f), (f, f),
             (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344),
             (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]:
        got = R.philox(np.array(ctr, dtype=np.uint64), key)
        assert tuple(int(v) for v in got) == want


def test_mask_numbering_and_rate():
    keep, s = R.keep_mask(3000, 40, 0.25, (7, 1))
    assert s == 65536 / 49152
    # 120000 draws of 3/4: five standard deviations are 0.0063
    assert abs(keep.double().mean().item() - 0.75) < 0.0063
    # a row's numbers go by its place alone
    again, _ = R.keep_mask(10, 40, 0.25, (7, 1), row0=55)
    assert torch.equal(again, keep[55:65])
    other, _ = R.keep_mask(3000, 40, 0.25, (7, 2))
    assert not torch.equal(other, keep)


def test_reference_gradient_against_differences():
    g = torch.Generator().manual_seed(2)
    h, x, dy = (torch.randn(5, 12, generator=g, dtype=torch.float64)
                for _ in range(3))
    gate = torch.randn(2, 12, generator=g, dtype=torch.float64)
    mod = torch.tensor([0, 0, 1, 1, 1])
    dh, dgate, _ = R.backward(dy, h, gate, 0.3, (1, 2), mod, 2)

    def loss(h, gate):
        return (R.forward(x, h, gate, 0.3, (1, 2), mod) * dy).sum()

    for i in range(60):
        d = torch.zeros(60, dtype=torch.float64)
        d[i] = 1e-4
        d = d.reshape(5, 12)
        diff = (loss(h + d, gate) - loss(h - d, gate)) / 2e-4
        assert float(diff) == pytest.approx(float(dh.flatten()[i]), abs=1e-8)
    for i in range(24):
        d = torch.zeros(24, dtype=torch.float64)
        d[i] = 1e-4
        d = d.reshape(2, 12)
        diff = (loss(h, gate + d) - loss(h, gate - d)) / 2e-4
        assert float(diff) == pytest.approx(float(dgate.flatten()[i]), abs=1e-8)


def _no_gpu():
    if torch.cuda.device_count() > 0:
        pytest.skip("host-validation tests run only without a GPU")


P = 0x1000  # 16-byte aligned, never dereferenced


def test_refusals_of_the_c_entry_points():
    _no_gpu()
    lib = A.load()
    f = lib.adaln_residual_fwd

    def fwd(x=P, h=P, g=P, p=0.1, rng=P, y=P, B=2, N=3, D=64, dt=1):
        return f(x, h, g, p, rng, y, B, N, D, dt, None)

    assert fwd(dt=7) == _lib.ERR_DTYPE
    assert fwd(B=-1) == fwd(N=-1) == fwd(D=0) == _lib.ERR_INVALID
    assert fwd(D=60) == fwd(D=62, dt=0) == _lib.ERR_ALIGN
    assert fwd(D=32776) == _lib.ERR_UNSUPPORTED
    assert fwd(h=None) == fwd(y=None) == fwd(rng=None) == _lib.ERR_INVALID
    assert fwd(x=P + 8) == fwd(h=P + 4) == fwd(g=P + 2) == fwd(y=P + 8) \
        == fwd(rng=P + 4) == _lib.ERR_ALIGN
    for p in (-0.1, 1.0, 1 - 2.0 ** -17, float("nan"), float("inf")):
        assert fwd(p=p) == _lib.ERR_INVALID
        assert b"p must be" in lib.adaln_last_error()
    assert fwd(x=None, h=None, y=None, rng=None, g=None, N=0) == _lib.OK

    b = lib.adaln_residual_bwd

    def bwd(dy=P, h=P, g=P, p=0.1, rng=P, dh=P, dg=P, ws=P, wb=1 << 30, B=2,
            N=4000, D=64, dt=1):
        return b(dy, h, g, p, rng, dh, dg, ws, wb, B, N, D, dt, None)

    assert bwd(dy=None) == bwd(h=None) == bwd(g=None) == bwd(dh=None) \
        == bwd(dg=None) == bwd(rng=None) == _lib.ERR_INVALID
    assert bwd(dg=P + 4) == bwd(ws=P + 4) == _lib.ERR_ALIGN
    need = lib.adaln_residual_bwd_workspace_bytes(2, 4000, 64, 1)
    assert need > 0
    assert bwd(wb=need - 1) == bwd(ws=None) == _lib.ERR_WORKSPACE
    # few tokens, no tokens and wrong arguments need none
    for args in ((2, 1, 64, 1), (2, 0, 64, 1), (2, 4000, 60, 1), (2, 3, 64, 9)):
        assert lib.adaln_residual_bwd_workspace_bytes(*args) == 0
    # without a gate, no samples: nothing to do
    assert bwd(dy=None, h=None, g=None, dh=None, dg=None, B=0) == _lib.OK


def test_refusals_of_the_segment_entry_points():
    _no_gpu()
    lib = A.load()
    off = (ctypes.c_int64 * 3)(0, 4, 9)
    mod = (ctypes.c_int32 * 2)(1, 0)

    def fwd(x=P, h=P, g=P, p=0.1, rng=P, y=P, off=off, mod=mod, nseg=2, nmod=2,
            D=64, dt=1):
        return lib.adaln_residual_fwd_segments(x, h, g, p, rng, y, off, mod,
                                               nseg, nmod, D, dt, None)

    assert fwd(nseg=129) == fwd(nseg=-1) == fwd(off=None) == fwd(nmod=1) \
        == _lib.ERR_INVALID
    assert fwd(off=(ctypes.c_int64 * 3)(0, 4, 3)) == _lib.ERR_INVALID
    assert fwd(off=(ctypes.c_int64 * 3)(1, 4, 5)) == _lib.ERR_INVALID
    assert fwd(g=None) == fwd(h=None) == fwd(p=2.0) == _lib.ERR_INVALID
    assert fwd(off=(ctypes.c_int64 * 3)(0, 0, 0), x=None, h=None, y=None,
               g=None, rng=None) == _lib.OK

    def bwd(dy=P, h=P, g=P, p=0.1, rng=P, dh=P, dg=P, ws=P, wb=1 << 30,
            off=off, mod=mod, nseg=2, nmod=2, D=64, dt=1):
        return lib.adaln_residual_bwd_segments(dy, h, g, p, rng, dh, dg, ws,
                                               wb, off, mod, nseg, nmod, D, dt,
                                               None)

    need = lib.adaln_residual_bwd_segments_workspace_bytes(off, 2, 64, 1)
    assert need > 0
    assert bwd(wb=need - 1) == bwd(ws=None) == _lib.ERR_WORKSPACE
    assert bwd(dg=None) == bwd(g=None) == bwd(dh=None) == _lib.ERR_INVALID
    assert lib.adaln_residual_bwd_segments_workspace_bytes(off, 2, 60, 1) == 0
    assert lib.adaln_residual_bwd_segments_workspace_bytes(off, 0, 64, 1) == 0


def test_refusals_of_the_binding():
    h = torch.zeros(2, 3, 64)
    with pytest.raises(ValueError, match="GPU tensor"):
        A.residual_fwd(h, h, h[:, 0])
    with pytest.raises(ValueError, match="\\[B, N, D\\]"):
        A.residual_fwd(h[0], h[0])
    with pytest.raises(TypeError, match="dtype"):
        A.residual_fwd(h.half(), h.half())
    with pytest.raises(ValueError, match="\\[T, D\\]"):
        A.residual_fwd_segments(h, h, h[:, 0], [0, 3])
    with pytest.raises(ValueError, match="ends at"):
        A.residual_bwd_segments(h[0], h[0], h[:, 0], [0, 2])
