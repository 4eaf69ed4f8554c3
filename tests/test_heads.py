"""Rotary positions and query/key norms without a GPU: the float64 reference
of the GPU tests against differences and hand values, the frequency table,
and the refusals of the C entry points and of the binding."""

import ctypes

import numpy as np
import pytest
import torch

import adaln_fwd_amd as A
from adaln_fwd_amd import _lib
from tests import ref_heads as R


def test_freqs_table():
    f = A.rope_freqs((2, 0, 3), theta=100.0)
    assert f.shape == (3, 5) and f.dtype == np.float64
    np.testing.assert_allclose(f[0], [1, 0.1, 0, 0, 0])
    assert not f[1].any()
    np.testing.assert_allclose(f[2, 2:], 100.0 ** (-np.arange(3) / 3))
    for bad in ((), (0, 0), (-1, 2)):
        with pytest.raises(ValueError):
            A.rope_freqs(bad)


def test_reference_by_hand():
    # one head of 6 features, two pairs, a quarter turn and none
    x = torch.arange(1.0, 7.0, dtype=torch.float64).reshape(1, 1, 1, 6)
    ang = torch.tensor([[torch.pi / 2, 0.0]], dtype=torch.float64)
    y = R.rotate(x, ang, "interleaved").flatten().tolist()
    assert y == pytest.approx([-2, 1, 3, 4, 5, 6])
    y = R.rotate(x, ang, "half").flatten().tolist()
    assert y == pytest.approx([-3, 2, 1, 4, 5, 6])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_reference_gradient_against_differences(layout):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2, 3, 2, 8, generator=g, dtype=torch.float64)
    w = torch.randn(8, generator=g, dtype=torch.float64)
    dy = torch.randn(2, 3, 2, 8, generator=g, dtype=torch.float64)
    pos = torch.randint(-50, 50, (3, 2), generator=g)
    ang = R.angles(pos, A.rope_freqs((1, 2)))
    dx, dw, _ = R.qk_bwd(dy, x, w, ang, layout, eps=1e-3)
    h = 1e-5

    def loss(x, w):
        return float((R.qk_fwd(x, w, ang, layout, eps=1e-3) * dy).sum())

    for i in (0, 17, 50, 95):
        d = torch.zeros(x.numel(), dtype=torch.float64)
        d[i] = h
        d = d.reshape(x.shape)
        assert (loss(x + d, w) - loss(x - d, w)) / (2 * h) == pytest.approx(
            float(dx.flatten()[i]), abs=1e-7)
    for i in range(8):
        d = torch.zeros(8, dtype=torch.float64)
        d[i] = h
        assert (loss(x, w + d) - loss(x, w - d)) / (2 * h) == pytest.approx(
            float(dw[i]), abs=1e-7)


# ------------------------------------------------------------------ refusals

P = 0x1000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.device_count() > 0:
        pytest.skip("host-validation tests run only without a GPU")
    return A.load()


def _h(data=P, b=64 * 2 * 5, n=64 * 2, h=64):
    return ctypes.byref(_lib.Heads(data, b, n, h))


_FREQS = np.ones((3, 32))


def _rot(pos=P, batch=0, freqs=_FREQS, axes=3, pairs=32, layout=0):
    return ctypes.byref(_lib.Rotation(
        pos, batch, None if freqs is None else freqs.ctypes.data, axes, pairs,
        layout))


def _rope(lib, q=None, k=None, rot=None, qo=None, ko=None, B=2, N=5, Hq=2,
          Hk=2, d=64, dt=1, entry="adaln_rope_fwd"):
    return getattr(lib, entry)(q or _h(), k or _h(), rot or _rot(), qo or _h(),
                               ko or _h(), B, N, Hq, Hk, d, dt, None)


REFUSED = [
    (dict(dt=7), _lib.ERR_DTYPE),
    (dict(B=-1), _lib.ERR_INVALID),
    (dict(Hk=-1), _lib.ERR_INVALID),
    (dict(d=0), _lib.ERR_INVALID),
    (dict(d=60), _lib.ERR_ALIGN),
    (dict(d=520), _lib.ERR_UNSUPPORTED),
    (dict(Hq=4097), _lib.ERR_INVALID),
    (dict(B=1 << 16, N=1 << 15), _lib.ERR_INVALID),
    (dict(rot=dict(axes=0)), _lib.ERR_INVALID),
    (dict(rot=dict(axes=5)), _lib.ERR_INVALID),
    (dict(rot=dict(pairs=33)), _lib.ERR_INVALID),
    (dict(rot=dict(pairs=0)), _lib.ERR_INVALID),
    (dict(rot=dict(layout=2)), _lib.ERR_INVALID),
    (dict(rot=dict(layout=1, pairs=28)), _lib.ERR_ALIGN),
    (dict(rot=dict(freqs=None)), _lib.ERR_INVALID),
    (dict(rot=dict(freqs=np.full((3, 32), np.nan))), _lib.ERR_INVALID),
    (dict(rot=dict(freqs=np.full((3, 32), -1e7))), _lib.ERR_INVALID),
    (dict(rot=dict(pos=None)), _lib.ERR_INVALID),
    (dict(rot=dict(pos=P + 2)), _lib.ERR_ALIGN),
    (dict(rot=dict(batch=-3)), _lib.ERR_INVALID),
    (dict(rot=dict(batch=4)), _lib.ERR_INVALID),
    (dict(rot=dict(axes=4, pairs=128), d=256), _lib.ERR_UNSUPPORTED),
    (dict(q=dict(data=None)), _lib.ERR_INVALID),
    (dict(q=dict(data=P + 8)), _lib.ERR_ALIGN),
    (dict(k=dict(n=132)), _lib.ERR_ALIGN),
    (dict(k=dict(n=-128)), _lib.ERR_INVALID),
    (dict(q=dict(h=1 << 34)), _lib.ERR_UNSUPPORTED),
    (dict(qo=dict(h=32)), _lib.ERR_INVALID),     # heads of the output overlap
    (dict(ko=dict(n=0)), _lib.ERR_INVALID),
    (dict(ko=dict(b=64 * 4)), _lib.ERR_INVALID),  # samples overlap
]


@pytest.mark.parametrize("case", range(len(REFUSED)))
def test_refusals(lib, case):
    kw, code = REFUSED[case]
    kw = {n: (_rot(**v) if n == "rot" else _h(**v)) if isinstance(v, dict)
          else v for n, v in kw.items()}
    for entry in ("adaln_rope_fwd", "adaln_rope_bwd"):
        assert _rope(lib, entry=entry, **kw) == code
        assert lib.adaln_last_error()
    a = dict(q=_h(), k=_h(), rot=_rot(), qo=_h(), ko=_h(), B=2, N=5, Hq=2,
             Hk=2, d=64, dt=1) | kw
    size = [a[n] for n in ("B", "N", "Hq", "Hk", "d", "dt")]
    assert lib.adaln_qk_norm_rope_fwd(a["q"], a["k"], P, P, 1e-6, a["rot"],
                                      a["qo"], a["ko"], *size, None) == code
    assert lib.adaln_qk_norm_rope_bwd(
        _h(), _h(), a["q"], a["k"], P, P, 1e-6, a["rot"], a["qo"], a["ko"], P,
        P, P, 1 << 40, *size, None) == code


def test_refusals_of_the_norm(lib):
    size = (2, 5, 2, 2, 64, 1, None)
    f = lib.adaln_qk_norm_rope_fwd
    for wq, wk, eps, code in [(None, P, 1e-6, _lib.ERR_INVALID),
                              (P, P + 4, 1e-6, _lib.ERR_ALIGN),
                              (P, P, -1.0, _lib.ERR_INVALID),
                              (P, P, float("nan"), _lib.ERR_INVALID),
                              (P, P, float("inf"), _lib.ERR_INVALID)]:
        assert f(_h(), _h(), wq, wk, eps, _rot(), _h(), _h(), *size) == code
    # so few tokens need no workspace; 500 per sample do
    assert lib.adaln_qk_norm_rope_bwd_workspace_bytes(*size[:-1]) == 0
    size = (2, 500) + size[2:]
    need = lib.adaln_qk_norm_rope_bwd_workspace_bytes(*size[:-1])
    assert need > 0 and need % (2 * 64 * 4) == 0

    def _far(data=P, b=64 * 2 * 500):
        return ctypes.byref(_lib.Heads(data, b, 128, 64))

    def g(dwq=P, dwk=P, ws=P, n=need, dy=None):
        return lib.adaln_qk_norm_rope_bwd(
            dy or _far(), _far(), _far(), _far(), P, P, 1e-6, _rot(), _far(),
            _far(), dwq, dwk, ws, n, *size)

    assert g(ws=None) == _lib.ERR_WORKSPACE
    assert g(n=need - 1) == _lib.ERR_WORKSPACE
    assert b"workspace" in lib.adaln_last_error()
    assert g(ws=P + 4) == _lib.ERR_ALIGN
    assert g(dwq=None) == _lib.ERR_INVALID
    assert g(dy=_far(data=None)) == _lib.ERR_INVALID


def test_empty_calls_need_nothing(lib):
    r = _rot(pos=None)
    for B, N, Hq, Hk in ((0, 5, 2, 2), (2, 0, 2, 2), (2, 5, 0, 0)):
        assert lib.adaln_rope_fwd(None, None, r, None, None, B, N, Hq, Hk, 64,
                                  1, None) == _lib.OK
        assert lib.adaln_qk_norm_rope_fwd(None, None, None, None, 1e-6, r,
                                          None, None, B, N, Hq, Hk, 64, 1,
                                          None) == _lib.OK
    ws = lib.adaln_qk_norm_rope_bwd_workspace_bytes
    assert ws(0, 5, 2, 2, 64, 1) == 0 and ws(1, 5, 2, 2, 60, 1) == 0


def test_binding_refuses():
    q = torch.zeros(2, 3, 64, dtype=torch.bfloat16)
    pos = torch.zeros(2, 3, dtype=torch.int32)
    f = A.rope_freqs((10, 11, 11))
    with pytest.raises(ValueError, match="GPU"):
        A.rope_fwd(q, q, pos, f)
    with pytest.raises(TypeError):
        A.rope_fwd(q.half(), q.half(), pos, f)
    with pytest.raises(ValueError, match="None"):
        A.rope_fwd(None, None, pos, f)
    with pytest.raises(ValueError):
        A.rope_fwd(q[0], q[0], pos, f)
