"""Linear attention without a GPU: the reference against the recurrence and
against differences, and the refusals of the C entry points and the binding."""

import ctypes

import pytest
import torch

import adaln_fwd_amd as A
from adaln_fwd_amd import _lib
from tests import ref_lin_attn as R

P = 0x1000


def _inputs(N, H, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = [torch.randn(N, H, d, generator=g, dtype=torch.float64)
         for _ in range(4)]
    s = [torch.randn(H, d, d, generator=g, dtype=torch.float64)
         for _ in range(2)]
    return t, s, torch.tensor([-0.1, -1.5, 0.0, float("-inf")])[:H]


def test_reference_is_the_recurrence():
    (q, k, v, _), (S0, _), decay = _inputs(9, 4, 3)
    o, last = R.forward(q, k, v, decay, 0.7, S0)
    S = S0.clone()
    for t in range(9):
        S = torch.exp(decay.double())[:, None, None] * S + \
            k[t][:, :, None] * v[t][:, None]
        want = 0.7 * torch.einsum("hij,hi->hj", S, q[t])
        torch.testing.assert_close(o[t], want, rtol=1e-12, atol=1e-12)
    torch.testing.assert_close(last, S, rtol=1e-12, atol=1e-12)


def test_reference_gradient_against_differences():
    (q, k, v, do), (S0, dS), decay = _inputs(7, 4, 3, seed=1)
    grads = R.backward(do, q, k, v, decay, 0.7, S0, dS)
    parts = [q, k, v, S0]

    def loss(parts):
        o, last = R.forward(*parts[:3], decay, 0.7, parts[3])
        return float((o * do).sum() + (last * dS).sum())

    for i, grad in enumerate(grads):
        for j in range(parts[i].numel()):
            d = torch.zeros(parts[i].numel(), dtype=torch.float64)
            d[j] = 1e-4
            d = d.reshape(parts[i].shape)
            up, down = list(parts), list(parts)
            up[i], down[i] = parts[i] + d, parts[i] - d
            assert (loss(up) - loss(down)) / 2e-4 == pytest.approx(
                float(grad.flatten()[j]), abs=1e-7)


def _no_gpu():
    if torch.cuda.device_count() > 0:
        pytest.skip("host-validation tests run only without a GPU")


def _heads(N, H, d, data=P, **kw):
    h = _lib.Heads(data, N * H * d, H * d, d)
    for k, v in kw.items():
        setattr(h, k, v)
    return ctypes.byref(h)


def test_refusals_of_the_c_entry_points():
    _no_gpu()
    lib = A.load()
    E = _lib

    def fwd(q="x", k="x", v="x", g=P, c=0.1, s=P, o="x", so=P, st=P,
            sb=1 << 40, off=None, nseg=0, B=2, N=4000, H=3, d=64, dt=1):
        x = _heads(4000, 3, 64)
        q, k, v, o = (x if t == "x" else t for t in (q, k, v, o))
        return lib.adaln_lin_attn_fwd(q, k, v, g, c, s, o, so, st, sb, off,
                                      nseg, B, N, H, d, dt, None)

    assert fwd(dt=5) == E.ERR_DTYPE
    assert fwd(B=-1) == fwd(N=-1) == fwd(H=-1) == fwd(d=0) == fwd(H=4097) \
        == fwd(B=1 << 21) == fwd(N=1 << 31) == fwd(c=float("nan")) \
        == fwd(c=float("inf")) == E.ERR_INVALID
    assert fwd(d=60) == fwd(d=62, dt=0) == E.ERR_ALIGN
    assert fwd(d=136) == E.ERR_UNSUPPORTED
    assert fwd(q=None) == fwd(k=None) == fwd(v=None) == fwd(o=None) \
        == fwd(g=None) == E.ERR_INVALID
    assert fwd(g=P + 2) == fwd(s=P + 4) == fwd(so=P + 8) == fwd(st=P + 4) \
        == E.ERR_ALIGN
    assert fwd(q=_heads(4000, 3, 64, data=P + 8)) == E.ERR_ALIGN
    assert fwd(q=_heads(4000, 3, 64, token_stride=100)) == E.ERR_ALIGN
    # an output's heads may not overlap; an input's may
    assert fwd(o=_heads(4000, 3, 64, head_stride=0)) == E.ERR_INVALID
    need = lib.adaln_lin_attn_states_bytes(None, 0, 2, 4000, 3, 64, 1)
    assert need > 0 and need % (3 * 64 * 64 * 4) == 0
    assert fwd(sb=need - 1) == fwd(st=None) == E.ERR_WORKSPACE
    off = (ctypes.c_int64 * 3)(0, 1000, 4000)
    assert fwd(off=off, nseg=2) == E.ERR_INVALID  # B is not 1
    assert fwd(off=off, nseg=2, B=1, N=3999) == E.ERR_INVALID
    assert fwd(off=off, nseg=0, B=1) == fwd(off=off, nseg=129, B=1) \
        == E.ERR_INVALID
    down = (ctypes.c_int64 * 3)(0, 4500, 4000)
    assert fwd(off=down, nseg=2, B=1) == E.ERR_INVALID
    need = lib.adaln_lin_attn_states_bytes(off, 2, 1, 4000, 3, 64, 1)
    assert fwd(off=off, nseg=2, B=1, sb=need - 1) == E.ERR_WORKSPACE
    # nothing to do
    for kw in (dict(B=0), dict(H=0)):
        assert fwd(q=None, k=None, v=None, o=None, g=None, s=None, so=None,
                   **kw) == E.OK
    # few tokens, and wrong arguments, need no states
    for args in ((2, 64, 3, 64, 1), (2, 0, 3, 64, 1), (2, 4000, 3, 60, 1),
                 (2, 4000, 3, 64, 7), (-1, 4000, 3, 64, 1)):
        assert lib.adaln_lin_attn_states_bytes(None, 0, *args) == 0

    def bwd(do="x", q="x", k="x", v="x", g=P, s=P, st=P, ds=P, dq="x", dk="x",
            dv="x", d0=P, ws=P, wb=1 << 40):
        x = _heads(4000, 3, 64)
        do, q, k, v, dq, dk, dv = (x if t == "x" else t for t in
                                   (do, q, k, v, dq, dk, dv))
        return lib.adaln_lin_attn_bwd(do, q, k, v, g, 0.1, s, st, ds, dq, dk,
                                      dv, d0, ws, wb, None, 0, 2, 4000, 3, 64,
                                      1, None)

    assert bwd(do=None) == bwd(q=None) == bwd(k=None) == bwd(v=None) \
        == bwd(dq=None) == bwd(dk=None) == bwd(dv=None) == bwd(g=None) \
        == E.ERR_INVALID
    assert bwd(s=P + 4) == bwd(st=P + 4) == bwd(ds=P + 4) == bwd(d0=P + 4) \
        == bwd(ws=P + 4) == E.ERR_ALIGN
    one = lib.adaln_lin_attn_bwd_workspace_bytes(1, None, 0, 2, 4000, 3, 64, 1)
    two = lib.adaln_lin_attn_bwd_workspace_bytes(0, None, 0, 2, 4000, 3, 64, 1)
    assert two == 2 * one > 0
    assert bwd(wb=one - 1) == bwd(st=None, wb=two - 1) == bwd(ws=None) \
        == E.ERR_WORKSPACE

    def step(q="x", k="x", v="x", g=P, s=P, o="x", so=P, B=2, H=3, d=64, dt=1):
        x = _heads(1, 3, 64)
        q, k, v, o = (x if t == "x" else t for t in (q, k, v, o))
        return lib.adaln_lin_attn_step(q, k, v, g, 0.1, s, o, so, B, H, d, dt,
                                       None)

    assert step(q=None) == step(k=None) == step(v=None) == step(o=None) \
        == step(g=None) == step(s=None) == step(so=None) == step(B=-1) \
        == E.ERR_INVALID
    assert step(s=P + 4) == step(so=P + 4) == step(d=60) == E.ERR_ALIGN
    assert step(d=136) == E.ERR_UNSUPPORTED
    assert step(B=0, s=None, so=None, q=None) == E.OK


def test_refusals_of_the_binding():
    q, g = torch.zeros(2, 3, 4, 8), torch.zeros(4)
    with pytest.raises(ValueError, match="GPU tensor"):
        A.lin_attn_fwd(q, q, q, g)
    with pytest.raises(ValueError, match="\\[T, H, d\\]"):
        A.lin_attn_fwd(q[0, 0], q, q, g)
    with pytest.raises(ValueError, match="packed tokens"):
        A.lin_attn_fwd(q, q, q, g, seg_offsets=[0, 3])
    with pytest.raises(ValueError, match="ends at"):
        A.lin_attn_bwd(q[0], q[0], q[0], q[0], g, seg_offsets=[0, 2])
    with pytest.raises(TypeError, match="dtype"):
        A.lin_attn_step(q[0].half(), q[0], q[0], g, q)
