"""Binding of the gated join with the residual stream and its dropout
(adaln_residual_*) for torch tensors.  Checks, streams and allocation are those
of :mod:`adaln_fwd_amd.ops`.

Dropout's mask is never stored: it follows from `rng`, an int64 tensor [2] on
the GPU holding a seed and the number of the call.  The forward and its
backward get the same numbers; raise the second one (``rng[1] += 1``, in a
captured graph too) before the next forward."""

from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from .glu import _out
from .ops import _DTYPES, _check, _code, _on, _ptr, _shape3, _stream, _table


def _rate(p, rng, dev):
    p = float(p)
    if not 0.0 <= p <= 1.0 - 2.0 ** -16:
        raise ValueError(f"p must be from 0 to 1 - 2^-16, got {p}")
    if rng is not None:
        _check(rng, "rng", (2,), torch.int64, dev)
    elif p > 0:
        raise ValueError("dropout needs rng, an int64 tensor [2] of seed and "
                         "call number")
    return p


def _workspace(workspace, need, like):
    """The workspace and its bytes: as given, or a new one."""
    if workspace is None:
        return like.new_empty(max(need, 1), dtype=torch.uint8), max(need, 1)
    if workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on "
                         f"{like.device}")
    return workspace, workspace.numel() * workspace.element_size()


def residual_fwd(x: Optional[torch.Tensor], h: torch.Tensor,
                 gate: Optional[torch.Tensor] = None, *, p: float = 0.0,
                 rng: Optional[torch.Tensor] = None,
                 y: Optional[torch.Tensor] = None, stream=None):
    """y = x + gate[b] * drop(h); returns y.

    x, h: [B, N, D] (x None: nothing is added); gate: [B, D] or None; drop(h)
    keeps an element with probability 1 - p (a multiple of 2^-16) and divides
    it by that.  y may be x or h."""
    B, N, D = _shape3(h)
    dev, dt = h.device, h.dtype
    code = _code(h)
    _check(h, "h", (B, N, D), dt, dev)
    if x is not None:
        _check(x, "x", (B, N, D), dt, dev)
    if gate is not None:
        _check(gate, "gate", (B, D), dt, dev)
    p = _rate(p, rng, dev)
    lib = _lib.load()
    with _on(dev, stream):
        y = _out(y, h, "y")
        rc = lib.adaln_residual_fwd(_ptr(x), _ptr(h), _ptr(gate), p, _ptr(rng),
                                    _ptr(y), B, N, D, code,
                                    _stream(dev, stream))
    _lib.check(rc, "adaln_residual_fwd")
    return y


def residual_bwd_workspace_bytes(B: int, N: int, D: int,
                                 dtype: torch.dtype) -> int:
    return int(_lib.load().adaln_residual_bwd_workspace_bytes(
        B, N, D, _DTYPES.get(dtype, -1)))


def residual_bwd(dy: torch.Tensor, h: Optional[torch.Tensor],
                 gate: Optional[torch.Tensor] = None, *, p: float = 0.0,
                 rng: Optional[torch.Tensor] = None,
                 dh: Optional[torch.Tensor] = None,
                 dgate: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None):
    """Backward of :func:`residual_fwd` (the gradient of x is dy itself);
    returns (dh, dgate), dgate in float32, or None without a gate (h is not
    read then and may be None).  dh may be dy or h.  The workspace (bytes from
    :func:`residual_bwd_workspace_bytes`) is allocated if not given."""
    B, N, D = _shape3(dy)
    dev, dt = dy.device, dy.dtype
    code = _code(dy)
    _check(dy, "dy", (B, N, D), dt, dev)
    if h is not None or gate is not None:
        _check(h, "h", (B, N, D), dt, dev)
    if gate is not None:
        _check(gate, "gate", (B, D), dt, dev)
    elif dgate is not None:
        raise ValueError("dgate was given without a gate")
    p = _rate(p, rng, dev)
    lib = _lib.load()
    wbytes = 0
    with _on(dev, stream):
        dh = _out(dh, dy, "dh")
        if gate is not None:
            if dgate is None:
                dgate = dy.new_empty((B, D), dtype=torch.float32)
            else:
                _check(dgate, "dgate", (B, D), torch.float32, dev)
            workspace, wbytes = _workspace(
                workspace, int(lib.adaln_residual_bwd_workspace_bytes(
                    B, N, D, code)), dy)
        rc = lib.adaln_residual_bwd(_ptr(dy), _ptr(h), _ptr(gate), p,
                                    _ptr(rng), _ptr(dh), _ptr(dgate),
                                    _ptr(workspace), wbytes, B, N, D, code,
                                    _stream(dev, stream))
    _lib.check(rc, "adaln_residual_bwd")
    return dh, dgate


def _packed(t, name, seg_offsets, seg_mod):
    tab = _table(seg_offsets, seg_mod)
    if t.dim() != 2:
        raise ValueError(f"{name} must be [T, D], got shape {tuple(t.shape)}")
    if t.shape[0] != tab.rows:
        raise ValueError(f"{name} has {t.shape[0]} rows, seg_offsets ends at "
                         f"{tab.rows}")
    return tab


def residual_fwd_segments(x: Optional[torch.Tensor], h: torch.Tensor,
                          gate: torch.Tensor, seg_offsets, seg_mod=None, *,
                          p: float = 0.0, rng: Optional[torch.Tensor] = None,
                          y: Optional[torch.Tensor] = None, stream=None):
    """:func:`residual_fwd` for packed sequences: x, h [T, D], gate [nmod, D],
    segment s joined by gate[seg_mod[s]] as in :func:`fwd_segments`."""
    tab = _packed(h, "h", seg_offsets, seg_mod)
    dev, dt = h.device, h.dtype
    code = _code(h)
    D = h.shape[1]
    _check(h, "h", h.shape, dt, dev)
    if x is not None:
        _check(x, "x", h.shape, dt, dev)
    nmod = gate.shape[0] if gate.dim() == 2 else -1
    _check(gate, "gate", (nmod, D), dt, dev)
    p = _rate(p, rng, dev)
    lib = _lib.load()
    with _on(dev, stream):
        y = _out(y, h, "y")
        rc = lib.adaln_residual_fwd_segments(
            _ptr(x), _ptr(h), _ptr(gate), p, _ptr(rng), _ptr(y),
            tab.offsets_ptr, tab.mod_ptr, tab.nseg, nmod, D, code,
            _stream(dev, stream))
    _lib.check(rc, "adaln_residual_fwd_segments")
    return y


def residual_bwd_segments_workspace_bytes(seg_offsets, D: int,
                                          dtype: torch.dtype) -> int:
    tab = _table(seg_offsets, None)
    return int(_lib.load().adaln_residual_bwd_segments_workspace_bytes(
        tab.offsets_ptr, tab.nseg, D, _DTYPES.get(dtype, -1)))


def residual_bwd_segments(dy: torch.Tensor, h: torch.Tensor,
                          gate: torch.Tensor, seg_offsets, seg_mod=None, *,
                          p: float = 0.0, rng: Optional[torch.Tensor] = None,
                          dh: Optional[torch.Tensor] = None,
                          dgate: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None,
                          stream=None):
    """Backward of :func:`residual_fwd_segments`; returns (dh, dgate) with
    dgate float32 [nmod, D] summed over every segment that uses the vector."""
    tab = _packed(dy, "dy", seg_offsets, seg_mod)
    dev, dt = dy.device, dy.dtype
    code = _code(dy)
    D = dy.shape[1]
    _check(dy, "dy", dy.shape, dt, dev)
    _check(h, "h", dy.shape, dt, dev)
    nmod = gate.shape[0] if gate.dim() == 2 else -1
    _check(gate, "gate", (nmod, D), dt, dev)
    p = _rate(p, rng, dev)
    lib = _lib.load()
    with _on(dev, stream):
        dh = _out(dh, dy, "dh")
        if dgate is None:
            dgate = dy.new_empty((nmod, D), dtype=torch.float32)
        else:
            _check(dgate, "dgate", (nmod, D), torch.float32, dev)
        workspace, wbytes = _workspace(
            workspace, int(lib.adaln_residual_bwd_segments_workspace_bytes(
                tab.offsets_ptr, tab.nseg, D, code)), dy)
        rc = lib.adaln_residual_bwd_segments(
            _ptr(dy), _ptr(h), _ptr(gate), p, _ptr(rng), _ptr(dh),
            _ptr(dgate), _ptr(workspace), wbytes, tab.offsets_ptr,
            tab.mod_ptr, tab.nseg, nmod, D, code, _stream(dev, stream))
    _lib.check(rc, "adaln_residual_bwd_segments")
    return dh, dgate
