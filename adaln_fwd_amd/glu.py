"""Binding of the gated feed-forward (adaln_glu_*) for torch tensors: token
rows [M, D] or [B, N, D], weights [F, D] as a linear layer keeps them.
Checks, streams and allocation are those of :mod:`adaln_fwd_amd.ops`; outputs
and the workspace must not overlap inputs or each other."""

from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from .ops import _DTYPES, _check, _code, _on, _ptr, _stream

_ACTS = {"silu": 0, "gelu": 1}


def _shapes(x, wg, wu, act):
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    code = _code(x)
    if x.dim() not in (2, 3):
        raise ValueError(f"x must be [M, D] or [B, N, D], got shape "
                         f"{tuple(x.shape)}")
    if act not in _ACTS:
        raise ValueError(f"act must be 'silu' or 'gelu', got {act!r}")
    lead, D = tuple(x.shape[:-1]), x.shape[-1]
    F = wg.shape[0] if isinstance(wg, torch.Tensor) and wg.dim() == 2 else -1
    _check(x, "x", lead + (D,), x.dtype, x.device)
    _check(wg, "wg", (F, D), x.dtype, x.device)
    _check(wu, "wu", (F, D), x.dtype, x.device)
    M = 1
    for n in lead:
        M *= n
    return lead, M, D, F, code


def _out(t, like, name):
    """An output: as given, or a new one."""
    if t is None:
        return torch.empty_like(like)
    _check(t, name, like.shape, like.dtype, like.device)
    return t


def glu_fwd(x: torch.Tensor, wg: torch.Tensor, wu: torch.Tensor, *,
            act: str = "silu", save: bool = False,
            h: Optional[torch.Tensor] = None,
            saved: Optional[torch.Tensor] = None, stream=None):
    """h = act(x wg^T) * (x wu^T), act "silu" or "gelu" (tanh form); returns
    h, or with ``save=True`` (h, saved), `saved` being what the backward
    needs to skip the two products: both projections in float32 [2, M, F]."""
    lead, M, D, F, code = _shapes(x, wg, wu, act)
    dev = x.device
    lib = _lib.load()
    with _on(dev, stream):
        if h is None:
            h = x.new_empty(lead + (F,))
        else:
            _check(h, "h", lead + (F,), x.dtype, dev)
        if saved is not None:
            if not save:
                raise ValueError("saved was given without save=True")
            _check(saved, "saved", (2, M, F), torch.float32, dev)
        elif save:
            saved = x.new_empty((2, M, F), dtype=torch.float32)
        rc = lib.adaln_glu_fwd(_ptr(x), _ptr(wg), _ptr(wu), _ptr(h),
                               _ptr(saved), M, D, F, _ACTS[act], code,
                               _stream(dev, stream))
    _lib.check(rc, "adaln_glu_fwd")
    return (h, saved) if save else h


def glu_bwd_workspace_bytes(M: int, D: int, F: int,
                            dtype: torch.dtype = torch.bfloat16) -> int:
    return int(_lib.load().adaln_glu_bwd_workspace_bytes(
        M, D, F, _DTYPES.get(dtype, -1)))


def glu_bwd(dh: torch.Tensor, x: torch.Tensor, wg: torch.Tensor,
            wu: torch.Tensor, saved: Optional[torch.Tensor] = None, *,
            act: str = "silu", dx: Optional[torch.Tensor] = None,
            dwg: Optional[torch.Tensor] = None,
            dwu: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None, stream=None):
    """Backward of :func:`glu_fwd`; returns (dx, dwg, dwu) in x's dtype.
    Without `saved` both projections are computed again.  The workspace
    (bytes from :func:`glu_bwd_workspace_bytes`) is allocated if not given."""
    lead, M, D, F, code = _shapes(x, wg, wu, act)
    dev, dt = x.device, x.dtype
    _check(dh, "dh", lead + (F,), dt, dev)
    if saved is not None:
        _check(saved, "saved", (2, M, F), torch.float32, dev)
    lib = _lib.load()
    need = int(lib.adaln_glu_bwd_workspace_bytes(M, D, F, code))
    with _on(dev, stream):
        dx = _out(dx, x, "dx")
        dwg = _out(dwg, wg, "dwg")
        dwu = _out(dwu, wu, "dwu")
        if workspace is None:
            wbytes = max(need, 1)
            workspace = x.new_empty(wbytes, dtype=torch.uint8)
        else:
            if workspace.device != dev or not workspace.is_contiguous():
                raise ValueError(f"workspace must be a contiguous tensor on "
                                 f"{dev}")
            wbytes = workspace.numel() * workspace.element_size()
        rc = lib.adaln_glu_bwd(_ptr(dh), _ptr(x), _ptr(wg), _ptr(wu),
                               _ptr(saved), _ptr(dx), _ptr(dwg), _ptr(dwu),
                               _ptr(workspace), wbytes, M, D, F, _ACTS[act], code,
                               _stream(dev, stream))
    _lib.check(rc, "adaln_glu_bwd")
    return dx, dwg, dwu
