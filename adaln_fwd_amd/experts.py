"""Binding of the way of tokens to the experts of a mixture and back
(adaln_experts_*) for torch tensors.  Checks, streams and allocation are those
of :mod:`adaln_fwd_amd.ops`.

    offsets, slot = experts_plan(expert, E)        # a router's choices [T, k]
    xs = experts_sort_fwd(x, slot)                 # rows by expert
    ...                                            # ys: each expert's rows
    y = experts_join_fwd(ys, slot, w)              # weighted, back at the tokens

Plan, sort and join go by what stands on the GPU, and a captured graph of them by
each replay's choices.  The experts' own products need their rows' limits on the
host (``offsets.tolist()``, which waits for the GPU); captured, they keep those."""

from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from .glu import _out
from .ops import _check, _code, _on, _ptr, _stream
from .residual import _workspace


def experts_plan_workspace_bytes(T: int, k: int, E: int) -> int:
    return int(_lib.load().adaln_experts_plan_workspace_bytes(T, k, E))


def experts_plan(expert: torch.Tensor, E: int, *,
                 offsets: Optional[torch.Tensor] = None,
                 slot: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None):
    """Where each choice stands when the choices are sorted by expert, those
    of one expert by token; returns (offsets, slot).

    expert: int32 or int64 [T, k]; a choice outside [0, E) is dropped.
    offsets: int32 [E + 1], expert e's sorted rows; slot: int32 [T, k], -1 for
    a dropped choice.  The workspace (bytes from
    :func:`experts_plan_workspace_bytes`) is allocated if not given."""
    if not isinstance(expert, torch.Tensor):
        raise TypeError("expert must be a torch.Tensor")
    if expert.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"expert has dtype {expert.dtype}, expected int32 or "
                        "int64")
    if expert.dim() != 2:
        raise ValueError(f"expert must be [T, k], got shape "
                         f"{tuple(expert.shape)}")
    T, k = expert.shape
    dev, E = expert.device, int(E)
    _check(expert, "expert", (T, k), expert.dtype, dev)
    lib = _lib.load()
    with _on(dev, stream):
        if offsets is None:
            offsets = expert.new_empty(max(E, 0) + 1, dtype=torch.int32)
        else:
            _check(offsets, "offsets", (E + 1,), torch.int32, dev)
        if slot is None:
            slot = expert.new_empty((T, k), dtype=torch.int32)
        else:
            _check(slot, "slot", (T, k), torch.int32, dev)
        need = int(lib.adaln_experts_plan_workspace_bytes(T, k, E))
        wbytes = 0
        if need or workspace is not None:
            workspace, wbytes = _workspace(workspace, need, expert)
        rc = lib.adaln_experts_plan(
            _ptr(expert), int(expert.dtype == torch.int64), _ptr(offsets),
            _ptr(slot), _ptr(workspace), wbytes, T, k, E,
            _stream(dev, stream))
    _lib.check(rc, "adaln_experts_plan")
    return offsets, slot


def _rows(one, many, slot, one_name, many_name):
    """Sizes of a call with a row per token (`one`) and sorted rows (`many`),
    either of which may be missing."""
    ref, name = (one, one_name) if one is not None else (many, many_name)
    if not isinstance(ref, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not isinstance(slot, torch.Tensor):
        raise TypeError("slot must be a torch.Tensor")
    code = _code(ref)
    if ref.dim() != 2 or slot.dim() != 2:
        raise ValueError(f"{name} must be [rows, D] and slot [T, k], got "
                         f"shapes {tuple(ref.shape)}, {tuple(slot.shape)}")
    T, k = slot.shape
    D = ref.shape[1]
    if one is not None:
        _check(one, one_name, (T, D), ref.dtype, ref.device)
    if many is not None:
        _check(many, many_name, (T * k, D), ref.dtype, ref.device)
    _check(slot, "slot", (T, k), torch.int32, ref.device)
    return T, k, D, code, ref.device


def _new(t, name, rows, D, like):
    if t is None:
        return like.new_empty((rows, D))
    _check(t, name, (rows, D), like.dtype, like.device)
    return t


def experts_sort_fwd(x: torch.Tensor, slot: torch.Tensor, *,
                     xs: Optional[torch.Tensor] = None, stream=None):
    """xs[slot[t, j]] = x[t]: the tokens' rows [T, D] in sorted order
    [T * k, D].  Rows from offsets[E] on (as many as choices were dropped) are
    left as they are."""
    T, k, D, code, dev = _rows(x, None, slot, "x", "")
    lib = _lib.load()
    with _on(dev, stream):
        xs = _new(xs, "xs", T * k, D, x)
        rc = lib.adaln_experts_sort_fwd(_ptr(x), _ptr(slot), _ptr(xs), T, k, D,
                                        code, _stream(dev, stream))
    _lib.check(rc, "adaln_experts_sort_fwd")
    return xs


def experts_sort_bwd(dxs: torch.Tensor, slot: torch.Tensor, *,
                     dx: Optional[torch.Tensor] = None, stream=None):
    """Backward of :func:`experts_sort_fwd`: dx[t] = sum_j dxs[slot[t, j]]."""
    T, k, D, code, dev = _rows(None, dxs, slot, "", "dxs")
    lib = _lib.load()
    with _on(dev, stream):
        dx = _new(dx, "dx", T, D, dxs)
        rc = lib.adaln_experts_sort_bwd(_ptr(dxs), _ptr(slot), _ptr(dx), T, k,
                                        D, code, _stream(dev, stream))
    _lib.check(rc, "adaln_experts_sort_bwd")
    return dx


def experts_join_fwd(ys: torch.Tensor, slot: torch.Tensor, w: torch.Tensor, *,
                     y: Optional[torch.Tensor] = None, stream=None):
    """y[t] = sum_j w[t, j] ys[slot[t, j]], w float32 [T, k]: the experts'
    outputs [T * k, D], weighted, back at their tokens [T, D]."""
    T, k, D, code, dev = _rows(None, ys, slot, "", "ys")
    _check(w, "w", (T, k), torch.float32, dev)
    lib = _lib.load()
    with _on(dev, stream):
        y = _new(y, "y", T, D, ys)
        rc = lib.adaln_experts_join_fwd(_ptr(ys), _ptr(slot), _ptr(w), _ptr(y),
                                        T, k, D, code, _stream(dev, stream))
    _lib.check(rc, "adaln_experts_join_fwd")
    return y


def experts_join_bwd(dy: torch.Tensor, ys: torch.Tensor, slot: torch.Tensor,
                     w: torch.Tensor, *, dys: Optional[torch.Tensor] = None,
                     dw: Optional[torch.Tensor] = None, stream=None):
    """Backward of :func:`experts_join_fwd`; returns (dys, dw): dys[slot[t, j]]
    = w[t, j] dy[t] and dw[t, j] = dy[t] . ys[slot[t, j]] (float32, zero for a
    dropped choice).  Rows of dys that no choice has are left as they are; dys
    may be ys."""
    T, k, D, code, dev = _rows(dy, ys, slot, "dy", "ys")
    _check(w, "w", (T, k), torch.float32, dev)
    lib = _lib.load()
    with _on(dev, stream):
        dys = _out(dys, ys, "dys")
        if dw is None:
            dw = torch.empty_like(w)
        else:
            _check(dw, "dw", (T, k), torch.float32, dev)
        rc = lib.adaln_experts_join_bwd(_ptr(dy), _ptr(ys), _ptr(slot),
                                        _ptr(w), _ptr(dys), _ptr(dw), T, k, D,
                                        code, _stream(dev, stream))
    _lib.check(rc, "adaln_experts_join_bwd")
    return dys, dw
