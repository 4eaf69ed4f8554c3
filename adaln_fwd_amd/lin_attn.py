"""Binding of linear attention with a decay for each head (adaln_lin_attn_*)
for torch tensors.

q, k and v are [B, N, H, d], or [T, H, d] for packed tokens, in any memory order
that keeps a head's features contiguous, as the rotations leave them: views of
one projection's output, or transposed [B, H, N, d].  Checks, streams and
allocation are those of :mod:`adaln_fwd_amd.ops`."""

from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from .heads import _ref, _wrong
from .ops import _DTYPES, _check, _code, _on, _ptr, _stream, _table
from .residual import _workspace

F32 = torch.float32


class _Call:
    """What the entry points share: shapes, device, sequences, descriptors."""

    __slots__ = ("dev", "index", "dt", "code", "shape", "four", "B", "N", "H",
                 "d", "tab", "seqs", "scale", "decay")

    def __init__(self, q, log_decay, scale, seg_offsets):
        if not isinstance(q, torch.Tensor):
            raise TypeError("q must be a torch.Tensor")
        shape = q.shape
        if len(shape) not in (3, 4):
            raise ValueError("q, k and v must be [B, N, H, d] or [T, H, d], "
                             f"got shape {tuple(shape)}")
        self.dev, self.dt, self.shape = q.device, q.dtype, shape
        self.index = q.get_device()
        self.code = _code(q)
        self.four = len(shape) == 4
        self.B = shape[0] if self.four else 1
        self.N, self.H, self.d = shape[-3:]
        self.tab = None
        if seg_offsets is not None:
            if self.four:
                raise ValueError("seg_offsets needs packed tokens [T, H, d]")
            self.tab = _table(seg_offsets, None)
            if self.tab.rows != self.N:
                raise ValueError(f"q has {self.N} tokens, seg_offsets ends at "
                                 f"{self.tab.rows}")
        self.seqs = self.B if self.tab is None else self.tab.nseg
        self.scale = self.d ** -0.5 if scale is None else float(scale)
        self.decay = log_decay
        _check(log_decay, "log_decay", (self.H,), F32, self.dev)

    def heads(self, t, name) -> _lib.Heads:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        shape, st = t.shape, t.stride()
        # one condition for calls that are right; which one failed comes after
        if not (t.is_cuda and t.get_device() == self.index
                and t.dtype is self.dt and shape == self.shape
                and (st[-1] == 1 or self.d == 1)):
            if shape != self.shape:
                raise ValueError(f"{name} has shape {tuple(shape)}, expected "
                                 f"{tuple(self.shape)}")
            _wrong(t, name, self.shape, self.dt, self.dev)
        return _lib.Heads(_ptr(t), st[0] if self.four else 0, st[-3], st[-2])

    def out(self, t, like, name):
        """An output and its descriptor: as given, or a contiguous one."""
        if t is None:
            t = torch.empty_like(like, memory_format=torch.contiguous_format)
        return t, self.heads(t, name)

    def state(self, t, name):
        if t is not None:
            _check(t, name, (self.seqs, self.H, self.d, self.d), F32, self.dev)
        return t

    def new_state(self, t, name, like):
        if t is None:
            return like.new_empty((self.seqs, self.H, self.d, self.d),
                                  dtype=F32)
        return self.state(t, name)

    def sequences(self):
        """seg_offsets and nseg, the entry points' own order."""
        if self.tab is None:
            return None, 0
        return self.tab.offsets_ptr, self.tab.nseg

    def sizes(self, stream):
        return (*self.sequences(), self.B, self.N, self.H, self.d, self.code,
                _stream(self.dev, stream))


def _bytes(f, seg_offsets, B, N, H, d, dtype, *first):
    tab = None if seg_offsets is None else _table(seg_offsets, None)
    return int(f(*first, None if tab is None else tab.offsets_ptr,
                 0 if tab is None else tab.nseg, B, N, H, d,
                 _DTYPES.get(dtype, -1)))


def lin_attn_states_bytes(B: int, N: int, H: int, d: int, dtype: torch.dtype,
                          seg_offsets=None) -> int:
    """Bytes of the states that the forward keeps within its sequences."""
    return _bytes(_lib.load().adaln_lin_attn_states_bytes, seg_offsets, B, N,
                  H, d, dtype)


def lin_attn_fwd(q, k, v, log_decay: torch.Tensor, *,
                 scale: Optional[float] = None,
                 state: Optional[torch.Tensor] = None, final: bool = False,
                 save: bool = False, seg_offsets=None,
                 o: Optional[torch.Tensor] = None,
                 state_out: Optional[torch.Tensor] = None,
                 saved: Optional[torch.Tensor] = None, stream=None):
    """S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T, o_t = scale * S_t^T q_t;
    returns (o, state_out, saved).

    log_decay: float32 [H], at most 0, a constant of the head (no gradient).
    scale: d^-1/2 if not given.  state: float32 [B, H, d, d], the state before
    the first token (rows are k's features), or None.  state_out, the state
    behind the last, is returned with ``final=True`` (or if given), else None.
    seg_offsets: packed sequences in [T, H, d], host numbers or a
    :class:`SegTable`; the states are then [nseg, H, d, d].  saved: with
    ``save=True``, what spares the backward one pass over k and v, else None
    (a workspace then, allocated unless given)."""
    c = _Call(q, log_decay, scale, seg_offsets)
    hq, hk, hv = c.heads(q, "q"), c.heads(k, "k"), c.heads(v, "v")
    c.state(state, "state")
    lib = _lib.load()
    need = int(lib.adaln_lin_attn_states_bytes(*c.sizes(0)[:-1]))
    with _on(c.dev, stream):
        o, ho = c.out(o, q, "o")
        if final or state_out is not None:
            state_out = c.new_state(state_out, "state_out", q)
        states, wbytes = _workspace(saved, need, q)
        rc = lib.adaln_lin_attn_fwd(
            _ref(hq), _ref(hk), _ref(hv), _ptr(log_decay), c.scale,
            _ptr(state), _ref(ho), _ptr(state_out), _ptr(states), wbytes,
            *c.sizes(stream))
    _lib.check(rc, "adaln_lin_attn_fwd")
    return o, state_out, states if save else None


def lin_attn_bwd_workspace_bytes(saved: bool, B: int, N: int, H: int, d: int,
                                 dtype: torch.dtype, seg_offsets=None) -> int:
    return _bytes(_lib.load().adaln_lin_attn_bwd_workspace_bytes, seg_offsets,
                  B, N, H, d, dtype, int(saved))


def lin_attn_bwd(do, q, k, v, log_decay: torch.Tensor, *,
                 scale: Optional[float] = None,
                 state: Optional[torch.Tensor] = None,
                 saved: Optional[torch.Tensor] = None,
                 dstate_out: Optional[torch.Tensor] = None, seg_offsets=None,
                 dq=None, dk=None, dv=None,
                 dstate: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None):
    """Backward of :func:`lin_attn_fwd`; returns (dq, dk, dv, dstate), the last
    None unless a state was given.  dstate_out: the gradient of state_out, or
    None.  saved: as the forward of the same sizes returned it, or None (the
    states are computed again).  The workspace (bytes from
    :func:`lin_attn_bwd_workspace_bytes`) is allocated if not given."""
    c = _Call(q, log_decay, scale, seg_offsets)
    hq, hk, hv = c.heads(q, "q"), c.heads(k, "k"), c.heads(v, "v")
    hdo = c.heads(do, "do")
    c.state(state, "state")
    c.state(dstate_out, "dstate_out")
    lib = _lib.load()
    sizes = c.sizes(0)[:-1]
    if saved is not None:
        kept, _ = _workspace(saved, 0, q)
        need = int(lib.adaln_lin_attn_states_bytes(*sizes))
        if kept.numel() * kept.element_size() < need:
            raise ValueError(f"saved has {kept.numel() * kept.element_size()} "
                             f"bytes, the forward of these sizes saves {need}")
    need = int(lib.adaln_lin_attn_bwd_workspace_bytes(int(saved is not None),
                                                      *sizes))
    with _on(c.dev, stream):
        dq, hdq = c.out(dq, q, "dq")
        dk, hdk = c.out(dk, k, "dk")
        dv, hdv = c.out(dv, v, "dv")
        if state is not None or dstate is not None:
            dstate = c.new_state(dstate, "dstate", q)
        workspace, wbytes = _workspace(workspace, need, q)
        rc = lib.adaln_lin_attn_bwd(
            _ref(hdo), _ref(hq), _ref(hk), _ref(hv), _ptr(log_decay), c.scale,
            _ptr(state), _ptr(saved), _ptr(dstate_out), _ref(hdq), _ref(hdk),
            _ref(hdv), _ptr(dstate), _ptr(workspace), wbytes,
            *c.sizes(stream))
    _lib.check(rc, "adaln_lin_attn_bwd")
    return dq, dk, dv, dstate


def lin_attn_step(q, k, v, log_decay: torch.Tensor, state: torch.Tensor, *,
                  scale: Optional[float] = None,
                  o: Optional[torch.Tensor] = None,
                  state_out: Optional[torch.Tensor] = None, stream=None):
    """One token of each sample: q, k, v [B, H, d], state float32
    [B, H, d, d], moved on in place unless state_out is given; returns
    (o, state_out)."""
    c = _Call(q, log_decay, scale, None)
    if c.four:
        raise ValueError(f"q must be [B, H, d], got shape {tuple(q.shape)}")
    c.seqs = B = q.shape[0]
    hq, hk, hv = c.heads(q, "q"), c.heads(k, "k"), c.heads(v, "v")
    _check(state, "state", (B, c.H, c.d, c.d), F32, c.dev)
    if state_out is None:
        state_out = state
    else:
        c.state(state_out, "state_out")
    lib = _lib.load()
    with _on(c.dev, stream):
        o, ho = c.out(o, q, "o")
        # [B, H, d]: the first dimension is the samples', there are no tokens
        for t in (hq, hk, hv, ho):
            t.batch_stride = t.token_stride
        rc = lib.adaln_lin_attn_step(
            _ref(hq), _ref(hk), _ref(hv), _ptr(log_decay), c.scale,
            _ptr(state), _ref(ho), _ptr(state_out), B, c.H, c.d, c.code,
            _stream(c.dev, stream))
    _lib.check(rc, "adaln_lin_attn_step")
    return o, state_out
