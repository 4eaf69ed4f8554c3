"""Binding of the rotary positions and the query/key norms (adaln_rope_*,
adaln_qk_norm_rope_*) for torch tensors.

q and k are [B, N, H, d], or [T, H, d] for packed tokens, in any memory order
that keeps a head's features contiguous: views of one projection's output, or
transposed [B, H, N, d].  Checks, streams and allocation are those of
:mod:`adaln_fwd_amd.ops`."""

from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import numpy as np
import torch

from . import _lib
from .ops import _check, _code, _on, _ptr, _stream

_LAYOUTS = {"interleaved": 0, "half": 1}


def rope_freqs(pairs: Sequence[int], theta: float = 10000.0) -> np.ndarray:
    """Frequencies of consecutive runs of pairs, one run per axis: axis a
    turns its pairs[a] pairs at theta^(-i / pairs[a]) radians per unit
    position, i = 0, 1, ...  Returns float64 [len(pairs), sum(pairs)], zero
    where an axis does not turn a pair."""
    pairs = [int(p) for p in pairs]
    if not pairs or min(pairs) < 0 or sum(pairs) < 1:
        raise ValueError(f"pairs must be counts of rotated pairs, got {pairs}")
    out = np.zeros((len(pairs), sum(pairs)))
    at = 0
    for a, p in enumerate(pairs):
        if p:
            out[a, at:at + p] = float(theta) ** (-np.arange(p) / p)
        at += p
    return out


def _wrong(t, name, shape, dtype, device):
    """Raises for what _heads found wrong with a tensor."""
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor, got {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.dim() != len(shape) or t.shape[:-2] != shape[:-2] \
            or t.shape[-1] != shape[-1]:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected "
                         f"{tuple(shape[:-2]) + ('H', shape[-1])}")
    raise ValueError(f"{name}: the features of a head must be contiguous")


class _Call:
    """What the four entry points share: shapes, device, the rotation and the
    descriptors of the inputs."""

    __slots__ = ("dev", "index", "dt", "code", "shape", "four", "B", "N", "d",
                 "q", "k", "Hq", "Hk", "freqs", "rot")

    def __init__(self, q, k, pos, freqs, layout):
        ref = q if q is not None else k
        if ref is None:
            raise ValueError("q and k are both None")
        if not isinstance(ref, torch.Tensor):
            raise TypeError("q and k must be torch.Tensors")
        shape = ref.shape
        if len(shape) not in (3, 4):
            raise ValueError("q and k must be [B, N, H, d] or [T, H, d], got "
                             f"shape {tuple(shape)}")
        self.dev, self.dt = ref.device, ref.dtype
        self.index = ref.get_device()
        self.code = _code(ref)
        self.shape = shape
        self.four = len(shape) == 4
        self.B = shape[0] if self.four else 1
        self.N = N = shape[-3]
        self.d = shape[-1]
        self.Hq = self.Hk = 0
        self.q = self.k = None
        if q is not None:
            self.q, self.Hq = self.heads(q, "q"), q.shape[-2]
        if k is not None:
            self.k, self.Hk = self.heads(k, "k"), k.shape[-2]
        if layout not in _LAYOUTS:
            raise ValueError("layout must be 'interleaved' or 'half', got "
                             f"{layout!r}")
        if isinstance(freqs, torch.Tensor):
            if freqs.device.type != "cpu":
                raise ValueError("freqs is read on the host: pass a CPU "
                                 "tensor or an array")
            freqs = freqs.numpy()
        # contiguous float64; the caller's own array when it already is
        self.freqs = freqs = np.ascontiguousarray(freqs, dtype=np.float64)
        if freqs.ndim != 2:
            raise ValueError("freqs must be [axes, pairs], got shape "
                             f"{freqs.shape}")
        axes, pairs = freqs.shape
        if not isinstance(pos, torch.Tensor):
            raise TypeError("pos must be a torch.Tensor")
        shared = pos.dim() == 2 or not self.four
        _check(pos, "pos", (N, axes) if shared else (self.B, N, axes),
               torch.int32, self.dev)
        self.rot = _lib.Rotation(_ptr(pos), 0 if shared else N * axes,
                                 freqs.__array_interface__["data"][0], axes,
                                 pairs, _LAYOUTS[layout])

    def heads(self, t, name, like=None) -> Optional[_lib.Heads]:
        """Descriptor of one tensor of heads, or None for None."""
        if t is None:
            return None
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        shape, st = t.shape, t.stride()
        if like is not None and shape != like.shape:
            raise ValueError(f"{name} has shape {tuple(shape)}, expected "
                             f"{tuple(like.shape)}")
        # one condition for calls that are right; which one failed comes after
        if not (t.is_cuda and t.get_device() == self.index
                and t.dtype is self.dt and len(shape) == len(self.shape)
                and shape[-1] == self.d and shape[-3] == self.N
                and shape[0] == self.shape[0] and (st[-1] == 1 or self.d == 1)):
            _wrong(t, name, self.shape, self.dt, self.dev)
        return _lib.Heads(_ptr(t), st[0] if self.four else 0, st[-3], st[-2])

    def out(self, t, like, name):
        """An output and its descriptor: as given, or a contiguous one."""
        if like is None:
            if t is not None:
                raise ValueError(f"{name} was given for a missing input")
            return None, None
        if t is not None:
            return t, self.heads(t, name, like)
        t = torch.empty_like(like, memory_format=torch.contiguous_format)
        row = like.shape[-2] * self.d
        return t, _lib.Heads(_ptr(t), self.N * row, row, self.d)

    def sizes(self, stream):
        return (self.B, self.N, self.Hq, self.Hk, self.d, self.code,
                _stream(self.dev, stream))


def _ref(h):
    return None if h is None else ctypes.byref(h)


def _rope(entry, q, k, pos, freqs, layout, q_out, k_out, stream):
    c = _Call(q, k, pos, freqs, layout)
    lib = _lib.load()
    with _on(c.dev, stream):
        q_out, ho = c.out(q_out, q, "q_out")
        k_out, hk = c.out(k_out, k, "k_out")
        rc = getattr(lib, entry)(_ref(c.q), _ref(c.k), ctypes.byref(c.rot),
                                 _ref(ho), _ref(hk), *c.sizes(stream))
    _lib.check(rc, entry)
    return q_out, k_out


def rope_fwd(q, k, pos: torch.Tensor, freqs, *, layout: str = "interleaved",
             q_out=None, k_out=None, stream=None):
    """Rotary positions with several axes on q and k (either may be None);
    returns (q_out, k_out).

    pos: int32 [N, axes], shared by the samples, or [B, N, axes]; freqs: host
    float64 [axes, pairs] (:func:`rope_freqs`): pair j of token n turns by
    sum_a pos[n, a] * freqs[a, j].  layout: pairs (2j, 2j+1) ("interleaved")
    or (j, j + pairs) ("half"); features past 2 * pairs pass through.  An
    output may be its own input."""
    return _rope("adaln_rope_fwd", q, k, pos, freqs, layout, q_out, k_out,
                 stream)


def rope_bwd(dq_out, dk_out, pos: torch.Tensor, freqs, *,
             layout: str = "interleaved", dq=None, dk=None, stream=None):
    """Backward of :func:`rope_fwd`; returns (dq, dk)."""
    return _rope("adaln_rope_bwd", dq_out, dk_out, pos, freqs, layout, dq, dk,
                 stream)


def _weights(c, wq, wk):
    if c.q is not None:
        _check(wq, "wq", (c.d,), c.dt, c.dev)
    if c.k is not None:
        _check(wk, "wk", (c.d,), c.dt, c.dev)


def _dw(dw, w, name, x, c):
    """A weight's gradient: as given, or a new one; None for a missing x."""
    if x is None:
        if dw is not None:
            raise ValueError(f"{name} was given for a missing input")
        return None
    if dw is None:
        return w.new_empty(c.d, dtype=torch.float32)
    _check(dw, name, (c.d,), torch.float32, c.dev)
    return dw


def qk_norm_rope_fwd(q, k, wq, wk, pos: torch.Tensor, freqs, *,
                     eps: float = 1e-6, layout: str = "interleaved",
                     q_out=None, k_out=None, stream=None):
    """The RMS norm of each head of q and k with weights wq, wk [d], then the
    rotation of :func:`rope_fwd`, in one pass; returns (q_out, k_out)."""
    c = _Call(q, k, pos, freqs, layout)
    _weights(c, wq, wk)
    lib = _lib.load()
    with _on(c.dev, stream):
        q_out, ho = c.out(q_out, q, "q_out")
        k_out, hk = c.out(k_out, k, "k_out")
        rc = lib.adaln_qk_norm_rope_fwd(
            _ref(c.q), _ref(c.k), _ptr(wq), _ptr(wk), eps, ctypes.byref(c.rot),
            _ref(ho), _ref(hk), *c.sizes(stream))
    _lib.check(rc, "adaln_qk_norm_rope_fwd")
    return q_out, k_out


def qk_norm_rope_bwd_workspace_bytes(B: int, N: int, Hq: int, Hk: int, d: int,
                                     dtype: torch.dtype) -> int:
    from .ops import _DTYPES
    return int(_lib.load().adaln_qk_norm_rope_bwd_workspace_bytes(
        B, N, Hq, Hk, d, _DTYPES.get(dtype, -1)))


def qk_norm_rope_bwd(dq_out, dk_out, q, k, wq, wk, pos: torch.Tensor, freqs, *,
                     eps: float = 1e-6, layout: str = "interleaved", dq=None,
                     dk=None, dwq: Optional[torch.Tensor] = None,
                     dwk: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """Backward of :func:`qk_norm_rope_fwd` from its inputs and the gradients
    of its outputs; returns (dq, dk, dwq, dwk), the weights' gradients in
    float32.  The workspace (bytes from
    :func:`qk_norm_rope_bwd_workspace_bytes`) is allocated if not given."""
    c = _Call(q, k, pos, freqs, layout)
    _weights(c, wq, wk)
    if (dq_out is None) != (q is None) or (dk_out is None) != (k is None):
        raise ValueError("a gradient and its input must both be given")
    hq, hk = c.heads(dq_out, "dq_out", q), c.heads(dk_out, "dk_out", k)
    lib = _lib.load()
    need = int(lib.adaln_qk_norm_rope_bwd_workspace_bytes(
        c.B, c.N, c.Hq, c.Hk, c.d, c.code))
    with _on(c.dev, stream):
        dq, ho = c.out(dq, q, "dq")
        dk, ko = c.out(dk, k, "dk")
        dwq = _dw(dwq, wq, "dwq", q, c)
        dwk = _dw(dwk, wk, "dwk", k, c)
        if workspace is None:
            wbytes = max(need, 1)
            workspace = (q if q is not None else k).new_empty(
                wbytes, dtype=torch.uint8)
        else:
            if workspace.device != c.dev or not workspace.is_contiguous():
                raise ValueError("workspace must be a contiguous tensor on "
                                 f"{c.dev}")
            wbytes = workspace.numel() * workspace.element_size()
        rc = lib.adaln_qk_norm_rope_bwd(
            _ref(hq), _ref(hk), _ref(c.q), _ref(c.k), _ptr(wq), _ptr(wk), eps,
            ctypes.byref(c.rot), _ref(ho), _ref(ko), _ptr(dwq), _ptr(dwk),
            _ptr(workspace), wbytes, *c.sizes(stream))
    _lib.check(rc, "adaln_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk
