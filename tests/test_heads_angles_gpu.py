"""Cosines and sines of the rotations, to a relative bound.

A pair (1, 0) rotates to (cos, sin) exactly as the kernel has them.  Each is
within 4 * 2^-24 of itself: the conversion of the phase to float32 and its
scaling round once each and sin x moves by at most as much as x relatively,
cos x by x tan x <= 0.79 of it; the polynomials round once at the end, and what
they add there (at most 0.1 of the sine, 0.44 of the cosine, four roundings or
fewer deep) brings the sum below 4.  On top of that stands what the frequency's
64-bit fraction of a turn rounds, half of 2^-64 turns per unit position and
axis, and the reference's float64 product, 2^-53 of the angle per axis."""

import math

import pytest
import torch

import adaln_fwd_amd as A

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"[heads] {msg}", flush=True)


def _cos_sin(pos, freqs, inverse=False):
    """[N, pairs] each, from float32 pairs (1, 0)."""
    N, pairs = pos.shape[0], freqs.shape[1]
    x = torch.zeros(1, N, 1, 2 * pairs)
    x[..., 0::2] = 1
    rotate = A.rope_bwd if inverse else A.rope_fwd
    y = rotate(x.cuda(), None, pos.cuda(), freqs)[0].cpu().double()[0, :, 0]
    return y[:, 0::2], (-1 if inverse else 1) * y[:, 1::2]


def _check(pos, freqs, inverse=False):
    f = torch.as_tensor(freqs)
    ang = pos.double() @ f
    size = pos.double().abs() @ f.abs()
    c, s = _cos_sin(pos, freqs, inverse)
    off = pos.double().abs().sum(-1, keepdim=True) * math.pi * 2.0 ** -64 \
        + 4 * 2.0 ** -53 * size
    for got, ref in ((c, ang.cos()), (s, ang.sin())):
        err = (got - ref).abs()
        bad = ~(err <= 4 * 2.0 ** -24 * ref.abs() + off)
        assert not bad.any(), (int(bad.sum()), float((err / ref.abs()).max()))


@pytest.mark.parametrize("inverse", [False, True])
def test_small_angles_keep_their_digits(inverse):
    """The first positions at the default frequencies of 64 and of 256 pairs,
    and far lower ones."""
    _say(f"small angles, inverse {inverse}")
    pos = torch.tensor([[0], [1], [-1], [2], [3], [7], [-64], [1000]],
                       dtype=torch.int32)
    for pairs in (64, 256):
        _check(pos, A.rope_freqs((pairs,)), inverse)
    low = 2.0 ** -torch.arange(3, 35, 0.25, dtype=torch.float64)
    _check(pos, low.reshape(1, -1).numpy(), inverse)


def test_angles_of_every_size():
    """Up to a few thousand turns, near the ends of the quarters too, where
    float64 angles leave the reference enough digits; by one axis and by sums
    over three."""
    _say("angles of every size")
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(-20000, 20000, (997, 1), generator=g,
                        dtype=torch.int32)
    _check(pos, torch.rand(1, 64, generator=g, dtype=torch.float64).numpy())
    quarters = torch.arange(-40, 41, dtype=torch.int32).reshape(-1, 1)
    near = math.pi / 4 * (1 + torch.tensor(
        [0.0] + [q * 2.0 ** -k for k in range(4, 36) for q in (-1, 1)[:1 + k % 2]]
        + [2.0 ** -36], dtype=torch.float64))
    _check(quarters, near.reshape(1, -1).numpy())
    pos = torch.randint(-2000, 2000, (500, 3), generator=g, dtype=torch.int32)
    dense = torch.rand(3, 64, generator=g, dtype=torch.float64) - 0.5
    _check(pos, dense.numpy())
