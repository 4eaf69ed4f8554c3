"""What the rotations and the query/key norms have to get exactly right:
features past the rotated ones, whatever they hold."""

import pytest
import torch

import adaln_fwd_amd as A

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _say(msg):
    print(f"[heads] {msg}", flush=True)


def _bits(t):
    return t.contiguous().view(torch.int16 if t.dtype is BF16 else torch.int32)


def _positions(N):
    return torch.arange(3, N + 3, dtype=torch.int32).reshape(N, 1).cuda()


# d, pairs, layout, dtype: the rotated part ends with a vector, inside one,
# and heads of an odd number of vectors
PARTS = [
    (64, 16, "interleaved", BF16), (64, 13, "interleaved", BF16),
    (72, 3, "interleaved", BF16), (64, 16, "half", BF16),
    (72, 8, "half", BF16), (512, 96, "half", BF16),
    (64, 16, "interleaved", F32), (64, 13, "interleaved", F32),
    (20, 1, "interleaved", F32), (64, 12, "half", F32), (36, 8, "half", F32),
    (512, 192, "interleaved", F32),
]

# infinities, quiet and signalling NaNs with and without a payload, both
# zeros, the smallest and the largest numbers, in bits
ODD_F32 = [0x7F800000, 0xFF800000, 0x7FC00000, 0xFFC12345, 0x7F800001,
           0xFFBFFFFF, 0x80000000, 0, 1, 0x80000001, 0x7F7FFFFF, 0xFF7FFFFF,
           0x3F800000]
ODD_BF16 = [0x7F80, 0xFF80, 0x7FC0, 0xFFC1, 0x7F81, 0xFFBF, 0x8000, 0, 1,
            0x8001, 0x7F7F, 0xFF7F, 0x3F80]


def _odd(shape, dtype, seed):
    table = torch.tensor(ODD_BF16 if dtype is BF16 else ODD_F32)
    g = torch.Generator().manual_seed(seed)
    i = torch.randint(0, len(table), shape, generator=g)
    if dtype is BF16:
        return table[i].to(torch.int32).to(torch.int16).view(BF16)
    return table[i].to(torch.int32).view(F32)


@pytest.mark.parametrize("d,pairs,layout,dtype", PARTS)
def test_features_past_the_rotated_ones_pass_through(d, pairs, layout, dtype):
    """Bit for bit, and without a trace in the rotated ones."""
    _say(f"pass through: {d} {pairs} {layout} {dtype}")
    B, N, Hq, Hk = 2, 37, 3, 2
    g = torch.Generator().manual_seed(d + pairs)
    pos = _positions(N)
    freqs = A.rope_freqs((pairs,))
    x = [torch.randn(B, N, H, d, generator=g).to(dtype) for H in (Hq, Hk)]
    odd = [t.clone() for t in x]
    for t in odd:
        t[..., 2 * pairs:] = _odd(t[..., 2 * pairs:].shape, dtype, pairs)
    for rotate in (A.rope_fwd, A.rope_bwd):
        clean = rotate(*[t.cuda() for t in x], pos, freqs, layout=layout)
        got = rotate(*[t.cuda() for t in odd], pos, freqs, layout=layout)
        for y, c, t in zip(got, clean, odd):
            assert torch.equal(_bits(y[..., 2 * pairs:]).cpu(),
                               _bits(t[..., 2 * pairs:]))
            assert torch.equal(_bits(y[..., :2 * pairs]),
                               _bits(c[..., :2 * pairs]))


@pytest.mark.parametrize("d,pairs,layout,dtype", PARTS)
def test_norms_keep_unrotated_features_apart(d, pairs, layout, dtype):
    """An infinite weight, input or gradient of one feature that is not
    rotated shows up in that feature alone (and in what the norm's sums carry
    everywhere)."""
    _say(f"norm past the rotated ones: {d} {pairs} {layout} {dtype}")
    N, H = 29, 3
    g = torch.Generator().manual_seed(d + pairs)
    pos = _positions(N)
    freqs = A.rope_freqs((pairs,))
    x, dy = [torch.randn(1, N, H, d, generator=g).to(dtype).cuda()
             for _ in range(2)]
    w = torch.ones(d, dtype=dtype, device="cuda")
    inf = float("inf")

    def fwd(x, w):
        return A.qk_norm_rope_fwd(x, None, w, None, pos, freqs,
                                  layout=layout)[0]

    def bwd(dy, x):
        return A.qk_norm_rope_bwd(dy, None, x, None, w, None, pos, freqs,
                                  layout=layout)

    y, dw = fwd(x, w), bwd(dy, x)[2]
    for j in sorted({2 * pairs, 2 * pairs + 1, d // 2 + pairs, d - 2, d - 1}):
        rest = torch.arange(d, device="cuda") != j
        for value in (inf, float("nan")):
            v = w.clone()
            v[j] = value
            got = fwd(x, v)
            assert torch.equal(got[..., rest], y[..., rest]), j
            assert not torch.isfinite(got[..., j]).any()
        # 1 / sqrt(inf) = 0: the head's other features are zeros
        u = x.clone()
        u[0, 5, 1, j] = -inf
        got = fwd(u, w)
        assert (got[0, 5, 1, rest] == 0).all() and got[0, 5, 1, j].isnan()
        got[0, 5, 1] = y[0, 5, 1]
        assert torch.equal(got, y)
        # t is infinite in feature j of one head alone, and so is dw
        u = dy.clone()
        u[0, 7, 2, j] = inf
        got = bwd(u, x)
        assert torch.equal(got[2][rest], dw[rest]) and got[2][j].isinf()
        # zeros keep their sign, beside negative and positive features
        u = x.clone()
        u[..., j] = -0.0
        assert fwd(u, w)[..., j].signbit().all()
