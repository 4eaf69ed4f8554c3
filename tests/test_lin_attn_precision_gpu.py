"""How exactly the linear attention carries its state within a long stretch of a
bf16 sequence, where later products see it and nobody else: by sums that cancel.

Within 64 tokens the decay is 1/3.  Of every 128 tokens the first 32 bring a
product x y^T into the state, with y three times whole numbers; 64 tokens later
the same x come with minus those numbers, which cancels them but for the rounding
of the decay; the last 32 look at what is left.  So what they see is the error of
the state, and no rounding of the output or of the products covers it.

Tolerance.  A term's way into the state: the power, its two products, the rest of
three bf16, the multiplication by the chunks' decay and the sum: six roundings of
at most 2^-24 each, independent of each other and of other terms'.  Their 2-norm
is at most sqrt(6) * 2^-24 of the 2-norm of the terms; twice that is allowed.
(A decayed value given as two bf16 is off by up to 2^-17, by 2^-19 in the mean
square.)"""

import math

import pytest
import torch

import adaln_fwd_amd as A

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("d", [32, 128])
@pytest.mark.parametrize("which", ["o", "dq", "dv", "dk"])
def test_a_state_within_a_stretch_takes_float32_values(which, d):
    # sequences times heads, for a stretch of 1024 tokens
    N, H = (4096, 128) if d == 32 else (8192, 64)
    n = A.lin_attn_states_bytes(1, N, H, d, BF16) // (4 * H * d * d)
    assert 1 < n <= N // 512                 # cut, in stretches of many chunks
    g = torch.Generator().manual_seed(d)
    at = torch.arange(N) // 32 % 4
    look = torch.randn(N, 2, d, generator=g) * (at == 3)[:, None, None]
    same = torch.randn(N // 128, 32, 2, d, generator=g)
    whole = torch.randint(-40, 41, (N // 128, 32, 2, d), generator=g).float()
    x, y = torch.zeros(2, N, 2, d)
    for part, times in ((0, 3), (2, -1)):
        x[at == part] = same.flatten(0, 1)
        y[at == part] = times * whole.flatten(0, 1)
    look, x, y = (t.to(BF16) for t in (look, x, y))
    decay = torch.full((H,), -math.log(3) / 64)

    # every head but the checked two is zero; backwards in time the tokens of
    # the two gradients that run so
    def put(t):
        full = torch.zeros(1, N, H, d, dtype=BF16)
        full[0, :, [0, H - 1]] = t.flip(0) if which in ("dv", "dk") else t
        return full.cuda()

    look_, x_, y_ = put(look), put(x), put(y)
    zero = torch.zeros_like(x_)
    q, k, v, do = {"o": (look_, x_, y_, zero), "dq": (zero, y_, x_, look_),
                   "dv": (x_, look_, zero, y_),
                   "dk": (y_, zero, look_, x_)}[which]
    if which == "o":
        got, _, _ = A.lin_attn_fwd(q, k, v, decay.cuda(), scale=1.0)
    else:
        got = A.lin_attn_bwd(do, q, k, v, decay.cuda(), scale=1.0)[
            ("dq", "dk", "dv").index(which)]
    got = got[0, :, [0, H - 1]].double().cpu()
    if which in ("dv", "dk"):
        got = got.flip(0)

    t = torch.nonzero(at == 3).flatten()
    gap = t[:, None] - torch.arange(N)
    power = torch.where(gap >= 0, torch.exp(decay[0].double() *
                                            gap.clamp(min=0)), 0.0)
    for h in range(2):
        a, b, c = (s[:, h].double() for s in (look[t], x, y))
        w = (a @ b.T) * power
        want = w @ c
        terms = ((a * a) @ (b * b).T * power ** 2) @ (c * c)
        off = float((got[t, h] - want).norm() / terms.sum().sqrt())
        print(f"[state] {which} {d}: {off * 2 ** 24:.2f} * 2^-24", flush=True)
        assert off <= 2 * math.sqrt(6) * 2.0 ** -24
