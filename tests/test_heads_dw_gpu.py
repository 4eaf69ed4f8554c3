"""The norms' weight gradients as whole numbers.

x is 1 or -1 everywhere, w = 1 and eps = 0, so r = 1 and xh = x; at position 0
nothing turns; dy is a whole number.  Then every partial sum of dw is a whole
number below 2^24, exact in float32 in any order, and dw is compared bit for
bit: no row may be missing or counted twice.  (d is a power of two, so that
the mean of d ones is 1; a mean of d whole numbers is exact too, and so dx is
a multiple of 1 / d, exact in float32.)"""

import pytest
import torch

import adaln_fwd_amd as A

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"[heads] {msg}", flush=True)


# B, N, Hq, Hk, d, layout, dtype: one workgroup without a second launch; one
# block per workgroup; several blocks per workgroup, the last one short; blocks
# of one token; heads of one vector and of 128
SIZES = [
    (1, 1, 1, 1, 64, "interleaved", "bf16"),
    (1, 3, 4, 2, 128, "half", "bf16"),
    (2, 5, 3, 1, 8, "interleaved", "bf16"),
    (1, 33, 7, 3, 128, "interleaved", "f32"),
    (5, 413, 6, 2, 64, "half", "bf16"),
    (1, 16391, 2, 1, 64, "interleaved", "bf16"),
    (1, 65537, 1, 1, 64, "half", "bf16"),
    (3, 27001, 2, 1, 8, "interleaved", "bf16"),
    (7, 3701, 3, 5, 32, "half", "f32"),
    (2, 9001, 1, 2, 512, "half", "f32"),
    (1, 20001, 2, 1, 512, "interleaved", "bf16"),
    (2, 4099, 40, 8, 128, "interleaved", "bf16"),
    (1500, 3, 5, 1, 16, "half", "f32"),
    (1, 1801, 96, 0, 128, "half", "bf16"),
    (1, 40009, 0, 4, 4, "interleaved", "f32"),
]


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_weight_gradients_miss_no_row(size):
    B, N, Hq, Hk, d, layout, dtype = size
    _say(f"whole dw {size}")
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(N + d)
    pos = torch.zeros(N, 1, dtype=torch.int32, device="cuda")
    freqs = A.rope_freqs((d // 2,))
    w = torch.ones(d, dtype=dt, device="cuda")

    def whole(H, lo, hi):
        return torch.randint(lo, hi + 1, (B, N, H, d), generator=g,
                             device="cuda", dtype=torch.int8).to(dt)

    x = [whole(H, 0, 1) * 2 - 1 for H in (Hq, Hk)]
    # of the first and the last token every head counts a thousandfold, which
    # bf16 holds as 1024 and no other row can make up for
    dy = [whole(H, -3, 3) for H in (Hq, Hk)]
    for t in dy:
        t[:, 0] = 1024
        t[:, -1] = -1024
    got = A.qk_norm_rope_bwd(*dy, *x, w, w, pos, freqs, eps=0.0, layout=layout)
    for dx, dw, a, b in zip(got[:2], got[2:], dy, x):
        t = a.double() * b.double()
        # (1024 B H of either end, 3 of the others: all sums below 2^24)
        assert not t.numel() or t.abs().sum((0, 1, 2)).max() < 2 ** 24
        assert torch.equal(dw.double(), t.sum((0, 1, 2)))
        want = a.double() - b.double() * t.mean(-1, keepdim=True)
        assert torch.equal(dx, want.float().to(dt))
