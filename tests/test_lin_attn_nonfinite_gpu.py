"""Linear attention, one token of which is infinite or no number: that it spoils
what the formulas let it reach, and nothing else.  An output goes by its own and
earlier tokens, and so does dq; dk and dv by their own and later ones.  All others
stay as they are, bit by bit: tokens, features, heads, samples and sequences."""

import pytest
import torch

import adaln_fwd_amd as A
from tests.test_lin_attn_gpu import _make

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
NAMES = ("q", "k", "v", "do")
# what each result is made of, x_t . sum of y_s z_s^T: x spoils its own token, y
# every feature from its token on, z its own feature from its token on
MADE = {"o": ("q", "k", "v"), "dq": ("do", "v", "k"), "dk": ("v", "do", "q"),
        "dv": ("k", "q", "do")}


def _run(ins, decay, tab=None):
    q, k, v, do = ins
    o, _, saved = A.lin_attn_fwd(q, k, v, decay, save=True, seg_offsets=tab)
    dq, dk, dv, _ = A.lin_attn_bwd(do, q, k, v, decay, saved=saved,
                                   seg_offsets=tab)
    return {"o": o, "dq": dq, "dk": dk, "dv": dv}


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N", [120, 700])   # whole, and cut in stretches
@pytest.mark.parametrize("d", [24, 64, 72, 128])
@pytest.mark.parametrize("value", [float("nan"), float("-inf")], ids=str)
def test_samples(dt, N, d, value):
    ins = [t.cuda() for t in _make(2, N, 3, d, dt)[:4]]
    decay = torch.tensor([-0.5, -0.01, 0.0], device="cuda")
    want = _run(ins, decay)
    for at in (0, 37, 63, 64, N // 2, N - 1):
        for i, name in enumerate(NAMES):
            for f in (5, d - 2):
                bad = [t.clone() for t in ins]
                bad[i][1, at, 1, f] = value
                print(f"[nonfinite] {name} of token {at}, {f}", flush=True)
                for n, got in _run(bad, decay).items():
                    hit = torch.zeros_like(got, dtype=torch.bool)
                    reach = slice(at, N) if n in ("o", "dq") else \
                        slice(0, at + 1)
                    if name in MADE[n]:
                        role = MADE[n].index(name)
                        hit[1, at if role == 0 else reach, 1,
                            f if role == 2 else slice(None)] = True
                    assert not got[hit].isfinite().any(), n
                    assert torch.equal(got[~hit], want[n][~hit]), n


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_packed_sequences(dt):
    off = [0, 50, 51, 380, 400]
    ins = [t[0].cuda() for t in _make(1, 400, 3, 64, dt)[:4]]
    decay = torch.tensor([-0.5, -0.01, 0.0], device="cuda")
    want = _run(ins, decay, off)
    for a, b in zip(off, off[1:]):
        keep = torch.ones(400, dtype=torch.bool, device="cuda")
        keep[a:b] = False
        for i in range(4):
            bad = [t.clone() for t in ins]
            bad[i][a:b] = float("nan")
            for n, got in _run(bad, decay, off).items():
                assert torch.equal(got[keep], want[n][keep]), n


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_padding_behind_a_sample(dt):
    """Samples of different lengths in one tensor, NaN behind their ends."""
    B, N, d = 3, 100, 64
    ins = [t.cuda() for t in _make(B, N, 2, d, dt)[:4]]
    decay = torch.tensor([-0.2, -0.01], device="cuda")
    want = _run(ins, decay)
    for b, n in enumerate((1, 45, 97)):
        for t in ins[:3]:
            t[b, n:] = float("nan")
    got = _run(ins, decay)
    for b, n in enumerate((1, 45, 97)):
        for name in ("o", "dq"):
            assert torch.equal(got[name][b, :n], want[name][b, :n])
            assert not got[name][b, n:].isfinite().any()
