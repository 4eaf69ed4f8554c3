"""Linear attention, one token of which is infinite or no number: which outputs
and gradients that may spoil, and that all the others stay as they are, bit by
bit.  An output goes by its own and earlier tokens, and so does dq; dk and dv by
their own and later ones.  Up to 31 tokens on the other side may be spoilt too;
other samples, heads and packed sequences never are."""

import pytest
import torch

import adaln_fwd_amd as A
from tests.test_lin_attn_gpu import _make

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
NAMES = ("q", "k", "v", "do")


def _run(ins, decay, tab=None):
    q, k, v, do = ins
    o, _, saved = A.lin_attn_fwd(q, k, v, decay, save=True, seg_offsets=tab)
    dq, dk, dv, _ = A.lin_attn_bwd(do, q, k, v, decay, saved=saved,
                                   seg_offsets=tab)
    return {"o": o, "dq": dq, "dk": dk, "dv": dv}


def _same(got, want, keep):
    for n in want:
        a, b = got[n][keep[n]], want[n][keep[n]]
        assert torch.equal(a, b), n


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N", [120, 700])   # whole, and cut in stretches
@pytest.mark.parametrize("d", [64, 72])
@pytest.mark.parametrize("value", [float("nan"), float("-inf")], ids=str)
def test_samples(dt, N, d, value):
    ins = [t.cuda() for t in _make(2, N, 3, d, dt)[:4]]
    decay = torch.tensor([-0.5, -0.01, 0.0], device="cuda")
    want = _run(ins, decay)
    for at in (0, 37, N // 2, N - 1):
        keep = {n: torch.ones(2, N, 3, dtype=torch.bool, device="cuda")
                for n in want}
        for n in want:
            gone = slice(max(0, at - 31), N) if n in ("o", "dq") else \
                slice(0, at + 32)
            keep[n][1, gone, 1] = False
        for i, name in enumerate(NAMES):
            bad = [t.clone() for t in ins]
            bad[i][1, at, 1, 5] = value
            print(f"[nonfinite] {name} of token {at}", flush=True)
            _same(_run(bad, decay), want, keep)


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
            _same(_run(bad, decay, off), want, {n: keep for n in want})
