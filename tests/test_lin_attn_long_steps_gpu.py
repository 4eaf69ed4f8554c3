"""Linear attention, thousands of single tokens from state to state: the decay of
a slowly forgetting head does not drift from that of a whole sequence.

Tolerance, of the state's 2-norm.  Each of n steps rounds the decayed state, and
the sum with k v^T, by at most 2^-24 and independently of the other steps: at most
sqrt(2 n) * 2^-24 together, and twice that is allowed.  The decay's own error goes
with every step: one of 2^-23 of 1 - l, n |log_decay| * 2^-23.  (l as a rounded
number is off by up to 2^-25, and n * 2^-25 in the end, 1.2e-4 of 4096 tokens.)"""

import pytest
import torch

import adaln_fwd_amd as A

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
N, B, H, D = 4096, 2, 8, 16


def _allow(decay, n=N):
    return 2 * (2 * n) ** 0.5 * 2.0 ** -24 + n * decay.abs() * 2.0 ** -23


def _norm(x):
    """2-norm of each head's elements."""
    return x.transpose(0, 1).flatten(1).square().sum(1).sqrt()


def _decay():
    # heads that remember some 3000 to 4100 tokens, as log1p gives them
    return torch.log1p(-1 / torch.linspace(3000, 4096, H)).float()


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_a_state_is_forgotten_at_its_rate(dt):
    g = torch.Generator().manual_seed(3)
    S0 = torch.randn(B, H, D, D, generator=g)
    decay = _decay()
    z = torch.zeros(B, H, D, device="cuda", dtype=dt)
    S, dec = S0.cuda(), decay.cuda()
    for _ in range(N):
        A.lin_attn_step(z, z, z, dec, S)
    want = S0.double() * torch.exp(decay.double() * N)[:, None, None]
    off = _norm(S.double().cpu() - want) / _norm(want)
    print(f"[steps] {off.tolist()}", flush=True)
    assert (off <= _allow(decay)).all()


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
def test_steps_of_a_whole_sequence(dt):
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(B, N, H, D, generator=g).to(dt) for _ in range(3))
    S0 = 60 * torch.randn(B, H, D, D, generator=g)
    decay = _decay()
    S, dec = S0.cuda(), decay.cuda()
    qs, ks, vs = (t.cuda() for t in (q, k, v))
    for t in range(N):
        o, _ = A.lin_attn_step(qs[:, t], ks[:, t], vs[:, t], dec, S)
    # the state behind, and the last token's output
    w = torch.exp(decay.double() * (N - 1 - torch.arange(N))[:, None])
    want = torch.exp(decay.double() * N)[:, None, None] * S0.double() + \
        torch.matmul((k.double() * w[..., None]).permute(0, 2, 3, 1),
                     v.double().permute(0, 2, 1, 3))
    off = _norm(S.double().cpu() - want) / _norm(want)
    print(f"[steps] {off.tolist()}", flush=True)
    assert (off <= _allow(decay)).all()
    last = D ** -0.5 * torch.matmul(q[:, -1, :, None].double(), want)[:, :, 0]
    half = 2.0 ** -8 if dt == BF16 else 2.0 ** -24
    # D products and sums more, and half a step of the type
    off = _norm(o.double().cpu() - last) / _norm(last)
    assert (off <= _allow(decay) + (D + 1) * 2.0 ** -24 + half).all()


def test_a_step_keeps_a_decays_digits():
    """One step of any decay: the power's error, at most 2^-23 of it, and one
    rounding."""
    g = torch.cat([-torch.logspace(-9, 1.9, 150), torch.tensor([-0.5, 0.0])])
    H = g.numel()
    S0 = torch.randn(1, H, D, D, generator=torch.Generator().manual_seed(5))
    z = torch.zeros(1, H, D, device="cuda")
    _, S = A.lin_attn_step(z, z, z, g.cuda(), S0.cuda())
    want = S0.double() * torch.exp(g.double())[:, None, None]
    # (2^-126: the least number with all its digits)
    allow = 3 * 2.0 ** -24 * want.abs() + 2.0 ** -126
    assert ((S.double().cpu() - want).abs() <= allow).all()


def test_without_memory_a_step_leaves_its_own_token_alone():
    S = torch.randn(1, 2, D, D, device="cuda")
    k, v = (torch.randn(1, 2, D, device="cuda") for _ in range(2))
    decay = torch.full((2,), float("-inf"), device="cuda")
    A.lin_attn_step(k, k, v, decay, S)
    assert torch.equal(S, k[..., None] * v[..., None, :])
