"""Linear attention where its launches and offsets reach furthest: more sequences
and heads than one launch takes, gradients past 32-bit offsets, and single tokens
in a captured graph from the state of a captured prompt.

Tolerances: those of test_lin_attn_gpu.py."""

import pytest
import torch

import adaln_fwd_amd as A
from tests import near
from tests import ref_lin_attn as R
from tests.test_lin_attn_gpu import HALF, U, _make, _near

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dt,d", [(BF16, 8), (F32, 4)], ids=["bf16", "f32"])
def test_more_sequences_and_heads_than_a_launch_takes(dt, d):
    """One token each, 2^20 + 12 of them, with states: S = l S0 + k v^T."""
    B, H, c = (1 << 18) + 3, 4, 0.4
    print(f"[reach] {B} samples of {H} heads of {d}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(d)

    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")

    q, k, v, do = (normal(B, 1, H, d).to(dt) for _ in range(4))
    S0, dS = normal(B, H, d, d), normal(B, H, d, d)
    decay = torch.tensor([-0.3, 0.0, -2.0, float("-inf")], device="cuda")
    o, last, _ = A.lin_attn_fwd(q, k, v, decay, scale=c, state=S0, final=True)
    dq, dk, dv, d0 = A.lin_attn_bwd(do, q, k, v, decay, scale=c, state=S0,
                                    dstate_out=dS)
    # a term: a power and its exponent (1 + |log_decay|) roundings, sums and
    # products 4 d + 64; of bf16 three numbers as two bf16 each
    lam = decay.double().exp()
    rel = (4 * d + 64) * U * (1 + decay.abs().clamp(max=100).double())
    more = 3 * 2.0 ** -16 if dt == BF16 else 0.0
    for a in (0, (1 << 18) - 2000, B - 2000):
        i = slice(a, min(B, a + 2000))
        s0, ds = S0[i].double(), dS[i].double()
        qi, ki, vi, oi = (t[i, 0].double() for t in (q, k, v, do))

        def check(got, terms, r, what):
            """terms: the last dimension is summed."""
            want, size = terms.sum(-1), terms.abs().sum(-1)
            r = r.view((1, H) + (1,) * (want.dim() - 2)) + more
            half = HALF[dt] if got.dtype == dt else U
            near.check(got, want, r * size + half * (want.abs() + r * size),
                       what)

        kv = ki[..., :, None] * vi[..., None, :]
        qo = c * qi[..., :, None] * oi[..., None, :]
        ls = lam[:, None, None]
        check(last[i], torch.stack([ls * s0, kv], -1), rel, "state")
        check(d0[i], ls[..., None] * torch.stack([ds, qo], -1), rel, "dstate")
        both = torch.cat([ls * s0, kv], -2)             # [b, h, 2 d, d]
        twice = torch.cat([ls * s0, kv], -1)            # [b, h, d, 2 d]
        check(o[i, 0], c * (torch.cat([qi, qi], -1)[..., None] * both)
              .transpose(-1, -2), rel, "o")
        check(dq[i, 0], c * twice * torch.cat([oi, oi], -1)[..., None, :], rel,
              "dq")
        both, twice = torch.cat([ds, qo], -2), torch.cat([ds, qo], -1)
        check(dk[i, 0], twice * torch.cat([vi, vi], -1)[..., None, :], rel,
              "dk")
        check(dv[i, 0], (torch.cat([ki, ki], -1)[..., None] * both)
              .transpose(-1, -2), rel, "dv")
    # no sequence was left out
    assert not (last == 0).flatten(1).all(1).any()
    assert not (dk == 0).flatten(1).all(1).any()


def test_gradients_past_32_bit_offsets():
    """A head's last tokens, 2^31 elements and more into the tensors."""
    N, H, d = 70000, 260, 128
    print("[reach] gradients of 2.3e9 elements", flush=True)
    x = torch.zeros(1, N, H, d, device="cuda", dtype=BF16)
    g = torch.Generator().manual_seed(2)
    tail = torch.randn(40, 3, d, generator=g).to(BF16)
    x[0, -40:, -3:] = tail.cuda()
    decay = torch.full((H,), -0.05, device="cuda")
    got = A.lin_attn_bwd(x, x, x, x, decay)
    args = (tail, tail, tail, tail, decay[:3].cpu(), d ** -0.5)
    want, sums = R.backward(*args), R.backward(*args, sums=True)
    for t, w, s, what in zip(got, want, sums, ("dq", "dk", "dv")):
        _near(t[0, -40:, -3:], w, s, 40, d, BF16, what)
        assert not t[0, :-40].any() and not t[0, -40:, :-3].any()


def test_a_captured_prompt_and_its_steps():
    ins = _make(2, 700, 3, 64, BF16)
    q, k, v, _, S0, _, decay = (t.cuda() for t in ins)

    def run():
        o, last, _ = A.lin_attn_fwd(q[:, :697], k[:, :697], v[:, :697], decay,
                                    state=S0, final=True)
        out = [o, last]
        for t in range(697, 700):
            y, last = A.lin_attn_step(q[:, t], k[:, t], v[:, t], decay, last,
                                      state_out=torch.empty_like(last))
            out += [y, last]
        return out

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for i in range(4):
        q.copy_(q.flip(1))
        S0.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i
