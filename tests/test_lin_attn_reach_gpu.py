"""Linear attention where its offsets reach furthest, and single tokens in a
captured graph from the state of a captured prompt.

Tolerances: those of test_lin_attn_gpu.py."""

import pytest
import torch

import adaln_fwd_amd as A
from tests import ref_lin_attn as R
from tests.test_lin_attn_gpu import _make, _near

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


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
