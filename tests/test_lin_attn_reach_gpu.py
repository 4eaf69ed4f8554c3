"""Linear attention's single tokens in a captured graph, from the state of a
captured prompt."""

import pytest
import torch

import adaln_fwd_amd as A
from tests.test_lin_attn_gpu import _make

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


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
