"""The stream that a call without one runs on: torch's current one, whichever
way its handle is asked for."""

import pytest
import torch

import adaln_fwd_amd as A
from adaln_fwd_amd import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("public", [False, True])
def test_the_current_stream(monkeypatch, public):
    if public:
        monkeypatch.setattr(ops, "_current", ops._current_stream)
    dev = torch.device("cuda", torch.cuda.current_device())
    x = torch.randn(1, 40, 2, 64, device=dev)
    pos = torch.arange(40, dtype=torch.int32, device=dev).reshape(-1, 1)
    f = A.rope_freqs((32,))
    want = A.rope_fwd(x, None, pos, f)[0]
    torch.cuda.synchronize()
    for s in (torch.cuda.default_stream(dev), torch.cuda.Stream(dev)):
        with torch.cuda.stream(s):
            assert ops._stream(dev, None) == s.cuda_stream
            got = A.rope_fwd(x, None, pos, f)[0]
        s.synchronize()
        assert torch.equal(got, want)
    assert ops._stream(dev, s) == s.cuda_stream == ops._stream(
        dev, s.cuda_stream)
