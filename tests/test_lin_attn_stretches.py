"""Where the linear attention starts to cut its sequences, without a GPU: the
number of equal sequences decides, not a token more or less of each."""

import pytest
import torch

import adaln_fwd_amd as A

BF16, F32 = torch.bfloat16, torch.float32


def _stretches(B, N, H, d, dt, seg=None):
    return A.lin_attn_states_bytes(B, N, H, d, dt, seg) // (4 * H * d * d)


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [40, 64, 128])
@pytest.mark.parametrize("B,H", [(16, 12), (16, 11), (19, 10), (9, 19)])
def test_171_sequences_and_more_stay_whole(B, H, d, dt):
    assert all(_stretches(B, N, H, d, dt) == 0 for N in range(1200, 2000))


@pytest.mark.parametrize("d", [8, 32, 64, 128])
@pytest.mark.parametrize("B,H", [(17, 10), (16, 10), (16, 9), (43, 3)])
def test_fewer_are_cut_in_three(B, H, d):
    for N in range(1600, 2400):
        n = _stretches(B, N, H, d, BF16)
        assert n == 3 * B, (N, n)


@pytest.mark.parametrize("B,H,cut", [(19, 10, True), (16, 12, False)])
def test_narrow_heads_are_cut_up_to_191(B, H, cut):
    for N in range(1600, 2000):
        assert (_stretches(B, N, H, 32, BF16) > 0) == cut, N


@pytest.mark.parametrize("B,H", [(16, 12), (16, 11), (17, 10), (8, 12)])
def test_packed_sequences_go_by_the_same_limit(B, H):
    for N in (1559, 1560, 1561, 1999):
        seg = [i * N for i in range(B + 1)]
        assert _stretches(1, B * N, H, 128, BF16, seg) == \
            _stretches(B, N, H, 128, BF16)
