"""The comparison that the values' tests use, without a GPU."""

import pytest
import torch

from tests import near


def test_what_is_off_or_no_number_is_refused():
    want = torch.tensor([0.0, 1.0, -2.0], dtype=torch.float64)
    allow = torch.tensor([0.0, 0.1, 0.1], dtype=torch.float64)
    near.check(torch.tensor([0.0, 1.05, -1.95]), want, allow, "within")
    for bad in ([0.0, 1.2, -2.0], [1e-30, 1.0, -2.0],
                [0.0, float("nan"), -2.0], [float("nan")] * 3,
                [0.0, float("inf"), -2.0], [0.0, 1.0, float("-inf")]):
        with pytest.raises(AssertionError):
            near.check(torch.tensor(bad), want, allow, "off")
    with pytest.raises(AssertionError):
        near.check(torch.zeros(2), want, allow, "shape")
    near.check(torch.zeros(0), torch.zeros(0, dtype=torch.float64),
               torch.zeros(0, dtype=torch.float64), "empty")
