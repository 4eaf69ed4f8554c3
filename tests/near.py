"""Comparison with a reference that a missing number never passes."""


def beyond(got, want, allow):
    """The largest part of its allowance that an element of got is off by;
    infinite where got is no number, or infinite, and want is not."""
    err = (got.double() - want).abs()
    off = (err / allow.clamp(min=1e-300)).masked_fill(err <= allow, 0.0)
    return float(off.nan_to_num(nan=float("inf"), posinf=float("inf")).max()) \
        if off.numel() else 0.0


def check(got, want, allow, what):
    assert got.shape == want.shape, what
    off = beyond(got, want, allow)
    assert off == 0.0, (what, off)
