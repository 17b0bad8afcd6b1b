"""The rounding that include/mha.h states for the 8-bit cache, on the plain form
(the GPU tests hold the kernel to its bits)."""
import numpy as np
import pytest
import torch

from tests import cache_util as cu


def rows_below(top):
    """A row per positive bf16 value below `top` (down to 2^-30 of it), beside `top`."""
    bits = torch.arange(1, 0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).double().numpy()
    x = bits[(bits < top) & (bits > top * 2.0 ** -30)]
    return np.stack([np.full_like(x, top), x], -1)


def error(rows):
    codes, scales = cu.quantise(rows)
    e = scales.astype(np.float64) - 127
    y = cu.VALUES[codes] * np.exp2(e)[:, None]
    return np.abs(y - rows)[:, 1], e


@pytest.mark.parametrize("at", [-40, 0, 7, 100])
@pytest.mark.parametrize("top", [225.0, 256.0, 448.0])   # just above a scale's step; one; a full one
def test_rounding_of_a_row(top, at):
    rows = rows_below(top * 2.0 ** at)
    x = rows[:, 1]
    err, e = error(rows)
    assert (e == at).all()
    assert (err <= np.maximum(2.0 ** -4 * x, 2.0 ** (e - 10))).all()
    large = x >= 2.0 ** -13 * rows[:, 0]
    assert (err[large] <= 2.0 ** -4 * x[large]).all()


def test_rounding_below_that():
    """One power of two less of the row's largest is not enough, and neither is a
    row below 2^-56."""
    rows = rows_below(225.0)
    err, _ = error(rows)
    x = rows[:, 1]
    assert (err > 2.0 ** -4 * x)[x >= 2.0 ** -14 * 225.0].any()
    rows = rows_below(2.0 ** -60)
    err, e = error(rows)
    x = rows[:, 1]
    assert (e == -64).all() and (err > 2.0 ** -4 * x)[x >= 2.0 ** -13 * 2.0 ** -60].any()
    assert (err <= np.maximum(2.0 ** -4 * x, 2.0 ** -74)).all()
