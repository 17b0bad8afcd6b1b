"""Moves of cached rows whose launch would pass a grid's largest size are refused on the host,
before any CUDA call (pointers below are never dereferenced)."""
import pytest

from tests.test_cache_host import SHAPE, lib  # noqa: F401
from tests.test_cache_q4_host import BF16, F8, Q4

KC, VC, KS, VS, PREFIX, PATH = (0x100_0000_0000 * i for i in range(1, 7))


@pytest.mark.parametrize("fmt,d", [(BF16, 8), (F8, 16), (Q4, 32), (Q4, 256)])
@pytest.mark.parametrize("B", [2 ** 30, 2 ** 30 + 1, 2 ** 30 + 77, 3 * 2 ** 29, 2 ** 31 - 1])
def test_a_compaction_of_more_blocks_than_a_grid_has(lib, fmt, d, B):  # noqa: F811
    """Two blocks to a sequence at least, for its keys and its values."""
    assert lib.mha_cache_compact(KC, VC, KS, VS, fmt, B, 1, 1, 1, d, PREFIX, PATH, None, None) == SHAPE
