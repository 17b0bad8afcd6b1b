"""Arguments of the 8-bit cache's entries that would reach the kernels as bad
addresses: refused by the C entries before any CUDA call (the pointers are
never dereferenced)."""
import pytest

from tests.test_cache_host import COUNTS, SHAPE, START, UNSUP, lib, read, write  # noqa: F401


@pytest.mark.parametrize("off", [1, 2, 3])
def test_misaligned_lengths(lib, off):  # noqa: F811
    """int32 arrays are read as such: 4-byte aligned, like those of the steps."""
    assert write(lib, start=START + off) == UNSUP
    assert write(lib, counts=COUNTS + off) == UNSUP
    assert read(lib, lens=START + off) == UNSUP
