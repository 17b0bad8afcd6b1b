"""Arguments that would reach the kernels as bad addresses: refused by the C
entries before any CUDA call (the pointers are never dereferenced)."""
import pytest

from tests import test_abi_host as abi
from tests.test_cache_host import ALIAS, COUNTS, K, SHAPE, START, UNSUP, lib, read, write  # noqa: F401


@pytest.mark.parametrize("off", [1, 2, 3])
def test_misaligned_lengths(lib, off):  # noqa: F811
    """int32 arrays are read as such: 4-byte aligned, like those of the steps."""
    assert write(lib, start=START + off) == UNSUP
    assert write(lib, counts=COUNTS + off) == UNSUP
    assert read(lib, lens=START + off) == UNSUP


def test_strides_that_wrap(lib):  # noqa: F811
    """Rows that reach further than 2^50 elements are refused, whichever stride takes
    them there: their last address would wrap, in the check for overlaps too."""
    far = 1 << 50
    assert write(lib, B=1 << 20, T=1, H=1, ss=far) == SHAPE
    assert write(lib, B=3, T=1, H=1, ss=far) == SHAPE
    assert write(lib, B=1 << 15, T=1, H=1, ss=1 << 36) == SHAPE
    assert write(lib, B=2, T=1 << 10, H=1, ts=1 << 40, ss=1 << 49) == SHAPE
    assert write(lib, B=1 << 20, T=1 << 20, H=1, ts=1 << 31) == SHAPE      # (dense rows: ss = T ts)
    # near the end, and with a single sequence, whose stride is of no account, the
    # check for overlaps has its say
    assert write(lib, B=1, T=5, H=3, ss=far, kc=K) == ALIAS
    assert write(lib, B=2, T=1, H=1, ss=far - 64, kc=K + 2 * (far - 64)) == ALIAS


@pytest.mark.parametrize("off", [1, 2, 3])
def test_misaligned_lengths_of_the_other_entries(lib, off):  # noqa: F811
    assert abi.dec(lib, lens=abi.LENS_D + off) == UNSUP
    for fn in ("mha_fwd", "mha_fwd_f32"):
        assert abi.fwd(lib, fn, mask=2, lens=abi.LENS + off) == UNSUP
    assert abi.bwd(lib, mask=2, lens=abi.LENS + off) == UNSUP
    assert abi.layer(lib, mask=2, lens=abi.LENS + off) == UNSUP
