"""The 4-bit cache's writes and reads at sizes whose launches divide the work otherwise:
tiles of 4, 8 and 16 positions, ragged at both ends, for each number of lanes to a row."""
import numpy as np
import pytest

from tests import test_cache_q4_gpu as q4
from tests.test_cache_gpu import mha  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [32, 64, 128, 224])
@pytest.mark.parametrize("B,T,H", [(2, 9, 11), (5, 37, 90), (9, 83, 130)], ids=["4", "8", "16"])
def test_write_tiles(mha, B, T, H, d):  # noqa: F811
    rng = np.random.default_rng(B)
    Lk = T + 5
    start = rng.integers(-3, 9, size=B).tolist()
    counts = rng.integers(0, T + 2, size=B).tolist()
    counts[0] = T
    q4.test_write(mha, (B, T, H, d, Lk, start, counts, d == 64))


@pytest.mark.parametrize("d", [32, 64, 128, 224])
@pytest.mark.parametrize("B,Lk,H", [(2, 9, 11), (5, 37, 90), (9, 83, 130)], ids=["4", "8", "16"])
def test_read_tiles(mha, B, Lk, H, d):  # noqa: F811
    lens = np.random.default_rng(B).integers(0, Lk + 1, size=B).tolist()
    lens[0] = Lk
    q4.test_read(mha, (B, Lk, H, d, lens))
