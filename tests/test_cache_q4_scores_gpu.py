"""Steps over a 4-bit cache whose scores are large and finite: past 2^24 a score's last place is
more than the distance that weights keep from a row's reference, and a row is its best key's
value all the same."""
import numpy as np
import pytest
import torch

from tests import cache_util as cu
from tests import parity_util as pu
from tests import q4_util as qu
from tests.test_cache_gpu import mha, on_gpu  # noqa: F401
from tests.test_cache_q4_gpu import call_step, make_step

pytestmark = pytest.mark.gpu

SIZES = [10, 18, 20, 22, 23, 24, 25, 26, 27, 28, 30, 40, 70, 100]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,G", [(1, 1), (1, 2), (8, 1), (16, 1), (8, 4), (40, 1), (20, 3)])
@pytest.mark.parametrize("n", [60, 500, 9000], ids=["a tile", "tiles", "splits"])
@pytest.mark.parametrize("sign", [1.0, -1.0], ids=["up", "down"])
def test_scores_past_float32s_places(mha, d, T, G, n, sign):  # noqa: F811
    """Queries and keys of one feature; keys of 20 to 100 units, one of 128 and one of 1, whose
    places change: queries of either sign have one best key, and the scores of all others
    are lower by 19 units or more, hundreds at the least.  The weight is rounded to fp16 (2^-11,
    the same in the value's offset and its code) and the output to bf16 (2^-8)."""
    case = make_step(d + T, 1, T, G, 1, d, n + T, [n], None, None)
    rng = np.random.default_rng(d + T + n)
    factor = 1 / np.sqrt(d)
    v, v_pairs = qu.cache_f64(case["vc"], case["vs"])
    room_of = qu.reach(v_pairs)
    for i, at in enumerate((0, n // 2, n - 1)):
        levels = rng.integers(20, 101, size=n + T)
        levels[at], levels[(at + n // 3 + 1) % n] = 128, 1
        k = torch.zeros((1, n + T, 1, d))
        k[0, :, 0, 5] = torch.from_numpy(levels).float()
        case["kc"], case["ks"] = qu.q4_cache(k.to(torch.bfloat16))
        kv, _ = qu.cache_f64(case["kc"], case["ks"])
        for size in SIZES[i::3]:
            case["q"][:] = 0.0
            case["q"][..., 5] = sign * 1.25 * 2.0 ** size
            case["q"][0, T // 2:, ..., 5] *= 1.5
            out, lse = call_step(mha, on_gpu(case), True)
            assert mha.mha_sync_status() == 0
            s = factor * cu.f64(case["q"])[0, :, :, 5, None] * kv[0, None, None, :n, 0, 5]   # (drafts: 20 to 100)
            j = s.argmax(-1)
            assert (j == j.flat[0]).all() and levels[j.flat[0]] in (1, 128)
            want, reach = v[0, j.flat[0], 0], room_of[0, j.flat[0], 0]
            got = cu.f64(out).reshape(T, G, d)
            assert np.isfinite(got).all(), f"2^{size}: not finite"
            worst = (np.abs(got - want) - 2.0 ** -8 * np.abs(want)).max()
            assert worst <= 2.0 ** -10 * reach, f"2^{size}: off by {worst:.3g}"
            # lse: beside the entries' tolerance, float32 places of the row's largest |score| S, which
            # its references pass on the way to the best key: a score is three products and sums
            # (3 x 2^-24 S), a reference that moves two differences of numbers up to 2 S
            # (4 x 2^-24 S) and its score's own, a score less it one more (2 x 2^-24 S): below 2^-20 S.
            ref = s.max(-1).T[None]
            room = pu.LSE_ABS + pu.LSE_REL * np.abs(ref) + 2.0 ** -20 * np.abs(s).max(-1).T[None]
            assert (np.abs(cu.f64(lse).reshape(1, G, T) - ref) <= room).all(), f"2^{size}: lse"
