"""Steps over a 4-bit cache whose products of codes cancel against those of offsets: what is
left shows how many places the products' sums keep.

Beside q4_util's tolerances (of float32 sums): the tensor cores add sixteen products at a time,
aligned by the exponents of their factors, and a code enters as an fp16 subnormal, c 2^-24, whose
exponent counts as 2^-14 whatever c is.  A product is cut 25 places below the largest sum of
exponents: at 2^-39 of the block's largest q (or weight), that is 2^-15 of it times a code of 1.
A score adds d products, an output sixteen to each sixteen keys, and each is off by less than that:
  scores   d 2^-15 scale max |q| max step
  outputs  sum over sixteen keys at a time of 16 2^-15 max a_j step_j
"""
import numpy as np
import pytest
import torch

from tests import cache_util as cu
from tests import parity_util as pu
from tests import q4_util as qu
from tests.test_cache_gpu import mha, on_gpu  # noqa: F401
from tests.test_cache_q4_gpu import call_step, make_step

pytestmark = pytest.mark.gpu

ROWS = [(1, 1), (1, 2), (8, 1), (16, 1), (16, 2), (40, 1), (16, 8)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,G", ROWS)
@pytest.mark.parametrize("n", [30, 700, 9000], ids=["a tile", "tiles", "splits"])
def test_values_that_cancel(mha, d, T, G, n):  # noqa: F811
    """One key has nearly all the weight, and its value is offset + 7 step, a few places from 0;
    the others' weights are 2^-5 to 2^-14 of its, and their values any."""
    case = make_step(d + T, 1, T, G, 1, d, n + T, [n], None, None)
    rng = np.random.default_rng(d + T + n)
    codes = rng.integers(0, 16, size=(1, n + T, 1, d)).astype(np.uint8)
    at = n // 2
    codes[0, at] = 7
    step = rng.integers(129, 256, size=(1, 1, n + T)) / 256.0
    case["vc"] = torch.from_numpy(qu.packed(codes))
    case["vs"] = torch.from_numpy(np.stack((-7 * step, step), -1)).to(torch.bfloat16)   # (offsets rounded)
    k = torch.zeros((1, n + T, 1, d))
    k[0, :, 0, 6] = torch.from_numpy(rng.uniform(0, 1, size=n + T)).float()
    k[0, at, 0, 6] = 0.0
    k[0, at, 0, 3] = 1.0
    case["kc"], case["ks"] = qu.q4_cache(k.to(torch.bfloat16))
    case["q"][:] = 0.0
    case["q"][..., 3], case["q"][..., 6] = 16.0, 6.0
    out, _ = call_step(mha, on_gpu(case), True, scale=1.0)
    assert mha.mha_sync_status() == 0
    (kv, k_pairs), (vv, v_pairs) = (qu.cache_f64(case[x + "c"], case[x + "s"]) for x in "kv")
    q = cu.f64(case["q"])
    for t in range(T):
        m = n + t + 1
        s = kv[0, :m, 0] @ q[0, t, 0]
        a = np.exp(s - s.max())
        a /= a.sum()
        ref, size = a @ vv[0, :m, 0], a @ np.abs(vv[0, :m, 0])
        big = np.pad(a * v_pairs[0, 0, :m, 1], (0, -m % 16)).reshape(-1, 16).max(-1).sum()
        span = qu.reach(v_pairs)[0, :m, 0, 0]
        ds = (d / 16 + 8) * 2.0 ** -23 * np.abs(q[0, t, 0]).sum() * qu.reach(k_pairs).max()
        # (float32 sums: of what a row's keys weigh in all, once to sixteen keys and 64 times beside)
        room = 2.0 ** -8 * np.abs(ref) + 1.01 * ((1 + 2.0 ** -11 + 2.0 ** -18) * np.exp(2 * ds) - 1) * size + \
            (m / 16 + 64) * 2.0 ** -23 * (a * span).sum() + 16 * 2.0 ** -15 * big
        got = cu.f64(out)[0, t]
        assert (np.abs(got - ref) <= room).all(), f"row {t}: {(np.abs(got - ref) / room).max():.3f} of the tolerance"


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,G", ROWS)
@pytest.mark.parametrize("sign", [False, True], ids=["any sign", "one sign"])
def test_scores_of_small_features_beside_a_large_one(mha, d, T, G, sign):  # noqa: F811
    """Queries of 1 in one feature, whose keys are offset + 7 step = 0, and of some 2^-10 in all
    others."""
    n = 150
    case = make_step(d + T, 1, T, G, 1, d, n + T, [n], None, None)
    rng = np.random.default_rng(d + T)
    codes = rng.integers(0, 16, size=(1, n + T, 1, d)).astype(np.uint8)
    at = int(rng.integers(0, d))
    codes[..., at] = 7
    step = 2.0 ** -rng.integers(0, 3, size=(1, 1, n + T)).astype(float)
    case["kc"] = torch.from_numpy(qu.packed(codes))
    case["ks"] = torch.from_numpy(np.stack((-7 * step, step), -1)).to(torch.bfloat16)
    case["q"] = (cu.random_rows(T, (1, T, G, d)).float() * 2.0 ** -10).to(torch.bfloat16)
    if sign:                                              # what is cut off adds up
        case["q"] = case["q"].abs()
    case["q"][..., at] = 1.0
    _, lse = call_step(mha, on_gpu(case), True, scale=64.0)
    assert mha.mha_sync_status() == 0
    kv, pairs = qu.cache_f64(case["kc"], case["ks"])
    q = cu.f64(case["q"])
    _, ref, _ = cu.attention(q, kv, kv, lambda b: cu.visible(b, T, n + T, [n], None, None), 64.0)
    ds = (d / 16 + 8) * 2.0 ** -23 * 64.0 * np.abs(q).sum(-1).max() * qu.reach(pairs).max() + \
        d * 2.0 ** -15 * 64.0 * np.abs(q).max() * pairs[..., 1].max()
    assert (np.abs(cu.f64(lse).reshape(ref.shape) - ref) <= pu.LSE_ABS + pu.LSE_REL * np.abs(ref) + ds).all()
