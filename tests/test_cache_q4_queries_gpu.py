"""Steps over a 4-bit cache with queries near the ends of bf16's range, where scores in float32
are finite (mha.h's bound on scale, queries and keys)."""
import numpy as np
import pytest
import torch

from tests import cache_util as cu
from tests import parity_util as pu
from tests import q4_util as qu
from tests.test_cache_gpu import mha, on_gpu  # noqa: F401
from tests.test_cache_q4_gpu import call_step, check_step, make_step

pytestmark = pytest.mark.gpu

ROWS = [(1, 1), (1, 2), (8, 1), (16, 1), (8, 4), (40, 1)]


def one_key_wins(case, mha, at, scale, what):  # noqa: F811
    """Queries and keys of one feature, `at`: no two keys are
    alike, and scores are so far apart that each row is its best key's value, rounded: the weight to
    fp16 (2^-11) and the output to bf16 (2^-8)."""
    B, T, H, d = case["q"].shape
    out, lse = call_step(mha, on_gpu(case), True, scale=scale)
    assert mha.mha_sync_status() == 0, what
    (k, _), (v, v_pairs) = (qu.cache_f64(case[n + "c"], case[n + "s"]) for n in "kv")
    q = cu.f64(case["q"])
    G = H // k.shape[2]
    factor = 1 / np.sqrt(d) if not scale else scale
    lse_ref = np.zeros((B, H, T))
    got = cu.f64(out)
    room_of = qu.reach(v_pairs)
    for h in range(H):
        for t in range(T):
            n = int(case["prefix"][0]) + t + 1
            s = factor * q[0, t, h, at] * k[0, :n, h // G, at]
            j = int(s.argmax())
            lse_ref[0, h, t] = s[j]
            want = v[0, j, h // G]
            room = 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * room_of[0, j, h // G]
            assert np.isfinite(got[0, t, h]).all(), f"{what}: row {t}, head {h} is not finite"
            assert (np.abs(got[0, t, h] - want) <= room).all(), f"{what}: row {t}, head {h}"
    assert lse_ref.max() < 2.0 ** 120
    pu.assert_lse_close(lse, lse_ref, what)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,G", ROWS)
@pytest.mark.parametrize("scale", [0.0, 1.0])
def test_large_queries(mha, d, T, G, scale):  # noqa: F811
    """Queries of one feature from 2^110 to the largest bf16, keys of 2^-55 to 2^-48."""
    n = 60
    case = make_step(d + T, 1, T, G, 1, d, n + T, [n], None, None)
    levels = 1 + np.random.default_rng(d + T).permutation(n + T)
    for at in (0, 7):
        k = torch.zeros((1, n + T, 1, d))
        k[0, :, 0, at] = torch.from_numpy(levels).float() * 2.0 ** -55
        case["kc"], case["ks"] = qu.q4_cache(k.to(torch.bfloat16))
        for size in (2.0 ** 110, 2.0 ** 117, 2.0 ** 118, 2.0 ** 121, 2.0 ** 125, 2.0 ** 127, 255 * 2.0 ** 120):
            case["q"][:] = 0.0
            case["q"][..., at] = size
            one_key_wins(case, mha, at, scale, f"feature {at}, |q| {size:.3g}")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,G", ROWS)
@pytest.mark.parametrize("scale", [0.0, 1.0])
def test_large_queries_of_keys_of_zeros(mha, d, T, G, scale):  # noqa: F811
    """Scores of 0, whatever the query: every key weighs the same."""
    case = make_step(d + T, 1, T, G, 1, d, 200 + T, [200], None, None)
    case["kc"], case["ks"] = qu.q4_cache(torch.zeros((1, 200 + T, 1, d), dtype=torch.bfloat16))
    plain = dict(case, q=torch.zeros_like(case["q"]))
    for size in (2.0 ** 121, 2.0 ** 127, 255 * 2.0 ** 120):
        case["q"][:] = size
        out, lse = call_step(mha, on_gpu(case), True, scale=scale)
        assert mha.mha_sync_status() == 0
        check_step(plain, out, lse, scale=scale or None, what=f"|q| {size:.3g}")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,G", [(2, 1), (8, 1), (16, 1), (40, 1)])
@pytest.mark.parametrize("big", [2.0 ** 122, 255 * 2.0 ** 120])
def test_a_large_query_beside_others(mha, d, T, G, big):  # noqa: F811
    """Rows of ordinary scores beside one of a huge query and one of a tiny: keys of 2^-20."""
    case = make_step(d + T, 1, T, G, 1, d, 300 + T, [300], None, None)
    k = cu.random_rows(5, (1, 300 + T, 1, d)).float() * 2.0 ** -20
    case["kc"], case["ks"] = qu.q4_cache(k.to(torch.bfloat16))
    case["q"] = (case["q"].float() * 2.0 ** 20).to(torch.bfloat16)
    if T > 2:
        case["q"][0, T // 2] = cu.random_rows(6, (G, d)) * 2.0 ** -90
    want = call_step(mha, on_gpu(case), True)
    spoilt = dict(case, q=case["q"].clone())
    spoilt["q"][0, T - 1] = big
    out, lse = call_step(mha, on_gpu(spoilt), True)
    assert mha.mha_sync_status() == 0
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    check_step(case, torch.cat((out[:, :-1], want[0][:, -1:]), 1), torch.cat((lse[..., :-1], want[1][..., -1:]), 2))


@pytest.mark.parametrize("T", [1, 2, 8, 16, 40])
def test_a_large_scale(mha, T):  # noqa: F811
    """The factor is the query's and the scale's together."""
    d, n = 128, 60
    case = make_step(T, 1, T, 1, 1, d, n + T, [n], None, None)
    k = torch.zeros((1, n + T, 1, d))
    k[0, :, 0, 3] = (1 + torch.arange(n + T)).float() * 2.0 ** -55
    case["kc"], case["ks"] = qu.q4_cache(k.to(torch.bfloat16))
    for size, scale in ((1.0, 2.0 ** 110), (2.0 ** 60, 2.0 ** 60), (2.0 ** -60, 2.0 ** 126), (2.0 ** 127, 2.0 ** -50)):
        case["q"][:] = 0.0
        case["q"][..., 3] = size
        one_key_wins(case, mha, 3, scale, f"|q| {size:.3g}, scale {scale:.3g}")


# What the header states of q: off by up to 2^-35 of its row's largest, and to 2^-27 where rows
# that share a factor are up to 2^8 larger.  In a packed row's even features it is 2^-39
# (2^-31): the odd ones' codes are 16 times too large, and q is rounded to fp16 16 times smaller.
EVEN, ODD = 2.0 ** -39, 2.0 ** -35


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,smaller", [(1, 0), (2, 0), (8, 0), (16, 0), (40, 0), (40, 8)])
@pytest.mark.parametrize("feature", [1, 2, 7, 20, 31])
def test_small_features_beside_a_large_one(mha, d, T, smaller, feature):  # noqa: F811
    """Queries of 1 in feature 0 (2^-8 in every second row, where the rows' common factor leaves
    eight binary places fewer) and of 2^-31 to 2^-28 in another, keys of that other alone, a scale
    of 2^30.  lse is off by no more than a score is: scale |k| times q's error."""
    n, scale = 150, 2.0 ** 30
    case = make_step(d + T, 1, T, 1, 1, d, n + T, [n], None, None)
    rng = np.random.default_rng(d + T + feature)
    k = torch.zeros((1, n + T, 1, d))
    k[0, :, 0, feature] = torch.from_numpy(rng.uniform(0.5, 3.0, size=n + T)).float()
    case["kc"], case["ks"] = qu.q4_cache(k.to(torch.bfloat16))
    case["q"][:] = 0.0
    case["q"][..., 0] = 1.0
    case["q"][:, 1::2, :, 0] = 2.0 ** -smaller
    case["q"][0, :, 0, feature] = torch.from_numpy(rng.uniform(-1, 1, size=T) * 2.0 ** -28).to(torch.bfloat16)
    _, lse = call_step(mha, on_gpu(case), True, scale=scale)
    assert mha.mha_sync_status() == 0
    kv, _ = qu.cache_f64(case["kc"], case["ks"])
    assert (kv[..., 0] == 0).all()
    s = scale * cu.f64(case["q"])[0, :, 0, feature, None] * kv[0, None, :, 0, feature]
    s = np.where(np.arange(n + T)[None] <= n + np.arange(T)[:, None], s, -np.inf)
    ref = np.log(np.exp(s - s.max(-1, keepdims=True)).sum(-1)) + s.max(-1)
    room = pu.LSE_ABS + pu.LSE_REL * np.abs(ref) + scale * (ODD if feature & 1 else EVEN) * kv.max()
    assert (np.abs(cu.f64(lse)[0, 0] - ref) <= room).all()
