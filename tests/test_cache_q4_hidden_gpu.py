"""A step over a 4-bit cache whose drafted positions hold keys or values that are no numbers:
the rows that see one are NaN, in out and in lse, and the rows that it is hidden from are what
they are without it (q4_util's plain forms)."""
import numpy as np
import pytest
import torch

from tests import cache_util as cu
from tests.test_cache_gpu import i32, mha, on_gpu  # noqa: F401
from tests.test_cache_q4_gpu import call_step, check_step, make_step

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
AS_WRITTEN = (NAN, 2.0 ** -60)     # what the write stores for a row that is not finite


def spoil(case, name, at, pair, heads=slice(None)):
    """The case with the pair of position `at` of sequence 0's keys or values (name: k, v)."""
    pairs = case[name + "s"].clone()
    pairs[0, heads, at] = torch.tensor(pair).to(torch.bfloat16)
    return dict(case, **{name + "s": pairs})


def check_spoilt(mha, case, bad, sees, what):  # noqa: F811
    """bad: the case spoilt; sees [B, T, H]: whose rows see it."""
    clean = call_step(mha, on_gpu(case), True)
    out, lse = call_step(mha, on_gpu(bad), True)
    assert mha.mha_sync_status() == 0
    sees = torch.from_numpy(sees).cuda()
    assert torch.isnan(out[sees]).all(), f"{what}: a row that sees it is no NaN"
    assert torch.isnan(lse.transpose(1, 2)[sees]).all(), f"{what}: its lse is no NaN"
    hidden = ~sees
    assert torch.isfinite(out[hidden]).all(), f"{what}: shows in a row that it is hidden from"
    assert not torch.isnan(lse.transpose(1, 2)[hidden]).any(), f"{what}: shows in the lse of such a row"
    out[sees] = clean[0][sees]
    lse = torch.where(sees.transpose(1, 2), clean[1], lse)
    check_step(case, out, lse, what=what)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,G", [(2, 1), (2, 2), (5, 1), (3, 2), (16, 1), (8, 2), (11, 2), (16, 2), (40, 1), (23, 2)])
@pytest.mark.parametrize("mask", [None, "tree"], ids=["chain", "tree"])
@pytest.mark.parametrize("prefix", [60, 9000], ids=["a tile", "splits"])
def test_a_drafted_value_that_is_no_number(mha, d, T, G, mask, prefix):  # noqa: F811
    """One, two, up to eight, up to sixteen and more rows per key head; the position spoilt is
    the first, one in the middle, the last."""
    case = make_step(d + T + G + prefix, 2, T, 2 * G, 2, d, prefix + T + 3, [prefix, 7], None, mask)
    bits = None if case["mask"] is None else case["mask"].numpy()
    visible = cu.visible(0, T, prefix + T + 3, case["prefix"].numpy(), None, bits)
    for j in sorted({0, T // 2, T - 1}) if prefix < 100 else [T // 2]:
        sees = np.zeros((2, T, 2 * G), dtype=bool)
        sees[0, :, :G] = visible[:, prefix + j, None]
        assert sees.any() and not sees.all()
        for name in "kv":
            bad = spoil(case, name, prefix + j, AS_WRITTEN, 0)     # of key head 0 alone
            check_spoilt(mha, case, bad, sees, f"{name} of draft {j}")


@pytest.mark.parametrize("T", [2, 5, 16, 40])
@pytest.mark.parametrize("pair", [(1.0, NAN), (1.0, 0.0), (0.0, 0.0), (1.0, INF), (INF, 1.0), (-INF, INF), (NAN, NAN),
                                  (1.0, 2.0 ** -130)], ids=str)
def test_pairs_that_the_write_does_not_store(mha, T, pair):  # noqa: F811
    """A value's pair of any bits: rows that it is hidden from do not know of it."""
    case = make_step(T, 1, T, 1, 1, 128, 100, [50], None, None)
    for name in "kv":
        out, lse = call_step(mha, on_gpu(spoil(case, name, 50 + T - 1, pair)), True)
        want, want_lse = call_step(mha, on_gpu(case), True)
        assert mha.mha_sync_status() == 0
        check_step(case, torch.cat((out[:, :-1], want[:, -1:]), 1), torch.cat((lse[..., :-1], want_lse[..., -1:]), 2))


@pytest.mark.parametrize("T", [1, 2, 6, 16, 40])
@pytest.mark.parametrize("prefix", [60, 9000], ids=["a tile", "splits"])
def test_a_value_of_the_prefix(mha, T, prefix):  # noqa: F811
    """All rows of its sequence and key head see it, and no other row does."""
    case = make_step(T + 1, 2, T, 2, 2, 64, prefix + T, [prefix, 20], None, None)
    sees = np.zeros((2, T, 2), dtype=bool)
    sees[0, :, 1] = True
    for at in (0, prefix // 2, prefix - 1):
        for name in "kv":
            check_spoilt(mha, case, spoil(case, name, at, AS_WRITTEN, 1), sees, f"{name} of position {at}")


@pytest.mark.parametrize("T", [2, 7, 16, 40])
def test_a_row_that_was_not_finite_when_written(mha, T):  # noqa: F811
    """By way of the write: a drafted token's value row holds an infinity."""
    B, H, d, Lk, n = 1, 2, 128, 80, 30
    k, v = (cu.random_rows(s, (B, n + T, H, d)) for s in (1, 2))
    v[0, n + T // 2, 0, 9] = INF
    q = cu.random_rows(3, (B, T, H, d))
    cache = [torch.zeros((B, Lk, H, d // 2), dtype=torch.uint8, device="cuda") for _ in range(2)] + \
        [torch.zeros((B, H, Lk, 2), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    mha.mha_cache_write_q4(k.cuda(), v.cuda(), *cache, i32([0]).cuda())
    out, lse = mha.mha_decode_tree_q4(q.cuda(), *cache, i32([n]).cuda(), return_lse=True)
    assert mha.mha_sync_status() == 0
    assert torch.isfinite(out[0, :, 1]).all() and torch.isfinite(lse[0, 1]).all()
    assert torch.isfinite(out[0, :T // 2, 0]).all() and torch.isfinite(lse[0, 0, :T // 2]).all()
    assert torch.isnan(out[0, T // 2:, 0]).all() and torch.isnan(lse[0, 0, T // 2:]).all()
