"""Edges of the steps over a cache, against the plain float64 forms with the
tolerances of cache_util."""
import numpy as np
import pytest
import torch

from tests import cache_util as cu
from tests.test_cache_gpu import call_step, check_step, make_step, mha, on_gpu  # noqa: F401

pytestmark = pytest.mark.gpu

KINDS = [(True, 64), (True, 128), (True, 256), (False, 64), (False, 128), (False, 256)]


def bits_of(sees):
    """Mask words int64 [1, T, ceil(T / 64)] of truth values [T, T]."""
    T = len(sees)
    words = np.zeros((1, T, (T + 63) // 64), dtype=np.uint64)
    for t, j in zip(*np.nonzero(sees)):
        words[0, t, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return torch.from_numpy(words.view(np.int64))


def one_feature_step(seed, T, H, d, Lk, prefix, sees, factor, f8):
    """A step whose scores lie in feature 0 alone: keys 8 to 15 there (exact in
    both caches), row t's queries factor[t].  A score is one exact product: its
    error is a few half steps of float32, so cache_util's ds < 2^-13 holds up to
    |score| 2^9."""
    case = make_step(seed, 1, T, H, H, d, Lk, [prefix], None, bits_of(sees), f8)
    k = torch.zeros((1, Lk, H, d), dtype=torch.bfloat16)
    k[0, :, :, 0] = (8 + torch.arange(Lk) % 8).to(torch.bfloat16)[:, None]
    case["q"][:] = 0.0
    case["q"][0, :, :, 0] = torch.tensor(factor, dtype=torch.float64).to(torch.bfloat16)[:, None]
    if f8:
        case["kc"], case["ks"] = cu.f8_cache(k)
        case["k_ref"] = cu.cache_values(cu.codes_of(case["kc"]), case["ks"].numpy())
    else:
        case["kc"], case["k_ref"] = k, cu.f64(k)
    return case


@pytest.mark.parametrize("f8,d", KINDS, ids=lambda x: str(x))
@pytest.mark.parametrize("values", ["ordinary", "zero"])
def test_rows_whose_first_key_comes_late(mha, f8, d, values):  # noqa: F811
    """No prefix, 200 drafted tokens: rows whose only keys lie in the second tile
    of 128 and score -100 to -375 are no empty rows; beside them rows that see
    keys of the first tile, and rows that see nothing."""
    T = 200
    t = np.arange(T)
    sees = np.zeros((T, T), dtype=bool)
    for i in t:
        if i % 4 == 0:
            sees[i, : i + 1] = True                    # from the first tile on
        elif i % 4 == 1:
            sees[i, 130 + i % 60: 130 + i % 60 + 3] = True
        elif i % 4 == 2:
            sees[i, 199] = True
    factor = np.where(t % 4 == 0, 1.0, np.where(t % 8 < 4, -12.5, -25.0))
    case = one_feature_step(31, T, 2, d, 230, 0, sees, factor, f8)
    if values == "zero":                               # (8-bit: the least scale)
        zero = torch.zeros((1, 230, 2, d), dtype=torch.bfloat16)
        if f8:
            case["vc"], case["vs"] = cu.f8_cache(zero)
        else:
            case["vc"] = zero
        case["v_ref"] = np.zeros((1, 230, 2, d))
    out, lse = call_step(mha, on_gpu(case), f8, True, scale=1.0)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, f8, scale=1.0, what=f"{d} features")


@pytest.mark.parametrize("f8,d", KINDS, ids=lambda x: str(x))
@pytest.mark.parametrize("prefix", [3840, 3968, 4000])
def test_late_first_keys_with_splits(mha, f8, d, prefix):  # noqa: F811
    """The same behind a prefix whose keys are in other splits: with a few tiles to
    a split, one that begins at the drafted tokens or just before them has rows
    that see nothing of its first tile."""
    T, Lk = 250, 4300
    t = np.arange(T)
    sees = np.zeros((T, T), dtype=bool)
    sees[t, t] = True
    sees[t % 3 == 1, 249] = True
    factor = np.where(t % 3 == 0, 1.0, np.where(t % 3 == 1, -12.5, -25.0))
    case = one_feature_step(32, T, 1, d, Lk, prefix, sees, factor, f8)
    out, lse = call_step(mha, on_gpu(case), f8, True, scale=1.0)
    assert mha.last_launch_info()["kernels"] == 2
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, f8, scale=1.0, what=f"{d} features")


HIDDEN = [
    # B, T, H, H_kv, Lk, prefix, drafts
    (1, 1, 2, 2, 40, [30], None),                  # the only drafted token does not see itself
    (2, 12, 4, 2, 300, [120, 0], None),            # over a tile's border; no prefix
    (3, 20, 4, 4, 290, [255, 40, 7], [20, 0, 13]),
    (1, 100, 3, 3, 500, [100], None),              # over three tiles
    (2, 200, 2, 1, 460, [250, 3], [200, 150]),     # blocks of rows; rows past the drafted tokens
    (1, 250, 8, 2, 4000, [3700], None),            # splits
]


@pytest.mark.parametrize("f8,d", KINDS, ids=lambda x: str(x))
@pytest.mark.parametrize("shape", HIDDEN, ids=lambda s: "x".join(map(str, s[:5])))
def test_drafted_positions_no_row_sees(mha, f8, d, shape):  # noqa: F811
    """A drafted position whose bit no row sets may hold anything: NaN and
    infinities (8-bit: NaN codes, the largest scale byte) reach no row."""
    B, T, H, H_kv, Lk, prefix, drafts = shape
    hidden = np.arange(T) % 5 == 2 if T > 1 else np.array([True])
    hidden[T // 2: T // 2 + 4] = True
    keep = cu.tree_bits(np.random.default_rng(T), B, T)
    words = (T + 63) // 64
    shown = bits_of(np.tile(~hidden, (T, 1)))[0, 0].reshape(1, 1, words)
    case = make_step(sum(shape[:5]) + d, B, T, H, H_kv, d, Lk, prefix, drafts, keep & shown, f8)
    for b in range(B):
        live = T if drafts is None else drafts[b]
        for j in np.nonzero(hidden[:live])[0]:
            at = prefix[b] + j
            for n in ("k", "v"):
                case[n + "_ref"][b, at] = 0.0
                if f8:
                    case[n + "c"].view(torch.uint8)[b, at] = 0x7F
                    case[n + "s"][b, :, at] = 255
                else:
                    case[n + "c"][b, at] = float("nan") if j % 2 else float("-inf")
    out, lse = call_step(mha, on_gpu(case), f8, True)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, f8, what=f"{shape[:5]} of {d}")


@pytest.mark.parametrize("f8,d", KINDS, ids=lambda x: str(x))
@pytest.mark.parametrize("shape", [(3, 7, 4, 2, 200), (2, 100, 2, 2, 500), (3, 40, 8, 2, 9000)],
                         ids=lambda s: "x".join(map(str, s)))
def test_rows_past_the_drafted_tokens_hold_anything(mha, f8, d, shape):  # noqa: F811
    """A padded batch: the queries of rows past draft_lens (NaN, the largest values)
    and their mask words reach no other row."""
    B, T, H, H_kv, Lk = shape
    drafts = [T - 3, 0, T][:B]
    case = make_step(B + T, B, T, H, H_kv, d, Lk, [Lk - T, 5, 40][:B], drafts, "tree", f8)
    for b, live in enumerate(drafts):
        case["q"][b, live:] = torch.tensor([float("nan"), float("inf"), 3e38, -3e38]).to(
            torch.bfloat16).repeat(d // 4)
        case["mask"][b, live:] = -1
    g = on_gpu(case)
    out, lse = call_step(mha, g, f8, True)
    assert mha.mha_sync_status() == 0
    for b, live in enumerate(drafts):
        case["q"][b, live:] = 0.0
    check_step(case, out, lse, f8, what=f"{shape} of {d}")


def test_nothing_to_do(mha):  # noqa: F811
    """No sequence, no token: nothing is launched, and shapes come back."""
    for B, T in ((0, 3), (2, 0)):
        case = make_step(1, B, T, 4, 2, 64, 30, [5] * B, None, None, True)
        g = on_gpu(case)
        for f8 in (True, False):
            if not f8:
                g["kc"], g["vc"] = (torch.zeros((B, 30, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv")
            out, lse = call_step(mha, g, f8, True)
            assert out.shape == (B, T, 4, 64) and lse.shape == (B, 4, T)
        k = torch.zeros((B, T, 2, 64), dtype=torch.bfloat16, device="cuda")
        mha.mha_cache_write_f8(k, k, *(on_gpu(case)[n] for n in ("kc", "vc", "ks", "vs")), g["prefix"])
    assert mha.mha_sync_status() == 0
