"""The 4-bit cache (mha_cache_write_q4, mha_cache_read_q4) and the steps over it
(mha_decode_q4, mha_decode_tree_q4) against their plain float64 forms (q4_util)."""
import numpy as np
import pytest
import torch

from tests import cache_util as cu
from tests import parity_util as pu
from tests import q4_util as qu
from tests.test_cache_edges_gpu import bits_of
from tests.test_cache_gpu import i32, mha, on_gpu  # noqa: F401
from tests.test_streams_gpu import behind_a_reader

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- write, read
WRITES = [
    # B, T, H, d, Lk, start, counts, packed
    (3, 1, 2, 32, 5, [0, 4, 2], None, False),
    (2, 7, 3, 96, 20, [13, 0], None, True),                    # odd heads, six lanes of eight
    (4, 33, 9, 64, 64, [31, 0, 40, -3], [33, 0, 33, 20], True),  # off both ends, none, more than a tile
    (1, 70, 17, 128, 101, [30], [69], False),
    (2, 40, 5, 256, 40, [0, 0], [100, -4], True),              # counts past T and below 0
    (2, 5, 4, 224, 300, [295, 297], None, False),
    (3, 6, 3, 160, 9, [5, -2, 2 ** 31 - 4], None, True),       # a start near the largest int
    (128, 1, 8, 64, 256, None, None, True),                    # a decode step's write
    (1, 1, 1, 128, 1, [0], [1], False),
]


def random_cache(seed, B, Lk, H, d):
    g = torch.Generator().manual_seed(seed)
    codes = [torch.randint(0, 256, (B, Lk, H, d // 2), generator=g, dtype=torch.uint8) for _ in range(2)]
    pairs = [torch.randn((B, H, Lk, 2), generator=g).to(torch.bfloat16) for _ in range(2)]
    return codes, pairs


def rows_of(seed, B, T, H, d, packed):
    """k, v on the GPU: row magnitudes from 2^-70 to 2^100; a row of zeros, of one
    value, of neighbouring values, of values on the middles between codes, and rows
    with a large offset; packed: inside a Q | K | V projection."""
    rng = np.random.default_rng(seed)
    x = cu.random_rows(seed, (B, T, 3, H, d)).float()
    x *= torch.from_numpy(np.exp2(rng.integers(-70, 100, size=(B, T, 3, H, 1)))).float()
    x[0, 0, 1, 0] = 0.0
    x[-1, -1, 1, -1] = -3.0
    x[-1, -1, 2, -1] = torch.arange(d) % 31 / 2 - 3.5            # step 1: halves are ties
    x[0, -1, 2, 0] = 100.0 + (torch.arange(d) % 2) * 0.5         # neighbours
    x[0, 0, 2, -1] = 1000.0 + torch.randn(d, generator=torch.Generator().manual_seed(seed))
    x = x.to(torch.bfloat16).cuda()
    if packed:
        return x[:, :, 1], x[:, :, 2]
    return x[:, :, 1].contiguous(), x[:, :, 2].contiguous()


@pytest.mark.parametrize("shape", WRITES, ids=lambda s: "x".join(map(str, s[:5])))
def test_write(mha, shape):  # noqa: F811
    B, T, H, d, Lk, start, counts, packed = shape
    if start is None:
        start = np.random.default_rng(2).integers(0, Lk, size=B).tolist()
    k, v = rows_of(7, B, T, H, d, packed)
    codes, pairs = random_cache(8, B, Lk, H, d)
    dev = [c.cuda() for c in codes] + [s.cuda() for s in pairs]
    mha.mha_cache_write_q4(k, v, *dev, i32(start).cuda(),
                           counts=None if counts is None else i32(counts).cuda())
    assert mha.mha_sync_status() == 0
    for x, c, s, got_c, got_s in zip((k, v), codes, pairs, dev[:2], dev[2:]):
        want_c, want_s = c.numpy().copy(), cu.f64(s).copy()
        qc, qs = qu.quantise(cu.f64(x))
        qc = qu.packed(qc)
        for b in range(B):
            for t in range(T if counts is None else int(np.clip(counts[b], 0, T))):
                if 0 <= start[b] + t < Lk:
                    want_c[b, start[b] + t] = qc[b, t]
                    want_s[b, :, start[b] + t] = qs[b, t]
        assert np.array_equal(got_c.cpu().numpy(), want_c)
        assert np.array_equal(cu.f64(got_s), want_s)


def test_write_rows_that_are_not_finite(mha):  # noqa: F811
    """A NaN, an infinity, a spread past float32: offset NaN, codes 0, and the rows
    beside them as ever.  The largest finite rows stay finite."""
    k = cu.random_rows(3, (1, 6, 1, 64))
    k[0, 0, 0, 5] = float("nan")
    k[0, 1, 0, 63] = float("-inf")
    k[0, 2, 0, 0] = float("inf")
    k[0, 3, 0, :2] = torch.tensor([3.3e38, -3.3e38])
    k[0, 4, 0, :2] = torch.tensor([3.3e38, 0.0])
    dev = [torch.full((1, 6, 1, 32), 0xAA, dtype=torch.uint8, device="cuda") for _ in range(2)] + \
        [torch.zeros((1, 1, 6, 2), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    mha.mha_cache_write_q4(k.cuda(), k.cuda(), *dev, i32([0]).cuda())
    back = mha.mha_cache_read_q4(*dev, i32([6]).cuda())
    assert mha.mha_sync_status() == 0
    for got, pairs, x in zip(dev[:2], dev[2:], back):
        assert torch.isnan(pairs[0, 0, :4, 0]).all() and torch.count_nonzero(got[0, :4]) == 0
        codes, want = qu.quantise(cu.f64(k)[:, 4:])
        assert np.array_equal(got[0, 4:].cpu().numpy(), qu.packed(codes)[0])
        assert np.array_equal(cu.f64(pairs)[0, 0, 4:], want[0, :, 0])
        assert torch.isnan(x[0, :4]).all() and torch.isfinite(x[0, 4:]).all()


READS = [(3, 5, 2, 32, [5, 0, 3]), (2, 70, 9, 128, [69, -2]), (2, 33, 3, 96, [33, 100]),
         (1, 130, 4, 256, [129]), (64, 512, 8, 64, None)]


@pytest.mark.parametrize("shape", READS, ids=lambda s: "x".join(map(str, s[:4])))
def test_read(mha, shape):  # noqa: F811
    B, Lk, H, d, lens = shape
    if lens is None:
        lens = np.random.default_rng(4).integers(0, Lk + 1, size=B).tolist()
    codes, pairs = random_cache(5, B, Lk, H, d)
    dev = [c.cuda() for c in codes] + [s.cuda() for s in pairs]
    kept = torch.full((B, Lk, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = mha.mha_cache_read_q4(*dev, i32(lens).cuda(), k=kept.clone())
    assert mha.mha_sync_status() == 0
    for got, c, s, rest in ((k, codes[0], pairs[0], 7.0), (v, codes[1], pairs[1], 0.0)):
        # lo + c step in float32, then bf16
        want = torch.from_numpy(qu.values(qu.unpacked(c.numpy()), cu.f64(s))).float().to(torch.bfloat16)
        for b in range(B):
            want[b, max(0, lens[b]):] = rest
        assert torch.equal(got.cpu(), want)


# ------------------------------------------------------------- steps over a cache
def make_step(seed, B, T, H, H_kv, d, Lk, prefix, drafts, mask, with_drafts=True, std=1.0):
    """A case on the CPU: positions no row may see hold random codes and NaN pairs."""
    rng = np.random.default_rng(seed)
    case = {"q": cu.random_rows(seed, (B, T, H, d), std), "prefix": i32(prefix),
            "drafts": None if drafts is None else i32(drafts),
            "mask": cu.tree_bits(rng, B, T) if mask == "tree" else mask}
    ends = []
    for b in range(B):
        n = int(np.clip(prefix[b], 0, Lk))
        live = T if drafts is None else int(np.clip(drafts[b], 0, T))
        ends.append(min(Lk, n + (live if with_drafts else 0)))
    for n, s in (("k", 1), ("v", 2)):
        case[n + "c"], case[n + "s"] = qu.q4_cache(cu.random_rows(seed * 10 + s, (B, Lk, H_kv, d), std), ends, seed)
    case["ends"] = ends
    return case


def call_step(mha, g, with_drafts, **kw):  # noqa: F811
    caches = (g["kc"], g["vc"], g["ks"], g["vs"])
    if not with_drafts:
        return mha.mha_decode_q4(g["q"][:, 0].contiguous(), *caches, g["prefix"], return_lse=True, **kw)
    return mha.mha_decode_tree_q4(g["q"], *caches, g["prefix"], draft_lens=g["drafts"], tree_mask=g["mask"],
                                  return_lse=True, **kw)


def check_step(case, out, lse, with_drafts=True, scale=None, what=""):
    B, T, H, d = case["q"].shape
    Lk = case["kc"].shape[1]
    drafts = None if case["drafts"] is None else case["drafts"].numpy()
    mask = None if case["mask"] is None else case["mask"].numpy()

    def sees(b):
        return cu.visible(b, T, Lk, case["prefix"].numpy(), drafts, mask, with_drafts)

    (k, k_pairs), (v, v_pairs) = (qu.cache_f64(case[n + "c"], case[n + "s"]) for n in "kv")
    q = np.nan_to_num(cu.f64(case["q"]), nan=0.0)
    ref, lse_ref, size = cu.attention(q, k, v, sees, scale)
    qu.assert_out_close(out, q, k_pairs, v_pairs, ref, size, sees, max(case["ends"], default=0), scale, what)
    pu.assert_lse_close(lse.reshape(B, H, T), lse_ref, what)
    empty = torch.from_numpy(np.isneginf(lse_ref).transpose(0, 2, 1))
    assert torch.count_nonzero(out.cpu().reshape(B, T, H, d)[empty]) == 0


DECODES = [
    # B, H, H_kv, d, Lk, lens
    (8, 4, 4, 64, 300, [300, 0, 1, 127, 128, 129, 299, 255]),
    (9, 2, 2, 128, 70, [1, 15, 16, 17, 31, 32, 33, 63, 64]),
    (3, 8, 2, 128, 257, [257, 256, 1]),
    (1, 2, 2, 128, 5000, [4321]),
    (2, 6, 2, 256, 700, [700, 13]),
    (2, 3, 1, 32, 130, [130, 77]),
    (2, 5, 5, 96, 640, [640, 577]),
    (1, 32, 1, 64, 1000, [999]),             # 32 query heads on one key head
    (1, 40, 1, 128, 400, [400]),             # more rows than a block of rows
    (2, 8, 8, 224, 1, [1, 0]),
    (64, 16, 16, 64, 96, None),
    (1, 4, 1, 128, 40000, [39999]),          # many splits
    (3, 2, 2, 192, 3000, [64, 3000, -5]),
    (2, 4, 4, 160, 1000, [7, 2000]),         # a length past the capacity
    (40, 2, 1, 64, 3000, None),              # more sequences than a balanced launch has
]


@pytest.mark.parametrize("shape", DECODES, ids=lambda s: "x".join(map(str, s[:5])))
def test_decode(mha, shape):  # noqa: F811
    B, H, H_kv, d, Lk, lens = shape
    if lens is None:
        lens = np.random.default_rng(5).integers(1, Lk + 1, size=B).tolist()
    case = make_step(sum(shape[:5]), B, 1, H, H_kv, d, Lk, lens, None, None, with_drafts=False)
    out, lse = call_step(mha, on_gpu(case), False)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, with_drafts=False, what=str(shape[:5]))


TREES = [
    # B, T, H, H_kv, d, Lk, prefix, drafts, mask
    (2, 1, 4, 4, 64, 200, [199, 0], None, None),
    (3, 5, 4, 2, 128, 300, [255, 123, 0], [5, 0, 3], "tree"),
    (2, 12, 8, 8, 64, 300, [280, 121], None, "tree"),
    (1, 16, 4, 1, 128, 2000, [1900], None, None),              # 64 rows on one key head
    (2, 63, 4, 2, 128, 1100, [1000, 65], [63, 17], "tree"),    # 126 rows: blocks of rows
    (1, 64, 2, 2, 64, 128, [64], None, "tree"),                # drafts end with a tile
    (1, 65, 3, 3, 96, 400, [300], None, "tree"),               # two mask words
    (1, 200, 2, 1, 64, 700, [450], [199], "tree"),             # four words, drafts over tiles
    (2, 7, 16, 2, 256, 900, [800, 3], None, None),
    (2, 9, 2, 2, 64, 40, [36, 40], None, None),                # drafts run past the capacity
    (1, 256, 1, 1, 128, 256, [0], None, None),                 # no prefix: causal attention
    (4, 3, 6, 3, 32, 77, [70, 1, 74, 30], [3, 3, -1, 9], "tree"),
    (1, 8, 2, 2, 128, 33000, [32000], None, "tree"),           # many splits
    (2, 20, 3, 1, 224, 500, [460, 130], None, "tree"),
    (33, 4, 2, 2, 128, 400, None, None, "tree"),               # more sequences than a warp has lanes
    (5, 9, 96, 96, 64, 900, [890, 3, 500, 0, 100], None, "tree"),  # longest first
]


@pytest.mark.parametrize("shape", TREES, ids=lambda s: "x".join(map(str, s[:6])))
def test_tree(mha, shape):  # noqa: F811
    B, T, H, H_kv, d, Lk, prefix, drafts, mask = shape
    if prefix is None:
        prefix = np.random.default_rng(6).integers(0, Lk - T, size=B).tolist()
    case = make_step(sum(shape[:6]), B, T, H, H_kv, d, Lk, prefix, drafts, mask)
    out, lse = call_step(mha, on_gpu(case), True)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, what=str(shape[:6]))


@pytest.mark.parametrize("d", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("T,G", [(1, 1), (3, 2), (9, 1), (5, 7), (17, 4)])
def test_widths_and_rows(mha, d, T, G):  # noqa: F811
    case = make_step(d + T, 2, T, 2 * G, 2, d, 150, [140 - T, 100], None, "tree")
    out, lse = call_step(mha, on_gpu(case), True)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, what=f"d {d}, {T} x {G} rows")


def test_rows_that_see_nothing(mha):  # noqa: F811
    """A mask that leaves a row nothing (no prefix, no bit), rows that see only
    a sibling, and bits past the drafted tokens, which count for nothing."""
    bits = torch.tensor([[[0], [1], [4], [15]], [[0], [0], [0], [0]]], dtype=torch.int64)
    case = make_step(3, 2, 4, 2, 2, 64, 40, [0, 5], [3, 4], bits)
    out, lse = call_step(mha, on_gpu(case), True)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_drafted_positions_that_no_row_sees(mha, d):  # noqa: F811
    """They may hold anything, and so may the queries of rows past the drafted ones."""
    T = 70
    sees = np.tril(np.ones((T, T), dtype=bool))
    hidden = [0, 7, 33, 64, 68]
    sees[:, hidden] = False
    case = make_step(5, 1, T, 2, 1, d, 200, [100], [66], bits_of(sees))
    for n in "kv":
        for j in hidden:
            case[n + "s"][0, :, 100 + j] = torch.tensor([float("nan"), 0.0])
        case[n + "s"][0, :, 100, 1] = float("inf")
    case["q"][0, 66:] = float("nan")
    out, lse = call_step(mha, on_gpu(case), True)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_whose_first_key_comes_late(mha, d):  # noqa: F811
    """No prefix, 200 drafted tokens: rows whose only keys lie behind the first tile
    and score low are no empty rows; beside them rows that see the first, and rows that
    see nothing."""
    T = 200
    sees = np.zeros((T, T), dtype=bool)
    for i in range(T):
        if i % 4 == 0:
            sees[i, : i + 1] = True
        elif i % 4 == 1:
            sees[i, 130 + i % 60: 130 + i % 60 + 3] = True
        elif i % 4 == 2:
            sees[i, 199] = True
    case = make_step(31, 1, T, 2, 2, d, 230, [0], None, bits_of(sees))
    k = torch.zeros((1, 230, 2, d), dtype=torch.bfloat16)
    k[0, :, :, 0] = (8 + torch.arange(230) % 8).to(torch.bfloat16)[:, None]
    case["kc"], case["ks"] = qu.q4_cache(k)
    case["q"][:] = 0.0
    factor = torch.where(torch.arange(T) % 4 == 0, 1.0, torch.where(torch.arange(T) % 8 < 4, -12.5, -25.0))
    case["q"][0, :, :, 0] = factor.to(torch.bfloat16)[:, None]
    out, lse = call_step(mha, on_gpu(case), True)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse)


@pytest.mark.parametrize("scale,std", [(1.0, 1.0), (0.01, 1.0), (0.0, 0.05)])
def test_scales(mha, scale, std):  # noqa: F811
    """Peaked rows (scale 1 on N(0, 1) rows moves the reference often) and nearly
    uniform ones."""
    case = make_step(17, 2, 5, 4, 2, 128, 900, [890, 400], None, "tree", std=std)
    out, lse = call_step(mha, on_gpu(case), True, scale=scale)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, scale=scale or None, what=f"scale {scale}")


def test_rising_scores(mha):  # noqa: F811
    """Every key scores higher than the one before: the reference moves in every tile."""
    case = make_step(18, 1, 3, 2, 1, 64, 1300, [1290], None, None)
    k = torch.zeros((1, 1300, 1, 64), dtype=torch.bfloat16)
    k[0, :, 0, 0] = torch.linspace(0.0, 60.0, 1300).to(torch.bfloat16)
    case["q"][:] = 0.0
    case["q"][..., 0] = 8.0
    case["kc"], case["ks"] = qu.q4_cache(k)
    out, lse = call_step(mha, on_gpu(case), True)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse)


def test_uneven_rows(mha):  # noqa: F811
    """Values whose magnitudes differ by 2^40 from position to position (each weight is
    kept relative to the row's own largest contribution), rows of one value and of
    zeros among them, and rows far from 0 whose spread is small."""
    B, H, d, Lk = 2, 4, 128, 600
    rng = np.random.default_rng(6)
    case = make_step(19, B, 1, H, H, d, Lk, [600, 130], None, None, with_drafts=False)
    for n in ("k", "v"):
        x = cu.random_rows(20, (B, Lk, H, d)).float()
        x *= torch.from_numpy(np.exp2(rng.integers(-40 if n == "v" else -6, 1, size=(B, Lk, H, 1)))).float()
        x[:, ::7] = 0.0
        x[:, 1::7] = 1.5
        x[:, 2::7] = -2.0 + x[:, 2::7] * 2.0 ** -6
        case[n + "c"], case[n + "s"] = qu.q4_cache(x.to(torch.bfloat16))
    out, lse = call_step(mha, on_gpu(case), False)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, with_drafts=False)


def test_zero_values_and_queries(mha):  # noqa: F811
    case = make_step(21, 1, 1, 2, 2, 64, 300, [300], None, None, with_drafts=False)
    case["vc"], case["vs"] = qu.q4_cache(torch.zeros((1, 300, 2, 64), dtype=torch.bfloat16))
    case["q"][0, 0, 1] = 0.0
    out, lse = call_step(mha, on_gpu(case), False)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, with_drafts=False)
    assert torch.count_nonzero(out) == 0
    assert abs(float(lse[0, 1]) - np.log(300)) < 1e-5


def test_a_visible_row_that_is_not_finite_shows(mha):  # noqa: F811
    """A value row that was not finite when it was written makes the rows that see it
    NaN, and no others."""
    case = make_step(25, 2, 2, 2, 1, 64, 100, [60, 60], None, None)
    case["vs"][0, 0, 61, 0] = float("nan")        # sequence 0's second drafted token
    out, _ = call_step(mha, on_gpu(case), True)
    assert mha.mha_sync_status() == 0
    assert torch.isnan(out[0, 1]).all() and torch.isfinite(out[1]).all()


def test_decode_matches_a_tree_of_one(mha):  # noqa: F811
    """A decode step whose own key is cached sees what a tree of one drafted token
    after a prefix one shorter sees."""
    case = make_step(22, 3, 1, 8, 4, 128, 700, [699, 20, 0], None, None)
    g = on_gpu(case)
    tree, lse_t = call_step(mha, g, True)
    g["prefix"] = g["prefix"] + 1
    one, lse_1 = call_step(mha, g, False)
    assert mha.mha_sync_status() == 0
    assert torch.equal(tree[:, 0], one) and torch.equal(lse_t[:, :, 0], lse_1)


def test_far_offsets(mha):  # noqa: F811
    """A cache of more than 2^32 bytes: the last sequence's rows start past it."""
    B, H_kv, d, Lk, n = 3, 8, 256, 1_500_000, 2000
    case = make_step(23, 1, 3, 16, H_kv, d, n, [n - 3], None, None)
    big = on_gpu(case)
    for c in ("kc", "vc"):
        t = torch.zeros((B, Lk, H_kv, d // 2), dtype=torch.uint8, device="cuda")
        t[B - 1, :n] = big[c][0]
        big[c] = t
    assert big["kc"].numel() > 2 ** 32
    for c in ("ks", "vs"):
        t = torch.zeros((B, H_kv, Lk, 2), dtype=torch.bfloat16, device="cuda")
        t[B - 1, :, :n] = big[c][0]
        big[c] = t
    big["q"] = big["q"].expand(B, -1, -1, -1).contiguous()
    big["prefix"] = i32([0, 0, n - 3]).cuda()
    big["drafts"] = i32([0, 0, 3]).cuda()
    out, lse = call_step(mha, big, True)
    assert mha.mha_sync_status() == 0
    check_step(case, out[B - 1:], lse[B - 1:])
    assert torch.count_nonzero(out[:B - 1]) == 0


def test_write_far_offsets(mha):  # noqa: F811
    B, H, d, Lk = 2, 8, 256, 2_200_000
    k, v = cu.random_rows(1, (B, 3, H, d)), cu.random_rows(2, (B, 3, H, d))
    dev = [torch.zeros((B, Lk, H, d // 2), dtype=torch.uint8, device="cuda") for _ in range(2)] + \
        [torch.zeros((B, H, Lk, 2), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    mha.mha_cache_write_q4(k.cuda(), v.cuda(), *dev, i32([5, Lk - 2]).cuda())
    assert mha.mha_sync_status() == 0
    codes, pairs = qu.quantise(cu.f64(v))
    assert np.array_equal(dev[1][1, Lk - 2:].cpu().numpy(), qu.packed(codes)[1, :2])
    assert np.array_equal(cu.f64(dev[3][1, :, Lk - 2:]), pairs[1, :2].transpose(1, 0, 2))
    assert torch.count_nonzero(dev[1][1, :Lk - 2]) == 0 and torch.count_nonzero(dev[1][0, 8:]) == 0


# ------------------------------------------------------------- streams, graphs, buffers
@pytest.mark.parametrize("with_drafts", [False, True], ids=["decode", "tree"])
def test_repeatable_and_other_streams(mha, with_drafts):  # noqa: F811
    """The same bits on every call, on another stream (as an object and as a handle),
    from two streams at once, and from a captured graph replayed after its inputs
    changed."""
    cases = [on_gpu(make_step(30 + i, 2, 5 if with_drafts else 1, 8, 2, 128, 9000, [8000, 33], None,
                              "tree" if with_drafts else None, with_drafts)) for i in range(2)]
    first = [call_step(mha, g, with_drafts) for g in cases]
    for g, (out, lse) in zip(cases, first):
        again = call_step(mha, g, with_drafts)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [call_step(mha, g, with_drafts, stream=s if i else s.cuda_stream)
               for i, (g, s) in enumerate(zip(cases, streams))]
        torch.cuda.synchronize()
        for (a, la), (b, lb) in zip(got, first):
            assert torch.equal(a, b) and torch.equal(la, lb)
    graph = torch.cuda.CUDAGraph()
    g = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in cases[0].items()}
    with torch.cuda.graph(graph):
        captured = call_step(mha, g, with_drafts)
    for i in (1, 0):
        for n, t in cases[i].items():
            if torch.is_tensor(t):
                g[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured[0], first[i][0]) and torch.equal(captured[1], first[i][1])
    assert mha.mha_sync_status() == 0


@pytest.mark.parametrize("with_drafts", [False, True], ids=["decode", "tree"])
def test_steps_wait_for_their_memory(mha, with_drafts):  # noqa: F811
    g = on_gpu(make_step(60, 2, 5 if with_drafts else 1, 8, 2, 128, 9000, [8000, 33], None, None, with_drafts))
    want = call_step(mha, g, with_drafts)
    got, reused, kept = behind_a_reader(want[0], lambda s: call_step(mha, g, with_drafts, stream=s))
    assert mha.mha_sync_status() == 0
    assert reused and kept
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_read_waits_for_its_memory(mha):  # noqa: F811
    codes, pairs = qu.q4_cache(cu.random_rows(1, (3, 400, 4, 64)))
    dev = [codes.cuda(), codes.cuda(), pairs.cuda(), pairs.cuda(), i32([400, 0, 77]).cuda()]
    want = mha.mha_cache_read_q4(*dev)
    got, reused, kept = behind_a_reader(want[0], lambda s: mha.mha_cache_read_q4(*dev, stream=s))
    assert mha.mha_sync_status() == 0
    assert reused and kept
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_caller_buffers(mha):  # noqa: F811
    """out, lse and the workspace of the caller's, with guards around them that stay
    as they were."""
    case = make_step(40, 2, 3, 4, 2, 64, 5000, [4990, 100], [3, 2], "tree")
    g = on_gpu(case)
    B, T, H, d = case["q"].shape
    guard = torch.full((B * T * H * d + 128,), 5.0, dtype=torch.bfloat16, device="cuda")
    out = guard[64:-64].view(B, T, H, d)
    lguard = torch.full((B * H * T + 8,), 5.0, device="cuda")
    lse = lguard[4:-4].view(B, H, T)
    need = mha.decode_tree_q4_workspace_bytes(B, T, H, 2, 5000, d)
    assert need >= 16
    ws = torch.full((need + 256,), 0xAB, dtype=torch.uint8, device="cuda")
    r = call_step(mha, g, True, out=out, lse=lse, workspace=ws[:need])
    assert mha.mha_sync_status() == 0
    assert r[0] is out and r[1] is lse
    check_step(case, out, lse)
    assert (guard[:64] == 5.0).all() and (guard[-64:] == 5.0).all()
    assert (lguard[:4] == 5.0).all() and (lguard[-4:] == 5.0).all()
    assert (ws[need:] == 0xAB).all()


def test_no_keys_at_all(mha):  # noqa: F811
    case = make_step(41, 2, 3, 4, 2, 64, 6, [0, 0], [0, 0], None)
    g = on_gpu(case)
    for n in "kv":
        g[n + "c"] = g[n + "c"][:, :0].contiguous()
        g[n + "s"] = g[n + "s"][:, :, :0].contiguous()
    out, lse = call_step(mha, g, True)
    assert mha.mha_sync_status() == 0
    assert torch.count_nonzero(out) == 0 and torch.isneginf(lse).all()


# ------------------------------------------------------------------- together
def test_a_decoding_loop(mha):  # noqa: F811
    """Prompts written in 4 bits, decoded a token at a time, a beam step's fork, a tree
    of drafted tokens verified, its accepted branch compacted, the cache read back:
    each step against the float64 form over the values that the cache should hold."""
    B, H, H_kv, d, Lk, T0, T = 4, 8, 4, 64, 200, 90, 10
    rng = np.random.default_rng(9)
    lens = [90, 90, 41, 41]                       # two prompts, two beams each
    cache = [torch.full((B, Lk, H_kv, d // 2), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2)] + \
        [torch.full((B, H_kv, Lk, 2), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    held = [np.zeros((B, Lk, H_kv, d)) for _ in range(2)]
    pairs = [np.zeros((B, H_kv, Lk, 2)) for _ in range(2)]

    def write(seed, n, start, counts):
        qkv = cu.random_rows(seed, (B, n, 3, H_kv, d)).cuda()
        k, v = qkv[:, :, 1], qkv[:, :, 2]
        mha.mha_cache_write_q4(k, v, *cache, i32(start).cuda(),
                               counts=None if counts is None else i32(counts).cuda())
        for x, h, p in zip((k, v), held, pairs):
            codes, new = qu.quantise(cu.f64(x))
            for b in range(B):
                m = n if counts is None else counts[b]
                h[b, start[b]:start[b] + m] = (new[b, :, :, :1] + codes[b] * new[b, :, :, 1:])[:m]
                p[b, :, start[b]:start[b] + m] = new[b, :m].transpose(1, 0, 2)

    def check(q, out, lse, sees, what):
        ref, lse_ref, size = cu.attention(cu.f64(q), *held, sees)
        qu.assert_out_close(out, cu.f64(q), *pairs, ref, size, sees, Lk, what=what)
        pu.assert_lse_close(lse.reshape(lse_ref.shape), lse_ref, what)

    write(100, T0, [0] * B, lens)
    for step in range(3):
        write(101 + step, 1, lens, None)
        lens = [n + 1 for n in lens]
        q = cu.random_rows(200 + step, (B, 1, H, d)).cuda()
        out, lse = mha.mha_decode_q4(q, *cache, i32(lens).cuda(), return_lse=True)
        assert mha.mha_sync_status() == 0
        check(q, out, lse, lambda b: cu.visible(b, 1, Lk, lens, None, None, False), f"step {step}")
        # the beams change places, or the second goes on with the first's
        parent = [1, 0, 2, 2] if step % 2 else [0, 0, 3, 2]
        mha.mha_cache_fork(cache[0], cache[1], i32(parent).cuda(), i32(lens).cuda(),
                           first=i32([85, 85, 0, 0]).cuda(), k_scale=cache[2], v_scale=cache[3])
        first = [85, 85, 0, 0]
        for x, y in zip(held, pairs):
            hx, py = x.copy(), y.copy()
            for b in range(B):
                x[b, first[b]:lens[b]] = hx[parent[b], first[b]:lens[b]]
                y[b, :, first[b]:lens[b]] = py[parent[b], :, first[b]:lens[b]]
    write(110, T, lens, None)
    bits = cu.tree_bits(rng, B, T)
    q = cu.random_rows(210, (B, T, H, d)).cuda()
    out, lse = mha.mha_decode_tree_q4(q, *cache, i32(lens).cuda(), tree_mask=bits.cuda(), return_lse=True)
    assert mha.mha_sync_status() == 0
    check(q, out, lse, lambda b: cu.visible(b, T, Lk, lens, None, bits.numpy()), "tree")
    path = [[j for j in range(T) if (int(bits[b, T - 1, 0]) >> j) & 1] for b in range(B)]
    accepted = [len(p) for p in path]
    rows = i32([j for p in path for j in p + [-1] * (T - len(p))]).reshape(B, T)
    mha.mha_cache_compact(cache[0], cache[1], i32(lens).cuda(), rows.cuda(), path_lens=i32(accepted).cuda(),
                          k_scale=cache[2], v_scale=cache[3])
    for x, y in zip(held, pairs):
        for b in range(B):
            at = [lens[b] + j for j in path[b]]
            x[b, lens[b]:lens[b] + accepted[b]] = x[b, at]
            y[b, :, lens[b]:lens[b] + accepted[b]] = y[b, :, at].transpose(1, 0, 2)
    lens = [n + a for n, a in zip(lens, accepted)]
    q = cu.random_rows(220, (B, 1, H, d)).cuda()
    out, lse = mha.mha_decode_q4(q, *cache, i32(lens).cuda(), return_lse=True)
    k16, v16 = mha.mha_cache_read_q4(*cache, i32(lens).cuda())
    assert mha.mha_sync_status() == 0
    check(q, out, lse, lambda b: cu.visible(b, 1, Lk, lens, None, None, False), "after the tree")
    for got, h in ((k16, held[0]), (v16, held[1])):
        want = torch.from_numpy(h).float().to(torch.bfloat16)
        for b in range(B):
            assert torch.equal(got[b, :lens[b]].cpu(), want[b, :lens[b]])
