"""The 8-bit cache (mha_cache_write_f8, mha_cache_read_f8) and the steps over a
cache (mha_decode_f8, mha_decode_tree, mha_decode_tree_f8) against their plain
float64 forms (cache_util)."""
import numpy as np
import pytest
import torch

from tests import cache_util as cu
from tests import parity_util as pu
from transformer_head_scaled_sdpa_gb300 import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mha():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for gpu tests")
    from transformer_head_scaled_sdpa_gb300 import binding, build
    build.build()
    return binding


def i32(v):
    return torch.tensor(list(v), dtype=torch.int32)


# ---------------------------------------------------------------- write, read
WRITES = [
    # B, T, H, d, Lk, start, counts, packed
    (3, 1, 2, 16, 5, [0, 4, 2], None, False),
    (2, 7, 3, 48, 20, [13, 0], None, True),                   # odd heads, three lanes of four
    (4, 33, 9, 64, 64, [31, 0, 40, -3], [33, 0, 33, 20], True),  # off both ends, none, more than a tile
    (1, 70, 17, 128, 101, [30], [69], False),
    (2, 40, 5, 256, 40, [0, 0], [100, -4], True),              # counts past T and below 0
    (2, 5, 4, 240, 300, [295, 297], None, False),
    (128, 1, 8, 64, 256, None, None, True),                    # a decode step's write
    (1, 1, 1, 128, 1, [0], [1], False),
]


def random_cache(seed, B, Lk, H, d):
    g = torch.Generator().manual_seed(seed)
    codes = [torch.randint(0, 256, (B, Lk, H, d), generator=g, dtype=torch.uint8) for _ in range(2)]
    scales = [torch.randint(0, 256, (B, H, Lk), generator=g, dtype=torch.uint8) for _ in range(2)]
    return codes, scales


def rows_of(seed, B, T, H, d, packed):
    """k, v on the GPU: row magnitudes from 2^-100 to 2^100, a zero row, values
    at the largest code's border; packed: inside a Q | K | V projection."""
    rng = np.random.default_rng(seed)
    x = cu.random_rows(seed, (B, T, 3, H, d)).float()
    x *= torch.from_numpy(np.exp2(rng.integers(-100, 100, size=(B, T, 3, H, 1)))).float()
    x[0, 0, 1, 0] = 0.0
    x[-1, -1, 2, -1] = torch.linspace(-448.0, 448.0, d)
    x[-1, -1, 1, -1, 0] = 3.0e38
    x = x.to(torch.bfloat16).cuda()
    if packed:
        return x[:, :, 1], x[:, :, 2]
    return x[:, :, 1].contiguous(), x[:, :, 2].contiguous()


@pytest.mark.parametrize("shape", WRITES, ids=lambda s: "x".join(map(str, s[:5])))
def test_write(mha, shape):
    B, T, H, d, Lk, start, counts, packed = shape
    if start is None:
        start = np.random.default_rng(2).integers(0, Lk, size=B).tolist()
    k, v = rows_of(7, B, T, H, d, packed)
    codes, scales = random_cache(8, B, Lk, H, d)
    dev = [c.cuda().view(torch.float8_e4m3fn) for c in codes] + [s.cuda() for s in scales]
    mha.mha_cache_write_f8(k, v, *dev, i32(start).cuda(),
                           counts=None if counts is None else i32(counts).cuda())
    assert mha.mha_sync_status() == 0
    for x, c, s, got_c, got_s in zip((k, v), codes, scales, dev[:2], dev[2:]):
        want_c, want_s = c.numpy().copy(), s.numpy().copy()
        qc, qs = cu.quantise(cu.f64(x))
        for b in range(B):
            for t in range(T if counts is None else int(np.clip(counts[b], 0, T))):
                if 0 <= start[b] + t < Lk:
                    want_c[b, start[b] + t] = qc[b, t]
                    want_s[b, :, start[b] + t] = qs[b, t]
        assert np.array_equal(cu.codes_of(got_c), want_c)
        assert np.array_equal(got_s.cpu().numpy(), want_s)


def test_write_keeps_nan_and_saturates_infinity(mha):
    k = torch.ones((1, 3, 1, 32), dtype=torch.bfloat16)
    k[0, 0, 0, 5] = float("nan")
    k[0, 1, 0, 6] = float("-inf")
    k[0, 2] = float("nan")
    v = torch.full_like(k, 2.0)
    c, s = torch.zeros((1, 4, 1, 32), dtype=torch.uint8), torch.zeros((1, 1, 4), dtype=torch.uint8)
    dev = [c.cuda().view(torch.float8_e4m3fn), c.cuda().view(torch.float8_e4m3fn), s.cuda(), s.cuda()]
    mha.mha_cache_write_f8(k.cuda(), v.cuda(), *dev, i32([0]).cuda())
    assert mha.mha_sync_status() == 0
    got, scale = cu.VALUES[cu.codes_of(dev[0])][0, :, 0], dev[2].cpu().numpy()[0, 0]
    assert np.isnan(got[0, 5]) and np.isnan(got[2]).all()
    assert np.array_equal(np.delete(got[0], 5), np.full(31, 256.0)) and scale[0] == 127 - 8
    assert got[1, 6] == -448.0 and scale[1] == 247           # largest code at the largest scale
    assert (cu.VALUES[cu.codes_of(dev[1])][0, :3] == 256.0).all()


def test_write_single_position_twice(mha):
    """Two steps in a row append: the second write leaves the first's row."""
    B, H, d, Lk = 2, 3, 64, 6
    k, v = cu.random_rows(1, (B, 2, H, d)), cu.random_rows(2, (B, 2, H, d))
    dev = [torch.zeros((B, Lk, H, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
           for _ in range(2)] + [torch.zeros((B, H, Lk), dtype=torch.uint8, device="cuda") for _ in range(2)]
    for t in range(2):
        mha.mha_cache_write_f8(k[:, t:t + 1].cuda(), v[:, t:t + 1].cuda(), *dev, i32([3 + t, t]).cuda())
    assert mha.mha_sync_status() == 0
    want, _ = cu.quantise(cu.f64(k))
    got = cu.codes_of(dev[0])
    assert np.array_equal(got[0, 3:5], want[0]) and np.array_equal(got[1, :2], want[1])
    assert (got[0, :3] == 0).all() and (got[1, 2:] == 0).all()


READS = [(3, 5, 2, 16, [5, 0, 3]), (2, 70, 9, 128, [69, -2]), (2, 33, 3, 48, [33, 100]),
         (1, 130, 4, 256, [129]), (64, 512, 8, 64, None)]


@pytest.mark.parametrize("shape", READS, ids=lambda s: "x".join(map(str, s[:4])))
def test_read(mha, shape):
    B, Lk, H, d, lens = shape
    if lens is None:
        lens = np.random.default_rng(4).integers(0, Lk + 1, size=B).tolist()
    rng = np.random.default_rng(5)
    codes = [rng.integers(0, 255, size=(B, Lk, H, d)).astype(np.uint8) for _ in range(2)]
    for c in codes:
        c[c == 0x7F] = 0x30
    scales = [rng.integers(63, 240, size=(B, H, Lk)).astype(np.uint8) for _ in range(2)]
    dev = [torch.from_numpy(c).cuda().view(torch.float8_e4m3fn) for c in codes] + \
        [torch.from_numpy(s).cuda() for s in scales]
    kept = torch.full((B, Lk, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = mha.mha_cache_read_f8(*dev, i32(lens).cuda(), k=kept.clone())
    assert mha.mha_sync_status() == 0
    for got, c, s, rest in ((k, codes[0], scales[0], 7.0), (v, codes[1], scales[1], 0.0)):
        want = cu.cache_values(c, s)
        for b in range(B):
            want[b, max(0, lens[b]):] = rest
        assert np.array_equal(cu.f64(got), want)


# ------------------------------------------------------------- steps over a cache
def on_gpu(case):
    return {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in case.items()}


def make_step(seed, B, T, H, H_kv, d, Lk, prefix, drafts, mask, f8, with_drafts=True, std=1.0):
    """A case on the CPU: positions no row may see hold NaN (8-bit: NaN codes and
    the largest scale)."""
    rng = np.random.default_rng(seed)
    case = {"q": cu.random_rows(seed, (B, T, H, d), std), "prefix": i32(prefix),
            "drafts": None if drafts is None else i32(drafts),
            "mask": cu.tree_bits(rng, B, T) if mask == "tree" else mask}
    ends = []
    for b in range(B):
        n = int(np.clip(prefix[b], 0, Lk))
        live = T if drafts is None else int(np.clip(drafts[b], 0, T))
        ends.append(min(Lk, n + (live if with_drafts else 0)))
    for n_, s in (("k", 1), ("v", 2)):
        x = cu.random_rows(seed * 10 + s, (B, Lk, H_kv, d), std)
        if f8:
            case[n_ + "c"], case[n_ + "s"] = cu.f8_cache(x, ends)
            case[n_ + "_ref"] = cu.cache_values(
                np.where(cu.codes_of(case[n_ + "c"]) == 0x7F, 0, cu.codes_of(case[n_ + "c"])),
                np.minimum(case[n_ + "s"].numpy(), 200))
        else:
            case[n_ + "_ref"] = cu.f64(x)
            for b, e in enumerate(ends):
                x[b, e:] = float("nan")
            case[n_ + "c"] = x
    case["ends"] = ends
    return case


def call_step(mha, g, f8, with_drafts, **kw):
    if not with_drafts:
        return mha.mha_decode_f8(g["q"][:, 0].contiguous(), g["kc"], g["vc"], g["ks"], g["vs"],
                                 g["prefix"], return_lse=True, **kw)
    caches = (g["kc"], g["vc"]) + ((g["ks"], g["vs"]) if f8 else ())
    fn = mha.mha_decode_tree_f8 if f8 else mha.mha_decode_tree
    return fn(g["q"], *caches, g["prefix"], draft_lens=g["drafts"], tree_mask=g["mask"],
              return_lse=True, **kw)


def check_step(case, out, lse, f8, with_drafts=True, scale=None, what=""):
    B, T, H, d = case["q"].shape
    Lk = case["k_ref"].shape[1]
    drafts = None if case["drafts"] is None else case["drafts"].numpy()
    mask = None if case["mask"] is None else case["mask"].numpy()
    ref, lse_ref, size = cu.attention(
        cu.f64(case["q"]), case["k_ref"], case["v_ref"],
        lambda b: cu.visible(b, T, Lk, case["prefix"].numpy(), drafts, mask, with_drafts), scale)
    cu.assert_out_close(out, ref, size, max(case["ends"], default=0), f8, what)
    pu.assert_lse_close(lse.reshape(B, H, T), lse_ref, what)
    empty = torch.from_numpy(np.isneginf(lse_ref).transpose(0, 2, 1))
    assert torch.count_nonzero(out.cpu().reshape(B, T, H, d)[empty]) == 0


DECODES = [
    # B, H, H_kv, d, Lk, lens
    (8, 4, 4, 64, 300, [300, 0, 1, 127, 128, 129, 299, 255]),
    (3, 8, 2, 128, 257, [257, 256, 1]),
    (1, 2, 2, 128, 5000, [4321]),
    (2, 6, 2, 256, 700, [700, 13]),
    (2, 3, 1, 16, 130, [130, 77]),
    (2, 5, 5, 80, 640, [640, 577]),
    (1, 32, 1, 64, 1000, [999]),             # 32 query heads on one key head
    (1, 40, 1, 128, 400, [400]),             # more rows than a block of rows
    (2, 8, 8, 208, 1, [1, 0]),
    (64, 16, 16, 64, 96, None),
    (1, 4, 1, 128, 40000, [39999]),          # many splits
    (3, 2, 2, 192, 3000, [64, 3000, -5]),
]


@pytest.mark.parametrize("shape", DECODES, ids=lambda s: "x".join(map(str, s[:5])))
def test_decode_f8(mha, shape):
    B, H, H_kv, d, Lk, lens = shape
    if lens is None:
        lens = np.random.default_rng(5).integers(1, Lk + 1, size=B).tolist()
    case = make_step(sum(shape[:5]), B, 1, H, H_kv, d, Lk, lens, None, None, True, with_drafts=False)
    out, lse = call_step(mha, on_gpu(case), True, False)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, True, with_drafts=False, what=str(shape[:5]))


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
    (4, 3, 6, 3, 48, 77, [70, 1, 74, 30], [3, 3, -1, 9], "tree"),
    (1, 8, 2, 2, 128, 33000, [32000], None, "tree"),           # many splits
]


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "f8"])
@pytest.mark.parametrize("shape", TREES, ids=lambda s: "x".join(map(str, s[:6])))
def test_tree(mha, shape, f8):
    B, T, H, H_kv, d, Lk, prefix, drafts, mask = shape
    case = make_step(sum(shape[:6]), B, T, H, H_kv, d, Lk, prefix, drafts, mask, f8)
    out, lse = call_step(mha, on_gpu(case), f8, True)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, f8, what=str(shape[:6]))


@pytest.mark.parametrize("d", [8, 24, 56, 136, 232])
def test_tree_bf16_widths(mha, d):
    case = make_step(d, 2, 6, 4, 2, d, 150, [140, 100], None, "tree", False)
    out, lse = call_step(mha, on_gpu(case), False, True)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, False, what=f"d {d}")


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "f8"])
def test_tree_rows_that_see_nothing(mha, f8):
    """A mask that leaves a row nothing (no prefix, no bit), rows that see only
    a sibling, and bits past the drafted tokens, which count for nothing."""
    B, T = 2, 4
    bits = torch.tensor([[[0], [1], [4], [15]], [[0], [0], [0], [0]]], dtype=torch.int64)
    case = make_step(3, B, T, 2, 2, 64, 40, [0, 5], [3, 4], bits, f8)
    out, lse = call_step(mha, on_gpu(case), f8, True)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, f8)


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "f8"])
@pytest.mark.parametrize("scale,std", [(1.0, 1.0), (0.01, 1.0), (0.0, 0.05)])
def test_tree_scales(mha, f8, scale, std):
    """Peaked rows (scale 1 on N(0, 1) rows moves the reference maximum often)
    and nearly uniform ones."""
    case = make_step(17, 2, 5, 4, 2, 128, 900, [890, 400], None, "tree", f8, std=std)
    out, lse = call_step(mha, on_gpu(case), f8, True, scale=scale)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, f8, scale=scale or None, what=f"scale {scale}")


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "f8"])
def test_tree_rising_scores(mha, f8):
    """Every key scores higher than the one before: the running reference moves
    in every tile."""
    case = make_step(18, 1, 3, 2, 1, 64, 1300, [1290], None, None, f8)
    ramp = torch.linspace(0.0, 60.0, 1300)
    k = torch.zeros((1, 1300, 1, 64), dtype=torch.bfloat16)
    k[0, :, 0, 0] = ramp.to(torch.bfloat16)
    case["q"][:] = 0.0
    case["q"][..., 0] = 8.0
    if f8:
        case["kc"], case["ks"] = cu.f8_cache(k)
        case["k_ref"] = cu.cache_values(cu.codes_of(case["kc"]), case["ks"].numpy())
    else:
        case["kc"], case["k_ref"] = k, cu.f64(k)
    out, lse = call_step(mha, on_gpu(case), f8, True)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, f8)


def test_decode_f8_uneven_rows(mha):
    """Cached rows whose magnitudes differ by 2^40 from position to position:
    each weight is kept relative to the row's own largest contribution."""
    B, H, d, Lk = 2, 4, 128, 600
    rng = np.random.default_rng(6)
    case = make_step(19, B, 1, H, H, d, Lk, [600, 130], None, None, True, with_drafts=False)
    for n in ("k", "v"):
        x = cu.random_rows(20, (B, Lk, H, d)).float()
        x *= torch.from_numpy(np.exp2(rng.integers(-40 if n == "v" else -6, 1, size=(B, Lk, H, 1)))).float()
        case[n + "c"], case[n + "s"] = cu.f8_cache(x.to(torch.bfloat16))
        case[n + "_ref"] = cu.cache_values(cu.codes_of(case[n + "c"]), case[n + "s"].numpy())
    out, lse = call_step(mha, on_gpu(case), True, False)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, True, with_drafts=False)


def test_decode_f8_zero_values(mha):
    case = make_step(21, 1, 1, 2, 2, 64, 300, [300], None, None, True, with_drafts=False)
    case["vc"], case["vs"] = cu.f8_cache(torch.zeros((1, 300, 2, 64), dtype=torch.bfloat16))
    case["v_ref"] = np.zeros_like(case["v_ref"])
    out, lse = call_step(mha, on_gpu(case), True, False)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, True, with_drafts=False)
    assert torch.count_nonzero(out) == 0


def test_decode_f8_matches_a_tree_of_one(mha):
    """A decode step whose own key is cached sees what a tree of one drafted
    token after a prefix one shorter sees."""
    case = make_step(22, 3, 1, 8, 4, 128, 700, [699, 20, 0], None, None, True)
    g = on_gpu(case)
    tree, lse_t = call_step(mha, g, True, True)
    g["prefix"] = g["prefix"] + 1
    one, lse_1 = call_step(mha, g, True, False)
    assert mha.mha_sync_status() == 0
    assert torch.equal(tree[:, 0], one) and torch.equal(lse_t[:, :, 0], lse_1)


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "f8"])
def test_far_offsets(mha, f8):
    """A cache of more than 2^32 bytes: the last sequence's rows start past it."""
    B, H_kv, d, Lk = 3, 8, 256, 800_000 if f8 else 400_000
    g = torch.Generator(device="cuda").manual_seed(5)
    n = 2000
    case = make_step(23, 1, 3, 16, H_kv, d, n, [n - 3], None, None, f8)
    dtype = torch.uint8 if f8 else torch.bfloat16
    big = on_gpu(case)
    for c in ("kc", "vc"):
        t = torch.zeros((B, Lk, H_kv, d), dtype=dtype, device="cuda")
        t[B - 1, :n] = big[c].view(dtype)[0]
        big[c] = t.view(torch.float8_e4m3fn) if f8 else t
    assert big["kc"].numel() * (1 if f8 else 2) > 2 ** 32
    for c in ("ks", "vs"):
        if f8:
            t = torch.zeros((B, H_kv, Lk), dtype=torch.uint8, device="cuda")
            t[B - 1, :, :n] = big[c][0]
            big[c] = t
    big["q"] = big["q"].expand(B, -1, -1, -1).contiguous()
    big["prefix"] = i32([0, 0, n - 3]).cuda()
    big["drafts"] = i32([0, 0, 3]).cuda()
    out, lse = call_step(mha, big, f8, True)
    assert mha.mha_sync_status() == 0
    check_step(case, out[B - 1:], lse[B - 1:], f8)
    assert torch.count_nonzero(out[:B - 1]) == 0
    del g


def test_write_far_offsets(mha):
    B, H, d, Lk = 2, 8, 256, 1_100_000
    k, v = cu.random_rows(1, (B, 3, H, d)), cu.random_rows(2, (B, 3, H, d))
    dev = [torch.zeros((B, Lk, H, d), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
           for _ in range(2)] + [torch.zeros((B, H, Lk), dtype=torch.uint8, device="cuda") for _ in range(2)]
    mha.mha_cache_write_f8(k.cuda(), v.cuda(), *dev, i32([5, Lk - 2]).cuda())
    assert mha.mha_sync_status() == 0
    codes, scales = cu.quantise(cu.f64(v))
    got = dev[1].view(torch.uint8)
    assert np.array_equal(got[1, Lk - 2:].cpu().numpy(), codes[1, :2])
    assert np.array_equal(dev[3][1, :, Lk - 2:].cpu().numpy(), scales[1, :2].T)
    assert torch.count_nonzero(got[1, :Lk - 2]) == 0 and torch.count_nonzero(got[0, 8:]) == 0


# ------------------------------------------------------------------- together
def test_a_run_of_them(mha):
    """Prompts written in 8 bits, decoded a token at a time, a tree of drafted
    tokens verified, the accepted branch committed, the cache read back: each
    step against the float64 form over the values the cache holds."""
    B, H, H_kv, d, Lk, T0 = 3, 8, 4, 64, 200, 90
    rng = np.random.default_rng(9)
    counts = [90, 41, 1]
    cache = [torch.full((B, Lk, H_kv, d), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
             for _ in range(2)] + [torch.full((B, H_kv, Lk), 255, dtype=torch.uint8, device="cuda")
                                   for _ in range(2)]
    held = [np.zeros((B, Lk, H_kv, d)), np.zeros((B, Lk, H_kv, d))]

    def write(seed, T, start, counts):
        qkv = cu.random_rows(seed, (B, T, 3, H_kv, d)).cuda()
        k, v = qkv[:, :, 1], qkv[:, :, 2]
        mha.mha_cache_write_f8(k, v, *cache, i32(start).cuda(),
                               counts=None if counts is None else i32(counts).cuda())
        for x, h in ((k, held[0]), (v, held[1])):
            codes, scales = cu.quantise(cu.f64(x))
            values = cu.VALUES[codes] * np.exp2(scales.astype(np.float64) - 127)[..., None]
            for b in range(B):
                for t in range(T if counts is None else counts[b]):
                    h[b, start[b] + t] = values[b, t]
        return k, v

    write(100, T0, [0] * B, counts)
    lens = list(counts)
    for step in range(3):
        write(101 + step, 1, lens, None)
        lens = [n + 1 for n in lens]
        q = cu.random_rows(200 + step, (B, H, d)).cuda()
        out, lse = mha.mha_decode_f8(q, *cache, i32(lens).cuda(), return_lse=True)
        assert mha.mha_sync_status() == 0
        ref, lse_ref, size = cu.attention(cu.f64(q)[:, None], *held,
                                          lambda b: cu.visible(b, 1, Lk, lens, None, None, False))
        cu.assert_out_close(out, ref, size, Lk, True, f"step {step}")
        pu.assert_lse_close(lse.reshape(B, H, 1), lse_ref, f"step {step}")
    T = 10
    k, v = write(110, T, lens, None)
    bits = cu.tree_bits(rng, B, T)
    q = cu.random_rows(210, (B, T, H, d)).cuda()
    out, lse = mha.mha_decode_tree_f8(q, *cache, i32(lens).cuda(), tree_mask=bits.cuda(), return_lse=True)
    assert mha.mha_sync_status() == 0
    ref, lse_ref, size = cu.attention(cu.f64(q), *held,
                                      lambda b: cu.visible(b, T, Lk, lens, None, bits.numpy()))
    cu.assert_out_close(out, ref, size, Lk, True, "tree")
    pu.assert_lse_close(lse, lse_ref, "tree")
    # the branch of the last drafted token is accepted: its rows move up behind the prefix
    path = [[j for j in range(T) if (int(bits[b, T - 1, 0]) >> j) & 1] for b in range(B)]
    accepted = [len(p) for p in path]
    rows = torch.tensor([p + [0] * (T - len(p)) for p in path], device="cuda")
    at = torch.arange(B, device="cuda")[:, None]
    mha.mha_cache_write_f8(k[at, rows].contiguous(), v[at, rows].contiguous(), *cache, i32(lens).cuda(),
                           counts=i32(accepted).cuda())
    for h in held:
        for b in range(B):
            h[b, lens[b]:lens[b] + accepted[b]] = h[b, [lens[b] + j for j in path[b]]]
    lens = [n + a for n, a in zip(lens, accepted)]
    k16, v16 = mha.mha_cache_read_f8(*cache, i32(lens).cuda())
    assert mha.mha_sync_status() == 0
    for got, h in ((k16, held[0]), (v16, held[1])):
        for b in range(B):
            assert np.array_equal(cu.f64(got)[b, :lens[b]], h[b, :lens[b]])
    # ... and the bf16 entries read what came back: the forward with the same key lengths
    q = cu.random_rows(220, (B, 1, H, d)).cuda()
    one, lse_1 = mha.mha_decode_f8(q, *cache, i32(lens).cuda(), return_lse=True)
    full, lse_f = mha.mha_fwd(q, k16.repeat_interleave(H // H_kv, 2), v16.repeat_interleave(H // H_kv, 2),
                              mask_kind=inputs.MASK_KEY_PADDING, key_lens=i32(lens).cuda(), return_lse=True)
    assert mha.mha_sync_status() == 0
    assert (one.float() - full.float()).abs().max() <= 2 ** -6
    assert (lse_1.reshape(-1) - lse_f.reshape(-1)).abs().max() <= 1e-3


@pytest.mark.parametrize("kind", ["decode_f8", "tree", "tree_f8"])
def test_repeatable_and_other_streams(mha, kind):
    """The same bits on every call, on another stream (as an object and as a
    handle), from two streams at once, and from a captured graph replayed after
    its inputs changed."""
    f8, with_drafts = kind != "tree", kind != "decode_f8"
    cases = [on_gpu(make_step(30 + i, 2, 5 if with_drafts else 1, 8, 2, 128, 9000, [8000, 33], None,
                              "tree" if with_drafts else None, f8, with_drafts)) for i in range(2)]
    first = [call_step(mha, g, f8, with_drafts) for g in cases]
    for g, (out, lse) in zip(cases, first):
        again = call_step(mha, g, f8, with_drafts)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [call_step(mha, g, f8, with_drafts, stream=s if i else s.cuda_stream)
               for i, (g, s) in enumerate(zip(cases, streams))]
        torch.cuda.synchronize()
        for (a, la), (b, lb) in zip(got, first):
            assert torch.equal(a, b) and torch.equal(la, lb)
    graph = torch.cuda.CUDAGraph()
    g = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in cases[0].items()}
    with torch.cuda.graph(graph):
        captured = call_step(mha, g, f8, with_drafts)
    for i in (1, 0):
        for n, t in cases[i].items():
            if torch.is_tensor(t):
                g[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured[0], first[i][0]) and torch.equal(captured[1], first[i][1])
    assert mha.mha_sync_status() == 0


def test_caller_buffers(mha):
    """out, lse and the workspace of the caller's, with guard rows around out
    and lse that stay as they were."""
    case = make_step(40, 2, 3, 4, 2, 64, 5000, [4990, 100], [3, 2], "tree", True)
    g = on_gpu(case)
    B, T, H, d = case["q"].shape
    guard = torch.full((B * T * H * d + 128,), 5.0, dtype=torch.bfloat16, device="cuda")
    out = guard[64:-64].view(B, T, H, d)
    lguard = torch.full((B * H * T + 8,), 5.0, device="cuda")
    lse = lguard[4:-4].view(B, H, T)
    need = mha.decode_tree_f8_workspace_bytes(B, T, H, 2, 5000, d)
    ws = torch.full((need + 256,), 0xAB, dtype=torch.uint8, device="cuda")
    r = call_step(mha, g, True, True, out=out, lse=lse, workspace=ws[:max(need, 16)])
    assert mha.mha_sync_status() == 0
    assert r[0] is out and r[1] is lse
    check_step(case, out, lse, True)
    assert (guard[:64] == 5.0).all() and (guard[-64:] == 5.0).all()
    assert (lguard[:4] == 5.0).all() and (lguard[-4:] == 5.0).all()
    assert (ws[need:] == 0xAB).all() if need >= 16 else True


def test_no_keys_at_all(mha):
    for f8 in (False, True):
        case = make_step(41, 2, 3, 4, 2, 64, 6, [0, 0], [0, 0], None, f8)
        g = on_gpu(case)
        for n in ("kc", "vc"):
            g[n] = g[n][:, :0].contiguous()
        for n in ("ks", "vs"):
            if f8:
                g[n] = g[n][:, :, :0].contiguous()
        out, lse = call_step(mha, g, f8, True)
        assert mha.mha_sync_status() == 0
        assert torch.count_nonzero(out) == 0 and torch.isneginf(lse).all()
