"""The forms a step over a cache takes beside that of a few rows over a long
cache: many rows of a bf16 cache (rows along the tensor core's M), a row or two
over a short 8-bit cache (CUDA cores), and key splits of ragged batches; against
the plain float64 forms, with the tolerances of cache_util."""
import numpy as np
import pytest
import torch

from tests import cache_util as cu
from tests import parity_util as pu
from tests.test_cache_gpu import call_step, check_step, i32, make_step, mha, on_gpu  # noqa: F401

pytestmark = pytest.mark.gpu

BLOCK_THREADS, SHORT_THREADS = 640, 128   # what the launch report tells the forms apart by


BLOCKS = [
    # B, T, H, H_kv, d, Lk, prefix, drafts, mask
    (1, 65, 1, 1, 64, 70, [5], None, "tree"),                      # 65 rows, one tile of rows
    (2, 33, 4, 2, 128, 200, [130, 1], [33, 20], "tree"),           # 66 rows of two query heads
    (1, 128, 1, 1, 128, 128, [0], None, None),                     # exactly one tile of rows, no prefix
    (1, 129, 1, 1, 128, 260, [128], None, "tree"),                 # one row in the second tile
    (3, 64, 8, 2, 128, 600, [500, 0, 77], [64, 0, 1], "tree"),     # 256 rows; a sequence without drafts
    (2, 65, 8, 2, 64, 400, [300, 335], None, "tree"),              # 260 rows: a second block; end of the cache
    (1, 256, 4, 2, 96, 900, [640], [255], "tree"),                 # 512 rows, four mask words
    (2, 200, 6, 1, 48, 300, [90, 300], [200, 200], None),          # 1200 rows; drafts past the capacity
    (1, 70, 2, 2, 8, 150, [60], None, "tree"),                     # 8 features
    (2, 70, 2, 2, 24, 150, [60, 3], None, None),
    (1, 80, 1, 1, 56, 300, [200], None, "tree"),
    (1, 80, 2, 2, 72, 300, [220], None, "tree"),
    (1, 80, 1, 1, 120, 300, [127], [79], "tree"),
    (2, 40, 8, 4, 128, 9000, [8900, 300], None, "tree"),           # splits of a ragged batch
    (40, 17, 4, 1, 64, 256, None, None, "tree"),                   # more sequences than are balanced
]


@pytest.mark.parametrize("shape", BLOCKS, ids=lambda s: "x".join(map(str, s[:6])))
def test_many_rows(mha, shape):  # noqa: F811
    B, T, H, H_kv, d, Lk, prefix, drafts, mask = shape
    if prefix is None:
        prefix = np.random.default_rng(3).integers(0, Lk - T + 1, size=B).tolist()
    case = make_step(sum(shape[:6]), B, T, H, H_kv, d, Lk, prefix, drafts, mask, False)
    out, lse = call_step(mha, on_gpu(case), False, True)
    assert mha.last_launch_info()["block"] == BLOCK_THREADS
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, False, what=str(shape[:6]))


def test_many_rows_that_see_nothing(mha):  # noqa: F811
    """Rows whose mask leaves nothing (no prefix), some of them in a row tile of
    their own, and rows whose only key comes after tiles they do not see."""
    B, T = 1, 200
    bits = np.zeros((B, T, 4), dtype=np.uint64)
    for t in range(T):
        if t % 3 == 1:
            bits[0, t, 3] = np.uint64(1) << np.uint64(199 - 192)   # the last drafted key alone
        elif t % 3 == 2:
            bits[0, t, 0] = np.uint64(1) << np.uint64(t % 64)
    bits = torch.from_numpy(bits.view(np.int64))
    case = make_step(3, B, T, 2, 2, 64, 220, [0], None, bits, False)
    out, lse = call_step(mha, on_gpu(case), False, True)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, False)


@pytest.mark.parametrize("scale,std", [(1.0, 1.0), (0.01, 1.0), (0.0, 0.05)])
def test_many_rows_scales(mha, scale, std):  # noqa: F811
    case = make_step(17, 2, 60, 4, 2, 128, 900, [840, 400], None, "tree", False, std=std)
    out, lse = call_step(mha, on_gpu(case), False, True, scale=scale)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, False, scale=scale or None, what=f"scale {scale}")


def test_many_rows_rising_scores(mha):  # noqa: F811
    """Every key of some rows scores higher than the one before, of others lower,
    so that only some rows of a warp move their references."""
    T, n = 70, 1200
    case = make_step(18, 1, T, 1, 1, 64, n + T, [n], None, None, False)
    k = torch.zeros((1, n + T, 1, 64), dtype=torch.bfloat16)
    k[0, :, 0, 0] = torch.linspace(0.0, 60.0, n + T).to(torch.bfloat16)
    case["q"][:] = 0.0
    case["q"][0, :, 0, 0] = torch.where(torch.arange(T) % 3 == 0, 8.0, -4.0).to(torch.bfloat16)
    case["kc"], case["k_ref"] = k, cu.f64(k)
    out, lse = call_step(mha, on_gpu(case), False, True)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, False)


SHORTS = [
    # B, H, H_kv, d, Lk, lens
    (5, 3, 3, 64, 256, [256, 0, 1, 129, 255]),
    (4, 6, 3, 64, 128, [128, 127, 3, 0]),         # two query heads to a key head
    (3, 2, 2, 16, 300, [300, 31, 8]),
    (2, 5, 5, 48, 77, [77, 76]),                  # three lanes of four hold a row
    (2, 4, 4, 128, 128, [128, 17]),
    (3, 4, 2, 80, 100, [100, 64, 99]),
    (2, 3, 3, 256, 64, [64, 5]),
    (1, 2, 1, 240, 33, [33]),
    (1, 1, 1, 64, 1, [1]),
    (130, 8, 8, 64, 64, None),
    (3, 2, 2, 64, 100, [-7, 100, 200]),           # lengths outside the cache
]


@pytest.mark.parametrize("shape", SHORTS, ids=lambda s: "x".join(map(str, s[:5])))
def test_short_decode(mha, shape):  # noqa: F811
    B, H, H_kv, d, Lk, lens = shape
    if lens is None:
        lens = np.random.default_rng(5).integers(0, Lk + 1, size=B).tolist()
    case = make_step(sum(shape[:5]), B, 1, H, H_kv, d, Lk, lens, None, None, True, with_drafts=False)
    out, lse = call_step(mha, on_gpu(case), True, False)
    assert mha.last_launch_info()["block"] == SHORT_THREADS
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, True, with_drafts=False, what=str(shape[:5]))


@pytest.mark.parametrize("mask", [None, [1, 0, 1, 3, 0]], ids=["chain", "bits"])
def test_short_tree_of_one(mha, mask):  # noqa: F811
    """A single drafted token: with and without its own bit, of a sequence that has
    no drafted token, and past the end of the cache."""
    bits = None if mask is None else torch.tensor(mask, dtype=torch.int64).reshape(5, 1, 1)
    case = make_step(8, 5, 1, 4, 4, 64, 50, [49, 0, 20, 50, 7], [1, 1, 0, 1, 5], bits, True)
    out, lse = call_step(mha, on_gpu(case), True, True)
    assert mha.last_launch_info()["block"] == SHORT_THREADS
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, True)


def test_short_decode_magnitudes(mha):  # noqa: F811
    """V rows whose magnitudes differ by 2^160, up to the largest: nothing
    overflows, and the small rows keep their weight in the sum."""
    B, H, d, Lk = 2, 2, 64, 200
    rng = np.random.default_rng(6)
    case = make_step(19, B, 1, H, H, d, Lk, [200, 130], None, None, True, with_drafts=False)
    x = torch.rand((B, Lk, H, d), generator=torch.Generator().manual_seed(3)) + 0.5
    x *= torch.from_numpy(np.exp2(rng.choice([-40.0, 0.0, 120.0], size=(B, Lk, H, 1)))).float()
    case["vc"], case["vs"] = cu.f8_cache(x.to(torch.bfloat16))
    case["v_ref"] = cu.cache_values(cu.codes_of(case["vc"]), case["vs"].numpy())
    out, lse = call_step(mha, on_gpu(case), True, False)
    assert mha.last_launch_info()["block"] == SHORT_THREADS
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, True, with_drafts=False)


RAGGED = [
    # B, T, H, H_kv, d, Lk, lens
    (5, 3, 4, 2, 128, 12000, [11990, 3, 0, 700, 5000]),
    (2, 5, 2, 2, 256, 20000, [19000, 100]),
    (32, 2, 1, 1, 64, 6000, None),                 # the most that are balanced
    (33, 2, 1, 1, 64, 6000, None),
    (4, 1, 2, 1, 64, 40000, [39000, 0, 0, 0]),     # one sequence has all the splits
    (3, 1, 4, 4, 128, 5000, [0, 0, 0]),
    (33, 40, 2, 1, 64, 2000, None),                # 80 rows, not balanced
    (6, 40, 2, 1, 128, 3000, None),                # 80 rows, balanced
]


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "f8"])
@pytest.mark.parametrize("shape", RAGGED, ids=lambda s: "x".join(map(str, s[:6])))
def test_ragged_splits(mha, shape, f8):  # noqa: F811
    B, T, H, H_kv, d, Lk, lens = shape
    if lens is None:
        lens = (Lk * np.random.default_rng(1).random(B) ** 3).astype(int).tolist()
    case = make_step(sum(shape[:6]), B, T, H, H_kv, d, Lk, lens, None, "tree", f8)
    out, lse = call_step(mha, on_gpu(case), f8, True)
    assert mha.last_launch_info()["kernels"] == 2
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, f8, what=str(shape[:6]))


def test_read_of_negative_lengths(mha):  # noqa: F811
    """A length below zero reads nothing, the least one too."""
    x = cu.random_rows(1, (3, 40, 2, 16))
    codes, scales = cu.f8_cache(x)
    out = [torch.full((3, 40, 2, 16), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    mha.mha_cache_read_f8(codes.cuda(), codes.cuda(), scales.cuda(), scales.cuda(),
                          i32([-2 ** 31, -1, 1]).cuda(), k=out[0], v=out[1])
    assert mha.mha_sync_status() == 0
    for t in out:
        assert (t[:2] == 7.0).all() and (t[2, 1:] == 7.0).all() and not (t[2, 0] == 7.0).all()


LONGEST_FIRST = [
    # B, T, H, H_kv, d, Lk, prefix, f8: more units than CTAs run at once, no splits
    (3, 65, 60, 60, 64, 130, [3, 65, 20], False),       # rows along M
    (2, 70, 80, 80, 16, 90, [0, 20], False),
    (32, 3, 10, 10, 64, 60, None, False),
    (5, 2, 70, 70, 128, 200, [1, 198, 0, 60, 198], True),
    (4, 20, 40, 40, 256, 60, [40, 0, 7, 39], True),
]


@pytest.mark.parametrize("shape", LONGEST_FIRST, ids=lambda s: "x".join(map(str, s[:6])))
def test_longest_first(mha, shape):  # noqa: F811
    B, T, H, H_kv, d, Lk, prefix, f8 = shape
    if prefix is None:
        prefix = np.random.default_rng(4).integers(0, Lk - T + 1, size=B).tolist()
    case = make_step(sum(shape[:6]), B, T, H, H_kv, d, Lk, prefix, None, "tree", f8)
    out, lse = call_step(mha, on_gpu(case), f8, True)
    launch = mha.last_launch_info()
    assert launch["kernels"] == 1 and launch["grid"] > 152
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, f8, what=str(shape[:6]))


@pytest.mark.parametrize("kind", ["block", "short"])
def test_forms_repeat(mha, kind):  # noqa: F811
    """The same bits on every call, from two streams at once, and from a captured
    graph replayed after its inputs changed."""
    f8 = kind == "short"
    shape = (2, 1, 8, 4, 64, 100) if f8 else (2, 40, 8, 2, 128, 9000)
    cases = [on_gpu(make_step(50 + i, *shape, [90 - 50 * i, 33] if f8 else [8900 - 900 * i, 33], None,
                              None if f8 else "tree", f8, not f8)) for i in range(2)]
    first = [call_step(mha, g, f8, not f8) for g in cases]
    assert not f8 or mha.last_launch_info()["block"] == SHORT_THREADS
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [call_step(mha, g, f8, not f8, stream=s) for g, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for (a, la), (b, lb) in zip(got, first):
            assert torch.equal(a, b) and torch.equal(la, lb)
    graph = torch.cuda.CUDAGraph()
    g = {n: (t.clone() if torch.is_tensor(t) else t) for n, t in cases[0].items()}
    with torch.cuda.graph(graph):
        captured = call_step(mha, g, f8, not f8)
    for i in (1, 0):
        for n, t in cases[i].items():
            if torch.is_tensor(t):
                g[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured[0], first[i][0]) and torch.equal(captured[1], first[i][1])
    assert mha.mha_sync_status() == 0


def test_many_rows_agree_with_the_forward(mha):  # noqa: F811
    """Without a prefix and with a chain, a step of T rows is causal attention: the
    forward over the same tensors.  Each rounds its output once (2^-8), and the
    forward its weights (2^-8 of a mean of |v|)."""
    from transformer_head_scaled_sdpa_gb300 import inputs
    B, T, H, d = 2, 192, 4, 128
    q, k, v = (cu.random_rows(s, (B, T, H, d)).cuda() for s in (1, 2, 3))
    out, lse = mha.mha_decode_tree(q, k, v, i32([0, 0]).cuda(), return_lse=True)
    full, lse_f = mha.mha_fwd(q, k, v, mask_kind=inputs.MASK_CAUSAL, return_lse=True)
    assert mha.mha_sync_status() == 0
    bound = 2 ** -8 * (out.float().abs() + full.float().abs() + 1.01 * v.float().abs().max())
    assert ((out.float() - full.float()).abs() <= bound).all()
    pu.assert_lse_close(lse, lse_f.double().cpu().numpy().reshape(B, H, T), "forward")


@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "f8"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T", [2, 8, 9, 16, 17, 32, 33, 64])
def test_every_count_of_rows(mha, T, d, f8):  # noqa: F811
    """Row counts around the sizes of a unit, over a ragged last tile, an empty
    prefix and several tiles."""
    case = make_step(T + d, 3, T, 2, 2, d, 300, [300 - T, 0, 17], [T, T - 1, T], "tree", f8)
    out, lse = call_step(mha, on_gpu(case), f8, True)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, f8, what=f"{T} rows of {d}")
