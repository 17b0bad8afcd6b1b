"""Steps over the 4-bit cache with many query rows per key head (a kernel of their own)
against their plain float64 forms (q4_util)."""
import numpy as np
import pytest
import torch

from tests import cache_util as cu
from tests import q4_util as qu
from tests.test_cache_gpu import mha, on_gpu  # noqa: F401
from tests.test_cache_q4_gpu import call_step, check_step, make_step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [32, 64, 96, 128, 192, 256])
@pytest.mark.parametrize("T,G", [(16, 1), (17, 1), (32, 1), (33, 1), (11, 4), (64, 1), (65, 1), (43, 3), (256, 1)])
def test_blocks_of_rows(mha, d, T, G):  # noqa: F811
    """A block of rows full, one row over it, one short of it; prefixes that end with a
    tile, inside one, and of nothing."""
    case = make_step(d + T + G, 3, T, 2 * G, 2, d, 700, [384, 129, 0], [T, max(0, T - 5), T], "tree")
    out, lse = call_step(mha, on_gpu(case), True)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, what=f"d {d}, {T} x {G} rows")


@pytest.mark.parametrize("d,H", [(64, 40), (128, 24), (128, 48), (256, 20), (256, 70)])
@pytest.mark.parametrize("lens", [[1], [0, 128], [5000, 127, 129], [300] * 40], ids=["1", "0-128", "5000", "40x300"])
def test_shared_heads(mha, d, H, lens):  # noqa: F811
    """A decode step with so many query heads on one key head: no key, one, splits, more
    sequences than a warp has lanes."""
    case = make_step(d + H, len(lens), 1, H, 1, d, max(lens) + 3, lens, None, None, with_drafts=False)
    out, lse = call_step(mha, on_gpu(case), False)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, with_drafts=False, what=f"d {d}, {H} heads")


@pytest.mark.parametrize("d", [64, 128, 256])
def test_moving_references(mha, d):  # noqa: F811
    """Scores that rise from tile to tile, for some rows steeply, for others not at all, and
    fall for the rest."""
    T, Lk = 50, 1500
    case = make_step(18, 1, T, 1, 1, d, Lk, [1400], None, None)
    k = torch.zeros((1, Lk, 1, d), dtype=torch.bfloat16)
    k[0, :, 0, 0] = torch.linspace(-30.0, 30.0, Lk).to(torch.bfloat16)
    case["q"][:] = 0.0
    case["q"][0, :, 0, 0] = torch.linspace(-16.0, 16.0, T).to(torch.bfloat16)
    case["kc"], case["ks"] = qu.q4_cache(k)
    out, lse = call_step(mha, on_gpu(case), True)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_values_far_apart(mha, d):  # noqa: F811
    B, H, Lk = 2, 40, 600
    rng = np.random.default_rng(6)
    case = make_step(19, B, 1, H, 1, d, Lk, [600, 130], None, None, with_drafts=False)
    for n in ("k", "v"):
        x = cu.random_rows(20, (B, Lk, 1, d)).float()
        x *= torch.from_numpy(np.exp2(rng.integers(-40 if n == "v" else -6, 1, size=(B, Lk, 1, 1)))).float()
        x[:, ::7] = 0.0
        x[:, 1::7] = 1.5
        case[n + "c"], case[n + "s"] = qu.q4_cache(x.to(torch.bfloat16))
    out, lse = call_step(mha, on_gpu(case), False)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse, with_drafts=False)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("spread", [0, 7, 9, 60])
def test_queries_far_apart(mha, d, spread):  # noqa: F811
    """Rows of one block that differ by powers of two, and rows of zeros."""
    T = 40
    case = make_step(23, 1, T, 1, 1, d, 500, [450], None, "tree")
    by = torch.exp2(-torch.arange(T, dtype=torch.float32) * spread / (T - 1)) * 2
    case["q"] = (case["q"].float() * by[None, :, None, None]).to(torch.bfloat16)
    case["q"][0, 3] = case["q"][0, 39] = 0.0
    out, lse = call_step(mha, on_gpu(case), True)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_queries_of_zeros(mha, d):  # noqa: F811
    case = make_step(24, 1, 36, 1, 1, d, 300, [200], None, None)
    case["q"][:] = 0.0
    out, lse = call_step(mha, on_gpu(case), True)
    assert mha.mha_sync_status() == 0
    check_step(case, out, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("inf"), float("nan"), 2.0 ** 120])
def test_a_bad_query_keeps_to_its_row(mha, d, bad):  # noqa: F811
    T, rows = 40, [0, 17, 35]
    case = make_step(25, 1, T, 1, 1, d, 500, [450], None, None)
    case["q"][0, rows] = 0.0
    out0, lse0 = call_step(mha, on_gpu(case), True)
    spoilt = dict(case, q=case["q"].clone())
    spoilt["q"][0, rows, 0, 5] = bad
    out, lse = call_step(mha, on_gpu(spoilt), True)
    assert mha.mha_sync_status() == 0
    if not np.isfinite(bad):
        assert torch.isnan(out[0, rows]).all()
    out[0, rows] = out0[0, rows]
    lse[..., rows] = lse0[..., rows]
    check_step(case, out, lse)


def test_two_streams_and_a_graph(mha):  # noqa: F811
    """Two steps at once on streams of their own, and one captured and replayed over new
    queries, give what they give alone, bit for bit."""
    a = on_gpu(make_step(26, 3, 20, 12, 3, 128, 3000, [2900, 1000, 64], None, "tree"))
    b = on_gpu(make_step(27, 2, 33, 4, 2, 256, 2000, [1900, 700], None, None))
    want = [call_step(mha, g, True) for g in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s, g in zip(streams, (a, b)):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(call_step(mha, g, True))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    other = a["q"].flip(0).contiguous()
    a2 = dict(a, q=other)
    want2 = call_step(mha, a2, True)
    held = dict(a, q=a["q"].clone())
    with torch.cuda.stream(streams[0]):
        call_step(mha, held, True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = call_step(mha, held, True)
    for q, (o, s) in ((a["q"], want[0]), (other, want2), (a["q"], want[0])):
        held["q"].copy_(q)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(lse, s)
    assert mha.mha_sync_status() == 0


@pytest.mark.parametrize("T,H", [(1, 1), (1, 2), (5, 1), (16, 1), (40, 1)])
@pytest.mark.parametrize("Lk", [1, 200, 9000], ids=["a key", "a split", "splits"])
def test_what_is_not_a_number_shows(mha, T, H, Lk):  # noqa: F811
    """A row whose every score is NaN, for its query's sake or its keys', is no empty row."""
    case = make_step(28, 1, T, H, 1, 128, Lk + T, [Lk], None, None)
    bad = dict(case, q=case["q"].clone())
    bad["q"][0, T - 1, 0, 7] = float("nan")
    out, lse = call_step(mha, on_gpu(bad), True)
    assert torch.isnan(out[0, T - 1, 0]).all() and torch.isnan(lse[0, 0, T - 1])
    assert torch.isfinite(out[0, : T - 1]).all() and torch.isfinite(out[0, :, 1:]).all()
    bad = dict(case, ks=case["ks"].clone())
    bad["ks"][..., 0] = float("nan")
    out, lse = call_step(mha, on_gpu(bad), True)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    assert mha.mha_sync_status() == 0
