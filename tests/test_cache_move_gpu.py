"""Rows of a cache moved in place (mha_cache_fork, mha_cache_compact) against plain
copies, bit for bit, in the three formats."""
import numpy as np
import pytest
import torch

from tests.test_cache_gpu import i32, mha  # noqa: F401

pytestmark = pytest.mark.gpu

FORMATS = ["bf16", "f8", "q4"]


def random_bytes(seed, fmt, B, Lk, H, d):
    """(k, v[, k scales, v scales]) of random bytes as the format's dtypes, CPU."""
    g = torch.Generator().manual_seed(seed)

    def rand(shape, dtype):
        return torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).view(dtype)

    if fmt == "bf16":
        return [rand((B, Lk, H, 2 * d), torch.bfloat16) for _ in range(2)]
    if fmt == "f8":
        return [rand((B, Lk, H, d), torch.float8_e4m3fn) for _ in range(2)] + \
            [rand((B, H, Lk), torch.uint8) for _ in range(2)]
    return [rand((B, Lk, H, d // 2), torch.uint8) for _ in range(2)] + \
        [rand((B, H, Lk, 4), torch.bfloat16) for _ in range(2)]


def raw(t):
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()


def by_position(t, i):
    """[B, Lk, H, bytes] of a cache's i-th tensor (scales lie by head)."""
    x = raw(t)
    if i < 2:
        return x
    return x.reshape(*x.shape[:3], -1).transpose(0, 2, 1, 3)


def scales_of(dev):
    return {"k_scale": dev[2], "v_scale": dev[3]} if len(dev) == 4 else {}


def check_fork(mha, cpu, dev, parent, first, lens):  # noqa: F811
    B, Lk = cpu[0].shape[:2]
    mha.mha_cache_fork(dev[0], dev[1], i32(parent).cuda(), i32(lens).cuda(),
                       first=None if first is None else i32(first).cuda(), **scales_of(dev))
    assert mha.mha_sync_status() == 0
    for i, (t, got) in enumerate(zip(cpu, dev)):
        old = by_position(t, i)
        want = old.copy()
        for b in range(B):
            f, e = max(0, 0 if first is None else first[b]), min(lens[b], Lk)
            if 0 <= parent[b] < B and f < e:
                want[b, f:e] = old[parent[b], f:e]
        assert np.array_equal(by_position(got, i), want)


FORKS = [
    # B, Lk, H, d, parent, first, lens
    (4, 40, 3, 64, [1, 0, 3, 2], None, [40, 40, 17, 17]),                # exchanges
    (4, 33, 8, 96, [1, 2, 3, 0], [5, 0, 31, 2], [33, 20, 33, 3]),        # a cycle, each its own range
    (3, 5, 1, 32, [0, 1, 2], None, [5, 5, 5]),                           # nothing moves
    (6, 70, 2, 128, [-1, 6, 0, 0, 0, 2 ** 31 - 1], [0, 0, -3, 69, 70, 0], [70, 70, 100, 70, 70, 70]),
    (1, 9, 2, 64, [0], None, [9]),
    (2, 300, 96, 128, [1, 1], [100, 0], [300, 300]),
    (2, 1, 1, 32, [1, 1], None, [1, 0]),
    (5, 1000, 2, 256, [4, 4, 4, 4, 0], [0, 1, 2, 3, 4], [-5, 0, 1000, 999, 5]),
    (130, 21, 3, 64, None, None, None),
    (1024, 3, 1, 32, None, None, None),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", FORKS, ids=lambda s: "x".join(map(str, s[:4])))
def test_fork(mha, shape, fmt):  # noqa: F811
    B, Lk, H, d, parent, first, lens = shape
    rng = np.random.default_rng(B)
    if parent is None:
        parent = rng.permutation(B).tolist() if B > 500 else rng.integers(-1, B + 1, size=B).tolist()
        first = rng.integers(0, Lk, size=B).tolist()
        lens = rng.integers(0, Lk + 1, size=B).tolist()
    cpu = random_bytes(1, fmt, B, Lk, H, d)
    check_fork(mha, cpu, [t.cuda() for t in cpu], parent, first, lens)


def check_compact(mha, cpu, dev, prefix, path, path_lens):  # noqa: F811
    B, Lk = cpu[0].shape[:2]
    T = len(path[0])
    mha.mha_cache_compact(dev[0], dev[1], i32(prefix).cuda(), torch.tensor(path, dtype=torch.int32).cuda(),
                          path_lens=None if path_lens is None else i32(path_lens).cuda(), **scales_of(dev))
    assert mha.mha_sync_status() == 0
    for i, (t, got) in enumerate(zip(cpu, dev)):
        old = by_position(t, i)
        want = old.copy()
        for b in range(B):
            n = int(np.clip(prefix[b], 0, Lk))
            for x in range(T if path_lens is None else int(np.clip(path_lens[b], 0, T))):
                if 0 <= path[b][x] < T and n + x < Lk and n + path[b][x] < Lk:
                    want[b, n + x] = old[b, n + path[b][x]]
        assert np.array_equal(by_position(got, i), want)


def ascending(rng, B, T, n):
    return [sorted(rng.choice(T, size=n, replace=False).tolist()) + [0] * (T - n) for _ in range(B)]


COMPACTS = [
    # B, Lk, H, d, T, prefix, path, path_lens
    (2, 40, 3, 64, 5, [3, 30], [[0, 2, 4, 9, 9], [1, 3, 4, 0, 0]], [3, 3]),
    (2, 40, 8, 96, 4, [0, 38], [[3, 2, 1, 0], [1, 0, 3, 2]], None),           # exchanges; past the capacity
    (1, 20, 2, 32, 6, [5], [[5, 5, 5, 0, 0, -1]], [6]),                        # one token in several places
    (3, 20, 1, 128, 3, [-4, 20, 25], [[2, 2, 2], [1, 1, 1], [1, 1, 1]], [100, 3, 3]),
    (2, 9, 2, 64, 3, [2, 2], [[2, 2 ** 31 - 1, -2 ** 31], [1, 2, 0]], [3, -1]),
    (1, 3, 1, 32, 1, [1], [[0]], None),                                        # nothing moves
    (4, 300, 96, 128, 63, [200, 0, 10, 290], None, 12),
    (2, 700, 5, 256, 256, [100, 444], None, 200),
    (40, 64, 8, 64, 12, None, None, 5),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", COMPACTS, ids=lambda s: "x".join(map(str, s[:5])))
def test_compact(mha, shape, fmt):  # noqa: F811
    B, Lk, H, d, T, prefix, path, path_lens = shape
    rng = np.random.default_rng(B + T)
    if prefix is None:
        prefix = rng.integers(0, Lk - T, size=B).tolist()
    if path is None:
        path, path_lens = ascending(rng, B, T, path_lens), [path_lens] * B
    cpu = random_bytes(2, fmt, B, Lk, H, d)
    check_compact(mha, cpu, [t.cuda() for t in cpu], prefix, path, path_lens)


def test_bf16_widths_that_are_multiples_of_8(mha):  # noqa: F811
    """Rows of 16 bytes and of an odd number of 16-byte pieces."""
    for d, H in ((8, 1), (24, 3), (200, 1)):
        cpu = random_bytes(3, "bf16", 3, 12, H, d)
        dev = [t.cuda() for t in cpu]
        check_fork(mha, cpu, dev, [2, 0, 1], [1, 0, 3], [12, 11, 12])
        cpu = [t.cpu() for t in dev]
        check_compact(mha, cpu, dev, [2, 9, 0], [[1, 2, 0], [2, 1, 0], [2, 2, 2]], None)


def test_far_offsets(mha):  # noqa: F811
    """Caches of more than 2^32 bytes: the moved rows lie past that."""
    B, H, d, Lk = 3, 8, 256, 1_500_000
    g = torch.Generator(device="cuda").manual_seed(1)
    dev = [torch.zeros((B, Lk, H, d // 2), dtype=torch.uint8, device="cuda") for _ in range(2)] + \
        [torch.zeros((B, H, Lk, 2), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    assert dev[0].numel() > 2 ** 32
    for t in dev[:2]:
        t[1:, -20:] = torch.randint(0, 256, (2, 20, H, d // 2), generator=g, device="cuda", dtype=torch.uint8)
    for t in dev[2:]:
        t[1:, :, -20:] = torch.randn((2, H, 20, 2), generator=g, device="cuda").to(torch.bfloat16)
    tails = [t[:, -20:].clone() if i < 2 else t[:, :, -20:].clone() for i, t in enumerate(dev)]
    mha.mha_cache_fork(dev[0], dev[1], i32([0, 2, 1]).cuda(), i32([Lk] * 3).cuda(),
                       first=i32([0, Lk - 18, Lk - 18]).cuda(), k_scale=dev[2], v_scale=dev[3])
    mha.mha_cache_compact(dev[0], dev[1], i32([0, Lk - 10, Lk - 10]).cuda(), i32([1, 0] * 3).reshape(3, 2).cuda(),
                          path_lens=i32([0, 2, 1]).cuda(), k_scale=dev[2], v_scale=dev[3])
    assert mha.mha_sync_status() == 0
    for i, (t, old) in enumerate(zip(dev, tails)):
        new = t[:, -20:] if i < 2 else t[:, :, -20:].transpose(1, 2)
        old = old if i < 2 else old.transpose(1, 2)
        want = old.clone()
        want[1, 2:], want[2, 2:] = old[2, 2:], old[1, 2:]
        want[1, 10], want[1, 11] = old[2, 11], old[2, 10]      # exchanged after the fork
        want[2, 10] = old[1, 11]
        assert torch.equal(new, want)
        assert torch.count_nonzero(t[0]) == 0


def test_streams_and_graphs(mha):  # noqa: F811
    """On another stream, and captured: a replay moves what the arrays then say."""
    cpu = random_bytes(4, "f8", 3, 50, 4, 64)
    parent, lens, first = i32([1, 2, 0]).cuda(), i32([50, 40, 50]).cuda(), i32([0, 3, 9]).cuda()
    path, prefix = i32([2, 3, 1, 0, 0, 0, 1, 1, 1]).reshape(3, 3).cuda(), i32([5, 44, 0]).cuda()

    def call(dev, **kw):
        mha.mha_cache_fork(dev[0], dev[1], parent, lens, first=first, **scales_of(dev), **kw)
        mha.mha_cache_compact(dev[0], dev[1], prefix, path, **scales_of(dev), **kw)

    want = [t.cuda() for t in cpu]
    call(want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = [t.cuda() for t in cpu]
        torch.cuda.synchronize()
        call(got, stream=stream)
        torch.cuda.synchronize()
        assert all(np.array_equal(raw(a), raw(b)) for a, b in zip(got, want))
    dev = [t.cuda() for t in cpu]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(dev)
    parent.copy_(i32([2, 0, 1]))
    path.copy_(i32([1, 1, 2, 2, 1, 0, 0, 0, 0]).reshape(3, 3))
    for t, c in zip(dev, cpu):
        t.view(torch.uint8).copy_(c.view(torch.uint8))
    graph.replay()
    again = [t.cuda() for t in cpu]
    call(again)
    assert mha.mha_sync_status() == 0
    assert all(np.array_equal(raw(a), raw(b)) for a, b in zip(dev, again))
    assert not np.array_equal(raw(dev[0]), raw(want[0]))
