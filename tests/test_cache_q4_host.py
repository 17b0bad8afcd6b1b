"""The 4-bit cache, the steps over it and the moves of cached rows on the host: the C
entries refuse bad arguments with the documented codes and the binding refuses bad
tensors, before any CUDA call (pointers below are never dereferenced); the plain forms
the GPU tests compare with are pinned here too."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from tests import cache_util as cu
from tests import q4_util as qu
from tests.test_cache_host import (ALIAS, BITS, COUNTS, K, KC, KS, LSE, MASK, NULL, O, OK, Q, SCALE, SHAPE, START,
                                   UNSUP, V, VC, VS, WORKSPACE, WS, lib)  # noqa: F401
from transformer_head_scaled_sdpa_gb300 import binding

PARENT, FIRST, LENS, PATH = 0x7_2000_0000, 0x7_3000_0000, 0x7_4000_0000, 0x7_5000_0000
BF16, F8, Q4 = 0, 1, 2


def write(lib, k=K, v=V, ts=0, ss=0, kc=KC, vc=VC, ks=KS, vs=VS, B=2, T=5, H=3, Lk=64, d=64,  # noqa: F811
          start=START, counts=None):
    return lib.mha_cache_write_q4(k, v, ts, ss, kc, vc, ks, vs, B, T, H, Lk, d, start, counts, None)


def test_write_refusals(lib):  # noqa: F811
    for name in ("B", "T", "H", "Lk", "ts", "ss"):
        assert write(lib, **{name: -1}) == SHAPE
    for d in (0, 8, 16, 48, 80, 100, 272, 288):
        assert write(lib, d=d) == UNSUP
    for name in ("k", "v", "kc", "vc", "ks", "vs", "start"):
        assert write(lib, **{name: None}) == NULL
    for name, p in (("k", K), ("v", V), ("kc", KC), ("vc", VC)):
        assert write(lib, **{name: p + 8}) == UNSUP
    for off in (1, 2, 3):
        assert write(lib, ks=KS + off) == UNSUP and write(lib, vs=VS + off) == UNSUP
        assert write(lib, start=START + off) == UNSUP and write(lib, counts=COUNTS + off) == UNSUP
    assert write(lib, ts=3 * 64 - 8) == SHAPE
    assert write(lib, ts=3 * 64 + 4) == UNSUP and write(lib, ss=3 * 64 + 4) == UNSUP
    assert write(lib, B=1 << 20, H=1 << 20) == SHAPE
    assert write(lib, B=1 << 15, H=1 << 12, Lk=1 << 20) == SHAPE
    assert write(lib, B=1, H=1, Lk=2 ** 31 - 1) == SHAPE
    assert write(lib, B=3, T=1, H=1, ss=1 << 50) == SHAPE
    # codes take 2 x 64 x 3 x 32 bytes, scales 2 x 3 x 64 x 4
    codes, scales = 2 * 64 * 3 * 32, 2 * 3 * 64 * 4
    assert write(lib, kc=K) == ALIAS and write(lib, vc=KC + codes - 16) == ALIAS
    assert write(lib, ks=KC) == ALIAS and write(lib, vs=KS + scales - 4) == ALIAS
    assert write(lib, kc=START - 16) == ALIAS and write(lib, vc=COUNTS - 16, counts=COUNTS) == ALIAS
    for name in ("B", "T", "H", "Lk"):
        assert write(lib, **{name: 0}) == OK
    assert write(lib, B=0, k=None, kc=None, start=None) == OK


def read(lib, kc=KC, vc=VC, ks=KS, vs=VS, k=K, v=V, B=2, H=3, Lk=64, d=64, lens=START):  # noqa: F811
    return lib.mha_cache_read_q4(kc, vc, ks, vs, k, v, B, H, Lk, d, lens, None)


def test_read_refusals(lib):  # noqa: F811
    for name in ("B", "H", "Lk"):
        assert read(lib, **{name: -1}) == SHAPE
        assert read(lib, **{name: 0}) == OK
    assert read(lib, d=48) == UNSUP
    for name in ("kc", "vc", "ks", "vs", "k", "v", "lens"):
        assert read(lib, **{name: None}) == NULL
    assert read(lib, k=K + 8) == UNSUP and read(lib, vc=VC + 4) == UNSUP
    assert read(lib, ks=KS + 2) == UNSUP and read(lib, lens=START + 1) == UNSUP
    assert read(lib, k=KC) == ALIAS and read(lib, v=KS) == ALIAS and read(lib, v=K + 16) == ALIAS
    values = 2 * 3 * 64 * 64 * 2
    assert read(lib, k=START - values + 16) == ALIAS and read(lib, v=K - values + 16) == ALIAS
    assert read(lib, B=1 << 16, H=1 << 16) == SHAPE


def step(lib, fn, q=Q, kc=KC, vc=VC, ks=KS, vs=VS, o=O, lse=None, B=2, T=4, H=6, H_kv=3, Lk=64,  # noqa: F811
         d=64, lens=START, drafts=None, bits=None, scale=0.0, ws=None, wsb=0):
    if fn == "mha_decode_q4":
        return lib.mha_decode_q4(q, kc, vc, ks, vs, o, lse, B, H, H_kv, Lk, d, lens, scale, ws, wsb, None)
    return lib.mha_decode_tree_q4(q, kc, vc, ks, vs, o, lse, B, T, H, H_kv, Lk, d, lens, drafts, bits, scale, ws,
                                  wsb, None)


@pytest.mark.parametrize("fn", ["mha_decode_q4", "mha_decode_tree_q4"])
def test_step_refusals(lib, fn):  # noqa: F811
    for name in ("B", "H", "Lk"):
        assert step(lib, fn, **{name: -1}) == SHAPE
    assert step(lib, fn, H=6, H_kv=4) == SHAPE and step(lib, fn, H_kv=0) == SHAPE
    assert step(lib, fn, B=1 << 20, H=1 << 12, H_kv=1) == SHAPE
    assert step(lib, fn, B=1, T=1, H=1, H_kv=1, Lk=2 ** 31 - 1) == SHAPE
    assert step(lib, fn, B=1, T=1, H=1 << 24, H_kv=1 << 24, Lk=1, d=256) == SHAPE   # a position of 2^31 bytes
    for d in (0, 8, 16, 48, 100, 264, 288):
        assert step(lib, fn, d=d) == UNSUP
    assert step(lib, fn, ks=None) == NULL and step(lib, fn, vs=None) == NULL
    assert step(lib, fn, ks=KS + 2) == UNSUP and step(lib, fn, vs=VS + 1) == UNSUP
    scales = 2 * 3 * 64 * 4
    assert step(lib, fn, o=KS + scales - 16) == ALIAS and step(lib, fn, lse=VS + scales - 4) == ALIAS
    if "tree" in fn:
        assert step(lib, fn, T=-1) == SHAPE and step(lib, fn, T=257) == UNSUP and step(lib, fn, T=0) == OK
        assert step(lib, fn, bits=BITS + 4) == UNSUP and step(lib, fn, drafts=COUNTS + 2) == UNSUP
        assert step(lib, fn, o=BITS, bits=BITS) == ALIAS and step(lib, fn, lse=COUNTS, drafts=COUNTS) == ALIAS
    for bad in (math.nan, math.inf, -1.0):
        assert step(lib, fn, scale=bad) == SCALE
    for name in ("q", "kc", "vc", "o"):
        assert step(lib, fn, **{name: None}) == NULL
    assert step(lib, fn, lens=None) == MASK
    for name, p in (("q", Q), ("kc", KC), ("vc", VC), ("o", O)):
        assert step(lib, fn, **{name: p + 8}) == UNSUP
    assert step(lib, fn, lse=LSE + 2) == UNSUP and step(lib, fn, lens=START + 2) == UNSUP
    assert step(lib, fn, o=Q) == ALIAS and step(lib, fn, o=KC + 64) == ALIAS
    assert step(lib, fn, lse=O) == ALIAS and step(lib, fn, o=START - 16) == ALIAS
    assert step(lib, fn, B=0) == OK and step(lib, fn, H=0, H_kv=0, q=None) == OK


def test_workspace_rules(lib):  # noqa: F811
    ws = lib.mha_decode_q4_workspace_bytes
    tree = lib.mha_decode_tree_q4_workspace_bytes
    assert ws(2, 32, 8, 65536, 48) == 0 and ws(2, 32, 5, 65536, 128) == 0
    assert ws(0, 32, 8, 65536, 128) == 0 and ws(-1, 32, 8, 65536, 128) == 0
    assert tree(2, 300, 32, 8, 65536, 128) == 0                    # T too large
    big = dict(B=1, T=4, H=8, H_kv=2, Lk=65536, d=128)
    for fn, need in (("mha_decode_q4", ws(1, 8, 2, 65536, 128)), ("mha_decode_tree_q4", tree(1, 4, 8, 2, 65536, 128))):
        assert need > 0
        assert step(lib, fn, **big) == WORKSPACE
        assert step(lib, fn, ws=WS, wsb=need - 1, **big) == WORKSPACE
        assert step(lib, fn, ws=WS + 8, wsb=need, **big) == WORKSPACE
        assert step(lib, fn, ws=O, wsb=need, **big) == ALIAS
        assert step(lib, fn, ws=VC, wsb=need, **big) == ALIAS
        assert step(lib, fn, ws=VS, wsb=need, **big) == ALIAS
        assert step(lib, fn, ws=LSE, wsb=need, lse=LSE, **big) == ALIAS


# ---- moves
def fork(lib, fmt=F8, kc=KC, vc=VC, ks=KS, vs=VS, B=2, H=3, Lk=64, d=64, parent=PARENT, first=None,  # noqa: F811
         lens=LENS):
    return lib.mha_cache_fork(kc, vc, ks, vs, fmt, B, H, Lk, d, parent, first, lens, None)


def compact(lib, fmt=F8, kc=KC, vc=VC, ks=KS, vs=VS, B=2, T=5, H=3, Lk=64, d=64, prefix=LENS, path=PATH,  # noqa: F811
            path_lens=None):
    return lib.mha_cache_compact(kc, vc, ks, vs, fmt, B, T, H, Lk, d, prefix, path, path_lens, None)


@pytest.mark.parametrize("call", [fork, compact])
def test_move_refusals(lib, call):  # noqa: F811
    for fmt in (-1, 3):
        assert call(lib, fmt=fmt) == UNSUP
    for name in ("B", "H", "Lk"):
        assert call(lib, **{name: -1}) == SHAPE
        assert call(lib, **{name: 0}) == OK
    for fmt, bad in ((BF16, (0, 4, 264)), (F8, (8, 24, 272)), (Q4, (16, 48, 288))):
        for d in bad:
            assert call(lib, fmt=fmt, d=d) == UNSUP
    assert call(lib, B=1 << 20, H=1 << 20) == SHAPE and call(lib, B=1, Lk=2 ** 31 - 1) == SHAPE
    for name in ("kc", "vc", "ks", "vs"):
        assert call(lib, **{name: None}) == NULL
    for name, p in (("kc", KC), ("vc", VC)):
        assert call(lib, **{name: p + 8}) == UNSUP
    for off in (1, 2, 3):
        assert call(lib, fmt=Q4, ks=KS + off) == UNSUP and call(lib, fmt=Q4, vs=VS + off) == UNSUP
    rows = 2 * 64 * 3
    for fmt, row, scale in ((BF16, 128, 0), (F8, 64, 1), (Q4, 32, 4)):
        end = rows * row - 16
        assert call(lib, fmt=fmt, vc=KC + end) == ALIAS and call(lib, fmt=fmt, kc=LENS - end) == ALIAS
        if scale:
            assert call(lib, fmt=fmt, ks=VC + rows * row - 4) == ALIAS
            assert call(lib, fmt=fmt, vs=KS + rows * scale - 4) == ALIAS
            assert call(lib, fmt=fmt, ks=LENS - rows * scale + 4) == ALIAS
    if call is fork:
        assert fork(lib, parent=None) == NULL and fork(lib, lens=None) == NULL
        for off in (1, 2, 3):
            assert fork(lib, parent=PARENT + off) == UNSUP and fork(lib, first=FIRST + off) == UNSUP
            assert fork(lib, lens=LENS + off) == UNSUP
        assert fork(lib, B=1025) == UNSUP
        assert fork(lib, kc=PARENT - 16) == ALIAS and fork(lib, vs=FIRST, first=FIRST) == ALIAS
    else:
        assert compact(lib, prefix=None) == NULL and compact(lib, path=None) == NULL
        for off in (1, 2, 3):
            assert compact(lib, path=PATH + off) == UNSUP and compact(lib, path_lens=COUNTS + off) == UNSUP
            assert compact(lib, prefix=LENS + off) == UNSUP
        assert compact(lib, T=-1) == SHAPE and compact(lib, T=257) == UNSUP and compact(lib, T=0) == OK
        assert compact(lib, kc=PATH + 2 * 5 * 4 - 8 & ~15) == ALIAS
        assert compact(lib, vs=COUNTS, path_lens=COUNTS) == ALIAS


# ---- the binding
def cache(B=2, Lk=8, H=2, d=32):
    return [torch.zeros((B, Lk, H, d // 2), dtype=torch.uint8) for _ in range(2)] + \
        [torch.zeros((B, H, Lk, 2), dtype=torch.bfloat16) for _ in range(2)]


def test_binding_refusals(lib):  # noqa: F811
    kc, vc, ks, vs = cache()
    lens = torch.zeros(2, dtype=torch.int32)
    k = torch.zeros((2, 3, 2, 32), dtype=torch.bfloat16)
    q = torch.zeros((2, 4, 32), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="cuda"):          # nothing runs on the CPU
        binding.mha_cache_write_q4(k, k.clone(), kc, vc, ks, vs, lens)
    with pytest.raises(ValueError, match="cuda"):
        binding.mha_cache_read_q4(kc, vc, ks, vs, lens)
    with pytest.raises(ValueError, match="cuda"):
        binding.mha_decode_q4(q, kc, vc, ks, vs, lens)
    with pytest.raises(ValueError, match="k_scale"):
        binding.mha_cache_read_q4(kc, vc, ks[..., 0], vs, lens)
    with pytest.raises(ValueError, match="d_k / 2"):
        binding.mha_cache_read_q4(kc, vc[:, :4], ks, vs, lens)
    with pytest.raises(ValueError, match="must be"):
        binding.mha_cache_write_q4(k[..., :16], k[..., :16], kc, vc, ks, vs, lens)
    with pytest.raises(TypeError, match="uint8"):
        binding.mha_cache_read_q4(kc.view(torch.int8), vc, ks, vs, lens)
    with pytest.raises(TypeError, match="bfloat16"):
        binding.mha_decode_q4(q.float(), kc, vc, ks, vs, lens)
    with pytest.raises(ValueError, match="match"):
        binding.mha_decode_q4(q[:, :3], kc, vc, ks, vs, lens)
    with pytest.raises(ValueError, match="tree_mask"):
        binding.mha_decode_tree_q4(q[:, None], kc, vc, ks, vs, lens, tree_mask=torch.zeros((2, 1), dtype=torch.int64))


def test_binding_refusals_of_moves(lib):  # noqa: F811
    kc, vc, ks, vs = cache()
    lens = torch.zeros(2, dtype=torch.int32)
    path = torch.zeros((2, 3), dtype=torch.int32)
    scales = {"k_scale": ks, "v_scale": vs}
    half = kc.to(torch.bfloat16)
    with pytest.raises(ValueError, match="cuda"):
        binding.mha_cache_fork(kc, vc, lens, lens, **scales)
    with pytest.raises(ValueError, match="cuda"):
        binding.mha_cache_compact(half, half, lens, path)
    with pytest.raises(TypeError, match="k_cache"):
        binding.mha_cache_fork(kc.float(), vc.float(), lens, lens)
    with pytest.raises(ValueError, match="needs k_scale"):
        binding.mha_cache_fork(kc, vc, lens, lens)
    with pytest.raises(ValueError, match="no scales"):
        binding.mha_cache_compact(half, half, lens, path, **scales)
    with pytest.raises(ValueError, match="alike"):
        binding.mha_cache_fork(half, half[:, :3], lens, lens)
    with pytest.raises(ValueError, match="path"):
        binding.mha_cache_compact(kc, vc, lens, path[:1], **scales)


# ---- the plain forms
def test_plain_quantise_by_fractions():
    """The plain form's step and codes against the definition in exact fractions."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((60, 32)) * np.exp2(rng.integers(-70, 80, size=(60, 1)).astype(float))
    x[0] = 0.0
    x[1] = -2.5
    x[2] = np.arange(32) % 31 / 2 - 3.5
    x[3] = 100 + rng.standard_normal(32)
    x[4] = np.abs(x[4])
    x = cu.f64(torch.from_numpy(x).to(torch.bfloat16))
    codes, pairs = qu.quantise(x)
    for row, c, (lo, step) in zip(x, codes, pairs):
        row = [Fraction(v) for v in row]
        need = max((max(row) - min(row)) / 15, max(abs(v) for v in row) / 8192, Fraction(1, 2 ** 60))
        up = torch.tensor(step, dtype=torch.float64).to(torch.bfloat16)
        assert float(up) == step and Fraction(step) >= need and lo == min(row)
        below = torch.tensor(up.view(torch.int16).item() - 1, dtype=torch.int16).view(torch.bfloat16)
        assert Fraction(float(below)) < need
        for v, code in zip(row, c):
            at = (v - Fraction(lo)) / Fraction(step)
            assert 0 <= code <= 15 and abs(at - int(code)) <= Fraction(1, 2)
            assert at - int(code) != Fraction(-1, 2)       # a tie takes the lower
    assert (codes[2, 1:30:2] == np.arange(15)).all()


def test_plain_pack():
    c = np.arange(16, dtype=np.uint8)[None, None, None]
    b = qu.packed(c)
    assert b[0, 0, 0, 0] == 0x10 and np.array_equal(qu.unpacked(b), c)
