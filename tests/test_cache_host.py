"""The 8-bit cache and the steps over a cache on the host: the C entries refuse
bad arguments with the documented codes and the binding refuses bad tensors,
before any CUDA call (pointers below are never dereferenced); the plain forms
the GPU tests compare with are pinned here too."""
import math

import numpy as np
import pytest
import torch

from tests import cache_util as cu
from transformer_head_scaled_sdpa_gb300 import binding, build

OK, NULL, SHAPE, UNSUP, MASK, SCALE, LAUNCH, TIMEOUT, ALIAS, WORKSPACE = range(10)

K, V, KC, VC = 0x1_0000_0000, 0x2_0000_0000, 0x3_0000_0000, 0x4_0000_0000
KS, VS, START, COUNTS = 0x5_0000_0000, 0x6_0000_0000, 0x7_0000_0000, 0x7_1000_0000
Q, O, LSE, WS, BITS = 0x8_0000_0000, 0x9_0000_0000, 0xA_0000_0000, 0xB_0000_0000, 0xC_0000_0000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def write(lib, k=K, v=V, ts=0, ss=0, kc=KC, vc=VC, ks=KS, vs=VS, B=2, T=5, H=3, Lk=64, d=64,
          start=START, counts=None):
    return lib.mha_cache_write_f8(k, v, ts, ss, kc, vc, ks, vs, B, T, H, Lk, d, start, counts, None)


def test_write_refusals(lib):
    for name in ("B", "T", "H", "Lk", "ts", "ss"):
        assert write(lib, **{name: -1}) == SHAPE
    for d in (0, 8, 24, 100, 272):
        assert write(lib, d=d) == UNSUP
    for name in ("k", "v", "kc", "vc", "ks", "vs", "start"):
        assert write(lib, **{name: None}) == NULL
    for name, p in (("k", K), ("v", V), ("kc", KC), ("vc", VC)):
        assert write(lib, **{name: p + 8}) == UNSUP
    assert write(lib, ts=3 * 64 - 8) == SHAPE            # a token's rows overlap the next one's
    assert write(lib, ts=3 * 64 + 4) == UNSUP            # rows not 16-byte aligned
    assert write(lib, ss=3 * 64 + 4) == UNSUP
    assert write(lib, B=1 << 20, H=1 << 20) == SHAPE
    assert write(lib, B=1 << 15, H=1 << 12, Lk=1 << 20) == SHAPE
    assert write(lib, kc=K) == ALIAS and write(lib, vc=KC + 64) == ALIAS
    assert write(lib, ks=KC) == ALIAS and write(lib, vs=KS + 16) == ALIAS
    assert write(lib, kc=START - 16) == ALIAS and write(lib, vc=COUNTS - 16, counts=COUNTS) == ALIAS
    # the last row of strided input: (B - 1) ss + (T - 1) ts + H d elements
    span = (1 * 4096 + 4 * 576 + 192) * 2
    assert write(lib, ts=576, ss=4096, kc=K + span - 16) == ALIAS
    for name in ("B", "T", "H", "Lk"):
        assert write(lib, **{name: 0}) == OK
    assert write(lib, B=0, k=None, kc=None, start=None) == OK


def read(lib, kc=KC, vc=VC, ks=KS, vs=VS, k=K, v=V, B=2, H=3, Lk=64, d=64, lens=START):
    return lib.mha_cache_read_f8(kc, vc, ks, vs, k, v, B, H, Lk, d, lens, None)


def test_read_refusals(lib):
    for name in ("B", "H", "Lk"):
        assert read(lib, **{name: -1}) == SHAPE
        assert read(lib, **{name: 0}) == OK
    assert read(lib, d=40) == UNSUP
    for name in ("kc", "vc", "ks", "vs", "k", "v", "lens"):
        assert read(lib, **{name: None}) == NULL
    assert read(lib, k=K + 8) == UNSUP and read(lib, vc=VC + 4) == UNSUP
    assert read(lib, k=KC) == ALIAS and read(lib, v=KS) == ALIAS and read(lib, v=K + 16) == ALIAS
    assert read(lib, v=START - 32) == ALIAS
    assert read(lib, B=1 << 16, H=1 << 16) == SHAPE


def step(lib, fn, q=Q, kc=KC, vc=VC, ks=KS, vs=VS, o=O, lse=None, B=2, T=4, H=6, H_kv=3, Lk=64,
         d=64, lens=START, drafts=None, bits=None, scale=0.0, ws=None, wsb=0):
    if fn == "mha_decode_f8":
        return lib.mha_decode_f8(q, kc, vc, ks, vs, o, lse, B, H, H_kv, Lk, d, lens, scale, ws, wsb,
                                 None)
    scales = (ks, vs) if fn.endswith("f8") else ()
    return getattr(lib, fn)(q, kc, vc, *scales, o, lse, B, T, H, H_kv, Lk, d, lens, drafts, bits,
                            scale, ws, wsb, None)


STEPS = ["mha_decode_f8", "mha_decode_tree", "mha_decode_tree_f8"]


@pytest.mark.parametrize("fn", STEPS)
def test_step_refusals(lib, fn):
    f8 = fn.endswith("f8")
    tree = "tree" in fn
    for name in ("B", "H", "Lk"):
        assert step(lib, fn, **{name: -1}) == SHAPE
    assert step(lib, fn, H=6, H_kv=4) == SHAPE and step(lib, fn, H_kv=0) == SHAPE
    assert step(lib, fn, H_kv=-3) == SHAPE
    assert step(lib, fn, B=1 << 20, H=1 << 12, H_kv=1) == SHAPE
    for d in (0, 4, 100, 264):
        assert step(lib, fn, d=d) == UNSUP
    if f8:
        assert step(lib, fn, d=24) == UNSUP
        assert step(lib, fn, ks=None) == NULL and step(lib, fn, vs=None) == NULL
        assert step(lib, fn, o=KS) == ALIAS
    if tree:
        assert step(lib, fn, T=-1) == SHAPE
        assert step(lib, fn, T=257) == UNSUP
        assert step(lib, fn, T=0) == OK
        assert step(lib, fn, bits=BITS + 4) == UNSUP and step(lib, fn, drafts=COUNTS + 2) == UNSUP
        assert step(lib, fn, o=BITS, bits=BITS) == ALIAS
        assert step(lib, fn, lse=COUNTS, drafts=COUNTS) == ALIAS
    for bad in (math.nan, math.inf, -1.0):
        assert step(lib, fn, scale=bad) == SCALE
    for name in ("q", "kc", "vc", "o"):
        assert step(lib, fn, **{name: None}) == NULL
    assert step(lib, fn, lens=None) == MASK
    for name, p in (("q", Q), ("kc", KC), ("vc", VC), ("o", O)):
        assert step(lib, fn, **{name: p + 8}) == UNSUP
    assert step(lib, fn, lse=LSE + 2) == UNSUP and step(lib, fn, lens=START + 2) == UNSUP
    assert step(lib, fn, o=Q) == ALIAS and step(lib, fn, o=KC + 64) == ALIAS
    assert step(lib, fn, lse=O) == ALIAS and step(lib, fn, lse=VC) == ALIAS
    assert step(lib, fn, o=START - 16) == ALIAS
    assert step(lib, fn, B=0) == OK and step(lib, fn, H=0, H_kv=0, q=None) == OK


def test_more_positions_than_an_int_counts(lib):
    """A capacity whose last tile would not fit an int is refused, not wrapped."""
    far = 2 ** 31 - 1
    assert write(lib, B=1, H=1, Lk=far, d=16) == SHAPE
    assert write(lib, B=1, H=1, T=far, d=16) == SHAPE
    assert write(lib, B=1, H=1, T=1 << 30, ts=1 << 40, d=16) == SHAPE
    assert read(lib, B=1, H=1, Lk=far, d=16) == SHAPE
    for fn in ("mha_decode_f8", "mha_decode_tree", "mha_decode_tree_f8"):
        assert step(lib, fn, B=1, T=1, H=1, H_kv=1, Lk=far, d=16) == SHAPE
    assert lib.mha_decode_f8_workspace_bytes(1, 1, 1, far, 16) == 0


def test_workspace_rules(lib):
    ws = lib.mha_decode_f8_workspace_bytes
    assert ws(2, 32, 8, 65536, 24) == 0 and ws(2, 32, 5, 65536, 128) == 0
    assert ws(0, 32, 8, 65536, 128) == 0 and ws(-1, 32, 8, 65536, 128) == 0
    assert lib.mha_decode_tree_workspace_bytes(2, 300, 32, 8, 65536, 128) == 0   # T too large
    for fn, need in (("mha_decode_f8", ws(1, 8, 2, 65536, 128)),
                     ("mha_decode_tree", lib.mha_decode_tree_workspace_bytes(1, 4, 8, 2, 65536, 128)),
                     ("mha_decode_tree_f8",
                      lib.mha_decode_tree_f8_workspace_bytes(1, 4, 8, 2, 65536, 128))):
        if need == 0:
            continue
        big = dict(B=1, T=4, H=8, H_kv=2, Lk=65536, d=128)
        assert step(lib, fn, **big) == WORKSPACE
        assert step(lib, fn, ws=WS, wsb=need - 1, **big) == WORKSPACE
        assert step(lib, fn, ws=WS + 8, wsb=need, **big) == WORKSPACE
        assert step(lib, fn, ws=O, wsb=need, **big) == ALIAS
        assert step(lib, fn, ws=VC, wsb=need, **big) == ALIAS
        assert step(lib, fn, ws=LSE, wsb=need, lse=LSE, **big) == ALIAS


def cache(B=2, Lk=8, H=2, d=16):
    return (torch.zeros((B, Lk, H, d), dtype=torch.uint8).view(torch.float8_e4m3fn),
            torch.zeros((B, Lk, H, d), dtype=torch.uint8).view(torch.float8_e4m3fn),
            torch.zeros((B, H, Lk), dtype=torch.uint8), torch.zeros((B, H, Lk), dtype=torch.uint8))


def test_binding_refusals(lib):
    kc, vc, ks, vs = cache()
    lens = torch.zeros(2, dtype=torch.int32)
    k = torch.zeros((2, 3, 2, 16), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="cuda"):          # nothing runs on the CPU
        binding.mha_cache_write_f8(k, k.clone(), kc, vc, ks, vs, lens)
    with pytest.raises(ValueError, match="cuda"):
        binding.mha_cache_read_f8(kc, vc, ks, vs, lens)
    with pytest.raises(ValueError, match="k_scale"):
        binding.mha_cache_write_f8(k, k, kc, vc, ks.transpose(1, 2), vs, lens)
    with pytest.raises(ValueError, match="must be"):
        binding.mha_cache_write_f8(k[:1], k[:1], kc, vc, ks, vs, lens)
    with pytest.raises(ValueError, match="overlap"):
        binding.mha_cache_write_f8(k[:, :1].expand(2, 3, 2, 16), k, kc, vc, ks, vs, lens)
    with pytest.raises(ValueError, match="contiguous"):
        binding.mha_cache_write_f8(torch.zeros((2, 3, 16, 2), dtype=torch.bfloat16).transpose(2, 3),
                                   k, kc, vc, ks, vs, lens)
    with pytest.raises(ValueError, match="strides"):
        binding.mha_cache_write_f8(torch.zeros((2, 3, 3, 2, 16), dtype=torch.bfloat16)[:, :, 1], k,
                                   kc, vc, ks, vs, lens)
    with pytest.raises(ValueError, match="start"):
        binding.mha_cache_write_f8(k, k, kc, vc, ks, vs, lens[:1])
    q = torch.zeros((2, 4, 16), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="float8"):
        binding.mha_cache_read_f8(kc.view(torch.uint8), vc, ks, vs, lens)
    with pytest.raises(TypeError, match="bfloat16"):
        binding.mha_decode_f8(q.float(), kc, vc, ks, vs, lens)
    with pytest.raises(ValueError, match="cuda"):
        binding.mha_decode_f8(q, kc, vc, ks, vs, lens)
    with pytest.raises(ValueError, match="match"):
        binding.mha_decode_f8(torch.zeros((2, 3, 16), dtype=torch.bfloat16), kc, vc, ks, vs, lens)
    with pytest.raises(ValueError, match="q must be"):
        binding.mha_decode_f8(torch.zeros((2, 2, 4, 16), dtype=torch.bfloat16), kc, vc, ks, vs, lens)
    with pytest.raises(ValueError, match="tree_mask"):
        binding.mha_decode_tree(torch.zeros((2, 3, 4, 16), dtype=torch.bfloat16),
                                kc.to(torch.bfloat16), vc.to(torch.bfloat16), lens,
                                tree_mask=torch.zeros((2, 3), dtype=torch.int64))


def test_row_strides_of_packed_projection():
    qkv = torch.zeros((2, 5, 3, 4, 16), dtype=torch.bfloat16)
    assert binding._row_strides(qkv[:, :, 1], "k") == (192, 960)
    assert binding._row_strides(qkv[:, :3, 2], "k") == (192, 960)
    assert binding._row_strides(qkv[:1, :1, 1], "k") == (64, 64)
    assert binding._row_strides(qkv[:, :0, 1], "k") == (0, 0)


# ---- the plain forms
def test_plain_quantise_against_torch():
    """The plain form's codes, from the format's definition, against torch's
    own float8 conversion of the scaled values."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((500, 32)) * np.exp2(rng.integers(-90, 100, size=(500, 1)).astype(float))
    x[0] = 0.0
    x[1] = 448.0 * 2.0 ** 5
    x[2, 0] = 448.5 * 2.0 ** 5
    x = torch.from_numpy(x).to(torch.bfloat16)
    codes, scales = cu.quantise(cu.f64(x))
    e = scales.astype(np.int64) - 127
    top = np.abs(cu.f64(x)).max(-1)
    assert (top <= 448.0 * np.exp2(e.astype(float))).all()
    assert ((top > 448.0 * np.exp2(e - 1.0)) | (e == -64)).all()
    y = torch.from_numpy(cu.f64(x) / np.exp2(e.astype(float))[:, None]).float()
    want = y.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes, want)
    assert scales[0] == 63 and scales[1] == 127 + 5 and scales[2] == 127 + (5 if float(x[2, 0]) <= 448 * 32 else 6)


def test_plain_attention_against_torch():
    q, k, v = (torch.randn(s, dtype=torch.float64) for s in ((2, 3, 4, 8), (2, 11, 2, 8), (2, 11, 2, 8)))
    bits = cu.tree_bits(np.random.default_rng(1), 2, 3)
    prefix, drafts = np.array([6, 8]), np.array([3, 2])
    out, lse, _ = cu.attention(q.numpy(), k.numpy(), v.numpy(),
                               lambda b: cu.visible(b, 3, 11, prefix, drafts, bits.numpy()))
    for b in range(2):
        sees = torch.from_numpy(cu.visible(b, 3, 11, prefix, drafts, bits.numpy()))
        live = int(drafts[b])
        ref = torch.nn.functional.scaled_dot_product_attention(
            q[b, :live].transpose(0, 1), k[b].transpose(0, 1).repeat_interleave(2, 0),
            v[b].transpose(0, 1).repeat_interleave(2, 0), attn_mask=sees[:live])
        assert np.allclose(out[b, :live], ref.transpose(0, 1).numpy(), atol=1e-12)
        assert (out[b, live:] == 0).all() and np.isneginf(lse[b, :, live:]).all()
