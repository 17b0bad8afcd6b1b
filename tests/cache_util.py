"""Plain float64 forms of the 8-bit cache and of the steps of a few rows over
a cache, for their tests.

Tolerances, from the formats' half steps (bf16 2^-8 relative, the weights'
pieces 2^-11 over an 8-bit cache and 2^-16 over a bf16 one) and float32 sums:
  out  |o - ref| <= 2^-8 |ref| + w * sum_j a_j |v_j| + 2^-8 * tiny, where
       w bounds the weights' relative error: the pieces' (2^-11 after an fp16
       rounding of 2^-11, or 2^-16), and the scores' absolute error ds, which
       moves every weight by a factor e^(2 ds).  ds <= (d + 2) 2^-24 sum|q k|
       scale in float32 sums, and over an 8-bit cache q's pieces leave 2^-22
       of the row's largest |q| on each of d terms; both stay below 2^-13 at
       the tests' |q k| sums.  So w = 2^-10 + 2^-12 (8-bit) or 2^-12 (bf16),
       and the float32 sum of n weights and products adds n 2^-24 at worst.
  lse  5e-4 + 1e-6 |lse| as for the other entries (parity_util).
"""
import numpy as np
import torch

E4M3_MAX = 448.0


def e4m3_values():
    """The 256 codes' values, by the format's definition (NaN at 0x7f, 0xff)."""
    v = np.empty(256)
    for c in range(256):
        sign = -1.0 if c & 0x80 else 1.0
        e, m = (c >> 3) & 15, c & 7
        v[c] = sign * (m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        if c & 0x7F == 0x7F:
            v[c] = np.nan
    return v


VALUES = e4m3_values()


def quantise(x):
    """Codes (uint8) and exponents (biased, uint8) of float64 rows [..., d] of
    finite values."""
    x = np.asarray(x, dtype=np.float64)
    top = np.abs(x).max(-1)
    m, ex = np.frexp(top / E4M3_MAX)            # top / 448 = m 2^ex, 1/2 <= m < 1
    e = np.where(m == 0.5, ex - 1, ex)          # the smallest e with top <= 448 * 2^e
    e = np.where(top == 0, -64, np.maximum(e, -64))
    y = x / np.exp2(e.astype(np.float64))[..., None]
    a = np.abs(y)
    _, ye = np.frexp(np.maximum(a, 2.0 ** -6))
    step = np.exp2(ye - 1 - 3.0)
    r = np.round(a / step) * step               # half to even
    r = np.minimum(r, E4M3_MAX)
    table = VALUES[:0x7F]
    codes = np.searchsorted(table, r)
    assert np.array_equal(table[codes], r)
    codes = codes | np.where(np.signbit(y), 0x80, 0)
    return codes.astype(np.uint8), (e + 127).astype(np.uint8)


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def codes_of(t):
    return t.detach().cpu().view(torch.uint8).numpy()


def cache_values(codes, scales):
    """float64 rows [B, L, H, d] of uint8 codes [B, L, H, d] and exponents
    [B, H, L]."""
    e = scales.astype(np.float64).transpose(0, 2, 1) - 127
    return VALUES[codes] * np.exp2(e)[..., None]


def visible(b, T, Lk, prefix, drafts, mask, with_drafts=True):
    """[T, Lk] truth values for sequence b."""
    n = int(np.clip(prefix[b], 0, Lk))
    live = T if drafts is None else int(np.clip(drafts[b], 0, T))
    sees = np.zeros((T, Lk), dtype=bool)
    for t in range(live):
        sees[t, :n] = True
        if not with_drafts:
            continue
        for j in range(live):
            if n + j >= Lk:
                break
            if mask is None:
                on = j <= t
            else:
                on = (int(mask[b, t, j // 64]) >> (j % 64)) & 1
            sees[t, n + j] = bool(on)
    return sees


def attention(q, k, v, sees_of, scale=None):
    """q [B, T, H, d], k, v [B, Lk, H_kv, d] float64 -> out, lse [B, H, T], and
    sum_j a_j |v_j| (the size the weights' errors are relative to)."""
    B, T, H, d = q.shape
    H_kv = k.shape[2]
    G = H // H_kv
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    out = np.zeros((B, T, H, d))
    size = np.zeros((B, T, H, d))
    lse = np.full((B, H, T), -np.inf)
    for b in range(B):
        sees = sees_of(b)
        cols = np.nonzero(sees.any(0))[0]
        if cols.size == 0:
            continue
        s_b = sees[:, cols]
        for h in range(H):
            kk, vv = k[b, cols, h // G], v[b, cols, h // G]
            s = np.where(s_b, (q[b, :, h] @ kk.T) * scale, -np.inf)
            m = s.max(-1)
            ok = np.isfinite(m)
            p = np.exp(s[ok] - m[ok, None])
            total = p.sum(-1)
            a = p / total[:, None]
            out[b, ok, h] = a @ vv
            size[b, ok, h] = a @ np.abs(vv)
            lse[b, h, ok] = m[ok] + np.log(total)
    return out, lse, size


def assert_out_close(got, ref, size, keys, f8, what=""):
    got = f64(got).reshape(ref.shape)
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    w = (2.0 ** -10 + 2.0 ** -12 if f8 else 2.0 ** -12) + keys * 2.0 ** -24
    excess = np.abs(got - ref) - (2.0 ** -8 * np.abs(ref) + 1.01 * w * size)
    assert excess.max(initial=-1.0) <= 0, \
        f"{what}: off by {excess.max():.3e} more than the roundings allow"


def tree_bits(rng, B, T, branch=0.2, back=6):
    """Ancestor bits int64 [B, T, ceil(T / 64)] of random trees (rng: numpy)."""
    words = (T + 63) // 64
    out = np.zeros((B, T, words), dtype=np.uint64)
    for b in range(B):
        for t in range(T):
            if t and rng.random() >= branch:
                out[b, t] = out[b, rng.integers(max(0, t - back), t)]
            out[b, t, t // 64] |= np.uint64(1) << np.uint64(t % 64)
    return torch.from_numpy(out.view(np.int64))


def random_rows(seed, shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def f8_cache(x, garbage_from=None):
    """(codes float8_e4m3fn, scales uint8) of bf16 rows [B, L, H, d]; positions
    from garbage_from[b] on are set to NaN codes with the largest scale byte."""
    codes, scales = quantise(f64(x))
    scales = np.ascontiguousarray(scales.transpose(0, 2, 1))
    if garbage_from is not None:
        for b, n in enumerate(garbage_from):
            codes[b, max(0, n):] = 0x7F
            scales[b, :, max(0, n):] = 255
    return torch.from_numpy(codes).view(torch.float8_e4m3fn), torch.from_numpy(scales)
