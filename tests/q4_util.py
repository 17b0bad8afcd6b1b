"""Plain float64 forms of the 4-bit cache and of moved rows, for their tests.

Tolerances of the steps over a 4-bit cache, from the formats' half steps (bf16
2^-8 relative, fp16 2^-11) and float32 sums on the tensor cores, whose additions
may cut: 2^-23 of what is summed so far, once per block of 16 products.
  out  |o - ref| <= 2^-8 |ref| + w sum_j a_j |v_j| + n sum_j a_j (|lo_j| + 15 step_j)
       w: the weights' relative error, 2^-11 (fp16, the same for a value's offset
       and code), a factor e^(2 ds) for the scores' absolute error ds, and 2^-18
       for exponentials, logarithms, reciprocals and the factors' products (each
       a few 2^-23); n: the products' sums, (keys / 16 + 64) 2^-23.
       ds = (d / 16 + 8) 2^-23 scale sum_f |q_f| (|lo| + 15 step) at its largest.
  lse  5e-4 + 1e-6 |lse| as for the other entries (parity_util); ds is below that.
"""
import numpy as np
import torch

from tests import cache_util as cu


def bf16_up(x):
    """The smallest bf16 numbers >= x (float64, positive, normal)."""
    m, e = np.frexp(x)
    return np.ldexp(np.ceil(m * 256.0), e - 8)


def quantise(x):
    """Codes (uint8 0 .. 15) and (offset, step) float64 [..., 2] of rows [..., d] of
    finite float64 values, by the definition: the step is checked against both of its
    sides, and a code counts the middles between neighbours that lie below x."""
    lo, hi = x.min(-1), x.max(-1)
    top = np.abs(x).max(-1)
    step = bf16_up(np.maximum(np.maximum((hi - lo) / 15, top * 2.0 ** -13), 2.0 ** -60))

    def enough(s):
        return (lo + 15 * s >= hi) & (s >= top * 2.0 ** -13) & (s >= 2.0 ** -60)

    below = np.nextafter(step, 0)
    m, e = np.frexp(below)
    below = np.ldexp(np.floor(m * 256.0), e - 8)
    assert enough(step).all() and not enough(below).any()
    codes = np.zeros(x.shape, dtype=np.uint8)
    for k in range(1, 16):
        codes += (x > lo[..., None] + (k - 0.5) * step[..., None]).astype(np.uint8)
    return codes, np.stack((lo, step), -1)


def packed(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpacked(b):
    return np.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], -1)


def values(codes, pairs):
    """float64 rows [B, L, H, d] of codes [B, L, H, d] and (offset, step) [B, H, L, 2]."""
    p = pairs.transpose(0, 2, 1, 3)
    return p[..., :1] + codes * p[..., 1:]


def q4_cache(x, garbage_from=None, seed=0):
    """(packed codes uint8, pairs bf16 [B, H, L, 2]) of bf16 rows [B, L, H, d];
    positions from garbage_from[b] on hold random codes and NaN pairs."""
    codes, pairs = quantise(cu.f64(x))
    codes, pairs = packed(codes), np.ascontiguousarray(pairs.transpose(0, 2, 1, 3))
    if garbage_from is not None:
        rng = np.random.default_rng(seed)
        for b, n in enumerate(garbage_from):
            codes[b, max(0, n):] = rng.integers(0, 256, size=codes[b, max(0, n):].shape)
            pairs[b, :, max(0, n):] = np.nan
    return torch.from_numpy(codes), torch.from_numpy(pairs).to(torch.bfloat16)


def cache_f64(codes, pairs):
    """What a cache's tensors stand for (NaN or infinite: 0)."""
    p = np.nan_to_num(cu.f64(pairs), nan=0.0, posinf=0.0)
    return values(unpacked(codes.cpu().numpy()), p), p


def reach(pairs):
    """|lo| + 15 step of (offset, step) [B, H, L, 2] as [B, L, H, 1]."""
    return (np.abs(pairs[..., 0]) + 15 * pairs[..., 1]).transpose(0, 2, 1)[..., None]


def assert_out_close(got, q, k_pairs, v_pairs, ref, size, sees_of, keys, scale=None, what=""):
    """q [B, T, H, d] float64, pairs [B, H_kv, L, 2] float64, ref and size from
    cache_util.attention over the cache's values."""
    B, T, H, d = ref.shape
    got = cu.f64(got).reshape(ref.shape)
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    G = H // k_pairs.shape[1]
    ds, span = np.zeros((B, T, H, 1)), np.zeros((B, T, H, 1))
    for b in range(B):
        cols = np.nonzero(sees_of(b).any(0))[0]
        if cols.size == 0:
            continue
        for h in range(H):
            rk, rv = (np.abs(p[b, h // G, cols, 0]) + 15 * p[b, h // G, cols, 1] for p in (k_pairs, v_pairs))
            ds[b, :, h, 0] = (d / 16 + 8) * 2.0 ** -23 * scale * np.abs(q[b, :, h]).sum(-1) * rk.max()
            span[b, :, h, 0] = rv.max()
    w = (1 + 2.0 ** -11 + 2.0 ** -18) * np.exp(2 * ds) - 1
    room = 2.0 ** -8 * np.abs(ref) + 1.01 * w * size + (keys / 16 + 64) * 2.0 ** -23 * span
    excess = np.abs(got - ref) - room
    assert excess.max(initial=-1.0) <= 0, f"{what}: off by {excess.max():.3e} more than the roundings allow"
