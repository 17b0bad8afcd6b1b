"""Every form of a step over a 4-bit cache gives the same bits on every call: over one, two, up
to eight, sixteen, 32 and more rows per key head, in one unit, in splits, and in launches
with more units than run at once, with other work between the calls."""
import pytest
import torch

from tests.test_cache_gpu import mha, on_gpu  # noqa: F401
from tests.test_cache_q4_gpu import call_step, make_step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,G", [(1, 1), (2, 1), (4, 2), (16, 1), (8, 2), (16, 2), (33, 1), (32, 4)])
@pytest.mark.parametrize("B,H_kv,Lk", [(1, 1, 300), (2, 2, 9000), (40, 40, 700)], ids=["a unit", "splits", "waves"])
def test_a_step_repeats(mha, d, T, G, B, H_kv, Lk):  # noqa: F811
    small = min(B, 4)
    case = make_step(d + T + B, small, T, small * G, small, d, Lk, [Lk - T - 37 * b for b in range(small)], None, "tree")
    g = on_gpu(case)
    if B > small:                       # more sequences and heads: the same ones again
        n = B // small
        g = {"q": g["q"].repeat(n, 1, n, 1), "prefix": g["prefix"].repeat(n), "drafts": None,
             "mask": g["mask"].repeat(n, 1, 1), "kc": g["kc"].repeat(n, 1, n, 1), "vc": g["vc"].repeat(n, 1, n, 1),
             "ks": g["ks"].repeat(n, n, 1, 1), "vs": g["vs"].repeat(n, n, 1, 1)}
    out, lse = call_step(mha, g, True)
    if B > small:                       # ... and so are their rows
        assert torch.equal(out[:small, :, :small * G], out[small:2 * small, :, small * G:2 * small * G])
    noise = torch.zeros(1 << 26, device="cuda")
    for i in range(12):
        if i % 3 == 0:
            noise.add_(1.0)             # (over what the caches hold of the inputs)
        again = call_step(mha, g, True)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    assert mha.mha_sync_status() == 0
