"""Calls on a stream other than the current one, whose outputs and workspaces
come from the current stream's memory: that memory may be a tensor's that was
just freed there and is still in use by what is queued on it."""
import pytest
import torch

from tests import cache_util as cu
from tests.test_cache_gpu import call_step, i32, make_step, mha, on_gpu  # noqa: F401

pytestmark = pytest.mark.gpu

SLEEP = 40_000_000   # cycles: some 20 ms, far more than a call takes


def behind_a_reader(like, call):
    """Calls `call` on another stream just after a tensor of `like`'s size was freed
    on the current one, where its last reader is still waiting; returns the call's
    result and whether that reader saw what the tensor held."""
    torch.cuda.synchronize()
    held = torch.full_like(like, 3.0)
    copy = torch.zeros_like(like)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(SLEEP)
    copy.copy_(held)
    at = held.data_ptr()
    del held
    result = call(side)
    first = result[0]
    reused = first.data_ptr() == at
    torch.cuda.synchronize()
    return result, reused, bool((copy == 3.0).all())


STEPS = [
    ("decode_f8", (8, 1, 8, 8, 64, 200), [200, 0, 1, 127, 128, 129, 199, 60]),   # CUDA cores
    ("decode_f8", (2, 1, 8, 2, 128, 9000), [8000, 33]),                          # splits: a workspace
    ("tree", (2, 5, 8, 2, 128, 9000), [8000, 33]),
    ("tree", (2, 40, 8, 2, 128, 900), [800, 33]),
    ("tree_f8", (2, 5, 8, 2, 128, 9000), [8000, 33]),
]


@pytest.mark.parametrize("kind,shape,lens", STEPS, ids=lambda x: str(x) if isinstance(x, str) else "")
@pytest.mark.parametrize("as_int", [True, False], ids=["handle", "object"])
def test_steps_wait_for_their_memory(mha, kind, shape, lens, as_int):  # noqa: F811
    f8, with_drafts = kind != "tree", kind != "decode_f8"
    g = on_gpu(make_step(60, *shape, lens, None, "tree" if with_drafts else None, f8, with_drafts))
    want = call_step(mha, g, f8, with_drafts)
    # (a tensor of the output's size is what the allocator hands out again)
    got, reused, kept = behind_a_reader(
        want[0], lambda s: call_step(mha, g, f8, with_drafts, stream=s.cuda_stream if as_int else s))
    assert mha.mha_sync_status() == 0
    assert reused and kept
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_read_waits_for_its_memory(mha):  # noqa: F811
    x = cu.random_rows(1, (3, 400, 4, 64))
    codes, scales = cu.f8_cache(x)
    dev = [codes.cuda(), codes.cuda(), scales.cuda(), scales.cuda(), i32([400, 0, 77]).cuda()]
    want = mha.mha_cache_read_f8(*dev)
    got, reused, kept = behind_a_reader(want[0], lambda s: mha.mha_cache_read_f8(*dev, stream=s))
    assert mha.mha_sync_status() == 0
    assert reused and kept
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_default_stream_from_another(mha):  # noqa: F811
    """stream=0, the default stream, while another is current."""
    g = on_gpu(make_step(61, 2, 1, 8, 2, 128, 9000, [8000, 33], None, None, True, False))
    want = call_step(mha, g, True, False)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for stream in (0, torch.cuda.default_stream()):
            got = call_step(mha, g, True, False, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert mha.mha_sync_status() == 0


def older_calls(mha):
    """The entries that read no 8-bit cache, on small inputs: (name, call(stream))."""
    def t(seed, *shape):
        return cu.random_rows(seed, shape).cuda()

    q, k, v, do = (t(s, 2, 96, 4, 64) for s in range(4))
    lens = i32([96, 50]).cuda()
    out, lse = mha.mha_fwd(q, k, v, return_lse=True)
    f = [x.float() for x in (q, k, v)]
    narrow, one = v[..., :32].contiguous(), q[:, 0].contiguous()
    x, w_qkv, w_o = t(5, 2, 96, 256), t(6, 256, 3 * 256), t(7, 256, 256)
    cache = [t(8 + i, 2, 3000, 4, 64) for i in range(2)]
    clens = i32([3000, 1700]).cuda()
    return {
        "mha_fwd": lambda s: mha.mha_fwd(q, k, v, stream=s, return_lse=True),
        "mha_fwd_dv": lambda s: mha.mha_fwd(q, k, narrow, stream=s, return_lse=True),
        "mha_fwd_f32": lambda s: mha.mha_fwd_f32(*f, mask_kind=2, key_lens=lens, stream=s, return_lse=True),
        "mha_bwd": lambda s: mha.mha_bwd(q, k, v, out, do, lse, stream=s),
        "mha_layer_fwd": lambda s: (mha.mha_layer_fwd(x, w_qkv, w_o, 4, stream=s),),
        "mha_gemm_bf16": lambda s: (mha.mha_gemm_bf16(x[0], w_qkv, stream=s),),
        "mha_decode": lambda s: mha.mha_decode(one, *cache, clens, stream=s, return_lse=True),
        "mha_decode_static": lambda s: mha.mha_decode_static(one, *cache, clens, stream=s, return_lse=True),
    }


@pytest.mark.parametrize("name", ["mha_fwd", "mha_fwd_dv", "mha_fwd_f32", "mha_bwd", "mha_layer_fwd",
                                  "mha_gemm_bf16", "mha_decode", "mha_decode_static"])
def test_other_entries_wait_for_their_memory(mha, name):  # noqa: F811
    call = older_calls(mha)[name]
    want = call(None)
    got, _, kept = behind_a_reader(want[0], call)
    assert mha.mha_sync_status() == 0
    assert kept
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_kernels_of_two_streams_share_the_machine(mha):  # noqa: F811
    """Steps of every form and the forward, each stream's calls one after the other
    and the two streams' at once: all of them want tensor memory, and each step
    lets its stream's next launch set itself up while it runs."""
    steps = []
    for i, (kind, shape, lens) in enumerate(STEPS):
        f8, with_drafts = kind != "tree", kind != "decode_f8"
        steps.append((on_gpu(make_step(70 + i, *shape, lens, None, "tree" if with_drafts else None, f8,
                                       with_drafts)), f8, with_drafts))
    q, k, v = (cu.random_rows(s, (2, 128, 8, 64)).cuda() for s in range(3))

    def round_of():
        got = [x for g, f8, drafts in steps for x in call_step(mha, g, f8, drafts)]
        return got + [mha.mha_fwd(q, k, v)]

    want = round_of()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    results = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                results.append(round_of())
    torch.cuda.synchronize()
    assert mha.mha_sync_status() == 0
    for got in results:
        for a, b in zip(got, want):
            assert torch.equal(a, b)
