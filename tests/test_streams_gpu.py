"""Wrappers that allocate for a call on another stream than the current one:
the call's memory is not handed out while the call has yet to run."""
import pytest
import torch

import cache_util as R
from gqa_flash_attention_prefill_gb300 import workloads as W
from test_cache_gpu import pkg  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def cases(pkg):  # noqa: F811
    """name -> (call of a stream, workspace bytes or 0)"""
    b = W.make_batch([0, 0], [1, 1], 16, 2, 64, "bf16", sink_mode="head", seed=1)
    b.prefix_lens = torch.tensor([5000, 40], dtype=torch.int32)
    cache = R.on_gpu(R.fill(W.empty_cache([5001, 41], 2, 64, 16, "bf16", "e4m3"), b, 2))
    dev = b.to("cuda")
    indptr = torch.tensor([0, 5001, 5042], dtype=torch.int32, device="cuda")
    full = W.make_batch([3000, 0], [40, 200], 16, 2, 64, "bf16", sink_mode="head", seed=3)
    paged = W.paged(full, 16, seed=4).to("cuda")
    words, mip = (t.cuda() for t in W.pack_custom_mask([W.random_tree_mask(n, seed=n) for n in (40, 200)]))
    full = full.to("cuda")
    return {
        "cache_attention": (lambda s: pkg.cache_attention(dev, cache, stream=s),
                            pkg.cache_attention_workspace(2, 2, 1, 16, 2, 64, "bf16", "e4m3")),
        "cache_read": (lambda s: pkg.cache_read(cache, indptr, 5042, torch.bfloat16, stream=s), 0),
        "prefill": (lambda s: pkg.prefill(full, stream=s), 0),
        "prefill_masked": (lambda s: pkg.prefill_masked(full, words, mip, stream=s), 0),
        "prefill_paged": (lambda s: pkg.prefill_paged(paged, stream=s), 0),
        "prefill_splitkv": (lambda s: pkg.prefill_splitkv(full, num_splits=4, stream=s),
                            pkg.splitkv_workspace(2, 240, 200, 16, 2, 64, "bf16", 0, 4)[1]),
    }


@pytest.mark.parametrize("name", ["cache_attention", "cache_read", "prefill", "prefill_masked", "prefill_paged",
                                  "prefill_splitkv"])
@pytest.mark.parametrize("handle", [False, True])
def test_memory_of_a_call_on_another_stream(pkg, name, handle):  # noqa: F811
    """The call waits behind a busy stream while the current stream takes and
    fills blocks of its sizes: neither sees the other's bytes."""
    call, nbytes = cases(pkg)[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(other):
            torch.cuda._sleep(20_000_000)  # some 10 ms
        got = call(other.cuda_stream if handle else other)
        sizes = [nbytes] * 4 if nbytes else []
        sizes += [t.numel() * t.element_size() for t in got] * 2
        blocks = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]
        other.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(bool((x == 255).all()) for x in blocks)
        del blocks
    assert pkg.get_device_status() == 0


def test_handles_name_their_stream(pkg):  # noqa: F811
    """A raw handle allocates on the stream it names, 0 on the default one."""
    other = torch.cuda.Stream()
    with torch.cuda.stream(torch.cuda.Stream()):
        mine = torch.cuda.current_stream().cuda_stream
        for stream, handle in ((None, mine), (0, 0), (other, other.cuda_stream), (other.cuda_stream, other.cuda_stream),
                               (torch.cuda.default_stream(), 0)):
            with pkg._allocating(stream):
                assert torch.cuda.current_stream().cuda_stream == handle
            assert torch.cuda.current_stream().cuda_stream == mine
