"""A step over a cache whose slots were never written: workloads.empty_cache
holds rows of zeros, which a token attends to like any others."""
import pytest
import torch

import cache_util as R
from gqa_flash_attention_prefill_gb300 import workloads as W
from test_cache_gpu import pkg, status_ok  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["16", "e4m3"])
@pytest.mark.parametrize("new", [1, 12])
def test_step_over_an_empty_prefix(pkg, new, kind):  # noqa: F811
    """Written tokens after an empty prefix, as in the README's example."""
    pre = [1000, 17, 4096, 300]
    b = W.make_batch([0] * 4, [new] * 4, 64, 8, 64, "bf16", sink_mode="head", seed=5)
    b.prefix_lens = torch.tensor(pre, dtype=torch.int32)
    dev = b.to("cuda")
    cache = W.empty_cache([p + new for p in pre], 8, 64, 64, "bf16", kind, device="cuda")
    pkg.cache_write(dev, cache)
    out, lse = pkg.cache_attention(dev, cache)
    status_ok(pkg)
    host = W.Cache(*(t.cpu() if t is not None else None for t in (
        cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales, cache.page_indptr, cache.page_indices)), kind)
    ref, z, bo, bl = R.attention(b.q, host, b.cu_seqlens_q.tolist(), pre, b.scale, 0, b.sinks)
    assert bool(((out.cpu().double() - ref).abs() <= bo).all())
    assert bool(((lse.cpu().double() - z).abs() <= bl).all())


@pytest.mark.parametrize("new", [1, 12])
def test_empty_rows_among_scales_far_apart(pkg, new):  # noqa: F811
    """Zeroed slots next to value rows 2^40 apart in one tile: the 128-row
    kernel then takes an exponent per key."""
    pre = [150, 20]
    b = W.make_batch([0, 0], [new] * 2, 16, 2, 64, "f16", sink_mode="none", seed=14)
    b.prefix_lens = torch.tensor(pre, dtype=torch.int32)
    cache = R.fill(W.empty_cache([p + new for p in pre], 2, 64, 16, "f16", "e4m3"), b, 15)
    gen = torch.Generator().manual_seed(3)
    cache.v_scales.copy_(torch.randint(95, 136, cache.v_scales.shape, generator=gen).to(torch.uint8))
    for i, p in enumerate(pre):
        for at in (R.keys_of(cache, i, 3, 9), R.keys_of(cache, i, p - 2, p)):
            for x in "kv":
                getattr(cache, x + "_pages").view(torch.uint8).flatten(0, 1)[at] = 0
                getattr(cache, x + "_scales").flatten(0, 1)[at] = 0
    from test_cache_gpu import check
    check(pkg, b, cache)
