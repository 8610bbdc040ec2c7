"""gqa_cache_attention where the units of one launch differ: row tiles that
come and go, and magnitudes that differ from tile to tile of the cache, so that
a tile taken with another tile's scale shows."""
import pytest
import torch

import cache_util as R
from gqa_flash_attention_prefill_gb300 import workloads as W
from test_cache_gpu import check, pkg  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def uneven_case(pre, new, hq, hkv, d, kind, tree, seed):
    """Keys and values whose scale changes by 2^-3 .. 2^3 from one run of 64
    keys to the next, and by 2^0 .. 2^3 between sequences."""
    b = W.make_batch([0] * len(pre), new, hq, hkv, d, "bf16", sink_mode="head", seed=seed)
    b.prefix_lens = torch.tensor(pre, dtype=torch.int32)
    cache = R.fill(W.empty_cache([p + n for p, n in zip(pre, new)], hkv, d, 64, "bf16", kind, seed=seed), b, seed + 1, 0)
    gen = torch.Generator().manual_seed(seed + 2)
    for i, (p, n) in enumerate(zip(pre, new)):
        own = int(torch.randint(0, 4, (1,), generator=gen))
        for k0 in range(0, p + n, 64):
            at = R.keys_of(cache, i, k0, min(k0 + 64, p + n))
            for x in "kv":
                e = int(torch.randint(-3, 4, (1,), generator=gen)) - own
                if kind == "e4m3":
                    getattr(cache, x + "_scales").flatten(0, 1)[at] = 120 + e
                else:
                    getattr(cache, x + "_pages").flatten(0, 1)[at] *= 2.0 ** (e - 1)
    keep = depths = None
    if tree:
        keep = [W.random_tree_mask(n, seed=seed + i) for i, n in enumerate(new)]
        depths = [[int(m[t].sum()) - 1 for t in range(m.shape[0])] for m in keep]
    return b, cache, keep, depths


# Query heads per KV head G, new tokens of the sequences: units of 256 rows, the
# last of a sequence narrower (at most 128 rows: its second row tile is empty).
@pytest.mark.parametrize("hq,hkv,d,pre,new,tree", [
    (64, 8, 64, [5000] * 6, [40] * 6, True),                       # 256 rows, then 64
    (64, 8, 64, [8192, 9000, 8000, 8100], [8, 64, 8, 64], True),   # 64 rows, then 512
    (32, 4, 128, [4096, 3000, 5000], [40, 8, 33], True),           # 64-key tiles
    (64, 8, 128, [3000, 2500, 2900, 3100], [16, 17, 3, 48], False),
    (8, 8, 64, [6000, 7000, 5000, 200], [60, 200, 100, 300], False),
    (64, 2, 64, [20000, 30000, 16000], [4, 12, 2], True)])
@pytest.mark.parametrize("kind", ["e4m3", "16"])
def test_row_tiles_that_come_and_go(pkg, hq, hkv, d, pre, new, tree, kind):  # noqa: F811
    """Units with one row tile before units with two, in shares of many key
    tiles: every row within its bound, and the same bits again."""
    b, cache, keep, depths = uneven_case(pre, new, hq, hkv, d, kind, tree, seed=sum(new) + d)
    first = check(pkg, b, cache, keep, depths)
    again = check(pkg, b, cache, keep, depths)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("hint", [0, 1, 5, 64, 2 ** 31 - 1])
@pytest.mark.parametrize("kind,window", [("e4m3", 0), ("16", 0), ("e4m3", 100), ("16", 33)])
def test_hint_of_the_longest_sequence_may_be_wrong(pkg, hint, kind, window):  # noqa: F811
    """max_seqlen_q shapes the launch; any value gives the same operation.
    Sequences without new tokens stand between and behind the others."""
    pre, new = [40, 700, 0, 1500, 9, 300], [0, 5, 0, 64, 1, 0]
    b, cache, keep, depths = uneven_case(pre, new, 16, 2, 64, kind, True, seed=hint % 1000 + window)
    b.window = window
    dev, gpu = b.to("cuda"), R.on_gpu(cache)
    mask, indptr = (t.cuda() for t in W.pack_custom_mask(keep))
    dep = torch.tensor(sum(([int(x) for x in r] for r in depths), []), dtype=torch.int32).cuda()
    size = pkg.cache_attention_workspace(len(pre), b.total_q, hint, 16, 2, 64, "bf16", kind)
    out = torch.full_like(dev.q, float("nan"))
    lse = torch.full(dev.q.shape[:2], float("nan"), device="cuda")
    pkg.gqa_cache_attention(dev.q, gpu.k_pages, gpu.v_pages, dev.cu_seqlens_q, dev.prefix_lens, gpu.page_indptr,
                            gpu.page_indices, dev.scale, torch.empty(size, dtype=torch.uint8, device="cuda"),
                            window=window, sinks=dev.sinks, k_scales=gpu.k_scales, v_scales=gpu.v_scales,
                            custom_mask=mask, mask_indptr=indptr, depths=dep, out=out, lse=lse, max_seqlen_q=hint)
    torch.cuda.synchronize()
    assert pkg.get_device_status() == 0
    ref, z, bo, bl = R.attention(b.q, cache, b.cu_seqlens_q.tolist(), pre, b.scale, window, b.sinks, False, keep, depths)
    assert bool(((out.cpu().double() - ref).abs() <= bo).all()) and bool(((lse.cpu().double() - z).abs() <= bl).all())


@pytest.mark.parametrize("kind", ["16", "e4m3"])
def test_one_graph_for_a_growing_cache(pkg, kind):  # noqa: F811
    """A decode step captured once and replayed while lengths, page table and
    tokens change in place, over buffers sized for the longest."""
    hq, hkv, d, page, cap = 16, 2, 64, 16, 700
    pool = W.empty_cache([cap] * 3, hkv, d, page, "bf16", kind, device="cuda")
    order = pool.page_indices.tolist()
    per = -(-cap // page)
    lens = [0, 655, 14]
    # earlier tokens: random rows, as a prompt left them
    host = R.fill(W.empty_cache([cap] * 3, hkv, d, page, "bf16", kind), None, 3)
    for f in ("k_pages", "v_pages", "k_scales", "v_scales"):
        if getattr(host, f) is not None:
            getattr(pool, f).copy_(getattr(host, f))
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, pre = torch.tensor([0, 1, 2, 3], **i32), torch.zeros(3, **i32)
    ip, idx = torch.zeros(4, **i32), torch.zeros(3 * per, **i32)
    q, k, v = (torch.empty(3, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    out, lse = torch.empty_like(q), torch.empty(3, hq, device="cuda")
    ws = torch.empty(pkg.cache_attention_workspace(3, 3, 1, hq, hkv, d, "bf16", kind), dtype=torch.uint8, device="cuda")

    def set_step(step):
        gen = torch.Generator().manual_seed(step)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=gen).to(torch.bfloat16))
        pre.copy_(torch.tensor(lens, dtype=torch.int32))
        table = [order[i * per:i * per + n // page + 1] for i, n in enumerate(lens)]
        ip.copy_(torch.tensor([0] + torch.tensor([len(t) for t in table]).cumsum(0).tolist(), dtype=torch.int32))
        flat = sum(table, [])
        idx[:len(flat)].copy_(torch.tensor(flat, dtype=torch.int32))

    def step():
        pkg.gqa_cache_write(k, v, cu, pre, ip, idx, pool.k_pages, pool.v_pages, k_scales=pool.k_scales,
                            v_scales=pool.v_scales)
        pkg.gqa_cache_attention(q, pool.k_pages, pool.v_pages, cu, pre, ip, idx, d ** -0.5, ws, k_scales=pool.k_scales,
                                v_scales=pool.v_scales, out=out, lse=lse, max_seqlen_q=1)

    set_step(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(20):
        set_step(n)
        graph.replay()
        torch.cuda.synchronize()
        assert pkg.get_device_status() == 0
        if n % 4 == 3:
            now = W.Cache(*(t.cpu() if t is not None else None for t in (
                pool.k_pages, pool.v_pages, pool.k_scales, pool.v_scales, ip, idx)), kind)
            ref, z, bo, bl = R.attention(q.cpu(), now, [0, 1, 2, 3], lens, d ** -0.5)
            assert bool(((out.cpu().double() - ref).abs() <= bo).all())
            assert bool(((lse.cpu().double() - z).abs() <= bl).all())
        lens = [x + 1 for x in lens]
