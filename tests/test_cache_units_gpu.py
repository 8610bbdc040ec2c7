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
