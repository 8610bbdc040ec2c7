"""gqa_cache_attention whose bounded waits run out: the call ends, reports it,
joins nothing, and the next call is right.  With a limit of 1 ms the warps that
wait for their first piece give up on the CTAs whose planning warp has to walk
some 10^5 row tiles to its share."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import json, sys
import torch
import gqa_flash_attention_prefill_gb300 as pkg
from gqa_flash_attention_prefill_gb300 import workloads as W
sys.path.insert(0, "tests")
import cache_util as R

hkv, tokens, group = (int(x) for x in sys.argv[1:4])
hq, d = hkv * group, 256

def call(b, cache, hkv):
    q = b.q.cuda() if not b.q.is_cuda else b.q
    size = pkg.cache_attention_workspace(1, b.total_q, b.max_seqlen_q, b.hq, hkv, d, "bf16", "16")
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    guard = torch.full((b.total_q + 2, b.hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):
        pkg.gqa_cache_attention(q, cache.k_pages, cache.v_pages, b.cu_seqlens_q.cuda(), b.prefix_lens.cuda(),
                                cache.page_indptr, cache.page_indices, b.scale, ws, out=guard[1:-1],
                                max_seqlen_q=b.max_seqlen_q)
    torch.cuda.synchronize()
    status = pkg.get_device_status()
    assert bool((guard[0] == 7).all() and (guard[-1] == 7).all())
    return guard[1:-1], status

cpu = W.make_batch([0], [1], 2 * hkv, hkv, d, "bf16")
cpu.prefix_lens = torch.tensor([700], dtype=torch.int32)
small = R.fill(W.empty_cache([701], hkv, d, 64, "bf16", "16"), None, 1)
ref, _, bound, _ = R.attention(cpu.q, small, [0, 1], [700], cpu.scale)

def right():  # a millisecond is short: a wait may run out by chance, and says so
    for _ in range(3):
        out, status = call(cpu, R.on_gpu(small), hkv)
        if status == 0:
            return bool(((out.cpu().double() - ref).abs() <= bound).all())
    return False

before = right()
cache = R.on_gpu(W.empty_cache([tokens], hkv, d, 64, "bf16", "16"))

class Big:
    q = torch.zeros(tokens, hq, d, dtype=torch.bfloat16, device="cuda")
    cu_seqlens_q, prefix_lens = torch.tensor([0, tokens], dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    scale, total_q, hq, max_seqlen_q = 0.0625, tokens, hkv * group, tokens

_, status = call(Big, cache, hkv)
print(json.dumps(dict(before=before, status=status, after=right())))
"""


# KV heads (8: a warp per head; 2, 1: four, eight warps that share a head's
# keys), new tokens, query heads per KV head.
@pytest.mark.parametrize("hkv,tokens,group", [(8, 64, 10000), (2, 200, 4000), (1, 300, 2200)])
def test_waits_that_run_out_end_the_call(hkv, tokens, group):
    import __graft_entry__
    __graft_entry__.build()
    import gqa_flash_attention_prefill_gb300 as pkg
    env = dict(os.environ, GQA_PREFILL_TIMEOUT_MS="1")
    res = subprocess.run([sys.executable, "-c", CHILD, str(hkv), str(tokens), str(group)], cwd=ROOT, env=env,
                         capture_output=True, text=True, timeout=200)
    assert res.returncode == 0, res.stdout + res.stderr
    got = json.loads(res.stdout.splitlines()[-1])
    assert got["before"] and got["after"] and got["status"] == pkg.GQA_DEV_TIMEOUT, got
