"""Host threads that make the first calls of a kernel at the same time, with
different amounts of shared memory."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import sys, threading
import torch
sys.path.insert(0, "tests")
import cache_util as R
import gqa_flash_attention_prefill_gb300 as pkg
from gqa_flash_attention_prefill_gb300 import workloads as W

pkg.load()
heads = [1, 2, 3, 5, 6, 7, 1, 3]  # KV heads: as many ring shapes of one kernel
errors = []
for d, kind, new in [(64, "e4m3", 1), (64, "16", 1), (128, "e4m3", 1), (128, "16", 1), (256, "e4m3", 1), (256, "16", 1),
                     (64, "e4m3", 10), (64, "16", 10), (64, "e4m3", 20), (128, "e4m3", 10), (128, "16", 12)]:
    runs = []
    for h in heads:
        b = W.make_batch([0], [new], h, h, d, "bf16", seed=h)
        b.prefix_lens = torch.tensor([90], dtype=torch.int32)
        cache = R.fill(W.empty_cache([90 + new], h, d, 16, "bf16", kind), b, h)
        dev = b.to("cuda")
        size = pkg.cache_attention_workspace(1, new, new, h, h, d, "bf16", kind)
        ws, out = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.zeros_like(dev.q)
        stream = torch.cuda.Stream()
        ref = R.attention(b.q, cache, [0, new], [90], b.scale, b.window, b.sinks, b.smooth)
        runs.append((dev, R.on_gpu(cache), ws, out, stream, ref))
    torch.cuda.synchronize()
    gate = threading.Barrier(len(runs))

    def go(dev, cache, ws, out, stream, wait):
        try:
            if wait:
                gate.wait()
            pkg.cache_attention(dev, cache, workspace=ws, out=out, with_lse=False, stream=stream)
        except Exception as e:
            errors.append((d, kind, new, dev.hkv, str(e)))

    threads = [threading.Thread(target=go, args=(*r[:5], True)) for r in runs]
    [t.start() for t in threads]
    [t.join() for t in threads]
    for r in runs:  # every shape again: the kernel has kept what the largest needs
        go(*r[:5], False)
    torch.cuda.synchronize()
    for *_, out, _, (ref, _, bound, _) in runs:
        assert bool(((out.cpu().double() - ref).abs() <= bound).all())
assert not errors, errors
assert pkg.get_device_status() == 0
print("ok")
"""


def test_first_calls_from_many_threads():
    import __graft_entry__
    __graft_entry__.build()
    for _ in range(3):
        res = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=200)
        assert res.returncode == 0 and res.stdout.strip() == "ok", res.stdout + res.stderr
