"""The attention's gradient when a bounded wait runs out: the call ends and says so, its cut units are not joined and the sinks'
gradient is not written, what it did write is right, and so is the next call on the same workspace."""
import os
import subprocess
import sys

import pytest

import give_up

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import sys
import torch
import gqa_flash_attention_prefill_gb300 as pkg
from gqa_flash_attention_prefill_gb300 import workloads as W

d, tokens, prefix = (int(x) for x in sys.argv[1:4])
b = W.make_batch([prefix, 0], [tokens, 9], 8, 2, d, "bf16", sink_mode="head").to("cuda")
out, lse = pkg.prefill(b)
dout = torch.randn(b.q.shape, generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
size = pkg.prefill_backward_workspace(2, b.total_q, b.total_kv, 8, 2, d, "bf16")
ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
assert pkg.get_device_status() == 0
for name in ("first", "again"):
    res = [torch.full_like(x, 7.0) for x in (b.q, b.k, b.v, b.sinks)]
    pkg.gqa_prefill_backward(b.q, b.k, b.v, b.cu_seqlens_q, b.prefix_lens, b.kv_indptr, b.scale, out, lse, dout, *res[:3], ws,
                             sinks=b.sinks, dsinks=res[3])
    torch.cuda.synchronize()
    status = pkg.get_device_status()
    torch.save(([x.cpu() for x in res], status), sys.argv[4] + name)
"""

# The limit's last digit is the warp of CTA 1 that gives up (0: the first softmax warp, 1: the one that loads, 2: the one that
# issues the products), the digits before it how many of its waits pass before.
PLACE = ("blockIdx.x == 1 && (threadIdx.x & 31) == 0 && "
         "threadIdx.x / 32 == (timeout_ns / 1000000 % 10 == 0 ? 0 : blockDim.x / 32 - 3 + timeout_ns / 1000000 % 10) && "
         "atomicAdd(&give_up_calls, 1) == (timeout_ns / 1000000 - 2000) / 10")


@pytest.fixture(scope="module")
def libraries(tmp_path_factory):
    made = {}

    def get(d):
        if d not in made:
            made[d] = give_up.library(str(tmp_path_factory.mktemp("give_up")), f"inst_bwd_d{d}.cu", "prefill_kernel.cuh", PLACE)
        return made[d]
    return get


def child(at, lib, limit, *args):
    import torch
    env = dict(os.environ, GQA_PREFILL_TIMEOUT_MS=str(limit))
    env.pop("GQA_PREFILL_LIB", None)
    if lib is not None:
        env["GQA_PREFILL_LIB"] = lib
    res = subprocess.run([sys.executable, "-c", CHILD, *(str(a) for a in args), at], cwd=ROOT, env=env, capture_output=True, text=True,
                         timeout=200)
    assert res.returncode == 0, res.stdout + res.stderr
    return [torch.load(at + x) for x in ("first", "again")]


# A unit or two a CTA, whose loads are all issued before the wait that gives up; and long streams of tiles.
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("tokens,prefix", [(40, 0), (900, 1100)])
def test_waits_that_run_out(libraries, tmp_path, d, tokens, prefix):
    import torch
    import gqa_flash_attention_prefill_gb300 as pkg
    own = child(str(tmp_path / "own"), None, 4000, d, tokens, prefix)
    want = own[0][0]
    assert all(status == 0 for _, status in own) and all(torch.equal(x, y) for x, y in zip(own[1][0], want))
    for which in (0, 1, 2):
        for passed in (0, 1, 4) if tokens < 100 else (0, 4, 9, 20):
            first, again = child(str(tmp_path / "cut"), libraries(d), 2000 + 10 * passed + which, d, tokens, prefix)
            if passed < (2 if tokens < 100 else 10):  # the waits that each of these warps has at least
                assert first[1] == pkg.GQA_DEV_TIMEOUT, (which, passed)
            if first[1] == 0:  # fewer waits than that: the call after it is the one that is cut short
                first, again = again, first
            if first[1] != 0:
                assert bool((first[0][3] == 7.0).all())
                for x, y in zip(first[0][:3], want):
                    assert bool(((x == y) | (x == 7.0)).all()), (which, passed)
            assert again[1] == 0 and all(torch.equal(x, y) for x, y in zip(again[0], want)), (which, passed)
