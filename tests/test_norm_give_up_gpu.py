"""The norm's gradient when a bounded wait runs out: the CTA stops where it is, for all its threads, issues no further copy and
waits for those in flight; dweight is not written; the call's other rows are right, and so is the next call."""
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

rows, n, stream = int(sys.argv[1]), int(sys.argv[2]), getattr(torch, sys.argv[3])
gen = torch.Generator(device="cuda").manual_seed(1)
randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")
dy, h, dh, w = randn(rows, n).bfloat16(), randn(rows, n).to(stream), randn(rows, n).to(stream), randn(n)
rstd = (h.float().square().mean(-1) + 1e-5).rsqrt()
ws = torch.full((pkg.rms_norm_backward_workspace(rows, 1, n, "bf16"),), 255, dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
for name in ("first", "again"):
    dx, dw = torch.full_like(dy, 7.0), torch.full((n,), 7.0, device="cuda")
    pkg.gqa_rms_norm_backward(dy, h, w, rstd, dx, dweight=dw, workspace=ws, dh=dh)
    torch.cuda.synchronize()
    status = pkg.get_device_status()
    torch.save((dx.cpu(), dw.cpu(), status), sys.argv[4] + name)
"""


# Stages of the ring: four, two, one.  CTA 1 gives up in its first warp alone, at the first row of its second time round
# the ring; CTA 2 in its last thread alone, at its first row.
PLACE = ("blockIdx.x == 1 ? parity == 1u && threadIdx.x < 32 : "
         "blockIdx.x == 2 && parity == 0u && threadIdx.x == blockDim.x - 1")


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    return give_up.library(str(tmp_path_factory.mktemp("give_up")), "rms_norm.cu", "prefill_kernel.cuh", PLACE)


@pytest.mark.parametrize("n,stream,stages,per_sm", [(4096, "bfloat16", 4, 2), (8200, "float32", 2, 1), (16384, "float32", 1, 1)])
def test_waits_that_run_out(library, tmp_path, n, stream, stages, per_sm):
    import torch
    import gqa_flash_attention_prefill_gb300 as pkg
    ctas = torch.cuda.get_device_properties(0).multi_processor_count * per_sm
    rows = ctas * 7 + 5
    got = {}
    for name, lib in (("own", None), ("cut", library)):
        env = dict(os.environ)
        env.pop("GQA_PREFILL_LIB", None)
        if lib is not None:
            env["GQA_PREFILL_LIB"] = lib
        at = str(tmp_path / name)
        res = subprocess.run([sys.executable, "-c", CHILD, str(rows), str(n), stream, at], cwd=ROOT, env=env, capture_output=True,
                             text=True, timeout=200)
        assert res.returncode == 0, res.stdout + res.stderr
        got[name] = [torch.load(at + x) for x in ("first", "again")]
    for dx, dw, status in got["own"]:
        assert status == 0 and torch.equal(dx, got["own"][0][0]) and torch.equal(dw, got["own"][0][1])
        assert bool(dw.isfinite().all()) and not bool((dw == 7.0).all())
    want = got["own"][0][0]
    for dx, dw, status in got["cut"]:
        assert status == pkg.GQA_DEV_TIMEOUT
        assert bool((dw == 7.0).all())
        row = torch.arange(rows)
        left = (row % ctas == 2) | ((row % ctas == 1) & (row // ctas >= stages))
        assert torch.equal(dx[~left], want[~left]) and bool((dx[left] == 7.0).all())
