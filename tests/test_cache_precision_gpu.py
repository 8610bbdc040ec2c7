"""What the probabilities of a decoded token keep of fp32: values that cancel,
so that the output is far smaller than its terms."""
import math

import pytest
import torch

import cache_util as R
from gqa_flash_attention_prefill_gb300 import workloads as W
from test_cache_gpu import DT, pkg, status_ok  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def cancelling(n, hkv, d, dtype, kind, seed):
    """Scores (natural, one 16-bit or e4m3 value each) and values of n keys;
    the last four keys, of falling weight, take up what the others leave."""
    gen = torch.Generator().manual_seed(seed)
    held = torch.float8_e4m3fn if kind == "e4m3" else DT[dtype]
    score = -torch.rand(n, hkv, generator=gen) * 2
    score[-3:] = torch.tensor([-3.0, -5.0, -7.0])[:, None]
    score = score.to(held).double()
    v = torch.randn(n, hkv, d, generator=gen).to(held).double()
    p = torch.softmax(score, 0)
    for i in range(n - 4, n):
        rest = (p[:, :, None] * v).sum(0) - p[i][:, None] * v[i]
        v[i] = (-rest / p[i][:, None]).float().to(held).double()
    return score, v, p, held


@pytest.mark.parametrize("dtype,kind", [("f16", "16"), ("bf16", "16"), ("f16", "e4m3")])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (8, 8, 128), (6, 3, 256), (64, 8, 64)])
@pytest.mark.parametrize("n", [6, 40, 700])
def test_probabilities_keep_more_than_the_output(pkg, hq, hkv, d, dtype, kind, n):  # noqa: F811
    """q is 1 at one place, so a score is one product, exact.  The bound: the
    output's half step; P in two terms (u^2 of each, u the half step of one;
    2^-30 of the largest where the second term leaves f16's range); and 2.5
    rho for fp32: the scale and log2 e (2^-24 each of the exponent, |s| log2 e
    up to 11), the exponential 2^-22, its argument's rounding (2^-23 of the
    exponent plus the reference, up to 32), the sums n 2^-24."""
    score, v, p, held = cancelling(n, hkv, d, dtype, kind, seed=n + d)
    cache = W.empty_cache([n], hkv, d, 16, dtype, kind)
    at = R.keys_of(cache, 0, 0, n)
    k = torch.zeros(n, hkv, d, dtype=torch.float64)
    k[:, :, 5] = score
    for pages, x in ((cache.k_pages, k), (cache.v_pages, v)):
        if kind == "e4m3":
            pages.view(torch.uint8).flatten(0, 1)[at] = x.float().to(held).view(torch.uint8)
        else:
            pages.flatten(0, 1)[at] = x.to(held)
    if kind == "e4m3":
        cache.k_scales.fill_(127)
        cache.v_scales.fill_(127)
    b = W.make_batch([0], [1], hq, hkv, d, dtype, sink_mode="none", scale=1.0)
    b.prefix_lens = torch.tensor([n - 1], dtype=torch.int32)
    b.q.zero_()
    b.q[0, :, 5] = 1.0
    out, _ = pkg.cache_attention(b.to("cuda"), R.on_gpu(cache))
    status_ok(pkg)
    want = (p[:, :, None] * v).sum(0).repeat_interleave(hq // hkv, 0)
    size = (p[:, :, None] * v.abs()).sum(0).repeat_interleave(hq // hkv, 0)
    total = v.abs().sum(0).repeat_interleave(hq // hkv, 0)
    u, up = R.U[DT[dtype]], R.U[torch.float16 if kind == "e4m3" else DT[dtype]]
    rho = 2 * 11 * 2.0 ** -24 + 2.0 ** -22 + 32 * 2.0 ** -23 + n * 2.0 ** -24
    tol = u * want.abs() + (1 + u) * ((up ** 2 + 2.5 * rho) * size + 2.0 ** -30 * total) + R.TINY[DT[dtype]]
    err = (out[0].cpu().double() - want).abs()
    assert bool((err <= tol).all()), (float((err / tol).max()), float((size / want.abs().clamp(min=1e-9)).median()))
    assert math.isfinite(float(err.max()))
