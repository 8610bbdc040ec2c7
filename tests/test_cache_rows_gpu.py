"""gqa_rope and gqa_cache_write where the forms of the other tests cannot tell:
angles of far positions next to the zeros of sine and cosine, rows that belong
to no sequence."""
import math
from fractions import Fraction

import pytest
import torch

import cache_util as R
from gqa_flash_attention_prefill_gb300 import workloads as W
from test_cache_gpu import pkg, rand, status_ok  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu
BITS = 160


def two_pi_inverse():
    """round(2^BITS / (2 pi)), pi by Machin's formula in integers."""
    one = 1 << (BITS + 40)

    def atan_inverse(n):
        term, total, k, sign = one // n, 0, 1, 1
        while term:
            total += sign * (term // k)
            term, k, sign = term // (n * n), k + 2, -sign
        return total

    pi = 4 * (4 * atan_inverse(5) - atan_inverse(239))
    return (one << BITS) // (2 * pi)


@pytest.mark.parametrize("top", [2 ** 31 - 1, 1000000])
def test_rope_of_far_positions(pkg, top):  # noqa: F811
    """Positions where a pair's cosine (or sine) is nearly zero, so that an f16
    result shows the angle itself.  Near a quarter turn the phase is off by
    2^-32 turns where it is cut, and position * 2^-64 from the step: 1.5 *
    2^-32 turns together.  Sine and products are fp32, the result f16: half a
    step, and 2^-20 for the rest.  The other value of the pair is near its
    largest: 2^-20 of it besides."""
    inverse = two_pi_inverse()
    freqs = (W.rope_frequencies(64, 10000.0)[0][:8].tolist() + W.rope_frequencies(128, 150000.0)[0][1:5].tolist()
             + [2.0 ** 20 + 0.37, 123456.789, -0.81, 6.2])
    mask = (1 << BITS) - 1
    rows = []  # (pair, position, 0 for the cosine or 1 for the sine, signed distance in turns)
    for j, f in enumerate(freqs):
        step = int(Fraction(f) * inverse)  # exact to 2^-BITS turns and a bit
        near = []
        for pos in range(top - 30000, top + 1):
            quarters, rest = divmod(4 * ((pos * step) & mask) + (1 << (BITS - 1)), 1 << BITS)
            near.append((abs(rest - (1 << (BITS - 1))), pos, quarters & 3, rest - (1 << (BITS - 1))))
        near.sort()
        rows += [(j, pos, quarter, Fraction(d, 4 << BITS)) for _, pos, quarter, d in near[:6]]
    n, half = len(rows), len(freqs)
    x = torch.zeros(n, 1, 2 * half, dtype=torch.float16)
    for r, (j, *_) in enumerate(rows):
        x[r, 0, j] = 1024.0
    pos = torch.tensor([p for _, p, *_ in rows], dtype=torch.int32)
    out = pkg.gqa_rope(x.cuda(), pos.cuda(), torch.tensor(freqs, dtype=torch.float64).cuda(), torch.empty_like(x, device="cuda"))
    status_ok(pkg)
    out = out.cpu().double()
    for r, (j, p, quarter, d) in enumerate(rows):
        s, c = math.sin(2 * math.pi * float(d)), math.cos(2 * math.pi * float(d))
        cos, sin = [(c, s), (-s, c), (-c, -s), (s, -c)][quarter]
        for got, want in ((out[r, 0, j], 1024 * cos), (out[r, 0, half + j], 1024 * sin)):
            tol = (2.0 ** -11 + 2.0 ** -20) * abs(want) + 1024 * 2 * math.pi * 1.5 * 2.0 ** -32
            assert abs(float(got) - want) <= tol, (freqs[j], p, float(got), want, tol)


@pytest.mark.parametrize("kind", ["16", "e4m3"])
@pytest.mark.parametrize("new,pad", [([3, 1], 5), ([700, 300], 200)])
def test_rows_without_a_place_change_nothing(pkg, new, pad, kind):  # noqa: F811
    """Rows behind the last sequence, and rows whose page is outside the pool:
    neither the pool nor q_out changes there; the others are as without them."""
    pre, hq, hkv, d, page = [20, 9], 6, 2, 64, 16
    used, total = sum(new), sum(new) + pad
    packed = rand(total, hq + 2 * hkv, d, seed=total, dtype=torch.bfloat16).cuda()
    q, k, v = packed.split([hq, hkv, hkv], 1)
    inv = W.rope_frequencies(64)[0].cuda()
    cu = torch.tensor([0, new[0], used], dtype=torch.int32, device="cuda")
    lens = torch.tensor(pre, dtype=torch.int32, device="cuda")
    runs = []
    for rows, bad in ((used, False), (total, False), (total, True)):
        cache = R.on_gpu(R.fill(W.empty_cache([p + n for p, n in zip(pre, new)], hkv, d, page, "bf16", kind), None, 5))
        table = cache.page_indices.clone()
        if bad:  # the last page of sequence 1
            table[-1] = cache.k_pages.shape[0] + 3
        q_out = torch.full((rows, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
        pkg.gqa_cache_write(k[:rows], v[:rows], cu, lens, cache.page_indptr, table, cache.k_pages, cache.v_pages,
                            k_scales=cache.k_scales, v_scales=cache.v_scales, rope=pkg.Rope(inv, q=q[:rows], q_out=q_out))
        torch.cuda.synchronize()
        assert pkg.get_device_status() == (pkg.GQA_DEV_BAD_METADATA if bad else 0)
        runs.append((q_out, [t.view(torch.uint8) for t in (cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales)
                             if t is not None], cache))
    (plain, pools, _), (padded, padded_pools, _), (broken, broken_pools, cache) = runs
    assert torch.equal(padded[:used], plain) and bool((padded[used:] == 7).all())
    assert all(torch.equal(a, b) for a, b in zip(padded_pools, pools))
    lost = (pre[1] + new[1] - 1) % page + 1  # keys on the last page
    lost = min(lost, new[1])
    assert torch.equal(broken[:used - lost], plain[:used - lost]) and bool((broken[used - lost:] == 7).all())
    before = R.on_gpu(R.fill(W.empty_cache([p + n for p, n in zip(pre, new)], hkv, d, page, "bf16", kind), None, 5))
    last = int(before.page_indices[-1])
    rest = [i for i in range(before.k_pages.shape[0]) if i != last]
    for name, a, b in zip(("k_pages", "v_pages", "k_scales", "v_scales"), broken_pools, pools):
        old = getattr(before, name).view(torch.uint8)
        assert torch.equal(a[rest], b[rest]) and torch.equal(a[last], old[last])
