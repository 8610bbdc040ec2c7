"""f16: rows whose dout is far below the largest of their own sequence lose nothing of dq, nor do tiles of keys
that only such rows see of dk and dv."""
import math

import pytest
import torch

import grad_util as R
from test_backward_gpu import batch, dout_of
from test_cache_gpu import pkg  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("below", [2.0 ** -12, 2.0 ** -17, 2.0 ** -20])
@pytest.mark.parametrize("pre,new,hq,hkv,d,window", [(0, 600, 8, 2, 64, 0), (0, 100, 2, 1, 64, 0), (0, 1500, 4, 1, 128, 0),
                                                     (300, 700, 4, 2, 128, 100), (0, 390, 2, 2, 128, 0), (40, 800, 2, 1, 256, 0),
                                                     (0, 500, 4, 4, 256, 64), (2500, 300, 8, 1, 64, 0)])
def test_small_rows_beside_large_ones(pkg, pre, new, hq, hkv, d, window, below):  # noqa: F811
    """Every 29th token of the first third has a dout 2^9, all others `below` times that.  Over the small rows' dq, and the dk and
    dv of the tiles of 128 keys whose query tiles are small rows alone, the error's norm is the results' own rounding (of values
    that may be subnormal), u / sqrt(3) of each term in the mean square where p and ds are held in one term (see
    test_one_term_costs_one_rounding), and the 2^-14 of the fp32 sums; 5% for the draw where 10^5 pairs and more are rounded,
    15% in the smaller calls."""
    b = batch([pre], [new], hq, hkv, d, "f16", window, "head")
    g = hq // hkv
    large = torch.zeros(new, dtype=torch.bool, device="cuda")
    large[:new // 3:29] = True
    last = int(large.nonzero().max())
    tail = min([a for a in range(0, pre + new, 128) if max(a - pre, 0) * g // 128 * 128 // g > last], default=pre + new)
    assert tail < pre + new or new < 200 or pre > 2000
    dout = dout_of(b, dtype=torch.float32)
    dout = (dout * torch.where(large, 512.0, 512.0 * below)[:, None, None]).half()
    out, lse = pkg.prefill(b)
    got = pkg.prefill_backward(b, out, lse, dout)
    torch.cuda.synchronize()
    assert pkg.get_device_status() == 0
    want, bounds = R.gradients(b, out, lse, dout)
    R.check(got, want, bounds)
    u, terms, keep = 2.0 ** -11, [0.0, 0.0, 0.0], R.visible(b, 0)
    for h in range(hq):
        q, do, o, k, v = (x.double() for x in (b.q[:, h], dout[:, h], out[:, h], b.k[:, h * hkv // hq], b.v[:, h * hkv // hq]))
        p = torch.exp(q @ k.T * b.scale - lse[:, h, None].double()).masked_fill(~keep, 0.0)
        ds = p * (do @ v.T - (do * o).sum(1)[:, None]) * b.scale
        terms[0] += float((ds[~large] ** 2 @ (k ** 2).sum(1)).sum())
        terms[1] += float(((ds ** 2).T @ (q ** 2).sum(1))[tail:].sum())
        terms[2] += float(((p ** 2).T @ (do ** 2).sum(1))[tail:].sum())
    one = new * g * (min(pre + new, window) if window else pre + new) > 2 ** 19
    for x, y, t in ((got[0][~large], want[0][~large], terms[0]), (got[1][tail:], want[1][tail:], terms[1]),
                    (got[2][tail:], want[2][tail:], terms[2])):
        if y.numel() == 0:
            continue
        own = float((y.half().double() - y).norm())
        room = 1.05 if one else 1.15
        assert float((x.double() - y).norm()) <= room * math.sqrt(own ** 2 + one * u ** 2 / 3 * t) + 2.0 ** -14 * float(y.norm())
