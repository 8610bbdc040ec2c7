"""The attention's gradient with P and dS in two 16-bit terms (sequences of few pairs) and in one (all others): which one a
sequence gets, that nothing but its own lengths and the window decide it, and the one-term form where it can go wrong."""
import math

import pytest
import torch

import grad_util as R
from gqa_flash_attention_prefill_gb300 import workloads as W
from test_backward_gpu import batch, dout_of, outside
from test_cache_gpu import pkg  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

LIMIT = 2 ** 19  # pairs of a KV head's query rows and the keys that one can see


def pairs(P, E, hq, hkv, window):
    return E * (hq // hkv) * (min(P + E, window) if window > 0 else P + E)


def backward(pkg, b, out, lse, dout, dlse=None, terms=None):  # noqa: F811
    """prefill_backward, and of the plan that its workspace holds afterwards the terms of each sequence's units."""
    size = pkg.prefill_backward_workspace(b.num_seqs, b.total_q, b.total_kv, b.hq, b.hkv, b.d, b.dtype_name)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    got = pkg.prefill_backward(b, out, lse, dout, dlse=dlse, workspace=ws)
    torch.cuda.synchronize()
    assert pkg.get_device_status() == 0
    words = ws[:-(size % 4) or None].view(torch.int32)
    units = words[64:64 + 16 * int(words[0])].view(-1, 16).cpu()  # 64 words of header, 16 a record
    seen = {}
    for kind, seq in zip(units[:, 0].tolist(), units[:, 12].tolist()):
        seen.setdefault(seq, set()).add(2 if kind & 4 else 1)
    for s in range(b.num_seqs):
        P, E = int(b.prefix_lens[s]), int(b.cu_seqlens_q[s + 1] - b.cu_seqlens_q[s])
        if P + E > 0:
            assert seen[s] == {2 if pairs(P, E, b.hq, b.hkv, b.window) <= LIMIT else 1}, (s, P, E)
    if terms is not None:
        assert set().union(*seen.values()) == {terms}
    return got


def run(pkg, b, dout=None, dlse=None, terms=1):  # noqa: F811
    out, lse = pkg.prefill(b)
    dout = dout_of(b) if dout is None else dout
    got = backward(pkg, b, out, lse, dout, dlse, terms)
    R.check(got, *R.gradients(b, out, lse, dout, dlse))
    return out, lse, dout, got


@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 64), (2, 2, 128), (4, 2, 256)])
def test_limit(pkg, hq, hkv, d):  # noqa: F811
    """Both sides of the limit, by a prefix key, beside one another."""
    E = 64
    keys = LIMIT // (E * hq // hkv)
    b = batch([keys - E, keys - E + 1, 0], [E, E, 9], hq, hkv, d, "bf16", sink="head")
    out, lse = pkg.prefill(b)
    dout = dout_of(b)
    R.check(backward(pkg, b, out, lse, dout), *R.gradients(b, out, lse, dout))


@pytest.mark.parametrize("pre,new,hq,hkv,d,dtype", [([0, 13, 0], [100, 37, 203], 8, 1, 64, "bf16"),
                                                    ([0, 20], [150, 41], 4, 2, 128, "f16"), ([5], [90], 2, 1, 256, "bf16")])
@pytest.mark.parametrize("junk", [1, 500, 40000])
def test_rows_outside_change_no_bit(pkg, pre, new, hq, hkv, d, dtype, junk):  # noqa: F811
    """However many rows stand behind the last sequence, and whatever they hold."""
    b = batch(pre, new, hq, hkv, d, dtype, sink="head")
    out, lse = pkg.prefill(b)
    dout = dout_of(b)
    want = pkg.prefill_backward(b, out, lse, dout)
    tail = lambda x: torch.cat([x, torch.full((junk, *x.shape[1:]), float("nan"), dtype=x.dtype, device="cuda")])  # noqa: E731
    w = W.Batch(tail(b.q), tail(b.k), tail(b.v), b.cu_seqlens_q, b.prefix_lens, b.kv_indptr, hq, hkv, d, b.window, b.sinks,
                b.smooth, b.scale, "", dict(b.meta))
    got = pkg.prefill_backward(w, tail(out), tail(lse), tail(dout))
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x[:len(y)], y)


@pytest.mark.parametrize("hq,hkv,d,dtype", [(8, 2, 64, "bf16"), (4, 1, 128, "f16"), (2, 1, 256, "bf16")])
def test_company_changes_no_bit(pkg, hq, hkv, d, dtype):  # noqa: F811
    """A few tokens have the bits, and so the accuracy, that they have in a call of their own: beside a long sequence the
    error of theirs is still their own rounding and 2^-14 (the bound of the calls of few tokens alone)."""
    long = 1500
    for few, behind in ((3, 0), (40, 7), (1, 300)):
        b = batch([0, behind], [long, few], hq, hkv, d, dtype, sink="head")
        out, lse = pkg.prefill(b)
        dout = dout_of(b)
        got = backward(pkg, b, out, lse, dout)
        own = W.Batch(b.q[long:].clone(), b.k[long:].clone(), b.v[long:].clone(), b.cu_seqlens_q[1:] - long, b.prefix_lens[1:],
                      b.kv_indptr[1:] - long, hq, hkv, d, b.window, b.sinks, b.smooth, b.scale, "", dict(b.meta))
        alone = backward(pkg, own, out[long:], lse[long:], dout[long:].contiguous(), terms=2)
        want, _ = R.gradients(own, out[long:], lse[long:], dout[long:])
        for x, y, z in zip(got[:3], alone, want):
            assert torch.equal(x[long:], y)
            off = float((y.double() - z).norm())
            assert off <= float((z.to(y.dtype).double() - z).norm()) + 2.0 ** -14 * float(z.norm())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv,d", [(16, 1, 64), (8, 4, 128), (4, 4, 256), (128, 1, 64), (64, 1, 128), (32, 1, 256)])
def test_heads(pkg, hq, hkv, d, dtype):  # noqa: F811
    g = hq // hkv
    n = math.isqrt(LIMIT // g) + 2
    run(pkg, batch([0, 37], [n, n], hq, hkv, d, dtype, sink="head"))


@pytest.mark.parametrize("d,hq,hkv,dtype", [(64, 16, 1, "bf16"), (128, 16, 1, "f16"), (256, 16, 1, "bf16")])
@pytest.mark.parametrize("window", [63, 64, 65, 127, 128, 129, 400])
def test_windows(pkg, window, d, hq, hkv, dtype):  # noqa: F811
    n = max(LIMIT // (16 * window) + 5, math.isqrt(LIMIT // 16) + 2)
    run(pkg, batch([0, 150], [n, n], hq, hkv, d, dtype, window=window, sink="head"))


@pytest.mark.parametrize("sink", ["none", "smooth", "head"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_sinks_and_lse(pkg, sink, d):  # noqa: F811
    b = batch([0, 20], [370, 410], 8, 2, d, "f16" if d == 128 else "bf16", sink=sink)
    run(pkg, b, dlse=torch.randn(b.q.shape[:2], device="cuda"))


@pytest.mark.parametrize("d,dtype,scale", [(64, "f16", 1e-6), (64, "f16", 3e3), (128, "f16", 1e-6), (256, "f16", 30.0),
                                           (64, "bf16", 1e-20), (128, "bf16", 1e15), (256, "bf16", 1e-20)])
def test_sizes_of_dout(pkg, d, dtype, scale):  # noqa: F811
    b = batch([0], [520], 4, 2, d, dtype, sink="head")
    run(pkg, b, dout=(dout_of(b, dtype=torch.float32) * scale).to(b.q.dtype))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_one_sequence_does_not_coarsen_another(pkg, d):  # noqa: F811
    """f16: the power of two that ds is held with is each sequence's and KV head's own."""
    b = batch([0, 0], [520, 520], 4, 2, d, "f16")
    dout = dout_of(b)
    dout[:520] *= 1000.0
    dout[520:] *= 2.0 ** -14
    run(pkg, b, dout=dout)


@pytest.mark.parametrize("d,window,dtype", [(64, 0, "bf16"), (128, 400, "f16"), (256, 0, "bf16")])
def test_true_gradient(pkg, d, window, dtype):  # noqa: F811
    """Against the gradient of the attention itself in 64 bits: out's own rounding enters D."""
    b = batch([0, 30], [365, 420], 8, 2, d, dtype, window, "head")
    out, lse = pkg.prefill(b)
    dout = dout_of(b)
    got = backward(pkg, b, out, lse, dout, terms=1)
    o, le = R.forward(b)
    # prefill rounds p and out once to the type (2 u), and lse is good to 2^-20 of its size at these lengths
    u = torch.finfo(b.q.dtype).eps / 2
    want, bounds = R.gradients(b, o, le, dout, out_error=2 * u + float((o - out.double()).abs().max() / o.abs().max()))
    R.check(got, want, bounds)


@pytest.mark.parametrize("d,hq,hkv,dtype", [(64, 8, 1, "bf16"), (128, 4, 2, "f16"), (256, 2, 2, "bf16")])
def test_rows_outside(pkg, d, hq, hkv, dtype):  # noqa: F811
    """Rows of no sequence may hold NaN and are not written, behind long sequences too."""
    n = math.isqrt(LIMIT * hkv // hq) + 1
    b = batch([0, 13], [n, n + 38], hq, hkv, d, dtype, sink="head")
    w, out, lse, dout = outside(pkg, b, float("nan"))
    mark = [torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda") for x in (w.q, w.k, w.v)]
    dsinks = torch.empty(hq, device="cuda")
    ws = torch.empty(pkg.prefill_backward_workspace(2, w.total_q, w.total_kv, hq, hkv, d, dtype), dtype=torch.uint8, device="cuda")
    pkg.gqa_prefill_backward(w.q, w.k, w.v, w.cu_seqlens_q, w.prefix_lens, w.kv_indptr, w.scale, out, lse, dout, *mark, ws,
                             sinks=w.sinks, dsinks=dsinks)
    torch.cuda.synchronize()
    assert pkg.get_device_status() == 0
    want, bounds = R.gradients(w, out, lse, dout)
    R.check([*mark, dsinks], want, bounds)
    for x, y in zip(mark, want):
        assert bool((x[y.isnan()] == 7.0).all())


@pytest.mark.parametrize("spread", [1.0, 8.0])
@pytest.mark.parametrize("pre,new,hq,hkv,d,dtype,window", [([0], [1500], 8, 1, 64, "bf16", 0), ([0], [1500], 8, 1, 64, "f16", 0),
                                                           ([900], [600], 4, 2, 128, "bf16", 0), ([0], [1100], 4, 1, 128, "f16", 0),
                                                           ([0], [900], 2, 1, 256, "bf16", 0), ([0], [900], 2, 1, 256, "f16", 300),
                                                           ([3000], [700], 8, 1, 64, "bf16", 128)])
def test_one_term_costs_one_rounding(pkg, pre, new, hq, hkv, d, dtype, window, spread):  # noqa: F811
    """The error's norm, not each element's bound: a result is a sum of terms p dout, ds k or ds q, whose p and ds are off by
    u / sqrt(3) of themselves in the mean square at most (a rounding's error is even over a step of 2 u times the power of two
    below), independently; so its square is that of the results' own rounding, and u^2 / 3 of the sum of the terms' squares.
    Beside it the 2^-14 of the fp32 sums and the exponential, and 5% for the draw: over 5 x 10^5 roundings and more it is below
    2% where every row has a term of its own.  One bit of P or dS lost would be u^2 4 / 3: over the bound.
    `spread` times the scores' spread: rows that one or two p make up."""
    b = batch(pre, new, hq, hkv, d, dtype, window=window, sink="head")
    b.q = (b.q * spread).to(b.q.dtype)
    out, lse, dout, got = run(pkg, b)
    want, _ = R.gradients(b, out, lse, dout)
    u = torch.finfo(b.q.dtype).eps / 2
    keep = R.visible(b, 0)
    terms = [0.0, 0.0, 0.0]
    for h in range(hq):
        q, do, o, k, v = (x.double() for x in (b.q[:, h], dout[:, h], out[:, h], b.k[:, h * hkv // hq], b.v[:, h * hkv // hq]))
        p = torch.exp(q @ k.T * b.scale - lse[:, h, None].double()).masked_fill(~keep, 0.0)
        ds = p * (do @ v.T - (do * o).sum(1)[:, None]) * b.scale
        terms[0] += float((ds ** 2 @ (k ** 2).sum(1)).sum())
        terms[1] += float(((ds ** 2).T @ (q ** 2).sum(1)).sum())
        terms[2] += float(((p ** 2).T @ (do ** 2).sum(1)).sum())
    for x, y, t in zip(got[:3], want, terms):
        own = float((y.to(x.dtype).double() - y).norm())
        assert float((x.double() - y).norm()) <= 1.05 * math.sqrt(own ** 2 + u ** 2 / 3 * t) + 2.0 ** -14 * float(y.norm())
