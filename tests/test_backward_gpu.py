"""The attention's gradient on the GPU against its formula in 64 bits."""
import pytest
import torch

import grad_util as R
from gqa_flash_attention_prefill_gb300 import workloads as W
from test_cache_gpu import pkg  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def batch(pre, new, hq, hkv, d, dtype="bf16", window=0, sink="none", seed=0, scale=None):
    return W.make_batch(pre, new, hq, hkv, d, dtype, window=window, sink_mode=sink, seed=seed, scale=scale).to("cuda")


def dout_of(b, seed=1, dtype=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(b.q.shape, generator=gen, device="cuda").to(dtype or b.q.dtype)


def run(pkg, b, dout=None, dlse=None):  # noqa: F811
    """Against the formula on the forward's own out and lse."""
    out, lse = pkg.prefill(b)
    dout = dout_of(b) if dout is None else dout
    got = pkg.prefill_backward(b, out, lse, dout, dlse=dlse)
    torch.cuda.synchronize()
    assert pkg.get_device_status() == 0
    R.check(got, *R.gradients(b, out, lse, dout, dlse))
    return out, lse, dout, got


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (8, 1, 64), (16, 2, 64), (6, 3, 128), (8, 2, 128), (4, 2, 256),
                                      (128, 1, 64), (128, 1, 256), (32, 1, 128)])
def test_heads(pkg, hq, hkv, d, dtype):  # noqa: F811
    run(pkg, batch([0, 3], [70, 131], hq, hkv, d, dtype, sink="head"))


@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (128, 4, 4), (256, 2, 1)])
@pytest.mark.parametrize("pre,new", [([0], [1]), ([5], [1]), ([0], [2]), ([127], [1]), ([128], [1]), ([0], [127]),
                                     ([0], [128]), ([0], [129]), ([0], [257]), ([300], [31]), ([1, 0, 129], [16, 15, 17]),
                                     ([0, 7, 0, 0, 2], [0, 0, 33, 0, 64])])
def test_lengths(pkg, pre, new, d, hq, hkv):  # noqa: F811
    run(pkg, batch(pre, new, hq, hkv, d, "bf16", sink="smooth", seed=len(new)))


@pytest.mark.parametrize("d,hq,hkv,dtype", [(64, 8, 1, "bf16"), (128, 4, 2, "f16"), (256, 2, 2, "bf16")])
@pytest.mark.parametrize("window", [1, 2, 63, 64, 127, 128, 129, 400, 2**31 - 1])
def test_windows(pkg, window, d, hq, hkv, dtype):  # noqa: F811
    run(pkg, batch([0, 500, 90], [300, 140, 1], hq, hkv, d, dtype, window=window, sink="head"))


@pytest.mark.parametrize("sink", ["none", "smooth", "head"])
@pytest.mark.parametrize("with_dlse", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_sinks_and_lse(pkg, sink, with_dlse, d):  # noqa: F811
    b = batch([0, 20], [200, 90], 8, 2, d, "f16" if d == 128 else "bf16", sink=sink)
    dlse = torch.randn(b.q.shape[:2], device="cuda") if with_dlse else None
    run(pkg, b, dlse=dlse)


@pytest.mark.parametrize("pre,new,hq,hkv,d,dtype,window", [
    ([0], [1500], 16, 1, 64, "bf16", 0), ([0], [1100], 8, 1, 128, "f16", 0), ([6000], [40], 8, 1, 64, "f16", 0),
    ([3000, 0], [100, 900], 4, 1, 256, "bf16", 0), ([0], [4000], 8, 1, 64, "bf16", 128), ([2500], [700], 2, 2, 128, "bf16", 300)])
def test_cut_units(pkg, pre, new, hq, hkv, d, dtype, window):  # noqa: F811
    """Few KV heads and long sequences: units are cut and joined."""
    run(pkg, batch(pre, new, hq, hkv, d, dtype, window, "head"))


def test_many_sequences(pkg):  # noqa: F811
    new = [(7 * i) % 23 for i in range(1500)]
    pre = [(5 * i) % 11 for i in range(1500)]
    run(pkg, batch(pre, new, 4, 2, 64, "bf16", sink="head"))


@pytest.mark.parametrize("d,dtype,scale", [(64, "f16", 1e-6), (64, "f16", 3e3), (128, "f16", 1e-6), (256, "f16", 30.0),
                                           (64, "bf16", 1e-20), (128, "bf16", 1e15)])
def test_sizes_of_dout(pkg, d, dtype, scale):  # noqa: F811
    """Gradients far from 1, in both directions: nothing is lost of dk, dq beyond the type's own range."""
    b = batch([0], [260], 4, 2, d, dtype, sink="head")
    run(pkg, b, dout=(dout_of(b, dtype=torch.float32) * scale).to(b.q.dtype))


def test_one_sequence_does_not_coarsen_another(pkg):  # noqa: F811
    """f16: the power of two that ds is held with is each sequence's and KV head's own."""
    b = batch([0, 0], [150, 150], 4, 2, 64, "f16")
    dout = dout_of(b)
    dout[:150] *= 1000.0
    dout[150:] *= 2.0 ** -14
    run(pkg, b, dout=dout)


def test_true_gradient(pkg):  # noqa: F811
    """Against the gradient of the attention itself in 64 bits: out's own rounding enters D."""
    for d, dtype, window in ((64, "bf16", 0), (128, "f16", 40), (256, "bf16", 0)):
        b = batch([0, 30], [130, 65], 8, 2, d, dtype, window, "head")
        out, lse = pkg.prefill(b)
        dout = dout_of(b)
        got = pkg.prefill_backward(b, out, lse, dout)
        o, le = R.forward(b)
        # prefill rounds p and out once to the type (2 u), and lse is good to 2^-20 of its size at these lengths
        u = torch.finfo(b.q.dtype).eps / 2
        want, bounds = R.gradients(b, o, le, dout, out_error=2 * u + float((o - out.double()).abs().max() / o.abs().max()))
        R.check(got, want, bounds)


def outside(pkg, b, junk):  # noqa: F811
    """The batch inside larger tensors whose other rows hold `junk`; returns (batch, out, lse, dout)."""
    out, lse = pkg.prefill(b)
    dout = dout_of(b)
    wide = lambda x, lo: torch.cat([torch.full((lo, *x.shape[1:]), junk, dtype=x.dtype, device="cuda"), x,  # noqa: E731
                                    torch.full((70, *x.shape[1:]), junk, dtype=x.dtype, device="cuda")])
    w = W.Batch(wide(b.q, 0), wide(b.k, 9), wide(b.v, 9), b.cu_seqlens_q, b.prefix_lens, b.kv_indptr + 9, b.hq, b.hkv, b.d,
                b.window, b.sinks, b.smooth, b.scale, "", dict(b.meta))
    return w, wide(out, 0), wide(lse, 0), wide(dout, 0)


@pytest.mark.parametrize("d,hq,hkv,dtype", [(64, 8, 1, "bf16"), (128, 4, 2, "f16"), (256, 2, 2, "bf16")])
def test_rows_outside(pkg, d, hq, hkv, dtype):  # noqa: F811
    """Rows of no sequence may hold NaN, are not written, and change nothing."""
    b = batch([0, 13, 0], [100, 37, 203], hq, hkv, d, dtype, sink="head")
    w, out, lse, dout = outside(pkg, b, float("nan"))
    mark = [torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda") for x in (w.q, w.k, w.v)]
    dsinks = torch.empty(hq, device="cuda")
    ws = torch.empty(pkg.prefill_backward_workspace(3, w.total_q, w.total_kv, hq, hkv, d, dtype), dtype=torch.uint8, device="cuda")
    pkg.gqa_prefill_backward(w.q, w.k, w.v, w.cu_seqlens_q, w.prefix_lens, w.kv_indptr, w.scale, out, lse, dout, *mark, ws,
                             sinks=w.sinks, dsinks=dsinks)
    torch.cuda.synchronize()
    assert pkg.get_device_status() == 0
    want, bounds = R.gradients(w, out, lse, dout)
    R.check([*mark, dsinks], want, bounds)
    for x, y in zip(mark, want):
        assert bool((x[y.isnan()] == 7.0).all())


def test_no_tokens(pkg):  # noqa: F811
    """Sequences without new tokens: their prefix's gradient is zero, the sinks' too."""
    b = batch([40, 0, 200], [0, 0, 0], 8, 2, 64, "bf16", sink="head")
    out, lse = torch.empty_like(b.q), torch.empty(0, 8, device="cuda")
    dq, dk, dv, dsinks = pkg.prefill_backward(b, out, lse, torch.empty_like(b.q))
    assert dq.shape[0] == 0 and not dk.any() and not dv.any() and not dsinks.any()
    none = batch([], [], 8, 2, 64, "bf16", sink="head")
    assert not pkg.prefill_backward(none, out, lse, torch.empty_like(b.q))[3].any()
    assert pkg.get_device_status() == 0


def test_same_bits(pkg):  # noqa: F811
    """The same run to run, and whatever the workspace held."""
    b = batch([700, 0], [300, 1100], 8, 1, 64, "bf16", sink="head")
    out, lse = pkg.prefill(b)
    dout = dout_of(b)
    size = pkg.prefill_backward_workspace(2, b.total_q, b.total_kv, 8, 1, 64, "bf16")
    first = None
    for fill in (0, 255, 85):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        got = [x.clone() for x in pkg.prefill_backward(b, out, lse, dout, workspace=ws)]
        first = first or got
        assert all(torch.equal(x, y) for x, y in zip(got, first))


def test_bad_metadata(pkg):  # noqa: F811
    """Nothing is written, and the status word says so."""
    b = batch([10, 0], [20, 30], 4, 2, 64, "bf16", sink="head")
    out, lse = pkg.prefill(b)
    dout = dout_of(b)
    ws = torch.empty(pkg.prefill_backward_workspace(2, 50, 60, 4, 2, 64, "bf16"), dtype=torch.uint8, device="cuda")
    for name, value in (("cu_seqlens_q", [0, 20, 51]), ("cu_seqlens_q", [0, 60, 50]), ("cu_seqlens_q", [1, 20, 50]),
                        ("prefix_lens", [11, 0]), ("prefix_lens", [-1, 0]), ("kv_indptr", [0, 30, 61]), ("kv_indptr", [-1, 30, 60])):
        m = {n: getattr(b, n) for n in ("cu_seqlens_q", "prefix_lens", "kv_indptr")}
        m[name] = torch.tensor(value, dtype=torch.int32, device="cuda")
        res = [torch.full_like(x, 3.0) for x in (b.q, b.k, b.v, b.sinks)]
        pkg.gqa_prefill_backward(b.q, b.k, b.v, m["cu_seqlens_q"], m["prefix_lens"], m["kv_indptr"], b.scale, out, lse, dout,
                                 *res[:3], ws, sinks=b.sinks, dsinks=res[3])
        torch.cuda.synchronize()
        assert pkg.get_device_status() == pkg.GQA_DEV_BAD_METADATA, (name, value)
        assert all(bool((x == 3.0).all()) for x in res)


def test_graphs_and_streams(pkg):  # noqa: F811
    """Two captured calls on workspaces of their own, replayed at once on two streams over new values."""
    calls = []
    for i, (d, dtype) in enumerate(((64, "bf16"), (128, "f16"))):
        b = batch([0, 100], [400, 77], 8, 2, d, dtype, sink="head", seed=i)
        out, lse = pkg.prefill(b)
        dout = dout_of(b)
        res = [torch.empty_like(x) for x in (b.q, b.k, b.v, b.sinks)]
        ws = torch.empty(pkg.prefill_backward_workspace(2, b.total_q, b.total_kv, 8, 2, d, dtype), dtype=torch.uint8, device="cuda")
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            pkg.gqa_prefill_backward(b.q, b.k, b.v, b.cu_seqlens_q, b.prefix_lens, b.kv_indptr, b.scale, out, lse, dout,
                                     *res[:3], ws, sinks=b.sinks, dsinks=res[3])
        calls.append((ws, b, out, lse, dout, res, stream, graph))  # what a graph points to stays alive
    for round_ in range(3):
        for _, b, out, lse, dout, res, stream, graph in calls:
            dout.copy_(dout_of(b, 10 + round_))
        torch.cuda.synchronize()
        for *_, stream, graph in calls:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for _, b, out, lse, dout, res, stream, graph in calls:
            R.check(res, *R.gradients(b, out, lse, dout))
    assert pkg.get_device_status() == 0


def test_memory_of_a_call_on_another_stream(pkg):  # noqa: F811
    b = batch([0], [500], 8, 2, 64, "bf16", sink="head")
    out, lse = pkg.prefill(b)
    dout = dout_of(b)
    want = [t.clone() for t in pkg.prefill_backward(b, out, lse, dout)]
    torch.cuda.synchronize()
    size = pkg.prefill_backward_workspace(1, 500, 500, 8, 2, 64, "bf16")
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        torch.cuda._sleep(20_000_000)
    got = pkg.prefill_backward(b, out, lse, dout, stream=other)
    blocks = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
              for n in [size] + [t.numel() * t.element_size() for t in got] * 2]
    other.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert all(bool((x == 255).all()) for x in blocks)


def test_offsets_past_32_bits(pkg):  # noqa: F811
    """A short sequence behind a long one, past 2^31 values of q: the rows of a call of its own."""
    long, pre, new, hq, hkv, d = 2 ** 18, 30, 90, 64, 2, 128
    b = W.make_batch([0, pre], [long, new], hq, hkv, d, "bf16", window=40, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    dout = torch.randn(b.q.shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    out, lse = pkg.prefill(b)
    got = pkg.prefill_backward(b, out, lse, dout)
    tail = batch([pre], [new], hq, hkv, d, "bf16", window=40, sink="head")
    tail.q, tail.k, tail.v, tail.sinks = b.q[long:].clone(), b.k[long:].clone(), b.v[long:].clone(), b.sinks
    assert long * hq * d >= 2 ** 31 and len(tail.k) == pre + new
    want, bounds = R.gradients(tail, out[long:], lse[long:], dout[long:])
    torch.cuda.synchronize()
    assert pkg.get_device_status() == 0
    R.check([got[0][long:], got[1][long:], got[2][long:]], want[:3], bounds[:3])
    assert bool(torch.stack([x.isfinite().all() for x in got]).all())


@pytest.mark.parametrize("pre,new,hq,hkv,d,dtype,window", [([0], [2], 2, 2, 128, "bf16", 0), ([34, 2], [3, 8], 2, 1, 256, "bf16", 128),
                                                           ([89], [2], 4, 4, 64, "f16", 0), ([0, 2966], [102, 14], 2, 1, 64, "bf16", 0),
                                                           ([0], [83], 1, 1, 64, "f16", 0), ([5112, 0], [36, 3], 4, 4, 64, "bf16", 128),
                                                           ([0, 0], [3, 2], 8, 2, 64, "f16", 128), ([0], [27], 2, 2, 256, "f16", 0)])
def test_small_calls_lose_nothing_to_p_and_ds(pkg, pre, new, hq, hkv, d, dtype, window):  # noqa: F811
    """Over a few rows an error is not averaged away, so P and dS are held in two terms: off by 2^-17 (bf16) at most.  With
    that, fp32 sums of d products ((d + 3) f of some 5 times the score) and the exponential a result is off by 2^-14 of
    its norm, beside its own rounding."""
    b = batch(pre, new, hq, hkv, d, dtype, window=window, sink="head")
    out, lse, dout, got = run(pkg, b)
    want, _ = R.gradients(b, out, lse, dout)
    for x, y in zip(got[:3], want[:3]):
        own = (y.to(b.q.dtype).double() - y).norm()
        assert float((x.double() - y).norm()) <= float(own) + 2.0 ** -14 * float(y.norm())
