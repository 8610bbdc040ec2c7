"""The gradient's formula against differences of the forward pass, in 64 bits,
and what gqa_prefill_backward refuses before any launch."""
import ctypes

import pytest
import torch

import grad_util as R
from gqa_flash_attention_prefill_gb300 import workloads as W

FAKE = 1 << 20  # a 256-byte-aligned non-null address; never dereferenced
STEP = 1 << 24  # between tensors, so that none overlaps another


@pytest.fixture(scope="module")
def lib():
    from gqa_flash_attention_prefill_gb300 import build
    import gqa_flash_attention_prefill_gb300 as pkg
    return pkg.load(build.build())


@pytest.mark.parametrize("sink", ["none", "smooth", "head"])
@pytest.mark.parametrize("window", [0, 3])
def test_formula_against_differences(sink, window):
    """Central differences of L = <dout, out> + <dlse, lse>: their own error is the third derivative's, h^2 = 1e-10."""
    b = W.make_batch([0, 4], [6, 3], 4, 2, 8, "f16", window=window, sink_mode=sink, seed=3)
    b.q, b.k, b.v = b.q.double(), b.k.double(), b.v.double()
    b.sinks = None if b.sinks is None else b.sinks.double()
    gen = torch.Generator().manual_seed(5)
    dout = torch.randn(b.q.shape, generator=gen, dtype=torch.float64)
    dlse = torch.randn(b.q.shape[:2], generator=gen, dtype=torch.float64)
    out, lse = R.forward(b)
    want, _ = R.gradients(b, out, lse, dout, dlse)

    def loss():
        o, le = R.forward(b)
        return float((dout * o).sum() + (dlse * le).sum())

    h = 1e-5
    for x, grad in zip((b.q, b.k, b.v, b.sinks), want):
        if x is None:
            continue
        flat = x.view(-1)
        for i in torch.randperm(flat.numel(), generator=gen)[:12].tolist():
            keep = float(flat[i])
            flat[i] = keep + h
            up = loss()
            flat[i] = keep - h
            down = loss()
            flat[i] = keep
            assert abs((up - down) / (2 * h) - float(grad.view(-1)[i])) < 1e-7


def call(lib, **over):
    a = dict(q=FAKE, k=FAKE + STEP, v=FAKE + 2 * STEP, cu=FAKE + 3 * STEP, pre=FAKE + 4 * STEP, kvi=FAKE + 5 * STEP, B=1, total_q=16,
             total_kv=16, hq=8, hkv=2, d=64, dtype=1, scale=0.125, window=0, out=FAKE + 6 * STEP, lse=FAKE + 7 * STEP,
             dout=FAKE + 8 * STEP, dlse=None, sinks=None, dq=FAKE + 9 * STEP, dk=FAKE + 10 * STEP, dv=FAKE + 11 * STEP, dsinks=None,
             ws=FAKE + 12 * STEP, size=1 << 40, stream=None)
    a.update(over)
    return lib.gqa_prefill_backward(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), -1), (dict(total_q=-1), -1), (dict(total_kv=-1), -1), (dict(hq=7), -1), (dict(hkv=0), -1), (dict(d=0), -1),
    (dict(dtype=2), -1), (dict(scale=0.0), -1), (dict(scale=float("inf")), -1), (dict(scale=float("nan")), -1),
    (dict(sinks=FAKE + 13 * STEP), -1), (dict(dsinks=FAKE + 13 * STEP), -1), (dict(cu=None), -1), (dict(pre=None), -1),
    (dict(kvi=None), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(out=None), -1), (dict(lse=None), -1),
    (dict(dout=None), -1), (dict(dq=None), -1), (dict(dk=None), -1), (dict(dv=None), -1), (dict(total_kv=0), -1),
    (dict(q=FAKE + 8), -1), (dict(dout=FAKE + 8 * STEP + 4), -1), (dict(dk=FAKE + 10 * STEP + 2), -1), (dict(lse=FAKE + 7 * STEP + 2), -1),
    (dict(ws=None), -1), (dict(size=1000), -1), (dict(ws=FAKE + 12 * STEP + 16), -1),
    (dict(dq=FAKE), -1), (dict(dq=FAKE + 8 * STEP), -1), (dict(dk=FAKE + STEP), -1), (dict(dv=FAKE + 10 * STEP + 256), -1),
    (dict(dk=FAKE + 6 * STEP + 64), -1), (dict(ws=FAKE + 2 * STEP), -1),
    (dict(sinks=FAKE + 13 * STEP, dsinks=FAKE + 13 * STEP), -1),
    (dict(d=96), -2), (dict(hq=12, hkv=4), -2), (dict(hq=256, hkv=1), -2), (dict(total_q=1 << 30, hq=8, hkv=8), -2),
    (dict(B=0, q=None), 0)])
def test_refusals(lib, over, code):
    assert call(lib, **over) == code


def test_workspace(lib):
    import gqa_flash_attention_prefill_gb300 as pkg
    small = pkg.prefill_backward_workspace(1, 10, 10, 8, 2, 64, "bf16")
    large = pkg.prefill_backward_workspace(5, 10000, 20000, 8, 2, 64, "bf16")
    assert 0 < small < large and small % 256 == 0
    assert pkg.prefill_backward_workspace(1, 10, 10, 8, 2, 64, torch.float16) >= small
    with pytest.raises(pkg.GQAError):
        pkg.prefill_backward_workspace(1, 10, 10, 8, 2, 80, "bf16")
    size = ctypes.c_size_t(0)
    assert lib.gqa_prefill_backward_workspace(1, 1, 1, 8, 2, 64, 1, None) == -1
    assert lib.gqa_prefill_backward_workspace(1, 1, 1, 8, 3, 64, 1, ctypes.byref(size)) == -1


def test_binding_refusals():
    import gqa_flash_attention_prefill_gb300 as pkg
    b = W.make_batch([0], [4], 4, 2, 64, "bf16")
    lse = torch.zeros(4, 4)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.gqa_prefill_backward(b.q, b.k, b.v, b.cu_seqlens_q, b.prefix_lens, b.kv_indptr, 0.1, b.q, lse, b.q, b.q, b.k, b.v, None)
    with pytest.raises(ValueError, match="float32"):
        pkg._float32((4, 4), lse=lse.double())
    with pytest.raises(ValueError, match="float32"):
        pkg._float32((4, 3), lse=lse)
