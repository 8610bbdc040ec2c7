"""What the norm and its gradient refuse before any launch."""
import ctypes

import pytest
import torch

FAKE = 1 << 20  # a 256-byte-aligned non-null address; never dereferenced
STEP = 1 << 28  # between tensors, so that none overlaps another


@pytest.fixture(scope="module")
def lib():
    from gqa_flash_attention_prefill_gb300 import build
    import gqa_flash_attention_prefill_gb300 as pkg
    return pkg.load(build.build())


def norm(lib, **over):
    a = dict(x=FAKE, xs=256, res=FAKE + STEP, h=FAKE + 2 * STEP, st=1, w=FAKE + 3 * STEP, wt=2, offset=0.0, eps=1e-5, rows=4, heads=1,
             n=256, dtype=1, kind=0, group=0, out=FAKE + 4 * STEP, os=256, scales=None, rstd=FAKE + 5 * STEP, stream=None)
    a.update(over)
    return lib.gqa_rms_norm(*a.values())


E4 = dict(kind=1, group=32, scales=FAKE + 6 * STEP)


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), -1), (dict(heads=0), -1), (dict(n=0), -1), (dict(dtype=2), -1), (dict(st=0), -1), (dict(wt=0), -1),
    (dict(st=3), -1), (dict(eps=0.0), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(offset=float("inf")), -1),
    (dict(kind=2), -1), (dict(E4, group=0), -1), (dict(E4, group=48), -1), (dict(E4, scales=None), -1),
    (dict(res=None), -1), (dict(h=None), -1), (dict(x=None), -1), (dict(w=None), -1), (dict(out=None), -1),
    (dict(x=FAKE + 8), -1), (dict(w=FAKE + 3 * STEP + 4), -1), (dict(out=FAKE + 4 * STEP + 2), -1), (dict(rstd=FAKE + 5 * STEP + 2), -1),
    (dict(xs=248), -1), (dict(xs=260), -1), (dict(os=128), -1),
    (dict(out=FAKE + 16), -1), (dict(out=FAKE, os=512), -1), (dict(h=FAKE + 16), -1), (dict(out=FAKE + 2 * STEP), -1),
    (dict(st=2, h=FAKE), -1), (dict(E4, out=FAKE), -1), (dict(E4, scales=FAKE + STEP), -1), (dict(rstd=FAKE + 4 * STEP), -1),
    (dict(out=FAKE + 3 * STEP), -1),
    (dict(n=12, xs=16, os=16), -2), (dict(n=16392, xs=16392, os=16392), -2), (dict(E4, group=16), -2), (dict(E4, group=8), -2),
    (dict(rows=1 << 30, heads=4, n=8, xs=32, os=32), -2),
    (dict(rows=0, x=None, w=None, out=None), 0)])
def test_norm_refusals(lib, over, code):
    assert norm(lib, **over) == code


def gradient(lib, **over):
    a = dict(dy=FAKE, ys=256, h=FAKE + STEP, hs=256, st=1, rstd=FAKE + 2 * STEP, w=FAKE + 3 * STEP, wt=1, offset=0.0, dh=FAKE + 4 * STEP,
             rows=4, heads=1, n=256, dtype=1, dx=FAKE + 5 * STEP, xs=256, dres=None, dw=FAKE + 6 * STEP, ws=FAKE + 7 * STEP,
             size=1 << 26, stream=None)
    a.update(over)
    return lib.gqa_rms_norm_backward(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), -1), (dict(heads=-1), -1), (dict(n=0), -1), (dict(dtype=5), -1), (dict(st=0), -1), (dict(wt=0), -1),
    (dict(offset=float("nan")), -1), (dict(dx=None, dw=None), -1), (dict(dy=None), -1), (dict(h=None), -1), (dict(rstd=None), -1),
    (dict(w=None), -1), (dict(ys=252), -1), (dict(hs=128), -1), (dict(xs=264 + 4), -1), (dict(dy=FAKE + 2), -1),
    (dict(dh=FAKE + 4 * STEP + 8), -1), (dict(dw=FAKE + 6 * STEP + 2), -1), (dict(ws=None), -1), (dict(ws=FAKE + 7 * STEP + 64), -1),
    (dict(size=256), -1), (dict(dx=FAKE + 32), -1), (dict(dx=FAKE, xs=512), -1), (dict(dres=FAKE + 5 * STEP), -1),
    (dict(dw=FAKE + 2 * STEP), -1), (dict(st=2, dx=FAKE + STEP), -1), (dict(ws=FAKE + 4 * STEP), -1),
    (dict(n=20, ys=24, hs=24, xs=24), -2), (dict(n=20000, ys=20000, hs=20000, xs=20000), -2),
    (dict(rows=0, dy=None, dw=None), 0)])
def test_gradient_refusals(lib, over, code):
    assert gradient(lib, **over) == code


def test_workspace(lib):
    import gqa_flash_attention_prefill_gb300 as pkg
    assert pkg.rms_norm_backward_workspace(4, 1, 4096, "bf16") >= 4 * 4096
    with pytest.raises(pkg.GQAError):
        pkg.rms_norm_backward_workspace(4, 1, 4097, "bf16")
    size = ctypes.c_size_t(0)
    assert lib.gqa_rms_norm_backward_workspace(4, 1, 64, 1, None) == -1
    assert lib.gqa_rms_norm_backward_workspace(-4, 1, 64, 1, ctypes.byref(size)) == -1


def test_binding_refusals():
    import gqa_flash_attention_prefill_gb300 as pkg
    x, w = torch.zeros(3, 64, dtype=torch.bfloat16), torch.zeros(64)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.gqa_rms_norm(x, w, x)
    with pytest.raises(ValueError, match="packed heads"):
        pkg._norm_rows("x", x.t())
    with pytest.raises(ValueError, match="shape of the rows"):
        pkg._norm_rows("out", x, (3, 1, 32))
    with pytest.raises(ValueError, match="one value per column"):
        pkg._norm_weight(w[:32], 64, x.dtype)
    with pytest.raises(TypeError, match="rows' type"):
        pkg._norm_weight(w.half(), 64, x.dtype)
    assert pkg._norm_weight(w, 64, x.dtype) == pkg.GQA_F32
    with pytest.raises(ValueError, match="contiguous"):
        pkg._norm_stream("residual", x.t(), (64, 1, 3))
    with pytest.raises(ValueError, match="rstd"):
        pkg._norm_rstd(w, 3, 1)
    # a slice of a packed projection: its stride is what is passed on
    assert pkg._norm_rows("x", torch.zeros(5, 8, 64)[:, 2:4]) == (5, 2, 64, 512)


def test_workspaces_refuse_other_types():
    import gqa_flash_attention_prefill_gb300 as pkg
    for dtype in (torch.float32, "f32", "float64"):
        with pytest.raises(TypeError, match="float16 or bfloat16"):
            pkg.rms_norm_backward_workspace(4, 1, 64, dtype)
        with pytest.raises(TypeError, match="float16 or bfloat16"):
            pkg.prefill_backward_workspace(1, 4, 4, 2, 1, 64, dtype)
    for names in (("bf16", torch.bfloat16), ("f16", torch.float16)):
        assert len({pkg.prefill_backward_workspace(1, 400, 400, 2, 1, 64, dtype) for dtype in names}) == 1
