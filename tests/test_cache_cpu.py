"""Refusals of the paged cache's operators, before any launch (fake addresses,
no device), and the host-side helpers."""
import ctypes
import math

import pytest
import torch

import cache_util as R
from gqa_flash_attention_prefill_gb300 import workloads as W

FAKE = 1 << 20  # a 16-byte-aligned non-null address; never dereferenced
FAR = 1 << 40   # another one, far from it


@pytest.fixture(scope="module")
def lib():
    from gqa_flash_attention_prefill_gb300 import build
    import gqa_flash_attention_prefill_gb300 as pkg
    return pkg.load(build.build())


def rope_args(**over):
    import gqa_flash_attention_prefill_gb300 as pkg
    a = dict(positions=FAKE, inv_freq=FAKE, rot_dim=64, interleaved=0, inverse=0, attn_factor=1.0, Hq=4, q=FAKE,
             q_stride=256, q_out=FAR, q_out_stride=256)
    a.update({k: v for k, v in over.items() if k in a})
    return pkg._RopeArgs(*a.values())


def call_rope(lib, **over):
    a = dict(k=FAKE, k_stride=128, k_out=FAR + (1 << 30), k_out_stride=128, rows=3, hkv=2, d=64, dtype=1, stream=None)
    a.update({k: v for k, v in over.items() if k in a})
    r = None if over.get("none") else ctypes.byref(rope_args(**over))
    return lib.gqa_rope(r, *a.values())


@pytest.mark.parametrize("over,code", [
    (dict(none=True), -1), (dict(rows=-1), -1), (dict(hkv=-1), -1), (dict(d=0), -1), (dict(dtype=2), -1),
    (dict(rot_dim=0), -1), (dict(rot_dim=7), -1), (dict(rot_dim=66), -1), (dict(interleaved=2), -1), (dict(inverse=5), -1),
    (dict(attn_factor=float("nan")), -1), (dict(attn_factor=float("inf")), -1), (dict(positions=None), -1),
    (dict(inv_freq=None), -1), (dict(inv_freq=FAKE + 4), -1), (dict(q=None), -1), (dict(q=FAKE + 8), -1),
    (dict(q_stride=248), -1), (dict(q_stride=260), -1), (dict(q_out=FAKE + 256), -1), (dict(k_out=FAKE), -1),
    (dict(q=FAR + (1 << 31), q_out=FAKE + 64), -1), (dict(k=FAR + (1 << 31), k_out=FAKE + 64), -1),
    (dict(k=None), -1), (dict(d=68, rot_dim=64), -2), (dict(d=2048), -2), (dict(d=1024, rot_dim=600), -2),
    (dict(rows=0, positions=None), 0), (dict(Hq=0, hkv=0), 0)])
def test_rope_refusals(lib, over, code):
    assert call_rope(lib, **over) == code


def call_write(lib, **over):
    a = dict(k=FAKE, ks=128, v=FAKE, vs=128, cu=FAKE, pre=FAKE, ip=FAKE, idx=FAKE, entries=4, page=16, pages=8, B=1, total=3,
             hkv=2, d=64, dtype=1, kind=1, kp=FAKE, vp=FAKE, ksc=FAKE, vsc=FAKE)
    a.update({k: v for k, v in over.items() if k in a})
    rope = ctypes.byref(rope_args(**over["rope"])) if "rope" in over else None
    return lib.gqa_cache_write(*a.values(), rope, None)


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), -1), (dict(total=-1), -1), (dict(hkv=0), -1), (dict(dtype=9), -1), (dict(kind=2), -1), (dict(page=12), -1),
    (dict(page=0), -1), (dict(pages=0), -1), (dict(pages=1 << 28), -1), (dict(entries=-1), -1), (dict(entries=0), -1),
    (dict(k=None), -1), (dict(v=FAKE + 2), -1), (dict(ks=100), -1), (dict(vs=132), -1), (dict(cu=None), -1),
    (dict(idx=None), -1), (dict(kp=None), -1), (dict(vp=FAKE + 8), -1), (dict(ksc=None), -1), (dict(d=96), -2),
    (dict(rope=dict(inverse=1)), -1), (dict(rope=dict(rot_dim=128)), -1), (dict(rope=dict(q_out=FAKE)), -1),
    (dict(B=0, k=None), 0), (dict(total=0), 0)])
def test_write_refusals(lib, over, code):
    assert call_write(lib, **over) == code


def call_read(lib, **over):
    a = dict(kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, kind=1, ip=FAKE, idx=FAKE, entries=4, page=16, pages=8, kvi=FAKE, first=None,
             B=1, total=3, hkv=2, d=64, dtype=1, k=FAKE, v=FAKE, stream=None)
    a.update(over)
    return lib.gqa_cache_read(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), -1), (dict(total=-1), -1), (dict(hkv=0), -1), (dict(dtype=3), -1), (dict(kind=-1), -1), (dict(page=4), -1),
    (dict(entries=0), -1), (dict(kp=None), -1), (dict(k=FAKE + 8), -1), (dict(ks=None), -1), (dict(kvi=None), -1),
    (dict(d=32), -2), (dict(total=0), 0), (dict(B=0), 0)])
def test_read_refusals(lib, over, code):
    assert call_read(lib, **over) == code


def call_attention(lib, **over):
    a = dict(q=FAKE, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, kind=1, cu=FAKE, pre=FAKE, ip=FAKE, idx=FAKE, entries=4, page=16,
             pages=8, B=1, total=3, max=3, hq=8, hkv=2, d=64, dtype=1, scale=0.125, window=0, sinks=None, smooth=0, mask=None,
             mip=None, words=0, depths=None, out=FAKE, lse=None, ws=FAKE, size=1 << 40, stream=None)
    a.update(over)
    return lib.gqa_cache_attention(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(B=-1), -1), (dict(total=-2), -1), (dict(max=-1), -1), (dict(hq=7), -1), (dict(hkv=0), -1), (dict(dtype=4), -1),
    (dict(kind=7), -1), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1), (dict(sinks=FAKE, smooth=1), -1),
    (dict(page=20), -1), (dict(pages=0), -1), (dict(entries=0), -1), (dict(words=-1), -1), (dict(q=None), -1),
    (dict(out=FAKE + 4), -1), (dict(ks=None), -1), (dict(vs=FAKE + 8), -1), (dict(mask=FAKE), -1), (dict(mip=FAKE), -1),
    (dict(mask=FAKE + 2, mip=FAKE), -1), (dict(ws=None), -1), (dict(ws=FAKE + 16), -1), (dict(size=100), -1), (dict(d=80), -2),
    (dict(hkv=1, hq=8, page=8), -2),  # e4m3 scales of a page: fewer than 16 bytes
    (dict(total=1 << 30, max=1), -2), (dict(B=0, q=None), 0), (dict(total=0), 0)])
def test_attention_refusals(lib, over, code):
    assert call_attention(lib, **over) == code


def test_attention_workspace(lib):
    import gqa_flash_attention_prefill_gb300 as pkg
    one = pkg.cache_attention_workspace(1, 1, 1, 64, 8, 64, "bf16", "e4m3")
    many = pkg.cache_attention_workspace(500, 500, 1, 64, 8, 64, "bf16", "e4m3")
    assert 0 < one <= many and many % 256 == 0
    with pytest.raises(pkg.GQAError):
        pkg.cache_attention_workspace(1, 1, 1, 64, 8, 96, "bf16", "16")
    with pytest.raises(ValueError):
        pkg.cache_attention_workspace(1, 1, 1, 64, 8, 64, "bf16", "int8")
    size = ctypes.c_size_t(0)
    assert lib.gqa_cache_attention_workspace(1, 1, 1, 64, 8, 64, 1, 1, None) == -1
    assert lib.gqa_cache_attention_workspace(1, 1, 1, 64, 7, 64, 1, 1, ctypes.byref(size)) == -1


def test_binding_refusals():
    """What the Python layer refuses before it takes a pointer (CPU tensors
    among it)."""
    import gqa_flash_attention_prefill_gb300 as pkg
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.gqa_rope(x, torch.zeros(3, dtype=torch.int32), torch.zeros(32, dtype=torch.float64), x.clone())
    with pytest.raises(ValueError, match="float64"):
        pkg.Rope(torch.zeros(32))
    with pytest.raises(ValueError, match="go together"):
        pkg.Rope(torch.zeros(32, dtype=torch.float64), q=x)
    with pytest.raises(ValueError, match="int32"):
        pkg.Rope(torch.zeros(32, dtype=torch.float64), positions=torch.zeros(3))
    with pytest.raises(ValueError, match="prepare_call"):
        pkg.prepare_call(pkg.gqa_flash_prefill)
    pages = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="no scales"):
        pkg._pool(pages, pages, torch.zeros(2, 16, 2, dtype=torch.uint8), None)
    with pytest.raises(TypeError, match="type of the rows"):
        pkg._pool(pages, pages, None, None, torch.float16)
    with pytest.raises(TypeError):
        pkg._pool(pages.float(), pages.float(), None, None)
    e4 = pages.to(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="byte tensor"):
        pkg._pool(e4, e4, None, None)
    with pytest.raises(ValueError, match="agree"):
        pkg._pool(pages, pages[:1], None, None)
    with pytest.raises(ValueError, match="packed heads"):
        pkg._rows("q", torch.zeros(3, 64, 2).transpose(1, 2))
    # rows of a packed projection are fine: their stride is what is passed on
    assert pkg._rows("k", torch.zeros(3, 8, 64)[:, 2:4]) == 512


def test_rope_frequencies():
    inv, f = W.rope_frequencies(64, 10000.0)
    assert f == 1.0 and inv.dtype == torch.float64 and float(inv[0]) == 1.0
    assert math.isclose(float(inv[1]), 10000 ** (-2 / 64), rel_tol=1e-14)
    assert torch.equal(W.rope_frequencies(64, 10000.0, "linear", 4.0)[0], inv / 4)
    stretched, _ = W.rope_frequencies(64, 10000.0, "base", 8.0)
    assert float(stretched[0]) == 1.0 and math.isclose(float(stretched[-1]), float(inv[-1]) / 8, rel_tol=1e-12)
    inv, _ = W.rope_frequencies(64, 150000.0)
    blend, f = W.rope_frequencies(64, 150000.0, "blend", 32.0)
    assert math.isclose(f, 0.1 * math.log(32) + 1)
    turns = inv * 4096 / (2 * math.pi)
    assert torch.allclose(blend[turns > 33], inv[turns > 33], rtol=1e-12)
    assert torch.allclose(blend[turns < 0.9], inv[turns < 0.9] / 32, rtol=1e-12)
    assert bool((blend <= inv).all() and (blend >= inv / 32 * (1 - 1e-12)).all())
    for bad in (dict(rot_dim=5), dict(rot_dim=64, base=1.0), dict(rot_dim=64, scaling="x"), dict(rot_dim=2, scaling="base")):
        with pytest.raises(ValueError):
            W.rope_frequencies(**bad)


def test_plain_forms_agree_with_closed_ones():
    """The reference forms of the GPU tests: e4m3 against torch's own
    conversion, scales on their borders, and attention over one key."""
    x = torch.randn(40, 3, 64, generator=torch.Generator().manual_seed(0)).double()
    code, e = R.quantise(x)
    assert torch.equal(code, (x * torch.exp2(-(e.double() - 127))[..., None]).float().to(torch.float8_e4m3fn).view(torch.uint8))
    assert [R.scale_exponent(v) for v in (448.0, 448.1, 224.0, 0.0, 1e-30, 896.0)] == [0, 1, -1, 0, -60, 1]
    cache = R.fill(W.empty_cache([1], 1, 64, 16, "bf16", "e4m3"), None, 3)
    q = torch.randn(1, 2, 64).to(torch.bfloat16)
    out, lse, bo, bl = R.attention(q, cache, [0, 1], [0], 0.125)
    v = R.dequantise(cache.v_pages, cache.v_scales).flatten(0, 1)[R.keys_of(cache, 0, 0, 1)]
    assert torch.allclose(out, v.expand(1, 2, 64), rtol=1e-12) and bool((bo > 0).all() and (bl > 0).all())
