"""The paged cache's operators on the GPU against plain 64-bit forms: rotary
positions, cache write, cache read, attention of a few new tokens, and a run
of them together."""
import math

import pytest
import torch

import cache_util as R
from gqa_flash_attention_prefill_gb300 import workloads as W

pytestmark = pytest.mark.gpu
DT = W.DTYPES


@pytest.fixture(scope="module")
def pkg():
    import __graft_entry__
    __graft_entry__.build()
    import gqa_flash_attention_prefill_gb300 as pkg
    pkg.load()
    return pkg


def status_ok(pkg):
    torch.cuda.synchronize()
    assert pkg.get_device_status() == 0


def rand(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


# ------------------------------------------------------------------ rope
@pytest.mark.parametrize("rows,hq,hkv,d,rot", [
    (1, 8, 1, 64, 64), (37, 5, 3, 128, 96), (700, 4, 2, 64, 20), (3, 2, 0, 256, 256), (9, 1, 1, 24, 6),
    (2, 3, 1, 1024, 512), (2500, 2, 1, 64, 64), (1, 1, 1, 8, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rope_matches_64_bits(pkg, rows, hq, hkv, d, rot, interleaved, dtype):
    inv, factor = W.rope_frequencies(rot, 10000.0)
    factor = 1.3
    pos = torch.randint(-3, 1 << 30, (rows,), generator=torch.Generator().manual_seed(rows), dtype=torch.int32)
    packed = rand(rows, hq + hkv + 1, d, seed=d, dtype=DT[dtype]).cuda()
    q, k = packed[:, 1:1 + hq], packed[:, 1 + hq:]
    out = torch.full((rows, hq, d), math.nan, dtype=DT[dtype], device="cuda")
    k_out = torch.full((rows, hkv, d), math.nan, dtype=DT[dtype], device="cuda")
    for inverse in (False, True):
        pkg.gqa_rope(q, pos.cuda(), inv.cuda(), out, k=k if hkv else None, k_out=k_out if hkv else None,
                     interleaved=interleaved, attn_factor=factor, inverse=inverse)
        status_ok(pkg)
        for x, y in ((q, out), (k, k_out)):
            # the angle in 64 bits is off by 2^-53 of up to 2^30: reduce it in exact integers instead
            step = [round(float(f) / (2 * math.pi) * 2.0 ** 64) for f in inv.tolist()]
            turns = torch.tensor([[((int(p) * s) % (1 << 64)) / 2.0 ** 64 for s in step] for p in pos.tolist()],
                                 dtype=torch.float64)
            ref, err = rotate_turns(x.cpu(), turns, factor, interleaved, inverse)
            tol = R.U[x.dtype] * ref.abs() + (1 + R.U[x.dtype]) * err + R.TINY[x.dtype]
            assert bool(((y.cpu().double() - ref).abs() <= tol).all())


def rotate_turns(x, turns, factor, interleaved, inverse):
    y = x.double().clone()
    rot = 2 * turns.shape[1]
    t = turns[:, None] * (-2 if inverse else 2) * math.pi
    c, s = t.cos() * factor, t.sin() * factor
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = y[..., ia], y[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    err = torch.zeros_like(y)
    err[..., ia] = err[..., ib] = (a.abs() + b.abs()) * factor * 2.0 ** -20
    return y, err


def test_rope_inverse_is_the_gradient(pkg):
    """<y(x + h u) - y(x - h u), w> / 2h = <u, inverse(w)>: the operator is
    linear, so the difference quotient is exact up to the roundings (f16 half
    steps of |y| with h = 1: 2^-11 of each of the sums' terms)."""
    rows, h, d = 13, 3, 64
    inv = W.rope_frequencies(48, 500.0, "blend", 8.0, 256)[0].cuda()
    pos = torch.arange(rows, dtype=torch.int32).cuda() * 977
    x, u, w = (rand(rows, h, d, seed=s, dtype=torch.float16).cuda() for s in (1, 2, 3))
    up, dn = (x + u), (x - u)
    y = [pkg.gqa_rope(t, pos, inv, torch.empty_like(t), attn_factor=1.2) for t in (up, dn)]
    back = pkg.gqa_rope(w, pos, inv, torch.empty_like(w), attn_factor=1.2, inverse=True)
    status_ok(pkg)
    lhs = ((y[0].double() - y[1].double()) / 2 * w.double()).sum()
    rhs = ((up.double() - dn.double()) / 2 * back.double()).sum()
    bound = 2.0 ** -11 * (((y[0].double().abs() + y[1].double().abs()) / 2 * w.double().abs()).sum()
                          + ((up.double() - dn.double()).abs() / 2 * back.double().abs()).sum()) * 1.01
    assert float((lhs - rhs).abs()) <= float(bound)


# ------------------------------------------------------------------ write and read
def write_case(pre, new, hkv, d, page, kind, dtype, seed=0):
    b = W.make_batch([0] * len(pre), new, 2 * hkv, hkv, d, dtype, seed=seed)
    b.prefix_lens = torch.tensor(pre, dtype=torch.int32)
    cache = R.fill(W.empty_cache([p + n for p, n in zip(pre, new)], hkv, d, page, dtype, kind, seed=seed), b, seed)
    return b, cache


@pytest.mark.parametrize("pre,new,hkv,d,page", [
    ([0], [1], 1, 64, 16), ([5, 0, 130], [1, 1, 1], 8, 64, 16), ([7, 64, 0, 31], [40, 0, 257, 1], 3, 128, 24),
    ([100], [600], 2, 256, 64), ([3] * 70, [2] * 70, 2, 64, 8), ([0, 9], [2000, 1900], 1, 64, 128)])
@pytest.mark.parametrize("kind", ["16", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_write_then_read(pkg, pre, new, hkv, d, page, kind, dtype):
    """Bytes and scales bit for bit, every other slot left as it was, and the
    read back (whole and its last 50 keys) as the values times the scales."""
    b, cache = write_case(pre, new, hkv, d, page, kind, dtype, seed=page)
    b.k[0, 0] = 0  # a row of zeros
    b.v[0, 0, 3:] = 0
    b.v[0, 0, :3] = torch.tensor([448.0, 1.75, -2.0 ** -9]).to(b.v.dtype)  # largest magnitude on the border
    gpu, dev = R.on_gpu(cache), b.to("cuda")
    pkg.cache_write(dev, gpu)
    status_ok(pkg)
    want = {x: getattr(cache, x + "_pages").view(torch.uint8 if kind == "e4m3" else torch.int16).clone().flatten(0, 1)
            for x in "kv"}
    scales = {x: None if kind == "16" else getattr(cache, x + "_scales").clone().flatten(0, 1) for x in "kv"}
    cu = b.cu_seqlens_q.tolist()
    for i, (p, n) in enumerate(zip(pre, new)):
        at = R.keys_of(cache, i, p, p + n)
        for x in "kv":
            rows = getattr(b, x)[cu[i]:cu[i + 1]]
            if kind == "16":
                want[x][at] = rows.view(torch.int16)
            else:
                want[x][at], scales[x][at] = R.quantise(rows)
    for x in "kv":
        got = getattr(gpu, x + "_pages").cpu().view(want[x].dtype).flatten(0, 1)
        assert torch.equal(got, want[x])
        if kind == "e4m3":
            assert torch.equal(getattr(gpu, x + "_scales").cpu().flatten(0, 1), scales[x])

    lens = [p + n for p, n in zip(pre, new)]
    for tail in (0, 50):
        first = [max(0, n - tail) if tail else 0 for n in lens]
        ip = torch.tensor([0] + torch.tensor([n - f for n, f in zip(lens, first)]).cumsum(0).tolist(), dtype=torch.int32)
        k, v = pkg.cache_read(gpu, ip.cuda(), int(ip[-1]), b.k.dtype,
                              first_keys=torch.tensor(first, dtype=torch.int32).cuda() if tail else None)
        status_ok(pkg)
        cpu = W.Cache(*(t.cpu() if t is not None else None for t in (
            gpu.k_pages, gpu.v_pages, gpu.k_scales, gpu.v_scales, gpu.page_indptr, gpu.page_indices)), gpu.kind)
        for x, got in (("k", k), ("v", v)):
            vals = R.dequantise(getattr(cpu, x + "_pages"), getattr(cpu, x + "_scales")).flatten(0, 1)
            ref = torch.cat([vals[R.keys_of(cache, i, f, n)] for i, (f, n) in enumerate(zip(first, lens))])
            assert torch.equal(got.cpu(), ref.to(b.k.dtype))


@pytest.mark.parametrize("rot,interleaved,explicit", [(64, False, False), (32, True, True), (12, False, True)])
@pytest.mark.parametrize("kind", ["16", "e4m3"])
def test_write_rotates_on_the_way(pkg, rot, interleaved, explicit, kind):
    """k from a packed projection rotated into the cache, q into q_out: each
    value within its own rounding (half an e4m3 step: 2^-4 relative, 2^-10 of
    the scale near zero) plus the rotation's."""
    pre, new, hq, hkv, d = [3, 700, 0], [5, 1, 300], 6, 2, 64
    total = sum(new)
    packed = rand(total, hq + 2 * hkv, d, seed=rot, dtype=torch.bfloat16)
    q, k, v = packed.split([hq, hkv, hkv], 1)
    inv, factor = W.rope_frequencies(rot, 150000.0, "blend", 32.0)
    pos = torch.cat([torch.arange(p, p + n) for p, n in zip(pre, new)])
    if explicit:
        pos = pos * 3 + 11
    cache = R.fill(W.empty_cache([p + n for p, n in zip(pre, new)], hkv, d, 16, "bf16", kind), None, 5)
    gpu = R.on_gpu(cache)
    cu = torch.tensor([0, 5, 6, 306], dtype=torch.int32)
    dq, dk, dv = packed.cuda().split([hq, hkv, hkv], 1)
    q_out = torch.empty(total, hq, d, dtype=torch.bfloat16, device="cuda")
    rope = pkg.Rope(inv.cuda(), positions=pos.to(torch.int32).cuda() if explicit else None, interleaved=interleaved,
                    attn_factor=factor, q=dq, q_out=q_out)
    pkg.gqa_cache_write(dk, dv, cu.cuda(), torch.tensor(pre, dtype=torch.int32).cuda(), gpu.page_indptr, gpu.page_indices,
                        gpu.k_pages, gpu.v_pages, k_scales=gpu.k_scales, v_scales=gpu.v_scales, rope=rope)
    status_ok(pkg)
    ref, err = R.rotate(q, pos, inv, factor, interleaved)
    assert bool(((q_out.cpu().double() - ref).abs() <= R.U[q.dtype] * ref.abs() + 1.01 * err).all())
    at = torch.cat([R.keys_of(cache, i, p, p + n) for i, (p, n) in enumerate(zip(pre, new))])
    ref, err = R.rotate(k, pos, inv, factor, interleaved)
    sc = None if kind == "16" else gpu.k_scales.cpu()
    got = R.dequantise(gpu.k_pages.cpu(), sc).flatten(0, 1)[at]
    if kind == "16":
        tol = R.U[k.dtype] * ref.abs() + 1.01 * err
    else:
        step = torch.exp2(sc.flatten(0, 1)[at].double() - 127)[..., None]
        amax = ref.abs().amax(-1, keepdim=True)
        near = 1 + 2.0 ** -18  # a row on the border of two scales may take either
        assert bool((amax <= 448 * step * near).all() and ((amax * near > 224 * step) | (step == 2.0 ** -60)).all())
        tol = 2.0 ** -4 * ref.abs() + 2.0 ** -10 * step + 1.1 * err
    assert bool(((got - ref).abs() <= tol).all())
    vq = v if kind == "16" else None
    got = R.dequantise(gpu.v_pages.cpu(), None if kind == "16" else gpu.v_scales.cpu()).flatten(0, 1)[at]
    if kind == "16":
        assert torch.equal(got, vq.double())
    else:
        code, e = R.quantise(v)
        assert torch.equal(got, R.TABLE[code.long()] * torch.exp2(e.double() - 127)[..., None])


def test_write_infinities_and_nan(pkg):
    b, cache = write_case([0], [3], 1, 64, 16, "e4m3", "bf16")
    b.k[0, 0, 5] = math.inf
    b.k[0, 0, 6] = -math.inf
    b.k[1, 0, 7] = math.nan
    b.v[2, 0] = math.nan
    gpu = R.on_gpu(cache)
    pkg.cache_write(b.to("cuda"), gpu)
    status_ok(pkg)
    at = R.keys_of(cache, 0, 0, 3)
    kb, ks = gpu.k_pages.cpu().view(torch.uint8).flatten(0, 1)[at], gpu.k_scales.cpu().flatten(0, 1)[at]
    vals = R.TABLE[kb.long()]
    assert float(vals[0, 0, 5]) == 448 and float(vals[0, 0, 6]) == -448
    assert math.isnan(float(vals[1, 0, 7]))
    rest = [i for i in range(64) if i != 7]
    clean = b.k[1].clone()
    clean[0, 7] = 0
    code, e = R.quantise(clean)
    assert torch.equal(kb[1, 0, rest], code[0, rest]) and int(ks[1, 0]) == int(e[0])
    vb = gpu.v_pages.cpu().view(torch.uint8).flatten(0, 1)[at]
    assert bool(((vb[2] & 127) == 127).all()) and int(gpu.v_scales.cpu().flatten(0, 1)[at][2, 0]) == 127


def test_write_and_read_report_bad_metadata(pkg):
    """A page outside the pool, and more keys than pages: those rows are left
    out, the others written, and the status word says so."""
    b, cache = write_case([0, 0], [20, 20], 2, 64, 16, "16", "f16", seed=3)
    gpu, dev = R.on_gpu(cache), b.to("cuda")
    before = gpu.k_pages.clone()
    bad = gpu.page_indices.clone()
    bad[3] = cache.k_pages.shape[0]
    args = (dev.cu_seqlens_q, dev.prefix_lens, gpu.page_indptr)
    pkg.gqa_cache_write(dev.k, dev.v, *args, bad, gpu.k_pages, gpu.v_pages)
    torch.cuda.synchronize()
    assert pkg.get_device_status() == pkg.GQA_DEV_BAD_METADATA
    want = before.cpu().flatten(0, 1)
    want[R.keys_of(cache, 0, 0, 20)] = b.k[:20]
    want[R.keys_of(cache, 1, 0, 16)] = b.k[20:36]
    assert torch.equal(gpu.k_pages.cpu().flatten(0, 1), want)
    k = torch.full((40, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    v = torch.full_like(k, 7.0)
    ip = torch.tensor([0, 40, 40], dtype=torch.int32).cuda()  # sequence 0 has two pages: 32 keys
    pkg.gqa_cache_read(gpu.k_pages, gpu.v_pages, gpu.page_indptr, gpu.page_indices, ip, k, v)
    torch.cuda.synchronize()
    assert pkg.get_device_status() == pkg.GQA_DEV_BAD_METADATA
    assert bool((k[32:] == 7).all()) and torch.equal(k[:20], dev.k[:20])


# ------------------------------------------------------------------ attention
def attention_case(pre, new, hq, hkv, d, page, kind, dtype, window=0, sink="none", tree=False, seed=0, scale=None):
    b = W.make_batch([0] * len(pre), new, hq, hkv, d, dtype, window=window, sink_mode=sink, seed=seed, scale=scale)
    b.prefix_lens = torch.tensor(pre, dtype=torch.int32)
    cache = R.fill(W.empty_cache([p + n for p, n in zip(pre, new)], hkv, d, page, dtype, kind, seed=seed), b, seed + 1)
    keep = depths = None
    if tree:
        keep = [W.random_tree_mask(n, seed=seed + i) for i, n in enumerate(new)]
        depths = [[int(m[t].sum()) - 1 for t in range(m.shape[0])] for m in keep]
    return b, cache, keep, depths


def poison(cache, pre, new):
    """NaN in every slot that holds no key of a sequence."""
    used = torch.zeros(cache.k_pages.shape[0] * cache.k_pages.shape[1], dtype=torch.bool)
    for i, (p, n) in enumerate(zip(pre, new)):
        used[R.keys_of(cache, i, 0, p + n)] = True
    for x in "kv":
        pages = getattr(cache, x + "_pages")
        raw = pages.view(torch.uint8 if cache.kind == "e4m3" else pages.dtype).flatten(0, 1)
        raw[~used] = 0x7F if cache.kind == "e4m3" else math.nan
        if cache.kind == "e4m3":
            getattr(cache, x + "_scales").flatten(0, 1)[~used] = 255


def run_attention(pkg, b, cache, keep=None, depths=None, workspace=None):
    dev, gpu = b.to("cuda"), R.on_gpu(cache)
    mask = indptr = dep = None
    if keep is not None:
        mask, indptr = (t.cuda() for t in W.pack_custom_mask(keep))
    if depths is not None:
        dep = torch.tensor(sum(([int(x) for x in r] for r in depths), []), dtype=torch.int32).cuda()
    out = torch.full_like(dev.q, math.nan)
    lse = torch.full(dev.q.shape[:2], math.nan, device="cuda")
    pkg.cache_attention(dev, gpu, custom_mask=mask, mask_indptr=indptr, depths=dep, out=out, lse=lse,
                        workspace=workspace)
    status_ok(pkg)
    return out, lse


def check(pkg, b, cache, keep=None, depths=None, workspace=None, label=""):
    out, lse = run_attention(pkg, b, cache, keep, depths, workspace)
    ref, z, bo, bl = R.attention(b.q, cache, b.cu_seqlens_q.tolist(), b.prefix_lens.tolist(), b.scale, b.window,
                                 b.sinks, b.smooth, keep, depths)
    n = b.cu_seqlens_q.tolist()[-1]
    got, gl = out.cpu().double()[:n], lse.cpu().double()[:n]
    over = (got - ref[:n]).abs() - bo[:n]
    assert bool((over <= 0).all()), f"{label} out of bound by {float(over.max()):.3g}, nan {bool(got.isnan().any())}"
    none = z[:n] == -math.inf
    assert torch.equal(gl[none], z[:n][none])
    over = (gl - z[:n]).abs()[~none] - bl[:n][~none]
    assert bool((over <= 0).all()), f"{label} lse out of bound by {float(over.max()):.3g}"
    return out, lse


@pytest.mark.parametrize("kind", ["16", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv,d,page", [
    (8, 1, 64, 16), (64, 8, 64, 16), (16, 2, 128, 64), (12, 4, 256, 32), (6, 6, 64, 48), (3, 3, 128, 16),
    (48, 16, 64, 16), (8, 8, 256, 8), (40, 2, 64, 128), (14, 14, 64, 24)])
def test_decode(pkg, hq, hkv, d, page, dtype, kind):
    """One token each over prefixes of 0 to 700 keys, odd lengths, every
    unwritten slot NaN."""
    pre, new = [0, 1, 15, 16, 333, 700], [1] * 6
    b, cache, _, _ = attention_case(pre, new, hq, hkv, d, page, kind, dtype, sink="head", seed=d + page)
    poison(cache, pre, new)
    check(pkg, b, cache)


@pytest.mark.parametrize("kind", ["16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d,window,sink", [
    (64, 8, 64, 0, "head"), (16, 2, 128, 100, "smooth"), (8, 1, 64, 1, "none"), (8, 2, 256, 7, "head"),
    (10, 5, 64, 64, "none"), (2, 2, 64, 0, "smooth")])
def test_trees(pkg, hq, hkv, d, window, sink, kind):
    """Draft trees of 1 to 70 tokens (over two mask words) with depths, over
    prefixes whose end falls inside a tile, windows that cut the tree too."""
    pre, new = [0, 129, 600, 31, 5], [7, 64, 3, 70, 1]
    b, cache, keep, depths = attention_case(pre, new, hq, hkv, d, 16, kind, "bf16", window, sink, tree=True, seed=hq)
    poison(cache, pre, new)
    check(pkg, b, cache, keep, depths)


def test_tree_without_depths_and_rows_without_keys(pkg):
    """Mask without depths; rows whose bitmap and window leave nothing give
    out = 0 and lse = -inf, with and without a sink."""
    for sink in ("none", "head"):
        pre, new = [0, 40], [9, 33]
        b, cache, keep, _ = attention_case(pre, new, 8, 2, 64, 8, "e4m3", "f16", 4, sink, tree=True, seed=9)
        keep[0][:] = False
        keep[1][20:, 10:] = False  # rows 20.. keep only tokens below 10, outside their window
        check(pkg, b, cache, keep)


@pytest.mark.parametrize("kind", ["16", "e4m3"])
@pytest.mark.parametrize("hq,hkv,d,new", [(8, 8, 64, 12), (4, 2, 256, 40), (16, 1, 64, 40), (40, 2, 128, 20)])
def test_hidden_tokens_may_hold_anything(pkg, hq, hkv, d, new, kind):
    """Drafted tokens that no row sees, by the bitmap or by their depth, keys
    below the window and their pages' table entries: NaN with NaN scales, and
    infinities, change nothing."""
    for window in (0, 30):
        pre = [37, 90]
        b, cache, keep, depths = attention_case(pre, [new] * 2, hq, hkv, d, 16, kind, "bf16", window, "none",
                                                tree=True, seed=7 + new)
        hidden = [1, 3, new - 1]
        for m in keep:
            m[:, hidden] = False
        if window:  # token 5 lies a window below every row that its bitmap gives it
            window = b.window = 2
            for m, dep in zip(keep, depths):
                dep[6:] = [max(x, 3) for x in dep[6:]]
                dep[5] = 0
                m[5, 5] = False
            hidden.append(5)
        want, _ = check(pkg, b, cache, keep, depths)
        for i, p in enumerate(pre):
            at = [R.keys_of(cache, i, p + h, p + h + 1) for h in hidden]
            at += [R.keys_of(cache, i, 0, p - window + 1)] if window else []
            for n, rows in enumerate(at):
                for x in "kv":
                    pages = getattr(cache, x + "_pages")
                    if kind == "e4m3":
                        pages.view(torch.uint8).flatten(0, 1)[rows] = 0x7F
                        getattr(cache, x + "_scales").flatten(0, 1)[rows] = 255
                    else:
                        pages.flatten(0, 1)[rows] = math.nan if n % 2 == 0 else math.inf
            if window:  # pages wholly below the window are no longer this sequence's
                first = int(cache.page_indptr[i])
                cache.page_indices[first:first + (p - window + 1) // 16] = -7
        got, _ = run_attention(pkg, b, cache, keep, depths)
        assert torch.equal(got, want)


def test_new_tokens_in_a_run_are_causal(pkg):
    """No mask: several new tokens are a causal chunk, also over 512 rows."""
    pre, new = [50, 0], [200, 19]
    b, cache, _, _ = attention_case(pre, new, 16, 4, 64, 16, "16", "f16", 0, "none", seed=4)
    check(pkg, b, cache)
    b, cache, _, _ = attention_case(pre, new, 16, 4, 64, 16, "e4m3", "f16", 30, "none", seed=5)
    check(pkg, b, cache)


@pytest.mark.parametrize("hq,hkv,d,kind", [(64, 8, 64, "e4m3"), (8, 1, 128, "16"), (4, 4, 256, "e4m3"), (16, 2, 64, "16")])
def test_long_sequence_is_split_and_joined(pkg, hq, hkv, d, kind):
    """A long sequence next to short ones: shares cut it over many CTAs.  Run
    twice on a workspace of 0xFF bytes, the results are equal bit for bit."""
    pre, new = [20000, 3, 1200], [2, 1, 1]
    b, cache, _, _ = attention_case(pre, new, hq, hkv, d, 64, kind, "bf16", 0, "head", seed=2)
    size = pkg.cache_attention_workspace(3, 4, 2, hq, hkv, d, "bf16", kind)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    first = check(pkg, b, cache, workspace=ws)
    again = check(pkg, b, cache, workspace=ws)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("hq,hkv,d,kind,window", [
    (64, 8, 64, "e4m3", 0), (16, 2, 128, "e4m3", 0), (64, 8, 64, "16", 0), (16, 2, 128, "16", 700), (16, 1, 64, "e4m3", 300)])
def test_many_rows_over_long_prefixes(pkg, hq, hkv, d, kind, window):
    """Trees whose rows fill several 128-row tiles (one a little, one half)
    over prefixes of many key tiles, and a sequence of a single tile."""
    pre, new = [5000, 3, 2500], [64, 20, 17]
    b, cache, keep, depths = attention_case(pre, new, hq, hkv, d, 64, kind, "bf16", window, "head", tree=True, seed=12)
    poison(cache, pre, new)
    first = check(pkg, b, cache, keep, depths)
    again = check(pkg, b, cache, keep, depths)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("hq,hkv,new,kind", [(64, 16, 64, "e4m3"), (64, 16, 64, "16"), (8, 8, 1, "16")])
def test_units_cut_into_many_pieces(pkg, hq, hkv, new, kind):
    """One sequence whose units are cut over nine CTAs or more each, with more
    rows than the join has blocks for them."""
    b, cache, _, _ = attention_case([12000], [new], hq, hkv, 64, 64, kind, "bf16", 0, "head", seed=15)
    check(pkg, b, cache)


@pytest.mark.parametrize("d,kind", [(256, "16"), (64, "e4m3")])
def test_long_chunk_of_many_row_tiles(pkg, d, kind):
    """A chunk of 700 tokens after 40 cached ones: many row tiles of one
    sequence, each with its own causal key range."""
    b, cache, _, _ = attention_case([40, 5], [700, 300], 4, 2, d, 16, kind, "bf16", 0, "none", seed=16)
    check(pkg, b, cache)
    b, cache, _, _ = attention_case([40, 5], [700, 300], 4, 2, d, 16, kind, "bf16", 200, "head", seed=17)
    check(pkg, b, cache)


def test_many_short_sequences_of_many_rows(pkg):
    """More units of one key tile than CTAs, each with 80 rows."""
    pre, new = [(5 * i) % 30 for i in range(200)], [10] * 200
    for kind in ("16", "e4m3"):
        b, cache, _, _ = attention_case(pre, new, 16, 2, 64, 16, kind, "bf16", 0, "head", seed=13)
        check(pkg, b, cache)


@pytest.mark.parametrize("new", [2, 40])
def test_value_scales_far_apart_in_a_tile(pkg, new):
    """V rows 2^40 apart in magnitude within one key tile, K rows as well."""
    pre = [150, 20]
    b, cache, _, _ = attention_case(pre, [new, new], 8, 2, 64, 16, "e4m3", "f16", 0, "none", seed=14)
    gen = torch.Generator().manual_seed(3)
    cache.v_scales.copy_(torch.randint(95, 136, cache.v_scales.shape, generator=gen).to(torch.uint8))
    cache.k_scales.copy_(torch.randint(90, 121, cache.k_scales.shape, generator=gen).to(torch.uint8))
    check(pkg, b, cache)


def test_more_sequences_than_one_launch(pkg):
    pre = [(7 * i) % 90 for i in range(1100)]
    b, cache, _, _ = attention_case(pre, [1] * 1100, 4, 2, 64, 16, "e4m3", "bf16", 0, "head", seed=6)
    check(pkg, b, cache)


def test_extreme_scales_and_scores(pkg):
    """Value scales 2^40 apart, keys that tower over the rest, and sinks far
    above and below the scores."""
    pre, new = [300, 40], [1, 2]
    b, cache, _, _ = attention_case(pre, new, 8, 2, 64, 16, "e4m3", "bf16", 0, "head", seed=8)
    gen = torch.Generator().manual_seed(1)
    cache.v_scales.copy_(torch.randint(95, 136, cache.v_scales.shape, generator=gen).to(torch.uint8))
    cache.k_scales.flatten(0, 1)[R.keys_of(cache, 0, 17, 18)] = 127
    b.sinks[:4] = 60.0
    b.sinks[4:] = -60.0
    check(pkg, b, cache)


def test_rows_outside_sequences_and_bad_tables(pkg):
    pre, new = [30, 12], [2, 1]
    b, cache, _, _ = attention_case(pre, new, 8, 2, 64, 16, "16", "bf16", seed=11)
    b.q = torch.cat((b.q, b.q))  # rows behind the last sequence
    out, lse = check(pkg, b, cache)
    assert bool(out[3:].isnan().all()) and bool(lse[3:].isnan().all())
    dev, gpu = b.to("cuda"), R.on_gpu(cache)
    short = gpu.page_indptr.clone()
    short[1] -= 1
    out.fill_(7.0)
    gpu.page_indptr = short
    pkg.cache_attention(dev, gpu, out=out, lse=lse)
    torch.cuda.synchronize()
    assert pkg.get_device_status() == pkg.GQA_DEV_BAD_METADATA and bool((out == 7).all())
    gpu = R.on_gpu(cache)
    gpu.page_indices[1] = 1 << 20
    pkg.cache_attention(dev, gpu, out=out, lse=lse)
    torch.cuda.synchronize()
    assert pkg.get_device_status() == pkg.GQA_DEV_BAD_METADATA


def test_matches_the_paged_prefill(pkg):
    """Over a 16-bit pool the operation is gqa_flash_prefill_paged's: both lie
    within the same bound of the 64-bit result."""
    b = W.make_batch([300, 17], [20, 5], 16, 2, 64, "bf16", window=90, sink_mode="head", seed=3)
    pb = W.paged(b, 16, seed=4).to("cuda")
    ref, lse = pkg.prefill_paged(pb)
    cache = W.Cache(pb.k_pages, pb.v_pages, None, None, pb.page_indptr, pb.page_indices, "16")
    out, lse2 = pkg.cache_attention(pb.batch, cache)
    status_ok(pkg)
    assert float((lse - lse2).abs().max()) <= 1e-5 * float(lse.abs().max())
    # both round P and the result to bf16: each within 2^-8 (|out| + sum p |v|), and sum p |v| <= max |v|
    assert float((out.double() - ref.double()).abs().max()) <= 2 * 2.0 ** -8 * 2 * float(b.v.abs().max())


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("kind", ["16", "e4m3"])
def test_prompt_then_tokens_then_tree(pkg, kind):
    """A prompt rotated and written, read back for the prefill kernel; decoded
    tokens written and attended one at a time (the step captured once per
    token and replayed); then a draft tree.  Every result against the 64-bit
    form on what the cache holds."""
    hq, hkv, d, dt = 16, 2, 64, torch.bfloat16
    prompt, steps, tree = [70, 33], 3, 9
    cap = [n + steps + tree for n in prompt]
    cache = W.empty_cache(cap, hkv, d, 16, "bf16", kind, device="cuda")
    inv, factor = W.rope_frequencies(d, 150000.0, "blend", 32.0)
    inv = inv.cuda()
    scale = d ** -0.5

    def table(lens):  # the pages the present lengths need, as a scheduler hands them over
        ip, idx = [0], []
        for i, n in enumerate(lens):
            s = int(cache.page_indptr[i])
            idx += cache.page_indices[s:s + -(-n // 16)].tolist()
            ip.append(len(idx))
        return (torch.tensor(ip, dtype=torch.int32, device="cuda"), torch.tensor(idx, dtype=torch.int32, device="cuda"))

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def step(pre, new, seed, keep=None, depths=None, graph=False):
        total = sum(new)
        packed = rand(total, hq + 2 * hkv, d, seed=seed, dtype=dt).cuda()
        q, k, v = packed.split([hq, hkv, hkv], 1)
        q_out = torch.full((total, hq, d), math.nan, dtype=dt, device="cuda")
        cu = i32([0] + torch.tensor(new).cumsum(0).tolist())
        plen = i32(pre)
        ip, idx = table([p + n for p, n in zip(pre, new)])
        pos = None
        mask = mip = dep = None
        if keep is not None:
            mask, mip = (t.cuda() for t in W.pack_custom_mask(keep))
            dep = i32(sum(depths, []))
            pos = i32([p + x for p, r in zip(pre, depths) for x in r])
        rope = pkg.Rope(inv, positions=pos, attn_factor=factor, q=q, q_out=q_out)
        out, lse = torch.empty_like(q_out), torch.empty(total, hq, device="cuda")
        ws = torch.empty(pkg.cache_attention_workspace(2, total, max(new), hq, hkv, d, "bf16", kind), dtype=torch.uint8,
                         device="cuda")

        def calls():
            pkg.gqa_cache_write(k, v, cu, plen, ip, idx, cache.k_pages, cache.v_pages, k_scales=cache.k_scales,
                                v_scales=cache.v_scales, rope=rope)
            pkg.gqa_cache_attention(q_out, cache.k_pages, cache.v_pages, cu, plen, ip, idx, scale, ws,
                                    k_scales=cache.k_scales, v_scales=cache.v_scales, custom_mask=mask, mask_indptr=mip,
                                    depths=dep, out=out, lse=lse, max_seqlen_q=max(new))
        if graph:
            g = torch.cuda.CUDAGraph()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                with torch.cuda.graph(g, stream=side):
                    calls()
            g.replay()
            g.replay()
        else:
            calls()
        status_ok(pkg)
        host = W.Cache(*(t.cpu() if t is not None else None for t in (
            cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales, ip, idx)), kind)
        ref, z, bo, bl = R.attention(q_out.cpu(), host, cu.tolist(), pre, scale, keep=keep, depths=depths)
        assert bool(((out.cpu().double() - ref).abs() <= bo).all()) and bool(((lse.cpu().double() - z).abs() <= bl).all())
        return q_out, out, (cu, plen, ip, idx)

    pre = [0, 0]
    q_out, out, (cu, plen, ip, idx) = step(pre, prompt, 1)
    k, v = pkg.gqa_cache_read(cache.k_pages, cache.v_pages, ip, idx, cu, torch.empty(sum(prompt), hkv, d, dtype=dt, device="cuda"),
                              torch.empty(sum(prompt), hkv, d, dtype=dt, device="cuda"), k_scales=cache.k_scales,
                              v_scales=cache.v_scales)
    again = torch.empty_like(q_out)
    pkg.gqa_flash_prefill(q_out, k, v, cu, plen, cu, scale, out=again)
    status_ok(pkg)
    # the prefill kernel on the values read back: two bf16 roundings each side, as above
    assert float((again.double() - out.double()).abs().max()) <= 2 * 2.0 ** -8 * 2 * float(v.double().abs().max())
    pre = list(prompt)
    for t in range(steps):
        step(pre, [1, 1], 10 + t, graph=True)
        pre = [p + 1 for p in pre]
    keep = [W.random_tree_mask(tree, seed=i) for i in range(2)]
    depths = [[int(m[t].sum()) - 1 for t in range(tree)] for m in keep]
    step(pre, [tree, tree], 40, keep, depths)


def test_two_graphs_share_a_workspace_in_turn(pkg):
    """Captured calls of two shapes that use one workspace, replayed one after
    the other and interleaved, keep their results."""
    cases = [attention_case([5000, 9], [1, 1], 8, 2, 64, 16, "e4m3", "bf16", seed=20),
             attention_case([40, 2500, 77], [3, 1, 2], 8, 2, 64, 16, "16", "bf16", seed=21)]
    ws = torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
    runs = []
    for b, cache, _, _ in cases:
        dev, gpu = b.to("cuda"), R.on_gpu(cache)
        out, lse = torch.empty_like(dev.q), torch.empty(dev.q.shape[:2], device="cuda")
        pkg.cache_attention(dev, gpu, workspace=ws, out=out, lse=lse)
        want = out.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkg.cache_attention(dev, gpu, workspace=ws, out=out, lse=lse)
        runs.append((g, out, want, dev, gpu, lse))
    for _ in range(3):
        for g, out, *_ in runs:
            out.zero_()
            g.replay()
    status_ok(pkg)
    for g, out, want, *_ in runs:
        assert torch.equal(out, want)


def test_prepared_call_and_other_stream(pkg):
    b, cache, _, _ = attention_case([1000, 3], [1, 1], 8, 2, 64, 16, "e4m3", "bf16", seed=30)
    want = check(pkg, b, cache)
    dev, gpu = b.to("cuda"), R.on_gpu(cache)
    st = torch.cuda.Stream()
    out, lse = torch.zeros_like(dev.q), torch.zeros(dev.q.shape[:2], device="cuda")
    ws = torch.empty(pkg.cache_attention_workspace(2, 2, 1, 8, 2, 64, "bf16", "e4m3"), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    call = pkg.prepare_call(pkg.gqa_cache_attention, dev.q, gpu.k_pages, gpu.v_pages, dev.cu_seqlens_q, dev.prefix_lens,
                            gpu.page_indptr, gpu.page_indices, dev.scale, ws, k_scales=gpu.k_scales, v_scales=gpu.v_scales,
                            out=out, lse=lse, stream=st, max_seqlen_q=1)
    call()
    st.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    pkg.set_call_flags(pkg.FLAG_METADATA_READY)
    try:
        out.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            call()
        st.synchronize()
    finally:
        pkg.set_call_flags(0)
    assert torch.equal(out, want[0])
    status_ok(pkg)


def test_slots_past_2_gib(pkg):
    """A page whose bytes lie behind 2^31 and 2^32 of the pool."""
    hkv, d, page = 8, 256, 64
    pages = (5 << 30) // (page * hkv * d * 2) + 1
    pool = [torch.zeros(pages, page, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    idx = torch.tensor([pages - 1, pages * 3 // 5, 1], dtype=torch.int32)
    b = W.make_batch([100], [40], 8, hkv, d, "bf16", seed=1)
    dev = b.to("cuda")
    ip = torch.tensor([0, 3], dtype=torch.int32).cuda()
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 140], dtype=torch.int32).cuda()
    pkg.gqa_cache_write(dev.k, dev.v, cu, zero, ip, idx.cuda(), *pool)
    k, v = pkg.gqa_cache_read(*pool, ip, idx.cuda(), cu, torch.empty_like(dev.k), torch.empty_like(dev.v))
    status_ok(pkg)
    assert torch.equal(k, dev.k) and torch.equal(v, dev.v)
    cache = W.Cache(*pool, None, None, ip, idx.cuda(), "16")
    out, lse = pkg.cache_attention(dev, cache)
    status_ok(pkg)
    small = [torch.stack([p[i] for i in idx.tolist()]).cpu() for p in pool]
    host = W.Cache(*small, None, None, ip.cpu(), torch.arange(3, dtype=torch.int32), "16")
    ref, z, bo, bl = R.attention(b.q, host, [0, 40], [100], b.scale, sinks=b.sinks)
    assert bool(((out.cpu().double() - ref).abs() <= bo).all())
