"""The root-mean-square norm and its gradient on the GPU against their formulas in 64 bits.

Bounds, with f = 2^-24 and u half a step of the output's type.  Sums of positive terms are made in a tree whose longest
path has at most 32 (a thread's values) + 10 (lanes, warps) additions, so a mean of squares is off by 46 f relative and
rstd by 23 f + 3 f; a norm's value takes three more roundings (30 f in all) and its own, u."""
import pytest
import torch

from test_cache_gpu import pkg  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
F = 2.0 ** -24
EPS = 1e-5


def randn(*shape, seed=0, dtype=torch.float32, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):  # half a step of the smallest values
    return 2.0 ** -25 if dtype == torch.float16 else 0.0


def check_out(out, scales, rstd, h, weight, offset, eps, dtype):
    """out (and scales) of the rows h [rows, heads, n]."""
    h = h.double()
    want_rstd = 1 / torch.sqrt(h.square().mean(-1) + eps)
    if rstd is not None:
        assert float(((rstd.double() - want_rstd) / want_rstd).abs().max()) <= 26 * F
    y = h * want_rstd[..., None] * (weight.double() + offset)
    slack = 30 * F * y.abs() + F * (h * want_rstd[..., None]).abs() * (weight.double().abs() + abs(offset))
    if scales is None:
        bad = (out.double() - y).abs() > half_step(dtype) * y.abs() + 1.01 * slack + tiny(dtype)
        assert not bool(bad.any())
        return
    group = h.shape[-1] // scales.shape[-1]
    e = scales.view(torch.uint8).double() - 127
    most = y.unflatten(-1, (-1, group)).abs().amax(-1)
    room = slack.unflatten(-1, (-1, group)).amax(-1)

    def exponent(x):
        return torch.where(x == 0, torch.zeros_like(x), torch.ceil(torch.log2(x / 448)).clamp(-60, 127))

    assert bool(((e == exponent(most - room)) | (e == exponent(most + room))).all())
    step = torch.exp2(e)[..., None].expand(*e.shape, group).flatten(-2)
    got = out.view(torch.float8_e4m3fn).double() * step
    assert not bool(((got - y).abs() > 2.0 ** -4 * y.abs() + 1.1 * slack + 2.0 ** -10 * step).any())


@pytest.mark.parametrize("dtype,stream,weight", [("bf16", "bf16", "bf16"), ("f16", "f32", "f32"), ("f16", "f16", "f32"),
                                                 ("bf16", "f32", "bf16")])
@pytest.mark.parametrize("rows,n", [(1, 8), (3, 72), (5, 256), (2, 1000), (7, 1024), (3, 1032), (1, 2048), (4, 2056), (2, 4096),
                                    (3, 8192), (2, 8200), (1, 16384)])
def test_rows(pkg, rows, n, dtype, stream, weight):  # noqa: F811
    x, w = randn(rows, n, seed=1, dtype=DT[dtype]), randn(n, seed=2, dtype=DT[weight])
    res = randn(rows, n, seed=3, dtype=DT[stream], scale=3.0)
    for offset, residual in ((0.0, None), (1.0, res)):
        out, _, h, rstd = pkg.rms_norm(x, w, EPS, offset, residual, with_rstd=True)
        if residual is not None:
            assert torch.equal(h, (x.float() + residual.float()).to(residual.dtype))
        check_out(out[:, None], None, rstd[:, None], h[:, None], w, offset, EPS, x.dtype)


@pytest.mark.parametrize("dtype,stream", [("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("rows,n,group", [(1, 4096, 128), (5, 4096, 32), (3, 5120, 64), (4, 64, 64), (9, 64, 32), (2, 128, 128),
                                          (3, 1000, 1000), (2, 2048, 2048), (1, 16384, 32), (7, 8, 8), (2, 96, 32), (2, 3104, 32)])
def test_eight_bits(pkg, rows, n, group, dtype, stream):  # noqa: F811
    x, w = randn(rows, n, seed=1, dtype=DT[dtype]), randn(n, seed=2)
    x[0, : n // 2] = 0  # groups of zeros, where there is no residual
    for residual in (None, randn(rows, n, seed=3, dtype=DT[stream])):
        out, scales, h, rstd = pkg.rms_norm(x, w, EPS, 0.5, residual, group, True)
        check_out(out[:, None], scales[:, None], rstd[:, None], h[:, None], w, 0.5, EPS, x.dtype)


@pytest.mark.parametrize("heads,n", [(1, 64), (3, 64), (8, 128), (64, 64), (5, 256), (2, 1032)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_heads_of_a_packed_projection(pkg, heads, n, dtype):  # noqa: F811
    """Each head's norm, in place in the projection; what lies beside is left."""
    rows = 37
    packed = randn(rows, heads + 3, n, seed=4, dtype=DT[dtype])
    before, w = packed.clone(), randn(n, seed=5)
    mine = packed[:, 1:heads + 1]
    rstd = torch.empty(rows, heads, device="cuda")
    pkg.gqa_rms_norm(mine, w, mine, eps=EPS, rstd=rstd)
    check_out(mine, None, rstd, before[:, 1:heads + 1], w, 0.0, EPS, mine.dtype)
    assert torch.equal(packed[:, :1], before[:, :1]) and torch.equal(packed[:, heads + 1:], before[:, heads + 1:])


def test_sizes_of_values(pkg):  # noqa: F811
    w = randn(512, seed=1)
    for scale in (1e-30, 1e-3, 1e15):
        x = randn(6, 512, seed=2, dtype=torch.bfloat16, scale=scale)
        x[3] = 0
        for group in (None, 32, 512):
            out, scales, h, rstd = pkg.rms_norm(x, w, EPS, group=group, with_rstd=True)
            check_out(out[:, None], None if scales is None else scales[:, None], rstd[:, None], h[:, None], w, 0.0, EPS, x.dtype)
    # A row that is not finite spoils none beside it.
    x = randn(8, 512, seed=3, dtype=torch.bfloat16)
    want = pkg.rms_norm(x, w)[0]
    x[2, 7], x[5, 100] = float("nan"), float("inf")
    got = pkg.rms_norm(x, w)[0]
    keep = [0, 1, 3, 4, 6, 7]
    assert torch.equal(got[keep], want[keep]) and bool(got[2].isnan().all())


def check_gradient(pkg, rows, heads, n, dtype, stream, weight, offset, with_dh, strided=False, seed=0):  # noqa: F811
    dt, st = DT[dtype], DT[stream]
    wide = (lambda t: torch.cat([t[:, :1], t, t[:, :1]], 1)[:, 1:heads + 1]) if strided else (lambda t: t)
    dy = wide(randn(rows, heads, n, seed=seed, dtype=dt))
    h = wide(randn(rows, heads, n, seed=seed + 1, dtype=st, scale=3.0))
    w = randn(n, seed=seed + 2, dtype=DT[weight])
    dh = randn(rows, heads, n, seed=seed + 3, dtype=st) if with_dh else None
    rstd = (h.float().square().mean(-1) + EPS).rsqrt().contiguous()
    dx, dres, dw = pkg.rms_norm_backward(dy, h, w, rstd, offset, dh)
    torch.cuda.synchronize()
    r = rstd.double()[..., None]
    t, d = h.double() * r, dy.double()
    g = d * (w.double() + offset)
    c = (g * t).mean(-1, keepdim=True)
    c_abs = (g * t).abs().mean(-1, keepdim=True)
    want = r * (g - t * c) + (0 if dh is None else dh.double())
    # g and t two roundings each (offset's sum one more, of the larger magnitude), the sum's tree 46, the result's four
    big = d.abs() * (w.double().abs() + abs(offset))
    slack = F * r * (8 * big + t.abs() * (56 * c_abs + 8 * (big * t.abs()).mean(-1, keepdim=True))) + 4 * F * want.abs()
    if dh is not None:
        slack = slack + F * dh.double().abs()
    for x in {id(dx): dx, id(dres): dres}.values():
        assert not bool(((x.double() - want).abs() > half_step(x.dtype) * want.abs() + 1.01 * slack + tiny(x.dtype)).any())
    want_w = (d * t).sum((0, 1))
    assert not bool(((dw.double() - want_w).abs() > F * (min(rows * heads, 600) + 60) * (d * t).abs().sum((0, 1))).any())
    return dy, h, w, rstd, dh, dx, dres, dw


@pytest.mark.parametrize("dtype,stream,weight,offset,with_dh", [("bf16", "bf16", "bf16", 0.0, True), ("f16", "f32", "f32", 1.0, True),
                                                                ("bf16", "f32", "bf16", 1.0, False), ("f16", "f16", "f32", 0.0, False)])
@pytest.mark.parametrize("rows,n", [(1, 8), (3, 72), (33, 1000), (700, 256), (2, 1024), (400, 1032), (3, 2056), (500, 4096), (2, 8200),
                                    (400, 16384)])
def test_gradient(pkg, rows, n, dtype, stream, weight, offset, with_dh):  # noqa: F811
    check_gradient(pkg, rows, 1, n, dtype, stream, weight, offset, with_dh)


@pytest.mark.parametrize("rows,heads,n", [(1, 1, 64), (50, 3, 64), (129, 8, 128), (40, 5, 256), (3, 2, 1032), (600, 2, 64)])
def test_gradient_of_heads(pkg, rows, heads, n):  # noqa: F811
    check_gradient(pkg, rows, heads, n, "bf16", "bf16", "f32", 0.0, False, strided=True)


def test_gradient_against_differences(pkg):  # noqa: F811
    """Differences of the forward kernel over an fp32 stream: <dy, out> moves by <dx, step> + <dw, step>."""
    x, dy = torch.zeros(4, 512, dtype=torch.float16, device="cuda"), randn(4, 512, seed=1, dtype=torch.float16)
    res, w = randn(4, 512, seed=2), randn(512, seed=3)
    _, _, h, rstd = pkg.rms_norm(x, w, EPS, residual=res, with_rstd=True)
    _, dres, dw = pkg.rms_norm_backward(dy, h, w, rstd)

    def loss(r, weight):  # the norm in 64 bits (the forward kernel's 16-bit output is too coarse to be differenced)
        r = r.double()
        return float((dy.double() * r / torch.sqrt(r.square().mean(-1, keepdim=True) + EPS) * weight.double()).sum())

    a, b, t = randn(4, 512, seed=4).double(), randn(512, seed=5).double(), 1e-4
    slope = (loss(res.double() + t * a, w.double() + t * b) - loss(res.double() - t * a, w.double() - t * b)) / (2 * t)
    got = float((dres.double() * a).sum() + (dw.double() * b).sum())
    size = float((dres.double() * a).abs().sum() + (dw.double() * b).abs().sum())
    assert abs(got - slope) <= size * 100 * F + 1e-5  # the difference's own error: t^2 = 1e-8 of third derivatives


def test_in_place_and_same_bits(pkg):  # noqa: F811
    x, res, w = randn(300, 2048, seed=1, dtype=torch.bfloat16), randn(300, 2048, seed=2, dtype=torch.bfloat16), randn(2048, seed=3)
    out, _, h, rstd = pkg.rms_norm(x, w, EPS, residual=res, with_rstd=True)
    x2, res2 = x.clone(), res.clone()
    pkg.gqa_rms_norm(x2, w, x2, eps=EPS, residual=res2, residual_out=res2)
    assert torch.equal(x2, out) and torch.equal(res2, h)
    dy, dh = randn(300, 2048, seed=4, dtype=torch.bfloat16), randn(300, 2048, seed=5, dtype=torch.bfloat16)
    dx, _, dw = pkg.rms_norm_backward(dy, h, w, rstd, dh=dh)
    ws = torch.full((pkg.rms_norm_backward_workspace(300, 1, 2048, "bf16"),), 255, dtype=torch.uint8, device="cuda")
    for target in ("dy", "dh", "h"):
        t = {"dy": dy.clone(), "dh": dh.clone(), "h": h.clone()}
        dw2 = torch.empty_like(dw)
        pkg.gqa_rms_norm_backward(t["dy"], t["h"], w, rstd, t[target], dweight=dw2, workspace=ws, dh=t["dh"])
        assert torch.equal(t[target], dx) and torch.equal(dw2, dw)


def test_no_rows(pkg):  # noqa: F811
    x, w = torch.empty(0, 256, dtype=torch.float16, device="cuda"), randn(256)
    assert pkg.rms_norm(x, w, with_rstd=True)[0].shape == (0, 256)
    dx, _, dw = pkg.rms_norm_backward(x, x, w, torch.empty(0, device="cuda"))
    assert dx.numel() == 0 and not bool(dw.any())


def test_graph_and_stream(pkg):  # noqa: F811
    """Captured and replayed over new values, and a call of another stream whose memory is not handed out."""
    x, res, w = randn(64, 4096, seed=1, dtype=torch.bfloat16), randn(64, 4096, seed=2, dtype=torch.bfloat16), randn(4096, seed=3)
    out, h, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(64, device="cuda")
    dw, dx = torch.empty(4096, device="cuda"), torch.empty_like(x)
    ws = torch.empty(pkg.rms_norm_backward_workspace(64, 1, 4096, "bf16"), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pkg.gqa_rms_norm(x, w, out, eps=EPS, residual=res, residual_out=h, rstd=rstd)
        pkg.gqa_rms_norm_backward(x, h, w, rstd, dx, dweight=dw, workspace=ws, dh=h)
    for seed in (7, 8):
        x.copy_(randn(64, 4096, seed=seed, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        want = pkg.rms_norm(x, w, EPS, residual=res, with_rstd=True)
        assert torch.equal(out, want[0]) and torch.equal(h, want[2]) and torch.equal(rstd, want[3])
        wx, _, ww = pkg.rms_norm_backward(x, h, w, rstd, dh=h)
        assert torch.equal(dx, wx) and torch.equal(dw, ww)
    for call in (lambda s: [t for t in pkg.rms_norm(x, w, EPS, residual=res, group=128, with_rstd=True, stream=s) if t is not None],
                 lambda s: list(pkg.rms_norm_backward(x, h, w, rstd, dh=h, stream=s))):
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        other = torch.cuda.Stream()
        with torch.cuda.stream(other):
            torch.cuda._sleep(20_000_000)
        got = call(other)
        blocks = [torch.full((t.numel() * t.element_size(),), 255, dtype=torch.uint8, device="cuda") for t in got * 2 + [ws]]
        other.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
        assert all(bool((b == 255).all()) for b in blocks)


def test_offsets_past_32_bits(pkg):  # noqa: F811
    """Rows past 2^31 values, forward and back."""
    rows, n = 2 ** 19 + 3, 4096
    x = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    x[-3:] = randn(3, n, seed=1, dtype=torch.bfloat16)
    weight = randn(n, seed=2)
    out, _, _, rstd = pkg.rms_norm(x, weight, EPS, with_rstd=True)
    check_out(out[-3:, None], None, rstd[-3:, None], x[-3:, None], weight, 0.0, EPS, torch.bfloat16)
    assert not bool(out[:-3].any())
    dx, _, dweight = pkg.rms_norm_backward(x, x, weight, rstd)
    few = pkg.rms_norm_backward(x[-3:].clone(), x[-3:].clone(), weight, rstd[-3:].clone())
    assert torch.equal(dx[-3:], few[0]) and not bool(dx[:-3].any())
    # Three rows' products, in another order at most: 3 f of the sum of magnitudes.
    t = x[-3:].double() * rstd[-3:, None].double()
    room = 2.0 ** -22 * (x[-3:].double() * t).abs().sum(0)
    assert bool(((dweight - few[2]).abs().double() <= room).all())


@pytest.mark.parametrize("dtype,stream,weight", [("bf16", "bf16", "f32"), ("f16", "f32", "f16")])
@pytest.mark.parametrize("rows", [1, 37, 311])
@pytest.mark.parametrize("n", [264, 504, 512, 520, 768, 1016, 1024, 1032, 1536, 2040, 2048])
def test_widths(pkg, rows, n, dtype, stream, weight):  # noqa: F811
    """A row in a warp of one, two or four groups a lane, or in a CTA of one or two a thread; teams with rows missing."""
    x, w = randn(rows, n, seed=1, dtype=DT[dtype]), randn(n, seed=2, dtype=DT[weight])
    res = randn(rows, n, seed=3, dtype=DT[stream], scale=3.0)
    out, _, h, rstd = pkg.rms_norm(x, w, EPS, 1.0, res, with_rstd=True)
    check_out(out[:, None], None, rstd[:, None], h[:, None], w, 1.0, EPS, x.dtype)
    for group in [g for g in (32, 128, n) if n % g == 0]:
        out, scales, h, rstd = pkg.rms_norm(x, w, EPS, 0.0, res, group, True)
        check_out(out[:, None], scales[:, None], rstd[:, None], h[:, None], w, 0.0, EPS, x.dtype)
    check_gradient(pkg, rows, 1, n, dtype, stream, weight, 1.0, rows != 37, strided=rows == 37)
