"""The norm and its gradient into buffers of NaN: every element is written, is finite, and within its bound.  The comparisons
ask for `<=` everywhere, so that a NaN fails them; the bounds are test_norm_gpu's."""
import pytest
import torch

from test_cache_gpu import pkg  # noqa: F401 (fixture)
from test_norm_gpu import DT, EPS, F, half_step, randn, tiny

pytestmark = pytest.mark.gpu

WIDTHS = [8, 64, 72, 256, 264, 504, 512, 520, 1000, 1016, 1024, 1032, 2040, 2048, 2056, 4096, 8192, 8200, 16384]
TYPES = [("bf16", "bf16", "bf16"), ("f16", "f32", "f32"), ("f16", "f16", "f32"), ("bf16", "f32", "bf16")]


def nan(*shape, dtype):
    if dtype == torch.uint8:
        return torch.full(shape, 255, dtype=dtype, device="cuda")  # e4m3's NaN; a scale of 2^128, which none has
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def within(got, want, bound):
    assert got.shape == want.shape
    assert bool(((got.double() - want).abs() <= bound).all())


def forward(pkg, x, w, offset, residual, group):  # noqa: F811
    rows, heads, n = x.shape
    h = None if residual is None else nan(*x.shape, dtype=residual.dtype)
    rstd = nan(rows, heads, dtype=torch.float32)
    out = nan(*x.shape, dtype=x.dtype if group is None else torch.uint8)
    scales = None if group is None else nan(rows, heads, n // group, dtype=torch.uint8)
    pkg.gqa_rms_norm(x, w, out, EPS, offset, residual, h, scales, rstd)
    torch.cuda.synchronize()
    v = x if residual is None else h
    if residual is not None:
        assert torch.equal(h, (x.float() + residual.float()).to(residual.dtype))
    v = v.double()
    r = 1 / torch.sqrt(v.square().mean(-1) + EPS)
    within(rstd, r, 26 * F * r)
    y = v * r[..., None] * (w.double() + offset)
    slack = 1.1 * (30 * F * y.abs() + F * (v * r[..., None]).abs() * (w.double().abs() + abs(offset)))
    if group is None:
        within(out, y, half_step(x.dtype) * y.abs() + slack + tiny(x.dtype))
        return
    e = scales.double() - 127
    assert float(e.max()) <= 127 and float(e.min()) >= -60
    step = torch.exp2(e)[..., None].expand(*e.shape, group).flatten(-2)
    within(out.view(torch.float8_e4m3fn).double() * step, y, 2.0 ** -4 * y.abs() + slack + 2.0 ** -10 * step)


@pytest.mark.parametrize("dtype,stream,weight", TYPES)
@pytest.mark.parametrize("n", WIDTHS)
def test_forward(pkg, n, dtype, stream, weight):  # noqa: F811
    rows = 37 if n <= 2048 else 5
    x, w = randn(rows, 1, n, seed=1, dtype=DT[dtype]), randn(n, seed=2, dtype=DT[weight])
    for residual in (None, randn(rows, 1, n, seed=3, dtype=DT[stream], scale=3.0)):
        for group in [None] + [g for g in sorted({32, 64, 128, n}) if n % g == 0]:
            forward(pkg, x, w, 0.5, residual, group)


@pytest.mark.parametrize("heads,n", [(3, 64), (8, 128), (64, 64), (5, 256), (2, 1032)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_forward_of_heads(pkg, heads, n, dtype):  # noqa: F811
    packed, w = randn(41, heads + 3, n, seed=4, dtype=DT[dtype]), randn(n, seed=5)
    for group in [None] + [g for g in (32, n) if n % g == 0]:
        forward(pkg, packed[:, 1:heads + 1], w, 0.0, None, group)


def gradient(pkg, dy, h, w, offset, dh, results):  # noqa: F811
    rows, heads, n = dy.shape
    rstd = (h.float().square().mean(-1) + EPS).rsqrt().contiguous()
    dx = nan(*dy.shape, dtype=dy.dtype) if "dx" in results else None
    dres = nan(*dy.shape, dtype=h.dtype) if "dresidual" in results else None
    dw = nan(n, dtype=torch.float32) if "dweight" in results else None
    ws = nan(pkg.rms_norm_backward_workspace(rows, heads, n, dy.dtype) // 4, dtype=torch.float32)
    pkg.gqa_rms_norm_backward(dy, h, w, rstd, dx, dres, dw, ws, offset, dh)
    torch.cuda.synchronize()
    assert pkg.get_device_status() == 0
    r, d = rstd.double()[..., None], dy.double()
    t = h.double() * r
    g = d * (w.double() + offset)
    want = r * (g - t * (g * t).mean(-1, keepdim=True)) + (0 if dh is None else dh.double())
    big = d.abs() * (w.double().abs() + abs(offset))
    slack = F * r * (8 * big + t.abs() * (56 * (g * t).abs().mean(-1, keepdim=True) + 8 * (big * t.abs()).mean(-1, keepdim=True)))
    slack = slack + 4 * F * want.abs() + (0 if dh is None else F * dh.double().abs())
    for x in (dx, dres):
        if x is not None:
            within(x, want, half_step(x.dtype) * want.abs() + 1.01 * slack + tiny(x.dtype))
    if dw is not None:
        within(dw, (d * t).sum((0, 1)), F * (min(rows * heads, 600) + 60) * (d * t).abs().sum((0, 1)))


@pytest.mark.parametrize("dtype,stream,weight", TYPES)
@pytest.mark.parametrize("n", WIDTHS)
def test_gradient(pkg, n, dtype, stream, weight):  # noqa: F811
    for rows, with_dh in ((1, True), (700 if n <= 4096 else 400, True), (37, False)):
        dy, h = randn(rows, 1, n, seed=1, dtype=DT[dtype]), randn(rows, 1, n, seed=2, dtype=DT[stream], scale=3.0)
        dh = randn(rows, 1, n, seed=3, dtype=DT[stream]) if with_dh else None
        gradient(pkg, dy, h, randn(n, seed=4, dtype=DT[weight]), 1.0, dh, ("dx", "dresidual", "dweight"))


@pytest.mark.parametrize("results", [("dx",), ("dresidual",), ("dweight",), ("dx", "dweight"), ("dresidual", "dweight")])
@pytest.mark.parametrize("n", [64, 512, 1024, 4096])
def test_some_results(pkg, n, results):  # noqa: F811
    dy, h = randn(50, 1, n, seed=1, dtype=torch.bfloat16), randn(50, 1, n, seed=2)
    gradient(pkg, dy, h, randn(n, seed=4), 0.0, None, results)


@pytest.mark.parametrize("heads,n", [(3, 64), (8, 128), (5, 256), (2, 1032), (64, 64)])
def test_gradient_of_heads(pkg, heads, n):  # noqa: F811
    wide = lambda t: torch.cat([t[:, :1], t, t[:, :1]], 1)[:, 1:heads + 1]  # noqa: E731
    dy, h = (wide(randn(130, heads, n, seed=s, dtype=torch.bfloat16)) for s in (1, 2))
    gradient(pkg, dy, h, randn(n, seed=4), 0.0, None, ("dx", "dweight"))


@pytest.mark.parametrize("rows,n", [(700, 1024), (400, 4096), (60, 16384), (700, 256)])
def test_values_that_are_not_finite(pkg, rows, n):  # noqa: F811
    """A NaN or an infinity of dy is written where it belongs: its row of dx, its column of dweight, and nowhere else."""
    dy, h, w = randn(rows, n, seed=1, dtype=torch.bfloat16), randn(rows, n, seed=2, dtype=torch.bfloat16), randn(n, seed=3)
    rstd = (h.float().square().mean(-1) + EPS).rsqrt()
    want = pkg.rms_norm_backward(dy, h, w, rstd)
    dy[5, 9], dy[rows - 2, n - 3] = float("nan"), float("inf")
    h[rows - 2, n - 3] = 1.0  # not zero: an infinity times zero is NaN
    ws = nan(pkg.rms_norm_backward_workspace(rows, 1, n, "bf16") // 4, dtype=torch.float32)
    dx, dw = torch.full_like(dy, 7.0), torch.full((n,), 7.0, device="cuda")
    pkg.gqa_rms_norm_backward(dy, h, w, rstd, dx, dweight=dw, workspace=ws)
    torch.cuda.synchronize()
    assert pkg.get_device_status() == 0
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[5] = rest[rows - 2] = False
    assert torch.equal(dx[rest], want[0][rest]) and not bool(dx[~rest].isfinite().any())
    col = torch.ones(n, dtype=torch.bool, device="cuda")
    col[9] = col[n - 3] = False
    assert bool(dw[9].isnan()) and bool(dw[n - 3].isinf()) and torch.equal(dw[col], want[2][col])
