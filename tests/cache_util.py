"""Plain 64-bit forms of the paged cache's operators, on the CPU, with bounds
on what the GPU's arithmetic may differ by."""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # half a step at zero


def rotate(x, pos, inv_freq, factor=1.0, interleaved=False, inverse=False):
    """Rotated x [rows, heads, d], and the bound on fp32 arithmetic: the phase
    is rounded to 2^-25 half turns (an angle of 1e-7), sine and cosine to two
    units in 2^-24, products and their sum to 2^-24 each; 2^-20 of |a| + |b|
    covers their sum (about 2^-21.3)."""
    y = x.double().clone()
    rot = 2 * inv_freq.numel()
    t = pos.double()[:, None, None] * inv_freq * (-1 if inverse else 1)
    c, s = t.cos() * factor, t.sin() * factor
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = y[..., ia], y[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    err = torch.zeros_like(y)
    err[..., ia] = err[..., ib] = (a.abs() + b.abs()) * factor * 2.0 ** -20
    return y, err


def e4m3_table():
    """Values of the 256 bytes, from the format: sign, 4 exponent bits (bias
    7), 3 mantissa bits, the two all-ones codes NaN."""
    out = []
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        v = math.nan if e == 15 and m == 7 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out.append(-v if b & 128 else v)
    return torch.tensor(out, dtype=torch.float64)


TABLE = e4m3_table()


def scale_exponent(amax):
    """Least e with amax <= 448 * 2^e, at least -60, 0 for zero (plain search)."""
    if amax == 0:
        return 0
    e = -60
    while amax > 448 * 2.0 ** e:
        e += 1
    return e


def quantise(x):
    """Bytes and exponents of rows x [..., d] in 64 bits, by a search of the
    nearest table value, ties to the even code."""
    x = x.double()
    e = torch.tensor([scale_exponent(v) for v in x.abs().amax(-1).flatten().tolist()],
                     dtype=torch.float64).view(x.shape[:-1])
    y = x * torch.exp2(-e)[..., None]
    pos = TABLE[:127]
    mag = y.abs().contiguous()
    hi = torch.searchsorted(pos, mag).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = mag - pos[lo], pos[hi] - mag
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = code + 128 * (torch.signbit(y)).long()
    return code.to(torch.uint8), (e + 127).to(torch.uint8)


def dequantise(pages, scales):
    """64-bit values of a pool (16-bit, or bytes with scale bytes)."""
    if scales is None:
        return pages.double()
    return TABLE[pages.view(torch.uint8).long()] * torch.exp2(scales.view(torch.uint8).double() - 127)[..., None]


def keys_of(cache, b, lo, hi):
    """Flat pool rows of keys lo .. hi - 1 of sequence b."""
    ps = cache.k_pages.shape[1]
    j = torch.arange(lo, hi)
    return cache.page_indices.long()[int(cache.page_indptr[b]) + j // ps] * ps + j % ps


def attention(q, cache, cu, pre, scale, window=0, sinks=None, smooth=False, keep=None, depths=None):
    """out, lse in 64 bits and their bounds.  keep: per sequence a boolean
    matrix over the new tokens, or None.

    The bound on out, element-wise: the output's own rounding; the rounding of
    each probability to 16 bits (u_p, against sum p |v|); and the relative
    error rho of a probability in fp32, which enters numerator and
    denominator: the scores' sums (d products of fp32 accuracy, the scaled
    query's 2^-25), the exponential (2^-22) and its argument's rounding
    (|s| 2^-23 in the log2 domain), the sums over the keys (n 2^-24)."""
    kd = dequantise(cache.k_pages, cache.k_scales).flatten(0, 1)
    vd = dequantise(cache.v_pages, cache.v_scales).flatten(0, 1)
    total, hq, d = q.shape
    hkv = kd.shape[1]
    g = hq // hkv
    out, lse = torch.zeros(total, hq, d, dtype=torch.float64), torch.full((total, hq), math.nan, dtype=torch.float64)
    bo, bl = torch.zeros_like(out), torch.zeros_like(lse)
    u_p = 2.0 ** -11 if cache.k_scales is not None else U[q.dtype]
    for b in range(len(pre)):
        lo, hi = cu[b], cu[b + 1]
        n, p = hi - lo, pre[b]
        if n == 0:
            continue
        rows = keys_of(cache, b, 0, p + n)
        k = kd[rows].repeat_interleave(g, 1).transpose(0, 1)
        v = vd[rows].repeat_interleave(g, 1).transpose(0, 1)
        qb = q[lo:hi].double().transpose(0, 1)
        ok = torch.ones(n, p + n, dtype=torch.bool).tril(p)
        if keep is not None:
            ok[:, p:] &= torch.as_tensor(keep[b])
        dep = list(range(n)) if depths is None else list(depths[b])
        if window > 0:
            place = torch.tensor(list(range(p)) + [p + x for x in dep])
            ok &= place[None] > p + torch.tensor(dep)[:, None] - window
        # keys no row sees may hold anything: take zeros for them
        seen = ok.any(0)
        k, v = k * seen[None, :, None], v * seen[None, :, None]
        k[:, ~seen], v[:, ~seen] = 0, 0
        s = qb @ k.transpose(1, 2) * scale
        s = s.masked_fill(~ok, -math.inf)
        x = torch.full((hq, 1, 1), -math.inf, dtype=torch.float64)
        if sinks is not None:
            x = sinks.double().cpu().view(hq, 1, 1)
        elif smooth:
            x = torch.zeros(hq, 1, 1, dtype=torch.float64)
        full = torch.cat((s, x.expand(hq, n, 1)), -1)
        any_key = ok.any(-1)[None].expand(hq, n)
        m = torch.where(any_key, full.amax(-1), torch.zeros(()).double())
        e = (s - m[..., None]).exp()
        den = e.sum(-1) + (x[..., 0] - m).exp()
        o = torch.where(any_key[..., None], e @ v / den[..., None], torch.zeros(()).double())
        z = torch.where(any_key, m + den.log(), torch.full((), -math.inf).double())
        av = torch.where(any_key[..., None], e @ v.abs() / den[..., None], torch.zeros(()).double())
        sa = (qb.abs() @ k.abs().transpose(1, 2) * scale).amax(-1)
        qk = qb.abs().amax(-1) * k.abs().sum(-1).amax(-1)[:, None] * scale
        rho = d * 2.0 ** -24 * sa + 2.0 ** -24 * qk + 2.0 ** -22 + sa * 2.0 ** -22 + (p + n) * 2.0 ** -24
        vmax = v.abs().amax() if v.numel() else 0.0
        bound = U[q.dtype] * o.abs() + (1 + U[q.dtype]) * (u_p + 2.5 * rho[..., None]) * av
        bound += TINY[q.dtype] + (p + n) * 2.0 ** -30 * vmax
        out[lo:hi], lse[lo:hi] = o.transpose(0, 1), z.transpose(0, 1)
        bo[lo:hi] = bound.transpose(0, 1)
        bl[lo:hi] = (2 * rho + 2.0 ** -22 * z.abs().nan_to_num(posinf=0)).transpose(0, 1)
    return out, lse, bo, bl


def fill(cache, batch, seed=0, spread=2):
    """Random contents for a whole pool: normal values, rows scaled by powers
    of two, in the pool's own type."""
    gen = torch.Generator().manual_seed(seed)
    shape = cache.k_pages.shape
    for x in "kv":
        y = torch.randn(shape, generator=gen)
        pages, scales = getattr(cache, x + "_pages"), getattr(cache, x + "_scales")
        if scales is None:
            pages.copy_(y.to(pages.dtype))
        else:
            e = torch.randint(120 - spread, 121 + spread, shape[:3], generator=gen)
            pages.copy_((y * 100).clamp(-448, 448).to(torch.float8_e4m3fn))
            scales.copy_(e.to(torch.uint8))
    return cache


def on_gpu(cache):
    import dataclasses
    return dataclasses.replace(cache, **{f: (t.cuda() if t is not None else None) for f, t in (
        (n, getattr(cache, n)) for n in ("k_pages", "v_pages", "k_scales", "v_scales", "page_indptr",
                                         "page_indices"))})
