"""The attention's gradient from its formula in 64 bits, and how far the kernels
may be from it, element by element."""
import torch


def visible(b, s):
    """[new, keys] truth table of sequence s of a batch."""
    P = int(b.prefix_lens[s])
    n = int(b.cu_seqlens_q[s + 1] - b.cu_seqlens_q[s])
    i = torch.arange(n, device=b.q.device)[:, None] + P
    j = torch.arange(P + n, device=b.q.device)[None]
    keep = j <= i
    if b.window > 0:
        keep = keep & (j > i - b.window)
    return keep


def forward(b):
    """out and lse in 64 bits."""
    g = b.hq // b.hkv
    out = torch.zeros(b.q.shape, dtype=torch.float64, device=b.q.device)
    lse = torch.full(b.q.shape[:2], -torch.inf, dtype=torch.float64, device=b.q.device)
    for s in range(b.num_seqs):
        ts, ks = _slices(b, s)
        if ts.stop == ts.start:
            continue
        keep = visible(b, s)
        for h in range(b.hq):
            x = (b.q[ts, h].double() @ b.k[ks, h // g].double().T * b.scale).masked_fill(~keep, -torch.inf)
            if b.sinks is not None or b.smooth:
                sink = b.sinks[h].double() if b.sinks is not None else torch.zeros((), dtype=torch.float64, device=x.device)
                x = torch.cat((x, sink.expand(x.shape[0], 1)), 1)
            lse[ts, h] = x.logsumexp(1)
            out[ts, h] = (x - lse[ts, h, None]).exp()[:, :keep.shape[1]] @ b.v[ks, h // g].double()
    return out, lse


def _slices(b, s):
    return (slice(int(b.cu_seqlens_q[s]), int(b.cu_seqlens_q[s + 1])),
            slice(int(b.kv_indptr[s]), int(b.kv_indptr[s + 1])))


def gradients(b, out, lse, dout, dlse=None, out_error=0.0):
    """(values, bounds) of dq, dk, dv and dsinks.  Rows outside every sequence are NaN in both.

    The bound of each element, with u half a step of the type and f = 2^-24:
      s     d fp32 additions:                    f (d + 3) scale sum |q| |k|
      p     exp of s - lse (3 roundings of either, 2^-22 for the exponential): a relative e_p
      D     d additions of |dout| |out| (and out_error relative in out, where out is not the forward's own rounding)
      ds    p (|dout . v - D| (e_p + 4 f) + f (d + 3) sum |dout| |v| + the error of D)
      p and ds are rounded to the type: u of each, times the other factor, and (f16) an absolute 2^-25 in units of
      their power of two: 2^-40 for p, 2^-38 times the largest |dout| |v| + |D| of the sequence and KV head for ds;
      sums over n terms in fp32, in any order: f (n + 8) of the sum of magnitudes; the result: u of it.
    """
    g, d = b.hq // b.hkv, b.d
    u = torch.finfo(b.q.dtype).eps / 2
    f = 2.0 ** -24
    f16 = b.q.dtype == torch.float16
    new = lambda x: [torch.full(x.shape, torch.nan, dtype=torch.float64, device=x.device) for _ in range(2)]  # noqa: E731
    (dq, eq), (dk, ek), (dv, ev) = new(b.q), new(b.k), new(b.v)
    dsink = torch.zeros(b.hq, dtype=torch.float64, device=b.q.device)
    esink = torch.zeros_like(dsink)
    for s in range(b.num_seqs):
        ts, ks = _slices(b, s)
        for x in (dq, eq):
            x[ts] = 0
        for x in (dk, ek, dv, ev):
            x[ks] = 0
        if ts.stop == ts.start:
            continue
        keep = visible(b, s)
        n_q, n_k = keep.shape
        for hk in range(b.hkv):
            k, v = b.k[ks, hk].double(), b.v[ks, hk].double()
            heads = range(hk * g, hk * g + g)
            most = (max(float(dout[ts, h].double().norm(dim=1).max()) for h in heads) * float(v.norm(dim=1).max())
                    + max(float((dout[ts, h].double() * out[ts, h].double()).sum(1).abs().max()) for h in heads))
            if dlse is not None:
                most += max(float(dlse[ts, h].abs().max()) for h in heads)
            for h in heads:
                q, do, o, le = (x[ts, h].double() for x in (b.q, dout, out, lse))
                sc = q @ k.T * b.scale
                p = torch.exp(sc - le[:, None]).masked_fill(~keep, 0.0)
                D = (do * o).sum(1)
                eD = (do.abs() * o.abs()).sum(1) * (f * (d + 3) + out_error)
                if dlse is not None:
                    D = D - dlse[ts, h].double()
                eD = eD + f * D.abs()
                dp = do @ v.T - D[:, None]
                ds = p * dp
                ep = f * (d + 3) * (q.abs() @ k.abs().T) * b.scale + 3 * f * (sc.abs() + le.abs()[:, None]) + 2.0 ** -22
                eds = p * (dp.abs() * (ep + 4 * f) + f * (d + 3) * (do.abs() @ v.abs().T) + eD[:, None])
                rp = (u + ep) * p + (2.0 ** -40 if f16 else 0.0) * keep
                rds = u * ds.abs() + (1 + u) * eds + (2.0 ** -38 * most if f16 else 0.0) * keep
                dq[ts, h] = ds @ k * b.scale
                eq[ts, h] = (rds @ k.abs() + f * (n_k + 8) * (ds.abs() @ k.abs())) * b.scale
                dk[ks, hk] += ds.T @ q * b.scale
                ek[ks, hk] += (rds.T @ q.abs() + f * (g * n_q + 8) * (ds.abs().T @ q.abs())) * b.scale
                dv[ks, hk] += p.T @ do
                ev[ks, hk] += rp.T @ do.abs() + f * (g * n_q + 8) * (p.T @ do.abs())
                if b.sinks is not None:
                    x = b.sinks[h].double()
                    w = torch.exp(x - le)
                    dsink[h] -= w @ D
                    ew = 2 * f * (x.abs() + le.abs()) + 2.0 ** -22
                    esink[h] += (w * (eD + D.abs() * (ew + 16 * f))).sum()
    esink = esink + f * dsink.abs()
    for x, e in ((dq, eq), (dk, ek), (dv, ev)):
        e += u * (x.abs() + e) + (2.0 ** -25 if f16 else 0.0)
    return (dq, dk, dv, dsink), (eq, ek, ev, esink)


def check(got, want, bounds, names=("dq", "dk", "dv", "dsinks")):
    """Every element of a sequence within its bound."""
    for name, x, y, e in zip(names, got, want, bounds):
        if x is None:
            continue
        real = ~y.isnan()
        assert bool(x[real].isfinite().all()), f"{name}: not finite"
        off = (x.double() - y).abs()[real] / e[real].clamp(min=1e-300)
        assert off.numel() == 0 or float(off.max()) <= 1.0, f"{name}: {float(off.max()):.3f} times the bound"
