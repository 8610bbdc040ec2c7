"""Cases of the operators beside the attention when its layer is trained: the
gradient of the attention, the root-mean-square norm of hidden rows or of query
heads (with the residual's addition, and an output in 16 bits or in e4m3 with
power-of-two scales), and the norm's gradient.

``own`` False computes them in elementary torch operations, ``own`` True
through the package's entry points.  Shapes follow the package's own
workloads: 64 / 8 heads of 64, window 128, prompts of 4k to 16k tokens.
"""
import math
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One full-attention layer of a 4k training sequence, with per-head sinks.
        dict(name="attention full", op="attention", pre="0", new="4096", hq=64, hkv=8, d=64, dtype="bf16", window=0,
             sink="head"),
        # The sliding-window layer beside it.
        dict(name="attention window", op="attention", pre="0", new="4096", hq=64, hkv=8, d=64, dtype="bf16",
             window=128, sink="head"),
        # Packed sequences of very different lengths, wide heads, the "+1" in the denominator.
        dict(name="attention ragged", op="attention", pre="0 0 0 0 0", new="1000 37 1 2047 513", hq=32, hkv=8, d=128,
             dtype="f16", window=0, sink="smooth"),
        # Chunks trained behind long prefixes, whose keys take gradients too.
        dict(name="attention chunks", op="attention", pre="8192 5001", new="300 255", hq=64, hkv=8, d=64, dtype="bf16",
             window=0, sink="none"),
        # Two short sequences of very wide heads: latency.
        dict(name="attention short", op="attention", pre="0 3", new="37 5", hq=8, hkv=4, d=256, dtype="bf16", window=0,
             sink="none"),
        # The norm in front of a layer's projections over a 16k prompt, adding the block before it.
        dict(name="norm prompt", op="norm", rows=16384, heads=1, n=4096, dtype="bf16", stream="bf16", residual=True,
             group=0, offset=0.0, weight="bf16"),
        # One decoded token, for a projection in 8 bits.
        dict(name="norm token", op="norm", rows=1, heads=1, n=4096, dtype="bf16", stream="bf16", residual=True,
             group=128, offset=0.0, weight="bf16"),
        # A ragged batch over a 32-bit residual stream, for a projection in 8 bits.
        dict(name="norm quantised", op="norm", rows=2047, heads=1, n=5120, dtype="f16", stream="f32", residual=True,
             group=32, offset=1.0, weight="f32"),
        # The norm of each query head, read from the packed projection, before its rotation.
        dict(name="norm heads", op="norm", rows=16384, heads=64, n=64, dtype="bf16", stream="bf16", residual=False,
             group=0, offset=0.0, weight="f32"),
        # The gradient of the prompt's norm, with what comes down the residual stream.
        dict(name="norm gradient", op="gradient", rows=16384, heads=1, n=4096, dtype="bf16", stream="bf16",
             residual=True, offset=0.0, weight="bf16"),
        # The gradient of the norm of query heads.
        dict(name="head gradient", op="gradient", rows=4095, heads=32, n=128, dtype="f16", stream="f16",
             residual=False, offset=0.0, weight="f32"),
        # A few rows of an odd width over a 32-bit residual stream: latency.
        dict(name="small gradient", op="gradient", rows=33, heads=1, n=1000, dtype="bf16", stream="f32", residual=True,
             offset=1.0, weight="bf16"),
    ]


def draw(rng):
    def spread(lo, hi):  # uniform in the logarithm
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    dtype = rng.choice(["bf16", "f16"])
    op = rng.choice(["attention", "attention", "norm", "gradient"])
    if op == "attention":
        d = rng.choice([64, 64, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 8])
        seqs = rng.choice([1, 1, 2, 3, 7])
        new = [spread(1, 4096) for _ in range(seqs)]
        pre = [rng.choice([0, 0, 0, spread(1, 8192)]) for _ in range(seqs)]
        # No more products, and no more memory in 32 bits, than 4096 tokens of 64 heads of 64 take.
        while seqs * max(new) * (max(new) + max(pre)) * hq * d > 4096 * 4096 * 64 * 64:
            new, pre = [(n + 1) // 2 for n in new], [p // 2 for p in pre]
        new[0] = max(new[0], 2)  # a token that sees one key alone, and no sink, has no gradient but of its value
        return dict(op=op, pre=" ".join(map(str, pre)), new=" ".join(map(str, new)), hq=hq, hkv=hkv, d=d, dtype=dtype,
                    window=rng.choice([0, 0, 128, spread(2, 2000)]), sink=rng.choice(["head", "smooth", "none"]))
    if rng.random() < 0.3:
        heads, n = rng.choice([1, 3, 8, 32, 64]), rng.choice([64, 128, 256])
        stream, residual = dtype, False
    else:
        heads, n = 1, 8 * spread(8, 2048)
        stream, residual = rng.choice([dtype, "f32"]), True
    rows = spread(1, max(2, min(16384, 16384 * 4096 // (heads * n * (2 if stream == "f32" else 1)))))
    c = dict(op=op, rows=rows, heads=heads, n=n, dtype=dtype, stream=stream, residual=residual,
             offset=rng.choice([0.0, 1.0]), weight=rng.choice([dtype, "f32"]))
    if op == "norm":  # a 16-bit output, or e4m3 with a scale for each `group` values
        c["group"] = rng.choice([0, 0] + [g for g in (32, 64, 128, n) if n % g == 0])
    return c


def _lengths(c):
    return [int(x) for x in c["pre"].split()], [int(x) for x in c["new"].split()]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DT[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = {"case": c}
    if c["op"] == "attention":
        pre, new = _lengths(c)
        hq, hkv, d = c["hq"], c["hkv"], c["d"]
        keys = [p + n for p, n in zip(pre, new)]

        def starts(lens):
            return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=dev)

        s["q"], s["dout"] = normal(sum(new), hq, d).to(dt), normal(sum(new), hq, d).to(dt)
        s["k"], s["v"] = normal(sum(keys), hkv, d).to(dt), normal(sum(keys), hkv, d).to(dt)
        s["cu"], s["kv_indptr"] = starts(new), starts(keys)
        s["prefix_lens"] = torch.tensor(pre, dtype=torch.int32, device=dev)
        s["sinks"] = normal(hq) if c["sink"] == "head" else None
        s["max_new"], s["max_keys"] = max(new), max(keys)
        # What the forward pass left: out and the logarithm of the denominator.
        p, lse, _, vs, place = _probabilities(s)
        s["out"] = _rows(p @ vs, place, c).to(dt)
        s["lse"] = _rows(lse[..., None], place, c)[..., 0].contiguous()
        s["dq"], s["dk"], s["dv"] = torch.empty_like(s["q"]), torch.empty_like(s["k"]), torch.empty_like(s["v"])
        s["dsinks"] = torch.empty(hq, device=dev) if c["sink"] == "head" else None
        return s

    rows, heads, n, stream = c["rows"], c["heads"], c["n"], DT[c["stream"]]
    s["weight"] = (1.0 - c["offset"] + 0.2 * normal(n)).to(DT[c["weight"]])
    if c["op"] == "norm":
        # Heads come from a packed projection with the keys' and values' heads behind them.
        packed = normal(rows, heads + (16 if heads > 1 else 0), n).to(dt)
        s["x"] = packed[:, :heads]
        s["residual"] = (4.0 * normal(rows, heads, n)).to(stream) if c["residual"] else None
        s["h"] = torch.empty(rows, heads, n, dtype=stream, device=dev) if c["residual"] else None
        s["rstd"] = torch.empty(rows, heads, device=dev)
        s["y"] = torch.empty(rows, heads, n, dtype=torch.float8_e4m3fn if c["group"] else dt, device=dev)
        s["scales"] = torch.empty(rows, heads, n // c["group"], dtype=torch.uint8, device=dev) if c["group"] else None
        return s
    s["h"] = (4.0 * normal(rows, heads, n)).to(stream)
    s["rstd"] = (s["h"].float().square().mean(-1) + EPS).rsqrt()
    s["dy"] = normal(rows, heads, n).to(dt)
    s["dh"] = normal(rows, heads, n).to(stream) if c["residual"] else None
    s["dx"] = torch.empty(rows, heads, n, dtype=dt, device=dev)
    s["dresidual"] = torch.empty(rows, heads, n, dtype=stream, device=dev) if c["stream"] != c["dtype"] else None
    s["dweight"] = torch.empty(n, device=dev)
    return s


# ------------------------------------------------------------------ plain forms
def _probabilities(s):
    """Padded to [sequence, KV head, token, query head of it, key], in 32 bits: the probabilities, lse, the scores'
    query rows, values, and where each padded token and key stands among the rows."""
    c = s["case"]
    n, length, hq, hkv, d = s["max_new"], s["max_keys"], c["hq"], c["hkv"], c["d"]
    g, dev = hq // hkv, s["q"].device
    pre, cu, kvi = s["prefix_lens"].long(), s["cu"].long(), s["kv_indptr"].long()
    i, j = torch.arange(n, device=dev), torch.arange(length, device=dev)
    new, keys = cu[1:] - cu[:-1], kvi[1:] - kvi[:-1]
    row = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)  # [B, n]
    key = (kvi[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)
    qs = s["q"][row].float().unflatten(2, (hkv, g)).permute(0, 2, 1, 3, 4)  # [B, hkv, n, g, d]
    ks, vs = (s[x][key].float().permute(0, 2, 1, 3)[:, :, None] for x in "kv")  # [B, hkv, 1, L, d]
    at = (pre[:, None] + i)[:, :, None]
    keep = (j <= at) & (i[:, None] < new[:, None, None]) & (j < keys[:, None, None])
    if c["window"] > 0:
        keep &= j > at - c["window"]
    score = (qs @ ks.transpose(-1, -2)).mul_(d ** -0.5).masked_fill_(~keep[:, None, :, None], -math.inf)
    sink = s["sinks"] if c["sink"] == "head" else torch.full((hq,), 0.0 if c["sink"] == "smooth" else -math.inf, device=dev)
    top = score.amax(-1).maximum(sink.view(hkv, 1, g)).clamp(min=-1e30)
    if "lse" in s:
        lse = s["lse"][row].unflatten(2, (hkv, g)).permute(0, 2, 1, 3)
    else:
        lse = top + ((score - top[..., None]).exp().sum(-1) + (sink.view(hkv, 1, g) - top).exp()).log()
    p = score.sub_(lse[..., None]).exp_().masked_fill_(~keep[:, None, :, None], 0.0)
    return p, lse, qs, vs, (row, key, i < new[:, None], j < keys[:, None])


def _rows(x, place, c):
    """[B, hkv, n, g, d] back to the rows [tokens, hq, d]."""
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)[place[2]]


def _plain_attention(s):
    c, dt = s["case"], s["q"].dtype
    g = c["hq"] // c["hkv"]
    p, lse, qs, vs, place = _probabilities(s)
    row, key, real, real_key = place
    split = lambda x: x[row].float().unflatten(2, (c["hkv"], g)).permute(0, 2, 1, 3, 4)  # noqa: E731
    do = split(s["dout"]).masked_fill(~real[:, None, :, None, None], 0.0)
    delta = (do * split(s["out"])).sum(-1)
    dv = p.flatten(2, 3).transpose(-1, -2) @ do.flatten(2, 3)  # [B, hkv, L, d]
    ds = (do @ vs.transpose(-1, -2)).sub_(delta[..., None]).mul_(p)
    del p
    ks = s["k"][key].float().permute(0, 2, 1, 3)
    dq = (ds.flatten(2, 3) @ ks).unflatten(2, qs.shape[2:4]) * c["d"] ** -0.5
    dk = ds.flatten(2, 3).transpose(-1, -2) @ qs.flatten(2, 3) * c["d"] ** -0.5
    out = [_rows(dq, place, c).to(dt)] + [x.transpose(1, 2)[real_key].to(dt) for x in (dk, dv)]
    if s["sinks"] is not None:  # a sum over every row: in 64 bits
        weight = (s["sinks"].view(c["hkv"], 1, g) - lse).exp().masked_fill(~real[:, None, :, None], 0.0)
        out.append(-(weight * delta).double().sum((0, 2)).flatten().float())
    return out


def _plain_norm(s):
    c = s["case"]
    h, out = s["x"], []
    if c["residual"]:
        h = (h.float() + s["residual"].float()).to(s["residual"].dtype)
        out.append(h)
    h = h.float()
    rstd = (h.square().mean(-1) + EPS).rsqrt()
    y = h * rstd[..., None] * (s["weight"].float() + c["offset"])
    if not c["group"]:
        return out + [rstd, y.to(s["x"].dtype)]
    y = y.unflatten(-1, (-1, c["group"]))
    mant, e = torch.frexp(y.abs().amax(-1))  # mant in [0.5, 1): the least power of two that keeps the group within 448
    e = (e - 9 + (mant > 0.875).int()).clamp(-60, 127)
    e = torch.where(mant == 0, torch.zeros_like(e), e)
    y = torch.ldexp(y, -e[..., None]).flatten(-2).to(torch.float8_e4m3fn)
    return out + [rstd, y, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)]


def _plain_gradient(s):
    c = s["case"]
    near, dy = s["h"].float() * s["rstd"][..., None], s["dy"].float()
    g = dy * (s["weight"].float() + c["offset"])
    dh = s["rstd"][..., None] * (g - near * (g * near).mean(-1, keepdim=True))
    if s["dh"] is not None:
        dh = dh + s["dh"].float()
    dw = (dy * near).flatten(0, 1).double().sum(0).float()  # a sum over every row: in 64 bits
    return [dh.to(s["dx"].dtype)] + ([dh] if s["dresidual"] is not None else []) + [dw]


# ------------------------------------------------------------------ one pass
def run(s):
    c, op = s["case"], s["case"]["op"]
    if not own:
        return {"attention": _plain_attention, "norm": _plain_norm, "gradient": _plain_gradient}[op](s)
    import gqa_flash_attention_prefill_gb300 as gqa
    call = s.get("call")  # marshalled at the first pass, as a program does for the buffers of a layer
    if call is None:
        if op == "attention":
            size = gqa.prefill_backward_workspace(s["prefix_lens"].numel(), s["q"].shape[0], s["k"].shape[0], c["hq"],
                                                  c["hkv"], c["d"], c["dtype"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
            call = gqa.prepare_call(gqa.gqa_prefill_backward, s["q"], s["k"], s["v"], s["cu"], s["prefix_lens"],
                                    s["kv_indptr"], c["d"] ** -0.5, s["out"], s["lse"], s["dout"], s["dq"], s["dk"],
                                    s["dv"], s["workspace"], window=c["window"], sinks=s["sinks"],
                                    dsinks=s["dsinks"])
        elif op == "norm":
            call = gqa.prepare_call(gqa.gqa_rms_norm, s["x"], s["weight"], s["y"], eps=EPS, offset=c["offset"],
                                    residual=s["residual"], residual_out=s["h"], scales=s["scales"], rstd=s["rstd"])
        else:
            size = gqa.rms_norm_backward_workspace(c["rows"], c["heads"], c["n"], c["dtype"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
            call = gqa.prepare_call(gqa.gqa_rms_norm_backward, s["dy"], s["h"], s["weight"], s["rstd"], s["dx"],
                                    dresidual=s["dresidual"], dweight=s["dweight"], workspace=s["workspace"],
                                    offset=c["offset"], dh=s["dh"])
        s["call"] = call
    call()
    if op == "attention":
        return [s["dq"], s["dk"], s["dv"]] + ([s["dsinks"]] if s["dsinks"] is not None else [])
    if op == "norm":
        return ([s["h"]] if c["residual"] else []) + [s["rstd"], s["y"]] + (
            [s["scales"].view(torch.float8_e8m0fnu)] if c["group"] else [])
    return [s["dx"]] + ([s["dresidual"]] if s["dresidual"] is not None else []) + [s["dweight"]]


# ------------------------------------------------------------------ what a pass has to do
def work(case):
    c = case
    if c["op"] == "attention":
        pre, new = _lengths(c)
        pairs = 0  # keys that the tokens of each sequence see
        for p, n in zip(pre, new):
            far = c["window"] or p + n
            short = max(0, min(n, far - p))  # tokens that see every key before them
            pairs += short * p + short * (short + 1) // 2 + (n - short) * far
        tokens, keys = sum(new), sum(pre) + sum(new)
        return {"bytes": 2 * c["d"] * (4 * c["hq"] * tokens + 4 * c["hkv"] * keys) + 4 * c["hq"] * tokens,
                "flops": 10 * c["d"] * c["hq"] * pairs}
    values = c["rows"] * c["heads"] * c["n"]
    e, es = 2, 4 if c["stream"] == "f32" else 2
    if c["op"] == "norm":
        out = 1 + 1 / c["group"] if c["group"] else e
        each = e + out + (2 * es if c["residual"] else 0)
    else:
        each = 2 * e + es + (es if c["residual"] else 0) + (es if c["stream"] != c["dtype"] else 0)
    return {"bytes": values * each + 4 * c["rows"] * c["heads"] + 4 * c["n"], "flops": 8 * values}


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "attention":
        pre, new = _lengths(c)
        g, scale = c["hq"] // c["hkv"], 1.0 / math.sqrt(c["d"])
        grads = [torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (s["q"], s["k"], s["v"])]
        dsinks = torch.zeros(c["hq"], dtype=torch.float64, device="cuda")
        t0 = k0 = 0
        for p, n in zip(pre, new):
            ts, kslice = slice(t0, t0 + n), slice(k0, k0 + p + n)
            hidden = torch.ones(n, p + n, dtype=torch.bool, device="cuda").triu(p + 1)
            if c["window"]:
                hidden |= torch.ones_like(hidden).tril(p - c["window"])
            for h in range(c["hq"]):
                q, do, o = (s[x][ts, h].double() for x in ("q", "dout", "out"))
                k, v = (s[x][kslice, h // g].double() for x in "kv")
                lse = s["lse"][ts, h].double()
                prob = torch.exp(q @ k.T * scale - lse[:, None]).masked_fill(hidden, 0.0)
                delta = torch.einsum("nd,nd->n", do, o)
                slope = prob * (do @ v.T - delta[:, None]) * scale
                grads[0][ts, h] = slope @ k
                grads[1][kslice, h // g] += slope.T @ q
                grads[2][kslice, h // g] += prob.T @ do
                if s["sinks"] is not None:
                    dsinks[h] -= torch.exp(s["sinks"][h].double() - lse) @ delta
            t0, k0 = t0 + n, k0 + p + n
        return grads + ([dsinks] if s["sinks"] is not None else [])

    w = s["weight"].double() + c["offset"]
    if c["op"] == "norm":
        h, out = s["x"].double(), []
        if c["residual"]:
            h = (h + s["residual"].double()).to(s["residual"].dtype).double()  # held in the stream's type
            out.append(h)
        rstd = 1.0 / torch.sqrt(torch.linalg.vector_norm(h, dim=-1) ** 2 / c["n"] + EPS)
        y = torch.einsum("rhn,rh,n->rhn", h, rstd, w)
        if not c["group"]:
            return out + [rstd, y]
        y = y.view(*y.shape[:2], -1, c["group"])
        most = y.abs().amax(-1, keepdim=True)
        e = torch.ceil(torch.log2(most / 448)).clamp(-60, 127)
        e = torch.where(most == 0, torch.zeros_like(e), e)
        y = y * torch.exp2(-e)
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        return out + [rstd, (torch.round(y / step) * step).view(s["y"].shape), torch.exp2(e[..., 0])]

    # The row's Jacobian, written as a projection: rstd (g - (h . g) h rstd^2 / n).
    h, rstd, dy = s["h"].double(), s["rstd"].double()[..., None], s["dy"].double()
    g = dy * w
    dh = rstd * g - h * (rstd ** 3 * torch.einsum("rhn,rhn->rh", h, g)[..., None] / c["n"])
    if s["dh"] is not None:
        dh += s["dh"].double()
    dw = torch.einsum("rhn,rhn,rh->n", dy, h, rstd[..., 0])
    return [dh] + ([dh] if s["dresidual"] is not None else []) + [dw]
