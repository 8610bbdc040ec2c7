"""Cases of the serving-side operators around a paged key/value cache: rotary
positions, writing a cache (16-bit, or e4m3 with one power-of-two scale per
token and head), reading it back, and the attention of a few new tokens (one
decoded token, or a tree of drafted ones) over it.

``own`` False computes them in elementary torch operations, ``own`` True
through the package's entry points.  Shapes follow the package's own
workloads: 64 / 8 heads of 64, window 128, prefixes of 1k to 16k tokens.
"""
import math
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One layer's query and key heads of a 16k prompt, positions up to 128k.
        dict(name="rope prompt", op="rope", rows=16384, hq=64, hkv=8, d=64, rot=64, dtype="bf16", interleaved=False,
             inverse=False, scaled=True, far=131072),
        # The gradient of the same step in a smaller model: part of the head, interleaved pairs.
        dict(name="rope gradient", op="rope", rows=2047, hq=32, hkv=8, d=128, rot=96, dtype="f16", interleaved=True,
             inverse=True, scaled=False, far=8192),
        # A decode step of 64 sequences: one token each, rotated and quantised into its page.
        dict(name="write decode", op="write", seqs=64, pre_lo=0, pre_hi=500, new_lo=1, new_hi=1, lens=1, hq=64, hkv=8,
             d=64, rot=64, dtype="bf16", cache="e4m3", page=16, interleaved=False),
        # A ragged prompt batch, written at once from the packed projection.
        dict(name="write prompt", op="write", seqs=6, pre_lo=0, pre_hi=1000, new_lo=700, new_hi=2600, lens=2, hq=64,
             hkv=8, d=64, rot=64, dtype="bf16", cache="e4m3", page=64, interleaved=False),
        # Drafted tokens of wide heads into a 16-bit cache, without positions.
        dict(name="write drafts", op="write", seqs=16, pre_lo=1, pre_hi=300, new_lo=3, new_hi=7, lens=3, hq=8, hkv=4,
             d=256, rot=0, dtype="f16", cache="16", page=8, interleaved=False),
        # The cached prefixes of a chunked prefill, back to 16 bits for the prefill kernel.
        dict(name="read prefix", op="read", seqs=8, pre_lo=8192, pre_hi=8192, lens=4, hkv=8, d=64, dtype="bf16",
             cache="e4m3", page=64, tail=0),
        # The last 128 keys of each sequence, for a sliding-window layer.
        dict(name="read window", op="read", seqs=64, pre_lo=40, pre_hi=2000, lens=5, hkv=2, d=128, dtype="f16",
             cache="e4m3", page=16, tail=128),
        # One user with a long context, one token at a time.
        dict(name="decode long", op="attention", seqs=1, pre_lo=131071, pre_hi=131071, new_lo=1, new_hi=1, lens=6,
             hq=64, hkv=8, d=64, dtype="bf16", cache="e4m3", page=64, window=0, sink="head", tree=False),
        # A sliding-window layer's decode step.
        dict(name="decode window", op="attention", seqs=128, pre_lo=1024, pre_hi=16384, new_lo=1, new_hi=1, lens=7,
             hq=64, hkv=8, d=64, dtype="bf16", cache="16", page=16, window=128, sink="head", tree=False),
        # A full-attention layer's decode step of a large batch.
        dict(name="decode batch", op="attention", seqs=256, pre_lo=1024, pre_hi=16384, new_lo=1, new_hi=1, lens=8,
             hq=64, hkv=8, d=64, dtype="bf16", cache="e4m3", page=64, window=0, sink="head", tree=False),
        # Verification of 64-token draft trees over 8k prefixes.
        dict(name="verify trees", op="attention", seqs=8, pre_lo=8192, pre_hi=8192, new_lo=64, new_hi=64, lens=9,
             hq=64, hkv=8, d=64, dtype="bf16", cache="e4m3", page=64, window=0, sink="head", tree=True),
        # A few small trees in a smaller model with a 16-bit cache.
        dict(name="verify small", op="attention", seqs=5, pre_lo=200, pre_hi=2900, new_lo=3, new_hi=7, lens=10, hq=16,
             hkv=2, d=128, dtype="f16", cache="16", page=16, window=0, sink="smooth", tree=True),
    ]


def draw(rng):
    def spread(lo, hi):  # uniform in the logarithm
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "write", "read", "attention", "attention", "attention"])
    dtype = rng.choice(["bf16", "f16"])
    d = rng.choice([64, 64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 4, 8])
    page = rng.choice([8, 16, 16, 64, 128]) if hkv > 1 else rng.choice([16, 64])
    cache = rng.choice(["16", "e4m3"])
    lens = rng.randrange(1 << 30)
    inter = rng.random() < 0.4
    if op == "rope":
        rows = spread(1, 16384 * 4608 // ((hq + hkv) * d))
        return dict(op=op, rows=min(rows, 32768), hq=hq, hkv=hkv, d=d, rot=rng.choice([d, d, d // 2, d // 4 + 2]),
                    dtype=dtype, interleaved=inter, inverse=rng.random() < 0.4, scaled=rng.random() < 0.5,
                    far=spread(2000, 1000000))
    if op == "write":
        new_hi = spread(1, 2600)
        return dict(op=op, seqs=max(1, min(64, spread(1, 64), 12000 // new_hi)), pre_lo=0, pre_hi=spread(1, 1000),
                    new_lo=max(1, new_hi // 3), new_hi=new_hi, lens=lens, hq=hq, hkv=hkv, d=d,
                    rot=rng.choice([0, d, d // 2]), dtype=dtype, cache=cache, page=page, interleaved=inter)
    if op == "read":
        hi = spread(50, 8192)
        return dict(op=op, seqs=max(1, min(64, spread(1, 64), 65536 * 512 // (hi * hkv * d))), pre_lo=max(1, hi // 4),
                    pre_hi=hi, lens=lens, hkv=hkv, d=d, dtype=dtype, cache=cache, page=page,
                    tail=rng.choice([0, 0, 128]))
    hi = spread(100, 16384)
    new = rng.choice([1, 1, spread(2, 64)])
    room = 256 * 8704 * 512 // (2 * hi * hkv * d * max(1, new // 2))
    return dict(op=op, seqs=max(1, min(256, spread(1, 256), room)), pre_lo=max(1, hi // 8), pre_hi=hi,
                new_lo=max(1, new // 2), new_hi=new, lens=lens, hq=hq, hkv=hkv, d=d, dtype=dtype, cache=cache, page=page,
                window=rng.choice([0, 0, 128, 1000]), sink=rng.choice(["head", "smooth", "none"]),
                tree=new > 1 and rng.random() < 0.8)


def _lengths(c):
    """(prefix, new) tokens of each sequence, from the case alone."""
    r = random.Random(c["lens"])
    pre = [r.randint(c["pre_lo"], c["pre_hi"]) for _ in range(c["seqs"])]
    return pre, [r.randint(c["new_lo"], c["new_hi"]) if "new_lo" in c else 0 for _ in range(c["seqs"])]


def _frequencies(c):
    """Angle per position of each pair, in 64 bits, and the factor on the
    rotated values.  ``scaled``: the long-context blend (32 times the original
    4096 positions; fast pairs keep their frequency, slow ones are divided)."""
    rot = c["rot"]
    base, factor, original = (150000.0, 32.0, 4096.0) if c.get("scaled", True) else (10000.0, 1.0, 4096.0)
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    inv = base ** (-i / rot)
    if factor == 1.0:
        return inv, 1.0
    pair_of = [rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
    ramp = ((i / 2 - pair_of[0]) / max(pair_of[1] - pair_of[0], 1e-3)).clamp(0, 1)
    return inv / factor * ramp + inv * (1 - ramp), 0.1 * math.log(factor) + 1.0


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DT[c["dtype"]]
    d, hkv = c["d"], c["hkv"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = {"case": c}
    if c["op"] == "rope":
        s["q"], s["k"] = normal(c["rows"], c["hq"], d).to(dt), normal(c["rows"], hkv, d).to(dt)
        s["positions"] = torch.randint(0, c["far"], (c["rows"],), generator=gen, device=dev, dtype=torch.int32)
        inv, s["factor"] = _frequencies(c)
        s["inv_freq"] = inv.to(dev)
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        return s

    # The page table: each sequence's pages, scattered over the pool.
    pre, new = _lengths(c)
    keys = [p + n for p, n in zip(pre, new)]
    ps = c["page"]
    counts = torch.tensor([-(-n // ps) for n in keys])
    pages = int(counts.sum())
    i32 = dict(dtype=torch.int32, device=dev)

    def starts(lens):
        return torch.tensor([0] + list(torch.tensor(lens).cumsum(0).tolist()), **i32)

    s["page_indptr"] = starts(counts.tolist())
    s["page_indices"] = torch.randperm(pages + 2, generator=gen, device=dev)[:pages].to(torch.int32)
    s["prefix_lens"] = torch.tensor(pre, **i32)
    s["cu"] = starts(new)
    total = sum(new)

    def pool():
        """Pages as an earlier call left them: 16-bit values, or e4m3 values with their scales."""
        x = normal(pages + 2, ps, hkv, d)
        if c["cache"] == "16":
            return x.to(dt), None
        x *= torch.exp2(torch.randint(-2, 3, (pages + 2, ps, hkv, 1), generator=gen, device=dev).float())
        mant, e = torch.frexp(x.abs().amax(-1))
        e = (e - 9 + (mant > 0.875).int()).clamp(-60, 127)
        x = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn)
        return x, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)

    s["k_pages"], s["k_scales"] = pool()
    s["v_pages"], s["v_scales"] = pool()
    if c["op"] == "read":
        first = [max(0, n - c["tail"]) if c["tail"] else 0 for n in pre]
        s["first_keys"] = torch.tensor(first, **i32) if c["tail"] else None
        s["kv_indptr"] = starts([n - f for n, f in zip(pre, first)])
        rows = sum(n - f for n, f in zip(pre, first))
        s["k"], s["v"] = (torch.empty(rows, hkv, d, dtype=dt, device=dev) for _ in range(2))
    if c["op"] == "write":
        packed = normal(total, c["hq"] + 2 * hkv, d).to(dt)  # the projection's output
        s["q"], s["k"], s["v"] = packed.split([c["hq"], hkv, hkv], 1)
        if c["rot"]:
            inv, s["factor"] = _frequencies(c)
            s["inv_freq"] = inv.to(dev)
            s["q_out"] = torch.empty(total, c["hq"], d, dtype=dt, device=dev)
    if c["op"] == "attention":
        s["q"] = normal(total, c["hq"], d).to(dt)
        s["sinks"] = normal(c["hq"]) if c["sink"] == "head" else None
        s["max_new"], s["max_keys"] = max(new), max(keys)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(total, c["hq"], device=dev)
        s["mask"] = s["mask_indptr"] = s["depths"] = None
        if c["tree"]:  # draft trees: a token hangs under one drawn before it, and sees its ancestors
            r = random.Random(seed)
            words, at, depths = [], [0], []
            for n in new:
                w = -(-n // 32)
                bits, depth = [], []
                for t in range(n):
                    up = r.randrange(max(0, t - 8), t) if t else None
                    bits.append((0 if up is None else bits[up]) | 1 << t)
                    depth.append(0 if up is None else depth[up] + 1)
                words += [(b >> 32 * k) & 0xFFFFFFFF for b in bits for k in range(w)]
                at.append(at[-1] + n * w)
                depths += depth
            s["mask"] = torch.tensor([x - (1 << 32) if x >> 31 else x for x in words], **i32)
            s["mask_indptr"], s["depths"] = torch.tensor(at, **i32), torch.tensor(depths, **i32)
    return s


# ------------------------------------------------------------------ plain forms
def _turned(x, angle, factor, interleaved, inverse):
    """x [rows, heads, d] in 32 bits, its first 2 * angle.shape[1] values rotated."""
    cos, sin = (angle.cos() * factor).float()[:, None], (angle.sin() * factor).float()[:, None]
    sin = -sin if inverse else sin
    h = angle.shape[1]
    head, rest = x[..., :2 * h], x[..., 2 * h:]
    a, b = (head[..., 0::2], head[..., 1::2]) if interleaved else (head[..., :h], head[..., h:])
    lo, hi = a * cos - b * sin, b * cos + a * sin
    head = torch.stack((lo, hi), -1).flatten(-2) if interleaved else torch.cat((lo, hi), -1)
    return torch.cat((head, rest), -1)


def _plain_rope(s):
    c = s["case"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    return [_turned(x.float(), angle, s["factor"], c["interleaved"], c["inverse"]).to(x.dtype) for x in (s["q"], s["k"])]


def _quantised(x):
    """e4m3 values and the exponent of the scale: the least power of two that keeps the row within 448."""
    mant, e = torch.frexp(x.abs().amax(-1))  # mant in [0.5, 1)
    e = (e - 9 + (mant > 0.875).int()).clamp(-60, 127)
    e = torch.where(mant == 0, torch.zeros_like(e), e)
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _plain_write(s):
    c, ps = s["case"], s["case"]["page"]
    row = torch.arange(s["k"].shape[0], device=s["k"].device)
    b = torch.searchsorted(s["cu"][1:].long(), row, right=True)
    at = s["prefix_lens"][b] + row - s["cu"][b]
    slot = s["page_indices"][s["page_indptr"][b] + at // ps].long() * ps + at % ps
    out, k = [], s["k"].float()
    if c["rot"]:
        angle = at.double()[:, None] * s["inv_freq"]
        out.append(_turned(s["q"].float(), angle, s["factor"], c["interleaved"], False).to(s["q"].dtype))
        k = _turned(k, angle, s["factor"], c["interleaved"], False)
    if c["cache"] == "16":
        s["k_pages"].flatten(0, 1)[slot] = k.to(s["k"].dtype)
        s["v_pages"].flatten(0, 1)[slot] = s["v"]
        return out + [s["k_pages"], s["v_pages"]]
    (kq, ke), (vq, ve) = _quantised(k), _quantised(s["v"].float())
    s["k_pages"].view(torch.uint8).flatten(0, 1)[slot] = kq.view(torch.uint8)
    s["v_pages"].view(torch.uint8).flatten(0, 1)[slot] = vq.view(torch.uint8)
    s["k_scales"].view(torch.uint8).flatten(0, 1)[slot] = ke
    s["v_scales"].view(torch.uint8).flatten(0, 1)[slot] = ve
    return out + [s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"]]


def _values(pages, scales, page):
    """The values of the given pages, in 32 bits."""
    if scales is None:
        return pages[page].float()
    return pages.view(torch.uint8)[page].view(pages.dtype).float() * scales.view(torch.uint8)[page].view(scales.dtype).float()[..., None]


def _plain_read(s):
    ps = s["case"]["page"]
    row = torch.arange(s["k"].shape[0], device=s["k"].device)
    b = torch.searchsorted(s["kv_indptr"][1:].long(), row, right=True)
    at = row - s["kv_indptr"][b] + (0 if s["first_keys"] is None else s["first_keys"][b])
    slot = s["page_indices"][s["page_indptr"][b] + at // ps].long() * ps + at % ps
    return [_values(s[x + "_pages"].flatten(0, 1), None if s[x + "_scales"] is None else s[x + "_scales"].flatten(0, 1),
                    slot).to(s["k"].dtype) for x in "kv"]


def _plain_attention(s):
    c, ps, q = s["case"], s["case"]["page"], s["q"]
    n, length, hq, hkv, d = s["max_new"], s["max_keys"], c["hq"], c["hkv"], c["d"]
    pre, cu, dev = s["prefix_lens"].long(), s["cu"].long(), q.device
    new = cu[1:] - cu[:-1]
    entry = s["page_indptr"][:-1, None] + torch.arange(-(-length // ps), device=dev)
    page = s["page_indices"][entry.clamp(max=s["page_indices"].numel() - 1)]
    k, v = (_values(s[x + "_pages"], s[x + "_scales"], page.long()).flatten(1, 2) for x in "kv")  # [B, L, hkv, d]
    i, j = torch.arange(n, device=dev), torch.arange(k.shape[1], device=dev)
    row = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)  # [B, n]
    qs = q[row].float().unflatten(2, (hkv, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, hkv, n G, d]
    score = (qs @ k.permute(0, 2, 3, 1)).unflatten(2, (n, hq // hkv)) * d ** -0.5  # [B, hkv, n, G, L]
    x = (j - pre[:, None])[:, None]  # [B, 1, L]: index among the new tokens
    depth = i.expand(row.shape) if s["depths"] is None else s["depths"][row].long()
    x_in = x.clamp(min=0).minimum(new[:, None, None] - 1)
    keep = (x <= i[:, None]) & (i[:, None] < new[:, None, None])
    if s["mask"] is not None:
        width = (new + 31) // 32
        word = s["mask_indptr"][:-1].long()[:, None, None] + i[:, None] * width[:, None, None] + x_in // 32
        bit = s["mask"][word.clamp(max=s["mask"].numel() - 1)] >> (x_in % 32) & 1
        keep &= (x < 0) | (bit != 0)
    if c["window"] > 0:
        place = torch.where(x < 0, x, depth.gather(1, x_in[:, 0])[:, None])  # position minus the prefix's length
        keep &= place > depth[:, :, None] - c["window"]
    score = score.masked_fill(~keep[:, None, :, None], -math.inf)
    sink = s["sinks"].float() if s["sinks"] is not None else torch.full((hq,), 0.0 if c["sink"] == "smooth" else -math.inf, device=dev)
    sink = sink.view(hkv, 1, hq // hkv)
    top = score.amax(-1).maximum(sink).clamp(min=-1e30)
    p = (score - top[..., None]).exp()
    total = p.sum(-1) + (sink - top).exp()
    o = (p.flatten(2, 3) @ v.permute(0, 2, 1, 3)).unflatten(2, (n, hq // hkv)) / total[..., None]
    o, lse = o.permute(0, 2, 1, 3, 4).flatten(2, 3), (top + total.log()).permute(0, 2, 1, 3).flatten(2, 3)
    real = i < new[:, None]
    return [o[real].to(q.dtype), lse[real]]


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"rope": _plain_rope, "write": _plain_write, "read": _plain_read, "attention": _plain_attention}[op](s)
    import gqa_flash_attention_prefill_gb300 as gqa
    c = s["case"]
    call = s.get("call")  # marshalled at the first pass, as a program does for the buffers of a layer
    if call is None:
        if op == "rope":
            call = gqa.prepare_call(gqa.gqa_rope, s["q"], s["positions"], s["inv_freq"], s["q_out"], k=s["k"],
                                    k_out=s["k_out"], interleaved=c["interleaved"], attn_factor=s["factor"],
                                    inverse=c["inverse"])
        elif op == "write":
            rope = gqa.Rope(s["inv_freq"], interleaved=c["interleaved"], attn_factor=s["factor"], q=s["q"],
                            q_out=s["q_out"]) if c["rot"] else None
            call = gqa.prepare_call(gqa.gqa_cache_write, s["k"], s["v"], s["cu"], s["prefix_lens"], s["page_indptr"],
                                    s["page_indices"], s["k_pages"], s["v_pages"], k_scales=s["k_scales"],
                                    v_scales=s["v_scales"], rope=rope)
        elif op == "read":
            call = gqa.prepare_call(gqa.gqa_cache_read, s["k_pages"], s["v_pages"], s["page_indptr"], s["page_indices"],
                                    s["kv_indptr"], s["k"], s["v"], first_keys=s["first_keys"], k_scales=s["k_scales"],
                                    v_scales=s["v_scales"])
        else:
            size = gqa.cache_attention_workspace(c["seqs"], s["q"].shape[0], s["max_new"], c["hq"], c["hkv"], c["d"],
                                                 c["dtype"], c["cache"])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
            call = gqa.prepare_call(gqa.gqa_cache_attention, s["q"], s["k_pages"], s["v_pages"], s["cu"],
                                    s["prefix_lens"], s["page_indptr"], s["page_indices"], c["d"] ** -0.5,
                                    s["workspace"], window=c["window"], sinks=s["sinks"],
                                    smooth_softmax=c["sink"] == "smooth", k_scales=s["k_scales"],
                                    v_scales=s["v_scales"], custom_mask=s["mask"], mask_indptr=s["mask_indptr"],
                                    depths=s["depths"], out=s["out"], lse=s["lse"], max_seqlen_q=s["max_new"])
        s["call"] = call
    call()
    if op == "rope":
        return [s["q_out"], s["k_out"]]
    if op == "write":
        return ([s["q_out"]] if c["rot"] else []) + [s["k_pages"], s["v_pages"]] + (
            [s["k_scales"], s["v_scales"]] if c["cache"] == "e4m3" else [])
    if op == "read":
        return [s["k"], s["v"]]
    return [s["out"], s["lse"]]


# ------------------------------------------------------------------ what a pass has to do
def work(case):
    c = case
    d, hkv = c["d"], c["hkv"]
    if c["op"] == "rope":
        n = c["rows"] * (c["hq"] + hkv) * d
        return {"bytes": 4 * n + 4 * c["rows"], "flops": 3 * n}
    pre, new = _lengths(c)
    row = hkv * (2 * d if c["cache"] == "16" else d + 1)  # one token's keys, or values, in the cache
    if c["op"] == "write":
        n = sum(new)
        q = 4 * n * c["hq"] * d if c["rot"] else 0
        return {"bytes": 2 * n * (2 * hkv * d + row) + q, "flops": 6 * n * hkv * d + q}
    if c["op"] == "read":
        n = sum(min(p, c["tail"]) if c["tail"] else p for p in pre)
        return {"bytes": 2 * n * (row + 2 * hkv * d), "flops": 2 * n * hkv * d}
    far = c["window"] or 1 << 30
    seen = [min(p, far - 1) + n for p, n in zip(pre, new)]  # keys some row of the sequence needs
    pairs = [n * min(p + (n + 1) // 2, far) for p, n in zip(pre, new)]
    return {"bytes": 2 * row * sum(seen) + (4 * d + 4) * c["hq"] * sum(new), "flops": 4 * d * c["hq"] * sum(pairs)}


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c, d = case, case["d"]
    pre, new = _lengths(c) if c["op"] != "rope" else ([], [])

    def turned(x, pos):
        """Each pair as a complex number, times e^(i angle)."""
        y = x.double().clone()
        rot = c["rot"]
        angle = pos.double()[:, None, None] * s["inv_freq"]
        turn = torch.polar(torch.full_like(angle, s["factor"]), -angle if c.get("inverse") else angle)
        one = (slice(0, rot, 2), slice(1, rot, 2)) if c["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(y[..., one[0]].contiguous(), y[..., one[1]].contiguous()) * turn
        y[..., one[0]], y[..., one[1]] = z.real, z.imag
        return y

    if c["op"] == "rope":
        return [turned(s["q"], s["positions"]), turned(s["k"], s["positions"])]

    def places(b, lo, hi):
        """Rows of the pool that hold keys lo .. hi - 1 of sequence b."""
        j = torch.arange(lo, hi, device="cuda")
        return s["page_indices"].long()[int(s["page_indptr"][b]) + j // c["page"]] * c["page"] + j % c["page"]

    def held(x, at):
        y = s[x + "_pages"].flatten(0, 1)
        if c["cache"] == "16":
            return y[at].double()
        return y.view(torch.uint8)[at].view(y.dtype).double() * torch.exp2(
            s[x + "_scales"].view(torch.uint8).flatten(0, 1)[at].double() - 127)[..., None]

    if c["op"] == "read":
        tails = [(b, max(0, n - c["tail"]) if c["tail"] else 0, n) for b, n in enumerate(pre)]
        return [torch.cat([held(x, places(b, lo, hi)) for b, lo, hi in tails]) for x in "kv"]

    first = [sum(new[:b]) for b in range(len(new) + 1)]
    if c["op"] == "write":
        pos = torch.cat([torch.arange(p, p + n, device="cuda") for p, n in zip(pre, new)])
        at = torch.cat([places(b, p, p + n) for b, (p, n) in enumerate(zip(pre, new))])
        out = [turned(s["q"], pos)] if c["rot"] else []
        values, scales = [], []
        for x in "kv":
            y = turned(s[x], pos) if c["rot"] and x == "k" else s[x].double()
            pool = s[x + "_pages"].double().flatten(0, 1)
            if c["cache"] == "e4m3":
                most = y.abs().amax(-1, keepdim=True)
                e = torch.ceil(torch.log2(most / 448)).clamp(-60, 127)
                e = torch.where(most == 0, torch.zeros_like(e), e)
                y = y * torch.exp2(-e)
                step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
                y = torch.round(y / step) * step
                old = torch.exp2(s[x + "_scales"].view(torch.uint8).flatten(0, 1).double() - 127)
                old[at] = torch.exp2(e[..., 0])
                scales.append(old.view(s[x + "_scales"].shape))
            pool[at] = y
            values.append(pool.view(s[x + "_pages"].shape))
        return out + values + scales

    outs, lses = [], []
    g = c["hq"] // c["hkv"]
    for b, (p, n) in enumerate(zip(pre, new)):
        k, v = (held(x, places(b, 0, p + n)).repeat_interleave(g, 1).transpose(0, 1) for x in "kv")
        q = s["q"][first[b]:first[b + 1]].double().transpose(0, 1)
        t = q @ k.transpose(1, 2) / math.sqrt(d)
        allowed = torch.ones(n, p + n, dtype=torch.bool).tril(p)
        depth = list(range(n)) if s["depths"] is None else s["depths"][first[b]:first[b + 1]].tolist()
        if c["tree"]:
            w = -(-n // 32)
            at = int(s["mask_indptr"][b])
            word = s["mask"][at:at + n * w].cpu().view(n, w).repeat_interleave(32, 1)[:, :n]
            allowed[:, p:] &= (word >> (torch.arange(n) % 32) & 1) != 0
        if c["window"]:
            where = torch.tensor(list(range(p)) + [p + x for x in depth])
            allowed &= where[None] > p + torch.tensor(depth)[:, None] - c["window"]
        t = t.masked_fill(~allowed.to(t.device), -math.inf)
        if c["sink"] != "none":
            x = s["sinks"].double() if c["sink"] == "head" else torch.zeros(c["hq"], dtype=torch.float64, device="cuda")
            t = torch.cat((t, x[:, None, None].expand(-1, n, 1)), -1)
        lses.append(t.logsumexp(-1).transpose(0, 1))
        outs.append((torch.softmax(t, -1)[..., :p + n] @ v).transpose(0, 1))
    return [torch.cat(outs), torch.cat(lses)]
