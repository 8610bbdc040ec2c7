"""The operators in the order in which a layer uses them: residual and norm, projections, the heads' norms, rotation,
attention, and back through all of them; and a decoded token after the same prompt, over a cache.

The reference is the same layer in 64 bits, differentiated by autograd.  Its tolerance is made with it: every tensor
that the operators keep in 16 bits, forward and backward (P and dS inside the attention among them), is multiplied by
1 + x with x at random in [-u, u], u half a step of the type.  The norm of what that does to a result is the norm that the
roundings' errors have, but for chance: a rounding is off by at most u and, over a binade, by 0.41 u in the mean square,
x by 0.58 u.  The kernels' own sums, of 32 bits, are 2^13 times finer than a step of f16.  So each result may be off by
one and a half times the most of eight such runs."""
import pytest
import torch

from test_cache_gpu import pkg  # noqa: F401 (fixture)
from gqa_flash_attention_prefill_gb300 import workloads as W

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5
HIDDEN = 256


class Kept(torch.autograd.Function):
    """A tensor off by at most `u`, and its gradient by at most `du`."""

    @staticmethod
    def forward(ctx, x, u, du, gen):
        ctx.du, ctx.gen = du, gen
        return x * (1 + u * noise(x, gen)) if u else x.clone()

    @staticmethod
    def backward(ctx, g):
        return g * (1 + ctx.du * noise(g, ctx.gen)) if ctx.du else g, None, None, None


def noise(x, gen):
    return 2 * torch.rand(x.shape, generator=gen, dtype=x.dtype, device=x.device) - 1


class Layer:
    def __init__(self, lens, hq, hkv, d, dtype, window, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*shape, scale=1.0, to=DT[dtype]):
            return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(to)

        total = sum(lens)
        self.lens, self.hq, self.hkv, self.d, self.dtype, self.window = lens, hq, hkv, d, DT[dtype], window
        self.batch = W.make_batch([0] * len(lens), lens, hq, hkv, d, dtype, window=window, sink_mode="head").to("cuda")
        self.x, self.stream = randn(total, HIDDEN), randn(total, HIDDEN, to=torch.float32)
        self.norm = randn(HIDDEN, scale=0.2) + 1
        self.q_norm, self.k_norm = randn(d, scale=0.2, to=torch.float32), randn(d, scale=0.2, to=torch.float32)  # from 1
        self.proj = randn(HIDDEN, (hq + 2 * hkv) * d, scale=HIDDEN ** -0.5)
        self.dout, self.dstream = randn(total, hq, d), randn(total, HIDDEN, to=torch.float32)
        self.positions = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
        self.inv_freq = W.rope_frequencies(d)[0].to("cuda")

    def split(self, qkv):
        qkv = qkv.unflatten(-1, (-1, self.d))
        return qkv[:, :self.hq], qkv[:, self.hq:self.hq + self.hkv], qkv[:, self.hq + self.hkv:]

    def run(self, g):
        """Results of the operators of module `g`: what is kept, and the gradients."""
        t, b = {}, self.batch
        y, _, t["h"], rstd = g.rms_norm(self.x, self.norm, EPS, residual=self.stream, with_rstd=True)
        q0, k0, v = self.split((y.float() @ self.proj.float()).to(self.dtype))
        qn, _, _, q_rstd = g.rms_norm(q0, self.q_norm, EPS, 1.0, with_rstd=True)
        kn, _, _, k_rstd = g.rms_norm(k0, self.k_norm, EPS, 1.0, with_rstd=True)
        b.q, b.k, b.v = torch.empty_like(qn), torch.empty_like(kn), v.contiguous()
        g.gqa_rope(qn, self.positions, self.inv_freq, b.q, kn, b.k)
        t["out"], lse = g.prefill(b)
        dq, dk, dv, t["dsinks"] = g.prefill_backward(b, t["out"], lse, self.dout)
        dqn, dkn = torch.empty_like(dq), torch.empty_like(dk)
        g.gqa_rope(dq, self.positions, self.inv_freq, dqn, dk, dkn, inverse=True)
        dq0, _, t["dq_norm"] = g.rms_norm_backward(dqn, q0, self.q_norm, q_rstd, 1.0)
        dk0, _, t["dk_norm"] = g.rms_norm_backward(dkn, k0, self.k_norm, k_rstd, 1.0)
        dqkv = torch.cat([dq0, dk0, dv], 1).flatten(1)
        t["dproj"] = y.float().T @ dqkv.float()
        dy = (dqkv.float() @ self.proj.float().T).to(self.dtype)
        t["dx"], t["dstream"], t["dnorm"] = g.rms_norm_backward(dy, t["h"], self.norm, rstd, dh=self.dstream)
        return t

    def formula(self, u, seed=0):
        """The same in 64 bits; what is kept in 16 bits is off by at most `u`."""
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def kept(x):  # both are kept in 16 bits
            return Kept.apply(x, u, u, gen)

        def alone(x):  # the tensor, not its gradient
            return Kept.apply(x, u, 0.0, gen)

        def gradient(x):  # the gradient, not the tensor
            return Kept.apply(x, 0.0, u, gen)

        leaves = {n: getattr(self, n).double().requires_grad_()
                  for n in ("x", "stream", "norm", "q_norm", "k_norm", "proj")}
        sinks = self.batch.sinks.double().requires_grad_()
        x, d = leaves["x"], self.d

        def norm(x, w):
            return x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w

        def rope(x):
            a = self.positions.double()[:, None, None] * self.inv_freq.double()
            p, q = x[..., :d // 2], x[..., d // 2:]
            return torch.cat([p * a.cos() - q * a.sin(), q * a.cos() + p * a.sin()], -1)

        t = {"h": gradient(x) + leaves["stream"]}
        y = kept(norm(t["h"], leaves["norm"]))
        q, k, v = self.split(kept(y @ leaves["proj"]))
        q = kept(rope(kept(norm(q, leaves["q_norm"] + 1))))
        k = kept(rope(kept(norm(k, leaves["k_norm"] + 1))))
        group, outs, at = self.hq // self.hkv, [], 0
        for n in self.lens:
            s = slice(at, at + n)
            at += n
            score = torch.einsum("ihd,jhd->hij", q[s], k[s].repeat_interleave(group, 1)) * self.batch.scale
            i, j = torch.arange(n, device="cuda")[:, None], torch.arange(n, device="cuda")[None]
            keep = (j <= i) if not self.window else (j <= i) & (j > i - self.window)
            score = gradient(score).masked_fill(~keep, float("-inf"))  # its gradient is dS
            p = torch.softmax(torch.cat([score, sinks[:, None, None].expand(-1, n, 1)], -1), -1)[..., :-1]
            outs.append(torch.einsum("hij,jhd->ihd", alone(p), v[s].repeat_interleave(group, 1)))
        t["out"] = alone(torch.cat(outs))
        loss = (t["out"] * self.dout.double()).sum() + (t["h"] * self.dstream.double()).sum()
        leaves["sinks"] = sinks
        for name, g in zip(leaves, torch.autograd.grad(loss, list(leaves.values()))):
            t["d" + name] = g
        return {n: v.detach() for n, v in t.items()}


def check(got, layer, names, rows=slice(None)):
    exact = layer.formula(0.0)
    u = torch.finfo(layer.dtype).eps / 2
    runs = [layer.formula(u, seed) for seed in range(8)]
    for name in names:
        part = rows if name == "out" else slice(None)
        want = exact[name][part]
        room = 1.5 * max(float((r[name][part] - want).norm()) for r in runs)
        # What is kept in 32 bits without an operator of 16 bits before it.
        room = max(room, 2.0 ** -20 * float(want.norm()))
        assert got[name].shape == want.shape
        assert float((got[name].double() - want).norm()) <= room, name


SHAPES = [([70, 1, 129], 8, 2, 64, "bf16", 0), ([70, 1, 129], 8, 2, 64, "f16", 48), ([33, 160], 4, 4, 128, "f16", 0),
          ([1, 5, 190], 8, 1, 128, "bf16", 100), ([65, 2], 4, 2, 256, "bf16", 0)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_layer_and_its_gradient(pkg, shape):  # noqa: F811
    layer = Layer(*shape, seed=1)
    got = layer.run(pkg)
    torch.cuda.synchronize()
    check(got, layer, ["h", "out", "dsinks", "dq_norm", "dk_norm", "dproj", "dx", "dstream", "dnorm"])


@pytest.mark.parametrize("shape", SHAPES[:1] + SHAPES[2:3], ids=str)
def test_a_captured_layer_repeats_it(pkg, shape):  # noqa: F811
    layer = Layer(*shape, seed=2)
    want = layer.run(pkg)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        got = layer.run(pkg)
    inputs = layer.x, layer.stream, layer.dout
    before = [t.clone() for t in inputs]
    for t in inputs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert not bool(got["out"].isnan().any()) and float(got["dx"].abs().max()) <= 1.01 * float(layer.dstream.abs().max())
    for t, b in zip(inputs, before):
        t.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    for name in want:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("shape", SHAPES[:2] + SHAPES[3:], ids=str)
def test_a_decoded_token_after_the_same_norms(pkg, shape):  # noqa: F811
    """The prompt's keys and values go into a cache, and the last token of each sequence attends over it."""
    layer = Layer(*shape, seed=3)
    lens, b = layer.lens, layer.batch
    y = pkg.rms_norm(layer.x, layer.norm, EPS, residual=layer.stream)[0]
    q0, k0, v = layer.split((y.float() @ layer.proj.float()).to(layer.dtype))
    q = pkg.rms_norm(q0, layer.q_norm, EPS, 1.0)[0]
    b.q, b.k, b.v = q, pkg.rms_norm(k0, layer.k_norm, EPS, 1.0)[0], v.contiguous()
    cache = W.empty_cache(lens, layer.hkv, layer.d, 16, shape[4], device="cuda")
    rotated = torch.empty_like(q)
    pkg.cache_write(b, cache, rope=pkg.Rope(layer.inv_freq, q=q, q_out=rotated))
    step = W.make_batch([n - 1 for n in lens], [1] * len(lens), layer.hq, layer.hkv, layer.d, shape[4],
                        window=layer.window, sink_mode="head").to("cuda")
    step.sinks = b.sinks
    last = torch.tensor(lens, device="cuda").cumsum(0) - 1
    out, _ = pkg.cache_attention(step, cache, q=rotated[last].contiguous())
    torch.cuda.synchronize()
    check({"out": out}, layer, ["out"], rows=last)
