"""A decoder layer's products with adapters, rotary positions, cache and
attention together, as a server runs them: a prompt, chunks, single tokens, and
the decode step captured."""
import os
import re

import pytest
import torch

import heterogeneous_adapter_batching_amd as hab
from attention_reference import Batch
from conftest import ROOT

pytestmark = pytest.mark.gpu

H, KH, D, W = 8, 2, 64, 512            # heads, key heads, their width, the model's
PAGE, PAGES = 32, 40


class Layer:
    """Weights, two adapters, the cache and the sequences' pages."""

    def __init__(self, seqs):
        g = torch.Generator(device="cuda").manual_seed(3)
        r = lambda *s, std: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
        self.widths = [H * D, KH * D, KH * D, W]
        self.w_qkv, self.w_o = r(sum(self.widths[:3]), W, std=W ** -0.5), r(W, H * D, std=W ** -0.5)
        self.norm = r(W, std=0.1) + 1
        self.pool = hab.Pool(1, [W, W, W, H * D], self.widths, r_max=16, dtype="bf16", slab_bytes=1 << 22)
        for i in (0, 1):
            self.pool.register(i, 8, 2.0, A=[r(1, 8, n, std=W ** -0.5) for n in (W, W, W, H * D)],
                               B=[r(1, n, 8, std=0.05) for n in self.widths])
        self.k = torch.full((PAGES, KH, PAGE, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.v = self.k.clone()
        self.pages = torch.randperm(PAGES, generator=g, device="cuda").to(torch.int32)[:seqs * 8].view(seqs, 8)
        self.freqs = hab.rotary_frequencies(D, device="cuda")

    def plans(self, new, kv, **kw):
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        adapters = hab.Plan(self.pool, starts[-1], starts, [s % 3 - 1 for s in range(len(new))]).upload(3)
        return adapters, hab.AttentionPlan(H, KH, D, PAGE, new, kv, **kw).upload()

    def step(self, h, adapters, attn):
        """h' = h + o(attention(rotary(qkv(norm(h))))), and what lies between."""
        _, x = hab.block_norm(h, pre_weight=self.norm)
        qkv = hab.sgmv_linear(self.pool, adapters, 0, (0, 1, 2), (0, H * D, (H + KH) * D), x, self.w_qkv)
        q, k, v = qkv.split(self.widths[:3], 1)
        q = hab.rotary_append(attn, q, k, v, self.k, self.v, self.pages, self.freqs, q_out=q)
        a = hab.paged_attention(attn, q, self.k, self.v, self.pages)
        return hab.sgmv_linear(self.pool, adapters, 0, (3,), (0,), a, self.w_o, residual=h), q, a

    def check(self, new, kv, q, a):
        b = Batch(new, kv, H, KH, D, PAGE)
        b.q, b.k, b.v, b.pages = q, self.k, self.v, self.pages
        o, mean, size = b.attention()
        tol = b.tolerance(o, mean, size, 2.0 ** -8)
        assert ((a.double().view(o.shape) - o).abs() <= tol).all()


def hidden(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, W, generator=g, device="cuda").to(torch.bfloat16)


def test_prompt_chunks_and_single_tokens():
    """The cache carries the sequences from call to call: whole prompts give
    what chunks and single tokens give."""
    layer = Layer(3)
    lens = [100, 37, 64]
    h = [hidden(n, s) for s, n in enumerate(lens)]
    whole, q, a = layer.step(torch.cat(h), *layer.plans(lens, lens))
    layer.check(lens, lens, q, a)
    whole = whole.split(lens)
    other = Layer(3)
    done = [0, 0, 0]
    got = [[] for _ in lens]
    for cut in ([60, 1, 30], [20, 30, 0], [1, 1, 1], [1, 1, 1], [18, 4, 32]):
        new, kv = cut, [d + c for d, c in zip(done, cut)]
        part = torch.cat([t[d:d + c] for t, d, c in zip(h, done, cut)])
        out, q, a = other.step(part, *other.plans(new, kv))
        other.check(new, kv, q, a)
        for g, t in zip(got, out.split(cut)):
            g.append(t)
        done = kv
    assert done == lens
    for s, w in enumerate(whole):
        # (the products' own parts along K, and the weights of prompts, differ by
        # a rounding here and there: bfloat16's, of outputs of size 1 to 4)
        assert (torch.cat(got[s]).float() - w.float()).abs().max() <= 8 * 2.0 ** -8 * w.float().abs().max()


def test_decode_steps_captured():
    """One graph for all decode steps of a batch: the plan rebuilt and uploaded,
    the hidden states copied in, the graph replayed; each step against the same
    calls made eagerly."""
    layer, eager = Layer(4), Layer(4)
    lens = [50, 3, 31, 64]
    h = hidden(sum(lens), 9)
    for one in (layer, eager):
        one.step(h, *one.plans(lens, lens))
    new, kv = [1] * 4, [n + 1 for n in lens]
    adapters, attn = layer.plans(new, kv, max_kv=8 * PAGE)
    x, out = hidden(4, 10), torch.empty(4, W, dtype=torch.bfloat16, device="cuda")
    keep = layer.k.clone(), layer.v.clone()
    layer.step(x, adapters, attn)
    torch.cuda.synchronize()
    layer.k.copy_(keep[0])
    layer.v.copy_(keep[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out.copy_(layer.step(x, adapters, attn)[0])
    plans = eager.plans(new, kv, max_kv=8 * PAGE)
    for step in range(40):
        x.copy_(hidden(4, 20 + step))
        attn.rebuild(new, kv).upload(ws=attn.ws)
        graph.replay()
        plans[1].rebuild(new, kv).upload(ws=plans[1].ws)
        want = eager.step(x, *plans)[0]
        torch.cuda.synchronize()
        assert torch.equal(out, want), step
        assert all(torch.equal(a[~a.isnan()], b[~b.isnan()])
                   for a, b in ((layer.k, eager.k), (layer.v, eager.v)))
        kv = [n + 1 for n in kv]


def test_readme_example():
    text = open(os.path.join(ROOT, "README.md")).read()
    code = re.search(r"## Attention from Python\n\n```python\n(.*?)```", text, re.S).group(1)
    names = dict(qkv=(torch.randn(40, 6144, device="cuda")).to(torch.bfloat16))
    exec(compile(code, "README.md", "exec"), names)
    torch.cuda.synchronize()
    assert names["attended"].shape == (40, 4096) and bool(names["attended"].isfinite().all())
