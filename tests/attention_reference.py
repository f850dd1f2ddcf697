"""Attention over a paged cache, and rotary positions, in 64 bits from their
definitions: what the tests of the library's kernels compare with."""
import math

import torch

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


class Batch:
    """Sequences of new tokens behind cached ones: random queries, a cache whose
    pages lie in a random order among others, NaN in every place that holds no
    key, and the page table."""

    def __init__(self, new, kv, heads=8, kv_heads=2, dim=64, page=16, dtype="bf16", causal=True,
                 window=0, seed=0, device="cuda", order="heads", std=1.0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.new, self.kv, self.heads, self.kv_heads = list(new), list(kv), heads, kv_heads
        self.dim, self.page, self.dtype, self.causal, self.window = dim, page, dtype, causal, window
        dt = DTYPES[dtype]
        self.tokens = sum(self.new)

        def rand(*shape):
            return torch.randn(*shape, generator=g, device=device)

        counts = [-(-n // page) for n in self.kv]
        total = sum(counts) + 2
        perm = torch.randperm(total, generator=g, device=device).to(torch.int32)
        self.pages = torch.full((max(len(self.new), 1), max(counts + [1])), -1, dtype=torch.int32,
                                device=device)
        held = torch.zeros(total, page, dtype=torch.bool, device=device)
        at = 0
        for s, (n, L) in enumerate(zip(counts, self.kv)):
            mine = perm[at:at + n]
            self.pages[s, :n] = mine
            at += n
            for i in range(n):
                held[int(mine[i]), :min(page, L - i * page)] = True
        # the cache as [pages][kv_heads][page][dim], whatever its order in memory
        k, v = (rand(total, kv_heads, page, dim).to(dt) for _ in range(2))
        nan = torch.full((), math.nan, dtype=dt, device=device)
        k, v = (torch.where(held[:, None, :, None], t, nan) for t in (k, v))
        if order == "tokens":                    # [pages][page][kv_heads][dim]
            k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
        elif order == "joined":                  # keys and values of a page side by side
            both = torch.stack([k, v], 1)
            k, v = both[:, 0], both[:, 1]
        self.k, self.v = k, v
        self.q = (rand(self.tokens, heads * dim) * std).to(dt)

    def seen(self, s):
        """[new][kv] truth values: the keys that each new token sees."""
        n, L = self.new[s], self.kv[s]
        key = torch.arange(L, device=self.q.device)
        place = torch.arange(L - n, L, device=self.q.device)[:, None]
        if not self.causal:
            return torch.ones(n, L, dtype=torch.bool, device=self.q.device)
        seen = key <= place
        return seen & (key > place - self.window) if self.window else seen

    def gather(self, cache, s, absent=None):
        """A sequence's keys or values [kv][kv_heads][dim] in 64 bits."""
        rows = self.pages[s, :-(-self.kv[s] // self.page)].long()
        rows = rows.clamp(0, cache.shape[0] - 1)
        return cache[rows].double().transpose(1, 2).flatten(0, 1)[:self.kv[s]]

    def attention(self, scale=None):
        """(o, the mean of |v| under the weights, the largest sum |q_i k_i|
        scale) in 64 bits, [tokens][heads][dim], the same, [tokens][heads]."""
        scale = self.dim ** -0.5 if scale is None else scale
        group = self.heads // self.kv_heads
        dev = self.q.device
        o = torch.zeros(self.tokens, self.heads, self.dim, dtype=torch.float64, device=dev)
        mean, size = torch.zeros_like(o), torch.zeros(self.tokens, self.heads, dtype=torch.float64,
                                                      device=dev)
        q = self.q.double().reshape(self.tokens, self.heads, self.dim)
        at = 0
        for s, (n, L) in enumerate(zip(self.new, self.kv)):
            if n and L:
                k, v = self.gather(self.k, s), self.gather(self.v, s)
                rows = self.pages[s, :-(-L // self.page)]
                there = ((rows >= 0) & (rows < self.k.shape[0])).repeat_interleave(self.page)[:L]
                seen = self.seen(s) & there
                for h in range(self.heads):
                    kh, vh = k[:, h // group], v[:, h // group]
                    # (what no token sees is left out: it may hold anything)
                    used = seen.any(0)
                    kh, vh, m = kh[used], vh[used], seen[:, used]
                    if not m.shape[1]:
                        continue
                    t = (q[at:at + n, h] @ kh.T) * scale
                    t = torch.where(m, t, -math.inf)
                    top = t.max(1, keepdim=True).values
                    p = torch.exp(t - torch.where(top == -math.inf, 0.0, top))
                    p = torch.where(m, p, 0.0)
                    total = p.sum(1, keepdim=True)
                    p = p / torch.where(total == 0, 1.0, total)
                    # (0 weights times infinities that only other tokens see)
                    if torch.isfinite(vh).all():
                        o[at:at + n, h], mean[at:at + n, h] = p @ vh, p @ vh.abs()
                    else:
                        for i in range(n):
                            o[at + i, h] = p[i, m[i]] @ vh[m[i]]
                            mean[at + i, h] = p[i, m[i]] @ vh[m[i]].abs()
                    sizes = (q[at:at + n, h].abs() @ kh.abs().T) * abs(scale)
                    size[at:at + n, h] = torch.where(m, sizes, 0.0).amax(1)
            at += n
        return o, mean, size

    def tolerance(self, o, mean, size, weight_eps):
        """What the kernels may be off by, from the roundings they make: the
        output's half step; the weights' to `weight_eps`; the scores' float32
        sums of dim products (2^-24 each of at most `size`, three times as much
        with the scaling and the exponent's own), which move a weight and the
        weights' sum; and the sums over the keys."""
        half = torch.finfo(DTYPES[self.dtype]).eps / 2
        scores = size[..., None] * (self.dim + 3) * 2.0 ** -24
        keys = (max(self.kv + [1]) + 32) * 2.0 ** -24
        return half * o.abs() + mean * (weight_eps + 2 * scores + 2 * keys + 2.0 ** -21) + 1e-30

    def turned(self, rows, heads, positions, freqs, layout, magnitude):
        """Rotary positions on rows [tokens][heads * dim], in 64 bits."""
        x = rows.double().reshape(rows.shape[0], heads, self.dim)
        if freqs is None:
            return x
        r = freqs.shape[0]
        a = (positions.double()[:, None] * freqs.double().to(x.device))[:, None]
        i = torch.arange(r, device=x.device)
        first, second = (i, i + r) if layout == "half" else (2 * i, 2 * i + 1)
        out = x.clone()
        out[..., first] = magnitude * (x[..., first] * torch.cos(a) - x[..., second] * torch.sin(a))
        out[..., second] = magnitude * (x[..., second] * torch.cos(a) + x[..., first] * torch.sin(a))
        return out

    def places(self):
        """The new tokens' positions among their keys, their pages and slots."""
        pos = [L - n + i for n, L in zip(self.new, self.kv) for i in range(n)]
        seq = [s for s, n in enumerate(self.new) for _ in range(n)]
        pos = torch.tensor(pos, dtype=torch.int64, device=self.q.device)
        seq = torch.tensor(seq, dtype=torch.int64, device=self.q.device)
        return pos, self.pages[seq, pos // self.page].long(), pos % self.page
