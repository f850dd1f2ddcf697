"""A decoder layer's attention around its products, and what it costs.

Three forms of two operators run between the q/k/v product and the o product of
a layer, over a cache of keys and values in pages:

  rotary   rotary positions on a batch's new queries and keys, which go, with
           the new values, into the pages of their sequences: with angle
           a_i = p f_i, pair (x, y) of a head at position p becomes
               (m (x cos a_i - y sin a_i), m (y cos a_i + x sin a_i)).
  attend   attention of the new tokens (a chunk of a prompt, or one token of a
           decode step) over the sequence's pages, the new ones among them:
               o = sum_j exp(s q.k_j - M) v_j / sum_j exp(s q.k_j - M),
           over keys j up to the token's own position, or the last `window`.
  cross    the same over an encoder's states of another length: all of them.

`own` selects between the plain form of each (elementary torch operations in
32 bits, angles in 64, rounded once at the end) and the library's calls.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases ----

def _case(name, **values):
    return ({"name": name} if name else {}) | values


def rotary(name, seqs, new, past, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16",
           rotary_dim=128, layout="half", scaling="none", factor=1.0, shift=0, lens=1):
    """seqs sequences of `new` tokens behind `past` cached ones each ("a" or
    "a-b": between them, by `lens`); shift: added to the positions (tokens
    whose early keys have left the cache)."""
    return _case(name, op="rotary", seqs=seqs, new=new, past=past, heads=heads, kv_heads=kv_heads,
                 dim=dim, page=page, dtype=dtype, rotary_dim=rotary_dim, layout=layout,
                 scaling=scaling, factor=factor, shift=shift, lens=lens)


def attend(name, seqs, new, past, heads=32, kv_heads=8, dim=128, page=64, dtype="bf16", window=0,
           lens=1):
    return _case(name, op="attend", seqs=seqs, new=new, past=past, heads=heads, kv_heads=kv_heads,
                 dim=dim, page=page, dtype=dtype, window=window, lens=lens)


def cross(name, seqs, new, past, heads=16, kv_heads=16, dim=64, page=64, dtype="bf16", lens=1):
    """past: the encoder's states of each sequence."""
    return _case(name, op="cross", seqs=seqs, new=new, past=past, heads=heads, kv_heads=kv_heads,
                 dim=dim, page=page, dtype=dtype, window=0, lens=lens)


def listed():
    return [
        # one request decoding: latency alone
        rotary("rotary_token", 1, "1", "500"),
        # a decode batch of 128 requests
        rotary("rotary_decode", 128, "1", "16-1024"),
        # ragged chunks in 32 bits, interleaved pairs in part of a head, far along a long context
        rotary("rotary_ragged_far_f32", 7, "1-90", "0-700", 12, 4, 80, 48, "f32", 32, "interleaved",
               "linear", 8.0, 1000000, 3),
        # four prompts of a context stretched by parts
        rotary("rotary_prompt", 4, "4096", "0", scaling="by_parts", factor=4.0),
        # one request decoding behind a short context
        attend("attend_token", 1, "1", "700"),
        # a decode batch of 128 requests of very different ages
        attend("attend_decode", 128, "1", "16-8192"),
        # four requests decoding behind very long contexts
        attend("attend_long_decode", 4, "1", "65536-131072", lens=2),
        # chunks of prompts behind their earlier chunks
        attend("attend_chunks", 8, "512", "0-16384", lens=4),
        # four whole prompts
        attend("attend_prompt", 4, "4096", "0"),
        # ragged chunks in 32 bits through a sliding window, an odd head and odd pages
        attend("attend_window_f32", 5, "1-60", "0-600", 9, 3, 72, 48, "f32", 100, 5),
        # 64 requests decoding over an encoder's states, a key head for each query head
        cross("cross_decode", 64, "1", "1500"),
        # their first tokens, over states of different lengths
        cross("cross_prompt", 24, "100-448", "300-1500", lens=6),
    ]


#: What one drawn case may cost at most: the largest listed ones.
MOST_FLOPS = 4.0 * 128 * 32 * 4 * 4096 * 4097 / 2
MOST_BYTES = 4.0 * 131072 * 8 * 128 * 2 * 2


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _spread(rng, lo, hi):
    """A range within lo .. hi, as a case writes it."""
    a, b = sorted((_log(rng, lo, hi), _log(rng, lo, hi)))
    return str(a) if rng.random() < 0.3 else "%d-%d" % (a, b)


def draw(rng):
    while True:
        op = rng.choice(["rotary", "attend", "attend", "cross"])
        kv_heads, group = rng.choice([1, 2, 3, 4, 8, 8, 16]), rng.choice([1, 1, 2, 3, 4, 4, 7, 8])
        if kv_heads * group > 64:
            continue
        dim = rng.choice([16, 40, 64, 64, 72, 80, 96, 128, 128, 128, 192, 256])
        shape = dict(heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                     page=rng.choice([16, 16, 32, 48, 64, 128, 256, 400]),
                     dtype="f32" if rng.random() < 0.25 else "bf16", lens=rng.randrange(1000))
        many = rng.random() < 0.5                    # a decode step; else chunks
        seqs = _log(rng, 1, 256) if many else _log(rng, 1, 24)
        new = "1" if many and rng.random() < 0.8 else _spread(rng, 1, 8 if many else 4096)
        if op == "rotary":
            part = dim if rng.random() < 0.5 else 2 * rng.randrange(1, dim // 2 + 1)
            scaling = rng.choice(["none", "linear", "by_parts"])
            case = rotary(None, seqs, new, _spread(rng, 1, 1024), rotary_dim=part,
                          layout=rng.choice(["half", "interleaved"]), scaling=scaling,
                          factor=1.0 if scaling == "none" else rng.choice([2.0, 8.0, 32.0]),
                          shift=rng.choice([0, 0, 1000, 4000000]), **shape)
        elif op == "attend":
            window = _log(rng, 1, 4096) if rng.random() < 0.25 else 0
            case = attend(None, seqs, new, _spread(rng, 1, 32768 if many else 8192), window=window,
                          **shape)
        else:
            case = cross(None, seqs, new, _spread(rng, 1, 4096), **shape)
        cost = work(case)
        # (32-bit products take eight times as long as 16-bit ones)
        if cost["flops"] * (8 if case["dtype"] == "f32" else 1) <= MOST_FLOPS and \
                cost["bytes"] <= MOST_BYTES and _cache_bytes(case) <= MOST_BYTES:
            return case


def _range(text):
    lo, _, hi = text.partition("-")
    return int(lo), int(hi or lo)


def _lens(case):
    """New tokens and cached keys (the new ones among them, unless they are an
    encoder's states) of every sequence."""
    rng = random.Random(case["lens"])

    def some(text):
        lo, hi = _range(text)
        return lo if lo == hi else min(hi, int((lo + 1) * math.exp(
            rng.random() * math.log((hi + 1) / (lo + 1)))) - 1 + (rng.random() < 0.5))

    new = [some(case["new"]) for _ in range(case["seqs"])]
    past = [some(case["past"]) for _ in range(case["seqs"])]
    return new, past if case["op"] == "cross" else [n + p for n, p in zip(new, past)]


def _pages(case, kv):
    return [-(-n // case["page"]) for n in kv]


def _cache_bytes(case):
    pages = sum(_pages(case, _lens(case)[1]))
    return pages * case["page"] * case["kv_heads"] * case["dim"] * 2 * DTYPES[case["dtype"]].itemsize


# ----------------------------------------------------------------- inputs ----

def _frequencies(case):
    """Radians a position turns each pair by, in 64 bits."""
    f = torch.pow(torch.tensor(10000.0, dtype=torch.float64),
                  -torch.arange(0, case["rotary_dim"], 2, dtype=torch.float64) / case["rotary_dim"])
    if case["scaling"] == "linear":
        return f / case["factor"]
    if case["scaling"] == "by_parts":
        # pairs that turn often within the trained length keep their angles, those that hardly
        # turn are stretched, and those between are blended
        keep = ((f * (4096 / (2 * math.pi)) - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return f * keep + f / case["factor"] * (1.0 - keep)
    return f


def _magnitude(case):
    return 1.0 + 0.1 * math.log(case["factor"]) if case["scaling"] == "by_parts" else 1.0


def _tensors(case, seed):
    """Every tensor of the case, on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    new, kv = _lens(case)
    T, H, KH, D = sum(new), case["heads"], case["kv_heads"], case["dim"]

    def rand(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dt)

    # a sequence's pages lie where the cache had room, some of them nobody's
    counts = _pages(case, kv)
    total = sum(counts) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    pages = torch.zeros(len(new), max(counts + [1]), dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(counts):
        pages[s, :n] = order[at:at + n]
        at += n
    s = {"pages": pages,
         "k_cache": rand(total, KH, case["page"], D), "v_cache": rand(total, KH, case["page"], D)}
    if case["op"] == "rotary":
        # q, k and v are slices of one product's rows
        qkv = rand(T, (H + 2 * KH) * D)
        s["q"], s["k"], s["v"] = qkv.split([H * D, KH * D, KH * D], 1)
        s["positions"] = torch.tensor([case["shift"] + L - n + i for n, L in zip(new, kv)
                                       for i in range(n)], dtype=torch.int32, device="cuda")
    else:
        # scores of standard deviation 1.5: some keys count more than others
        s["q"] = rand(T, H * D, std=1.5)
    return s


def prepare(case, seed):
    s = _tensors(case, seed)
    s["case"], (s["new"], s["kv"]) = case, _lens(case)
    if case["op"] == "rotary":
        s["freqs"] = _frequencies(case).to("cuda")
        # where each new token's key and value go
        page, slot = [], []
        for n, L in zip(s["new"], s["kv"]):
            page.append(torch.arange(L - n, L) // case["page"])
            slot.append(torch.arange(L - n, L) % case["page"])
        row = torch.repeat_interleave(torch.arange(len(s["new"])), torch.tensor(s["new"]))
        s["page"] = s["pages"][row.cuda(), torch.cat(page).cuda()].long()
        s["slot"] = torch.cat(slot).cuda()
    if own:
        import heterogeneous_adapter_batching_amd as hab
        s["plan"] = hab.AttentionPlan(
            case["heads"], case["kv_heads"], case["dim"], case["page"], s["new"], s["kv"],
            dtype=case["dtype"], causal=case["op"] != "cross",
            window=case.get("window", 0)).upload()
        s["out"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
        if case["op"] == "rotary":
            s["freqs"] = hab.rotary_frequencies(
                case["rotary_dim"], base=10000.0, scaling=case["scaling"], factor=case["factor"],
                original_length=4096, device="cuda")
    return s


# ------------------------------------------------------------------- runs ----

def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return _plain_rotary(case, state) if case["op"] == "rotary" else _plain_attend(case, state)


def _own(case, s):
    import heterogeneous_adapter_batching_amd as hab
    if case["op"] == "rotary":
        q = hab.rotary_append(s["plan"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"],
                              s["pages"], s["freqs"], layout=case["layout"],
                              magnitude=_magnitude(case), q_out=s["out"],
                              positions=s["positions"] if case["shift"] else None)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    return hab.paged_attention(s["plan"], s["q"], s["k_cache"], s["v_cache"], s["pages"],
                               o=s["out"])


def _plain_turn(case, rows, cos, sin):
    """The pairs of every head of rows [T][heads][dim], turned."""
    x, r = rows.float(), case["rotary_dim"]
    a, b = (x[..., :r // 2], x[..., r // 2:r]) if case["layout"] == "half" else \
        (x[..., 0:r:2], x[..., 1:r:2])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([a, b], -1) if case["layout"] == "half" else \
        torch.stack([a, b], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1).to(rows.dtype)


def _plain_rotary(case, s):
    T, D = s["q"].shape[0], case["dim"]
    angle = s["positions"].double()[:, None] * s["freqs"]
    cos, sin = ((f(angle) * _magnitude(case)).float()[:, None] for f in (torch.cos, torch.sin))
    q = _plain_turn(case, s["q"].reshape(T, -1, D), cos, sin)
    s["k_cache"][s["page"], :, s["slot"]] = _plain_turn(case, s["k"].reshape(T, -1, D), cos, sin)
    s["v_cache"][s["page"], :, s["slot"]] = s["v"].reshape(T, -1, D)
    return {"q": q.reshape(T, -1), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(case, s):
    KH, D, group = case["kv_heads"], case["dim"], case["heads"] // case["kv_heads"]
    outs, at = [], 0
    for i, (n, L) in enumerate(zip(s["new"], s["kv"])):
        rows = s["pages"][i, :-(-L // case["page"])].long()
        k, v = (s[c][rows].transpose(0, 1).reshape(KH, -1, D)[:, :L].float()
                for c in ("k_cache", "v_cache"))
        q = s["q"][at:at + n].float().reshape(n, KH, group, D).permute(1, 0, 2, 3)
        at += n
        t = (q.reshape(KH, n * group, D) @ k.transpose(1, 2)) * (1.0 / math.sqrt(D))
        t = t.reshape(KH, n, group, L)
        if case["op"] == "attend":
            key = torch.arange(L, device="cuda")
            place = torch.arange(L - n, L, device="cuda")[:, None]
            hidden = key > place
            if case["window"]:
                hidden = hidden | (key <= place - case["window"])
            t = torch.where(hidden[:, None], -math.inf, t)
        t = torch.exp(t - t.max(-1, keepdim=True).values)
        o = (t.reshape(KH, n * group, L) @ v) / t.sum(-1).reshape(KH, n * group, 1)
        outs.append(o.reshape(KH, n, group, D).permute(1, 0, 2, 3).reshape(n, -1))
    return torch.cat(outs).to(s["q"].dtype)


# ------------------------------------------------------------- accounting ----

def work(case):
    e, D, H, KH = DTYPES[case["dtype"]].itemsize, case["dim"], case["heads"], case["kv_heads"]
    new, kv = _lens(case)
    T = sum(new)
    if case["op"] == "rotary":
        # q, k and v read and written once; a pair's turn is 6 operations
        return {"bytes": 2 * T * (H + 2 * KH) * D * e + 4 * T + 4 * case["rotary_dim"],
                "flops": 3 * T * (H + KH) * case["rotary_dim"]}
    w = case["window"]
    keys, pairs = 0, 0
    for n, L in zip(new, kv):
        if case["op"] == "cross":
            keys, pairs = keys + L, pairs + n * L
            continue
        # token i of the chunk sees L - n + i + 1 keys, at most w of them
        first = L - n + 1
        keys += L if not w else min(L, n + w - 1)
        if not w or L <= w:
            pairs += n * (first + L) // 2
        else:
            short = max(0, min(n, w - first))
            pairs += short * (2 * first + short - 1) // 2 + (n - short) * w
    return {"bytes": e * D * (2 * T * H + 2 * keys * KH) + 4 * sum(_pages(case, kv)),
            "flops": 4 * pairs * H * D}


# ------------------------------------------------------------------ exact ----

def exact(case, seed):
    """The definitions in 64 bits, unrounded, from the same inputs."""
    s = _tensors(case, seed)
    new, kv = _lens(case)
    D, ps = case["dim"], case["page"]
    starts = [sum(new[:i]) for i in range(len(new))]
    if case["op"] == "rotary":
        r = case["rotary_dim"]
        turn = torch.polar(torch.full((1,), _magnitude(case), dtype=torch.float64, device="cuda"),
                           torch.outer(s["positions"].double(), _frequencies(case).cuda()))

        def turned(rows):
            x = rows.double().unflatten(1, (-1, D)).clone()
            head = x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2) \
                if case["layout"] == "half" else x[..., :r].unflatten(-1, (r // 2, 2))
            z = torch.view_as_real(torch.view_as_complex(head.contiguous()) * turn[:, None])
            x[..., :r] = (z.transpose(-1, -2) if case["layout"] == "half" else z).flatten(-2)
            return x

        out = {"q": turned(s["q"]).flatten(1), "k_cache": s["k_cache"].double(),
               "v_cache": s["v_cache"].double()}
        k, v = turned(s["k"]), s["v"].double().unflatten(1, (-1, D))
        for i, (a, n, L) in enumerate(zip(starts, new, kv)):
            j = 0
            while j < n:                                  # page by page
                p, o = divmod(L - n + j, ps)
                m = min(ps - o, n - j)
                page = int(s["pages"][i, p])
                for name, rows in (("k_cache", k), ("v_cache", v)):
                    out[name][page, :, o:o + m] = rows[a + j:a + j + m].transpose(0, 1)
                j += m
        return out
    group = case["heads"] // case["kv_heads"]
    o = torch.zeros(sum(new), case["heads"], D, dtype=torch.float64, device="cuda")
    q = s["q"].double().unflatten(1, (-1, D))
    for i, (a, n, L) in enumerate(zip(starts, new, kv)):
        pages = s["pages"][i, :-(-L // ps)].long()
        for h in range(case["kv_heads"]):
            k = s["k_cache"][pages, h].double().flatten(0, 1)[:L]
            v = s["v_cache"][pages, h].double().flatten(0, 1)[:L]
            mine = slice(h * group, (h + 1) * group)
            t = torch.einsum("ngd,ld->ngl", q[a:a + n, mine], k) / math.sqrt(D)
            if case["op"] == "attend":
                behind = torch.arange(L - n, L, device="cuda")[:, None] - \
                    torch.arange(L, device="cuda")
                seen = behind >= 0
                if case["window"]:
                    seen &= behind < case["window"]
                t.masked_fill_(~seen[:, None], -math.inf)
            o[a:a + n, mine] = torch.einsum("ngl,ld->ngd", torch.softmax(t, -1), v)
    return o.flatten(1)
