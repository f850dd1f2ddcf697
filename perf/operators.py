"""The operators around the adapters' delta, and what they cost.

Three operators run next to the multi-adapter delta in a decoder layer:

  norm     the residual stream's update and the norms before and after a block:
               h' = beta h + alpha g . N_post(o),   u = N_pre(h')
           (o the block's output, g its gate, N an RMS or layer norm, or
           nothing), computed from the unrounded h' for u.
  linear   the frozen layer's product with its epilogue:
               y = act(x W^T + b) + residual, or with a gated pair of weights
               y = act(x Wg^T + bg) . (x Wu^T + bu) + residual.
  adapted  the same with every token's LoRA delta inside the activation:
               y = act(x W^T + b + s_i B_i (A_i x)) + residual.

`own` selects between the plain form of each (elementary torch operations in
32 bits, rounded once at the end) and the library's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases ----

def _case(name, **values):
    return ({"name": name} if name else {}) | values


def norm(name, tokens, width, dtype="bf16", stream="bf16", post="none", pre="rms", gate="none",
         gate_act="none", bias=False, alpha=1.0, beta=1.0):
    return _case(name, op="norm", tokens=tokens, width=width, dtype=dtype, stream=stream,
                 post=post, pre=pre, gate=gate, gate_act=gate_act, bias=bias, alpha=alpha,
                 beta=beta)


def linear(name, tokens, k, n, dtype="bf16", act="none", glu=False, bias=False, residual=False):
    return _case(name, op="linear", tokens=tokens, k=k, n=n, dtype=dtype, act=act, glu=glu,
                 bias=bias, residual=residual)


def adapted(name, tokens, k, widths, ranks, pool, segment, dtype="bf16", act="none", glu=False,
            bias=False, residual=False, skew=1.1, idle=0.0):
    """widths: output widths of the projections that share x, comma-separated
    (two equal ones, gate and up, with glu); ranks: the pool's ranks, dealt in
    turn; segment: tokens of one request; skew: Zipf exponent of the adapters'
    popularity (0: uniform); idle: share of requests without an adapter."""
    return _case(name, op="adapted", tokens=tokens, k=k, widths=widths, ranks=ranks, pool=pool,
                 segment=segment, dtype=dtype, act=act, glu=glu, bias=bias, residual=residual,
                 skew=skew, idle=idle)


def listed():
    return [
        # one request decoding: the residual add and the norm before the next block
        norm("norm_token", 1, 4096),
        # a decode batch of a model with norms on both sides of a block and a layer scale
        norm("norm_decode_both", 128, 4096, post="rms", gate="vector", alpha=0.22),
        # a ragged batch of odd width in 32 bits: layer norms with biases, a gate row per token
        norm("norm_ragged_f32", 1021, 5003, dtype="f32", stream="f32", post="layer", pre="layer",
             gate="rows", gate_act="tanh", bias=True, alpha=0.5, beta=1.25),
        # a long prompt batch with the residual stream kept in 32 bits
        norm("norm_long_prompt", 16384, 4096, stream="f32", post="rms"),
        # one request decoding: gate and up of the MLP, where the weights' bytes count
        linear("linear_token_glu", 1, 4096, 14336, act="silu", glu=True),
        # a decode batch through the MLP's down projection onto the residual stream
        linear("linear_decode_down", 128, 14336, 4096, residual=True),
        # a small ragged product in 32 bits with bias and activation
        linear("linear_ragged_f32", 77, 1016, 1003, dtype="f32", act="gelu", bias=True),
        # a prompt batch through gate and up: a large matrix product
        linear("linear_prompt_glu", 4096, 4096, 14336, act="silu", glu=True),
        # a decode batch of 128 requests over 1000 rank-16 adapters through q, k and v
        adapted("adapted_decode_qkv", 128, 4096, "4096,1024,1024", "16", 1000, 1),
        # a decode batch of mixed ranks through the gated MLP
        adapted("adapted_multirank_glu", 256, 4096, "14336,14336", "8,16,32,64", 64, 1,
                act="silu", glu=True, skew=0.0),
        # 8 prompts of 512 tokens with an adapter each through o onto the residual stream
        adapted("adapted_prompt_o", 4096, 4096, "4096", "16", 8, 512, residual=True, skew=0.0),
        # a few short prompts in 32 bits, some without an adapter
        adapted("adapted_ragged_f32", 45, 1032, "520,264", "8,24,64", 6, 7, dtype="f32",
                act="gelu_tanh", bias=True, residual=True, skew=0.0, idle=0.3),
    ]


#: What one drawn case may cost at most: the largest listed ones.
MOST_FLOPS = 2.0 * 4096 * 4096 * 28672
MOST_BYTES = 16384 * 4096 * 12.0


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "adapted"])
    f32 = rng.random() < 0.3
    dtype = "f32" if f32 else "bf16"
    if op == "norm":
        width = _log(rng, 64, 16384)
        tokens = _log(rng, 1, min(16384, MOST_BYTES / (16 * width)))
        post = rng.choice(["none", "rms", "layer"])
        return norm(None, tokens, width, dtype, "f32" if f32 else rng.choice(["bf16", "f32"]), post,
                    rng.choice(["none", "rms", "layer"]), rng.choice(["none", "vector", "rows"]),
                    rng.choice(["none", "sigmoid", "tanh"]), rng.random() < 0.5,
                    rng.choice([1.0, 0.22]), rng.choice([1.0, 1.25]))
    glu = rng.random() < 0.35
    act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"]) if glu or rng.random() < 0.4 else "none"
    k = 8 * _log(rng, 8, 1792)
    n = _log(rng, 16, 14336)
    most = min(4096.0, MOST_FLOPS / (2.0 * k * n * (2 if glu else 1)))
    tokens = _log(rng, 1, min(most, 512 if f32 else most))
    bias, residual = rng.random() < 0.4, rng.random() < 0.4
    if op == "linear":
        return linear(None, tokens, k, n, dtype, act, glu, bias, residual)
    n = max(8, n // 8 * 8)
    widths = "%d,%d" % (n, n) if glu else ",".join(
        str(w) for w in ([n] if rng.random() < 0.5 else [max(8, n // 16 * 8), max(8, n // 32 * 8)]))
    # (the pools' ranks together stay within what the largest listed case costs)
    ranks, pool = rng.choice([("8", 1), ("8", 1000), ("16", 8), ("16", 250), ("64", 8),
                              ("64", 64), ("8,16,32,64", 4), ("8,16,32,64", 64)])
    return adapted(None, tokens, k, widths, ranks, pool, rng.choice([1, 1, 7, 128, 512]), dtype,
                   act, glu, bias, residual, rng.choice([0.0, 1.1]), rng.choice([0.0, 0.25]))


# ----------------------------------------------------------------- inputs ----

def _tensors(case, seed):
    """Every tensor of the case, on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def rand(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    T = case["tokens"]
    if case["op"] == "norm":
        d = case["width"]
        s = {"h": rand(T, d, std=2.0, dtype=DTYPES[case["stream"]]), "o": rand(T, d, std=0.5)}
        for side in ("post", "pre"):
            s[side + "_weight"] = rand(d, std=0.1, mean=1.0) if case[side] != "none" else None
            s[side + "_bias"] = rand(d, std=0.1) if case[side] != "none" and case["bias"] else None
        s["gate"] = {"none": lambda: None, "vector": lambda: rand(d, std=0.5),
                     "rows": lambda: rand(T, d, std=0.5)}[case["gate"]]()
        return s
    widths = [case["n"]] * (1 + case["glu"]) if case["op"] == "linear" else \
        [int(w) for w in case["widths"].split(",")]
    k, wide = case["k"], sum(widths)
    out = wide // 2 if case["glu"] else wide
    s = {"x": rand(T, k), "w": rand(wide, k, std=1.0 / math.sqrt(k)),
         "bias": rand(wide, std=0.1) if case["bias"] else None,
         "residual": rand(T, out) if case["residual"] else None}
    if case["op"] == "adapted":
        _adapters(case, seed, s, widths, rand)
    return s


def _adapters(case, seed, s, widths, rand):
    """The requests' adapters and their weights: A ~ N(0, 1/(3 k)), B ~ N(0, 0.02^2), scale
    alpha / r with alpha = 2 r, one request after another."""
    r = np.random.default_rng(seed)
    T, pool = case["tokens"], case["pool"]
    starts = np.minimum(np.arange(0, T + case["segment"], case["segment"]), T).astype(np.int32)
    p = 1.0 / np.arange(1, pool + 1) ** case["skew"]
    ids = r.choice(pool, size=len(starts) - 1, p=p / p.sum()).astype(np.int32)
    ids[r.random(len(ids)) < case["idle"]] = -1
    ranks = [int(v) for v in case["ranks"].split(",")]
    used = sorted({int(i) for i in ids if i >= 0})
    s["starts"], s["ids"], s["widths"] = starts, ids, widths
    s["adapters"] = {i: {"rank": ranks[i % len(ranks)], "scale": 2.0} for i in used}
    for i in used:
        a = s["adapters"][i]
        a["A"] = [rand(a["rank"], case["k"], std=1.0 / math.sqrt(3 * case["k"])) for _ in widths]
        a["B"] = [rand(w, a["rank"], std=0.02) for w in widths]


def prepare(case, seed):
    s = _tensors(case, seed)
    s["case"] = case
    T, dt = case["tokens"], DTYPES[case["dtype"]]
    if case["op"] == "adapted":
        # the token's adapter, and the adapters' weights stacked along the ranks
        token = np.repeat(s["ids"], np.diff(s["starts"]))
        s["token"] = torch.from_numpy(token).to("cuda", torch.int64)
        A = list(s["adapters"].values())
        s["owner"] = torch.tensor([i for i, a in s["adapters"].items() for _ in range(a["rank"])],
                                  dtype=torch.int64, device="cuda")
        s["scale"] = torch.tensor([a["scale"] for a in A for _ in range(a["rank"])],
                                  dtype=torch.float32, device="cuda")
        s["A_all"] = [torch.cat([a["A"][p] for a in A]) if A else
                      torch.zeros(0, case["k"], dtype=dt, device="cuda")
                      for p in range(len(s["widths"]))]
        s["B_all"] = [torch.cat([a["B"][p] for a in A], 1) if A else
                      torch.zeros(w, 0, dtype=dt, device="cuda")
                      for p, w in enumerate(s["widths"])]
    if own:
        _handles(case, s, T, dt)
    return s


def _handles(case, s, T, dt):
    """What a serving loop keeps from call to call: the adapter pool, the batch's plan, outputs
    and workspaces."""
    import heterogeneous_adapter_batching_amd as hab
    if case["op"] == "norm":
        s["h_out"], s["u"] = torch.empty_like(s["h"]), torch.empty_like(s["o"])
        return
    wide, k = s["w"].shape
    s["y"] = torch.empty(T, wide // 2 if case["glu"] else wide, dtype=dt, device="cuda")
    if case["op"] == "linear":
        n = hab.linear_workspace_bytes(T, s["y"].shape[1], k, case["dtype"], case["glu"])
    else:
        widths, adapters = s["widths"], s["adapters"]
        pool = hab.Pool(1, [k] * len(widths), widths, r_max=64, dtype=case["dtype"],
                        slab_bytes=1 << 20)
        size = sum(pool.extent_bytes(a["rank"]) for a in adapters.values()) + (1 << 20)
        pool = hab.Pool(1, [k] * len(widths), widths, r_max=64, dtype=case["dtype"],
                        slab_bytes=size)
        for i, a in adapters.items():
            pool.register(i, a["rank"], a["scale"], [m.unsqueeze(0) for m in a["A"]],
                          [m.unsqueeze(0) for m in a["B"]])
        s["pool"] = pool
        s["plan"] = hab.Plan(pool, T, s["starts"], s["ids"]).upload(max_proj=len(widths))
        n = hab.sgmv_linear_workspace_bytes(pool, T, s["y"].shape[1], k, len(widths), case["glu"])
        s["projs"] = tuple(range(len(widths)))
        s["offsets"] = tuple(int(o) for o in np.cumsum([0] + widths[:-1]))
    s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------- runs ----

def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return {"norm": _plain_norm, "linear": _plain_linear, "adapted": _plain_adapted}[case["op"]](
        case, state)


def _own(case, s):
    import heterogeneous_adapter_batching_amd as hab
    if case["op"] == "norm":
        h, u = hab.block_norm(
            s["h"], s["o"], post=case["post"], post_weight=s["post_weight"],
            post_bias=s["post_bias"], gate=s["gate"], gate_act=case["gate_act"],
            alpha=case["alpha"], beta=case["beta"], pre=case["pre"], pre_weight=s["pre_weight"],
            pre_bias=s["pre_bias"], eps=1e-5, h_out=s["h_out"],
            u=s["u"] if case["pre"] != "none" else None)
        return {"h": h} if u is None else {"h": h, "u": u}
    epilogue = {"bias": s["bias"], "act": case["act"], "glu": case["glu"],
                "residual": s["residual"], "y": s["y"], "ws": s["ws"]}
    if case["op"] == "linear":
        return hab.frozen_linear(s["x"], s["w"], **epilogue)
    return hab.sgmv_linear(s["pool"], s["plan"], 0, s["projs"], s["offsets"], s["x"], s["w"],
                           **epilogue)


def _norm_rows(t, kind, weight, bias):
    if kind == "none":
        return t
    if kind == "layer":
        t = t - t.mean(1, keepdim=True)
    t = t / torch.sqrt((t * t).mean(1, keepdim=True) + 1e-5)
    t = t * weight.float()
    return t if bias is None else t + bias.float()


def _plain_norm(case, s):
    n = _norm_rows(s["o"].float(), case["post"], s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        g = s["gate"].float()
        n = n * {"none": lambda v: v, "sigmoid": lambda v: 1.0 / (1.0 + torch.exp(-v)),
                 "tanh": torch.tanh}[case["gate_act"]](g)
    h = s["h"].float() * case["beta"] + n * case["alpha"]
    out = {"h": h.to(s["h"].dtype)}
    if case["pre"] != "none":
        out["u"] = _norm_rows(h, case["pre"], s["pre_weight"], s["pre_bias"]).to(s["o"].dtype)
    return out


def _activate(t, act):
    if act == "relu":
        return torch.where(t > 0, t, torch.zeros_like(t))
    if act == "silu":
        return t / (1.0 + torch.exp(-t))
    if act == "gelu":
        return 0.5 * t * (1.0 + torch.erf(t * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * t * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (t + 0.044715 * t * t * t)))
    return t


def _epilogue(case, s, t):
    if s["bias"] is not None:
        t = t + s["bias"].float()
    if case["glu"]:
        n = t.shape[1] // 2
        t = _activate(t[:, :n], case["act"]) * t[:, n:]
    else:
        t = _activate(t, case["act"])
    if s["residual"] is not None:
        t = t + s["residual"].float()
    return t.to(s["x"].dtype)


def _plain_linear(case, s):
    return _epilogue(case, s, s["x"].float() @ s["w"].float().t())


def _plain_adapted(case, s):
    x = s["x"].float()
    # every token against every adapter in hand; the mask keeps its own one's ranks
    mask = (s["token"][:, None] == s["owner"][None, :]).float() * s["scale"]
    delta = torch.cat([((x @ A.float().t()) * mask) @ B.float().t()
                       for A, B in zip(s["A_all"], s["B_all"])], 1)
    return _epilogue(case, s, x @ s["w"].float().t() + delta)


# ------------------------------------------------------------- accounting ----

def work(case):
    T, e = case["tokens"], DTYPES[case["dtype"]].itemsize
    if case["op"] == "norm":
        d, hs = case["width"], DTYPES[case["stream"]].itemsize
        vectors = ((case["post"] != "none") + (case["pre"] != "none")) * (1 + case["bias"])
        rows = e + 2 * hs + (e if case["pre"] != "none" else 0)
        rows += e if case["gate"] == "rows" else 0
        vectors += case["gate"] == "vector"
        per = 4 + 6 * (case["post"] != "none") + 6 * (case["pre"] != "none")
        return {"bytes": T * d * rows + vectors * d * e, "flops": T * d * per}
    k = case["k"]
    widths = [case["n"]] * (1 + case["glu"]) if case["op"] == "linear" else \
        [int(w) for w in case["widths"].split(",")]
    wide = sum(widths)
    out = wide // 2 if case["glu"] else wide
    b = e * (T * k + wide * k + T * out * (1 + case["residual"]) + wide * case["bias"])
    f = 2 * T * k * wide
    if case["op"] == "adapted":
        # the adapters that a batch of these requests names, on average over draws
        requests = -(-T // case["segment"])
        p = 1.0 / np.arange(1, case["pool"] + 1) ** case["skew"]
        p = p / p.sum() * (1 - case["idle"])
        ranks = [int(v) for v in case["ranks"].split(",")]
        r = np.array([ranks[i % len(ranks)] for i in range(case["pool"])], dtype=np.float64)
        b += int(e * float(((1 - (1 - p) ** requests) * r).sum()) * sum(k + w for w in widths))
        f += int(2 * T * float((p * r).sum()) * sum(k + w for w in widths))
    return {"bytes": int(b), "flops": int(f)}


# ------------------------------------------------------------------ exact ----

def exact(case, seed):
    """The definitions in 64 bits, unrounded, from the same inputs."""
    s = {n: t.double() if torch.is_tensor(t) else t for n, t in _tensors(case, seed).items()}

    def normed(v, kind, weight, bias):
        if kind == "none":
            return v
        centre = v.mean(-1, keepdim=True) if kind == "layer" else 0.0
        power = (v - centre).square().mean(-1, keepdim=True)
        w = (v - centre) * torch.rsqrt(power + 1e-5) * weight
        return w + bias if bias is not None else w

    def acted(v):
        return {"none": lambda: v, "relu": lambda: v.clamp(min=0), "silu": lambda: v * torch.sigmoid(v),
                "gelu": lambda: v * 0.5 * torch.erfc(-v / math.sqrt(2.0)),
                "gelu_tanh": lambda: v * torch.sigmoid(
                    2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))}[case["act"]]()

    if case["op"] == "norm":
        n = normed(s["o"], case["post"], s["post_weight"], s["post_bias"])
        if s["gate"] is not None:
            n = n * {"none": lambda g: g, "sigmoid": torch.sigmoid, "tanh": torch.tanh}[
                case["gate_act"]](s["gate"])
        h = torch.add(case["beta"] * s["h"], n, alpha=case["alpha"])
        if case["pre"] == "none":
            return {"h": h}
        return {"h": h, "u": normed(h, case["pre"], s["pre_weight"], s["pre_bias"])}
    y = torch.matmul(s["x"], s["w"].t())
    if case["op"] == "adapted":
        edges = np.cumsum([0] + s["widths"])
        for lo, hi, i in zip(s["starts"][:-1], s["starts"][1:], s["ids"]):
            if i < 0:
                continue
            a = s["adapters"][int(i)]
            for p, (A, B) in enumerate(zip(a["A"], a["B"])):
                v = torch.matmul(s["x"][lo:hi], A.double().t())
                y[lo:hi, edges[p]:edges[p + 1]] += a["scale"] * torch.matmul(v, B.double().t())
    if s["bias"] is not None:
        y = y + s["bias"]
    if case["glu"]:
        gate, up = y.chunk(2, 1)
        y = acted(gate) * up
    else:
        y = acted(y)
    return y if s["residual"] is None else y + s["residual"]
