"""Run with HAB_LORA_LIB naming the bounds-checked debug build: attention and
rotary positions on plans whose device tables a stray write has changed.

Each field of the entries that the kernels read (parts, joins, tokens) is set
outside what the batch holds.  Every launch completes and sets the field's bit,
what lies around the outputs stays as it was, and the plan uploaded again gives
the first result with no bit set.  Tensors, cache, page table and workspace lie
inside larger ones, and the changed values stay small, so that even an access
that no check held back would be inside them.
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for p in (ROOT, os.path.join(ROOT, "tests")):
    if p not in sys.path:
        sys.path.insert(0, p)

import torch  # noqa: E402

import heterogeneous_adapter_batching_amd as hab  # noqa: E402
from attention_reference import Batch  # noqa: E402

TOKEN, ROW = hab.LORA_DEBUG_TOKEN, hab.LORA_DEBUG_ROW
SPARE = 64                       # rows around the outputs, and of the page table

# (float32, new tokens, keys): single tokens in parts and not, chunks, float32
BATCHES = (("bf16", [1, 1, 1], [3000, 40, 700]), ("bf16", [1, 1], [90, 40]),
           ("bf16", [40, 70], [9000, 300]), ("f32", [20, 3], [400, 30]))


def around(t, spare, rows):
    """A copy of t inside a larger tensor, as (the larger one, t)."""
    big = torch.full((t.shape[0] + 2 * spare, *t.shape[1:]), 3, dtype=t.dtype, device="cuda")
    big[spare:spare + rows] = t
    return big, big[spare:spare + rows]


def words(ws, at, count):
    return ws.view(torch.int32)[at // 4:at // 4 + count]


def main():
    torch.cuda.set_device(0)
    enabled, _ = hab.debug_checks(clear=True)
    assert enabled, f"{hab.LIB_PATH} is not the debug build"
    for dtype, new, kv in BATCHES:
        b = Batch(new, kv, heads=8, kv_heads=2, dim=64, page=64, dtype=dtype, seed=1)
        T, S = b.tokens, len(new)
        q_all, q = around(b.q, SPARE, T)
        (k_all, k), (v_all, v) = (around(t.nan_to_num(), 40, t.shape[0]) for t in (b.k, b.v))
        # (a table of more sequences and pages than the batch's, all of them valid)
        table = torch.zeros(S + SPARE, b.pages.shape[1] + SPARE, dtype=torch.int32, device="cuda")
        table[:S, :b.pages.shape[1]] = b.pages.clamp(min=0)
        pages = table[:, :b.pages.shape[1]]
        plan = hab.AttentionPlan(8, 2, 64, 64, new, kv, dtype=dtype)
        ws = torch.zeros(plan.workspace_bytes() + (1 << 20), dtype=torch.uint8, device="cuda")
        plan.upload(ws=ws)
        o_all, o = around(torch.zeros_like(q), SPARE, T)
        stats = plan.stats()

        def attend():
            o_all.fill_(3)
            hab.paged_attention(plan, q, k, v, pages, o=o)
            torch.cuda.synchronize()
            assert (o_all[:SPARE] == 3).all() and (o_all[SPARE + T:] == 3).all()
            return o.clone()

        first = attend()
        assert hab.debug_checks(clear=True)[1] == 0, "bits set by a sound plan"
        assert first.isfinite().all()
        units = -(-8 * T // 256) * 256
        joins = units + -(-36 * stats["units"] // 256) * 256
        keys = pages.shape[1] * 64
        changes = [("unit", units, 9, i, f, x, bit) for i in (0, stats["units"] - 1) for f, x, bit in (
            (0, S, ROW), (0, S + 5, ROW), (1, 2, TOKEN), (1, -1, TOKEN), (2, -16, TOKEN),
            (3, 8 * T + 64, TOKEN), (4, -1, TOKEN), (4, T, TOKEN), (6, 16, ROW), (6, -64, ROW),
            (7, keys + 1, ROW), (7, keys + 64, ROW), (8, 3000, ROW), (8, -2, ROW))]
        changes += [("join", joins, 6, i, f, x, bit) for i in range(min(stats["joins"], 2)) for f, x, bit in (
            (0, T, TOKEN), (1, 2, TOKEN), (2, -16, TOKEN), (3, 8 * T + 64, TOKEN), (4, -1, ROW),
            (4, 3000, ROW), (5, 3000, ROW), (5, -1, ROW))]
        for what, at, size, i, f, x, bit in changes:
            print(f"[debug] {dtype} {new} {kv}: {what} {i}, word {f} = {x}", flush=True)
            words(ws, at + 4 * (size * i + f), 1).fill_(x)
            torch.cuda.synchronize()
            attend()
            bits = hab.debug_checks(clear=True)[1]
            assert bits == bit, (bits, bit)
            plan.upload(ws=ws)
            assert torch.equal(attend(), first)
            assert hab.debug_checks(clear=True)[1] == 0

        # rotary positions: a token that is outside goes nowhere
        n = b.kv_heads * b.dim
        rows = torch.randn(T, 2 * n, device="cuda").to(q.dtype)
        freqs = hab.rotary_frequencies(64, device="cuda")
        for f, x in ((0, S), (0, S + 5), (0, -1), (1, keys), (1, keys + 70)):
            print(f"[debug] {dtype} {new} {kv}: token 0, word {f} = {x}", flush=True)
            words(ws, 4 * f, 1).fill_(x)
            torch.cuda.synchronize()
            before = k_all.clone(), v_all.clone()
            hab.rotary_append(plan, None, rows[:, :n], rows[:, n:], k, v, pages, freqs)
            torch.cuda.synchronize()
            bits = hab.debug_checks(clear=True)[1]
            assert bits == ROW, bits
            pos, page, slot = b.places()
            for was, now, one in ((before[0], k_all, k), (before[1], v_all, v)):
                mine = torch.zeros_like(one, dtype=torch.bool)
                mine[page[1:], :, slot[1:]] = True
                free = torch.ones_like(now, dtype=torch.bool)
                free[40:40 + one.shape[0]] = ~mine
                assert torch.equal(was[free], now[free])
            plan.upload(ws=ws)
    print("[debug] all checks passed", flush=True)


if __name__ == "__main__":
    main()
