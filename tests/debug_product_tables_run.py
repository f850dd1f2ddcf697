"""Run with HAB_LORA_LIB naming the bounds-checked debug build: sgmv_linear on
plans whose device tables a stray write has changed.

Each kind of entry that the product's kernels read (a token row, a position's
group, a group's first position, its padded rank, a block's token count) is
set outside what the plan holds.  Every launch completes and sets the kind's
bit, rows of y in front of and behind the batch stay as they were, and the
plan uploaded again gives the exact result with no bit set.  x, y and the
residual lie inside larger tensors, and the changed values stay small, so that
even an access that no check held back would be inside them.
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for p in (ROOT, os.path.join(ROOT, "tests")):
    if p not in sys.path:
        sys.path.insert(0, p)

import numpy as np  # noqa: E402
import torch  # noqa: E402

import heterogeneous_adapter_batching_amd as hab  # noqa: E402

SPARE = 16                       # rows in front of and behind every tensor
RANKS = (8, 40)
# a few tokens; a product in parts; one launch with the delta's own tiles
SIZES = ((6, 256, 64, 1), (100, 2048, 256, 1), (2048, 64, 4096, 512))
SLAB, TOKEN, ROW = hab.LORA_DEBUG_SLAB, hab.LORA_DEBUG_TOKEN, hab.LORA_DEBUG_ROW


def ints(g, *shape):
    return torch.randint(-1, 2, shape, generator=g).to(torch.bfloat16).cuda()


def tables(img, pool, T, groups):
    """Where the plan's image (32-bit words) keeps what the kernels read: the
    words of token rows, position groups, groups' first positions and ranks,
    blocks' token counts."""
    w = img.view(np.int32)
    w8, w4 = w[:w.size // 8 * 8].reshape(-1, 8), w[:w.size // 4 * 4].reshape(-1, 4)
    ext = {}
    for a in range(groups):
        q = pool.query(a)
        ext[a] = (np.uint32(q["offset"] & 0xffffffff).view(np.int32), q["offset"] >> 32, q["r_pad"])
    found = {"token": np.arange(T), "group": [], "first": [], "rank": [], "rows": []}
    one = np.float32(1.0).view(np.int32)
    is_pos = np.zeros(len(w8), bool)
    for lo, hi, r in ext.values():
        pos = (w8[:, 0] == lo) & (w8[:, 1] == hi) & (w8[:, 2] == r) & (w8[:, 6] == one) & (w8[:, 7] == 0)
        is_pos |= pos
        found["group"] += list(np.nonzero(pos)[0] * 8 + 3)
        blk = (w8[:, 2] == r) & (w8[:, 4] == one) & (w8[:, 6] == lo) & (w8[:, 7] == hi)
        found["rows"] += list(np.nonzero(blk)[0] * 8 + 1)
    for lo, hi, r in ext.values():
        grp = (w4[:, 0] == lo) & (w4[:, 1] == hi) & (w4[:, 2] == r) & ~np.repeat(is_pos, 2)[:len(w4)]
        found["first"] += list(np.nonzero(grp)[0] * 4 + 3)
        found["rank"] += list(np.nonzero(grp)[0] * 4 + 2)
    return found


def main():
    torch.cuda.set_device(0)
    enabled, _ = hab.debug_checks(clear=True)
    assert enabled, f"{hab.LIB_PATH} is not the debug build"
    g = torch.Generator().manual_seed(2)
    for T, k, n, seg in SIZES:
        pool = hab.Pool(1, [k], [n], 64, "bf16", slab_bytes=8 << 20)
        ads = []
        for a, rank in enumerate(RANKS):
            ads.append((ints(g, 1, rank, k), ints(g, 1, n, rank)))
            pool.register(a, rank, 1.0, [ads[a][0]], [ads[a][1]])
        starts = np.minimum(np.arange(0, T + seg, seg), T).astype(np.int32)
        ids = np.arange(len(starts) - 1, dtype=np.int32) % 2
        plan = hab.Plan(pool, T, starts, ids).upload(1)
        ws = plan.ws
        xb, rb = ints(g, T + 2 * SPARE, k), ints(g, T + 2 * SPARE, n)
        yb = torch.empty(T + 2 * SPARE, n, dtype=torch.bfloat16, device="cuda")
        w = ints(g, n, k)
        x, r, y = (t[SPARE:SPARE + T] for t in (xb, rb, yb))
        token = torch.from_numpy(np.repeat(ids, np.diff(starts))).cuda()
        ref = x.double() @ w.double().t()
        for a, (A, B) in enumerate(ads):
            rows = token == a
            ref[rows] += (x[rows].double() @ A[0].double().t()) @ B[0].double().t()
        ref = (ref + r.double()).to(torch.bfloat16)

        def call():
            yb.fill_(7.0)
            hab.sgmv_linear(pool, plan, 0, [0], [0], x, w, residual=r, y=y)
            _, bits = hab.debug_checks(clear=True)
            assert bool((yb[:SPARE] == 7).all()) and bool((yb[SPARE + T:] == 7).all())
            return bits

        assert call() == 0 and torch.equal(y, ref), T
        good = ws.cpu().numpy().copy()
        at = tables(good, pool, T, len(RANKS))
        assert len(at["group"]) == T and len(at["first"]) == len(RANKS) and at["rows"]
        kinds = [("token", v, TOKEN) for v in (T, T + 9, -2, -9)] + [("rows", 1 << 20, ROW)]
        if T == 2048:                    # the walk over groups is the one launch's
            kinds += [("group", len(RANKS) + 3, ROW), ("group", -4, ROW), ("first", T + 5, ROW),
                      ("first", -3, ROW), ("rank", 1 << 20, SLAB), ("rank", 0, SLAB), ("rank", -8, SLAB)]
        for kind, value, bit in kinds:
            print(f"[debug] {T} tokens: {kind} {value}", flush=True)
            img = good.copy()
            img.view(np.int32)[at[kind][::3] if kind == "token" else at[kind]] = value
            ws.copy_(torch.from_numpy(img))
            bits = call()
            assert bits & bit, (T, kind, value, bits)
            plan.upload(1, ws=ws)
            assert call() == 0 and torch.equal(y, ref), (T, kind, value)
    print("[debug] all checks passed", flush=True)


if __name__ == "__main__":
    main()
