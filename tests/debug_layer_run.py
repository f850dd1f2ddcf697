"""Run with HAB_LORA_LIB naming the bounds-checked debug build: the product
with adapters on good plans fails no check and gives the exact result; with
its plan tables' extents moved past the slab, as a stray write would leave
them, every launch completes and the slab bit is set."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for p in (ROOT, os.path.join(ROOT, "tests")):
    if p not in sys.path:
        sys.path.insert(0, p)

import numpy as np  # noqa: E402
import torch  # noqa: E402

import heterogeneous_adapter_batching_amd as hab  # noqa: E402


def ints(g, *shape):
    return torch.randint(-1, 2, shape, generator=g).to(torch.bfloat16).cuda()


def main():
    torch.cuda.set_device(0)
    enabled, _ = hab.debug_checks(clear=True)
    assert enabled, f"{hab.LIB_PATH} is not the debug build"
    g = torch.Generator().manual_seed(1)
    # a few tokens; a joined product; one launch with the delta's own tiles
    for T, k, n, seg in ((6, 256, 64, 1), (100, 2048, 256, 1), (2048, 64, 4096, 512)):
        pool = hab.Pool(1, [k], [n], 64, "bf16", slab_bytes=8 << 20)
        ads = []
        for a, rank in enumerate((8, 40)):
            ads.append((ints(g, 1, rank, k), ints(g, 1, n, rank)))
            pool.register(a, rank, 1.0, [ads[a][0]], [ads[a][1]])
        starts = np.minimum(np.arange(0, T + seg, seg), T).astype(np.int32)
        ids = np.arange(len(starts) - 1, dtype=np.int32) % 2
        plan = hab.Plan(pool, T, starts, ids).upload(1)
        x, w = ints(g, T, k), ints(g, n, k)
        y = hab.sgmv_linear(pool, plan, 0, [0], [0], x, w)
        token = torch.from_numpy(np.repeat(ids, np.diff(starts))).cuda()
        ref = x.double() @ w.double().t()
        for a, (A, B) in enumerate(ads):
            rows = token == a
            ref[rows] += (x[rows].double() @ A[0].double().t()) @ B[0].double().t()
        assert torch.equal(y, ref.to(torch.bfloat16)), T
        _, bits = hab.debug_checks(clear=True)
        assert bits == 0, (T, bits)
        img = plan.ws.cpu().numpy().copy()
        words = img[:img.size // 16 * 16].view(np.int32).reshape(-1, 4)
        hits = 0
        for a in range(2):
            q = pool.query(a)
            at = (words[:, 0] == (q["offset"] & 0xffffffff)) & (words[:, 1] == q["offset"] >> 32) & \
                 (words[:, 2] == q["r_pad"])
            words[at, 0] = pool.slab.numel()
            hits += int(at.sum())
        assert hits
        plan.ws.copy_(torch.from_numpy(img))
        hab.sgmv_linear(pool, plan, 0, [0], [0], x, w)
        _, bits = hab.debug_checks(clear=True)
        assert bits & hab.LORA_DEBUG_SLAB, (T, bits)
        print(f"[debug] {T} tokens: {hits} extents moved, bits {bits:#x}", flush=True)
    print("[debug] all checks passed", flush=True)


if __name__ == "__main__":
    main()
