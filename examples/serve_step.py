"""A small serving loop on the paged pool, end to end (needs an MI355X):

    python examples/serve_step.py

  1. a cached 1024-token chunk is rehydrated at its new position into the pool (kamera.h);
  2. every request forks the chunk's last, partly filled page and goes on from there;
  3. decode steps: per layer, append the new token's K/V rows and attend to the shared chunk
     and the request's own tokens;
  4. half the requests end; the pages of the rest are moved together and decoding goes on.

Random weights stand in for a model; each step's attention is checked against 64-bit NumPy.
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from oracle import step_oracle as so  # noqa: E402
from position_free_kv_amd import abi, step  # noqa: E402

LAYERS, HEADS, KV_HEADS, DIM, PAGE = 4, 16, 4, 128, 16
F = KV_HEADS * DIM
CHUNK, START, REQUESTS, STEPS, PAGES = 1000, 5000, 6, 12, 256


def main() -> None:
    torch.manual_seed(0)
    dev = "cuda"
    lay = abi.make_layout(abi.GQA, abi.BF16, LAYERS, num_kv_heads=KV_HEADS, head_dim=DIM, rope_base=1e6, page_size=PAGE)
    k_pool, v_pool = (torch.zeros(LAYERS, PAGES, PAGE, F, dtype=torch.bfloat16, device=dev) for _ in range(2))
    pool = abi.make_pool(k_pool, v_pool, PAGES)
    free = list(np.random.default_rng(0).permutation(PAGES))  # the caller keeps the books

    # 1. the shared chunk: canonical rows turned to their new position, straight into pages
    shared = np.array([free.pop() for _ in range(-(-CHUNK // PAGE))], np.int32)
    canon = [torch.randn(LAYERS, CHUNK, F, device=dev).bfloat16() for _ in range(2)]
    chunk = abi.ChunkDesc(num_tokens=CHUNK, delta=START, flags=0, k_src=canon[0], v_src=canon[1], block_table=shared)
    ws = torch.empty(abi.batch_workspace_bytes(lay, [chunk]), dtype=torch.uint8, device=dev)
    abi.rehydrate_batched(lay, [chunk], pool, ws)

    # 2. whole pages of the chunk are shared; its tail page is copied for every request
    whole, tail = CHUNK // PAGE, CHUNK % PAGE
    tables = np.zeros((REQUESTS, 8), np.int32)
    tables[:, 0] = [free.pop() for _ in range(REQUESTS)]
    copies = torch.empty(step.copy_pages_workspace_bytes(PAGES), dtype=torch.uint8, device=dev)
    step.copy_pages(lay, pool, np.full(REQUESTS, shared[whole]), tables[:, 0], copies)

    s = step.Step(num_q_heads=HEADS, block_tables=tables, num_tokens=tail, num_queries=1, prefix=0, position0=START + whole * PAGE,
                  prefixes=[dict(block_table=shared, num_tokens=whole * PAGE)])
    qw, kw = (1 + 0.1 * torch.randn(DIM, device=dev)).bfloat16(), (1 + 0.1 * torch.randn(DIM, device=dev)).bfloat16()
    scale, worst = DIM ** -0.5, 0.0
    for t in range(STEPS):
        # 3. one token a request: its page, the step's description, then the layers
        s.requests["num_tokens"] += 1
        n = len(s.requests)
        for r in range(n):
            last = int(s.requests["num_tokens"][r]) - 1
            if last % PAGE == 0:
                tables[r, last // PAGE] = free.pop()
        work = torch.empty(step.workspace_bytes(lay, s), dtype=torch.uint8, device=dev)
        plan = step.upload(lay, s, pool, work)
        for layer in range(LAYERS):
            rows = torch.randn(n, (HEADS + 2 * KV_HEADS) * DIM, device=dev).bfloat16()  # a layer's fused projection
            q, out = torch.empty(n, HEADS * DIM, dtype=torch.bfloat16, device=dev), torch.empty(n, HEADS * DIM, dtype=torch.bfloat16, device=dev)
            step.append(plan, layer, q=rows[:, :HEADS * DIM], k=rows[:, HEADS * DIM:-F], v=rows[:, -F:], q_out=q, q_weight=qw, k_weight=kw)
            step.attend(plan, layer, q, out, scale)
        # the last layer, in 64 bits
        k, v = (p[LAYERS - 1].view(-1, F).double().cpu().numpy() for p in (k_pool, v_pool))
        q64, g = q.double().cpu().numpy().reshape(n, HEADS, DIM), HEADS // KV_HEADS
        for r in range(n):
            own = int(s.requests["num_tokens"][r])
            at = np.concatenate([so.slots(shared, 0, whole * PAGE, PAGE), so.slots(tables[r], 0, own, PAGE)])
            for h in range(KV_HEADS):
                sl = slice(h * DIM, (h + 1) * DIM)
                o, _, a, _ = so.attend(q64[r:r + 1, h * g:(h + 1) * g], k[at, sl], v[at, sl], scale, [at.size - 1])
                got = out[r, h * g * DIM:(h + 1) * g * DIM].double().cpu().numpy().reshape(g, DIM)
                worst = max(worst, float((np.abs(got - o[0]) / (a[0] + np.abs(o[0]))).max()))
        if t == STEPS // 2:
            # 4. half the requests leave: what they held is free, the rest moves to the pool's start
            tables = tables[:n // 2].copy()
            used = -(-s.requests["num_tokens"][:n // 2] // PAGE)
            live = [shared] + [tables[r, :used[r]] for r in range(n // 2)]
            count = step.compact_pages(lay, pool, live, copies)
            free = list(range(PAGES - 1, count - 1, -1))
            s = step.Step(num_q_heads=HEADS, block_tables=tables, num_tokens=s.requests["num_tokens"][:n // 2].copy(), num_queries=1, prefix=0,
                          position0=START + whole * PAGE, prefixes=[dict(block_table=shared, num_tokens=whole * PAGE)])
            print(f"step {t}: {n} -> {n // 2} requests, {count} live pages together", flush=True)
    # a probability and an output rounded to bf16: 2^-8 of the weighted |v| each
    assert worst < 2.0 ** -7, worst
    print(f"serve_step ok: {STEPS} steps, worst difference {worst:.2e} of the weighted |v|", flush=True)


if __name__ == "__main__":
    main()
