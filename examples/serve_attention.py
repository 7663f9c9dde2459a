#!/usr/bin/env python3
"""Serving steps with attention over the unified pool: adapters and KV cache share one
paged pool, the scheduler admits requests by its free pages, and every step runs the
layer's LoRA projection (q, k and v packed), builds the block tables, stores the new
tokens' keys and values with rotary positions, and attends: new prompts over themselves,
running requests over their caches.

    python examples/serve_attention.py --steps 16 --requests 24
"""

import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import workloads  # noqa: E402
from heterogeneous_lora_amd import runtime  # noqa: E402


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=16)
    p.add_argument("--requests", type=int, default=24)
    p.add_argument("--window", type=int, default=0, help="sliding window, 0: none")
    p.add_argument("--softcap", type=float, default=0.0)
    p.add_argument("--kv-bits", type=int, default=16, choices=(16, 4), help="of a cached value")
    p.add_argument("--seed", type=int, default=0)
    args = p.parse_args()
    heads, kv_heads, dim = 16, 4, 64
    wl = workloads.random_small(args.seed + 400, dtype="f16", n_adapters=16, d_in=1024,
                                d_out=(heads + 2 * kv_heads) * dim, page_elems=512, n_tokens=1, n_segments=0,
                                rank_choices=(8, 16, 32, 64))
    loop = runtime.AttentionLoop(wl, n_pages=20000, n_q_heads=heads, n_kv_heads=kv_heads, head_dim=dim, max_len=256,
                                 rope=runtime.Rope(dim), attention=dict(window=args.window, softcap=args.softcap),
                                 max_batch_tokens=1024, max_running=64, kv_bits=args.kv_bits)
    rng = np.random.default_rng(args.seed)
    for r in range(args.requests):
        loop.submit(r, int(rng.integers(wl.n_adapters)), int(rng.integers(8, 160)), int(rng.integers(4, 32)))
    for step in range(args.steps):
        start = time.perf_counter()
        b, qkv, out = loop.step(seed=step)
        torch.cuda.synchronize()
        ms = 1e3 * (time.perf_counter() - start)
        size = 0.0 if out is None else float(out.float().abs().mean())
        print(f"step {b['step']}: {b['n_tokens']} tokens ({len(b['seg_adapter'])} prompts, "
              f"{b['token_adapter'].size} running), {b['free_pages']} pages free, mean |out| {size:.4f}, {ms:.1f} ms",
              flush=True)
    loop.close()


if __name__ == "__main__":
    main()
