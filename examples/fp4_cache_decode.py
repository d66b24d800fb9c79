"""Decoding over a 4-bit KV cache: insert, attend, gather the keys' weights, evict.

A toy server on cuda:0: a few requests fill their caches token by token.  Every step
normalises and rotates the queries and inserts the new KV rows (qnorm_rope_kv_fp4_insert),
attends (fp4_attention) and adds up what attention each key got (fp4_attention_weights).
When a request reaches its limit, its rows of low weight leave (fp4_evict) and decoding
goes on over the rest.  The attention's output stands in for the layer's: it makes the
next token's queries and KV row.

    python examples/fp4_cache_decode.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kv_norm_rope_gb300 as k  # noqa: E402

BLOCK, EPS = 16, 1e-6


class Pool:
    """The cache's free blocks."""

    def __init__(self, blocks):
        self.blocks = blocks
        self.free = list(range(blocks))
        self.cache = torch.zeros(k.fp4_cache_bytes(blocks, BLOCK), dtype=torch.uint8, device="cuda")

    def take(self, n):
        taken, self.free = self.free[:n], self.free[n:]
        return taken


def main(steps=96, batch=3, heads=16, limit=64, budget=40, recent=8, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    wide = -(-limit // BLOCK)
    pool = Pool(2 * batch * wide)
    tables = [pool.take(wide) for _ in range(batch)]
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    weights = torch.zeros(batch, limit, device="cuda")
    norm_weight = (1 + 0.1 * randn(512)).to(torch.bfloat16)
    angles = torch.arange(steps + 1, device="cuda")[:, None] * 10000.0 ** (-torch.arange(32, device="cuda") / 32)
    cos_sin = torch.cat([angles.cos(), angles.sin()], 1).float()
    out = torch.empty(batch, 1, heads, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(batch, 1, heads, device="cuda")
    error = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, evictions = randn(batch, 512), 0
    for step in range(steps):
        # the new token of each request: its queries, its KV row, its slot
        q = (x[:, None, None] + randn(batch, 1, heads, 512)).to(torch.bfloat16)
        kv = (x + 0.5 * randn(batch, 512)).to(torch.bfloat16)
        positions = torch.full((batch,), step, dtype=torch.int64, device="cuda")
        at = lens.tolist()
        slots = torch.tensor([tables[b][n // BLOCK] * BLOCK + n % BLOCK for b, n in enumerate(at)], device="cuda")
        table = torch.tensor(tables, dtype=torch.int32, device="cuda")
        k.qnorm_rope_kv_fp4_insert(q.view(batch, heads, 512), kv, norm_weight, positions, cos_sin, slots,
                                   pool.cache, pool.blocks, BLOCK, EPS, device_error=error)
        lens += 1
        k.fp4_attention(q, pool.cache, pool.blocks, BLOCK, table, lens, 512 ** -0.5, out, lse=lse,
                        device_error=error)
        k.fp4_attention_weights(q, pool.cache, pool.blocks, BLOCK, table, lens, 512 ** -0.5, lse, weights,
                                device_error=error)
        x = out.float().mean((1, 2))
        if int(lens.max()) == limit:
            new = [pool.take(wide) for _ in range(batch)]
            new_table = torch.tensor(new, dtype=torch.int32, device="cuda")
            kept = torch.empty(batch, budget, dtype=torch.int32, device="cuda")
            new_weights = torch.empty(batch, budget, device="cuda")
            k.fp4_evict(pool.cache, pool.blocks, BLOCK, table, lens, weights, budget, recent, new_table,
                        kept, lens, new_weights, device_error=error)
            for old in tables:
                pool.free += old
            tables = new
            weights = torch.nn.functional.pad(new_weights, (0, limit - budget))
            evictions += 1
    if int(error.item()) != 0:
        raise RuntimeError(f"device error {int(error.item())}")
    print(f"{steps} steps, {evictions} evictions; lengths {lens.tolist()}; "
          f"attention kept so far {[round(float(w), 2) for w in weights.sum(1)]}")
    return lens.tolist(), weights, x


if __name__ == "__main__":
    main()
