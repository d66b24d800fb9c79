"""Decoding with trees of drafted tokens over the FP8 KV cache.

A toy server on cuda:0.  Every step drafts a small tree of tokens for each request, inserts their
KV rows behind the context (qnorm_rope_kv_quant_insert), attends for all of them at once, each over
the context and its own ancestors (latent_attention with tree), turns the output's trailing dims
back by the token's position (rope_rows), accepts one path and moves its rows together
(tree_keep).  The angles are those of a context stretched by YaRN (rope_frequencies,
rope_table).  The attention's output stands in for the layer's.

    python examples/tree_decode.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kv_norm_rope_gb300 as k  # noqa: E402

BLOCK, EPS = 16, 1e-6
PARENTS = [None, 0, 0, 1, 1, 2, 3]  # of the drafted tokens: two guesses behind the first, and so on


def tree_words():
    words = []
    for j, parent in enumerate(PARENTS):
        words.append(1 << j | (0 if parent is None else words[parent]))
    return words


def main(steps=32, batch=3, heads=16, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    drafted, words = len(PARENTS), tree_words()
    depth = torch.tensor([bin(word).count("1") - 1 for word in words], device="cuda")
    paths = [[i for i in range(drafted) if word >> i & 1] for word in words]
    longest = max(len(path) for path in paths)
    wide = -(-(steps * longest + drafted) // BLOCK)
    blocks = batch * wide
    cache = torch.zeros(k.fp8_cache_bytes(blocks, BLOCK), dtype=torch.uint8, device="cuda")
    table = torch.arange(blocks, dtype=torch.int32, device="cuda").view(batch, wide)
    cos_sin = torch.empty(wide * BLOCK, 64, device="cuda")
    k.rope_table(k.rope_frequencies(64, 10000.0, k.ROPE_YARN, factor=4.0, original_positions=64.0), cos_sin)
    norm_weight = (1 + 0.1 * randn(512)).to(torch.bfloat16)
    tree = torch.tensor(words, device="cuda").repeat(batch, 1)
    workspace = torch.empty(k.latent_attention_workspace_bytes(), dtype=torch.uint8, device="cuda")
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    error = torch.zeros(1, dtype=torch.int32, device="cuda")
    x, accepted = randn(batch, 512), 0
    requests = torch.arange(batch, device="cuda")
    for step in range(steps):
        # the drafted tokens: their queries, KV rows, positions (the depth in the tree) and slots
        q = (x[:, None, None] + randn(batch, drafted, heads, 512)).to(torch.bfloat16)
        kv = (x[:, None] + 0.5 * randn(batch, drafted, 512)).to(torch.bfloat16)
        positions = (lens[:, None] + depth).long().view(-1)
        at = lens[:, None].long() + torch.arange(drafted, device="cuda")
        slots = (table[requests[:, None], at // BLOCK].long() * BLOCK + at % BLOCK).view(-1)
        k.qnorm_rope_kv_quant_insert(q.view(-1, heads, 512), kv.view(-1, 512), norm_weight, positions, cos_sin,
                                     slots, cache, blocks, BLOCK, EPS, device_error=error)
        lens += drafted
        out = torch.empty_like(q)
        k.latent_attention(k.STORE_FP8, q, cache, blocks, BLOCK, table, lens, 512 ** -0.5, out, tree=tree,
                           workspace=workspace, device_error=error)
        k.rope_rows(out.view(-1, heads, 512), positions, cos_sin, inverse=True, device_error=error)
        # a drafter's guesses that hold: here, the path of the token with the largest output
        best = out.float().square().mean((2, 3)).argmax(1).tolist()
        path = torch.full((batch, drafted), -1, dtype=torch.int32)
        for b, j in enumerate(best):
            path[b, :len(paths[j])] = torch.tensor(paths[j], dtype=torch.int32)
        path_lens = torch.tensor([len(paths[j]) for j in best], dtype=torch.int32)
        k.tree_keep(k.STORE_FP8, cache, blocks, BLOCK, table, lens, path.cuda(), path_lens.cuda(), lens,
                    device_error=error)
        accepted += int(path_lens.sum())
        x = out.float().mean(2)[requests, best]
    if int(error.item()) != 0:
        raise RuntimeError(f"device error {int(error.item())}")
    print(f"{steps} steps, {accepted / (steps * batch):.2f} tokens accepted in one; lengths {lens.tolist()}")
    return lens.tolist(), x


if __name__ == "__main__":
    main()
