"""Decoding with drafted trees over one layer's latent cache: prompts and drafts
are appended (normalised, rotated, the indexer's keys encoded), the tree's nodes
attend to the context and their ancestors, the accepted path is kept, and the
indexer chooses keys for the token behind it.

    python examples/draft_tree.py

Random activations stand in for a model's projections, and a random node of
each tree for the longest accepted one.
"""
import os
import random
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fp8_scoring_exact_gb300 import binding as B  # noqa: E402

H, DC, DP, DI, PAGE = 16, 512, 64, 128, 64
SCALE = 192 ** -0.5
BF16, I32 = torch.bfloat16, torch.int32


def rotations(n):
    """cos and sin of 32 angles at every position."""
    a = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def ints(v):
    return torch.tensor(v, dtype=I32, device="cuda")


def draft(rng, n):
    """Parents of a tree's nodes (node 0 is the last accepted token), and each node's ancestors with itself."""
    parents = [-1] + [rng.randrange(i) for i in range(1, n)]
    seen = []
    for i, p in enumerate(parents):
        seen.append((seen[p] if p >= 0 else []) + [i])
    return seen


def main(prompts=(300, 61, 700), nodes=16, steps=4, topk=128, seed=0, say=print):
    g, rng = torch.Generator(device="cuda").manual_seed(seed), random.Random(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=BF16)

    nb, pages = len(prompts), [-(-(n + nodes * (steps + 1)) // PAGE) for n in prompts]
    order = list(range(sum(pages)))
    rng.shuffle(order)
    table = torch.full((nb, max(pages)), -1, dtype=I32)
    for b, n in enumerate(pages):
        table[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=I32)
    table = table.cuda()
    P = sum(pages)
    ckv, kpe = (torch.zeros((P, PAGE, d), dtype=BF16, device="cuda") for d in (DC, DP))
    k_cache, k_scale = torch.zeros((P, PAGE, DI), dtype=torch.uint8, device="cuda"), torch.ones((P, PAGE), device="cuda")
    cos_sin = rotations(2048)
    norm = dict(c_norm=(torch.ones(DC, device="cuda"), 1e-6),
                index_norm=(torch.ones(DI, device="cuda"), torch.zeros(DI, device="cuda"), 1e-6))
    lens = torch.zeros(nb, dtype=I32, device="cuda")

    def append(counts, positions=None):
        """Latents, rope parts and index keys of counts[b] new tokens per sequence."""
        cu, T = [sum(counts[:i]) for i in range(nb + 1)], sum(counts)
        joint = normal(T, DC + DP)
        B.latent_cache_append(joint[:, :DC], joint[:, DC:], cos_sin, ints(cu), table, lens, ckv, kpe, index_k=normal(T, DI),
                              hadamard=True, k_cache=k_cache, k_cache_scale=k_scale, positions=positions, new_lens=lens,
                              **norm)

    append(list(prompts))
    say(f"prompts of {lens.tolist()} tokens in {P} pages")
    for step in range(steps):
        trees = [draft(rng, nodes) for _ in range(nb)]
        before = lens.tolist()
        # a node's position is its depth behind the context; its slot is its place among the nodes
        positions = ints([n + len(s) - 1 for n, t in zip(before, trees) for s in t])
        append([nodes] * nb, positions)
        q_nope, q_pe, x = normal(nb, nodes, H, DC), normal(nb * nodes, H, DP), normal(nb * nodes, 64, DI)
        codes, scale, q_pe = B.indexer_encode(x, cos_sin, positions, hadamard=True, pe=q_pe)
        mask = torch.tensor([[[sum(1 << j for j in s)] for s in t] for t in trees], dtype=torch.int64, device="cuda")
        out, lse = B.latent_attention_tree(q_nope, q_pe.view(nb, nodes, H, DP), ckv, kpe, table, lens, mask, SCALE)
        # what a model would accept: some node and its ancestors
        paths = [t[rng.randrange(nodes)] for t in trees]
        B.latent_cache_accept(ckv, kpe, table, lens, ints([nodes] * nb),
                              ints([p + [-1] * (nodes - len(p)) for p in paths]), ints([len(p) for p in paths]),
                              k_cache=k_cache, k_cache_scale=k_scale, new_lens=lens)
        say(f"step {step}: {nodes} nodes a sequence, accepted {[len(p) for p in paths]}, lengths {lens.tolist()}")
    # the indexer's choice for the last accepted token of each sequence
    last = torch.tensor([b * nodes + p[-1] for b, p in enumerate(paths)], device="cuda")
    w = torch.randn((nb, 1, 64), generator=g, device="cuda")
    chosen = B.indexer_topk_paged(codes[last][:, None].contiguous(), scale[last][:, None].contiguous(), k_cache, k_scale, w,
                                  table, lens, K=topk)
    status = B.latent_last_status()
    say(f"top {topk} of {lens.tolist()} keys: {[int((c >= 0).sum()) for c in chosen[:, 0]]} slots, status {status}")
    return lens.tolist(), out, lse, chosen, status


if __name__ == "__main__":
    main()
