"""Serving one latent-attention layer: prefill in the expanded form, decode over
the paged latent cache with accumulated key weights, eviction to a budget, and
decode of a batch behind a shared prompt.

    python examples/latent_decode.py

A layer with random weights stands in for a model's: per head h, k_nope = W_uk[h] c
and v = W_uv[h] c of a token's latent vector c.  Decode works on the latents
themselves (the absorbed form): the query is multiplied by W_uk[h] once, and the
output, a sum of latents, by W_uv[h].
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fp8_scoring_exact_gb300 import binding as B  # noqa: E402

H, DC, DN, DP, DV, PAGE = 16, 512, 128, 64, 128, 64
SCALE = (DN + DP) ** -0.5
BF16 = torch.bfloat16


class Layer:
    def __init__(self, gen):
        self.gen = gen
        self.w_uk = self.normal(H, DN, DC, scale=DC ** -0.5)
        self.w_uv = self.normal(H, DV, DC, scale=DC ** -0.5)

    def normal(self, *shape, scale=1.0):
        return (torch.randn(shape, generator=self.gen, device="cuda") * scale).to(BF16)

    def token(self, *rows):
        """Latents, rope keys and queries of new tokens (a model's projections)."""
        return self.normal(*rows, DC), self.normal(*rows, DP), self.normal(*rows, H, DN), self.normal(*rows, H, DP)

    def prefill(self, ckv, kpe, q_nope, q_pe, cu):
        """Every prompt token's output, [T, H, DV]: keys and values expanded per head."""
        k_nope = torch.einsum("tc,hdc->thd", ckv, self.w_uk)
        v = torch.einsum("tc,hdc->thd", ckv, self.w_uv)
        out, _ = B.latent_attention_prefill(torch.cat([q_nope, q_pe], -1), k_nope, kpe, v, cu, cu, SCALE)
        return out

    def absorb(self, q_nope):
        return torch.einsum("...hd,hdc->...hc", q_nope, self.w_uk).contiguous()

    def values(self, latent):
        return torch.einsum("...hc,hdc->...hd", latent, self.w_uv)


class Cache:
    """Pages of latents; sequence b's logical token s is in slot table[b, s // 64] * 64 + s % 64."""

    def __init__(self, pages, batch, max_pages):
        self.ckv = torch.zeros((pages, PAGE, DC), dtype=BF16, device="cuda")
        self.kpe = torch.zeros((pages, PAGE, DP), dtype=BF16, device="cuda")
        self.table = torch.full((batch, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.weights = torch.zeros((batch, max_pages * PAGE), device="cuda")
        self.free = list(range(pages))

    def append(self, b, ckv, kpe):
        start, n = int(self.lens[b]), ckv.shape[0]
        while int((self.table[b] >= 0).sum()) * PAGE < start + n:
            self.table[b, int((self.table[b] >= 0).sum())] = self.free.pop()
        at = torch.arange(start, start + n, device="cuda")
        slots = self.table[b].long()[at // PAGE] * PAGE + at % PAGE
        self.ckv.view(-1, DC)[slots], self.kpe.view(-1, DP)[slots] = ckv, kpe
        self.lens[b] += n


def main(prompts=(700, 1500, 90), steps=8, budget=512, recent=64, seed=0, say=print):
    layer = Layer(torch.Generator(device="cuda").manual_seed(seed))
    nb = len(prompts)
    cache = Cache(sum(-(-(n + steps) // PAGE) + 1 for n in prompts), nb, -(-(max(prompts) + steps) // PAGE) + 1)

    # the prompts, all at once, in the expanded form; their latents go to the cache
    cu = torch.tensor([sum(prompts[:i]) for i in range(nb + 1)], dtype=torch.int32, device="cuda")
    ckv, kpe, q_nope, q_pe = layer.token(sum(prompts))
    prompt_out = layer.prefill(ckv, kpe, q_nope, q_pe, cu)
    for b in range(nb):
        cache.append(b, ckv[cu[b]:cu[b + 1]], kpe[cu[b]:cu[b + 1]])

    # both forms say the same of the last prompt token
    last = (cu[1:] - 1).long()
    latent, _ = B.latent_attention_paged(layer.absorb(q_nope[last])[:, None], q_pe[last][:, None].contiguous(), cache.ckv,
                                         cache.kpe, cache.table, cache.lens, SCALE, weights=cache.weights)
    off = (layer.values(latent[:, 0]) - prompt_out[last]).float().norm() / prompt_out[last].float().norm()
    say(f"prefill {list(prompts)} tokens; absorbed against expanded form: relative difference {float(off):.1e}")

    # decode under a budget: what keys receive is added up, and a sequence past
    # its budget keeps its latest keys and those with the most
    for step in range(steps):
        ckv, kpe, q_nope, q_pe = layer.token(nb, 1)
        for b in range(nb):
            cache.append(b, ckv[b], kpe[b])
        latent, lse = B.latent_attention_paged(layer.absorb(q_nope), q_pe, cache.ckv, cache.kpe, cache.table, cache.lens,
                                               SCALE, weights=cache.weights)
        layer.values(latent)
        if step == steps // 2:
            before = cache.lens.tolist()
            kept, _ = B.latent_cache_evict(cache.ckv, cache.kpe, cache.weights, cache.table, cache.lens, budget, recent,
                                           new_lens=cache.lens)
            say(f"step {step}: lengths {before} cut to {cache.lens.tolist()}")
    status = B.latent_last_status()
    say(f"lengths after {steps} steps {cache.lens.tolist()}, device status {status}")

    # a batch that continues one prompt: its pages are read once for all
    shared, n = 1, int(cache.lens[1])
    pages = cache.table[shared, :-(-n // PAGE)].contiguous()
    own = Cache(4 * nb, nb, 4)
    own.ckv, own.kpe = torch.cat([cache.ckv, own.ckv]), torch.cat([cache.kpe, own.kpe])
    own.free = list(range(cache.ckv.shape[0], own.ckv.shape[0]))
    ckv, kpe, q_nope, q_pe = layer.token(nb, 3)
    for b in range(nb):
        own.append(b, ckv[b], kpe[b])
    q = layer.absorb(q_nope[:, -1:])
    latent, lse = B.latent_attention_shared_prefix(q, q_pe[:, -1:].contiguous(), own.ckv, own.kpe, pages, cache.lens[1:2],
                                                   own.table, own.lens, SCALE)
    say(f"shared prompt of {n} keys for {nb} sequences: out {list(layer.values(latent).shape)}, lse "
        f"{[round(float(x), 2) for x in lse[:, 0, 0]]}")
    return float(off), cache.lens.tolist(), status, latent, lse


if __name__ == "__main__":
    main()
