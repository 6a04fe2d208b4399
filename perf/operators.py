"""Workloads of the latent-attention operators: decode over a paged latent
cache (with and without the accumulated attention weight of every key), decode
of a batch that shares a long prefix, eviction from the cache by accumulated
weight, and prefill in the expanded form.

Sizes are those of the indexer's own workloads (16 heads per tensor-parallel
shard, 512 + 64 dims per latent key, 64-token pages, the paged decode batch of
64 sequences x 2 tokens with lengths up to 131072, the causal chunk of 2048
rows over 16384 keys) and generic small, odd and ragged ones around them.
`run` computes a case in plain 32-bit torch operations, or with `own` set
through the package's entry points."""
import math
import random

import torch

own = False

DC, DP = 512, 64   # compressed dims and rope dims of a latent key
DN, DV = 128, 128  # expanded no-rope key dims and value dims of a head
PAGE = 64
INF = float("inf")
LOG2E = 1.0 / math.log(2.0)
SM_SCALE = 1.0 / math.sqrt(DN + DP)


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one sequence with a short history: a first tokens' step, all latency
        {"name": "decode_b1_len200", "op": "decode", "B": 1, "nn": 1, "H": 16, "lo": 200, "hi": 200, "lens_seed": 1,
         "weights": False},
        # the paged decode batch of the indexer: 64 sequences, 2 tokens each, 1K to 128K keys
        {"name": "decode_b64_nn2_128k", "op": "decode", "B": 64, "nn": 2, "H": 16, "lo": 1024, "hi": 131072,
         "lens_seed": 4, "weights": False},
        # every head of the model on one GPU, a few long sequences
        {"name": "decode_b7_h128_32k", "op": "decode", "B": 7, "nn": 1, "H": 128, "lo": 9001, "hi": 32768,
         "lens_seed": 5, "weights": False},
        # decode under a cache budget: the keys' weights are accumulated as well
        {"name": "decode_weights_b32_16k", "op": "decode", "B": 32, "nn": 1, "H": 16, "lo": 500, "hi": 16384,
         "lens_seed": 6, "weights": True},
        # a few requests behind one system prompt
        {"name": "prefix_b12_2k", "op": "prefix", "B": 12, "nn": 1, "H": 16, "prefix": 2000, "lo": 1, "hi": 300,
         "lens_seed": 7},
        # a large batch over one long document, two tokens each
        {"name": "prefix_b64_nn2_32k", "op": "prefix", "B": 64, "nn": 2, "H": 16, "prefix": 32768, "lo": 1, "hi": 2048,
         "lens_seed": 8},
        # one sequence a little over its budget
        {"name": "evict_b1_3k", "op": "evict", "B": 1, "lo": 3000, "hi": 3000, "lens_seed": 9, "budget": 2048,
         "recent": 256, "indexer": False},
        # a whole batch cut to its budget, the indexer's keys moved along
        {"name": "evict_b64_32k", "op": "evict", "B": 64, "lo": 3500, "hi": 32768, "lens_seed": 10, "budget": 4096,
         "recent": 512, "indexer": True},
        # long histories, a large budget
        {"name": "evict_b5_128k", "op": "evict", "B": 5, "lo": 60001, "hi": 131072, "lens_seed": 11, "budget": 16384,
         "recent": 1000, "indexer": False},
        # one short prompt
        {"name": "prefill_100", "op": "prefill", "S": 1, "H": 16, "qlo": 100, "qhi": 100, "past": 0, "lens_seed": 12},
        # the causal chunk of 2048 rows over 16384 keys
        {"name": "prefill_q2048_n16k", "op": "prefill", "S": 1, "H": 16, "qlo": 2048, "qhi": 2048, "past": 14336,
         "lens_seed": 13},
        # a ragged batch of prompts without a history
        {"name": "prefill_ragged_9", "op": "prefill", "S": 9, "H": 16, "qlo": 1, "qhi": 2500, "past": 0,
         "lens_seed": 14},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefix", "evict", "prefill"])
    seed = rng.randrange(1 << 30)
    if op == "decode":
        weights = rng.random() < 0.4
        B, nn, H = _log(rng, 1, 64), rng.choice([1, 1, 2, 3, 4]), rng.choice([5, 8, 16, 16, 24, 32, 64, 128])
        if B * nn * H > 4096:
            nn = 1
            H = min(H, 4096 // B)
        hi = max(1, min(131072, _log(rng, 64, 131072), (1 << 20 if weights else 3 << 20) * 16 // (B * max(16, nn * H))))
        return {"op": op, "B": B, "nn": nn, "H": H, "lo": max(1, hi // rng.choice([1, 2, 16])), "hi": hi,
                "lens_seed": seed, "weights": weights}
    if op == "prefix":
        B, nn, H = _log(rng, 2, 64), rng.choice([1, 1, 2]), rng.choice([8, 16, 16, 20, 32])
        while B * nn * H > 2048:
            B = max(1, B // 2)
        hi = _log(rng, 1, 2048)
        return {"op": op, "B": B, "nn": nn, "H": H, "prefix": _log(rng, 500, 32768), "lo": max(1, hi // 8), "hi": hi,
                "lens_seed": seed}
    if op == "evict":
        B, hi = _log(rng, 1, 64), _log(rng, 1000, 32768)
        budget = max(64, int(hi * rng.uniform(0.1, 0.8)))
        return {"op": op, "B": B, "lo": max(1, hi // 4), "hi": hi, "lens_seed": seed, "budget": budget,
                "recent": rng.randrange(0, budget // 2), "indexer": rng.random() < 0.5}
    S, qhi = _log(rng, 1, 12), _log(rng, 1, 2048)
    past = rng.choice([0, 0, _log(rng, 1, 8192)])
    while S * qhi > 8192:
        S = max(1, S // 2)
    if S * S * qhi * (qhi + past) > 2048 * 16384:
        past = 0
    return {"op": op, "S": S, "H": rng.choice([4, 16, 16, 31]), "qlo": max(1, qhi // 8), "qhi": qhi, "past": past,
            "lens_seed": seed}


def _lens(case, n, lo, hi):
    r = random.Random(case["lens_seed"])
    return [r.randint(lo, hi) for _ in range(n)]


# ------------------------------------------------------------------ inputs --
def _pages(lens, seed):
    """Block table of a random permutation of the pages; unused entries -1."""
    r = random.Random(seed)
    n = [-(-x // PAGE) for x in lens]
    perm = list(range(sum(n)))
    r.shuffle(perm)
    table = torch.full((len(lens), max(n)), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(n):
        table[b, :c] = torch.tensor(perm[at:at + c], dtype=torch.int32)
        at += c
    return table.cuda(), at


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + case["lens_seed"])

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    op = case["op"]
    s = {"op": op}
    if op == "prefill":
        q = _lens(case, case["S"], case["qlo"], case["qhi"])
        k = [x + case["past"] for x in q]
        kv = normal(sum(k), case["H"], DN + DV)  # as one projection of the latent leaves them
        s.update(q=normal(sum(q), case["H"], DN + DP), k_nope=kv[..., :DN], v=kv[..., DN:], k_pe=normal(sum(k), DP),
                 cu_q=_ints([sum(q[:i]) for i in range(len(q) + 1)]),
                 cu_k=_ints([sum(k[:i]) for i in range(len(k) + 1)]))
        return s
    lens = _lens(case, case["B"], case["lo"], case["hi"])
    own_pages = sum(-(-x // PAGE) for x in lens)
    if op == "prefix":
        n = -(-case["prefix"] // PAGE)
        table, _ = _pages(lens, seed)
        order = torch.randperm(own_pages + n, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
        s["block_table"] = torch.where(table >= 0, order[table.clamp(min=0).long()], -1).to(torch.int32)
        s["prefix_table"], s["prefix_len"] = order[own_pages:].contiguous(), _ints([case["prefix"]])
        own_pages += n
    else:
        s["block_table"], _ = _pages(lens, seed)
    s.update(seq_lens=_ints(lens), ckv=normal(own_pages, PAGE, DC), kpe=normal(own_pages, PAGE, DP))
    width = s["block_table"].shape[1] * PAGE
    if op == "evict":
        # what accumulates in use: a few keys with much weight, a long tail, and new keys without any
        w = torch.exp(2.0 * torch.randn((case["B"], width), generator=g, device="cuda"))
        s["weights"] = w * (torch.rand(w.shape, generator=g, device="cuda") > 0.02)
        s.update(budget=case["budget"], recent=case["recent"])
        if case["indexer"]:
            s["k_cache"] = normal(own_pages, PAGE, 128).to(torch.float8_e4m3fn).view(torch.uint8)
            s["k_scale"] = torch.rand((own_pages, PAGE), generator=g, device="cuda") + 0.5
        return s
    s.update(q_nope=normal(case["B"], case["nn"], case["H"], DC), q_pe=normal(case["B"], case["nn"], case["H"], DP))
    if case.get("weights"):
        s["weights"] = torch.zeros((case["B"], width), device="cuda")
    return s


# ------------------------------------------------------------- plain forms --
def _gather(s, table, length):
    """Latent keys [B, length, 576] in 32 bits behind a block table."""
    at = torch.arange(length, device="cuda")
    slots = table.clamp(min=0).long()[..., at // PAGE] * PAGE + at % PAGE
    return torch.cat([s["ckv"].view(-1, DC)[slots], s["kpe"].view(-1, DP)[slots]], -1).float()


def _attend(scores, mask, values):
    """(out, lse, probabilities) over the last axis of `scores`, in base 2."""
    u = torch.where(mask, scores * (SM_SCALE * LOG2E), -INF)
    m = u.amax(-1, keepdim=True)
    e = torch.exp2(u - torch.where(m == -INF, 0.0, m))
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    lse = (m + torch.log2(total)).squeeze(-1)
    return (p @ values).to(torch.bfloat16), lse, p


def _plain_decode(s):
    B, nn, H, _ = s["q_nope"].shape
    q = torch.cat([s["q_nope"], s["q_pe"]], -1).float().reshape(B, nn * H, DC + DP)
    lens = s["seq_lens"].long()
    limit = lens[:, None] - nn + 1 + torch.arange(nn, device="cuda")  # [B, nn]
    keys = _gather(s, s["block_table"], s["block_table"].shape[1] * PAGE)
    at = torch.arange(keys.shape[1], device="cuda")
    mask = at < limit.repeat_interleave(H, 1)[..., None]
    if s["op"] == "prefix":
        n = s["prefix_table"].shape[0] * PAGE
        first = _gather(s, s["prefix_table"], n)
        keys = torch.cat([first.expand(B, n, DC + DP), keys], 1)
        seen = (torch.arange(n, device="cuda") < s["prefix_len"]).expand(B, nn * H, n)
        mask = torch.cat([seen, mask], -1)
    out, lse, p = _attend(q @ keys.transpose(1, 2), mask, keys[..., :DC])
    out = {"out": out.view(B, nn, H, DC), "lse": lse.view(B, nn, H)}
    if "weights" in s:
        s["weights"] += p.sum(1)
        out["weights"] = s["weights"]
    return out


def _plain_evict(s):
    w, lens, budget, recent = s["weights"], s["seq_lens"].long(), s["budget"], s["recent"]
    B, width = w.shape
    at = torch.arange(width, device="cuda").expand(B, width)
    new = lens.clamp(max=budget)
    key = torch.where(at >= (lens - recent)[:, None], INF, w)
    key = torch.where(at >= lens[:, None], -INF, key)
    first = torch.argsort(key, dim=1, descending=True, stable=True)[:, :min(budget, width)]
    place = torch.arange(first.shape[1], device="cuda")
    kept = torch.where(place < new[:, None], first, width).sort(1).values
    valid = kept < width
    src = kept.clamp(max=width - 1)
    page = s["block_table"].long()
    old = (page.gather(1, src // PAGE) * PAGE + src % PAGE)[valid]
    dst = (page[:, place // PAGE] * PAGE + place % PAGE)[valid]
    for name in ("ckv", "kpe", "k_cache", "k_scale"):
        if name in s:
            flat = s[name].view(-1, *s[name].shape[2:])
            flat[dst] = flat[old]
    head = torch.where(valid, w.gather(1, src), 0.0)
    w[:, :first.shape[1]] = torch.where((at[:, :first.shape[1]] < lens[:, None]), head, w[:, :first.shape[1]])
    w.masked_fill_((at >= new[:, None]) & (at < lens[:, None]), 0.0)
    full = torch.full((B, budget), -1, dtype=torch.int32, device="cuda")
    full[:, :first.shape[1]] = torch.where(valid, kept, -1).to(torch.int32)
    return _evicted(s, full, new.to(torch.int32))


def _evicted(s, kept, new_lens):
    out = {"kept": kept, "new_lens": new_lens, "weights": s["weights"], "ckv": s["ckv"], "kpe": s["kpe"]}
    if "k_cache" in s:
        out["k_cache"], out["k_scale"] = s["k_cache"], s["k_scale"]
    return out


def _plain_prefill(s):
    Tq, H, _ = s["q"].shape
    Tk = s["v"].shape[0]
    k = torch.cat([s["k_nope"], s["k_pe"][:, None].expand(Tk, H, DP)], -1).float().transpose(0, 1)
    i, j = torch.arange(Tq, device="cuda"), torch.arange(Tk, device="cuda")
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    of_q, of_k = torch.searchsorted(cu_q, i, right=True) - 1, torch.searchsorted(cu_k, j, right=True) - 1
    # query i of a sequence sees that sequence's keys up to its own place, the last query all of them
    last = cu_k[of_q + 1] - (cu_q[of_q + 1] - 1 - i)
    mask = (of_q[:, None] == of_k) & (j < last[:, None])
    out, lse, _ = _attend(s["q"].float().transpose(0, 1) @ k.transpose(1, 2), mask, s["v"].float().transpose(0, 1))
    return {"out": out.transpose(0, 1).contiguous(), "lse": lse.transpose(0, 1).contiguous()}


def run(s):
    op = s["op"]
    if not own:
        return {"decode": _plain_decode, "prefix": _plain_decode, "evict": _plain_evict,
                "prefill": _plain_prefill}[op](s)
    from fp8_scoring_exact_gb300 import binding
    if op == "decode":
        out, lse = binding.latent_attention_paged(s["q_nope"], s["q_pe"], s["ckv"], s["kpe"], s["block_table"],
                                                  s["seq_lens"], SM_SCALE, weights=s.get("weights"))
        return {"out": out, "lse": lse, **({"weights": s["weights"]} if "weights" in s else {})}
    if op == "prefix":
        out, lse = binding.latent_attention_shared_prefix(s["q_nope"], s["q_pe"], s["ckv"], s["kpe"],
                                                          s["prefix_table"], s["prefix_len"], s["block_table"],
                                                          s["seq_lens"], SM_SCALE)
        return {"out": out, "lse": lse}
    if op == "evict":
        kept, new_lens = binding.latent_cache_evict(s["ckv"], s["kpe"], s["weights"], s["block_table"], s["seq_lens"],
                                                    s["budget"], s["recent"], k_cache=s.get("k_cache"),
                                                    k_cache_scale=s.get("k_scale"))
        return _evicted(s, kept, new_lens)
    out, lse = binding.latent_attention_prefill(s["q"], s["k_nope"], s["k_pe"], s["v"], s["cu_q"], s["cu_k"], SM_SCALE)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------ work and truth --
def work(case):
    op = case["op"]
    if op == "prefill":
        q = _lens(case, case["S"], case["qlo"], case["qhi"])
        k = [x + case["past"] for x in q]
        pairs = case["H"] * sum(x * y - x * (x - 1) // 2 for x, y in zip(q, k))
        per_q = case["H"] * (2 * (DN + DP + DV) + 4)
        return {"bytes": sum(q) * per_q + sum(k) * (case["H"] * 2 * (DN + DV) + 2 * DP),
                "flops": 2 * (DN + DP + DV) * pairs}
    lens = _lens(case, case["B"], case["lo"], case["hi"])
    row = 2 * (DC + DP)
    if op == "evict":
        cut = sum(x > case["budget"] for x in lens)
        kept = sum(min(x, case["budget"]) for x in lens)
        moved = cut * case["budget"] * 2 * (row + (132 if case["indexer"] else 0))
        return {"bytes": moved + 4 * (sum(x for x in lens if x > case["budget"]) * 2 + kept), "flops": 0}
    nn, H = case["nn"], case["H"]
    rows = case["B"] * nn * H
    pairs = H * sum(max(0, x - i) for x in lens for i in range(nn)) + rows * case.get("prefix", 0)
    keys = sum(lens) + case.get("prefix", 0)
    return {"bytes": keys * (row + (8 if case.get("weights") else 0)) + rows * (row + 2 * DC + 4),
            "flops": 2 * (2 * DC + DP) * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    scale = SM_SCALE / math.log(2.0)

    def one(q, k, v, visible):
        """Softmax in base 2 of q k^T over the first visible[r] keys of each row r."""
        u = (q @ k.T) * scale
        u[torch.arange(k.shape[0], device="cuda")[None] >= visible[:, None]] = -INF
        lse = torch.logsumexp(u * math.log(2.0), 1) / math.log(2.0)
        p = torch.exp2(u - lse[:, None]).nan_to_num(0.0)
        return p @ v, lse, p

    if case["op"] == "prefill":
        q = s["q"].double()
        out = torch.empty(q.shape[:2] + (DV,), dtype=torch.float64, device="cuda")
        lse = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
        cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
        for a, b, c, d in zip(cq, cq[1:], ck, ck[1:]):
            pe = s["k_pe"][c:d].double()
            for h in range(q.shape[1]):
                k = torch.cat([s["k_nope"][c:d, h].double(), pe], 1)
                sees = (d - c) - (b - a) + 1 + torch.arange(b - a, device="cuda")
                out[a:b, h], lse[a:b, h], _ = one(q[a:b, h], k, s["v"][c:d, h].double(), sees)
        return {"out": out, "lse": lse}
    table, lens = s["block_table"].tolist(), s["seq_lens"].tolist()
    if case["op"] == "evict":
        w = s["weights"].double()
        kept = torch.full((case["B"], case["budget"]), -1, dtype=torch.int64)
        new = torch.tensor([min(x, case["budget"]) for x in lens])
        caches = {n: s[n].clone() for n in ("ckv", "kpe", "k_cache", "k_scale") if n in s}
        for b, length in enumerate(lens):
            n = min(length, case["budget"])
            if n < length:
                old = w[b, :length - case["recent"]].cpu().numpy()
                best = sorted(range(len(old)), key=lambda i: (-old[i], i))[:n - case["recent"]]
                rows = sorted(best) + list(range(length - case["recent"], length))
            else:
                rows = list(range(length))
            kept[b, :n] = torch.tensor(rows)
            slot = [table[b][i // PAGE] * PAGE + i % PAGE for i in range(length)]
            for name, c in caches.items():
                c.view(-1, *c.shape[2:])[slot[:n]] = s[name].view(-1, *c.shape[2:])[[slot[i] for i in rows]]
            moved = w[b, rows].clone()
            w[b, :length] = 0.0
            w[b, :n] = moved
        return {"kept": kept, "new_lens": new, "weights": w, "ckv": caches["ckv"].double(),
                "kpe": caches["kpe"].double(), **({"k_cache": caches["k_cache"], "k_scale": caches["k_scale"].double()}
                                                  if "k_cache" in caches else {})}
    B, nn, H = case["B"], case["nn"], case["H"]
    flat, flat_pe = s["ckv"].view(-1, DC), s["kpe"].view(-1, DP)
    out = torch.empty((B, nn, H, DC), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, nn, H), dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if "weights" in s else None
    for b, length in enumerate(lens):
        at = [p * PAGE + i for p in table[b] if p >= 0 for i in range(PAGE)][:length]
        before = 0
        if case["op"] == "prefix":
            before = case["prefix"]
            at = [p * PAGE + i for p in s["prefix_table"].tolist() for i in range(PAGE)][:before] + at
        at = torch.tensor(at, device="cuda")
        v = flat[at].double()
        k = torch.cat([v, flat_pe[at].double()], 1)
        q = torch.cat([s["q_nope"][b].double(), s["q_pe"][b].double()], -1).view(nn * H, DC + DP)
        sees = (before + length - nn + 1 + torch.arange(nn, device="cuda")).repeat_interleave(H)
        o, l, p = one(q, k, v, sees)
        out[b], lse[b] = o.view(nn, H, DC), l.view(nn, H)
        if weights is not None:
            weights[b, :length] += p.sum(0)
    return {"out": out, "lse": lse, **({"weights": weights} if weights is not None else {})}
