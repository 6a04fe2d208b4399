"""Workloads of the operators that make, place and verify tokens of a paged latent cache: encoding rows for the
indexer (norm, rotation, Hadamard transform, FP8) together with the rotation of the attention's rope parts,
appending tokens to the cache, attention of a tree of drafted tokens over it, and keeping the accepted path.

Sizes are those of the indexer's own workloads (64 index heads of 128 dims, 16 heads per tensor-parallel shard,
512 + 64 dims per latent key, 64-token pages, the paged decode batch of 64 sequences x 2 tokens, the causal chunk
of 4096 rows, histories of up to 131072 keys) and generic small, odd and ragged ones around them.
`run` computes a case in plain 32-bit torch operations, or with `own` set through the package's entry points."""
import math
import random

import torch

own = False

DC, DP = 512, 64  # compressed dims and rope dims of a latent key
DI, G = 128, 64   # dims and heads of the indexer
PAGE = 64
E4M3_MAX = 448.0
EPS = 1e-6
INF = float("inf")
LOG2E = 1.0 / math.log(2.0)
SM_SCALE = 1.0 / math.sqrt(192.0)
BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # the queries of the paged decode batch: 64 sequences, 2 tokens each, anywhere in histories of 128K
        {"name": "encode_queries_128", "op": "encode", "T": 128, "G": 64, "H": 16, "norm": False, "hadamard": True,
         "interleaved": False, "first": -1, "shape_seed": 1},
        # the queries of the causal chunk of 4096 rows that ends at 128K
        {"name": "encode_queries_4096", "op": "encode", "T": 4096, "G": 64, "H": 16, "norm": False, "hadamard": True,
         "interleaved": False, "first": 126976, "shape_seed": 2},
        # all keys of a 128K prompt, dense, for the indexer's prefill form
        {"name": "encode_keys_128k", "op": "encode", "T": 131072, "G": 1, "H": 1, "norm": True, "hadamard": True,
         "interleaved": False, "first": 0, "shape_seed": 3},
        # a decode step of 64 sequences: one token each, latents and index keys
        {"name": "append_b64_1", "op": "append", "B": 64, "nlo": 1, "nhi": 1, "lo": 1024, "hi": 16384, "index": True,
         "dense": False, "interleaved": True, "shape_seed": 4},
        # a prompt of 16K tokens into an empty cache
        {"name": "append_prompt_16k", "op": "append", "B": 1, "nlo": 16384, "nhi": 16384, "lo": 0, "hi": 0,
         "index": True, "dense": False, "interleaved": True, "shape_seed": 5},
        # a ragged batch of prompts behind what they share; the normed latents are wanted for the expanded form too
        {"name": "append_ragged_9", "op": "append", "B": 9, "nlo": 1, "nhi": 2500, "lo": 0, "hi": 777, "index": False,
         "dense": True, "interleaved": True, "shape_seed": 6},
        # one sequence, a small tree behind a short history: all latency
        {"name": "tree_b1_n8_2k", "op": "tree", "B": 1, "nn": 8, "ragged": False, "H": 16, "lo": 2000, "hi": 2000,
         "shape_seed": 7},
        # the decode batch with a tree of 8 nodes per sequence: at the border of bandwidth and arithmetic
        {"name": "tree_b64_n8_32k", "op": "tree", "B": 64, "nn": 8, "ragged": False, "H": 16, "lo": 1024, "hi": 32768,
         "shape_seed": 8},
        # few sequences with large trees of their own sizes
        {"name": "tree_b7_n64_8k", "op": "tree", "B": 7, "nn": 64, "ragged": True, "H": 16, "lo": 2999, "hi": 8192,
         "shape_seed": 9},
        # every head of the model on one GPU
        {"name": "tree_b4_n16_h128", "op": "tree", "B": 4, "nn": 16, "ragged": False, "H": 128, "lo": 5000,
         "hi": 16384, "shape_seed": 10},
        # one sequence keeps the accepted path of its tree
        {"name": "accept_b1_n16", "op": "accept", "B": 1, "nn": 16, "lo": 700, "hi": 700, "index": False,
         "shape_seed": 11},
        # a whole batch, large trees, the indexer's keys moved along
        {"name": "accept_b64_n64", "op": "accept", "B": 64, "nn": 64, "lo": 1024, "hi": 8192, "index": True,
         "shape_seed": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["encode", "append", "tree", "tree", "accept"])
    seed = rng.randrange(1 << 30)
    if op == "encode":
        keys = rng.random() < 0.4
        T = _log(rng, 1, 131072 if keys else 4096)
        return {"op": op, "T": T, "G": 1 if keys else 64, "H": 1 if keys else rng.choice([5, 8, 16, 16, 32, 128]),
                "norm": rng.random() < (0.8 if keys else 0.2), "hadamard": rng.random() < 0.6,
                "interleaved": rng.random() < 0.3, "first": rng.choice([-1, rng.randrange(0, 163840 - T)]),
                "shape_seed": seed}
    if op == "append":
        B, nhi = _log(rng, 1, 64), _log(rng, 1, 16384)
        while B * nhi > 16384:
            B = max(1, B // 2)
        hi = rng.choice([0, _log(rng, 1, 8192)])
        return {"op": op, "B": B, "nlo": rng.choice([0, 1, nhi]), "nhi": nhi, "lo": rng.randrange(0, hi + 1), "hi": hi,
                "index": rng.random() < 0.6, "dense": rng.random() < 0.3, "interleaved": rng.random() < 0.7,
                "shape_seed": seed}
    B, nn = _log(rng, 1, 64), _log(rng, 1, 64)
    if op == "accept":
        hi = _log(rng, nn, 8192)
        return {"op": op, "B": B, "nn": nn, "lo": max(nn, hi // 8), "hi": hi, "index": rng.random() < 0.5,
                "shape_seed": seed}
    H = rng.choice([5, 8, 16, 16, 24, 32, 64, 128])
    while B * nn * H > 8192:
        B, nn = (max(1, B // 2), nn) if B > 1 else (B, max(1, nn // 2))
    hi = max(nn, min(32768, _log(rng, 64, 32768), (1 << 27) // (B * nn * H)))
    return {"op": op, "B": B, "nn": nn, "ragged": rng.random() < 0.5, "H": H, "lo": max(nn, hi // rng.choice([1, 2, 16])),
            "hi": hi, "shape_seed": seed}


def _spread(case, lo, hi, salt):
    r = random.Random(case["shape_seed"] * 16 + salt)
    return [r.randint(lo, hi) for _ in range(case["B"])]


# ------------------------------------------------------------------ inputs --
def _pages(lens, seed):
    """Block table of a random permutation of the pages; unused entries -1."""
    r = random.Random(seed)
    n = [-(-x // PAGE) for x in lens]
    perm = list(range(sum(n)))
    r.shuffle(perm)
    table = torch.full((len(lens), max(1, max(n))), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(n):
        table[b, :c] = torch.tensor(perm[at:at + c], dtype=torch.int32)
        at += c
    return table.cuda(), max(1, at)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _rotations(n):
    """cos and sin of 32 angles at every position, from 64 bits: a model's table, kept by its program."""
    f = 10000.0 ** (-torch.arange(0, DP, 2, dtype=torch.float64, device="cuda") / DP)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def _trees(case, seed):
    """Parents of every sequence's drafted nodes (node 0: the last accepted token)."""
    r = random.Random(seed * 7919 + case["shape_seed"])
    n = [r.randint(1, case["nn"]) if case.get("ragged") else case["nn"] for _ in range(case["B"])]
    return [[-1] + [r.randrange(0, i) for i in range(1, k)] for k in n]


def _path(parents, node):
    p = []
    while node >= 0:
        p.append(node)
        node = parents[node]
    return p[::-1]


def _masks(parents, nn):
    """Bit j of word j // 64: node i sees node j (its ancestors and itself)."""
    words = -(-nn // 64)
    out = []
    for p in parents:
        seen = []
        for i, parent in enumerate(p):
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
        for s in seen + [0] * (nn - len(p)):
            w = [(s >> 64 * k) & (1 << 64) - 1 for k in range(words)]
            out.append([x - (1 << 64) if x >> 63 else x for x in w])
    return torch.tensor(out, dtype=torch.int64).view(len(parents), nn, words).cuda()


def _cache(s, case, total, g, index):
    """Pages for `total` keys per sequence, filled with what tokens leave there."""
    s["block_table"], pages = _pages(total, case["shape_seed"])
    s["ckv"] = torch.randn((pages, PAGE, DC), generator=g, device="cuda", dtype=BF16)
    s["kpe"] = torch.randn((pages, PAGE, DP), generator=g, device="cuda", dtype=BF16)
    if index:
        s["k_cache"] = torch.randn((pages, PAGE, DI), generator=g, device="cuda").mul_(120.0).clamp_(-448, 448).to(FP8)
        s["k_scale"] = torch.rand((pages, PAGE), generator=g, device="cuda") * 0.01 + 0.001


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + case["shape_seed"])

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=BF16)

    op = case["op"]
    s = {"op": op}
    if op == "encode":
        T = case["T"]
        s["x"] = normal(T, case["G"], DI)
        s["x"][:, :, 5] *= 8  # a few dims of activations are much larger than the others
        # the rope parts lie where a projection leaves them: behind a query's or a latent's other dims
        s["pe"] = normal(T, case["H"], 128 + DP)[..., 128:] if case["G"] > 1 else normal(T, 1, DC + DP)[..., DC:]
        s["cos_sin"] = _rotations(163840)
        at = torch.arange(T, device="cuda", dtype=torch.int32)
        s["positions"] = at + case["first"] if case["first"] >= 0 else torch.randint(
            0, 131072, (T,), generator=g, device="cuda", dtype=torch.int32)
        s["norm"] = (1 + 0.2 * torch.randn(DI, generator=g, device="cuda"),
                     0.1 * torch.randn(DI, generator=g, device="cuda"), EPS) if case["norm"] else None
        s.update(hadamard=case["hadamard"], interleaved=case["interleaved"])
        return s
    if op == "append":
        n, lens = _spread(case, case["nlo"], case["nhi"], 1), _spread(case, case["lo"], case["hi"], 2)
        n[0] = case["nhi"]
        _cache(s, case, [a + b for a, b in zip(n, lens)], g, case["index"])
        T = sum(n)
        joint = normal(T, DC + DP)  # one projection gives both
        s.update(c=joint[:, :DC], k_pe=joint[:, DC:], seq_lens=_ints(lens),
                 cu_new=_ints([sum(n[:i]) for i in range(len(n) + 1)]), cos_sin=_rotations(32768),
                 c_norm=(1 + 0.2 * torch.randn(DC, generator=g, device="cuda"), EPS),
                 dense=case["dense"], interleaved=case["interleaved"])
        if case["index"]:
            s["index_k"] = normal(T, DI)
            s["index_norm"] = (1 + 0.2 * torch.randn(DI, generator=g, device="cuda"),
                               0.1 * torch.randn(DI, generator=g, device="cuda"), EPS)
        return s
    lens = _spread(case, case["lo"], case["hi"], 1)
    parents = _trees(case, seed)
    _cache(s, case, lens, g, case.get("index", False))
    s.update(seq_lens=_ints(lens), draft_lens=_ints([len(p) for p in parents]))
    if op == "tree":
        rows = (case["B"], case["nn"], case["H"])
        s.update(q_nope=normal(*rows, DC), q_pe=normal(*rows, DP), tree_mask=_masks(parents, case["nn"]))
        return s
    paths = _accepted(case, seed, parents)
    s["path"] = _ints([p + [-1] * (case["nn"] - len(p)) for p in paths])
    s["path_lens"] = _ints([len(p) for p in paths])
    return s


def _accepted(case, seed, parents):
    r = random.Random(seed * 31 + case["shape_seed"])
    return [_path(p, r.randrange(len(p))) for p in parents]


# ------------------------------------------------------------- plain forms --
def _rotate(x, cs, interleaved):
    """x [..., 64] in 32 bits by the angles of its token: pairs (2i, 2i + 1), or (i, i + 32)."""
    cos, sin = cs[..., :DP // 2], cs[..., DP // 2:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    a, b = x[..., :DP // 2], x[..., DP // 2:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _hadamard_matrix():
    i = torch.arange(DI, device="cuda")
    both = i[:, None] & i[None, :]
    ones = sum((both >> k) & 1 for k in range(7))
    return (1.0 - 2.0 * (ones % 2)).float()


def _encode(x, cs, norm, hadamard, interleaved):
    """Codes and scales of rows x [T, G, 128] (bf16), cs [T, 64]."""
    x = x.float()
    if norm is not None:
        w, b, eps = norm
        d = x - x.mean(-1, keepdim=True)
        x = d / torch.sqrt(d.square().mean(-1, keepdim=True) + eps) * w + b
    x = torch.cat([_rotate(x[..., :DP], cs[:, None], interleaved), x[..., DP:]], -1)
    if hadamard:
        x = x @ (_hadamard_matrix() / math.sqrt(DI))
    amax = x.abs().amax((-2, -1))
    scale = torch.where(amax > 0, amax / E4M3_MAX, 1.0)
    return (x / scale[:, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(FP8), scale


def _plain_encode(s):
    cs = s["cos_sin"][s["positions"].long()]
    codes, scale = _encode(s["x"], cs, s["norm"], s["hadamard"], s["interleaved"])
    return {"codes": codes, "scale": scale, "pe": _rotate(s["pe"].float(), cs[:, None], True).to(BF16)}


def _plain_append(s):
    cu, lens = s["cu_new"].long(), s["seq_lens"].long()
    t = torch.arange(s["c"].shape[0], device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    at = lens[b] + t - cu[b]
    slots = s["block_table"].long()[b, at // PAGE] * PAGE + at % PAGE
    cs = s["cos_sin"][at]
    g, eps = s["c_norm"]
    c = s["c"].float()
    c = (c / torch.sqrt(c.square().mean(-1, keepdim=True) + eps) * g).to(BF16)
    pe = _rotate(s["k_pe"].float(), cs, s["interleaved"]).to(BF16)
    s["ckv"].view(-1, DC)[slots] = c
    s["kpe"].view(-1, DP)[slots] = pe
    new_lens = (lens + cu[1:] - cu[:-1]).to(torch.int32)
    if "index_k" in s:
        codes, scale = _encode(s["index_k"][:, None], cs, s["index_norm"], True, False)
        s["k_cache"].view(torch.uint8).view(-1, DI)[slots] = codes[:, 0].view(torch.uint8)
        s["k_scale"].view(-1)[slots] = scale
    return _appended(s, new_lens, c, pe)


def _appended(s, new_lens, c, pe):
    out = {"new_lens": new_lens, "ckv": s["ckv"], "kpe": s["kpe"]}
    if "index_k" in s:
        out["k_cache"], out["k_scale"] = s["k_cache"], s["k_scale"]
    if s["dense"]:
        out["c"], out["pe"] = c, pe
    return out


def _plain_tree(s):
    B, nn, H, _ = s["q_nope"].shape
    q = torch.cat([s["q_nope"], s["q_pe"]], -1).float().reshape(B, nn * H, DC + DP)
    at = torch.arange(s["block_table"].shape[1] * PAGE, device="cuda")
    slots = s["block_table"].clamp(min=0).long()[:, at // PAGE] * PAGE + at % PAGE
    keys = torch.cat([s["ckv"].view(-1, DC)[slots], s["kpe"].view(-1, DP)[slots]], -1).float()
    n = s["draft_lens"].long()
    d = at - (s["seq_lens"].long() - n)[:, None]  # place among the drafted nodes
    word = (d.clamp(min=0) // 64).clamp(max=s["tree_mask"].shape[2] - 1)
    bits = s["tree_mask"].gather(2, word[:, None].expand(B, nn, -1)) >> (d % 64)[:, None] & 1
    mask = (d < 0)[:, None] | ((d < n[:, None])[:, None] & (bits == 1))
    mask &= (torch.arange(nn, device="cuda") < n[:, None])[..., None]
    u = torch.where(mask.repeat_interleave(H, 1), (q @ keys.transpose(1, 2)) * (SM_SCALE * LOG2E), -INF)
    m = u.amax(-1, keepdim=True)
    e = torch.exp2(u - torch.where(m == -INF, 0.0, m))
    total = e.sum(-1, keepdim=True)
    out = (e / torch.where(total > 0, total, 1.0)) @ keys[..., :DC]
    lse = (m + torch.log2(total)).squeeze(-1)
    return {"out": out.to(BF16).view(B, nn, H, DC), "lse": lse.view(B, nn, H)}


def _plain_accept(s):
    before = (s["seq_lens"] - s["draft_lens"]).long()
    valid = torch.arange(s["path"].shape[1], device="cuda") < s["path_lens"][:, None]
    b, j = valid.nonzero(as_tuple=True)
    old, new = before[b] + s["path"].long()[b, j], before[b] + j
    table = s["block_table"].long()
    src, dst = table[b, old // PAGE] * PAGE + old % PAGE, table[b, new // PAGE] * PAGE + new % PAGE
    for name in ("ckv", "kpe", "k_cache", "k_scale"):
        if name in s:
            flat = s[name].view(torch.uint8) if name == "k_cache" else s[name]
            flat = flat.view(-1, *flat.shape[2:])
            flat[dst] = flat[src]
    return _kept(s, (before + s["path_lens"]).to(torch.int32))


def _kept(s, new_lens):
    return {"new_lens": new_lens, **{k: s[k] for k in ("ckv", "kpe", "k_cache", "k_scale") if k in s}}


def run(s):
    op = s["op"]
    if not own:
        return {"encode": _plain_encode, "append": _plain_append, "tree": _plain_tree, "accept": _plain_accept}[op](s)
    from fp8_scoring_exact_gb300 import binding
    if op == "encode":
        codes, scale, pe = binding.indexer_encode(s["x"], s["cos_sin"], s["positions"], norm=s["norm"],
                                                  interleaved=s["interleaved"], hadamard=s["hadamard"], pe=s["pe"])
        return {"codes": codes, "scale": scale, "pe": pe}
    if op == "append":
        dense = (torch.empty_like(s["c"], memory_format=torch.contiguous_format),
                 torch.empty_like(s["k_pe"], memory_format=torch.contiguous_format)) if s["dense"] else (None, None)
        new_lens = binding.latent_cache_append(s["c"], s["k_pe"], s["cos_sin"], s["cu_new"], s["block_table"],
                                               s["seq_lens"], s["ckv"], s["kpe"], c_norm=s["c_norm"],
                                               pe_interleaved=s["interleaved"], index_k=s.get("index_k"),
                                               index_norm=s.get("index_norm"), hadamard=True,
                                               k_cache=s.get("k_cache"), k_cache_scale=s.get("k_scale"),
                                               c_out=dense[0], k_pe_out=dense[1])
        return _appended(s, new_lens, *dense)
    if op == "tree":
        out, lse = binding.latent_attention_tree(s["q_nope"], s["q_pe"], s["ckv"], s["kpe"], s["block_table"],
                                                 s["seq_lens"], s["tree_mask"], SM_SCALE, draft_lens=s["draft_lens"])
        return {"out": out, "lse": lse}
    return _kept(s, binding.latent_cache_accept(s["ckv"], s["kpe"], s["block_table"], s["seq_lens"], s["draft_lens"],
                                                s["path"], s["path_lens"], k_cache=s.get("k_cache"),
                                                k_cache_scale=s.get("k_scale")))


# ------------------------------------------------------------ work and truth --
def work(case):
    op = case["op"]
    if op == "encode":
        return {"bytes": case["T"] * (case["G"] * DI * 3 + 4 + 4 + case["H"] * 4 * DP + 4 * DP), "flops": 0}
    if op == "append":
        n = _spread(case, case["nlo"], case["nhi"], 1)
        n[0] = case["nhi"]
        token = 4 * (DC + DP) + 4 * DP + (DI * 3 + 4 if case["index"] else 0) + (2 * (DC + DP) if case["dense"] else 0)
        return {"bytes": sum(n) * token + 12 * case["B"], "flops": 0}
    lens = _spread(case, case["lo"], case["hi"], 1)
    if op == "accept":
        kept = sum(len(p) for p in _accepted(case, 0, _trees(case, 0)))
        return {"bytes": kept * (2 * (2 * (DC + DP) + (132 if case["index"] else 0)) + 4) + 16 * case["B"], "flops": 0}
    rows, pairs, keys = case["B"] * case["nn"] * case["H"], 0, 0
    for length, p in zip(lens, _trees(case, 0)):
        pairs += case["H"] * sum(length - len(p) + len(_path(p, i)) for i in range(len(p)))
        keys += length
    return {"bytes": 2 * keys * (DC + DP) + rows * (2 * (DC + DP) + 2 * DC + 4), "flops": 2 * (2 * DC + DP) * pairs}


def _exact_rotate(x, cs, interleaved):
    """Each pair as a complex number, times cos + i sin."""
    pair = x.view(*x.shape[:-1], 32, 2) if interleaved else torch.stack([x[..., :32], x[..., 32:]], -1)
    turned = torch.view_as_complex(pair.contiguous()) * torch.complex(cs[..., :32], cs[..., 32:])
    pair = torch.view_as_real(turned)
    return pair.reshape(x.shape) if interleaved else torch.cat([pair[..., 0], pair[..., 1]], -1)


def _exact_encode(x, cs, norm, hadamard, interleaved):
    x = x.double()
    if norm is not None:
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        x = (x - mean) * (var + norm[2]) ** -0.5 * norm[0].double() + norm[1].double()
    x = torch.cat([_exact_rotate(x[..., :DP].contiguous(), cs[:, None].expand(-1, x.shape[1], -1), interleaved),
                   x[..., DP:]], -1)
    if hadamard:
        h = torch.ones((1, 1), dtype=torch.float64, device="cuda")
        for _ in range(7):
            h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
        x = torch.einsum("tgi,ij->tgj", x, h) / 128.0 ** 0.5
    top = x.abs().flatten(1).max(1).values
    scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    return x / scale[:, None, None], scale  # the values that the codes round


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "encode":
        cs = s["cos_sin"].index_select(0, s["positions"].long()).double()
        codes, scale = _exact_encode(s["x"], cs, s["norm"], case["hadamard"], case["interleaved"])
        pe = _exact_rotate(s["pe"].double().contiguous(), cs[:, None].expand(-1, s["pe"].shape[1], -1), True)
        return {"codes": codes, "scale": scale, "pe": pe}
    table = s["block_table"].tolist()
    lens = s["seq_lens"].tolist()

    def slots(b, first, n):
        return torch.tensor([table[b][i // PAGE] * PAGE + i % PAGE for i in range(first, first + n)], device="cuda",
                            dtype=torch.long)

    if op == "append":
        cu = s["cu_new"].tolist()
        out = {k: s[k].double() for k in ("ckv", "kpe", "k_cache", "k_scale") if k in s}
        dense_c, dense_pe = s["c"].double().contiguous(), s["k_pe"].double().contiguous()
        for b, first in enumerate(lens):
            lo, hi = cu[b], cu[b + 1]
            if lo == hi:
                continue
            at = slots(b, first, hi - lo)
            cs = s["cos_sin"][first:first + hi - lo].double()
            c = s["c"][lo:hi].double()
            dense_c[lo:hi] = c * ((c * c).sum(1, keepdim=True) / DC + s["c_norm"][1]) ** -0.5 * s["c_norm"][0].double()
            dense_pe[lo:hi] = _exact_rotate(s["k_pe"][lo:hi].double().contiguous(), cs, case["interleaved"])
            out["ckv"].view(-1, DC)[at], out["kpe"].view(-1, DP)[at] = dense_c[lo:hi], dense_pe[lo:hi]
            if case["index"]:
                codes, scale = _exact_encode(s["index_k"][lo:hi, None], cs, s["index_norm"], True, False)
                out["k_cache"].view(-1, DI)[at], out["k_scale"].view(-1)[at] = codes[:, 0], scale
        out["new_lens"] = torch.tensor([x + cu[b + 1] - cu[b] for b, x in enumerate(lens)])
        if case["dense"]:
            out["c"], out["pe"] = dense_c, dense_pe
        return out
    parents = _trees(case, seed)
    if op == "accept":
        out = {k: s[k].double() for k in ("ckv", "kpe", "k_cache", "k_scale") if k in s}
        new_lens = []
        for b, p in enumerate(_accepted(case, seed, parents)):
            before = lens[b] - len(parents[b])
            node = slots(b, before, len(parents[b]))
            for j, i in enumerate(p):
                for k, v in out.items():
                    v.view(-1, *v.shape[2:])[node[j]] = s[k].view(-1, *s[k].shape[2:])[node[i]].double()
            new_lens.append(before + len(p))
        return {**out, "new_lens": torch.tensor(new_lens)}
    B, nn, H = case["B"], case["nn"], case["H"]
    out = torch.zeros((B, nn, H, DC), dtype=torch.float64, device="cuda")
    lse = torch.full((B, nn, H), -INF, dtype=torch.float64, device="cuda")
    for b, length in enumerate(lens):
        n = len(parents[b])
        at = slots(b, 0, length)
        v = s["ckv"].view(-1, DC)[at].double()
        k = torch.cat([v, s["kpe"].view(-1, DP)[at].double()], 1)
        hidden = torch.ones((n, length), dtype=torch.bool)
        hidden[:, :length - n] = False
        for i in range(n):
            hidden[i, [length - n + j for j in _path(parents[b], i)]] = False
        q = torch.cat([s["q_nope"][b, :n].double(), s["q_pe"][b, :n].double()], -1).view(n * H, DC + DP)
        u = (q @ k.T) * (SM_SCALE / math.log(2.0))
        u.view(n, H, length).masked_fill_(hidden.cuda()[:, None], -INF)
        top = torch.logsumexp(u * math.log(2.0), 1) / math.log(2.0)
        out[b, :n] = (torch.exp2(u - top[:, None]) @ v).view(n, H, DC)
        lse[b, :n] = top.view(n, H)
    return {"out": out, "lse": lse}
