"""What the operators that encode, append, verify and keep tokens promise at the ends of their arguments: borders that do
not ascend, norms of very large and very small rows, threads, releases, and more work than a grid has threads."""
import numpy as np
import pytest
import torch

from oracle import latent_attention as la
from oracle import token_encode as te
from test_gpu_token_ops import (B, BF, BF16, MAXPOS, Cache, Pages, _check_tree, _ints, _mask, _normal, _np,  # noqa: F401
                                _np_norm, _queries, _random_tree, _seen_of, _table, _tokens, _tree, check_codes)

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------- borders --
def _append_with_borders(B, cu, T, lens):  # noqa: F811
    """Appends T plain tokens (no norm, positions 0, where a rotation changes nothing) and holds every slot and length
    against one rule: a sequence whose length moved has all of its tokens, nothing else is written."""
    n, table = len(cu) - 1, torch.cat([torch.ones(4, 32), torch.zeros(4, 32)], 1)
    p = Pages([x + T for x in lens], seed=3)
    g = torch.Generator().manual_seed(T)
    c, k_pe = _tokens(g, T, joint=False)
    new = B.latent_cache_append(c.cuda(), k_pe.cuda(), table.cuda(), _ints(cu), p.table.cuda(), _ints(lens), p.ckv, p.kpe,
                                positions=torch.zeros(T, dtype=torch.int32, device="cuda")).tolist()
    status = B.latent_last_status()
    want, want_pe = torch.full((p.P * 64, 512), 3.0, dtype=BF16), torch.full((p.P * 64, 64), 3.0, dtype=BF16)
    for b in range(n):
        if new[b] != lens[b]:
            lo, hi = int(cu[b]), int(cu[b + 1])
            assert 0 <= lo < hi <= T and new[b] == lens[b] + hi - lo, (cu, new)
            at = torch.from_numpy(p.slots(b, lens[b], hi - lo))
            want[at], want_pe[at] = c[lo:hi], k_pe[lo:hi]
    assert torch.equal(p.ckv.cpu().reshape(-1, 512), want), (cu, new)
    assert torch.equal(p.kpe.cpu().reshape(-1, 64), want_pe), (cu, new)
    return new, status


@pytest.mark.parametrize("cu", [[0, 5, 3, 8], [0, 6, 2, 8, 8], [0, 8, 0, 8], [8, 0, 8], [0, 3, 3, 1, 8], [4, 2, 6, 8, 8],
                                [0, 2, 9, 4, 8], [0, 2, -1, 4, 8], [0, 7, 6, 5, 4, 3, 2, 1, 8],
                                [0, 2 ** 31 - 1, 4, 8], [0, -2 ** 31, 4, 8]])
def test_append_with_borders_that_do_not_ascend(B, cu):  # noqa: F811
    lens = [5 * i + 60 for i in range(len(cu) - 1)]
    _, status = _append_with_borders(B, cu, 8, lens)
    assert status == B.DSA_ERR_RANGE


def test_append_with_any_borders(B):  # noqa: F811
    rng = np.random.default_rng(5)
    moved = 0
    for _ in range(300):
        n = int(rng.integers(1, 12))
        cu = rng.integers(0, 24, n + 1) if rng.random() < 0.5 else np.sort(rng.integers(0, 24, n + 1))
        for _ in range(int(rng.integers(0, 3))):  # and a few that are out of place
            cu[int(rng.integers(0, n + 1))] = int(rng.integers(-3, 27))
        lens = rng.integers(0, 70, n).tolist()
        new, status = _append_with_borders(B, cu.tolist(), 24, lens)
        fits = bool(np.all(np.diff(cu) >= 0) and cu[0] >= 0 and cu[-1] <= 24)
        assert (status == 0) == fits
        if fits:
            assert new == (np.asarray(lens) + np.diff(cu)).tolist()
        else:
            moved += sum(a != b for a, b in zip(new, lens))
    assert moved > 100  # (sequences are written beside borders that do not ascend, so the rule above is tried)


# ----------------------------------------------------------- calls and ends --
def test_replays_beside_each_other_leave_nothing_behind(B):  # noqa: F811
    """Graphs captured on one stream share its status, and have to be replayed in turn.  Two that are not, of grids of
    different sizes, spoil no call behind them: its lengths, rows and status are its own."""
    g, table, s = torch.Generator().manual_seed(9), _table().cuda(), torch.cuda.Stream()
    new, lens = [40 * i % 97 for i in range(64)], [i % 70 for i in range(64)]
    cu, after = np.concatenate([[0], np.cumsum(new)]), [a + b for a, b in zip(new, lens)]
    T = sum(new)
    p = Pages(after, seed=10)
    c, k_pe = (x.cuda() for x in _tokens(g, T, joint=False))
    dcu, bt, before, dl = _ints(cu), p.table.cuda(), _ints(lens), _ints(lens)
    x, pos = _normal(g, 3, 64, 128).cuda(), _ints([1, 2, 3])
    codes, scale = torch.empty((3, 64, 128), dtype=torch.uint8, device="cuda"), torch.empty(3, device="cuda")

    def append():
        dl.copy_(before)
        B.latent_cache_append(c, k_pe, table, dcu, bt, dl, p.ckv, p.kpe, new_lens=dl)

    def encode():
        B.indexer_encode(x, table, pos, codes=codes, scale=scale)

    graphs = []
    torch.cuda.synchronize()
    for call in (append, encode):
        with torch.cuda.stream(s):
            call()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            call()
    want = codes.clone()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    slots = [torch.from_numpy(p.slots(b, lens[b], new[b])).cuda() for b in range(64)]
    for _ in range(60):
        for _ in range(8):
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        p.ckv.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):  # in turn, on the stream that they shared
            append()
            ok, got = B.latent_last_status(), dl.tolist()
            B.indexer_encode(x, table, _ints([1, MAXPOS, 3]), codes=codes, scale=scale)
            bad = B.latent_last_status()
            encode()
            again = B.latent_last_status()
        assert got == after and (ok, bad, again) == (0, B.DSA_ERR_RANGE, 0) and torch.equal(codes, want)
        for b in range(64):
            assert torch.equal(p.ckv.view(-1, 512)[slots[b]], c[int(cu[b]):int(cu[b + 1])])


def test_calls_beside_releases(B):  # noqa: F811
    """dsa_indexer_release on one thread while others call: a call's status is not freed before its kernels are done."""
    from concurrent.futures import ThreadPoolExecutor
    g, table = torch.Generator().manual_seed(11), _table().cuda()
    x, pos = _normal(g, 40, 64, 128).cuda(), _ints(range(40))
    c, k_pe = (t.cuda() for t in _tokens(g, 8, joint=False))
    want = B.indexer_encode(x, table, pos, hadamard=True)
    cu, tables = _ints([0, 8]), [_ints([[2 * k, 2 * k + 1]]) for k in range(3)]
    ckv, kpe = (torch.zeros((6, 64, d), dtype=BF16, device="cuda") for d in (512, 64))
    lens, drafts, path, plens = _ints([60]), _ints([8]), _ints([[0, 3, 7]]), _ints([3])
    torch.cuda.synchronize()

    def calls(k):
        s = torch.cuda.Stream()
        codes, scale = torch.empty((40, 64, 128), dtype=torch.uint8, device="cuda"), torch.empty(40, device="cuda")
        n1, n2 = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        for _ in range(300):
            B.indexer_encode(x, table, pos, hadamard=True, codes=codes, scale=scale, stream=s)
            B.latent_cache_append(c, k_pe, table, cu, tables[k], lens, ckv, kpe, new_lens=n1, stream=s)
            B.latent_cache_accept(ckv, kpe, tables[k], n1, drafts, path, plens, new_lens=n2, stream=s)
        s.synchronize()
        return codes, scale, n1.tolist(), n2.tolist(), tables[k][0].tolist()

    def releases():
        for _ in range(150):
            B.release()

    with ThreadPoolExecutor(4) as pool:
        done = [pool.submit(calls, k) for k in range(3)]
        pool.submit(releases).result()
        done = [d.result() for d in done]
    torch.cuda.synchronize()
    for codes, scale, n1, n2, pages in done:
        assert torch.equal(codes, want[0].view(torch.uint8)) and torch.equal(scale, want[1])
        assert n1 == [68] and n2 == [63]
        flat = ckv[pages].view(-1, 512)
        assert torch.equal(flat[60:63], c[[0, 3, 7]]) and torch.equal(flat[63:68], c[3:8])


class PerThread:
    """cudaStreamPerThread: one handle, of a stream of its own on every thread."""
    cuda_stream = 2


def test_the_streams_of_threads_are_apart(B):  # noqa: F811
    from concurrent.futures import ThreadPoolExecutor
    s, table, x = PerThread(), _table().cuda(), torch.zeros((1, 64, 128), dtype=BF16, device="cuda")
    codes, scale = torch.empty((1, 64, 128), dtype=torch.uint8, device="cuda"), torch.empty(1, device="cuda")
    good, bad = _ints([0]), _ints([MAXPOS])
    torch.cuda.synchronize()

    def encode(pos):
        B.indexer_encode(x, table, pos, codes=codes, scale=scale, stream=s)
        return B.latent_last_status(s)

    with ThreadPoolExecutor(1) as first, ThreadPoolExecutor(1) as second:
        assert first.submit(encode, bad).result() == B.DSA_ERR_RANGE
        assert second.submit(B.latent_last_status, s).result() == 0  # (nothing has run on this thread's)
        assert second.submit(encode, good).result() == 0
        assert first.submit(B.latent_last_status, s).result() == B.DSA_ERR_RANGE
        assert first.submit(encode, good).result() == 0


def test_threads_append_on_their_streams_at_once(B):  # noqa: F811
    """Calls of different sizes, in place, on four threads' own streams."""
    from concurrent.futures import ThreadPoolExecutor
    s, table = PerThread(), _table().cuda()

    def work(k):
        g = torch.Generator().manual_seed(20 + k)
        new = [(k + 1) * 37 % 61 + 300 * k, 5, 64 * k]
        lens, T = [3, 60, 64], sum(new)
        p = Pages([a + b for a, b in zip(new, lens)], seed=k)
        c, k_pe = (t.cuda() for t in _tokens(g, T, joint=False))
        cu, bt, dl, before = _ints(np.concatenate([[0], np.cumsum(new)])), p.table.cuda(), _ints(lens), _ints(lens)
        x, pos = _normal(g, 5 + 90 * k, 64, 128).cuda(), _ints(range(5 + 90 * k))
        codes = torch.empty((len(pos), 64, 128), dtype=torch.uint8, device="cuda")
        scale = torch.empty(len(pos), device="cuda")
        out = torch.empty(3, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        for _ in range(100):
            B.latent_cache_append(c, k_pe, table, cu, bt, before, p.ckv, p.kpe, new_lens=out, stream=s)
            B.indexer_encode(x, table, pos, hadamard=True, codes=codes, scale=scale, stream=s)
        B.latent_cache_append(c, k_pe, table, cu, bt, dl, p.ckv, p.kpe, new_lens=dl, stream=s)
        status = B.latent_last_status(s)
        flat = p.ckv.view(-1, 512)
        for b, (a, n) in enumerate(zip(lens, new)):
            lo = sum(new[:b])
            assert torch.equal(flat[torch.from_numpy(p.slots(b, a, n)).cuda()], c[lo:lo + n])
        assert out.tolist() == dl.tolist() == [a + n for a, n in zip(lens, new)]
        return status

    with ThreadPoolExecutor(4) as pool:
        assert list(pool.map(work, range(4))) == [0] * 4


# ------------------------------------------------------------------- norms --
SIZES = [1e-38, 1e-30, 1e-22, 1e-12, 1e15, 3e18, 1e25, 1e38]


def _sized(g, size, *shape):
    """Normal values times `size`, as far as bf16 goes."""
    return (torch.randn(shape, generator=g, dtype=torch.float64) * size).clamp(-3.3e38, 3.3e38).to(BF16)


@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-6, 1e20])
@pytest.mark.parametrize("G,had", [(64, True), (1, False)])
def test_layer_norm_of_rows_of_any_size(B, G, had, eps):  # noqa: F811
    """A norm's result does not depend on whether the squares of its row fit fp32; rows of all sizes in one call, so that
    warps and tokens mix them.  The bounds are those of every encoding, relative to the norm's own terms: a power of two
    loses nothing, and eps times two of them one rounding, or all of what is below 2^-149 of a sum of at least 1/128."""
    g, table, T = torch.Generator().manual_seed(31), _table(), 8 * len(SIZES)
    x = torch.stack([_sized(g, SIZES[t % len(SIZES)], G, 128) for t in range(T)])
    x[5] = torch.stack([_sized(g, SIZES[(3 * r) % len(SIZES)], 128) for r in range(G)])  # and one token that has them all
    pos, nm = torch.arange(T, dtype=torch.int32), (torch.randn(128, generator=g), torch.randn(128, generator=g), eps)
    codes, s, _ = B.indexer_encode(x.cuda(), table.cuda(), pos.cuda(), norm=(nm[0].cuda(), nm[1].cuda(), eps), hadamard=had)
    # (the oracle works out the square of eps' fp32 value)
    y, reach = te.index_rows(_np(x), _np(table)[:T], (_np(nm[0]), _np(nm[1]), float(np.float32(eps))), False, had)
    assert B.latent_last_status() == 0
    check_codes(codes, s, y, reach)


@pytest.mark.parametrize("ctas", [0, 3])
@pytest.mark.parametrize("G,H,T", [(64, 4, 300), (1, 1, 5000), (1, 3, 900)])
def test_a_large_row_changes_no_other(B, G, H, T, ctas):  # noqa: F811
    """Tokens beside one that is taken again are taken again with it: with the same bits, and rope parts in place are
    rotated once."""
    g, table = torch.Generator().manual_seed(34), _table(T).cuda()
    x, pe, pos = _normal(g, T, G, 128), _normal(g, T, H, 64), torch.arange(T, dtype=torch.int32).cuda()
    nm = (torch.randn(128, generator=g).cuda(), torch.randn(128, generator=g).cuda(), 1e-6)
    large = torch.randperm(T, generator=g)[:T // 40]
    x2 = x.clone()
    x2[large, -1] = _sized(g, 1e38, len(large), 128)
    rest = torch.ones(T, dtype=torch.bool)
    rest[large] = False
    rest = rest.cuda()
    B.set_option("grid_ctas", ctas)
    try:
        codes, scale, out = B.indexer_encode(x.cuda(), table, pos, norm=nm, hadamard=True, pe=pe.cuda())
        there = pe.cuda()
        codes2, scale2, _ = B.indexer_encode(x2.cuda(), table, pos, norm=nm, hadamard=True, pe=there, pe_out=there)
        assert B.latent_last_status() == 0
    finally:
        B.set_option("grid_ctas", 0)
    assert torch.equal(there, out) and torch.equal(scale[rest], scale2[rest])
    assert torch.equal(codes.view(torch.uint8)[rest], codes2.view(torch.uint8)[rest])


@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-6, 1e20])
def test_append_norms_of_any_size(B, eps):  # noqa: F811
    g, table, T = torch.Generator().manual_seed(32), _table(), 8 * len(SIZES) + 3
    c = torch.stack([_sized(g, SIZES[t % len(SIZES)], 512) for t in range(T)])
    ik = torch.stack([_sized(g, SIZES[t % len(SIZES)], 128) for t in range(T)])
    k_pe, p = _normal(g, T, 64), Pages([T + 9], seed=33)
    # (weights that keep the smallest results in bf16's normal range: x / sqrt(eps) is 1e-48 and more of 1e-38 and 1e20)
    w = (1 + 0.3 * torch.rand(512, generator=g)) * (1e20 if eps > 1 else 1.0)
    nm = torch.randn(128, generator=g), torch.randn(128, generator=g), float(np.float32(eps))
    B.latent_cache_append(c.cuda(), k_pe.cuda(), table.cuda(), _ints([0, T]), p.table.cuda(), _ints([9]), p.ckv, p.kpe,
                          c_norm=(w.cuda(), eps), index_k=ik.cuda(), index_norm=(nm[0].cuda(), nm[1].cuda(), eps),
                          hadamard=True, k_cache=p.kc, k_cache_scale=p.ks)
    assert B.latent_last_status() == 0
    s = p.slots(0, 9, T)
    want, got = te.rms_norm(_np(c), _np(w), float(np.float32(eps))), _np(p.ckv).reshape(-1, 512)[s]
    # below bf16's normal range a step is 2^-133, and below fp32's a product's half a step of 2^-149 comes before it
    assert np.all(np.abs(got - want) <= (BF + 2.0 ** -18) * np.abs(want) + 2.0 ** -133)
    at = torch.from_numpy(s).cuda()
    check_codes(p.kc.view(-1, 128)[at][:, None], p.ks.view(-1)[at],
                *te.index_rows(_np(ik)[:, None], _np(table)[9:9 + T], _np_norm(nm), False, True))


# --------------------------------------------------------------- refusals --
def test_arguments_of_any_kind_are_refused_not_taken(B):  # noqa: F811
    """Every tensor argument in turn as something else: an exception of the bindings' own kinds, and nothing launched."""
    def z(*shape, dtype=BF16):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    i32, f32 = dict(dtype=torch.int32), dict(dtype=torch.float32)
    table, norm = z(100, 64, **f32), (z(128, **f32), z(128, **f32), 1e-6)
    cache = dict(ckv_cache=z(3, 64, 512), kpe_cache=z(3, 64, 64), block_table=z(2, 2, **i32), seq_lens=z(2, **i32))
    keys = dict(k_cache=z(3, 64, 128, dtype=torch.uint8), k_cache_scale=z(3, 64, **f32))
    calls = {
        B.indexer_encode: dict(x=z(4, 64, 128), cos_sin=table, positions=z(4, **i32), pe=z(4, 2, 64), pe_out=z(4, 2, 64),
                               codes=z(4, 64, 128, dtype=torch.uint8), scale=z(4, **f32), norm=norm),
        B.latent_cache_append: dict(c=z(4, 512), k_pe=z(4, 64), cos_sin=table, cu_new=z(3, **i32), **cache, **keys,
                                    c_norm=(z(512, **f32), 1e-6), index_k=z(4, 128), index_norm=norm,
                                    positions=z(4, **i32), c_out=z(4, 512), k_pe_out=z(4, 64), new_lens=z(2, **i32)),
        B.latent_attention_tree: dict(q_nope=z(2, 3, 16, 512), q_pe=z(2, 3, 16, 64), **cache, sm_scale=0.1,
                                      tree_mask=z(2, 3, 1, dtype=torch.int64), draft_lens=z(2, **i32),
                                      out=z(2, 3, 16, 512), lse=z(2, 3, 16, **f32)),
        B.latent_cache_accept: dict(**cache, **keys, draft_lens=z(2, **i32), path=z(2, 5, **i32), path_lens=z(2, **i32),
                                    new_lens=z(2, **i32))}
    optional = {"pe_out", "codes", "scale", "norm", "positions", "c_norm", "index_norm", "c_out", "k_pe_out", "new_lens",
                "draft_lens", "out", "lse"}
    before = B.launch_count()
    for fn, args in calls.items():
        for name, value in args.items():
            if isinstance(value, float):
                continue
            if isinstance(value, tuple):
                wrong = [(None, *value[1:]), (value[0].cpu(), *value[1:]), (value[0][None], *value[1:])]
            else:
                wrong = [3, [1, 2], "x", value.cpu(), value[0], value[None], value.double(), value.reshape(-1)[:1]]
                if name not in optional or (fn is B.indexer_encode and name == "positions") or (
                        fn is B.latent_cache_accept and name == "draft_lens"):
                    wrong.append(None)
            for v in wrong:
                if fn is B.indexer_encode and name in ("x", "pe") and v is None:
                    continue  # (optional, but for what goes with them)
                with pytest.raises((TypeError, ValueError, B.IndexerError)):
                    fn(**dict(args, **{name: v}))
                    pytest.fail(f"{fn.__name__}: {name} was taken")
    assert B.launch_count() == before


# ------------------------------------------- more work than threads or CTAs --
def _tree_call(B, nn, H, seqs, seed):  # noqa: F811
    """A tree's call over sequences of (length, nodes), one node of each that nobody sees holding NaN or infinity,
    padding queries NaN; held against the oracle, and run again for the same bits."""
    rng = np.random.default_rng(seed)
    lens, drafts = [a for a, _ in seqs], [n for _, n in seqs]
    c = Cache(lens, seed=seed)
    seen = [_seen_of(_random_tree(rng, n)) for n in drafts]
    for b, n in enumerate(drafts):
        if n > 2:
            j = int(rng.integers(1, n))
            seen[b] = [s - {j} for s in seen[b]]
            slot = la.slots_of(c.table[b].numpy(), lens[b])[lens[b] - n + j]
            c.data.view(-1, 576)[slot] = float("nan") if b % 2 else float("inf")
    qn, qp = _queries(len(lens), nn, H, seed=seed + 1)
    for b, n in enumerate(drafts):
        qn[b, n:] = float("nan")
    mask = _mask(seen, nn)
    out, lse = _tree(B, c, qn, qp, mask, drafts)
    assert B.latent_last_status() == 0
    again, lse2 = _tree(B, c, qn, qp, mask, drafts)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16)) and torch.equal(lse2, lse)
    c.data = torch.nan_to_num(c.data, nan=0.0, posinf=0.0)
    _check_tree(c, qn, qp, out, lse, seen)


@pytest.mark.parametrize("ctas", [0, 1, 7, 40])
@pytest.mark.parametrize("nn,H,n", [(5, 16, 450), (5, 30, 260), (3, 16, 700)])
def test_tree_of_more_items_than_threads(B, nn, H, n, ctas):  # noqa: F811
    """Items are numbered in rounds of a CTA's threads (384, or 352): one or two blocks of 128 rows a sequence, and
    blocks of 64; many items a run, and whole ones, or without a key."""
    seqs = [(i * 7 % 301, min(i * 7 % 301, i * 5 % (nn + 1))) for i in range(n)]
    B.set_option("grid_ctas", ctas)
    try:
        _tree_call(B, nn, H, seqs, seed=n + ctas)
    finally:
        B.set_option("grid_ctas", 0)


@pytest.mark.parametrize("nn,H,seqs", [(8, 16, [(33000, 8)]), (5, 16, [(131080, 5)]), (2, 16, [(131080, 2)]),
                                       (40, 16, [(70000, 33), (300, 40)])])
def test_tree_behind_long_histories(B, nn, H, seqs):  # noqa: F811
    """Rows cut into a piece for nearly every pair of CTAs, which are joined by eight warps in several rounds."""
    _tree_call(B, nn, H, seqs, seed=nn)
