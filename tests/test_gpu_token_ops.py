"""GPU parity of the operators that encode, append, verify and keep tokens, against the float64 oracle.

Tolerances, from the kernels' arithmetic (u = 2^-24, half a step of fp32):
  index values  a mean of 128: 7 additions in a lane's tree or 33 in a row, 34 u of mean |x| in all; the difference u;
           the reciprocal root 2 ulp and the squares' sum, 24 u; products and the bias 3 u; a rotation 3 u and the sines'
           sum of magnitudes; the Hadamard transform 8 u of the sum of magnitudes: 73 u of the `reach` (the sum of all
           magnitudes that went into a value), rounded up to 80 u = 5 2^-20
  scale    the same of the token's largest reach / 448, and 2^-22 of it for its own two roundings
  codes    half a step of e4m3: 2^-4 of the value, 2^-10 below the normal range; and the value's error; 2^-22 of the value
           for the reciprocal
  rope     half a step of bf16, 2^-8 of the value, and 4 u of the reach
  latent   2^-8 of the value, 2^-18 of it for the root of a sum of 512 squares (at most 23 additions deep) and 2 products
  tree     as attention over the paged cache (test_gpu_latent)"""
import numpy as np
import pytest
import torch

from oracle import indexer
from oracle import latent_attention as la
from oracle import token_encode as te
from test_gpu_latent import BF, B, SCALE, Cache, _check_rows, _ints, _queries  # noqa: F401
from helpers import check_rows_parallel  # noqa: F401

pytestmark = pytest.mark.gpu

VALUE = 5 * 2.0 ** -20
MAXPOS = 1000
BF16 = torch.bfloat16


def _normal(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(BF16)


def _table(n=MAXPOS):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(32) / 32.0)
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1)).float()


def _norm(g, n=128):
    return 1 + 0.3 * torch.randn(n, generator=g), 0.2 * torch.randn(n, generator=g), 1e-6


def _np(t):
    return t.detach().cpu().double().numpy()


def _np_norm(norm):
    return None if norm is None else (_np(norm[0]), _np(norm[1]), norm[2])


def check_codes(codes, scale, y, reach):
    """codes [T, G, 128] (uint8 or e4m3), scale [T] against the oracle's y and reach."""
    codes = codes.view(torch.uint8).cpu().numpy()
    s = _np(scale)
    t = VALUE * reach
    want = te.scales(y)
    assert np.all(np.abs(s - want) <= t.max((1, 2)) / 448 + 2.0 ** -22 * want), (s, want)
    got = te.values(codes)
    assert np.all(np.isfinite(got))
    s = s[:, None, None]
    tol = np.maximum(2.0 ** -4 * (np.abs(y) + t), 2.0 ** -10 * s) + t + 2.0 ** -22 * np.abs(y)
    err = np.abs(got * s - y)
    assert np.all(err <= tol), float((err / tol).max())
    # and almost all of them are the nearest ones, which the bound above does not ask for (a value whose error can
    # carry it over a border between codes may be its neighbour: with t of a few 2^-18 of a step of 2^-3 that is rare)
    assert (codes != te.nearest_codes(np.clip(y / s, -448, 448))).mean() <= 0.01


def check_rope(got, x, cs, interleaved):
    want = te.rotate(x, cs, interleaved)
    reach = np.abs(x).max(-1, keepdims=True) * 2
    err = np.abs(_np(got) - want)
    assert np.all(err <= BF * np.abs(want) + 4 * 2.0 ** -24 * reach), float(err.max())


# ------------------------------------------------------------------ encode --
@pytest.mark.parametrize("T,G,H", [(1, 64, 16), (2, 64, 1), (65, 64, 5), (7, 64, 128), (1, 1, 1), (63, 1, 1), (64, 1, 3),
                                   (333, 1, 1), (9, 64, None), (70, 1, None), (33, None, 7), (1, None, 64)])
@pytest.mark.parametrize("norm,had,inter,pe_inter", [(False, False, False, True), (True, True, False, True),
                                                     (True, False, True, False), (False, True, True, True)])
def test_encode_matches_oracle(B, T, G, H, norm, had, inter, pe_inter):  # noqa: F811
    g = torch.Generator().manual_seed(T * 7 + (G or 0) + (H or 0))
    table = _table()
    pos = torch.randint(0, MAXPOS, (T,), generator=g, dtype=torch.int32)
    cs = _np(table)[pos.numpy()]
    x = None if G is None else _normal(g, T, G, 128)
    pe = None if H is None else _normal(g, T, H, 64)
    nm = _norm(g) if norm and G else None
    dev = None if nm is None else (nm[0].cuda(), nm[1].cuda(), nm[2])
    codes, scale, out = B.indexer_encode(None if x is None else x.cuda(), table.cuda(), pos.cuda(), norm=dev,
                                         interleaved=inter, hadamard=had, pe=None if pe is None else pe.cuda(),
                                         pe_interleaved=pe_inter)
    assert B.latent_last_status() == 0
    if G:
        check_codes(codes, scale, *te.index_rows(_np(x), cs, _np_norm(nm), inter, had))
    else:
        assert codes is None and scale is None
    if H:
        check_rope(out, _np(pe), cs[:, None], pe_inter)


@pytest.mark.parametrize("G", [64, 1])
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e30, 3e37])
def test_encode_ends_of_the_range(B, G, scale):  # noqa: F811
    """Scales below fp32's normal range, large ones, and a token of zeros."""
    g = torch.Generator().manual_seed(5)
    x = _normal(g, 70, G, 128, scale=scale)
    x[3] = 0
    x[4] = 0
    x[4, -1, 127] = scale
    pos, table = torch.arange(70, dtype=torch.int32), _table()
    codes, s, _ = B.indexer_encode(x.cuda(), table.cuda(), pos.cuda())
    y, reach = te.index_rows(_np(x), _np(table)[:70], None, False, False)
    # below the normal range a step is 2^-149, whatever the value; the products of a rotation lose one each
    sub = 8 * 2.0 ** -149 / VALUE
    got = te.values(codes.view(torch.uint8).cpu().numpy())
    s = _np(s)
    assert s[3] == 1.0 and np.all(got[3] == 0)
    t = VALUE * (reach + sub)
    want = te.scales(y)
    assert np.all(np.abs(s - want) <= t.max((1, 2)) / 448 + 2.0 ** -22 * want + 2.0 ** -149)
    s = s[:, None, None]
    tol = np.maximum(2.0 ** -4 * (np.abs(y) + t), 2.0 ** -10 * s) + t + 2.0 ** -22 * np.abs(y)
    # (a scale below the normal range is itself off by up to half a step of 2^-149, and code times it by 448 of those)
    assert np.all(np.abs(got * s - y) <= tol + 448 * 2.0 ** -149)
    assert got[4, -1, 127] == 448


@pytest.mark.parametrize("had", [False, True])
@pytest.mark.parametrize("G", [64, 1])
@pytest.mark.parametrize("steps", [3, 50, 100, 3000, 10 ** 6])
def test_encode_scales_of_few_bits(B, G, steps, had):  # noqa: F811
    """Values of some `steps` of 2^-149, by a norm's weights: a scale that rounds to 0 is 1, and the codes are of the
    scale that is stored."""
    g, step, T = torch.Generator().manual_seed(steps), 2.0 ** -149, 70
    x, pos, table = _normal(g, T, G, 128), torch.arange(T, dtype=torch.int32), _table()
    nm = torch.full((128,), steps * step, dtype=torch.float64).float(), torch.zeros(128), 1e-6
    assert float(nm[0][0]) == steps * step
    codes, s, _ = B.indexer_encode(x.cuda(), table.cuda(), pos.cuda(), norm=(nm[0].cuda(), nm[1].cuda(), nm[2]),
                                   hadamard=had)
    y, reach = te.index_rows(_np(x), _np(table)[:T], _np_norm(nm), False, had)
    got, s = te.values(codes.view(torch.uint8).cpu().numpy()), _np(s)
    # a normalised value is off by half a step and turned to half of sqrt(2), each of a rotation's two products by half:
    # below 2; the transform adds 128 of those and multiplies by 1 / sqrt(128), and rounds: below 24
    off = (24 if had else 2) * step + VALUE * reach
    assert np.all(np.abs(np.where(s == 1, 0, s) - _top(y)) <= step / 2 + off.max((1, 2)) / 448 + 2.0 ** -22 * _top(y))
    assert np.all(got[s == 1] == 0)
    s = np.where(s == 1, 0, s)[:, None, None]
    # a code is off by 2^-4 or 2^-10 of the scale; a scale by half a step, which 448 times is what is cut off at most
    tol = np.maximum(2.0 ** -4 * (np.abs(y) + off), 2.0 ** -10 * s) + off + 224 * step + off.max((1, 2), keepdims=True)
    assert np.all(np.abs(got * s - y) <= tol)


def _top(y):
    return np.abs(y).max((1, 2)) / 448


@pytest.mark.parametrize("G", [64, 1])
def test_encode_padding_strides_and_in_place(B, G):  # noqa: F811
    """Positions below 0 are padding, at or past the table's end an error: outputs stay as they were.  Rows are parts of
    wider arrays; the rope parts are rotated in place, where their neighbours have to stay."""
    g = torch.Generator().manual_seed(6)
    T, H, table = 67, 6, _table()
    wide = _normal(g, T, G, 192).cuda()
    q = _normal(g, T, H, 200).cuda()
    pos = torch.randint(0, MAXPOS, (T,), generator=g, dtype=torch.int32)
    pos[[0, 20, 66]] = torch.tensor([-1, -(2 ** 31), -5], dtype=torch.int32)
    keep = pos >= 0
    cs = _np(table)[pos.clamp(min=0).numpy()]
    before = q.clone()
    codes = torch.full((T, G, 128), 0x55, dtype=torch.uint8, device="cuda")
    scale = torch.full((T,), -3.0, device="cuda")
    r = B.indexer_encode(wide[..., 64:], table.cuda(), pos.cuda(), hadamard=True, pe=q[..., 128:192], codes=codes,
                         scale=scale, pe_out=q[..., 128:192])
    assert r[0] is codes and r[1] is scale and B.latent_last_status() == 0
    y, reach = te.index_rows(_np(wide[..., 64:]), cs, None, False, True)
    check_codes(codes[keep.cuda()], scale[keep.cuda()], y[keep.numpy()], reach[keep.numpy()])
    check_rope(q[..., 128:192].cpu()[keep], _np(before[..., 128:192])[keep.numpy()], cs[keep.numpy()][:, None], True)
    assert torch.all(codes[~keep.cuda()] == 0x55) and torch.all(scale[~keep.cuda()] == -3.0)
    assert torch.equal(q[~keep.cuda()], before[~keep.cuda()])
    assert torch.equal(q[..., :128], before[..., :128]) and torch.equal(q[..., 192:], before[..., 192:])
    # the same with a position past the table
    pos2 = pos.clone()
    pos2[[5, 40]] = torch.tensor([MAXPOS, 2 ** 31 - 1], dtype=torch.int32)
    again, s2 = torch.full_like(codes, 0x55), torch.full_like(scale, -3.0)
    out = torch.full((T, H, 64), 7.0, dtype=BF16, device="cuda")
    B.indexer_encode(wide[..., 64:], table.cuda(), pos2.cuda(), hadamard=True, pe=before[..., 128:192], codes=again,
                     scale=s2, pe_out=out)
    assert B.latent_last_status() == B.DSA_ERR_RANGE
    ok = keep.clone()
    ok[[5, 40]] = False
    ok = ok.cuda()
    assert torch.equal(again[ok], codes[ok]) and torch.equal(s2[ok], scale[ok]) and torch.equal(out[ok], q[ok][..., 128:192])
    assert torch.all(again[~ok] == 0x55) and torch.all(s2[~ok] == -3.0) and torch.all(out[~ok] == 7.0)
    B.indexer_encode(wide[..., 64:], table.cuda(), pos.cuda())
    assert B.latent_last_status() == 0


def test_encode_rows_far_apart(B):  # noqa: F811
    """Token strides whose offsets pass 32 bits."""
    g = torch.Generator().manual_seed(7)
    step = (1 << 30) + 8
    store = torch.empty(2 * step + 64 * 128, dtype=BF16, device="cuda")
    x, pe = store.as_strided((3, 64, 128), (step, 128, 1)), store.as_strided((3, 4, 64), (step, 64, 1))
    vals, pos, table = _normal(g, 3, 64, 128), torch.tensor([3, 500, 999], dtype=torch.int32), _table()
    x.copy_(vals)
    codes, scale, out = B.indexer_encode(x, table.cuda(), pos.cuda(), pe=pe)
    cs = _np(table)[pos.numpy()]
    check_codes(codes, scale, *te.index_rows(_np(vals), cs, None, False, False))
    check_rope(out, _np(vals).reshape(3, -1)[:, :256].reshape(3, 4, 64), cs[:, None], True)


def test_encoded_rows_go_to_the_indexer(B):  # noqa: F811
    """Queries and keys as the dense indexer takes them: its choice over the codes is exact."""
    from oracle import checks
    g = torch.Generator().manual_seed(8)
    Q, N, K, table = 5, 900, 128, _table().cuda()
    q, s, _ = B.indexer_encode(_normal(g, Q, 64, 128).cuda(), table, torch.arange(895, 900, dtype=torch.int32).cuda(),
                               hadamard=True)
    k, ks, _ = B.indexer_encode(_normal(g, N, 1, 128).cuda(), table, torch.arange(N, dtype=torch.int32).cuda(),
                                hadamard=True, norm=tuple(x.cuda() if torch.is_tensor(x) else x for x in _norm(g)))
    w = torch.randn((Q, 64), generator=g)
    lo, hi = torch.zeros(Q, dtype=torch.int32), torch.arange(896, 901, dtype=torch.int32)
    out = B.indexer_topk(q, s, k[:, 0], ks, w.cuda(), lo.cuda(), hi.cuda(), K=K)
    o = indexer.DenseOracle(q.view(torch.uint8).cpu().numpy(), s.cpu().numpy(), k[:, 0].view(torch.uint8).cpu().numpy(),
                            ks.cpu().numpy(), w.numpy(), lo.numpy(), hi.numpy(), K)
    for t in range(Q):
        ids, scores, E = o.row_scores(t)
        assert not checks.check_row(out[t].cpu().numpy(), ids, scores, E, K)


# ------------------------------------------------------------------ append --
class Pages:
    """An empty paged cache for sequences of these final lengths, filled with a pattern; joint: one [P, 64, 576] array."""

    def __init__(self, totals, seed, joint=False, spare=2):
        g = torch.Generator().manual_seed(seed)
        n = [-(-max(0, x) // 64) for x in totals]
        self.P = sum(n) + spare
        perm = torch.randperm(self.P, generator=g).tolist()
        self.table = torch.full((len(totals), max(1, max(n))), -1, dtype=torch.int32)
        for b, c in enumerate(n):
            self.table[b, :c] = torch.tensor(perm[:c], dtype=torch.int32)
            perm = perm[c:]
        both = torch.full((self.P, 64, 576), 3.0, dtype=BF16, device="cuda")
        self.ckv, self.kpe = (both[..., :512], both[..., 512:]) if joint else (both[..., :512].clone(),
                                                                               both[..., 512:].clone())
        self.kc = torch.full((self.P, 64, 128), 0x33, dtype=torch.uint8, device="cuda")
        self.ks = torch.full((self.P, 64), -2.0, device="cuda")

    def slots(self, b, first, n):
        at = np.arange(first, first + n)
        return self.table[b].numpy()[at // 64].astype(np.int64) * 64 + at % 64


def _tokens(g, T, joint=True):
    c = _normal(g, T, 576)
    return (c[:, :512], c[:, 512:]) if joint else (c[:, :512].clone(), c[:, 512:].clone())


def check_appended(p, cu, lens, c, k_pe, table, c_norm=None, pe_inter=True, index=None, positions=None, skip=(),
                   dense=None):
    """Every slot of the cache: the new tokens' as the oracle has them, all others as they were.  index = (rows, norm,
    interleaved, hadamard); skip: tokens that are not written; dense = (c_out, k_pe_out), filled with 9 before."""
    ckv, kpe = _np(p.ckv).reshape(-1, 512), _np(p.kpe).reshape(-1, 64)
    kc, ks = p.kc.view(torch.uint8).reshape(-1, 128), p.ks.reshape(-1)
    free = np.ones(len(ckv), bool)
    done = []
    for b in range(len(lens)):
        lo, hi = int(cu[b]), int(cu[b + 1])
        t = np.array([i for i in range(lo, hi) if i not in skip], int)
        done += t.tolist()
        if not len(t):
            continue
        at = lens[b] + t - lo
        s = p.slots(b, 0, int(at.max()) + 1)[at]
        free[s] = False
        cs = _np(table)[at if positions is None else positions.numpy()[t]]
        x = _np(c)[t]
        want = x if c_norm is None else te.rms_norm(x, _np(c_norm[0]), c_norm[1])
        tol = 0 if c_norm is None else (BF + 2.0 ** -18) * np.abs(want)
        assert np.all(np.abs(ckv[s] - want) <= tol), b
        check_rope(torch.from_numpy(kpe[s]), _np(k_pe)[t], cs, pe_inter)
        if dense is not None:
            assert np.array_equal(_np(dense[0])[t], ckv[s]) and np.array_equal(_np(dense[1])[t], kpe[s])
        if index is not None:
            rows, norm, inter, had = index
            si = torch.from_numpy(s).cuda()
            check_codes(kc[si][:, None], ks[si], *te.index_rows(_np(rows)[t][:, None], cs, _np_norm(norm), inter, had))
    assert np.all(ckv[free] == 3.0) and np.all(kpe[free] == 3.0)
    f = torch.from_numpy(free).cuda() if index is not None else slice(None)
    assert torch.all(kc[f] == 0x33) and torch.all(ks[f] == -2.0)
    if dense is not None:
        rest = np.setdiff1d(np.arange(len(c)), done)
        assert np.all(_np(dense[0])[rest] == 9.0) and np.all(_np(dense[1])[rest] == 9.0)


APPEND = [([1], [0]), ([1], [63]), ([1], [64]), ([130], [0]), ([1] * 70, list(range(70))), ([0, 3, 0, 65, 1, 0], [5, 62, 0, 127, 64, 9]),
          ([700], [100]), ([200, 17], [0, 300])]


@pytest.mark.parametrize("new,lens", APPEND)
@pytest.mark.parametrize("norm,index,dense,pe_inter,joint,pad", [
    (True, None, False, True, False, 0), (True, (True, False, True), True, True, True, 3),
    (False, (False, True, False), False, False, False, 1), (False, None, True, False, True, 70),
    (True, (True, True, True), False, False, True, 0)])
def test_append_matches_oracle(B, new, lens, norm, index, dense, pe_inter, joint, pad):  # noqa: F811
    g = torch.Generator().manual_seed(sum(new) + len(new) + pad)
    n, T, table = len(new), sum(new) + pad, _table()
    p = Pages([a + b for a, b in zip(new, lens)], seed=pad, joint=joint)
    c, k_pe = _tokens(g, T, joint)
    cu = np.concatenate([[0], np.cumsum(new)])
    cn = (1 + 0.3 * torch.randn(512, generator=g), 1e-5) if norm else None
    ix = nm = None
    if index:
        ix, nm = _normal(g, T, 128), _norm(g) if index[0] else None
    outs = (torch.full((T, 512), 9.0, dtype=BF16, device="cuda"),
            torch.full((T, 64), 9.0, dtype=BF16, device="cuda")) if dense else (None, None)
    new_lens = B.latent_cache_append(
        c.cuda() if not joint else torch.cat([c, k_pe], 1).cuda()[:, :512], k_pe.cuda(), table.cuda(), _ints(cu),
        p.table.cuda(), _ints(lens), p.ckv, p.kpe, c_norm=None if cn is None else (cn[0].cuda(), cn[1]),
        pe_interleaved=pe_inter, index_k=None if ix is None else ix.cuda(),
        index_norm=None if nm is None else (nm[0].cuda(), nm[1].cuda(), nm[2]), interleaved=bool(index and index[1]),
        hadamard=bool(index and index[2]), k_cache=p.kc if index else None, k_cache_scale=p.ks if index else None,
        c_out=outs[0], k_pe_out=outs[1])
    assert B.latent_last_status() == 0
    assert new_lens.tolist() == [a + b for a, b in zip(new, lens)]
    check_appended(p, cu, lens, c, k_pe, table, cn, pe_inter, None if not index else (ix, nm, index[1], index[2]),
                   dense=outs if dense else None)


def test_append_at_given_positions_and_in_place(B):  # noqa: F811
    """Angles of given positions (a tree's depths, an evicted cache), new_lens in the place of seq_lens, and the dense
    copies in the place of the inputs."""
    g = torch.Generator().manual_seed(11)
    new, lens, table = [5, 40, 1], [60, 0, 200], _table()
    T, p = sum(new), Pages([65, 40, 201], seed=12)
    c, k_pe = _tokens(g, T)
    both = torch.cat([c, k_pe], 1).cuda()
    pos = torch.randint(0, MAXPOS, (T,), generator=g, dtype=torch.int32)
    cu, dl = np.concatenate([[0], np.cumsum(new)]), _ints(lens)
    cn = (torch.rand(512, generator=g), 1e-6)
    r = B.latent_cache_append(both[:, :512], both[:, 512:], table.cuda(), _ints(cu), p.table.cuda(), dl, p.ckv, p.kpe,
                              c_norm=(cn[0].cuda(), cn[1]), positions=pos.cuda(), c_out=both[:, :512],
                              k_pe_out=both[:, 512:], new_lens=dl)
    assert r is dl and dl.tolist() == [65, 40, 201] and B.latent_last_status() == 0
    check_appended(p, cu, lens, c, k_pe, table, cn, positions=pos, dense=(both[:, :512], both[:, 512:]))


def test_append_new_lens_in_place_of_many_tokens(B):  # noqa: F811
    """Thousands of CTAs read the lengths that the last of them replaces."""
    g = torch.Generator().manual_seed(13)
    new, lens, table = [9000, 1, 4000], [100, 64, 0], _table(10000)
    T, p = sum(new), Pages([9100, 65, 4000], seed=14)
    c, k_pe = (x.cuda() for x in _tokens(g, T, joint=False))
    cu = np.concatenate([[0], np.cumsum(new)])
    first = None
    for _ in range(20):
        dl = _ints(lens)
        B.latent_cache_append(c, k_pe, table.cuda(), _ints(cu), p.table.cuda(), dl, p.ckv, p.kpe, new_lens=dl)
        assert dl.tolist() == [9100, 65, 4000]
        got = (p.ckv.clone(), p.kpe.clone())
        assert first is None or (torch.equal(got[0], first[0]) and torch.equal(got[1], first[1]))
        first = got
    check_appended(p, cu, lens, c.cpu(), k_pe.cpu(), table)


def test_append_reports_and_skips_what_does_not_fit(B):  # noqa: F811
    g = torch.Generator().manual_seed(15)
    new, lens, table = [3, 4, 5, 6], [10, 62, 0, 64], _table(100)
    T, totals = sum(new), [13, 66, 5, 70]
    c, k_pe = _tokens(g, T, joint=False)
    cu = np.concatenate([[0], np.cumsum(new)])

    def run(p, cu=cu, lens=lens, btable=None, pos=None):
        out = torch.full((T, 512), 9.0, dtype=BF16, device="cuda"), torch.full((T, 64), 9.0, dtype=BF16, device="cuda")
        r = B.latent_cache_append(c.cuda(), k_pe.cuda(), table.cuda(), _ints(cu),
                                  (p.table if btable is None else btable).cuda(), _ints(lens), p.ckv, p.kpe,
                                  positions=None if pos is None else pos.cuda(), c_out=out[0], k_pe_out=out[1])
        return r.tolist(), B.latent_last_status(), out

    # a page outside the cache: that page's tokens are not written (logical slots 62, 63 of sequence 1 are)
    for page in (-1, 10 ** 6):
        p = Pages(totals, seed=16)
        bad = p.table.clone()
        bad[1, 1] = page
        r, status, out = run(p, btable=bad)
        assert r == totals and status == B.DSA_ERR_RANGE
        check_appended(p, cu, lens, c, k_pe, table, skip={5, 6}, dense=out)
    # a position outside the table
    pos = torch.arange(T, dtype=torch.int32)
    pos[[2, 9]] = torch.tensor([-1, 100], dtype=torch.int32)
    p = Pages(totals, seed=17)
    r, status, out = run(p, pos=pos)
    assert r == totals and status == B.DSA_ERR_RANGE
    check_appended(p, cu, lens, c, k_pe, table, skip={2, 9}, positions=pos, dense=out)
    # lengths that do not fit the table (two pages here)
    for wrong in (-1, 125, 2 ** 31 - 1):
        p = Pages(totals, seed=18)
        r, status, out = run(p, lens=[10, wrong, 0, 64])
        assert r == [13, wrong, 5, 70] and status == B.DSA_ERR_RANGE
        check_appended(p, cu, [10, 0, 0, 64], c, k_pe, table, skip={3, 4, 5, 6}, dense=out)
    # borders outside the arrays: the sequences beside them are skipped (a 0-token sequence with a sound border is not)
    p = Pages(totals, seed=19)
    r, status, out = run(p, cu=np.array([0, 3, 7, 12, 19]))
    assert r == [13, 66, 5, 64] and status == B.DSA_ERR_RANGE
    check_appended(p, cu, lens, c, k_pe, table, skip=set(range(12, 18)), dense=out)
    p = Pages(totals, seed=20)
    r, status, out = run(p, cu=np.array([-2, 3, 7, 12, 18]))
    assert r == [10, 66, 5, 70] and status == B.DSA_ERR_RANGE
    check_appended(p, cu, lens, c, k_pe, table, skip={0, 1, 2}, dense=out)
    # the next call starts from no status
    p = Pages(totals, seed=21)
    r, status, out = run(p)
    assert r == totals and status == 0
    check_appended(p, cu, lens, c, k_pe, table, dense=out)


def test_append_into_a_cache_past_32_bits(B):  # noqa: F811
    """Slots whose element and byte offsets pass 2^31."""
    g = torch.Generator().manual_seed(22)
    P, table = 68000, _table()
    ckv = torch.zeros((P, 64, 512), dtype=BF16, device="cuda")
    kpe = torch.zeros((P, 64, 64), dtype=BF16, device="cuda")
    c, k_pe = _tokens(g, 3, joint=False)
    bt = torch.tensor([[P - 1], [0], [P - 2]], dtype=torch.int32)
    B.latent_cache_append(c.cuda(), k_pe.cuda(), table.cuda(), _ints([0, 1, 2, 3]), bt.cuda(), _ints([63, 0, 5]), ckv, kpe)
    assert B.latent_last_status() == 0
    for t, (page, off) in enumerate([(P - 1, 63), (0, 0), (P - 2, 5)]):
        assert torch.equal(ckv[page, off].cpu(), c[t])
    # the path of a tree in the last pages
    n = B.latent_cache_accept(ckv, kpe, bt.cuda(), _ints([64, 1, 6]), _ints([1, 1, 6]), _ints([[0] * 2, [0] * 2, [5] * 2]),
                              _ints([1, 1, 1]))
    assert n.tolist() == [64, 1, 1] and torch.equal(ckv[P - 2, 0].cpu(), c[2])


# -------------------------------------------------------------------- tree --
def _random_tree(rng, n):
    return [-1] + [int(rng.integers(0, i)) for i in range(1, n)] if n else []


def _seen_of(parents):
    seen = []
    for i, p in enumerate(parents):
        seen.append((seen[p] if p >= 0 else set()) | {i})
    return seen


def _mask(seen, nn):
    words = -(-nn // 64)
    m = np.zeros((len(seen), nn, words), np.uint64)
    for b, rows in enumerate(seen):
        for i, s in enumerate(rows):
            for j in s:
                m[b, i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return torch.from_numpy(m.view(np.int64))


def _tree(B, c, qn, qp, mask, drafts, lens=None):  # noqa: F811
    ck, kp = c.device()
    out, lse = B.latent_attention_tree(qn.cuda(), qp.cuda(), ck, kp, c.table.cuda(), _ints(c.lens if lens is None else lens),
                                       mask.cuda(), SCALE, draft_lens=None if drafts is None else _ints(drafts))
    torch.cuda.synchronize()
    return out, lse


def _check_tree(c, qn, qp, out, lse, seen, only=None):
    ckv, kpe = c.flat()
    R = qn.shape[1] * qn.shape[2]
    ref = la.tree(_np(torch.nan_to_num(qn)), _np(torch.nan_to_num(qp)), ckv, kpe, c.table.numpy(), c.lens, seen, SCALE)
    for b in range(len(c.lens)) if only is None else only:
        _check_rows(_np(out[b]).reshape(R, 512), _np(lse[b]).reshape(R), ref[b], 576)


TREE = [
    # nn, H, (length, nodes) of each sequence
    (1, 16, [(1, 1), (64, 1), (65, 1), (500, 1)]), (8, 16, [(2000, 8)]), (8, 16, [(8, 8), (9, 8), (64, 8), (70, 8), (129, 8), (700, 8)]),
    (16, 16, [(300, 16), (16, 3), (5, 0), (0, 0), (1000, 1), (130, 15)]), (64, 16, [(64, 64), (1000, 64), (333, 17), (128, 64)]),
    (65, 3, [(65, 65), (190, 64), (500, 65)]), (130, 4, [(130, 130), (777, 128), (200, 1), (260, 129)]), (7, 5, [(100, 7), (90, 2)]),
    (16, 128, [(300, 16), (100, 9)]), (3, 100, [(65, 3), (64, 2)]), (33, 1, [(600, 33), (70, 33), (40, 20)]),
    (12, 24, [(4000, 12), (90, 5)]), (2, 16, [(30000, 2)]), (5, 16, [(5 * i, i % 6) for i in range(1, 60)]),
]


@pytest.mark.parametrize("nn,H,seqs", TREE)
def test_tree_matches_oracle(B, nn, H, seqs):  # noqa: F811
    """Random trees; nodes that nobody sees, and queries behind a sequence's nodes, hold NaN."""
    rng = np.random.default_rng(nn * 100 + H)
    lens, drafts = [a for a, _ in seqs], [n for _, n in seqs]
    c = Cache(lens, seed=nn + H, joint=bool(H % 2))
    seen = [_seen_of(_random_tree(rng, n)) for n in drafts]
    for b, n in enumerate(drafts):
        if n > 3:  # one node is left out by everybody
            j = int(rng.integers(1, n))
            seen[b] = [s - {j} for s in seen[b]]
            slot = la.slots_of(c.table[b].numpy(), lens[b])[lens[b] - n + j]
            c.data.view(-1, 576)[slot] = float("nan") if b % 2 else float("inf")
    qn, qp = _queries(len(lens), nn, H, seed=H)
    for b, n in enumerate(drafts):
        qn[b, n:] = float("nan")
    out, lse = _tree(B, c, qn, qp, _mask(seen, nn), drafts)
    assert B.latent_last_status() == 0
    c.data = torch.nan_to_num(c.data, nan=0.0, posinf=0.0)
    _check_tree(c, qn, qp, out, lse, seen)
    for _ in range(3):  # and the same bits again
        o2, l2 = _tree(B, c, qn, qp, _mask(seen, nn), drafts)
        assert torch.equal(o2, out) and torch.equal(l2, lse)


@pytest.mark.parametrize("nn,H,lens", [(4, 16, [4, 100, 64, 1000]), (70, 2, [70, 133, 500]), (40, 16, [300, 90])])
def test_tree_any_mask(B, nn, H, lens):  # noqa: F811
    """Masks that are no trees: rows that see no node (and without keys before the nodes nothing at all), all nodes,
    later ones; bits past the sequence's nodes do not count."""
    rng = np.random.default_rng(nn)
    c = Cache(lens, seed=nn)
    seen = []
    for L in lens:
        rows = [set(np.flatnonzero(rng.random(nn) < 0.5).tolist()) for _ in range(nn)]
        rows[0], rows[-1] = set(), set(range(nn))
        seen.append(rows)
    qn, qp = _queries(len(lens), nn, H, seed=H)
    out, lse = _tree(B, c, qn, qp, _mask(seen, nn), None)
    _check_tree(c, qn, qp, out, lse, seen)
    n = nn // 2 + 1
    out, lse = _tree(B, c, qn, qp, _mask(seen, nn), [n] * len(lens))
    cut = [[{j for j in s if j < n} for s in rows[:n]] for rows in seen]
    _check_tree(c, qn, qp, out, lse, cut)


def test_tree_of_a_chain_is_decode(B):  # noqa: F811
    """A chain of nodes gives the bits that decode gives."""
    c = Cache([500, 3, 130, 64, 0, 2], seed=31)
    qn, qp = _queries(6, 3, 16, seed=32)
    seen = [_seen_of([-1, 0, 1])] * 6
    out, lse = _tree(B, c, qn, qp, _mask(seen, 3), None)
    ck, kp = c.device()
    o2, l2 = B.latent_attention_paged(qn.cuda(), qp.cuda(), ck, kp, c.table.cuda(), _ints(c.lens), SCALE)
    for b in (0, 1, 2, 3, 4):
        assert torch.equal(out[b], o2[b]) and torch.equal(lse[b], l2[b])
    # a sequence with fewer keys than queries: here its first queries are the nodes, in decode its last ones see keys
    _check_tree(c, qn, qp, out, lse, seen[:4] + [[], seen[5][:2]], only=[4, 5])


def test_tree_far_logits(B):  # noqa: F811
    """Logits over thousands of units, and a node whose logits tower over the context's."""
    c = Cache([700, 90], seed=33)
    seen = [_seen_of(_random_tree(np.random.default_rng(1), 16))] * 2
    for b, L in enumerate(c.lens):
        c.data.view(-1, 576)[la.slots_of(c.table[b].numpy(), L)[-16:]] *= 8
    qn, qp = _queries(2, 16, 16, seed=34, scale=10.0)
    out, lse = _tree(B, c, qn, qp, _mask(seen, 16), None)
    _check_tree(c, qn, qp, out, lse, seen)


def test_tree_reports_bad_arguments(B):  # noqa: F811
    c = Cache([200, 200, 200, 200], seed=35)
    seen = [_seen_of(_random_tree(np.random.default_rng(b), 8)) for b in range(4)]
    qn, qp = _queries(4, 8, 16, seed=36)
    good = c.table.clone()
    for drafts, lens in (([8, -1, 8, 8], None), ([8, 9, 8, 8], None), ([8, 5, 8, 8], [200, 4, 200, 200]),
                         ([8] * 4, [200, -1, 200, 200]), ([8] * 4, [200, 10 ** 6, 200, 200])):
        out, lse = _tree(B, c, qn, qp, _mask(seen, 8), drafts, lens)
        assert B.latent_last_status() == B.DSA_ERR_RANGE
        assert torch.all(out[1] == 0) and torch.all(torch.isneginf(lse[1]))
        _check_tree(c, qn, qp, out, lse, seen, only=[0, 2, 3])
    c.table[2, 1] = c.P
    out, lse = _tree(B, c, qn, qp, _mask(seen, 8), [8] * 4)
    assert B.latent_last_status() == B.DSA_ERR_RANGE
    c.table = good
    _check_tree(c, qn, qp, out, lse, seen, only=[0, 1, 3])
    _tree(B, c, qn, qp, _mask(seen, 8), [8] * 4)
    assert B.latent_last_status() == 0


@pytest.mark.parametrize("nn,H", [(3, 16), (8, 16), (16, 128)])
def test_tree_wait_limit_ends_the_kernels(B, nn, H):  # noqa: F811
    """With a test option the first keys are never loaded, so that the waits for them (limit 50 ms here) run out: the
    call comes back, says so, and the next one is right."""
    c = Cache([3000, 500], seed=37)
    seen = [_seen_of(_random_tree(np.random.default_rng(b), nn)) for b in range(2)]
    qn, qp = _queries(2, nn, H, seed=38)
    B.set_option("wait_limit_us", 50000)
    B.set_option("test_withhold", 1)
    try:
        _tree(B, c, qn, qp, _mask(seen, nn), None)
        assert B.latent_last_status() == B.DSA_ERR_TIMEOUT
    finally:
        B.set_option("test_withhold", 0)
        B.set_option("wait_limit_us", 2000000)
    out, lse = _tree(B, c, qn, qp, _mask(seen, nn), None)
    assert B.latent_last_status() == 0
    _check_tree(c, qn, qp, out, lse, seen)


# ------------------------------------------------------------------ accept --
@pytest.mark.parametrize("seqs", [
    # (length, nodes, path) of each sequence
    [(10, 4, [0, 2])], [(70, 16, [0, 1, 2, 3]), (64, 1, [0]), (65, 2, [1]), (5, 0, []), (0, 0, []), (200, 7, [])],
    [(300, 200, list(range(0, 200, 2)))], [(300, 200, list(range(50, 200)))], [(129, 64, [63]), (1000, 64, [0, 5, 9, 33, 40, 63])],
    [(260, 130, [j for j in range(130) if j % 7 != 3])], [(40 + i, i, list(range(i // 2, i))) for i in range(1, 40)],
    [(100, 40, list(range(16, 40))), (100, 40, list(range(40)))]])
@pytest.mark.parametrize("indexer,joint,alias", [(False, False, False), (True, True, True)])
def test_accept_matches_oracle(B, seqs, indexer, joint, alias):  # noqa: F811
    lens = [a for a, _, _ in seqs]
    c = Cache(lens, seed=len(seqs), joint=joint)
    g = torch.Generator().manual_seed(40)
    kc = torch.randint(0, 256, (c.P, 64, 128), generator=g, dtype=torch.uint8)
    ks = torch.rand((c.P, 64), generator=g)
    width = max(1, max(len(p) for _, _, p in seqs)) + 2
    path = torch.full((len(seqs), width), -7, dtype=torch.int32)
    for b, (_, _, p) in enumerate(seqs):
        path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    ck, kp = c.device()
    dk, ds, dl = kc.cuda(), ks.cuda(), _ints(lens)
    new = B.latent_cache_accept(ck, kp, c.table.cuda(), dl, _ints([n for _, n, _ in seqs]), path.cuda(),
                                _ints([len(p) for _, _, p in seqs]), k_cache=dk if indexer else None,
                                k_cache_scale=ds if indexer else None, new_lens=dl if alias else None)
    assert B.latent_last_status() == 0 and (new is dl or not alias)
    assert new.tolist() == [a - n + len(p) for a, n, p in seqs]
    want = c.data.clone().view(torch.int16).reshape(-1, 576)
    old, wk, ws = want.clone(), kc.clone().reshape(-1, 128), ks.clone().reshape(-1)
    for b, (L, n, p) in enumerate(seqs):
        node = la.slots_of(c.table[b].numpy(), L)[L - n:]
        want[node[:len(p)]] = old[node[p]]
        if indexer:
            wk[node[:len(p)]], ws[node[:len(p)]] = kc.reshape(-1, 128)[node[p]], ks.reshape(-1)[node[p]]
    assert torch.equal(ck.cpu().contiguous().view(torch.int16).reshape(-1, 512), want[:, :512])
    assert torch.equal(kp.cpu().contiguous().view(torch.int16).reshape(-1, 64), want[:, 512:])
    assert torch.equal(dk.cpu().reshape(-1, 128), wk) and torch.equal(ds.cpu().reshape(-1), ws)


def test_accept_reports_and_leaves_what_is_no_path(B):  # noqa: F811
    c = Cache([200, 200, 200], seed=41)
    good = dict(lens=[200] * 3, drafts=[70] * 3, path=[[0, 3, 69]] * 3, plens=[3] * 3, table=c.table)
    bad_table = c.table.clone()
    bad_table[1, 3] = c.P  # the page of nodes 62 .. 69
    for change, moved, lens in [
            ({"path": [[0, 3, 69], [0, 3, 3], [0, 3, 69]]}, 0, 200), ({"path": [[0, 3, 69], [3, 0, 69], [0, 3, 69]]}, 0, 200),
            ({"path": [[0, 3, 69], [0, 3, 70], [0, 3, 69]]}, 0, 200), ({"path": [[0, 3, 69], [-1, 3, 69], [0, 3, 69]]}, 0, 200),
            ({"plens": [3, 4, 3]}, 0, 200), ({"plens": [3, -1, 3]}, 0, 200), ({"drafts": [70, 201, 70]}, 0, 200),
            ({"drafts": [70, -1, 70]}, 0, 200), ({"lens": [200, -1, 200]}, 0, -1), ({"lens": [200, 10 ** 6, 200]}, 0, 10 ** 6),
            ({"table": bad_table}, 2, 133)]:
        a = dict(good, **change)
        ck, kp = c.device()
        new = B.latent_cache_accept(ck, kp, a["table"].cuda(), _ints(a["lens"]), _ints(a["drafts"]), _ints(a["path"]),
                                    _ints(a["plens"]))
        assert B.latent_last_status() == B.DSA_ERR_RANGE and new.tolist() == [133, lens, 133], change
        want = c.data.clone().view(torch.int16).reshape(-1, 576)
        old = want.clone()
        for b, m in ((0, 3), (1, moved), (2, 3)):
            node = la.slots_of(c.table[b].numpy(), 200)[130:]
            want[node[:m]] = old[node[[0, 3, 69][:m]]]
        assert torch.equal(ck.cpu().contiguous().view(torch.int16).reshape(-1, 512), want[:, :512]), change
        assert torch.equal(kp.cpu().contiguous().view(torch.int16).reshape(-1, 64), want[:, 512:])
    ck, kp = c.device()
    B.latent_cache_accept(ck, kp, c.table.cuda(), _ints([200] * 3), _ints([70] * 3), _ints([[0, 3, 69]] * 3), _ints([3] * 3))
    assert B.latent_last_status() == 0


# ------------------------------------------------- streams, graphs, together --
def test_from_graphs_side_by_side_on_streams_of_their_own(B):  # noqa: F811
    """Encoding, appending, the tree and the path captured on two streams, replayed together with other contents, lengths
    and trees than they were captured with."""
    g = torch.Generator().manual_seed(50)
    table, nn, H = _table(), 8, 16
    runs = []
    for k in range(2):
        rng = np.random.default_rng(k)
        c = Cache([300, 70, 64], seed=51 + k)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        qn, qp = (x.cuda() for x in _queries(3, nn, H, seed=53 + k))
        ck, kp = c.device()
        x, pos = _normal(g, 24, 64, 128).cuda(), torch.zeros(24, dtype=torch.int32, device="cuda")
        new_c, new_pe = (t.cuda() for t in _tokens(g, 24, joint=False))
        st = dict(c=c, s=s, qn=qn, qp=qp, ck=ck, kp=kp, x=x, pos=pos, new_c=new_c, new_pe=new_pe, table=c.table.cuda(),
                  cs=table.cuda(), cu=_ints([0, 8, 16, 24]), before=_ints([0, 0, 0]), lens=_ints([8, 8, 8]), drafts=_ints([8, 8, 8]),
                  mask=_mask([_seen_of([-1] * nn)] * 3, nn).cuda(), path=_ints([[0] * nn] * 3), plens=_ints([1, 1, 1]),
                  codes=torch.empty((24, 64, 128), dtype=torch.uint8, device="cuda"), scale=torch.empty(24, device="cuda"),
                  out=torch.empty((3, nn, H, 512), dtype=BF16, device="cuda"), lse=torch.empty((3, nn, H), device="cuda"),
                  end=torch.empty(3, dtype=torch.int32, device="cuda"))

        def step(st=st):
            B.indexer_encode(st["x"], st["cs"], st["pos"], hadamard=True, codes=st["codes"], scale=st["scale"])
            B.latent_cache_append(st["new_c"], st["new_pe"], st["cs"], st["cu"], st["table"], st["before"], st["ck"],
                                  st["kp"], positions=st["pos"], new_lens=st["lens"])
            B.latent_attention_tree(st["qn"], st["qp"], st["ck"], st["kp"], st["table"], st["lens"], st["mask"], SCALE,
                                    draft_lens=st["drafts"], out=st["out"], lse=st["lse"])
            B.latent_cache_accept(st["ck"], st["kp"], st["table"], st["lens"], st["drafts"], st["path"], st["plens"],
                                  new_lens=st["end"])

        with torch.cuda.stream(s):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
        st["graph"] = graph
        # other contents: sequences of 300, 70 and 64 keys of which the tree's nodes are the last
        st["parents"] = [_random_tree(rng, n) for n in (8, 5, 8)]
        st["n"] = [8, 5, 8]
        st["seen"] = [_seen_of(p) for p in st["parents"]]
        st["paths"] = [sorted(st["seen"][b][int(rng.integers(0, st["n"][b]))]) for b in range(3)]
        for t, v in ((ck, c.data[..., :512]), (kp, c.data[..., 512:]), (st["mask"], _mask(st["seen"], nn)),
                     (st["cu"], _ints([0, 8, 13, 21])), (st["before"], _ints([292, 65, 56])), (st["drafts"], _ints(st["n"])),
                     (st["path"], _ints([p + [-1] * (nn - len(p)) for p in st["paths"]])),
                     (st["plens"], _ints([len(p) for p in st["paths"]])),
                     (pos, torch.randint(0, MAXPOS, (24,), generator=g, dtype=torch.int32))):
            t.copy_(v)
        runs.append(st)
    torch.cuda.synchronize()
    for _ in range(3):
        for st in runs:
            st["ck"].copy_(st["c"].data[..., :512])
            st["kp"].copy_(st["c"].data[..., 512:])
        torch.cuda.synchronize()
        for st in runs:
            with torch.cuda.stream(st["s"]):
                st["graph"].replay()
        torch.cuda.synchronize()
        for st in runs:
            assert B.latent_last_status(st["s"]) == 0
            c, d = st["c"], Cache([300, 70, 64], seed=1)
            cs = _np(table)[st["pos"].cpu().numpy()]
            check_codes(st["codes"], st["scale"], *te.index_rows(_np(st["x"]), cs, None, False, True))
            # the oracle's cache: as it was, with the nodes (rotated rope parts rounded to bf16) behind
            d.table, d.P, d.data = c.table, c.P, c.data.clone()
            rope = torch.from_numpy(te.rotate(_np(st["new_pe"]), cs, True)).to(BF16)
            at = 0
            for b, (L, n) in enumerate(zip(c.lens, st["n"])):
                slots = la.slots_of(c.table[b].numpy(), L)[L - n:]
                d.data.view(-1, 576)[slots] = torch.cat([st["new_c"].cpu()[at:at + n], rope[at:at + n]], 1)
                at += n
            _check_tree(d, st["qn"].cpu(), st["qp"].cpu(), st["out"], st["lse"], st["seen"])
            assert st["end"].tolist() == [L - n + len(p) for L, n, p in zip(c.lens, st["n"], st["paths"])]
            for b, (L, n, p) in enumerate(zip(c.lens, st["n"], st["paths"])):
                node = la.slots_of(c.table[b].numpy(), L)[L - n:]
                got = st["ck"].cpu().reshape(-1, 512)[node[:len(p)]]
                assert torch.equal(got, d.data.view(-1, 576)[node[p], :512])


def test_a_first_call_in_a_capture_leaves_it_whole(B):  # noqa: F811
    """The status of a stream is allocated by the first call on it, which a capture cannot hold."""
    x, pos, table = torch.zeros((4, 64, 128), dtype=BF16, device="cuda"), _ints([0, 1, 2, 3]), _table().cuda()
    codes, scale = torch.empty((4, 64, 128), dtype=torch.uint8, device="cuda"), torch.zeros(4, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    B.release()
    y = torch.zeros(3, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        with pytest.raises(B.IndexerError) as e:
            B.indexer_encode(x, table, pos, codes=codes, scale=scale)
        y.add_(1.0)
    assert e.value.code == B.DSA_ERR_CUDA
    g.replay()
    torch.cuda.synchronize()
    assert torch.all(y == 1.0) and torch.all(scale == 0.0)


def test_outputs_on_a_given_stream(B):  # noqa: F811
    """Outputs that a call makes for a stream that is not the current one lie in that stream's memory."""
    g = torch.Generator().manual_seed(55)
    x, pe, pos, table = _normal(g, 200, 64, 128).cuda(), _normal(g, 200, 16, 64).cuda(), _ints(range(200)), _table().cuda()
    want = B.indexer_encode(x, table, pos, pe=pe)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        for t in want:  # memory of the current stream that a slow kernel has yet to fill
            y = torch.empty_like(t)
            torch.cuda._sleep(2_000_000)
            y.view(torch.uint8).fill_(0x44)
            del y
        got = B.indexer_encode(x, table, pos, pe=pe, stream=s)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_a_drafted_step_as_a_server_runs_it(B):  # noqa: F811
    """Prompts and drafts appended, the indexer and the tree's attention over them, the accepted path kept: decode over
    what is left gives what the tree gave for the path, and the indexer's keys are those of the path."""
    from oracle import checks
    g, rng = torch.Generator().manual_seed(60), np.random.default_rng(60)
    prompts, nn, H, K = [200, 61, 130], 12, 16, 96
    nb, table = 3, _table()
    p = Pages([x + nn for x in prompts], seed=61)
    cs, bt = table.cuda(), p.table.cuda()
    cn, nm = (1 + 0.1 * torch.randn(512, generator=g), 1e-6), _norm(g)
    dcn, dnm = (cn[0].cuda(), cn[1]), (nm[0].cuda(), nm[1].cuda(), nm[2])
    opt = dict(c_norm=dcn, index_norm=dnm, hadamard=True, k_cache=p.kc, k_cache_scale=p.ks)
    lens = torch.zeros(nb, dtype=torch.int32, device="cuda")
    c, k_pe = _tokens(g, sum(prompts))
    ik = _normal(g, sum(prompts), 128)
    B.latent_cache_append(c.cuda(), k_pe.cuda(), cs, _ints(np.concatenate([[0], np.cumsum(prompts)])), bt, lens, p.ckv, p.kpe,
                          index_k=ik.cuda(), new_lens=lens, **opt)
    assert lens.tolist() == prompts
    # a tree behind every prompt: a node's position is its depth behind the prompt, not its slot
    parents = [_random_tree(rng, nn) for _ in range(nb)]
    seen = [_seen_of(t) for t in parents]
    pos = torch.tensor([[prompts[b] + len(s) - 1 for s in seen[b]] for b in range(nb)], dtype=torch.int32)
    c, k_pe, ik = *_tokens(g, nb * nn), _normal(g, nb * nn, 128)
    B.latent_cache_append(c.cuda(), k_pe.cuda(), cs, _ints([0, nn, 2 * nn, 3 * nn]), bt, lens, p.ckv, p.kpe, index_k=ik.cuda(),
                          positions=pos.view(-1).cuda(), new_lens=lens, **opt)
    q_nope, q_rope, xq = _normal(g, nb, nn, H, 512), _normal(g, nb, nn, H, 64), _normal(g, nb * nn, 64, 128)
    codes, scale, q_pe = B.indexer_encode(xq.cuda(), cs, pos.view(-1).cuda(), hadamard=True,
                                          pe=q_rope.cuda().view(nb * nn, H, 64))
    out, lse = B.latent_attention_tree(q_nope.cuda(), q_pe.view(nb, nn, H, 64), p.ckv, p.kpe, bt, lens,
                                       _mask(seen, nn).cuda(), SCALE)
    # a path to a leaf of each is accepted
    paths = [sorted(seen[b][nn - 1 - b]) for b in range(nb)]
    drafts = _ints([nn] * nb)
    B.latent_cache_accept(p.ckv, p.kpe, bt, lens, drafts, _ints([x + [-1] * (nn - len(x)) for x in paths]),
                          _ints([len(x) for x in paths]), k_cache=p.kc, k_cache_scale=p.ks, new_lens=lens)
    assert lens.tolist() == [a + len(x) for a, x in zip(prompts, paths)] and B.latent_last_status() == 0
    for b in range(nb):
        rows = paths[b]
        m = len(rows)
        sel = torch.tensor(rows, device="cuda")
        o, l = B.latent_attention_paged(q_nope[b:b + 1, rows].cuda(), q_pe.view(nb, nn, H, 64)[b:b + 1, sel].contiguous(),
                                        p.ckv, p.kpe, bt[b:b + 1], lens[b:b + 1], SCALE)
        # the same keys in the same order but for where tiles end: rounding apart, the same
        assert torch.allclose(o[0].float(), out[b, sel].float(), rtol=4 * BF, atol=4 * BF)
        assert torch.allclose(l[0], lse[b, sel], rtol=0, atol=1e-4)
        # the indexer's keys are those of the path, at their positions
        slots = torch.from_numpy(p.slots(b, prompts[b], m)).cuda()
        at = [b * nn + r for r in rows]
        y, reach = te.index_rows(_np(ik)[at][:, None], _np(table)[pos.view(-1).numpy()[at]], _np_norm(nm), False, True)
        check_codes(p.kc.view(-1, 128)[slots][:, None], p.ks.view(-1)[slots], y, reach)
    # the indexer over the cache, for the last accepted token of each
    last = torch.tensor([b * nn + paths[b][-1] for b in range(nb)], device="cuda")
    q, s, w = codes[last][:, None].contiguous(), scale[last][:, None].contiguous(), torch.randn((nb, 1, 64), generator=g)
    top = B.indexer_topk_paged(q, s, p.kc, p.ks, w.cuda(), bt, lens, K=K).cpu().numpy()
    o = indexer.PagedOracle(q.view(torch.uint8).cpu().numpy(), s.cpu().numpy(), p.kc.cpu().numpy(), p.ks.cpu().numpy(),
                            w.numpy(), p.table.numpy(), lens.cpu().numpy(), K)
    for b in range(nb):
        slots, scores, E = o.row_scores(b, 0)
        assert not checks.check_row(top[b, 0], slots, scores, E, K, order_key=np.arange(len(slots)))


@pytest.fixture(params=[1, 2, 7, 40])
def few_ctas(request, B):  # noqa: F811
    """The kernels' CTAs limited, so that each takes many tokens, items and pieces in turn."""
    B.set_option("grid_ctas", request.param)
    yield request.param
    B.set_option("grid_ctas", 0)  # the SM count again


@pytest.mark.parametrize("G,H,T,norm,had", [(64, 16, 40, False, True), (64, 100, 21, True, True), (64, 3, 33, False, False),
                                            (1, 1, 1500, True, True), (1, 2, 700, False, True), (1, None, 900, True, False)])
def test_encode_by_few_ctas(B, few_ctas, G, H, T, norm, had):  # noqa: F811
    g = torch.Generator().manual_seed(T)
    table, x, pe = _table(), _normal(g, T, G, 128), None if H is None else _normal(g, T, H, 64)
    pos = torch.randint(-MAXPOS // 4, MAXPOS, (T,), generator=g, dtype=torch.int32)  # some are padding
    nm = _norm(g) if norm else None
    codes, scale = torch.zeros((T, G, 128), dtype=torch.uint8, device="cuda"), torch.full((T,), -1.0, device="cuda")
    out = None if H is None else torch.full((T, H, 64), 5.0, dtype=BF16, device="cuda")
    B.indexer_encode(x.cuda(), table.cuda(), pos.cuda(), norm=None if nm is None else (nm[0].cuda(), nm[1].cuda(), nm[2]),
                     hadamard=had, pe=None if H is None else pe.cuda(), codes=codes, scale=scale, pe_out=out)
    assert B.latent_last_status() == 0
    keep = (pos >= 0).numpy()
    kd = torch.from_numpy(keep).cuda()
    cs = _np(table)[pos.numpy()[keep]]
    y, reach = te.index_rows(_np(x)[keep], cs, _np_norm(nm), False, had)
    check_codes(codes[kd], scale[kd], y, reach)
    assert torch.all(codes[~kd] == 0) and torch.all(scale[~kd] == -1.0)
    if H is not None:
        check_rope(out[kd], _np(pe)[keep], cs[:, None], True)
        assert torch.all(out[~kd] == 5.0)


@pytest.mark.parametrize("index", [False, True])
def test_append_by_few_ctas(B, few_ctas, index):  # noqa: F811
    g = torch.Generator().manual_seed(70)
    new, lens, table = [130, 0, 1, 600, 33, 64], [3, 9, 63, 0, 200, 64], _table()
    T = sum(new) + 5
    p = Pages([a + b for a, b in zip(new, lens)], seed=71, joint=index)
    c, k_pe = _tokens(g, T)
    cu, cn, nm, ix = np.concatenate([[0], np.cumsum(new)]), (torch.rand(512, generator=g), 1e-6), _norm(g), _normal(g, T, 128)
    dl = _ints(lens)
    B.latent_cache_append(c.cuda().contiguous(), k_pe.cuda().contiguous(), table.cuda(), _ints(cu), p.table.cuda(), dl, p.ckv,
                          p.kpe, c_norm=(cn[0].cuda(), cn[1]), index_k=ix.cuda() if index else None,
                          index_norm=(nm[0].cuda(), nm[1].cuda(), nm[2]) if index else None, hadamard=index,
                          k_cache=p.kc if index else None, k_cache_scale=p.ks if index else None, new_lens=dl)
    assert B.latent_last_status() == 0 and dl.tolist() == [a + b for a, b in zip(new, lens)]
    check_appended(p, cu, lens, c, k_pe, table, cn, index=(ix, nm, False, True) if index else None)


@pytest.mark.parametrize("nn,H,seqs", [
    (8, 16, [(1500, 8), (9, 8), (130, 3), (0, 0), (700, 8), (64, 8)]), (20, 16, [(300, 20), (2000, 11), (20, 20), (128, 1)]),
    (65, 3, [(500, 65), (65, 65), (190, 64)]), (3, 16, [(400, 3), (2, 2), (65, 3)])])
def test_tree_by_few_ctas(B, few_ctas, nn, H, seqs):  # noqa: F811
    """Runs of many items and pieces: whole items, cut ones, and ones that start and end in a run."""
    rng = np.random.default_rng(few_ctas + nn)
    lens, drafts = [a for a, _ in seqs], [n for _, n in seqs]
    c = Cache(lens, seed=nn)
    seen = [_seen_of(_random_tree(rng, n)) for n in drafts]
    qn, qp = _queries(len(lens), nn, H, seed=H)
    for b, n in enumerate(drafts):
        qn[b, n:] = float("nan")
    out, lse = _tree(B, c, qn, qp, _mask(seen, nn), drafts)
    assert B.latent_last_status() == 0
    _check_tree(c, qn, qp, out, lse, seen)


def test_binding_refuses_what_does_not_fit(B):  # noqa: F811
    """Wrong types, shapes, strides and combinations: an exception, and nothing is written."""
    def z(*shape, dtype=BF16):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    i32 = dict(dtype=torch.int32)
    table, pos = z(100, 64, dtype=torch.float32), z(4, **i32)
    x, pe = z(4, 64, 128), z(4, 16, 64)
    norm = z(128, dtype=torch.float32), z(128, dtype=torch.float32), 1e-6
    ckv, kpe, kc, ks = z(3, 64, 512), z(3, 64, 64), z(3, 64, 128, dtype=torch.uint8), z(3, 64, dtype=torch.float32)
    bt, lens, cu = z(2, 2, **i32), z(2, **i32), z(3, **i32)
    c, kp, ik = z(4, 512), z(4, 64), z(4, 128)
    cn = z(512, dtype=torch.float32), 1e-6
    qn, qp, mask = z(2, 3, 16, 512), z(2, 3, 16, 64), z(2, 3, 1, dtype=torch.int64)
    path, n2 = z(2, 5, **i32), z(2, **i32)
    bad = [
        lambda: B.indexer_encode(z(4, 2, 128), table, pos), lambda: B.indexer_encode(z(5, 64, 128), table, pos),
        lambda: B.indexer_encode(x.float(), table, pos), lambda: B.indexer_encode(x, table.double(), pos),
        lambda: B.indexer_encode(x, z(100, 32, dtype=torch.float32), pos), lambda: B.indexer_encode(x, table, pos.long()),
        lambda: B.indexer_encode(x, table, pos, norm=(norm[0][:64], norm[1], 1e-6)),
        lambda: B.indexer_encode(x, table, pos, norm=(norm[0], norm[1], -1.0)),
        lambda: B.indexer_encode(None, table, pos), lambda: B.indexer_encode(None, table, pos, pe=pe, norm=norm),
        lambda: B.indexer_encode(x, table, pos, pe_out=pe), lambda: B.indexer_encode(x, table, pos, pe=pe[..., :32]),
        lambda: B.indexer_encode(x, table, pos, pe=z(4, 16, 128)[..., ::2]),
        lambda: B.indexer_encode(x, table, pos, pe=z(4, 16, 68)[..., :64]),       # head stride no multiple of 8
        lambda: B.indexer_encode(x, table, pos, pe=z(4, 1, 64).expand(4, 16, 64)),  # head stride 0
        lambda: B.indexer_encode(x, table, pos, pe=z(4, 16, 72)[..., 4:68]),       # not 16-byte aligned
        lambda: B.indexer_encode(x, table, pos, codes=z(4, 64, 64, dtype=torch.uint8)),
        lambda: B.indexer_encode(x, table, pos, scale=z(5, dtype=torch.float32)),
        lambda: B.indexer_encode(x[:0], table, pos[:0]), lambda: B.indexer_encode(x.cpu(), table, pos),
        lambda: B.latent_cache_append(c, kp[:3], table, cu, bt, lens, ckv, kpe),
        lambda: B.latent_cache_append(c, kp, table, cu[:2], bt, lens, ckv, kpe),
        lambda: B.latent_cache_append(c, kp, table, cu, bt, lens[:1], ckv, kpe),
        lambda: B.latent_cache_append(c, kp, table, cu, bt, lens, ckv[:2], kpe),
        lambda: B.latent_cache_append(c, kp, table, cu, bt, lens, ckv, kpe, index_k=ik),
        lambda: B.latent_cache_append(c, kp, table, cu, bt, lens, ckv, kpe, k_cache=kc, k_cache_scale=ks),
        lambda: B.latent_cache_append(c, kp, table, cu, bt, lens, ckv, kpe, index_k=ik, k_cache=kc),
        lambda: B.latent_cache_append(c, kp, table, cu, bt, lens, ckv, kpe, index_norm=norm),
        lambda: B.latent_cache_append(c, kp, table, cu, bt, lens, ckv, kpe, c_norm=(cn[0][:128], 1e-6)),
        lambda: B.latent_cache_append(c, kp, table, cu, bt, lens, ckv, kpe, positions=pos[:3]),
        lambda: B.latent_cache_append(c, kp, table, cu, bt, lens, ckv, kpe, c_out=z(4, 576)),
        lambda: B.latent_cache_append(c, kp, table, cu, bt, lens, ckv, kpe, new_lens=z(3, **i32)),
        lambda: B.latent_cache_append(z(1, 512).expand(4, 512), kp, table, cu, bt, lens, ckv, kpe),
        lambda: B.latent_attention_tree(qn, qp, ckv, kpe, bt, lens, z(2, 3, 2, dtype=torch.int64), SCALE),
        lambda: B.latent_attention_tree(qn, qp, ckv, kpe, bt, lens, mask.int(), SCALE),
        lambda: B.latent_attention_tree(qn, qp[:, :2], ckv, kpe, bt, lens, mask, SCALE),
        lambda: B.latent_attention_tree(qn[0], qp, ckv, kpe, bt, lens, mask, SCALE),
        lambda: B.latent_attention_tree(qn, qp, ckv, kpe, bt[:1], lens, mask, SCALE),
        lambda: B.latent_attention_tree(qn, qp, ckv, kpe, bt, lens, mask, 0.0),
        lambda: B.latent_attention_tree(qn, qp, ckv, kpe, bt, lens, mask, SCALE, draft_lens=n2[:1]),
        lambda: B.latent_attention_tree(qn, qp, ckv, kpe, bt, lens, mask, SCALE, out=qn.float()),
        lambda: B.latent_attention_tree(qn.transpose(1, 2), qp, ckv, kpe, bt, lens, mask, SCALE),
        lambda: B.latent_cache_accept(ckv, kpe, bt, lens, n2, path[0], n2),
        lambda: B.latent_cache_accept(ckv, kpe, bt, lens, n2, path[:, :0], n2),
        lambda: B.latent_cache_accept(ckv, kpe, bt, lens, n2, path.long(), n2),
        lambda: B.latent_cache_accept(ckv, kpe, bt, lens, n2[:1], path, n2),
        lambda: B.latent_cache_accept(ckv, kpe, bt, lens, n2, path, n2, k_cache=kc),
        lambda: B.latent_cache_accept(ckv, kpe, bt, lens, n2, path, n2, k_cache=kc[:2], k_cache_scale=ks),
        lambda: B.latent_cache_accept(ckv, kpe, bt, lens, n2, path.t(), n2)]
    before = B.launch_count()
    for k, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError, B.IndexerError)):
            call()
            pytest.fail(f"call {k} was taken")
    assert B.launch_count() == before


def test_example_runs(B):  # noqa: F811
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_tree.py")
    spec = importlib.util.spec_from_file_location("draft_tree", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    said = []
    lens, out, lse, chosen, status = m.main(say=said.append)
    assert status == 0 and len(said) == 6 and all(n > p for n, p in zip(lens, (300, 61, 700)))
    assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(lse).all())
    for b, n in enumerate(lens):
        row = chosen[b, 0].tolist()
        assert sum(c >= 0 for c in row) == min(128, n) and len(set(c for c in row if c >= 0)) == min(128, n)
