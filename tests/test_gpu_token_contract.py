"""What the operators that encode, append, verify and keep tokens promise at the ends of their arguments: borders that do
not ascend, norms of very large and very small rows, threads, releases, and more work than a grid has threads."""
import numpy as np
import pytest
import torch

from test_gpu_token_ops import B, BF16, MAXPOS, Pages, _ints, _normal, _np, _table, _tokens  # noqa: F401

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
