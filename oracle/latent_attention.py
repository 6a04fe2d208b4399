"""Latent attention and cache eviction in float64 (test infrastructure only:
the oracle of the CUDA latent-attention operators).

Definitions:

  absorbed form   u_s = sm_scale log2(e) (q_nope . ckv[s] + q_pe . kpe[s]);
                  lse = log2(sum_s 2^u_s); out = sum_s 2^(u_s - lse) ckv[s];
                  token i of next_n sees the first len - next_n + i + 1 keys
  shared prefix   every row sees the prefix keys, then its own sequence's
  tree            node i of a sequence's last n keys sees the keys before them
                  and the nodes named for it
  key weights     sum over the rows that see key s of 2^(u_s - lse)
  expanded form   the same softmax over keys (k_nope[s, h] | k_pe[s]) and
                  values v[s, h]; query i of n sees the first m - n + i + 1 of
                  m keys with the causal mask
  eviction        of L > budget keys the last `recent` and the budget - recent
                  others with the largest weights (ties: the lowest index; NaN
                  above everything), in index order

A row that sees no key has out = 0 and lse = -inf.  Next to each output the
magnitude sum_s p_s |value_s| and the largest sum_d |q_d k_d| of its row are
returned: what rounding errors are relative to.
"""
from __future__ import annotations

import math

import numpy as np

LOG2E = 1.0 / math.log(2.0)
PAGE = 64


def rows_over_keys(q, k, v, visible, sm_scale):
    """q [R, D], k [N, D], v [N, E] float64, visible [R] keys from the first on, or [R, N]
    truth values: (out [R, E], lse [R], p [R, N], magnitude [R, E], spread [R])."""
    R, N = q.shape[0], k.shape[0]
    if N == 0:
        e = np.zeros((R, v.shape[1]))
        return e, np.full(R, -np.inf), np.zeros((R, 0)), e, np.zeros(R)
    visible = np.asarray(visible)
    see = visible if visible.ndim == 2 else np.arange(N)[None, :] < visible[:, None]
    u = np.where(see, (q @ k.T) * (sm_scale * LOG2E), -np.inf)
    m = np.where(see.any(1), u.max(1), 0.0)
    e = np.exp2(u - m[:, None])
    total = e.sum(1)
    p = e / np.where(total > 0, total, 1.0)[:, None]
    with np.errstate(divide="ignore"):
        lse = np.where(total > 0, m + np.log2(total), -np.inf)
    spread = np.where(see, np.abs(q) @ np.abs(k).T, 0.0).max(1) * (sm_scale * LOG2E)
    return p @ v, lse, p, p @ np.abs(v), spread


def slots_of(table, length):
    s = np.arange(length)
    return np.asarray(table, np.int64)[s // PAGE] * PAGE + s % PAGE


def decode(q_nope, q_pe, ckv, kpe, block_table, seq_lens, sm_scale, prefix_table=None, prefix_len=0):
    """Per sequence: (out [nn H, 512], lse, p [nn H, prefix + len], magnitude, spread).
    Arrays are float64 (q [B, nn, H, .], caches flat over slots)."""
    B, nn, H, _ = q_nope.shape
    res = []
    for b in range(B):
        L = int(seq_lens[b])
        slots = slots_of(block_table[b], L)
        if prefix_table is not None:
            slots = np.concatenate([slots_of(prefix_table, prefix_len), slots])
        v = ckv[slots]
        k = np.concatenate([v, kpe[slots]], 1)
        q = np.concatenate([q_nope[b], q_pe[b]], -1).reshape(nn * H, -1)
        sees = prefix_len + np.repeat(np.maximum(0, L - nn + 1 + np.arange(nn)), H)
        res.append(rows_over_keys(q, k, v, sees, sm_scale))
    return res


def tree(q_nope, q_pe, ckv, kpe, block_table, seq_lens, seen, sm_scale):
    """decode() for drafted nodes: seen[b] is the list of sets of nodes that each node of sequence b sees
    (its last len(seen[b]) keys); queries behind them see nothing."""
    B, nn, H, _ = q_nope.shape
    res = []
    for b in range(B):
        L, n = int(seq_lens[b]), len(seen[b])
        slots = slots_of(block_table[b], L)
        v = ckv[slots]
        k = np.concatenate([v, kpe[slots]], 1)
        q = np.concatenate([q_nope[b], q_pe[b]], -1).reshape(nn * H, -1)
        sees = np.zeros((nn, L), bool)
        for i, s in enumerate(seen[b]):
            sees[i, :L - n] = True
            sees[i, [L - n + j for j in s]] = True
        hidden = ~sees.any(0)  # what nobody sees may hold anything
        v[hidden], k[hidden] = 0.0, 0.0
        res.append(rows_over_keys(q, k, v, np.repeat(sees, H, 0), sm_scale))
    return res


def kept_keys(weights, length, budget, recent):
    """Old indices, ascending, of the keys a sequence keeps."""
    if length <= budget:
        return np.arange(length)
    cand = length - recent
    w = np.asarray(weights[:cand], np.float64)
    rank = np.where(np.isnan(w), np.inf, w)
    order = np.lexsort((np.arange(cand), -rank, ~np.isnan(w)))
    return np.concatenate([np.sort(order[:budget - recent]), np.arange(cand, length)]).astype(np.int64)
