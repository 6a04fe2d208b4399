"""Rows of new tokens in float64 (test infrastructure only: the oracle of the
CUDA operators that encode rows for the indexer and fill the latent cache).

Definitions:

  layer norm   (x - mean) / sqrt(mean (x - mean)^2 + eps) * weight + bias over the last axis
  RMS norm     x / sqrt(mean x^2 + eps) * weight
  rotation     of 64 dims by 32 angles: (a, b) -> (a cos - b sin, a sin + b cos),
               pairs (2 i, 2 i + 1) if interleaved, else (i, i + 32)
  Hadamard     y[d] = sum_e (-1)^popcount(d & e) x[e] / sqrt(n)
  codes        scale = max |y| / 448 over a token (1 where all are 0); the e4m3
               value nearest to y / scale, ties to the even code

Beside a row's values their `reach` is returned: the sum of the magnitudes that
were added up to form them, which rounding errors are relative to.
"""
from __future__ import annotations

import numpy as np

from . import e4m3


def layer_norm(x, weight, bias, eps):
    mean = x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    return (x - mean) * r * weight + bias, (np.abs(x) + np.abs(x).mean(-1, keepdims=True)) * r * np.abs(weight) + np.abs(bias)


def rms_norm(x, weight, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight


def rotate(x, cos_sin, interleaved):
    """x [..., 64], cos_sin [..., 64] (32 cosines, 32 sines) broadcast against it."""
    c, s = cos_sin[..., :32], cos_sin[..., 32:]
    out = np.empty(np.broadcast_shapes(x.shape, cos_sin.shape))
    first, second = (slice(0, 64, 2), slice(1, 64, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    a, b = x[..., first], x[..., second]
    out[..., first] = a * c - b * s
    out[..., second] = a * s + b * c
    return out


def hadamard(n):
    return np.array([[(-1.0) ** bin(d & e).count("1") for e in range(n)] for d in range(n)]) / np.sqrt(n)


def index_rows(x, cos_sin, norm, interleaved, had):
    """x [T, G, 128] float64, cos_sin [T, 64] -> (y, reach), both [T, G, 128]."""
    y, reach = layer_norm(x, *norm) if norm is not None else (x, np.abs(x))
    cs = cos_sin[:, None]
    y = np.concatenate([rotate(y[..., :64], cs, interleaved), y[..., 64:]], -1)
    # |a cos - b sin| <= |a| + |b|
    lo, hi = (slice(0, 64, 2), slice(1, 64, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    both = np.empty_like(reach[..., :64])
    both[..., lo] = both[..., hi] = reach[..., :64][..., lo] + reach[..., :64][..., hi]
    reach = np.concatenate([both, reach[..., 64:]], -1)
    if had:
        y = y @ hadamard(128)
        reach = np.broadcast_to(reach.sum(-1, keepdims=True) / np.sqrt(128.0), y.shape)
    return y, reach


def scales(y):
    top = np.abs(y).max(axis=tuple(range(1, y.ndim)))
    return np.where(top > 0, top / 448.0, 1.0)


_VALUES = e4m3.table_f64()


def nearest_codes(v):
    """The codes of the e4m3 values nearest to v (|v| <= 448), ties to the even code."""
    mags = _VALUES[:127]  # codes 0 .. 126 ascend
    a = np.abs(v)
    hi = np.clip(np.searchsorted(mags, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up = (a - mags[lo] > mags[hi] - a) | ((a - mags[lo] == mags[hi] - a) & (hi % 2 == 0))
    code = np.where((a == mags[hi]) | up, hi, lo)
    return (code | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def values(codes):
    return _VALUES[np.asarray(codes)]
