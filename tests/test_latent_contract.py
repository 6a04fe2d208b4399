"""Argument limits and host-side promises of the latent operators (CPU: a refused call returns before any CUDA
work)."""
import numpy as np
import pytest
import torch

from fp8_scoring_exact_gb300 import binding as B
from oracle import latent_attention as la
from test_latent_abi import EVICT, _call

UNSUPPORTED = B.DSA_ERR_UNSUPPORTED


@pytest.mark.parametrize("budget", [1 << 30, (1 << 31) - 64, (1 << 31) - 1])
def test_evict_refuses_a_budget_whose_indices_pass_32_bits(budget):
    """The kernels step through a list of `budget` entries in strides of up to 8192: from 2^31 - 8192 on an index
    would wrap to a negative one, and the count of 64-entry chunks as well."""
    assert _call("dsa_latent_cache_evict", EVICT, {"B": 1, "budget": budget}) == UNSUPPORTED


# Errors of fp32 key weights and lse for N(0, 1) queries and keys (D = 576, scale 1 / sqrt(192)), on the average over
# keys and rows rather than at worst, from the kernel's arithmetic:
#   logits   a key's weight comes from rows whose logit is some 1.73 standard deviations (24) up, 41; it grows over 36
#            additions, kept in two accumulators of 18 where weights are wanted (partial sums of 250 in all, each), that
#            lose half a step of 2^-23 of the partial sum each: 3e-5, times scale / ln 2 ln 2 = 0.0722: 2.2e-6 of a
#            weight.  In one accumulator (partial sums of 1000 in all) 6e-5, times scale / ln 2 = 0.104: 6.2e-6 of lse
#   argument 2^-24 of up to 16 units from the fused multiply-add and 1.5 2^-24 of it from the rounded scale, times
#            ln 2: 0.7e-6 + 0.7e-6 of a weight; 2.4e-6 of lse with its own rounding
#   exponential and sums 0.2e-6
WEIGHT_RMS, LSE_RMS = 4e-6, 1e-5


def relative_rms(got, want):
    return float(np.sqrt(np.mean(((got - want) / want) ** 2)))


def check_weights(got, p):
    """Key weights against the float64 probabilities p [rows, keys]."""
    assert relative_rms(got, p.sum(0)) <= WEIGHT_RMS


def check_lse(got, want):
    assert float(np.sqrt(np.mean((got - want) ** 2))) <= LSE_RMS


@pytest.mark.parametrize("keys,rows", [(200, 16), (2100, 128), (30000, 16)])
def test_the_key_weight_check_notices_fewer_bits(keys, rows):
    """What the check has to reject: weights from bf16 probabilities, and ones a thousandth off."""
    rng = np.random.default_rng(keys)
    q, k = rng.standard_normal((rows, 576)), rng.standard_normal((keys, 576))
    _, lse, p, _, _ = la.rows_over_keys(q, k, k[:, :1], [keys] * rows, 1.0 / np.sqrt(192.0))
    check_weights(p.astype(np.float32).astype(np.float64).sum(0).astype(np.float32), p)
    check_lse(lse.astype(np.float32), lse)
    few = torch.from_numpy(p).to(torch.bfloat16).double().numpy()
    for bad in (few.sum(0), p.sum(0) * 1.001, p.sum(0) * 0.9999):
        with pytest.raises(AssertionError):
            check_weights(bad, p)
    for bad in (lse + 1e-4, lse * (1 + 2.0 ** -13), lse.astype(np.float16).astype(np.float64)):
        with pytest.raises(AssertionError):
            check_lse(bad, lse)
