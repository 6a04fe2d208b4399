"""Argument limits and host-side promises of the latent operators (CPU: a refused call returns before any CUDA
work)."""
import pytest

from fp8_scoring_exact_gb300 import binding as B
from test_latent_abi import EVICT, _call

UNSUPPORTED = B.DSA_ERR_UNSUPPORTED


@pytest.mark.parametrize("budget", [1 << 30, (1 << 31) - 64, (1 << 31) - 1])
def test_evict_refuses_a_budget_whose_indices_pass_32_bits(budget):
    """The kernels step through a list of `budget` entries in strides of up to 8192: from 2^31 - 8192 on an index
    would wrap to a negative one, and the count of 64-entry chunks as well."""
    assert _call("dsa_latent_cache_evict", EVICT, {"B": 1, "budget": budget}) == UNSUPPORTED
