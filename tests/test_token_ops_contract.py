"""Host-side promises of the operators that encode, append, verify and keep tokens (CPU: a refused call returns before
any CUDA work)."""
import pytest
import torch

from fp8_scoring_exact_gb300 import binding as B


@pytest.mark.parametrize("other", [None, 3, [1.0], "cache"])
def test_caches_that_are_no_tensors_are_a_type_error(other):
    """What is no tensor is refused as such, in the place of either cache."""
    t = torch.zeros((2, 64, 512), dtype=torch.bfloat16)
    for args in ((other, t), (t, other), (other, other)):
        with pytest.raises(TypeError):
            B._latent_cache(*args)
