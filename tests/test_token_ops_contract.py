"""Host-side promises of the operators that encode, append, verify and keep tokens (CPU: a refused call returns before
any CUDA work)."""
import pytest
import torch

from fp8_scoring_exact_gb300 import binding as B
from test_latent_abi import ARG, P, UNSUPPORTED, _call
from test_token_ops_abi import APPEND, ENCODE


@pytest.mark.parametrize("other", [None, 3, [1.0], "cache"])
def test_caches_that_are_no_tensors_are_a_type_error(other):
    """What is no tensor is refused as such, in the place of either cache."""
    t = torch.zeros((2, 64, 512), dtype=torch.bfloat16)
    for args in ((other, t), (t, other), (other, other)):
        with pytest.raises(TypeError):
            B._latent_cache(*args)


MANY = 1 << 30  # tokens: more than are supported, which is looked at behind the strides, so that nothing is launched


@pytest.mark.parametrize("T,H,token,head,code", [
    (MANY, 16, 1024, 64, UNSUPPORTED), (MANY, 16, 64, 64 << 30, UNSUPPORTED), (MANY, 16, 1032, 64, UNSUPPORTED),
    (MANY, 1, 64, 8, UNSUPPORTED), (MANY, 2, 192, 128, UNSUPPORTED), (1 << 20, 1 << 16, 64, 64 << 20, UNSUPPORTED),
    (MANY, 16, 1016, 64, ARG), (MANY, 16, 64, (64 << 30) - 8, ARG), (MANY, 16, 1024, 56, ARG), (MANY, 1, 56, 8, ARG),
    (MANY, 2, 184, 128, ARG), (1 << 20, 1 << 16, 64, (64 << 20) - 8, ARG), (1 << 20, 1 << 16, 56, 64 << 20, ARG),
    (4, 16, 64, 64, ARG), (4, 16, 64, 8, ARG), (4, 16, 8, 64, ARG), (1, 16, 8, 56, ARG), (4, 1, 56, 8, ARG),
    (4, (1 << 31) - 1, (1 << 37) - 128, 64, ARG)])
def test_encode_refuses_output_rows_that_share_memory(T, H, token, head, code):
    """Each would be written by several CTAs, in any order."""
    assert _call("dsa_indexer_encode", ENCODE, dict(T=T, H=H, pt=64, ph=64, ot=token, oh=head)) == code


@pytest.mark.parametrize("change", [{"co": P(0x2000), "cos": 504}, {"co": P(0x2000), "cos": 8}, {"ko": P(0x2000), "kos": 56}])
def test_append_refuses_dense_copies_that_share_memory(change):
    assert _call("dsa_latent_cache_append", APPEND, change) == ARG
