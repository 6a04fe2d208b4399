"""What the latent operators promise around their results: the same bits from every run, waits that run out
and leave the cache alone, statuses of replayed graphs, streams, scratch and arguments of other types."""
import numpy as np
import pytest
import torch

from oracle import latent_attention as la
from test_gpu_latent import B, SCALE, Cache, _check_decode, _check_prefill, _ints, _prefill_inputs, _queries  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,qs,ks", [(16, [300, 1, 90, 700], [300, 129, 90, 1400]), (4, [2048], [4096])])
def test_prefill_repeats_bit_for_bit(B, H, qs, ks):  # noqa: F811
    """Copies, products and the softmax meet at barriers of both CTAs of a pair: no result may depend on who came first."""
    q, kv, kp, dev, cu = _prefill_inputs(qs, ks, H, seed=81, joint=True)
    first, lse1 = B.latent_attention_prefill(*dev, SCALE)
    runs = [B.latent_attention_prefill(*dev, SCALE) for _ in range(40)]
    assert B.latent_last_status() == 0
    for out, lse in runs:
        assert torch.equal(out.view(torch.int16), first.view(torch.int16))
        assert torch.equal(lse.view(torch.int32), lse1.view(torch.int32))
    if sum(ks) < 2000:
        _check_prefill(q, kv, kp, cu, first, lse1, True)
