"""Argument checks of the latent-attention entry points (CPU: every refused
call returns before any CUDA work)."""
import ctypes

import pytest
import torch

from fp8_scoring_exact_gb300 import binding as B

P = ctypes.c_void_p
OK, MIS = P(0x1000), P(0x1002)  # never dereferenced: validation fails first
ARG, UNSUPPORTED = B.DSA_ERR_ARG, B.DSA_ERR_UNSUPPORTED


def _call(name, args, change):
    a = dict(args, **change)
    return getattr(B.lib(), name)(*a.values())


PAGED = dict(qn=OK, qp=OK, ckv=OK, cs=512, kpe=OK, ks=64, bt=OK, sl=OK, B=2, nn=1, H=16, mp=4, np=8, scale=0.1, out=OK,
             lse=OK, w=None, ldw=0, stream=None)
PREFIX = dict(qn=OK, qp=OK, ckv=OK, cs=512, kpe=OK, ks=64, pt=OK, pl=OK, pp=4, bt=OK, sl=OK, B=2, nn=1, H=16, mp=4,
              np=8, scale=0.1, out=OK, lse=OK, stream=None)
EVICT = dict(ckv=OK, cs=512, kpe=OK, ks=64, kc=None, kcs=None, w=OK, ldw=256, bt=OK, sl=OK, B=2, mp=4, np=8, budget=64,
             recent=8, kept=OK, nl=OK, stream=None)
PREFILL = dict(q=OK, qs=16 * 192, qh=192, kn=OK, kns=2048, knh=128, kp=OK, kps=64, v=OK, vs=2048, vh=128, cq=OK, ck=OK,
               S=1, Tq=8, Tk=8, H=16, causal=1, scale=0.1, out=OK, lse=OK, stream=None)


@pytest.mark.parametrize("change,code", [
    *[({k: None}, ARG) for k in ("qn", "qp", "ckv", "kpe", "bt", "sl", "out", "lse")],
    *[({k: MIS}, ARG) for k in ("qn", "qp", "ckv", "kpe", "out")],
    *[({k: v}, ARG) for k in ("B", "nn", "H", "mp", "np") for v in (0, -1)],
    ({"scale": 0.0}, ARG), ({"scale": -1.0}, ARG), ({"scale": float("nan")}, ARG), ({"scale": float("inf")}, ARG),
    ({"cs": 504}, ARG), ({"cs": 516}, ARG), ({"ks": 56}, ARG), ({"ks": 65}, ARG),
    ({"w": OK, "ldw": 255}, ARG),
    ({"B": 65536}, UNSUPPORTED), ({"np": 1 << 25}, UNSUPPORTED), ({"mp": 1 << 24}, UNSUPPORTED),
    ({"H": 1 << 25}, UNSUPPORTED), ({"H": 4097, "w": OK, "ldw": 256}, UNSUPPORTED)])
def test_paged_refusals(change, code):
    assert _call("dsa_latent_attention_paged", PAGED, change) == code


@pytest.mark.parametrize("change,code", [
    ({"pt": None}, ARG), ({"pl": None}, ARG), ({"pp": 0}, ARG), ({"pp": 1 << 24}, UNSUPPORTED), ({"qn": None}, ARG),
    ({"H": 0}, ARG), ({"scale": 0.0}, ARG)])
def test_prefix_refusals(change, code):
    assert _call("dsa_latent_attention_shared_prefix", PREFIX, change) == code


@pytest.mark.parametrize("change,code", [
    *[({k: None}, ARG) for k in ("ckv", "kpe", "w", "bt", "sl", "kept", "nl")],
    ({"kc": OK}, ARG), ({"kcs": OK}, ARG), ({"kc": MIS, "kcs": OK}, ARG), ({"ckv": MIS}, ARG),
    ({"budget": 0}, ARG), ({"recent": -1}, ARG), ({"recent": 65}, ARG), ({"ldw": 255}, ARG), ({"cs": 508}, ARG),
    ({"B": 0}, ARG), ({"B": 65536}, UNSUPPORTED), ({"mp": 1 << 24, "ldw": 1 << 30}, UNSUPPORTED)])
def test_evict_refusals(change, code):
    assert _call("dsa_latent_cache_evict", EVICT, change) == code


@pytest.mark.parametrize("change,code", [
    *[({k: None}, ARG) for k in ("q", "kn", "kp", "v", "cq", "ck", "out", "lse")],
    *[({k: MIS}, ARG) for k in ("q", "kn", "kp", "v", "out")],
    *[({k: 0}, ARG) for k in ("S", "Tq", "Tk", "H", "qs", "kns", "kps", "vs", "vh")],
    ({"qh": 100}, ARG), ({"vs": -8}, ARG), ({"scale": 0.0}, ARG), ({"S": 65536}, UNSUPPORTED),
    ({"Tq": 1 << 28}, UNSUPPORTED)])
def test_prefill_refusals(change, code):
    assert _call("dsa_latent_attention_prefill", PREFILL, change) == code


def test_binding_takes_cuda_tensors_only():
    t = torch.zeros((1, 1, 16, 512), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        B.latent_attention_paged(t, t, t, t, t, t, 0.1)
    with pytest.raises(TypeError):
        B.latent_attention_prefill(t[0], t[0], t[0], t[0], t, t, 0.1)
    with pytest.raises(TypeError):
        B.latent_cache_evict(t, t, t, t, t, 4, 1)
