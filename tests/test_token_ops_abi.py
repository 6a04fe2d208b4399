"""Argument checks of the encoding, appending, tree and accepting entry points (CPU: every refused call returns
before any CUDA work)."""
import pytest
import torch

from fp8_scoring_exact_gb300 import binding as B
from test_latent_abi import ARG, MIS, OK, P, UNSUPPORTED, _call

ENCODE = dict(x=OK, xt=64 * 128, xh=128, G=64, nw=None, nb=None, eps=1e-6, pe=OK, pt=16 * 192, ph=192, H=16, cs=OK, mp=100,
              pos=OK, T=4, flags=0, codes=OK, scale=OK, po=P(0x2000), ot=1024, oh=64, stream=None)
APPEND = dict(c=OK, cs=576, kp=OK, kps=576, ik=OK, iks=128, cn=OK, ceps=1e-6, inw=OK, inb=OK, ieps=1e-6, rot=OK, mpos=100,
              pos=None, cu=OK, bt=OK, sl=OK, B=2, T=5, mp=4, np=8, flags=0, ckv=OK, ckvs=512, kpe=OK, kpes=64, kc=OK,
              kcs=OK, co=None, cos=0, ko=None, kos=0, nl=OK, stream=None)
TREE = dict(qn=OK, qp=OK, ckv=OK, cs=512, kpe=OK, ks=64, bt=OK, sl=OK, mask=OK, dl=None, B=2, nn=3, H=16, mp=4, np=8,
            scale=0.1, out=OK, lse=OK, stream=None)
ACCEPT = dict(ckv=OK, cs=512, kpe=OK, ks=64, kc=None, kcs=None, bt=OK, sl=OK, dl=OK, path=OK, pl=OK, B=2, mp=4, np=8,
              maxp=5, nl=OK, stream=None)
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("change,code", [
    *[({k: None}, ARG) for k in ("cs", "pos", "codes", "scale", "po", "x", "pe")],
    ({"x": None, "codes": None, "scale": None, "pe": None, "po": None}, ARG),
    *[({k: MIS}, ARG) for k in ("x", "pe", "cs", "codes", "po")],
    *[({k: v}, ARG) for k in ("T", "mp", "H") for v in (0, -1)],
    *[({"G": g}, ARG) for g in (0, 2, 63, 128, -1)],
    *[({k: v}, ARG) for k in ("xt", "xh", "pt", "ph", "ot", "oh") for v in (0, -8, 12, 1 << 38)],
    ({"nw": OK}, ARG), ({"nb": OK}, ARG), ({"nw": MIS, "nb": OK}, ARG), ({"nw": OK, "nb": MIS}, ARG),
    *[({"nw": OK, "nb": OK, "eps": e}, ARG) for e in (-1.0, NAN, INF)],
    ({"x": None, "codes": None, "scale": None, "nw": OK, "nb": OK}, ARG),
    ({"flags": 8}, ARG), ({"flags": -1}, ARG), ({"po": OK}, ARG), ({"T": 1 << 30}, UNSUPPORTED)])
def test_encode_refusals(change, code):
    assert _call("dsa_indexer_encode", ENCODE, change) == code


@pytest.mark.parametrize("change,code", [
    *[({k: None}, ARG) for k in ("c", "kp", "ik", "kc", "kcs", "rot", "cu", "bt", "sl", "ckv", "kpe", "nl", "inw", "inb")],
    *[({k: MIS}, ARG) for k in ("c", "kp", "ik", "cn", "inw", "inb", "rot", "ckv", "kpe", "kc", "co", "ko")],
    *[({k: v}, ARG) for k in ("B", "T", "mp", "np", "mpos") for v in (0, -1)],
    *[({k: v}, ARG) for k in ("cs", "kps", "iks") for v in (0, -8, 12)],
    ({"ckvs": 504}, ARG), ({"ckvs": 516}, ARG), ({"kpes": 56}, ARG), ({"kpes": 65}, ARG),
    ({"ik": None, "kc": None, "kcs": None}, ARG),  # (a norm of what is not there)
    *[({k: e}, ARG) for k in ("ceps", "ieps") for e in (-1.0, NAN, INF)],
    ({"co": OK, "cos": 512}, ARG), ({"ko": OK, "kos": 64}, ARG),  # in place with other strides
    ({"co": P(0x2000), "cos": 0}, ARG), ({"ko": P(0x2000), "kos": 4}, ARG),
    ({"flags": 8}, ARG), ({"mp": 1 << 24}, UNSUPPORTED), ({"np": 1 << 25}, UNSUPPORTED), ({"B": 65536}, UNSUPPORTED),
    ({"T": 1 << 30}, UNSUPPORTED)])
def test_append_refusals(change, code):
    assert _call("dsa_latent_cache_append", APPEND, change) == code


@pytest.mark.parametrize("change,code", [
    *[({k: None}, ARG) for k in ("qn", "qp", "ckv", "kpe", "bt", "sl", "mask", "out", "lse")],
    *[({k: MIS}, ARG) for k in ("qn", "qp", "ckv", "kpe", "mask", "out")],
    *[({k: v}, ARG) for k in ("B", "nn", "H", "mp", "np") for v in (0, -1)],
    ({"scale": 0.0}, ARG), ({"scale": NAN}, ARG), ({"cs": 504}, ARG), ({"ks": 65}, ARG),
    ({"B": 65536}, UNSUPPORTED), ({"nn": 65536}, UNSUPPORTED), ({"H": 1 << 25}, UNSUPPORTED),
    ({"mp": 1 << 24}, UNSUPPORTED), ({"np": 1 << 25}, UNSUPPORTED)])
def test_tree_refusals(change, code):
    assert _call("dsa_latent_attention_tree", TREE, change) == code


@pytest.mark.parametrize("change,code", [
    *[({k: None}, ARG) for k in ("ckv", "kpe", "bt", "sl", "dl", "path", "pl", "nl")],
    ({"kc": OK}, ARG), ({"kcs": OK}, ARG), ({"kc": MIS, "kcs": OK}, ARG), ({"ckv": MIS}, ARG), ({"kpe": MIS}, ARG),
    *[({k: v}, ARG) for k in ("B", "mp", "np", "maxp") for v in (0, -1)], ({"cs": 508}, ARG), ({"ks": 8}, ARG),
    ({"B": 65536}, UNSUPPORTED), ({"mp": 1 << 24}, UNSUPPORTED), ({"np": 1 << 25}, UNSUPPORTED),
    ({"maxp": 1 << 30}, UNSUPPORTED)])
def test_accept_refusals(change, code):
    assert _call("dsa_latent_cache_accept", ACCEPT, change) == code


def test_binding_takes_cuda_tensors_only():
    t, i = torch.zeros((1, 1, 16, 512), dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        B.latent_attention_tree(t, t, t, t, i, i, i, 0.1)
    with pytest.raises(TypeError):
        B.indexer_encode(t[0], t, i)
    with pytest.raises(TypeError):
        B.latent_cache_append(t[0, 0], t[0, 0], t, i, i, i, t, t)
    with pytest.raises(TypeError):
        B.latent_cache_accept(t, t, i[None], i, i, i[None], i)
