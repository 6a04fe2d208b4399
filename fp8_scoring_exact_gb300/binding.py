"""Thin Python binding of libdsa_indexer.so (include/dsa_indexer.h).

Argument marshalling only: every step of the operator runs in the library's
CUDA kernels.  Tensors are torch CUDA tensors (FP8 data as uint8 or
torch.float8_e4m3fn); they are passed to the C ABI as raw device pointers
together with the current (or given) CUDA stream.  indexer_topk_host takes
CPU tensors instead (the library does the copies).  There is no CPU fallback:
if the library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None

DSA_OK, DSA_ERR_ARG, DSA_ERR_UNSUPPORTED, DSA_ERR_CUDA, DSA_ERR_TIMEOUT, DSA_ERR_RANGE = 0, -1, -2, -3, -4, -5
STATUS_NAMES = {0: "DSA_OK", -1: "DSA_ERR_ARG", -2: "DSA_ERR_UNSUPPORTED", -3: "DSA_ERR_CUDA",
                -4: "DSA_ERR_TIMEOUT", -5: "DSA_ERR_RANGE"}
OPTIONS = {"chunk_tiles": 1, "tau_bias": 2, "profile": 3, "grid_ctas": 4, "sample_target": 5,
           "host_chunk_rows": 6, "unit_order": 7, "wait_limit_us": 8, "test_withhold": 9,
           "matrix_row_min": 10}
HEADS, HEAD_DIM, MAX_K = 64, 128, 2048

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64

# C ABI signatures, name -> (restype, argtypes)
SIGNATURES = {
    "dsa_indexer_topk": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "dsa_indexer_topk_host": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "dsa_indexer_topk_paged": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P]),
    "dsa_indexer_topk_unfused": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "dsa_indexer_scores": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _P, _I64, _P]),
    "dsa_indexer_topk_from_scores": (_I, [_P, _I64, _P, _P, _I, _I, _I, _P, _P]),
    "dsa_indexer_topk_from_scores_noalloc": (_I, [_P, _I64, _P, _P, _I, _I, _I, _P, _P]),
    "dsa_indexer_math_control": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _P]),
    "dsa_sparse_attention": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P]),
    "dsa_sparse_attention_last_status": (_I, [_P]),
    "dsa_latent_attention_paged": (_I, [_P, _P, _P, _I64, _P, _I64, _P, _P, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P,
                                        _P, _I64, _P]),
    "dsa_latent_attention_shared_prefix": (_I, [_P, _P, _P, _I64, _P, _I64, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I,
                                                ctypes.c_float, _P, _P, _P]),
    "dsa_latent_attention_tree": (_I, [_P, _P, _P, _I64, _P, _I64, _P, _P, _P, _P, _I, _I, _I, _I, _I, ctypes.c_float,
                                       _P, _P, _P]),
    "dsa_indexer_encode": (_I, [_P, _I64, _I64, _I, _P, _P, ctypes.c_float, _P, _I64, _I64, _I, _P, _I, _P, _I, _I, _P,
                                _P, _P, _I64, _I64, _P]),
    "dsa_latent_cache_append": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, ctypes.c_float, _P, _P, ctypes.c_float, _P, _I,
                                     _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _I64, _P, _I64, _P, _P, _P, _I64, _P, _I64,
                                     _P, _P]),
    "dsa_latent_cache_accept": (_I, [_P, _I64, _P, _I64, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "dsa_latent_cache_evict": (_I, [_P, _I64, _P, _I64, _P, _P, _P, _I64, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P]),
    "dsa_latent_attention_prefill": (_I, [_P, _I64, _I64, _P, _I64, _I64, _P, _I64, _P, _I64, _I64, _P, _P, _I, _I, _I,
                                          _I, _I, ctypes.c_float, _P, _P, _P]),
    "dsa_latent_last_status": (_I, [_P]),
    "dsa_indexer_last_device_status": (_I, [_P, _P]),
    "dsa_indexer_last_repaired_rows": (_I, [_P, _P, _I]),
    "dsa_indexer_set_option": (_I, [_I, _I64]),
    "dsa_indexer_get_option": (_I64, [_I]),
    "dsa_indexer_profiled_main_ms": (ctypes.c_float, [_P]),
    "dsa_indexer_launch_count": (_I64, []),
    "dsa_indexer_version": (ctypes.c_char_p, []),
    "dsa_indexer_release": (_I, []),
}


class IndexerError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} returned {STATUS_NAMES.get(code, code)}")
        self.code = code


def library_path() -> str:
    return _build.LIB


def lib():
    """Load the library (building it first if the sources are newer)."""
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path) or not _build.up_to_date():
            _build.build()
        if not os.path.exists(path):
            raise RuntimeError(f"CUDA library {path} is missing; build it with "
                               "python -m fp8_scoring_exact_gb300.build")
        L = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _LIB = L
    return _LIB


def _check(fn, code):
    if code != DSA_OK:
        raise IndexerError(fn, code)


def _stream_ptr(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _u8(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype == torch.float8_e4m3fn:
        t = t.view(torch.uint8)
    if t.dtype != torch.uint8:
        raise TypeError(f"{name} must hold e4m3 codes (uint8 or float8_e4m3fn), got {t.dtype}")
    return _dev(t, name)


def _dev(t: torch.Tensor, name: str, dtype=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def indexer_topk(q, q_scale, k, k_scale, w, row_begin, row_end, K=2048, out=None, stream=None,
                 unfused=False):
    """Exact top-K indices per row; q [Q,64,128], k [N,128] e4m3; returns int32 [Q,K]."""
    q, k = _u8(q, "q"), _u8(k, "k")
    q_scale = _dev(q_scale, "q_scale", torch.float32)
    k_scale = _dev(k_scale, "k_scale", torch.float32)
    w = _dev(w, "w", torch.float32)
    row_begin = _dev(row_begin, "row_begin", torch.int32)
    row_end = _dev(row_end, "row_end", torch.int32)
    Q, N = q.shape[0], k.shape[0]
    if tuple(q.shape[1:]) != (HEADS, HEAD_DIM) or tuple(k.shape[1:]) != (HEAD_DIM,):
        raise ValueError("q must be [Q,64,128] and k [N,128]")
    if out is None:
        out = torch.empty((Q, K), dtype=torch.int32, device=q.device)
    _dev(out, "out", torch.int32)
    fn = "dsa_indexer_topk_unfused" if unfused else "dsa_indexer_topk"
    rc = getattr(lib(), fn)(_ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), _ptr(w), _ptr(row_begin),
                            _ptr(row_end), Q, N, K, _ptr(out), _stream_ptr(stream))
    _check(fn, rc)
    return out


def _host(t: torch.Tensor, name: str, dtype=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.is_cuda:
        raise TypeError(f"{name} must be a CPU tensor")
    if t.dtype == torch.float8_e4m3fn:
        t = t.view(torch.uint8)
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def indexer_topk_host(q, q_scale, k, k_scale, w, row_begin, row_end, K=2048, out=None, stream=None):
    """dsa_indexer_topk_host: the fused operator on CPU tensors (pinned memory lets the
    library overlap its copies with the scoring); returns int32 [Q,K] on the CPU.
    Synchronous."""
    q, k = _host(q, "q", torch.uint8), _host(k, "k", torch.uint8)
    q_scale = _host(q_scale, "q_scale", torch.float32)
    k_scale = _host(k_scale, "k_scale", torch.float32)
    w = _host(w, "w", torch.float32)
    row_begin = _host(row_begin, "row_begin", torch.int32)
    row_end = _host(row_end, "row_end", torch.int32)
    Q, N = q.shape[0], k.shape[0]
    if tuple(q.shape[1:]) != (HEADS, HEAD_DIM) or tuple(k.shape[1:]) != (HEAD_DIM,):
        raise ValueError("q must be [Q,64,128] and k [N,128]")
    if out is None:
        out = torch.empty((Q, K), dtype=torch.int32, pin_memory=q.is_pinned())
    _host(out, "out", torch.int32)
    rc = lib().dsa_indexer_topk_host(_ptr(q), _ptr(q_scale), _ptr(k), _ptr(k_scale), _ptr(w), _ptr(row_begin),
                                     _ptr(row_end), Q, N, K, _ptr(out), _stream_ptr(stream))
    _check("dsa_indexer_topk_host", rc)
    return out


def indexer_topk_unfused(*args, **kw):
    return indexer_topk(*args, unfused=True, **kw)


def indexer_topk_paged(q, q_scale, k_cache, k_cache_scale, w, block_table, seq_lens, K=2048, out=None,
                       stream=None):
    """Paged variant; q [B,next_n,64,128], k_cache [P,64,128]; returns int32 [B,next_n,K] of
    physical slots (block_table[b][s//64]*64 + s%64)."""
    q, k_cache = _u8(q, "q"), _u8(k_cache, "k_cache")
    q_scale = _dev(q_scale, "q_scale", torch.float32)
    k_cache_scale = _dev(k_cache_scale, "k_cache_scale", torch.float32)
    w = _dev(w, "w", torch.float32)
    block_table = _dev(block_table, "block_table", torch.int32)
    seq_lens = _dev(seq_lens, "seq_lens", torch.int32)
    B, nn = q.shape[0], q.shape[1]
    P = k_cache.shape[0]
    maxp = block_table.shape[1]
    if out is None:
        out = torch.empty((B, nn, K), dtype=torch.int32, device=q.device)
    _dev(out, "out", torch.int32)
    rc = lib().dsa_indexer_topk_paged(_ptr(q), _ptr(q_scale), _ptr(k_cache), _ptr(k_cache_scale), _ptr(w),
                                      _ptr(block_table), _ptr(seq_lens), B, nn, maxp, P, K, _ptr(out),
                                      _stream_ptr(stream))
    _check("dsa_indexer_topk_paged", rc)
    return out


def indexer_scores(q, q_scale, k, k_scale, w, row_begin, row_end, scores=None, stream=None):
    """FP32 scores [Q, ld] (valid entries of every row; -inf elsewhere in touched tiles)."""
    q, k = _u8(q, "q"), _u8(k, "k")
    Q, N = q.shape[0], k.shape[0]
    if scores is None:
        ld = (N + 3) // 4 * 4
        scores = torch.full((Q, ld), float("nan"), dtype=torch.float32, device=q.device)
    _dev(scores, "scores", torch.float32)
    rc = lib().dsa_indexer_scores(_ptr(q), _ptr(_dev(q_scale, "q_scale", torch.float32)), _ptr(k),
                                  _ptr(_dev(k_scale, "k_scale", torch.float32)),
                                  _ptr(_dev(w, "w", torch.float32)),
                                  _ptr(_dev(row_begin, "row_begin", torch.int32)),
                                  _ptr(_dev(row_end, "row_end", torch.int32)), Q, N, _ptr(scores),
                                  scores.shape[1], _stream_ptr(stream))
    _check("dsa_indexer_scores", rc)
    return scores


def topk_from_scores(scores, row_begin, row_end, K=2048, N=None, out=None, stream=None):
    """Exact top-K of each row of an fp32 score matrix over [row_begin, row_end)."""
    scores = _dev(scores, "scores", torch.float32)
    Q, ld = scores.shape
    N = ld if N is None else N
    if out is None:
        out = torch.empty((Q, K), dtype=torch.int32, device=scores.device)
    rc = lib().dsa_indexer_topk_from_scores(_ptr(scores), ld, _ptr(_dev(row_begin, "row_begin", torch.int32)),
                                            _ptr(_dev(row_end, "row_end", torch.int32)), Q, N, K,
                                            _ptr(_dev(out, "out", torch.int32)), _stream_ptr(stream))
    _check("dsa_indexer_topk_from_scores", rc)
    return out


def topk_from_scores_noalloc(scores, row_begin, row_end, K=2048, N=None, out=None, stream=None):
    """Same as topk_from_scores, through the entry point that allocates nothing
    (its scratch is a fixed array in device memory; at most 4096 rows).  The
    output tensor is the caller's: pass `out` to avoid even that allocation."""
    scores = _dev(scores, "scores", torch.float32)
    Q, ld = scores.shape
    N = ld if N is None else N
    if out is None:
        out = torch.empty((Q, K), dtype=torch.int32, device=scores.device)
    rc = lib().dsa_indexer_topk_from_scores_noalloc(_ptr(scores), ld,
                                                    _ptr(_dev(row_begin, "row_begin", torch.int32)),
                                                    _ptr(_dev(row_end, "row_end", torch.int32)), Q, N, K,
                                                    _ptr(_dev(out, "out", torch.int32)), _stream_ptr(stream))
    _check("dsa_indexer_topk_from_scores_noalloc", rc)
    return out


def math_control(q, q_scale, k, k_scale, w, row_begin, row_end, K=2048, checksum=None, stream=None):
    """The math-only control (a measurement): the fused call's main scorer with its
    score reduction and candidate filter removed.  Returns the checksum tensor
    (one device float, added to)."""
    q, k = _u8(q, "q"), _u8(k, "k")
    if checksum is None:
        checksum = torch.zeros(1, dtype=torch.float32, device=q.device)
    rc = lib().dsa_indexer_math_control(_ptr(q), _ptr(_dev(q_scale, "q_scale", torch.float32)), _ptr(k),
                                        _ptr(_dev(k_scale, "k_scale", torch.float32)),
                                        _ptr(_dev(w, "w", torch.float32)),
                                        _ptr(_dev(row_begin, "row_begin", torch.int32)),
                                        _ptr(_dev(row_end, "row_end", torch.int32)), q.shape[0], k.shape[0], K,
                                        _ptr(_dev(checksum, "checksum", torch.float32)), _stream_ptr(stream))
    _check("dsa_indexer_math_control", rc)
    return checksum


def sparse_attention(q_nope, q_pe, ckv, kpe, indices, sm_scale, out=None, lse=None, stream=None):
    """Sparse-attention decode over top-K slots: q_nope [T,H,512], q_pe [T,H,64] bf16,
    ckv [S,512], kpe [S,64] bf16 (slot-major cache), indices [T,K] int32 (-1: padding).
    Returns (out [T,H,512] bf16, lse [T,H] fp32, base 2)."""
    q_nope = _dev(q_nope, "q_nope", torch.bfloat16)
    q_pe = _dev(q_pe, "q_pe", torch.bfloat16)
    ckv = _dev(ckv, "ckv", torch.bfloat16)
    kpe = _dev(kpe, "kpe", torch.bfloat16)
    indices = _dev(indices, "indices", torch.int32)
    T, H = q_nope.shape[0], q_nope.shape[1]
    if tuple(q_nope.shape[2:]) != (512,) or tuple(q_pe.shape) != (T, H, 64):
        raise ValueError("q_nope must be [T,H,512] and q_pe [T,H,64]")
    ckv2, kpe2 = ckv.reshape(-1, 512), kpe.reshape(-1, 64)
    if ckv2.shape[0] != kpe2.shape[0]:
        raise ValueError("ckv and kpe must hold the same slots")
    K = indices.shape[-1]
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=q_nope.device)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=q_nope.device)
    rc = lib().dsa_sparse_attention(_ptr(q_nope), _ptr(q_pe), _ptr(ckv2), _ptr(kpe2), _ptr(indices), T, H, K,
                                    ckv2.shape[0], float(sm_scale), _ptr(_dev(out, "out", torch.bfloat16)),
                                    _ptr(_dev(lse, "lse", torch.float32)), _stream_ptr(stream))
    _check("dsa_sparse_attention", rc)
    return out, lse


def sparse_attention_last_status(stream=None) -> int:
    return int(lib().dsa_sparse_attention_last_status(_stream_ptr(stream)))


# ---------------------------------------------------------- latent attention --
# Scratch belongs to the stream of the call or of the capture: calls and replays that share one have to run one
# after the other (a graph that is to run beside others is captured on a stream of its own).
LATENT_DC, LATENT_DP, LATENT_DN, LATENT_DV = 512, 64, 128, 128
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _full(t, name, shape, dtype):
    """Address of a contiguous CUDA tensor of this shape and type."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous()):
        _dev(t, name, dtype)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _strided(t, name, dtype=_BF16):
    """Strides of a CUDA tensor whose last axis is contiguous; the others are the caller's."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    s = t.stride()
    if s[-1] != 1:
        raise ValueError(f"{name} must be contiguous in its last axis")
    return s


def _latent_stream(stream):
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()) if stream is None else stream.cuda_stream


def _new(shape, dtype, device, stream):
    """An output, in memory of the stream that writes it: memory of another one may still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):  # any object that names a stream will do
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _slot_stride(t, name, pages, d):
    s = _strided(t, name)
    if t.shape != (pages, 64, d):
        raise ValueError(f"{name} must be [P,64,{d}] with one P for both caches, got {list(t.shape)}")
    if pages > 1 and s[0] != 64 * s[1]:
        raise ValueError(f"{name}: slots must be evenly spaced (page stride 64 times the slot stride)")
    return s[1]


def _latent_cache(ckv, kpe):
    """(ckv, its slot stride, kpe, its slot stride), pages of a cache [P,64,512] and [P,64,64]; either
    may be part of a wider array (slots evenly spaced)."""
    pages = ckv.shape[0] if isinstance(ckv, torch.Tensor) and ckv.dim() else 0
    if (isinstance(ckv, torch.Tensor) and isinstance(kpe, torch.Tensor) and ckv.is_cuda and kpe.is_cuda and
            ckv.dtype is kpe.dtype is _BF16 and ckv.shape == (pages, 64, LATENT_DC) and
            kpe.shape == (pages, 64, LATENT_DP)):  # (nothing to refuse, in short)
        (a0, a1, a2), (b0, b1, b2) = ckv.stride(), kpe.stride()
        if a2 == b2 == 1 and a0 == 64 * a1 and b0 == 64 * b1:
            return (ckv.data_ptr(), a1, kpe.data_ptr(), b1), pages
    cs, ks = _slot_stride(ckv, "ckv_cache", pages, LATENT_DC), _slot_stride(kpe, "kpe_cache", pages, LATENT_DP)
    return (ckv.data_ptr(), cs, kpe.data_ptr(), ks), pages


def _latent_queries(q_nope, q_pe, out, lse, stream):
    rows = _dev(q_nope, "q_nope", _BF16).shape
    if len(rows) != 4 or rows[3] != LATENT_DC:
        raise ValueError(f"q_nope must be [B,next_n,H,512], got {list(rows)}")
    rows = rows[:3]
    queries = q_nope.data_ptr(), _full(q_pe, "q_pe", (*rows, LATENT_DP), _BF16)
    if out is None:
        out = _new((*rows, LATENT_DC), _BF16, q_nope.device, stream)
    else:
        _full(out, "out", (*rows, LATENT_DC), _BF16)
    if lse is None:
        lse = _new(rows, _F32, q_nope.device, stream)
    else:
        _full(lse, "lse", rows, _F32)
    return rows, queries, out, lse


def _tables(block_table, seq_lens, B):
    shape = _dev(block_table, "block_table", _I32).shape
    if len(shape) != 2 or shape[0] != B:
        raise ValueError(f"block_table must be [{B},max_pages], got {list(shape)}")
    return (block_table.data_ptr(), _full(seq_lens, "seq_lens", (B,), _I32)), shape[1]


def _key_weights(weights, B, max_pages):
    shape = _dev(weights, "weights", _F32).shape
    if len(shape) != 2 or shape[0] != B or shape[1] < 64 * max_pages:
        raise ValueError(f"weights must be [{B}, at least {64 * max_pages}], got {list(shape)}")
    return weights.data_ptr(), shape[1]


def latent_attention_paged(q_nope, q_pe, ckv_cache, kpe_cache, block_table, seq_lens, sm_scale, out=None, lse=None,
                           weights=None, stream=None):
    """Latent attention over a paged cache, absorbed form: q_nope [B,next_n,H,512], q_pe [B,next_n,H,64],
    ckv_cache [P,64,512], kpe_cache [P,64,64] bf16, block_table int32 [B,max_pages], seq_lens int32 [B];
    token i of sequence b sees its first seq_lens[b] - next_n + i + 1 keys.  Returns (out
    [B,next_n,H,512] bf16, lse [B,next_n,H] fp32, base 2).  weights fp32 [B, >= 64 max_pages]: the
    softmax weight of every key, summed over the sequence's rows, is added to it (at the cost of scratch
    that grows with the table's width: 256 B max_pages bytes per row of a sequence)."""
    rows, queries, out, lse = _latent_queries(q_nope, q_pe, out, lse, stream)
    cache, pages = _latent_cache(ckv_cache, kpe_cache)
    tables, maxp = _tables(block_table, seq_lens, rows[0])
    w, ldw = (None, 0) if weights is None else _key_weights(weights, rows[0], maxp)
    rc = lib().dsa_latent_attention_paged(*queries, *cache, *tables, *rows, maxp, pages, float(sm_scale),
                                          out.data_ptr(), lse.data_ptr(), w, ldw, _latent_stream(stream))
    _check("dsa_latent_attention_paged", rc)
    return out, lse


def latent_attention_shared_prefix(q_nope, q_pe, ckv_cache, kpe_cache, prefix_table, prefix_len, block_table, seq_lens,
                                   sm_scale, out=None, lse=None, stream=None):
    """latent_attention_paged for a batch that shares a prefix: every row also sees the prefix_len[0]
    keys behind prefix_table (int32 [prefix_pages]), which are read once for the whole batch; seq_lens
    counts a sequence's own keys."""
    rows, queries, out, lse = _latent_queries(q_nope, q_pe, out, lse, stream)
    cache, pages = _latent_cache(ckv_cache, kpe_cache)
    tables, maxp = _tables(block_table, seq_lens, rows[0])
    n = prefix_table.numel()
    rc = lib().dsa_latent_attention_shared_prefix(*queries, *cache, _full(prefix_table, "prefix_table", (n,), _I32),
                                                  _full(prefix_len, "prefix_len", (1,), _I32), n, *tables, *rows, maxp,
                                                  pages, float(sm_scale), out.data_ptr(), lse.data_ptr(),
                                                  _latent_stream(stream))
    _check("dsa_latent_attention_shared_prefix", rc)
    return out, lse


def _here(t, name, shape, dtype, dev):
    """Address of a contiguous tensor of this shape and type on the current device."""
    if (isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype is dtype and t.shape == shape and
            t.is_contiguous()):
        return t.data_ptr()
    raise _refusal(t, name, shape, dtype, dev)


def _refusal(t, name, shape, dtype, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        return ValueError(f"{name} is on device {t.get_device()}, the current one is {dev}")
    if t.dtype is not dtype:
        return TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        return ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return ValueError(f"{name} must be contiguous")


def _rows_here(t, name, shape, dev):
    """The same for bf16 rows contiguous in their last axis, with the strides of the other axes."""
    if isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype is _BF16 and t.shape == shape:
        *s, last = t.stride()
        if last == 1:
            return t.data_ptr(), *s
        raise ValueError(f"{name} must be contiguous in its last axis")
    raise _refusal(t, name, shape, _BF16, dev)


def _axes(t, name, layout):
    """Shape of a tensor of as many axes as `layout` names."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != layout.count(",") + 1:
        raise ValueError(f"{name} must be [{layout}], got {list(t.shape)}")
    return t.shape


def _current_device(t):
    """Index of the current device; `t`: some tensor of the call (without a CUDA tensor CUDA is not asked)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("tensors must be CUDA tensors")
    return torch._C._cuda_getDevice()


def _pages_here(ckv, kpe, block_table, seq_lens, dev):
    """((ckv, its slot stride, kpe, its slot stride), (block_table, seq_lens), (B, max_pages, pages))."""
    cache, pages = _latent_cache(ckv, kpe)
    if not ckv.get_device() == kpe.get_device() == dev:
        raise ValueError(f"the caches must be on the current device, {dev}")
    shape = _axes(block_table, "block_table", "B,max_pages")
    return (cache, (_here(block_table, "block_table", shape, _I32, dev),
                    _here(seq_lens, "seq_lens", shape[:1], _I32, dev)), (*shape, pages))


def _index_cache(k_cache, k_cache_scale, pages, dev):
    if k_cache is None and k_cache_scale is None:
        return None, None
    if k_cache is None or k_cache_scale is None:
        raise ValueError("k_cache and k_cache_scale go together")
    return (_codes_here(k_cache, "k_cache", (pages, 64, HEAD_DIM), dev),
            _here(k_cache_scale, "k_cache_scale", (pages, 64), _F32, dev))


def _codes_here(t, name, shape, dev):
    if isinstance(t, torch.Tensor) and t.dtype is torch.float8_e4m3fn:
        return _here(t, name, shape, torch.float8_e4m3fn, dev)
    return _here(t, name, shape, torch.uint8, dev)


def latent_attention_tree(q_nope, q_pe, ckv_cache, kpe_cache, block_table, seq_lens, tree_mask, sm_scale,
                          draft_lens=None, out=None, lse=None, stream=None):
    """latent_attention_paged for drafted tokens that form a tree: the last draft_lens[b] (int32 [B]; without it
    next_n, or all keys if there are fewer) of a sequence's keys are its nodes; query i sees the keys before them and
    node j where bit j % 64 of tree_mask[b, i, j // 64] is set (int64 [B, next_n, ceil(next_n / 64)]).  Queries past
    draft_lens[b] are padding: zeros and lse -inf.  A node that any query sees has to be finite.  No key weights."""
    dev = _current_device(q_nope)
    cache, tables, (B, maxp, pages) = _pages_here(ckv_cache, kpe_cache, block_table, seq_lens, dev)
    nn, H = _axes(q_nope, "q_nope", "B,next_n,H,512")[1:3]
    shape, rows = (B, nn, H, LATENT_DC), (B, nn, H)
    queries = _here(q_nope, "q_nope", shape, _BF16, dev), _here(q_pe, "q_pe", (B, nn, H, LATENT_DP), _BF16, dev)
    mask = _here(tree_mask, "tree_mask", (B, nn, (nn + 63) // 64), torch.int64, dev)
    drafts = None if draft_lens is None else _here(draft_lens, "draft_lens", (B,), _I32, dev)
    if out is None:
        out = _new(shape, _BF16, q_nope.device, stream)
    else:
        _here(out, "out", shape, _BF16, dev)
    if lse is None:
        lse = _new(rows, _F32, q_nope.device, stream)
    else:
        _here(lse, "lse", rows, _F32, dev)
    rc = lib().dsa_latent_attention_tree(*queries, *cache, *tables, mask, drafts, *rows, maxp, pages, float(sm_scale),
                                         out.data_ptr(), lse.data_ptr(), _latent_stream(stream))
    _check("dsa_latent_attention_tree", rc)
    return out, lse


def latent_cache_accept(ckv_cache, kpe_cache, block_table, seq_lens, draft_lens, path, path_lens, k_cache=None,
                        k_cache_scale=None, new_lens=None, stream=None):
    """Keeps the accepted path of every sequence's drafted nodes (its last draft_lens[b] keys): node path[b, j] (int32
    [B, max_path], ascending), j < path_lens[b], moves to the j-th place behind the keys before the nodes, with the
    indexer's keys and scales if given.  Returns new_lens int32 [B], which may be seq_lens itself."""
    dev = _current_device(ckv_cache)
    cache, tables, (B, maxp, pages) = _pages_here(ckv_cache, kpe_cache, block_table, seq_lens, dev)
    keys = _index_cache(k_cache, k_cache_scale, pages, dev)
    width = _axes(path, "path", "B,max_path")[1]
    nodes = _here(path, "path", (B, width), _I32, dev)
    if new_lens is None:
        new_lens = _new((B,), _I32, ckv_cache.device, stream)
    else:
        _here(new_lens, "new_lens", (B,), _I32, dev)
    rc = lib().dsa_latent_cache_accept(*cache, *keys, *tables, _here(draft_lens, "draft_lens", (B,), _I32, dev), nodes,
                                       _here(path_lens, "path_lens", (B,), _I32, dev), B, maxp, pages, width,
                                       new_lens.data_ptr(), _latent_stream(stream))
    _check("dsa_latent_cache_accept", rc)
    return new_lens


_ENCODE_PAIRS, _ENCODE_HADAMARD, _ENCODE_PE_HALVES = 1, 2, 4


def _encode_flags(interleaved, hadamard, pe_interleaved):
    return ((_ENCODE_PAIRS if interleaved else 0) | (_ENCODE_HADAMARD if hadamard else 0) |
            (0 if pe_interleaved else _ENCODE_PE_HALVES))


def _layer_norm(norm, name, dev):
    if norm is None:
        return None, None, 0.0
    weight, bias, eps = norm
    return (_here(weight, f"{name} weight", (HEAD_DIM,), _F32, dev), _here(bias, f"{name} bias", (HEAD_DIM,), _F32, dev),
            float(eps))


def _rotation_table(cos_sin, dev):
    n = _axes(cos_sin, "cos_sin", "max_positions,64")[0]
    return _here(cos_sin, "cos_sin", (n, LATENT_DP), _F32, dev), n


def indexer_encode(x, cos_sin, positions, norm=None, interleaved=False, hadamard=False, pe=None, pe_interleaved=True,
                   codes=None, scale=None, pe_out=None, stream=None):
    """Rows for the indexer from a projection's output x [T,64,128] (queries) or [T,1,128] (keys) bf16: LayerNorm with
    norm = (weight [128], bias [128], eps), the first 64 dims rotated by the angles of cos_sin [max_positions,64] fp32
    (32 cosines, 32 sines) at positions int32 [T] (negative: padding, left as it was), the Hadamard transform, e4m3
    codes with one scale a token.  pe [T,H,64] bf16 are rope parts of the same tokens, rotated to pe_out (which may be
    pe).  interleaved: pairs (2 i, 2 i + 1), else (i, i + 32).  Token and head strides are the caller's.  Returns (codes
    float8_e4m3fn [T,G,128], scale fp32 [T], pe_out or None); x may be None, and codes and scale are then too."""
    dev = _current_device(positions)
    T = positions.numel()
    at = _here(positions, "positions", (T,), _I32, dev)
    table, n = _rotation_table(cos_sin, dev)
    G = H = 1
    rows = parts = out = (None, 0, 0)
    to = (None, None)
    if x is not None:
        G = _axes(x, "x", "T,G,128")[1]
        if G != HEADS and G != 1:
            raise ValueError(f"x must be [T,64,128] or [T,1,128], got {list(x.shape)}")
        shape = (T, G, HEAD_DIM)
        rows = _rows_here(x, "x", shape, dev)
        if codes is None:
            codes = _new(shape, torch.float8_e4m3fn, x.device, stream)
        else:
            _codes_here(codes, "codes", shape, dev)
        if scale is None:
            scale = _new((T,), _F32, x.device, stream)
        else:
            _here(scale, "scale", (T,), _F32, dev)
        to = codes.data_ptr(), scale.data_ptr()
    elif norm is not None or codes is not None or scale is not None:
        raise ValueError("norm, codes and scale go with x")
    if pe is not None:
        H = _axes(pe, "pe", "T,H,64")[1]
        shape = (T, H, LATENT_DP)
        parts = _rows_here(pe, "pe", shape, dev)
        if pe_out is None:
            pe_out = _new(shape, _BF16, pe.device, stream)
            out = pe_out.data_ptr(), H * LATENT_DP, LATENT_DP
        else:
            out = _rows_here(pe_out, "pe_out", shape, dev)
    elif pe_out is not None:
        raise ValueError("pe_out goes with pe")
    rc = lib().dsa_indexer_encode(*rows, G, *_layer_norm(norm, "norm", dev), *parts, H, table, n, at, T,
                                  _encode_flags(interleaved, hadamard, pe_interleaved), *to, *out,
                                  _latent_stream(stream))
    _check("dsa_indexer_encode", rc)
    return codes, scale, pe_out


def latent_cache_append(c, k_pe, cos_sin, cu_new, block_table, seq_lens, ckv_cache, kpe_cache, c_norm=None,
                        pe_interleaved=True, index_k=None, index_norm=None, interleaved=False, hadamard=False,
                        k_cache=None, k_cache_scale=None, positions=None, c_out=None, k_pe_out=None, new_lens=None,
                        stream=None):
    """New tokens into the paged cache: tokens cu_new[b]..cu_new[b+1] (int32) of c [T,512] and k_pe [T,64] bf16 behind
    the seq_lens[b] keys of sequence b: c normalised with c_norm = (weight [512] fp32, eps), k_pe rotated, index_k
    [T,128] encoded as indexer_encode does (index_norm, interleaved, hadamard) into k_cache [P,64,128] and k_cache_scale
    [P,64].  positions int32 [T]: of the angles, by default a token's place in its sequence.  c_out and k_pe_out get
    what the cache gets.  Returns new_lens int32 [B], which may be seq_lens itself."""
    dev = _current_device(c)
    T = _axes(c, "c", "T,512")[0]
    rows, parts = _rows_here(c, "c", (T, LATENT_DC), dev), _rows_here(k_pe, "k_pe", (T, LATENT_DP), dev)
    cache, tables, (B, maxp, pages) = _pages_here(ckv_cache, kpe_cache, block_table, seq_lens, dev)
    keys = _index_cache(k_cache, k_cache_scale, pages, dev)
    if (index_k is None) != (k_cache is None):
        raise ValueError("index_k and k_cache go together")
    if index_k is None and index_norm is not None:
        raise ValueError("index_norm goes with index_k")
    index = (None, 0) if index_k is None else _rows_here(index_k, "index_k", (T, HEAD_DIM), dev)
    weight, eps = (None, 0.0) if c_norm is None else (_here(c_norm[0], "c_norm weight", (LATENT_DC,), _F32, dev),
                                                      float(c_norm[1]))
    table, n = _rotation_table(cos_sin, dev)
    if new_lens is None:
        new_lens = _new((B,), _I32, ckv_cache.device, stream)
    else:
        _here(new_lens, "new_lens", (B,), _I32, dev)
    rc = lib().dsa_latent_cache_append(
        *rows, *parts, *index, weight, eps, *_layer_norm(index_norm, "index_norm", dev), table, n,
        None if positions is None else _here(positions, "positions", (T,), _I32, dev),
        _here(cu_new, "cu_new", (B + 1,), _I32, dev), *tables, B, T, maxp, pages,
        _encode_flags(interleaved, hadamard, pe_interleaved), *cache, *keys,
        *((None, 0) if c_out is None else _rows_here(c_out, "c_out", (T, LATENT_DC), dev)),
        *((None, 0) if k_pe_out is None else _rows_here(k_pe_out, "k_pe_out", (T, LATENT_DP), dev)),
        new_lens.data_ptr(), _latent_stream(stream))
    _check("dsa_latent_cache_append", rc)
    return new_lens


def latent_cache_evict(ckv_cache, kpe_cache, weights, block_table, seq_lens, budget, recent, k_cache=None,
                       k_cache_scale=None, kept=None, new_lens=None, stream=None):
    """Cuts every sequence to `budget` keys in place: its last `recent` keys and the others with the
    largest weights (ties: the lowest index), in their old order, with their weights and, if given, the
    indexer's keys k_cache [P,64,128] and scales [P,64].  Returns (kept int32 [B,budget]: old indices,
    then -1; new_lens int32 [B], which may be seq_lens itself)."""
    cache, pages = _latent_cache(ckv_cache, kpe_cache)
    B = block_table.shape[0]
    tables, maxp = _tables(block_table, seq_lens, B)
    w, ldw = _key_weights(weights, B, maxp)
    if (k_cache is None) != (k_cache_scale is None):
        raise ValueError("k_cache and k_cache_scale go together")
    keys = (None, None)
    if k_cache is not None:
        keys = (_full(_u8(k_cache, "k_cache"), "k_cache", (pages, 64, HEAD_DIM), torch.uint8),
                _full(k_cache_scale, "k_cache_scale", (pages, 64), _F32))
    budget, recent = int(budget), int(recent)
    if kept is None:
        kept = _new((B, max(0, budget)), _I32, ckv_cache.device, stream)
    if new_lens is None:
        new_lens = _new((B,), _I32, ckv_cache.device, stream)
    rc = lib().dsa_latent_cache_evict(*cache, *keys, w, ldw, *tables, B, maxp, pages, budget, recent,
                                      _full(kept, "kept", (B, max(0, budget)), _I32),
                                      _full(new_lens, "new_lens", (B,), _I32), _latent_stream(stream))
    _check("dsa_latent_cache_evict", rc)
    return kept, new_lens


def latent_attention_prefill(q, k_nope, k_pe, v, cu_q, cu_k, sm_scale, causal=True, out=None, lse=None, stream=None):
    """Latent attention of a ragged batch, expanded form: q [Tq,H,192], k_nope and v [Tk,H,128] (token and
    head strides positive multiples of 8), k_pe [Tk,64] bf16; sequence z has queries cu_q[z]..cu_q[z+1] and
    keys cu_k[z]..cu_k[z+1] (int32), its last query sees all its keys.  Returns (out [Tq,H,128] bf16, lse
    [Tq,H] fp32, base 2)."""
    sq, sk, sp, sv = _strided(q, "q"), _strided(k_nope, "k_nope"), _strided(k_pe, "k_pe"), _strided(v, "v")
    if q.dim() != 3 or q.shape[2] != LATENT_DN + LATENT_DP:
        raise ValueError(f"q must be [Tq,H,192], got {list(q.shape)}")
    Tq, H = q.shape[:2]
    Tk = v.shape[0]
    if k_nope.shape != (Tk, H, LATENT_DN) or v.shape != (Tk, H, LATENT_DV):
        raise ValueError("k_nope and v must be [Tk,H,128]")
    if k_pe.shape != (Tk, LATENT_DP):
        raise ValueError("k_pe must be [Tk,64]")
    S = cu_q.numel() - 1
    cu = _full(cu_q, "cu_q", (S + 1,), _I32), _full(cu_k, "cu_k", (S + 1,), _I32)
    if out is None:
        out = _new((Tq, H, LATENT_DV), _BF16, q.device, stream)
    if lse is None:
        lse = _new((Tq, H), _F32, q.device, stream)
    rc = lib().dsa_latent_attention_prefill(q.data_ptr(), sq[0], sq[1], k_nope.data_ptr(), sk[0], sk[1],
                                            k_pe.data_ptr(), sp[0], v.data_ptr(), sv[0], sv[1], *cu, S, Tq, Tk, H,
                                            1 if causal else 0, float(sm_scale),
                                            _full(out, "out", (Tq, H, LATENT_DV), _BF16),
                                            _full(lse, "lse", (Tq, H), _F32), _latent_stream(stream))
    _check("dsa_latent_attention_prefill", rc)
    return out, lse


def latent_last_status(stream=None) -> int:
    return int(lib().dsa_latent_last_status(_stream_ptr(stream)))


def last_device_status(stream=None):
    """(status code, {underflow, overflow, trivial, candidates}) of the last call on the stream."""
    buf = (ctypes.c_int32 * 4)()
    rc = lib().dsa_indexer_last_device_status(_stream_ptr(stream), buf)
    return rc, {"underflow": buf[0], "overflow": buf[1], "trivial": buf[2], "candidates": buf[3]}


def last_repaired_rows(stream=None, cap=1 << 20):
    """Row ids the last selecting call on the stream sent to exact repair."""
    buf = (ctypes.c_int32 * cap)()
    n = lib().dsa_indexer_last_repaired_rows(_stream_ptr(stream), buf, cap)
    if n < 0:
        raise IndexerError("dsa_indexer_last_repaired_rows", n)
    return [buf[i] for i in range(min(n, cap))]


def set_option(name: str, value: int):
    _check("dsa_indexer_set_option", lib().dsa_indexer_set_option(OPTIONS[name], int(value)))


def get_option(name: str) -> int:
    return int(lib().dsa_indexer_get_option(OPTIONS[name]))


def profiled_main_ms(stream=None) -> float:
    return float(lib().dsa_indexer_profiled_main_ms(_stream_ptr(stream)))


def launch_count() -> int:
    return int(lib().dsa_indexer_launch_count())


def version() -> str:
    return lib().dsa_indexer_version().decode()


def release():
    _check("dsa_indexer_release", lib().dsa_indexer_release())
