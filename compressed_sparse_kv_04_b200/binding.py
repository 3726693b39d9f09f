"""Thin binding of libcsa.so (include/csa.h), same entry-point names: ctypes, and
for the short calls of the 4-bit cache the native module _calls.

Argument marshalling only: every step runs in the library's CUDA kernels.
Tensors are torch tensors on the current CUDA device; the current torch
stream is passed as the `stream` argument.  Loading fails loudly when the
library has not been built: there is no CPU fallback.
"""
from __future__ import annotations

import ctypes as C
import math
import os

import torch

from . import build

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa.so")

CSA_OK = 0
STATUS_NAMES = {0: "CSA_OK", 1: "CSA_ERR_INVALID_ARG", 2: "CSA_ERR_UNSUPPORTED_SHAPE",
                3: "CSA_ERR_CAPACITY", 4: "CSA_ERR_WORKSPACE", 5: "CSA_ERR_CUDA",
                6: "CSA_ERR_DEVICE_TIMEOUT", 7: "CSA_ERR_DEVICE_INDEX"}
OP_INDEX_TOPK, OP_SPARSE_MQA, OP_DENSE_MQA, OP_PREFILL, OP_HCA_PREFILL = 1, 2, 3, 4, 5
OP_CSA_DECODE_STEP, OP_HCA_DECODE_STEP = 6, 7

EXPORTS = ["csa_version", "csa_last_error", "csa_workspace_bytes", "hca_compress",
           "csa_compress", "lightning_index_topk", "lightning_index_scores", "topk_select",
           "sparse_mqa_decode", "dense_mqa_decode", "csa_prefill_chunk",
           "lightning_index_topk_static", "csa_rope_yarn", "hca_prefill_chunk",
           "csa_decode_step", "hca_decode_step", "grouped_out_proj",
           "grouped_out_proj_workspace_bytes", "csa_shard_candidates", "csa_merge_candidates",
           "sparse_mqa_partials", "mqa_merge_partials", "csa_copy_async", "csa_copy_rows_async",
           "mxfp4_row_bytes", "mxfp4_cache_write", "mxfp4_cache_read", "hca_compress_mxfp4",
           "csa_compress_mxfp4", "sparse_mqa_decode_mxfp4", "dense_mqa_decode_mxfp4",
           "csa_prefill_chunk_mxfp4", "hca_prefill_chunk_mxfp4", "csa_decode_step_mxfp4",
           "hca_decode_step_mxfp4", "mxfp4_scale_bytes", "mxfp4_quantize",
           "grouped_out_proj_mxfp4", "grouped_out_proj_mxfp4_workspace_bytes"]
# Entry points that return a size, not a status.
_SIZES = ("csa_version", "csa_last_error", "csa_workspace_bytes",
          "grouped_out_proj_workspace_bytes", "mxfp4_row_bytes", "mxfp4_scale_bytes",
          "grouped_out_proj_mxfp4_workspace_bytes")


class CsaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class csa_params(C.Structure):
    _fields_ = [("B", C.c_int), ("d", C.c_int), ("H", C.c_int), ("H_I", C.c_int),
                ("D_I", C.c_int), ("k", C.c_int), ("window", C.c_int), ("rope_dim", C.c_int),
                ("m", C.c_int), ("eps", C.c_float), ("softmax_scale", C.c_float),
                ("rope_inv_freq", C.POINTER(C.c_double)), ("overlap", C.c_int),
                ("entry_offset", C.c_int64)]


_lib = None


def lib():
    """The loaded libcsa.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libcsa.so not found at {LIB_PATH}; build it with "
                               "`python -m compressed_sparse_kv_04_b200.build`")
        L = C.CDLL(LIB_PATH)
        _declare(L)
        _lib = L
    return _lib


_calls = None


def _native():
    """The native calls, on the loaded library's entry points."""
    global _calls
    if _calls is None:
        L = lib()
        try:
            from . import _calls as m
        except ImportError as e:
            raise RuntimeError("_calls.so not found or not loadable; build it with "
                               "`python -m compressed_sparse_kv_04_b200.build`") from e
        built_for = getattr(m, "built_for", "an unknown torch")
        if built_for != build.calls_tag():
            raise RuntimeError(f"_calls.so was built for {built_for}, this is "
                               f"{build.calls_tag()}; build it again with "
                               "`python -m compressed_sparse_kv_04_b200.build`")
        m.bind(*(C.cast(f, C.c_void_p).value for f in (
            L.mxfp4_row_bytes, L.mxfp4_cache_write, L.mxfp4_cache_read,
            L.sparse_mqa_decode_mxfp4, L.dense_mqa_decode_mxfp4, L.grouped_out_proj_mxfp4)))
        _calls = m
    return _calls


def _declare(L):
    vp, i32, i64, sz = C.c_void_p, C.c_int, C.c_int64, C.c_size_t
    P = C.POINTER(csa_params)
    L.csa_version.restype = i32
    L.csa_last_error.restype = C.c_char_p
    L.csa_workspace_bytes.argtypes = [P, i32, i32, i64]
    L.csa_workspace_bytes.restype = sz
    L.hca_compress.argtypes = [P, vp, i64, vp, vp, vp, vp, i64, i64, vp, i64, vp, vp]
    L.csa_compress.argtypes = [P, vp, i64, vp, vp, vp, vp, i64, i64, vp, i64, vp, vp, vp, vp,
                               vp, vp, vp]
    L.lightning_index_topk.argtypes = [P, i32, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp, sz,
                                       vp, vp]
    L.lightning_index_scores.argtypes = [P, i32, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp]
    L.topk_select.argtypes = [P, i32, vp, i64, vp, vp, vp, vp, vp]
    L.sparse_mqa_decode.argtypes = [P, vp, vp, vp, i64, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp,
                                    sz, vp, vp]
    L.dense_mqa_decode.argtypes = [P, vp, vp, vp, i64, vp, i64, vp, vp, vp, vp, vp, vp, sz, vp,
                                   vp]
    L.csa_prefill_chunk.argtypes = [P, i64, i32, vp, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp,
                                    i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    L.lightning_index_topk_static.argtypes = [P, i32, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp,
                                              vp]
    L.hca_prefill_chunk.argtypes = [P, i64, i32, vp, i64, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp,
                                    vp, vp, sz, vp, vp]
    L.csa_decode_step.argtypes = [P, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp, vp,
                                  vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    L.hca_decode_step.argtypes = [P, vp, vp, i64, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp, vp,
                                  sz, vp, vp]
    L.csa_rope_yarn.argtypes = [i32, C.c_double, C.c_double, C.c_double, C.c_double,
                                C.c_double, i32, C.POINTER(C.c_double), C.POINTER(C.c_double),
                                C.POINTER(C.c_float)]
    L.grouped_out_proj.argtypes = [i32, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp,
                                   vp]
    L.grouped_out_proj_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
    L.grouped_out_proj_workspace_bytes.restype = sz
    L.csa_shard_candidates.argtypes = [P, i32, vp, i64, vp, vp, vp, vp, vp, vp]
    L.csa_merge_candidates.argtypes = [P, i32, i32, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp]
    L.sparse_mqa_partials.argtypes = [P, i32, vp, vp, vp, i64, vp, vp, vp, i64, vp, vp, vp, vp,
                                      vp, vp]
    L.mqa_merge_partials.argtypes = [P, i32, vp, vp, vp, vp, vp, vp, vp, vp]
    L.csa_copy_async.argtypes = [vp, vp, sz, vp]
    L.csa_copy_rows_async.argtypes = [vp, sz, vp, sz, sz, sz, vp]
    # The calls on a 4-bit cache take the arguments of the bf16 ones.
    for name in EXPORTS:
        if name.endswith("_mxfp4") and name[:-6] in EXPORTS and name != "grouped_out_proj_mxfp4":
            getattr(L, name).argtypes = getattr(L, name[:-6]).argtypes
    L.mxfp4_row_bytes.argtypes = [i32]
    L.mxfp4_row_bytes.restype = sz
    L.mxfp4_cache_write.argtypes = [P, vp, i64, i64, vp, vp, vp, i64, vp, vp]
    L.mxfp4_cache_read.argtypes = [P, vp, i64, vp, vp, vp, i64, vp, vp, vp]
    L.mxfp4_scale_bytes.argtypes = [i64, i64]
    L.mxfp4_scale_bytes.restype = sz
    L.mxfp4_quantize.argtypes = [i64, i64, vp, i64, vp, vp, vp]
    L.grouped_out_proj_mxfp4_workspace_bytes.argtypes = [i32] * 6
    L.grouped_out_proj_mxfp4_workspace_bytes.restype = sz
    L.grouped_out_proj_mxfp4.argtypes = [i32] * 6 + [vp] * 8 + [sz, vp, vp]
    for name in EXPORTS:
        if name not in _SIZES:
            getattr(L, name).restype = i32


def make_params(B, d, H=0, H_I=0, D_I=0, k=0, window=0, rope_dim=0, m=4, eps=1e-6,
                softmax_scale=0.0, rope_inv_freq=None, overlap=0, entry_offset=0):
    p = csa_params(B, d, H, H_I, D_I, k, window, rope_dim, m, eps, softmax_scale, None, overlap,
                   entry_offset)
    if rope_inv_freq is not None:
        arr = (C.c_double * len(rope_inv_freq))(*rope_inv_freq)
        p.rope_inv_freq = C.cast(arr, C.POINTER(C.c_double))
        p._keep = arr
    return p


def params_for(w, B=None, **kw):
    """csa_params for a Workload (compressed_sparse_kv_04_b200.configs).  A
    workload with YaRN settings gets the library's YaRN frequency table and
    logit scale (csa_rope_yarn), unless the caller passes its own."""
    if w.yarn is not None and w.rope_dim > 0 and "rope_inv_freq" not in kw:
        tab, _, scale = rope_yarn(w.rope_dim, *w.yarn, d=w.d)
        kw["rope_inv_freq"] = tab
        kw.setdefault("softmax_scale", scale)
    kw.setdefault("overlap", w.overlap)
    return make_params(B or w.B, w.d, w.H, w.H_I, w.D_I, w.k, w.W, w.rope_dim, w.m, **kw)


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"expected a torch.Tensor, got {type(t)}")
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return C.c_void_p(t.data_ptr())


def _cache_ptr(p, kv_c):
    """Address of a bf16 cache [B, N_cap, d], which has to hold its entries' bytes
    (a 4-bit cache holds about a quarter of them: the calls would pass its end)."""
    need = p.B * kv_c.shape[1] * p.d * 2
    if kv_c.nbytes < need:
        raise ValueError(f"kv_c holds {kv_c.nbytes} bytes, {p.B} x {kv_c.shape[1]} bf16 entries of "
                         f"{p.d} take {need} (a 4-bit cache goes to the _mxfp4 calls)")
    return _ptr(kv_c)


def _weight_ptr(w, name, *shape):
    """Address of a bf16 weight, which has to hold that many values' bytes."""
    need = 2 * math.prod(shape)
    if w.nbytes < need:
        raise ValueError(f"{name} holds {w.nbytes} bytes, {list(shape)} in bf16 take {need} "
                         "(4-bit weights go to grouped_out_proj_mxfp4)")
    return _ptr(w)


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _check(status):
    if status != CSA_OK:
        raise CsaError(status, lib().csa_last_error().decode())


def version():
    return lib().csa_version()


def workspace_bytes(p, op, Q, N_cap):
    n = lib().csa_workspace_bytes(C.byref(p), op, Q, N_cap)
    if n == 0:
        raise CsaError(1, lib().csa_last_error().decode())
    return n


def workspace(p, op, Q, N_cap, device=None):
    """A zero-filled workspace (the decode step's score histogram starts
    cleared; each call leaves it so)."""
    return torch.zeros(workspace_bytes(p, op, Q, N_cap), dtype=torch.uint8,
                       device=torch.cuda.current_device() if device is None else device)


def hca_compress(p, kv_tok, ctx_len, w_s, b_pos, gamma, first_block, n_blocks, kv_c,
                 dev_status=None, stream=None):
    _check(lib().hca_compress(C.byref(p), _ptr(kv_tok), kv_tok.shape[1], _ptr(ctx_len),
                              _ptr(w_s), _ptr(b_pos), _ptr(gamma), first_block, n_blocks,
                              _cache_ptr(p, kv_c), kv_c.shape[1], _ptr(dev_status),
                              _stream(stream)))


def csa_compress(p, kv_tok, ctx_len, w_s, b_pos, gamma, first_block, n_blocks, kv_c,
                 idx_tok=None, w_s_idx=None, b_pos_idx=None, idx_key=None, idx_scale=None,
                 dev_status=None, stream=None):
    _check(lib().csa_compress(C.byref(p), _ptr(kv_tok), kv_tok.shape[1], _ptr(ctx_len),
                              _ptr(w_s), _ptr(b_pos), _ptr(gamma), first_block, n_blocks,
                              _cache_ptr(p, kv_c), kv_c.shape[1], _ptr(idx_tok), _ptr(w_s_idx),
                              _ptr(b_pos_idx), _ptr(idx_key), _ptr(idx_scale),
                              _ptr(dev_status), _stream(stream)))


def lightning_index_topk(p, Q, q_idx, q_scale, w, idx_key, idx_scale, pos_q, topk_idx,
                         topk_cnt, scores_out=None, ws=None, dev_status=None, stream=None):
    _check(lib().lightning_index_topk(
        C.byref(p), Q, _ptr(q_idx), _ptr(q_scale), _ptr(w), _ptr(idx_key), _ptr(idx_scale),
        idx_key.shape[1], _ptr(pos_q), _ptr(topk_idx), _ptr(topk_cnt), _ptr(scores_out),
        _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _ptr(dev_status),
        _stream(stream)))


def lightning_index_topk_static(p, Q, q_idx, q_scale, w, idx_key, idx_scale, pos_q, topk_idx,
                                topk_cnt, dev_status=None, stream=None):
    """lightning_index_topk with the scores in the library's own device array
    (no workspace; B*Q*N_cap <= 2**21)."""
    _check(lib().lightning_index_topk_static(
        C.byref(p), Q, _ptr(q_idx), _ptr(q_scale), _ptr(w), _ptr(idx_key), _ptr(idx_scale),
        idx_key.shape[1], _ptr(pos_q), _ptr(topk_idx), _ptr(topk_cnt), _ptr(dev_status),
        _stream(stream)))


def rope_yarn(rope_dim, factor, beta_fast, beta_slow, original_len, base=10000.0, d=1):
    """YaRN frequency table, logit gain and logit scale for head dim d (host
    only, computed by the library): returns (list of rope_dim/2 frequencies
    for make_params(rope_inv_freq=...), logit gain, softmax_scale)."""
    tab = (C.c_double * max(1, rope_dim // 2))()
    gain = C.c_double()
    scale = C.c_float()
    _check(lib().csa_rope_yarn(rope_dim, base, factor, beta_fast, beta_slow, original_len, d, tab,
                               C.byref(gain), C.byref(scale)))
    return list(tab)[: rope_dim // 2], gain.value, scale.value


def lightning_index_scores(p, Q, q_idx, q_scale, w, idx_key, idx_scale, pos_q, scores,
                           dev_status=None, stream=None):
    _check(lib().lightning_index_scores(
        C.byref(p), Q, _ptr(q_idx), _ptr(q_scale), _ptr(w), _ptr(idx_key), _ptr(idx_scale),
        idx_key.shape[1], _ptr(pos_q), _ptr(scores), _ptr(dev_status), _stream(stream)))


def topk_select(p, Q, scores, pos_q, topk_idx, topk_cnt, dev_status=None, stream=None):
    _check(lib().topk_select(C.byref(p), Q, _ptr(scores), scores.shape[-1], _ptr(pos_q),
                             _ptr(topk_idx), _ptr(topk_cnt), _ptr(dev_status), _stream(stream)))


def sparse_mqa_decode(p, q, pos_q, kv_c, topk_idx, topk_cnt, kv_tok, sink, out, gamma_q=None,
                      gamma_kv=None, lse=None, ws=None, dev_status=None, stream=None):
    _check(lib().sparse_mqa_decode(
        C.byref(p), _ptr(q), _ptr(pos_q), _cache_ptr(p, kv_c), kv_c.shape[1], _ptr(topk_idx),
        _ptr(topk_cnt), _ptr(kv_tok), kv_tok.shape[1], _ptr(sink), _ptr(gamma_q),
        _ptr(gamma_kv), _ptr(out), _ptr(lse), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _ptr(dev_status), _stream(stream)))


def dense_mqa_decode(p, q, pos_q, kv_c, kv_tok, sink, out, gamma_q=None, gamma_kv=None,
                     lse=None, ws=None, dev_status=None, stream=None):
    _check(lib().dense_mqa_decode(
        C.byref(p), _ptr(q), _ptr(pos_q), _cache_ptr(p, kv_c), kv_c.shape[1], _ptr(kv_tok),
        kv_tok.shape[1], _ptr(sink), _ptr(gamma_q), _ptr(gamma_kv), _ptr(out), _ptr(lse),
        _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _ptr(dev_status),
        _stream(stream)))


def csa_prefill_chunk(p, P, T, kv_tok, idx_tok, w_s, b_pos, gamma, w_s_idx, b_pos_idx, kv_c,
                      idx_key, idx_scale, q, q_idx, q_scale, w, sink, topk_idx, topk_cnt, out,
                      gamma_q=None, gamma_kv=None, ws=None, dev_status=None, stream=None):
    _check(lib().csa_prefill_chunk(
        C.byref(p), P, T, _ptr(kv_tok), _ptr(idx_tok), kv_tok.shape[1], _ptr(w_s), _ptr(b_pos),
        _ptr(gamma), _ptr(w_s_idx), _ptr(b_pos_idx), _cache_ptr(p, kv_c), _ptr(idx_key),
        _ptr(idx_scale), kv_c.shape[1], _ptr(q), _ptr(q_idx), _ptr(q_scale), _ptr(w), _ptr(sink),
        _ptr(gamma_q), _ptr(gamma_kv), _ptr(topk_idx), _ptr(topk_cnt), _ptr(out), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _ptr(dev_status), _stream(stream)))


def hca_prefill_chunk(p, P, T, kv_tok, w_s, b_pos, gamma, kv_c, q, sink, out, gamma_q=None,
                      gamma_kv=None, lse=None, ws=None, dev_status=None, stream=None):
    """HCA prefill chunk (B = 1): compression of the chunk's blocks, then dense
    MQA per new query.  kv_tok [1, L_cap, d]; kv_c [1, N_cap, d]; q/out [T, H, d]."""
    _check(lib().hca_prefill_chunk(
        C.byref(p), P, T, _ptr(kv_tok), kv_tok.shape[1], _ptr(w_s), _ptr(b_pos), _ptr(gamma),
        _cache_ptr(p, kv_c), kv_c.shape[1], _ptr(q), _ptr(sink), _ptr(gamma_q), _ptr(gamma_kv),
        _ptr(out), _ptr(lse), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
        _ptr(dev_status), _stream(stream)))


def csa_decode_step(p, pos_q, kv_tok, idx_tok, w_s, b_pos, gamma, w_s_idx, b_pos_idx, kv_c,
                    idx_key, idx_scale, q, q_idx, q_scale, w, sink, topk_idx, topk_cnt, out,
                    gamma_q=None, gamma_kv=None, lse=None, ws=None, dev_status=None, stream=None):
    """One CSA decode step (newest-block compression, indexer, top-k, sparse
    MQA) for B sequences at positions pos_q [B]."""
    _check(lib().csa_decode_step(
        C.byref(p), _ptr(pos_q), _ptr(kv_tok), _ptr(idx_tok), kv_tok.shape[1], _ptr(w_s),
        _ptr(b_pos), _ptr(gamma), _ptr(w_s_idx), _ptr(b_pos_idx), _cache_ptr(p, kv_c),
        _ptr(idx_key), _ptr(idx_scale), kv_c.shape[1], _ptr(q), _ptr(q_idx), _ptr(q_scale),
        _ptr(w), _ptr(sink), _ptr(gamma_q), _ptr(gamma_kv), _ptr(topk_idx), _ptr(topk_cnt),
        _ptr(out), _ptr(lse), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _ptr(dev_status),
        _stream(stream)))


class CsaDecodeStep:
    """csa_decode_step (or, with a 4-bit cache, csa_decode_step_mxfp4) for a
    fixed set of sequences: the arguments that stay the same from step to step
    (token buffers, caches, weights, sink and gains, the selection outputs,
    workspace and status word) are checked and converted once; each call
    passes the step's positions, queries and outputs.  Same C entry point and
    the same device-side work as the plain call (argument marshalling only)."""

    def __init__(self, p, kv_tok, idx_tok, w_s, b_pos, gamma, w_s_idx, b_pos_idx, kv_c, idx_key,
                 idx_scale, sink, topk_idx, topk_cnt, ws, gamma_q=None, gamma_kv=None,
                 dev_status=None):
        mx = _is_mxfp4(p, kv_c, kv_tok)
        self._fn = lib().csa_decode_step_mxfp4 if mx else lib().csa_decode_step
        self._keep = (p, kv_tok, idx_tok, w_s, b_pos, gamma, w_s_idx, b_pos_idx, kv_c, idx_key,
                      idx_scale, sink, topk_idx, topk_cnt, ws, gamma_q, gamma_kv, dev_status)
        self._head = (C.byref(p),)
        self._mid = (_ptr(kv_tok), _ptr(idx_tok), kv_tok.shape[1], _ptr(w_s), _ptr(b_pos),
                     _ptr(gamma), _ptr(w_s_idx), _ptr(b_pos_idx),
                     _ptr(kv_c) if mx else _cache_ptr(p, kv_c), _ptr(idx_key), _ptr(idx_scale),
                     kv_c.shape[1])
        self._sink = (_ptr(sink), _ptr(gamma_q), _ptr(gamma_kv), _ptr(topk_idx), _ptr(topk_cnt))
        self._tail = (_ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_status))

    def _args(self, pos_q, q, q_idx, q_scale, w, out, lse, stream):
        return (*self._head, _ptr(pos_q), *self._mid, _ptr(q), _ptr(q_idx), _ptr(q_scale),
                _ptr(w), *self._sink, _ptr(out), _ptr(lse), *self._tail, _stream(stream))

    def __call__(self, pos_q, q, q_idx, q_scale, w, out, lse=None, stream=None):
        _check(self._fn(*self._args(pos_q, q, q_idx, q_scale, w, out, lse, stream)))

    def bind(self, pos_q, q, q_idx, q_scale, w, out, lse=None, stream=None):
        """The step with its per-step buffers fixed as well (a decode loop
        that writes each step's positions and queries into the same
        buffers): returns f() that runs one step on `stream`."""
        fn, args = self._fn, self._args(pos_q, q, q_idx, q_scale, w, out, lse, stream)
        keep = (self, pos_q, q, q_idx, q_scale, w, out, lse, stream)

        def run(_keep=keep):
            _check(fn(*args))
        return run


class HcaDecodeStep:
    """hca_decode_step (or, with a 4-bit cache, hca_decode_step_mxfp4) for a
    fixed set of sequences (see CsaDecodeStep)."""

    def __init__(self, p, kv_tok, w_s, b_pos, gamma, kv_c, sink, ws, gamma_q=None, gamma_kv=None,
                 dev_status=None):
        mx = _is_mxfp4(p, kv_c, kv_tok)
        self._fn = lib().hca_decode_step_mxfp4 if mx else lib().hca_decode_step
        self._keep = (p, kv_tok, w_s, b_pos, gamma, kv_c, sink, ws, gamma_q, gamma_kv, dev_status)
        self._head = (C.byref(p),)
        self._mid = (_ptr(kv_tok), kv_tok.shape[1], _ptr(w_s), _ptr(b_pos), _ptr(gamma),
                     _ptr(kv_c) if mx else _cache_ptr(p, kv_c), kv_c.shape[1])
        self._gains = (_ptr(sink), _ptr(gamma_q), _ptr(gamma_kv))
        self._tail = (_ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_status))

    def _args(self, pos_q, q, out, lse, stream):
        return (*self._head, _ptr(pos_q), *self._mid, _ptr(q), *self._gains, _ptr(out),
                _ptr(lse), *self._tail, _stream(stream))

    def __call__(self, pos_q, q, out, lse=None, stream=None):
        _check(self._fn(*self._args(pos_q, q, out, lse, stream)))

    def bind(self, pos_q, q, out, lse=None, stream=None):
        """The step with its per-step buffers fixed (see CsaDecodeStep.bind)."""
        fn, args = self._fn, self._args(pos_q, q, out, lse, stream)
        keep = (self, pos_q, q, out, lse, stream)

        def run(_keep=keep):
            _check(fn(*args))
        return run


def _rows_of(t):
    """(rows, row_bytes, pitch_bytes) of a tensor whose first dimension
    strides over rows that are each contiguous."""
    if t.dim() == 0:
        return 1, t.element_size(), t.element_size()
    inner = t[0] if t.shape[0] > 0 else t
    if t.shape[0] > 0 and not inner.is_contiguous():
        raise ValueError("each row (first-dimension slice) must be contiguous")
    row = (t.numel() // max(1, t.shape[0])) * t.element_size()
    pitch = t.stride(0) * t.element_size() if t.shape[0] > 1 else row
    return t.shape[0], row, pitch


class PreparedCopy:
    """One asynchronous copy between two tensors of the same shape and dtype
    (page-locked host <-> device, either direction) with its addresses and
    stream fixed: csa_copy_async when both are contiguous, else
    csa_copy_rows_async over the first dimension (each row contiguous, e.g.
    kv_tok[:, pos:pos+1] of a [B, L_cap, d] token buffer).  f() enqueues it."""

    def __init__(self, dst, src, stream=None):
        if dst.shape != src.shape or dst.dtype != src.dtype:
            raise ValueError(f"copy between {tuple(src.shape)} {src.dtype} and "
                             f"{tuple(dst.shape)} {dst.dtype}")
        for t in (dst, src):
            if not t.is_cuda and not t.is_pinned():
                raise ValueError("host tensors of a prepared copy must be page-locked")
        self._keep = (dst, src, stream)
        L = lib()
        st = _stream(stream)
        if dst.is_contiguous() and src.is_contiguous():
            fn = L.csa_copy_async
            args = (C.c_void_p(dst.data_ptr()), C.c_void_p(src.data_ptr()),
                    dst.numel() * dst.element_size(), st)
        else:
            rows, row, dp = _rows_of(dst)
            _, srow, sp = _rows_of(src)
            fn = L.csa_copy_rows_async
            args = (C.c_void_p(dst.data_ptr()), dp, C.c_void_p(src.data_ptr()), sp, row, rows, st)
        self.bytes = dst.numel() * dst.element_size()
        self._fn, self._args = fn, args

    def __call__(self):
        _check(self._fn(*self._args))


def hca_decode_step(p, pos_q, kv_tok, w_s, b_pos, gamma, kv_c, q, sink, out, gamma_q=None,
                    gamma_kv=None, lse=None, ws=None, dev_status=None, stream=None):
    """One HCA decode step (newest-block compression, dense MQA) for B
    sequences at positions pos_q [B]."""
    _check(lib().hca_decode_step(
        C.byref(p), _ptr(pos_q), _ptr(kv_tok), kv_tok.shape[1], _ptr(w_s), _ptr(b_pos),
        _ptr(gamma), _cache_ptr(p, kv_c), kv_c.shape[1], _ptr(q), _ptr(sink), _ptr(gamma_q),
        _ptr(gamma_kv), _ptr(out), _ptr(lse), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _ptr(dev_status), _stream(stream)))


def grouped_out_proj_workspace_bytes(T, H, D, g, d_g, d_model):
    n = lib().grouped_out_proj_workspace_bytes(T, H, D, g, d_g, d_model)
    if n == 0:
        raise CsaError(2, lib().csa_last_error().decode())
    return n


def grouped_out_proj(o, w_g, w_o, z, y=None, ws=None, dev_status=None, stream=None):
    """Grouped output projection: o [T, H, D] -> y [T, g*d_g] -> z [T, d_model]
    (w_g [g, d_g, H/g*D], w_o [d_model, g*d_g], all bf16).  The workspace is
    allocated here when not given."""
    T, H, D = o.shape
    g, d_g, _ = w_g.shape
    d_model = w_o.shape[0]
    if ws is None:
        ws = torch.empty(grouped_out_proj_workspace_bytes(T, H, D, g, d_g, d_model),
                         dtype=torch.uint8, device=o.device)
    _check(lib().grouped_out_proj(T, H, D, g, d_g, d_model, _ptr(o),
                                  _weight_ptr(w_g, "w_g", g, d_g, H // max(g, 1) * D),
                                  _weight_ptr(w_o, "w_o", d_model, g * d_g), _ptr(y), _ptr(z),
                                  _ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_status),
                                  _stream(stream)))


# -------------------------------------------------------------- 4-bit (MXFP4) cache --
def mxfp4_row_bytes(d):
    """Bytes of a 4-bit cache row of d values (d/2 of codes, d/32 of scales,
    padded to 16)."""
    n = lib().mxfp4_row_bytes(d)
    if n == 0:
        raise CsaError(2, lib().csa_last_error().decode())
    return n


def mxfp4_cache(p, N_cap, device=None):
    """An empty (all zero) 4-bit cache [B, N_cap, row bytes] for these params."""
    return torch.zeros(p.B, N_cap, mxfp4_row_bytes(p.d), dtype=torch.uint8,
                       device=torch.cuda.current_device() if device is None else device)


_ROW_BYTES = {}
_Tensor = torch.Tensor


def _device():
    """The current CUDA device, which every tensor of a call has to be on; -2
    (no tensor's device) where there is none."""
    try:
        return torch._C._cuda_getDevice()
    except (AttributeError, RuntimeError):
        return -2


def _row_bytes(d):
    n = _ROW_BYTES.get(d)
    if n is None:
        n = _ROW_BYTES[d] = mxfp4_row_bytes(d)
    return n


def _need(dev, t, name, dtype, *shape):
    """Address of a tensor that must have this dtype and shape (None: any
    length), be contiguous and sit on the current device; None passes."""
    if t is None:
        return None
    # The usual case in few steps: a decode step makes a dozen of these checks.
    if (type(t) is _Tensor and t.dtype is dtype and t.shape == shape and t.is_contiguous() and
            t.get_device() == dev):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t)}")
    if t.dtype != dtype or t.dim() != len(shape) or any(
            n is not None and n != m for n, m in zip(shape, t.shape)):
        want = ", ".join("*" if n is None else str(n) for n in shape)
        raise ValueError(f"{name} must be {dtype} [{want}], not {t.dtype} {list(t.shape)}")
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on the current CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _size(t, name, dim):
    """Length of a dimension that the call itself reads."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t)}")
    if t.dim() <= dim:
        raise ValueError(f"{name} has {t.dim()} dimensions")
    return t.size(dim)


def _need_cache(dev, p, kv4):
    return _need(dev, kv4, "kv4", torch.uint8, p.B, _size(kv4, "kv4", 1), _row_bytes(p.d))


def _need_tok(dev, p, kv_tok):
    return _need(dev, kv_tok, "kv_tok", torch.bfloat16, p.B, _size(kv_tok, "kv_tok", 1), p.d)


def _status(dev, dev_status):
    return None if dev_status is None else _need(dev, dev_status, "dev_status", torch.int32, 1)


def _raw_stream(dev, stream):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(dev)


def _is_mxfp4(p, kv_c, kv_tok):
    """Whether a prepared step's cache is a 4-bit one: uint8 rows of that format's
    width (bytes of any other width are a bf16 cache's)."""
    if kv_c.dtype != torch.uint8 or kv_c.shape[-1] != lib().mxfp4_row_bytes(p.d):
        return False
    dev = _device()
    _need_cache(dev, p, kv_c)
    _need_tok(dev, p, kv_tok)
    return True


def _ws(dev, ws):
    """Address and bytes of a workspace (any type and shape, on the current
    device)."""
    if ws is None:
        return None, 0
    return _need(dev, ws, "ws", getattr(ws, "dtype", None), *getattr(ws, "shape", ())), ws.nbytes


def _empty(dev, stream, *shape):
    """uint8 memory that belongs to the stream of the call."""
    if stream is None:
        return torch.empty(*shape, dtype=torch.uint8, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(*shape, dtype=torch.uint8, device=dev)


def mxfp4_cache_write(p, rows, kv4, first_entry=None, count=None, dev_status=None, stream=None):
    """Quantises rows [B, n, d] (bf16; each sequence's rows contiguous) into
    entries first_entry[b] + i, i < count[b], of kv4."""
    st = (_calls or _native()).cache_write(p, rows, kv4, first_entry, count, dev_status, stream)
    if st:
        _check(st)


def mxfp4_cache_read(p, kv4, rows, idx=None, first_entry=None, count=None, dev_status=None,
                     stream=None):
    """The values of entries idx[b, i] (int32, -1 skipped) or first_entry[b] + i,
    i < count[b], of kv4 into rows [B, n, d] (bf16)."""
    st = (_calls or _native()).cache_read(p, kv4, rows, idx, first_entry, count, dev_status, stream)
    if st:
        _check(st)


def _pool_args(dev, p, w_s, b_pos, gamma):
    f32 = torch.float32
    return (_need(dev, w_s, "w_s", f32, p.d), _need(dev, b_pos, "b_pos", f32, p.m + p.overlap),
            _need(dev, gamma, "gamma", f32, p.d))


def _index_pool_args(dev, p, idx_tok, w_s_idx, b_pos_idx, idx_key, idx_scale, L_cap, N_cap):
    f32 = torch.float32
    return (_need(dev, idx_tok, "idx_tok", torch.bfloat16, p.B, L_cap, p.D_I),
            _need(dev, w_s_idx, "w_s_idx", f32, p.D_I),
            _need(dev, b_pos_idx, "b_pos_idx", f32, p.m + p.overlap),
            _need(dev, idx_key, "idx_key", torch.uint8, p.B, N_cap, p.D_I),
            _need(dev, idx_scale, "idx_scale", f32, p.B, N_cap))


def hca_compress_mxfp4(p, kv_tok, ctx_len, w_s, b_pos, gamma, first_block, n_blocks, kv4,
                       dev_status=None, stream=None):
    """hca_compress into a 4-bit cache."""
    dev = _device()
    _check(lib().hca_compress_mxfp4(
        C.byref(p), _need_tok(dev, p, kv_tok), kv_tok.shape[1],
        _need(dev, ctx_len, "ctx_len", torch.int64, p.B), *_pool_args(dev, p, w_s, b_pos, gamma),
        first_block,
        n_blocks, _need_cache(dev, p, kv4), kv4.shape[1], _status(dev, dev_status),
        _raw_stream(dev, stream)))


def csa_compress_mxfp4(p, kv_tok, ctx_len, w_s, b_pos, gamma, first_block, n_blocks, kv4,
                       idx_tok=None, w_s_idx=None, b_pos_idx=None, idx_key=None, idx_scale=None,
                       dev_status=None, stream=None):
    """csa_compress into a 4-bit cache (indexer keys as csa_compress)."""
    dev = _device()
    L, N = kv_tok.shape[1], kv4.shape[1]
    _check(lib().csa_compress_mxfp4(
        C.byref(p), _need_tok(dev, p, kv_tok), L,
        _need(dev, ctx_len, "ctx_len", torch.int64, p.B), *_pool_args(dev, p, w_s, b_pos, gamma),
        first_block,
        n_blocks, _need_cache(dev, p, kv4), N,
        *_index_pool_args(dev, p, idx_tok, w_s_idx, b_pos_idx, idx_key, idx_scale, L, N),
        _status(dev, dev_status), _raw_stream(dev, stream)))


def _mqa_inputs(dev, p, rows, q, kv4, kv_tok, sink, out, gamma_q, gamma_kv, lse):
    """Checked pointers of the attention's tensors, `rows` queries."""
    bf, f32 = torch.bfloat16, torch.float32
    return dict(q=_need(dev, q, "q", bf, rows, p.H, p.d), kv4=_need_cache(dev, p, kv4),
                kv_tok=_need_tok(dev, p, kv_tok),
                sink=_need(dev, sink, "sink", f32, p.H),
                gq=_need(dev, gamma_q, "gamma_q", f32, p.d),
                gkv=_need(dev, gamma_kv, "gamma_kv", f32, p.d),
                out=_need(dev, out, "out", bf, rows, p.H, p.d),
                lse=_need(dev, lse, "lse", f32, rows, p.H))


def sparse_mqa_decode_mxfp4(p, q, pos_q, kv4, topk_idx, topk_cnt, kv_tok, sink, out, gamma_q=None,
                            gamma_kv=None, lse=None, ws=None, dev_status=None, stream=None):
    """sparse_mqa_decode over a 4-bit cache."""
    st = (_calls or _native()).sparse_decode(p, q, pos_q, kv4, topk_idx, topk_cnt, kv_tok, sink,
                                             out, gamma_q, gamma_kv, lse, ws, dev_status, stream)
    if st:
        _check(st)


def dense_mqa_decode_mxfp4(p, q, pos_q, kv4, kv_tok, sink, out, gamma_q=None, gamma_kv=None,
                           lse=None, ws=None, dev_status=None, stream=None):
    """dense_mqa_decode over a 4-bit cache."""
    st = (_calls or _native()).dense_decode(p, q, pos_q, kv4, kv_tok, sink, out, gamma_q, gamma_kv,
                                            lse, ws, dev_status, stream)
    if st:
        _check(st)


def csa_prefill_chunk_mxfp4(p, P, T, kv_tok, idx_tok, w_s, b_pos, gamma, w_s_idx, b_pos_idx, kv4,
                            idx_key, idx_scale, q, q_idx, q_scale, w, sink, topk_idx, topk_cnt,
                            out, gamma_q=None, gamma_kv=None, ws=None, dev_status=None,
                            stream=None):
    """csa_prefill_chunk on a 4-bit cache (B = 1)."""
    dev = _device()
    a = _mqa_inputs(dev, p, T, q, kv4, kv_tok, sink, out, gamma_q, gamma_kv, None)
    L, N = kv_tok.shape[1], kv4.shape[1]
    it, wsi, bpi, ik, isc = _index_pool_args(dev, p, idx_tok, w_s_idx, b_pos_idx, idx_key,
                                             idx_scale, L, N)
    _check(lib().csa_prefill_chunk_mxfp4(
        C.byref(p), P, T, a["kv_tok"], it, L, *_pool_args(dev, p, w_s, b_pos, gamma), wsi, bpi,
        a["kv4"],
        ik, isc, N, a["q"], _need(dev, q_idx, "q_idx", torch.uint8, T, p.H_I, p.D_I),
        _need(dev, q_scale, "q_scale", torch.float32, T, p.H_I),
        _need(dev, w, "w", torch.float32, T, p.H_I),
        a["sink"], a["gq"], a["gkv"], _need(dev, topk_idx, "topk_idx", torch.int32, T, p.k),
        _need(dev, topk_cnt, "topk_cnt", torch.int32, T), a["out"], *_ws(dev, ws),
        _status(dev, dev_status),
        _raw_stream(dev, stream)))


def hca_prefill_chunk_mxfp4(p, P, T, kv_tok, w_s, b_pos, gamma, kv4, q, sink, out, gamma_q=None,
                            gamma_kv=None, lse=None, ws=None, dev_status=None, stream=None):
    """hca_prefill_chunk on a 4-bit cache (B = 1)."""
    dev = _device()
    a = _mqa_inputs(dev, p, T, q, kv4, kv_tok, sink, out, gamma_q, gamma_kv, lse)
    _check(lib().hca_prefill_chunk_mxfp4(
        C.byref(p), P, T, a["kv_tok"], kv_tok.shape[1], *_pool_args(dev, p, w_s, b_pos, gamma),
        a["kv4"],
        kv4.shape[1], a["q"], a["sink"], a["gq"], a["gkv"], a["out"], a["lse"], *_ws(dev, ws),
        _status(dev, dev_status), _raw_stream(dev, stream)))


def csa_decode_step_mxfp4(p, pos_q, kv_tok, idx_tok, w_s, b_pos, gamma, w_s_idx, b_pos_idx, kv4,
                          idx_key, idx_scale, q, q_idx, q_scale, w, sink, topk_idx, topk_cnt, out,
                          gamma_q=None, gamma_kv=None, lse=None, ws=None, dev_status=None,
                          stream=None):
    """csa_decode_step on a 4-bit cache."""
    dev = _device()
    a = _mqa_inputs(dev, p, p.B, q, kv4, kv_tok, sink, out, gamma_q, gamma_kv, lse)
    L, N = kv_tok.shape[1], kv4.shape[1]
    it, wsi, bpi, ik, isc = _index_pool_args(dev, p, idx_tok, w_s_idx, b_pos_idx, idx_key,
                                             idx_scale, L, N)
    _check(lib().csa_decode_step_mxfp4(
        C.byref(p), _need(dev, pos_q, "pos_q", torch.int64, p.B), a["kv_tok"], it, L,
        *_pool_args(dev, p, w_s, b_pos, gamma), wsi, bpi, a["kv4"], ik, isc, N, a["q"],
        _need(dev, q_idx, "q_idx", torch.uint8, p.B, p.H_I, p.D_I),
        _need(dev, q_scale, "q_scale", torch.float32, p.B, p.H_I),
        _need(dev, w, "w", torch.float32, p.B, p.H_I), a["sink"], a["gq"], a["gkv"],
        _need(dev, topk_idx, "topk_idx", torch.int32, p.B, p.k),
        _need(dev, topk_cnt, "topk_cnt", torch.int32, p.B), a["out"], a["lse"], *_ws(dev, ws),
        _status(dev, dev_status), _raw_stream(dev, stream)))


def hca_decode_step_mxfp4(p, pos_q, kv_tok, w_s, b_pos, gamma, kv4, q, sink, out, gamma_q=None,
                          gamma_kv=None, lse=None, ws=None, dev_status=None, stream=None):
    """hca_decode_step on a 4-bit cache."""
    dev = _device()
    a = _mqa_inputs(dev, p, p.B, q, kv4, kv_tok, sink, out, gamma_q, gamma_kv, lse)
    _check(lib().hca_decode_step_mxfp4(
        C.byref(p), _need(dev, pos_q, "pos_q", torch.int64, p.B), a["kv_tok"], kv_tok.shape[1],
        *_pool_args(dev, p, w_s, b_pos, gamma), a["kv4"], kv4.shape[1], a["q"], a["sink"], a["gq"],
        a["gkv"], a["out"], a["lse"], *_ws(dev, ws), _status(dev, dev_status), _raw_stream(dev, stream)))


def mxfp4_scale_bytes(rows, cols):
    """Bytes of an operand's scale tiles."""
    n = lib().mxfp4_scale_bytes(rows, cols)
    if n == 0:
        raise CsaError(2, lib().csa_last_error().decode())
    return n


def mxfp4_quantize(x, codes=None, scales=None, stream=None):
    """x [rows, cols] (bf16, each row contiguous) as an operand of the 4-bit
    product: (codes [rows, cols/2], scale tiles), allocated when not given."""
    dev = _device()
    rows, cols = _size(x, "x", 0), _size(x, "x", 1)
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1 or not x.is_cuda or \
            x.get_device() != torch.cuda.current_device():
        raise ValueError("x must be bfloat16 [rows, cols] with contiguous rows, on the current "
                         "CUDA device")
    n = mxfp4_scale_bytes(rows, cols) if rows else 0
    if codes is None:
        codes = _empty(dev, stream, rows, cols // 2)
    if scales is None:
        scales = _empty(dev, stream, n)
    _check(lib().mxfp4_quantize(rows, cols, x.data_ptr(), x.stride(0) if rows > 1 else cols,
                                _need(dev, codes, "codes", torch.uint8, rows, cols // 2),
                                _need_scales(dev, scales, "scales", n), _raw_stream(dev, stream)))
    return codes, scales


def _need_scales(dev, t, name, n):
    """Scale tiles: `n` bytes in any shape."""
    if isinstance(t, torch.Tensor) and t.numel() != n:
        raise ValueError(f"{name} must hold {n} bytes, not {t.numel()}")
    return _need(dev, t, name, torch.uint8, *(t.shape if isinstance(t, torch.Tensor) else ()))


def grouped_out_proj_mxfp4_workspace_bytes(T, H, D, g, d_g, d_model):
    n = lib().grouped_out_proj_mxfp4_workspace_bytes(T, H, D, g, d_g, d_model)
    if n == 0:
        raise CsaError(2, lib().csa_last_error().decode())
    return n


def grouped_out_proj_mxfp4(o, w_g, w_g_scale, w_o, w_o_scale, z, y=None, ws=None, dev_status=None,
                           stream=None):
    """grouped_out_proj with 4-bit weights and activations: o [T, H, D] bf16,
    w_g [g, d_g, H/g*D/2] and w_o [d_model, g*d_g/2] codes with their scale
    tiles (mxfp4_quantize).  The workspace is allocated here when not given."""
    native = _calls or _native()
    if ws is None:
        if not isinstance(o, torch.Tensor) or o.dim() != 3:
            raise ValueError("o must be [T, H, D]")
        ws = _empty(_device(), stream, grouped_out_proj_mxfp4_workspace_bytes(
            *o.shape, _size(w_g, "w_g", 0), _size(w_g, "w_g", 1), _size(w_o, "w_o", 0)))
    st = native.out_proj(o, w_g, w_g_scale, w_o, w_o_scale, z, y, ws, dev_status, stream)
    if st:
        _check(st)


# ------------------------------------------- context split over several devices --
def csa_shard_candidates(p, Q, scores, topk_idx, topk_cnt, cand_score, cand_idx,
                         dev_status=None, stream=None):
    _check(lib().csa_shard_candidates(C.byref(p), Q, _ptr(scores), scores.shape[-1],
                                      _ptr(topk_idx), _ptr(topk_cnt), _ptr(cand_score),
                                      _ptr(cand_idx), _ptr(dev_status), _stream(stream)))


def csa_merge_candidates(p, Q, G, cand_score, cand_idx, cand_cnt, N_cap, topk_idx, topk_cnt,
                         local_idx, local_cnt, dev_status=None, stream=None):
    _check(lib().csa_merge_candidates(C.byref(p), Q, G, _ptr(cand_score), _ptr(cand_idx),
                                      _ptr(cand_cnt), N_cap, _ptr(topk_idx), _ptr(topk_cnt),
                                      _ptr(local_idx), _ptr(local_cnt), _ptr(dev_status),
                                      _stream(stream)))


def sparse_mqa_partials(p, splits, q, pos_q, kv_c, topk_idx, topk_cnt, kv_tok, part_o, part_ml,
                        gamma_q=None, gamma_kv=None, dev_status=None, stream=None):
    _check(lib().sparse_mqa_partials(C.byref(p), splits, _ptr(q), _ptr(pos_q), _cache_ptr(p, kv_c),
                                     kv_c.shape[1], _ptr(topk_idx), _ptr(topk_cnt), _ptr(kv_tok),
                                     kv_tok.shape[1], _ptr(gamma_q), _ptr(gamma_kv),
                                     _ptr(part_o), _ptr(part_ml), _ptr(dev_status),
                                     _stream(stream)))


def mqa_merge_partials(p, splits, part_o, part_ml, pos_q, sink, out, lse=None, dev_status=None,
                       stream=None):
    _check(lib().mqa_merge_partials(C.byref(p), splits, _ptr(part_o), _ptr(part_ml), _ptr(pos_q),
                                    _ptr(sink), _ptr(out), _ptr(lse), _ptr(dev_status),
                                    _stream(stream)))
