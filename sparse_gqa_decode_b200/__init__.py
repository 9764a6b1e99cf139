"""Single-token GQA decode attention for B200 (sm_100a): output-aware token dropping (OAM),
an INT8 KV cache and split-KV flash-decoding with an exact log-sum-exp merge.

This module is a thin binding over the C ABI of ``libsgd.so`` (``include/sgd.h``): it turns
torch tensors into device pointers, allocates outputs and the workspace with torch, and
passes the current CUDA stream.  Every step of the computation runs in the library's CUDA
kernels; there is no CPU or PyTorch fallback, and importing fails loudly when the library
has not been built (``python sparse_gqa_decode_b200/build.py``).

A decode step, as the benchmark runs it::

    kc, vc, ks, vs, idx, cu_kept, ws = quantize_select(q, k, v, cu, G, beta, eps, 1, 8, "A", lengths)
    out, lse, ws = decode_attn(q, G, kc, vc, cu, k_scale=ks, v_scale=vs, scheme="A",
                               n_parts_=n_parts(lengths), idx=idx, cu_kept=cu_kept,
                               kept_total_=idx.shape[1])

Variants: ``oam_select`` on a bf16/f32 cache or on the INT8 cache with stored value norms;
``decode_attn(..., q_quant="token"|"tensor")`` for INT8 query codes; ``oam_select_multi`` /
``decode_attn_multi`` for several query tokens per sequence (speculative decoding);
``oam_select_blocks`` / ``decode_attn_blocks`` for whole 64-token blocks.

A speculative step over a paged cache (``PagedKv``; all state stays on the device)::

    grown, _ = pages_reserve(cache, n_nodes)              # room for the step's nodes
    n_nodes = grown - cache.lens                          # 0 everywhere if the pool had too few pages
    cu_new = torch.nn.functional.pad(n_nodes.cumsum(0, dtype=torch.int32), (1, 0))
    step = cache.with_lens(grown)
    pages_append(step, k_new, v_new, cu_new)              # their keys and values
    out, lse, _ = paged_attn(q, G, step, parent=parent, n_nodes=n_nodes, window=0, sinks=0)
    n_path, path, token, _ = verify_tree(p, tokens, parent, u_accept, u_sample, q=draft_p, n_nodes=n_nodes)
    lens, _ = pages_accept(step, path, n_path, n_nodes)   # the accepted nodes stay
    cache = cache.with_lens(lens)

``pages_fork`` branches a sequence, ``pages_keep`` cuts it to selected tokens (as ``oam_select``
returns them), ``pages_release`` gives pages back.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import torch

__all__ = [
    "lib", "quantize_kv", "oam_select", "oam_select_multi", "oam_select_blocks", "quantize_select",
    "quantize_select_multi", "quantize_select_blocks", "decode_attn",
    "decode_attn_multi", "decode_attn_blocks", "decode_attn_noalloc", "plan_segments", "workspace_status",
    "workspace_size", "decode_num_ctas", "kept_total", "kept_blocks_total", "n_parts", "kernel_timing_start",
    "kernel_timing_stop", "test_pipeline_timeout", "stream_read", "gather_read", "SGD_F32", "SGD_BF16", "SGD_I8", "SCHEME_A", "SCHEME_B",
    "SCHEME_A_CALIBRATED", "SCHEME_B_CALIBRATED", "STATUS_BITS", "ROW_COST", "PAGE", "MAX_NODES", "PagedKv",
    "paged_workspace_size", "paged_attn", "verify_tree", "pages_reserve", "pages_append", "pages_fork",
    "pages_release", "pages_accept", "pages_keep",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsgd.so")

SGD_F32, SGD_BF16, SGD_I8 = 0, 1, 2
SCHEME_A, SCHEME_B, SCHEME_A_CALIBRATED, SCHEME_B_CALIBRATED = 0, 1, 2, 3
ROW_COST = 512  # SGD_ROW_COST: the automatic split's work charge per row, in tokens
OP_QUANTIZE, OP_OAM_SELECT, OP_DECODE, OP_QUANTIZE_SELECT = 0, 1, 2, 3
PARTITION = 64
STATUS_BITS = {0x1: "empty sequence", 0x2: "wait timeout", 0x4: "size mismatch", 0x8: "bad index",
               0x10: "bad calibrated scale", 0x20: "too few free pages", 0x40: "shared page",
               0x80: "no positive probability"}
PAGE = 64  # SGD_PAGE: tokens of a page of the paged cache
MAX_NODES = 64  # SGD_MAX_NODES: query tokens of a sequence in one step of the paged calls

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python sparse_gqa_decode_b200/build.py` "
                      "(there is no fallback implementation)")


class SgdKv(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int),
        ("B", ctypes.c_int32),
        ("Hkv", ctypes.c_int32),
        ("D", ctypes.c_int32),
        ("T", ctypes.c_int64),
        ("cu_seqlens", ctypes.c_void_p),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("scheme", ctypes.c_int),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("n_parts", ctypes.c_int64),
        ("v_norm", ctypes.c_void_p),
    ]


_vp, _sz, _i64, _i32, _f = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_int, ctypes.c_float
_kvp = ctypes.POINTER(SgdKv)

lib = ctypes.CDLL(LIB_PATH)
lib.sgd_version.restype = ctypes.c_int
lib.sgd_error_string.argtypes = [ctypes.c_int]
lib.sgd_error_string.restype = ctypes.c_char_p
lib.sgd_workspace_size.argtypes = [_i32, _kvp, _i32, _i32, _i32]
lib.sgd_workspace_size.restype = _sz
lib.sgd_decode_num_ctas.argtypes = [_kvp, _i32, _vp, _i32, _i32]
lib.sgd_quantize_kv.argtypes = [_kvp, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
lib.sgd_oam_select.argtypes = [_vp, _i32, _i32, _kvp, _f, _f, _i32, _i32, _vp, _vp, _i64, _vp, _sz, _vp]
lib.sgd_decode_attn.argtypes = [_vp, _i32, _i32, _kvp, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _sz, _vp]
lib.sgd_decode_attn_multi.argtypes = [_vp, _i32, _i32, _i32, _kvp, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp,
                                      _sz, _vp]
lib.sgd_oam_select_multi.argtypes = [_vp, _i32, _i32, _i32, _kvp, _f, _f, _i32, _i32, _vp, _vp, _i64, _vp, _sz, _vp]
lib.sgd_oam_select_blocks.argtypes = [_vp, _i32, _i32, _kvp, _f, _f, _i32, _i32, _i64, _vp, _vp, _i64, _vp, _sz,
                                      _vp]
lib.sgd_decode_attn_blocks.argtypes = [_vp, _i32, _i32, _kvp, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _sz,
                                       _vp]
lib.sgd_test_pipeline_timeout.argtypes = [_i64, _i32]
lib.sgd_stream_read.argtypes = [_vp, _sz, _i32, _vp, _vp, _vp]
lib.sgd_gather_read.argtypes = [_vp, _vp, ctypes.c_int64, _vp, ctypes.c_int64, _vp, _vp]
lib.sgd_kernel_timing_start.argtypes = [_i32]
lib.sgd_kernel_timing_stop.argtypes = [ctypes.POINTER(ctypes.c_float), _i32, ctypes.POINTER(ctypes.c_int32)]
lib.sgd_kernel_timing_name.argtypes = [_i32]
lib.sgd_kernel_timing_name.restype = ctypes.c_char_p
lib.sgd_plan_segments.argtypes = [_vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _sz, _vp]
lib.sgd_workspace_status.argtypes = [_vp, ctypes.POINTER(ctypes.c_int32), _vp]
lib.sgd_quantize_select.argtypes = [_vp, _i32, _i32, _kvp, _f, _f, _i32, _i32, _i32, _i64, _vp, _vp, _vp, _vp,
                                    _vp, _vp, _vp, _i64, _vp, _sz, _vp]
lib.sgd_quantize_select_multi.argtypes = [_vp, _i32, _i32, _i32, _kvp, _f, _f, _i32, _i32, _i32, _i64, _vp, _vp, _vp,
                                          _vp, _vp, _vp, _vp, _i64, _vp, _sz, _vp]
lib.sgd_quantize_select_blocks.argtypes = [_vp, _i32, _i32, _kvp, _f, _f, _i32, _i32, _i32, _i64, _vp, _vp, _vp,
                                           _vp, _vp, _i64, _vp, _vp, _i64, _vp, _sz, _vp]
lib.sgd_decode_attn_noalloc.argtypes = [_vp, _i32, _i32, _kvp, _vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp,
                                        _vp]


class _PagedKvStruct(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int),
        ("B", ctypes.c_int32),
        ("Hkv", ctypes.c_int32),
        ("D", ctypes.c_int32),
        ("n_pages", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p),
        ("lens", ctypes.c_void_p),
        ("held", ctypes.c_void_p),
        ("ref_count", ctypes.c_void_p),
    ]


_pkvp = ctypes.POINTER(_PagedKvStruct)
lib.sgd_paged_workspace_size.argtypes = [_pkvp, _i32, _i32]
lib.sgd_paged_workspace_size.restype = _sz
lib.sgd_paged_attn.argtypes = [_vp, _i32, _i32, _pkvp, _vp, _vp, _i32, _i32, _vp, _vp, _vp, _sz, _vp]
lib.sgd_verify_tree.argtypes = [_vp, _i32, _vp, _i32, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
lib.sgd_pages_reserve.argtypes = [_pkvp, _vp, _vp, _vp, _sz, _vp]
lib.sgd_pages_append.argtypes = [_pkvp, _vp, _vp, _vp, _i64, _vp, _sz, _vp]
lib.sgd_pages_fork.argtypes = [_pkvp, _vp, _vp, _i32, _vp, _sz, _vp]
lib.sgd_pages_release.argtypes = [_pkvp, _vp, _vp, _sz, _vp]
lib.sgd_pages_accept.argtypes = [_pkvp, _vp, _vp, _vp, _i32, _vp, _vp, _sz, _vp]
lib.sgd_pages_keep.argtypes = [_pkvp, _vp, _vp, _i64, _vp, _vp, _sz, _vp]

_DT = {torch.float32: SGD_F32, torch.bfloat16: SGD_BF16, torch.int8: SGD_I8}
_QQ = {"none": 0, "token": 1, "tensor": 2}


class SgdError(RuntimeError):
    pass


def _check(rc: int, what: str):
    if rc != 0:
        raise SgdError(f"{what}: {lib.sgd_error_string(rc).decode()} ({rc})")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def n_parts(lengths: Sequence[int]) -> int:
    """Scheme-A K partitions over all sequences: sum_b ceil(L_b / 64) (a buffer size)."""
    return int(sum((int(L) + PARTITION - 1) // PARTITION for L in lengths))


def kept_total(lengths: Sequence[int], keep_num: int, keep_den: int) -> int:
    """Size of the kept-index buffer per KV head: sum_b clamp(ceil(L_b*num/den), 1, L_b)."""
    return int(sum(max(1, min(int(L), -(-int(L) * keep_num // keep_den))) for L in lengths))


def kept_blocks_total(lengths: Sequence[int], keep_num: int, keep_den: int) -> int:
    """Size of the kept-block buffer per KV head: sum_b clamp(ceil(nb_b*num/den), 1, nb_b) with
    nb_b = ceil(L_b / 64) blocks."""
    return kept_total([(int(L) + PARTITION - 1) // PARTITION for L in lengths], keep_num, keep_den)


def _kv(k, v, cu_seqlens, k_scale=None, v_scale=None, scheme=SCHEME_A, parts=0, v_norm=None) -> SgdKv:
    if k.dim() != 3 or k.shape != v.shape or k.dtype != v.dtype:
        raise ValueError("k and v must both be [Hkv, T, D] of one dtype")
    if k.dtype not in _DT:
        raise ValueError(f"unsupported cache dtype {k.dtype}")
    if not (k.is_contiguous() and v.is_contiguous() and cu_seqlens.is_contiguous()):
        raise ValueError("k, v and cu_seqlens must be contiguous")
    if cu_seqlens.dtype != torch.int32:
        raise ValueError("cu_seqlens must be int32")
    Hkv, T, D = k.shape
    return SgdKv(_DT[k.dtype], cu_seqlens.numel() - 1, Hkv, D, T, cu_seqlens.data_ptr(), k.data_ptr(),
                 v.data_ptr(), scheme, None if k_scale is None else k_scale.data_ptr(),
                 None if v_scale is None else v_scale.data_ptr(), int(parts),
                 None if v_norm is None else v_norm.data_ptr())


def workspace_size(op: int, kv: SgdKv, G: int = 1, schedule: int = 0, n_splits: int = 0) -> int:
    n = lib.sgd_workspace_size(op, ctypes.byref(kv), G, schedule, n_splits)
    if n == 0:
        raise SgdError("sgd_workspace_size rejected the arguments")
    return int(n)


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise SgdError("workspace too small")
        return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def workspace_status(workspace: torch.Tensor, stream=None) -> int:
    """Device status bits recorded by the last call that used ``workspace`` (synchronises)."""
    st = ctypes.c_int32(0)
    _check(lib.sgd_workspace_status(_ptr(workspace), ctypes.byref(st), _stream(stream)), "sgd_workspace_status")
    return int(st.value)


def _quant_scheme(scheme: str, k_scale_in, v_scale_in) -> int:
    """The C scheme value: A / B, or their calibrated forms when per-tensor scales are given."""
    if scheme not in ("A", "B"):
        raise ValueError("scheme must be 'A' or 'B'")
    if v_scale_in is None:
        if k_scale_in is not None:
            raise ValueError("a calibrated K scale goes with a calibrated V scale")
        return SCHEME_A if scheme == "A" else SCHEME_B
    if scheme == "A" and k_scale_in is not None:
        raise ValueError("scheme A computes its K partition scales: no k_scale_in")
    if scheme == "B" and k_scale_in is None:
        raise ValueError("scheme B with calibrated scales takes k_scale_in too")
    return SCHEME_A_CALIBRATED if scheme == "A" else SCHEME_B_CALIBRATED


def _scale_buffers(k, sch: int, parts: int, k_scale_in, v_scale_in):
    """k_scale / v_scale of a quantisation: the calibrated inputs where given, else new outputs."""
    Hkv = k.shape[0]
    if sch in (SCHEME_A, SCHEME_A_CALIBRATED):
        ks = torch.empty((Hkv, parts), dtype=torch.float32, device=k.device)
    else:
        ks = k_scale_in if k_scale_in is not None else torch.empty(1, dtype=torch.float32, device=k.device)
    vs = v_scale_in if v_scale_in is not None else torch.empty(1, dtype=torch.float32, device=k.device)
    return ks, vs


def quantize_kv(k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, scheme: str,
                lengths: Sequence[int], out=None, workspace=None, stream=None, v_norm=None,
                k_scale_in=None, v_scale_in=None):
    """INT8 codes and scales of a bf16/f32 cache.  Returns (k_codes, v_codes, k_scale, v_scale, ws).

    ``lengths`` are the host copies of the sequence lengths (buffer sizes only).  ``v_norm``: an
    optional float32 [Hkv, T] tensor that receives ||v_t|| (for oam_select over the INT8 cache).
    ``v_scale_in`` (and, scheme B, ``k_scale_in``): calibrated per-tensor scales, float32 [1] device
    tensors, used instead of max|x| / 127; they are returned as the scales.
    """
    sch = _quant_scheme(scheme, k_scale_in, v_scale_in)
    Hkv, T, D = k.shape
    parts = n_parts(lengths) if sch in (SCHEME_A, SCHEME_A_CALIBRATED) else 0
    kv = _kv(k, v, cu_seqlens)
    if out is None:
        kc = torch.empty((Hkv, T, D), dtype=torch.int8, device=k.device)
        vc = torch.empty_like(kc)
        ks, vs = _scale_buffers(k, sch, parts, k_scale_in, v_scale_in)
    else:
        kc, vc, ks, vs = out
    ws = _workspace(workspace_size(OP_QUANTIZE, kv), k.device, workspace)
    _check(lib.sgd_quantize_kv(ctypes.byref(kv), sch, parts, _ptr(kc), _ptr(vc), _ptr(ks), _ptr(vs), _ptr(v_norm),
                               _ptr(ws), ws.numel(), _stream(stream)), "sgd_quantize_kv")
    return kc, vc, ks, vs, ws


def oam_select(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, G: int,
               beta: float, eps: float, keep_num: int, keep_den: int, lengths: Sequence[int],
               out=None, workspace=None, stream=None, k_scale=None, v_scale=None, scheme: str = "A",
               n_parts_: int = 0, v_norm=None):
    """Kept token positions per (sequence, KV head).  Returns (idx [Hkv, Kt], cu_kept [B+1], ws).

    k, v bf16/f32: the cache before quantisation.  k, v int8: the quantised cache, scored on
    k_code * k_scale with ||v|| from ``v_norm`` (as written by quantize_kv / quantize_select)."""
    Hkv = k.shape[0]
    Kt = kept_total(lengths, keep_num, keep_den)
    kv = _kv(k, v, cu_seqlens, k_scale, v_scale, SCHEME_A if scheme == "A" else SCHEME_B, n_parts_, v_norm)
    if out is None:
        idx = torch.empty((Hkv, Kt), dtype=torch.int32, device=k.device)
        cu_kept = torch.empty(cu_seqlens.numel(), dtype=torch.int32, device=k.device)
    else:
        idx, cu_kept = out
    ws = _workspace(workspace_size(OP_OAM_SELECT, kv, G), k.device, workspace)
    _check(lib.sgd_oam_select(_ptr(q), _DT[q.dtype], G, ctypes.byref(kv), beta, eps, keep_num, keep_den, _ptr(idx),
                              _ptr(cu_kept), Kt, _ptr(ws), ws.numel(), _stream(stream)), "sgd_oam_select")
    return idx, cu_kept, ws


def oam_select_multi(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, G: int,
                     beta: float, eps: float, keep_num: int, keep_den: int, lengths: Sequence[int],
                     out=None, workspace=None, stream=None, k_scale=None, v_scale=None, scheme: str = "A",
                     n_parts_: int = 0, v_norm=None):
    """One kept set per (sequence, KV head) for the M query tokens of q [B, M, Hq, D] (the group
    maximum over all M * G query rows).  Returns (idx [Hkv, Kt], cu_kept [B+1], ws)."""
    Hkv, M = k.shape[0], q.shape[1]
    Kt = kept_total(lengths, keep_num, keep_den)
    kv = _kv(k, v, cu_seqlens, k_scale, v_scale, SCHEME_A if scheme == "A" else SCHEME_B, n_parts_, v_norm)
    if out is None:
        idx = torch.empty((Hkv, Kt), dtype=torch.int32, device=k.device)
        cu_kept = torch.empty(cu_seqlens.numel(), dtype=torch.int32, device=k.device)
    else:
        idx, cu_kept = out
    ws = _workspace(workspace_size(OP_OAM_SELECT, kv, G * M), k.device, workspace)
    _check(lib.sgd_oam_select_multi(_ptr(q), _DT[q.dtype], G, M, ctypes.byref(kv), beta, eps, keep_num, keep_den,
                                    _ptr(idx), _ptr(cu_kept), Kt, _ptr(ws), ws.numel(), _stream(stream)),
           "sgd_oam_select_multi")
    return idx, cu_kept, ws


def oam_select_blocks(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, G: int,
                      beta: float, eps: float, keep_num: int, keep_den: int, lengths: Sequence[int],
                      out=None, workspace=None, stream=None, k_scale=None, v_scale=None, scheme: str = "A",
                      n_parts_: int = 0, v_norm=None):
    """Kept 64-token blocks per (sequence, KV head), ranked by their best token's OAM score.
    Returns (blk [Hkv, NBt], cu_kept_blocks [B+1], ws); the cache arguments as in oam_select."""
    Hkv = k.shape[0]
    NBt = kept_blocks_total(lengths, keep_num, keep_den)
    kv = _kv(k, v, cu_seqlens, k_scale, v_scale, SCHEME_A if scheme == "A" else SCHEME_B, n_parts_, v_norm)
    if out is None:
        blk = torch.empty((Hkv, NBt), dtype=torch.int32, device=k.device)
        cu_kb = torch.empty(cu_seqlens.numel(), dtype=torch.int32, device=k.device)
    else:
        blk, cu_kb = out
    ws = _workspace(workspace_size(OP_OAM_SELECT, kv, G), k.device, workspace)
    _check(lib.sgd_oam_select_blocks(_ptr(q), _DT[q.dtype], G, ctypes.byref(kv), beta, eps, keep_num, keep_den,
                                     n_parts(lengths), _ptr(blk), _ptr(cu_kb), NBt, _ptr(ws), ws.numel(),
                                     _stream(stream)), "sgd_oam_select_blocks")
    return blk, cu_kb, ws


def _quantize_select(q, k, v, cu_seqlens, G, M, beta, eps, keep_num, keep_den, scheme, lengths, out, workspace,
                     stream, v_norm, k_scale_in, v_scale_in, blocks):
    sch = _quant_scheme(scheme, k_scale_in, v_scale_in)
    Hkv, T, D = k.shape
    nb = n_parts(lengths)
    parts = nb if sch in (SCHEME_A, SCHEME_A_CALIBRATED) else 0
    Kt = kept_blocks_total(lengths, keep_num, keep_den) if blocks else kept_total(lengths, keep_num, keep_den)
    kv = _kv(k, v, cu_seqlens)
    if out is None:
        kc = torch.empty((Hkv, T, D), dtype=torch.int8, device=k.device)
        vc = torch.empty_like(kc)
        ks, vs = _scale_buffers(k, sch, parts, k_scale_in, v_scale_in)
        idx = torch.empty((Hkv, Kt), dtype=torch.int32, device=k.device)
        cu_kept = torch.empty(cu_seqlens.numel(), dtype=torch.int32, device=k.device)
    else:
        kc, vc, ks, vs, idx, cu_kept = out
    ws = _workspace(workspace_size(OP_QUANTIZE_SELECT, kv, G * M), k.device, workspace)
    common = (beta, eps, keep_num, keep_den, sch, parts, _ptr(kc), _ptr(vc), _ptr(ks), _ptr(vs), _ptr(v_norm))
    tail = (_ptr(idx), _ptr(cu_kept), Kt, _ptr(ws), ws.numel(), _stream(stream))
    if blocks:
        rc = lib.sgd_quantize_select_blocks(_ptr(q), _DT[q.dtype], G, ctypes.byref(kv), *common, nb, *tail)
        name = "sgd_quantize_select_blocks"
    elif M > 1:
        rc = lib.sgd_quantize_select_multi(_ptr(q), _DT[q.dtype], G, M, ctypes.byref(kv), *common, *tail)
        name = "sgd_quantize_select_multi"
    else:
        rc = lib.sgd_quantize_select(_ptr(q), _DT[q.dtype], G, ctypes.byref(kv), *common, *tail)
        name = "sgd_quantize_select"
    _check(rc, name)
    return kc, vc, ks, vs, idx, cu_kept, ws


def quantize_select(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, G: int,
                    beta: float, eps: float, keep_num: int, keep_den: int, scheme: str, lengths: Sequence[int],
                    out=None, workspace=None, stream=None, v_norm=None, k_scale_in=None, v_scale_in=None):
    """quantize_kv and oam_select of one cache in one call (K and V read once for both).
    Returns (k_codes, v_codes, k_scale, v_scale, idx, cu_kept, ws); ``v_norm``, ``k_scale_in`` and
    ``v_scale_in`` as in quantize_kv (with calibrated scales one pass writes every code)."""
    return _quantize_select(q, k, v, cu_seqlens, G, 1, beta, eps, keep_num, keep_den, scheme, lengths, out,
                            workspace, stream, v_norm, k_scale_in, v_scale_in, False)


def quantize_select_multi(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, G: int,
                          beta: float, eps: float, keep_num: int, keep_den: int, scheme: str, lengths: Sequence[int],
                          out=None, workspace=None, stream=None, v_norm=None, k_scale_in=None, v_scale_in=None):
    """quantize_select for the M query tokens of q [B, M, Hq, D]: one kept set per (sequence, KV
    head) from the group maximum over all M * G query rows, as oam_select_multi."""
    return _quantize_select(q, k, v, cu_seqlens, G, q.shape[1], beta, eps, keep_num, keep_den, scheme, lengths, out,
                            workspace, stream, v_norm, k_scale_in, v_scale_in, False)


def quantize_select_blocks(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, G: int,
                           beta: float, eps: float, keep_num: int, keep_den: int, scheme: str, lengths: Sequence[int],
                           out=None, workspace=None, stream=None, v_norm=None, k_scale_in=None, v_scale_in=None):
    """quantize_select keeping whole 64-token blocks, as oam_select_blocks.  Returns (k_codes,
    v_codes, k_scale, v_scale, blk [Hkv, NBt], cu_kept_blocks [B+1], ws)."""
    return _quantize_select(q, k, v, cu_seqlens, G, 1, beta, eps, keep_num, keep_den, scheme, lengths, out,
                            workspace, stream, v_norm, k_scale_in, v_scale_in, True)


def decode_attn(q: torch.Tensor, G: int, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                k_scale=None, v_scale=None, scheme: str = "A", n_parts_: int = 0,
                idx=None, cu_kept=None, kept_total_: int = 0, schedule: int = 0, n_splits: int = 0,
                out=None, workspace=None, stream=None, q_quant: str = "none"):
    """Attention output and log-sum-exp per query head.  Returns (out [B,Hq,D] f32, lse [B,Hq] f32, ws).

    ``q_quant`` (INT8 cache, bf16 q, D = 128): "none", "token" (one query scale per (sequence,
    head) row) or "tensor" (one scale for all of q); q.k then runs on the INT8 codes."""
    sch = SCHEME_A if scheme == "A" else SCHEME_B
    kv = _kv(k, v, cu_seqlens, k_scale, v_scale, sch, n_parts_)
    B = cu_seqlens.numel() - 1
    Hq = k.shape[0] * G
    D = k.shape[2]
    if out is None:
        o = torch.empty((B, Hq, D), dtype=torch.float32, device=k.device)
        lse = torch.empty((B, Hq), dtype=torch.float32, device=k.device)
    else:
        o, lse = out
    ws = _workspace(workspace_size(OP_DECODE, kv, G, schedule, n_splits), k.device, workspace)
    _check(lib.sgd_decode_attn(_ptr(q), _DT[q.dtype], G, ctypes.byref(kv), _ptr(idx), _ptr(cu_kept),
                               int(kept_total_), schedule, n_splits, _QQ[q_quant], _ptr(o), _ptr(lse), _ptr(ws),
                               ws.numel(),
                               _stream(stream)), "sgd_decode_attn")
    return o, lse, ws


def decode_attn_multi(q: torch.Tensor, G: int, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                      k_scale=None, v_scale=None, scheme: str = "A", n_parts_: int = 0,
                      idx=None, cu_kept=None, kept_total_: int = 0, schedule: int = 0, n_splits: int = 0,
                      out=None, workspace=None, stream=None, q_quant: str = "none"):
    """M query tokens per sequence, q [B, M, Hq, D]; token m attends causally to positions
    <= L_b - M + m.  Returns (out [B, M, Hq, D] f32, lse [B, M, Hq] f32, ws)."""
    sch = SCHEME_A if scheme == "A" else SCHEME_B
    kv = _kv(k, v, cu_seqlens, k_scale, v_scale, sch, n_parts_)
    B, M = q.shape[0], q.shape[1]
    Hq = k.shape[0] * G
    D = k.shape[2]
    if out is None:
        o = torch.empty((B, M, Hq, D), dtype=torch.float32, device=k.device)
        lse = torch.empty((B, M, Hq), dtype=torch.float32, device=k.device)
    else:
        o, lse = out
    ws = _workspace(workspace_size(OP_DECODE, kv, G * M, schedule, n_splits), k.device, workspace)
    _check(lib.sgd_decode_attn_multi(_ptr(q), _DT[q.dtype], G, M, ctypes.byref(kv), _ptr(idx), _ptr(cu_kept),
                                     int(kept_total_), schedule, n_splits, _QQ[q_quant], _ptr(o), _ptr(lse),
                                     _ptr(ws), ws.numel(), _stream(stream)), "sgd_decode_attn_multi")
    return o, lse, ws


def decode_attn_blocks(q: torch.Tensor, G: int, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                       blk: torch.Tensor, cu_kept_blocks: torch.Tensor, k_scale=None, v_scale=None,
                       scheme: str = "A", n_parts_: int = 0, schedule: int = 0, n_splits: int = 0, out=None,
                       workspace=None, stream=None, q_quant: str = "none"):
    """Decode over kept 64-token blocks (as oam_select_blocks returns them).
    Returns (out [B, Hq, D] f32, lse [B, Hq] f32, ws)."""
    sch = SCHEME_A if scheme == "A" else SCHEME_B
    kv = _kv(k, v, cu_seqlens, k_scale, v_scale, sch, n_parts_)
    B = cu_seqlens.numel() - 1
    Hq = k.shape[0] * G
    D = k.shape[2]
    if out is None:
        o = torch.empty((B, Hq, D), dtype=torch.float32, device=k.device)
        lse = torch.empty((B, Hq), dtype=torch.float32, device=k.device)
    else:
        o, lse = out
    ws = _workspace(workspace_size(OP_DECODE, kv, G, schedule, n_splits), k.device, workspace)
    _check(lib.sgd_decode_attn_blocks(_ptr(q), _DT[q.dtype], G, ctypes.byref(kv), _ptr(blk), _ptr(cu_kept_blocks),
                                      int(blk.shape[1]), schedule, n_splits, _QQ[q_quant], _ptr(o), _ptr(lse),
                                      _ptr(ws), ws.numel(), _stream(stream)), "sgd_decode_attn_blocks")
    return o, lse, ws


def decode_attn_noalloc(q: torch.Tensor, G: int, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                        k_scale=None, v_scale=None, scheme: str = "A", n_parts_: int = 0,
                        idx=None, cu_kept=None, kept_total_: int = 0, schedule: int = 0, n_splits: int = 0,
                        out=None, status=None, stream=None, q_quant: str = "none"):
    """decode_attn without a workspace: the library's built-in device scratch array is used
    (for callers that cannot allocate).  ``out`` = (out, lse) and ``status`` ([1] int32) are
    optional preallocated device outputs.  Returns (out, lse)."""
    sch = SCHEME_A if scheme == "A" else SCHEME_B
    kv = _kv(k, v, cu_seqlens, k_scale, v_scale, sch, n_parts_)
    B = cu_seqlens.numel() - 1
    if out is None:
        o = torch.empty((B, k.shape[0] * G, k.shape[2]), dtype=torch.float32, device=k.device)
        lse = torch.empty((B, k.shape[0] * G), dtype=torch.float32, device=k.device)
    else:
        o, lse = out
    _check(lib.sgd_decode_attn_noalloc(_ptr(q), _DT[q.dtype], G, ctypes.byref(kv), _ptr(idx), _ptr(cu_kept),
                                       int(kept_total_), schedule, n_splits, _QQ[q_quant], _ptr(o), _ptr(lse),
                                       _ptr(status),
                                       _stream(stream)), "sgd_decode_attn_noalloc")
    return o, lse


def stream_read(buf: torch.Tensor, method: int = 0, sink=None, status=None, stream=None):
    """Measurement aid: read every byte of ``buf`` once (method 0: 16-byte loads, 1: bulk copies
    into shared memory), XOR-folded into ``sink`` ([1] int64).  Returns (sink, status)."""
    if sink is None:
        sink = torch.zeros(1, dtype=torch.int64, device=buf.device)
    if status is None:
        status = torch.zeros(1, dtype=torch.int32, device=buf.device)
    nbytes = buf.numel() * buf.element_size() // 16 * 16
    _check(lib.sgd_stream_read(_ptr(buf), nbytes, int(method), _ptr(sink), _ptr(status), _stream(stream)),
           "sgd_stream_read")
    return sink, status


def gather_read(a: torch.Tensor, rows: torch.Tensor, row_bytes: int, b=None, sink=None, stream=None,
                check: bool = True):
    """Measurement aid: read rows ``rows`` (int32 row numbers) of ``row_bytes`` bytes from ``a``
    (and ``b``) once, XOR-folded into ``sink`` ([1] int64).  ``check`` first verifies on the host
    that every row lies inside the tensors (a synchronising reduction: leave it to an untimed
    first call).  Returns sink."""
    if sink is None:
        sink = torch.zeros(1, dtype=torch.int64, device=a.device)
    if check and rows.numel():
        lo, hi = int(rows.min()), int(rows.max())
        for t in (a, b):
            if t is not None and (lo < 0 or (hi + 1) * row_bytes > t.numel() * t.element_size()):
                raise ValueError("a row lies outside the tensor")
    _check(lib.sgd_gather_read(_ptr(a), _ptr(b), int(row_bytes), _ptr(rows), rows.numel(), _ptr(sink),
                               _stream(stream)), "sgd_gather_read")
    return sink


def test_pipeline_timeout(polls: int, idle_producer: bool) -> None:
    """Test aid: lower the bounded pipeline-wait limit to ``polls`` polls (0 = the built-in limit)
    and, with ``idle_producer``, keep the kernels' producer warps from issuing copies, so that the
    waits run out and report SGD_STATUS_WAIT_TIMEOUT.  Affects calls made afterwards."""
    _check(lib.sgd_test_pipeline_timeout(int(polls), 1 if idle_producer else 0), "sgd_test_pipeline_timeout")


def kernel_timing_start(max_launches: int = 256) -> None:
    """Bracket each kernel the library launches from now on with a CUDA event pair (a
    measurement aid; see kernel_timing_stop)."""
    _check(lib.sgd_kernel_timing_start(int(max_launches)), "sgd_kernel_timing_start")


def kernel_timing_stop(max_launches: int = 4096):
    """Stop bracketing; returns [(mangled kernel name, milliseconds), ...] in launch order."""
    ms = (ctypes.c_float * max_launches)()
    n = ctypes.c_int32(0)
    _check(lib.sgd_kernel_timing_stop(ms, max_launches, ctypes.byref(n)), "sgd_kernel_timing_stop")
    return [(lib.sgd_kernel_timing_name(k).decode(), float(ms[k])) for k in range(min(n.value, max_launches))]


def decode_num_ctas(k, v, cu_seqlens, G: int, indexed: bool = False, schedule: int = 0, n_splits: int = 0) -> int:
    kv = _kv(k, v, cu_seqlens)
    n = lib.sgd_decode_num_ctas(ctypes.byref(kv), G, ctypes.c_void_p(1) if indexed else None, schedule, n_splits)
    _check(min(n, 0), "sgd_decode_num_ctas")
    return int(n)


def plan_segments(cu: torch.Tensor, B: int, Hkv: int, n_req: int, min_chunk: int, mode: int, row_cost: int = 0,
                  stream=None):
    """The split-KV partition: int32 [n_segs, 4] rows (cta, row, start, length), and the CTA count.
    ``row_cost``: positions charged to each row beside its tokens (the decode's automatic split
    uses ROW_COST)."""
    R = B * Hkv
    cap = n_req + R + 8
    segs = torch.full((cap, 4), -1, dtype=torch.int32, device=cu.device)
    nseg = torch.zeros(2, dtype=torch.int32, device=cu.device)
    n = R if mode == 1 else n_req
    nbytes = 2048 + 4 * (B + 2 * R + 3 * n + 6) + 32 * R  # the bound sgd.h states
    ws = torch.empty(nbytes, dtype=torch.uint8, device=cu.device)
    _check(lib.sgd_plan_segments(_ptr(cu), B, Hkv, n_req, min_chunk, mode, int(row_cost), _ptr(segs), cap, _ptr(nseg),
                                 _ptr(ws), ws.numel(), _stream(stream)), "sgd_plan_segments")
    n, ncta = (int(x) for x in nseg.tolist())
    return segs[:n].cpu(), ncta


# ------------------------------------------------------------------------------------------
# the paged cache
# ------------------------------------------------------------------------------------------
def _want(t, name: str, dtype, shape, device):
    """Raises ValueError unless ``t`` is a contiguous tensor of this dtype and shape on ``device``."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}" + ("" if t.is_contiguous() else ", strided"))


class PagedKv:
    """A paged KV cache: the pool ``k``, ``v`` [n_pages, Hkv, 64, D] (bfloat16, or int8 codes under the
    per-tensor ``k_scale``, ``v_scale`` float32 [1]), ``page_table`` int32 [B, max_pages], ``lens`` int32
    [B], and for the upkeep calls ``held`` int32 [B] and ``ref_count`` int32 [n_pages].  The tensors stay
    the caller's; the object only checks them once and holds their addresses."""

    def __init__(self, k, v, page_table, lens, held=None, ref_count=None, k_scale=None, v_scale=None):
        if k.dim() != 4 or k.shape[2] != PAGE:
            raise ValueError("k must be [n_pages, Hkv, 64, D]")
        if k.dtype not in (torch.bfloat16, torch.int8):
            raise ValueError(f"unsupported cache dtype {k.dtype}")
        if page_table.dim() != 2:
            raise ValueError("page_table must be [B, max_pages]")
        if (k.dtype == torch.int8) != (k_scale is not None) or (k_scale is None) != (v_scale is None):
            raise ValueError("an int8 cache, and no other, has k_scale and v_scale")
        B, dev, i32 = page_table.shape[0], k.device, torch.int32
        _want(k, "k", k.dtype, k.shape, dev)
        _want(v, "v", k.dtype, k.shape, dev)
        _want(page_table, "page_table", i32, page_table.shape, dev)
        _want(lens, "lens", i32, (B,), dev)
        for t, name, dt, n in ((held, "held", i32, B), (ref_count, "ref_count", i32, k.shape[0]),
                               (k_scale, "k_scale", torch.float32, 1), (v_scale, "v_scale", torch.float32, 1)):
            if t is not None:
                _want(t, name, dt, (n,), dev)
        self.k, self.v, self.page_table, self.lens = k, v, page_table, lens
        self.held, self.ref_count, self.k_scale, self.v_scale = held, ref_count, k_scale, v_scale
        self.device, self.B, self.Hkv, self.D = dev, B, k.shape[1], k.shape[3]
        address = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self._struct = _PagedKvStruct(_DT[k.dtype], B, self.Hkv, self.D, k.shape[0], page_table.shape[1], k.data_ptr(),
                                      v.data_ptr(), address(k_scale), address(v_scale), page_table.data_ptr(),
                                      lens.data_ptr(), address(held), address(ref_count))
        self._ref = ctypes.byref(self._struct)

    def with_lens(self, lens: torch.Tensor) -> "PagedKv":
        """The same cache with other lengths (as pages_reserve, pages_accept and pages_keep return them)."""
        return PagedKv(self.k, self.v, self.page_table, lens, self.held, self.ref_count, self.k_scale, self.v_scale)


def paged_workspace_size(cache: PagedKv, G: int = 1, M: int = 0) -> int:
    """Bytes of a workspace for any paged call with up to ``M`` query tokens and ``G`` heads per KV head
    (M = 0: for the upkeep calls alone)."""
    n = lib.sgd_paged_workspace_size(cache._ref, G, M)
    if n == 0:
        raise SgdError("sgd_paged_workspace_size rejected the arguments")
    return int(n)


class _On:
    """The raw stream of a call, and new tensors that belong to it: a tensor made for a call on another
    stream than the current one is allocated on that stream, so that its memory is not handed on while
    the call may still run."""

    def __init__(self, device, stream):
        if device.type != "cuda":
            raise ValueError(f"the tensors are on {device}, not on a CUDA device")
        if device.index != torch.cuda.current_device():
            raise ValueError(f"the tensors are on {device}, the current device is cuda:{torch.cuda.current_device()}")
        self.device, self.stream = device, stream
        self.raw = (stream if stream is not None else torch.cuda.current_stream(device)).cuda_stream

    def empty(self, shape, dtype):
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def workspace(self, nbytes, workspace):
        if workspace is None:
            return self.empty(nbytes, torch.uint8)
        if workspace.device != self.device or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {self.device}")
        return workspace


def _int32(n: int) -> int:
    """The nearest 32-bit number: what lies beyond either end means the same to the call, or is refused like it."""
    return max(min(n, 2 ** 31 - 1), -2 ** 31)


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def paged_attn(q: torch.Tensor, G: int, cache: PagedKv, parent=None, n_nodes=None, window: int = 0, sinks: int = 0,
               out=None, workspace=None, stream=None):
    """Attention of a step's query tokens q [B, M, Hkv * G, D] (bf16, M <= 64) over the paged cache, whose
    last entries they are: a tree of drafted tokens (``parent`` int32 [B, M]), a chain (``parent`` None)
    or one token (M = 1); ``n_nodes`` int32 [B] where a sequence has fewer than M.  ``window`` > 0 limits
    each query to the window's positions and the first ``sinks`` ones.
    Returns (out [B, M, Hq, D] bf16, lse [B, M, Hq] f32, ws)."""
    if q.dim() != 4:
        raise ValueError("q must be [B, M, Hq, D]")
    M, Hq = q.shape[1], cache.Hkv * G
    dev = cache.device
    _want(q, "q", torch.bfloat16, (cache.B, M, Hq, cache.D), dev)
    if parent is not None:
        _want(parent, "parent", torch.int32, (cache.B, M), dev)
    if n_nodes is not None:
        _want(n_nodes, "n_nodes", torch.int32, (cache.B,), dev)
    on = _On(dev, stream)
    if out is None:
        o, lse = on.empty(q.shape, torch.bfloat16), on.empty((cache.B, M, Hq), torch.float32)
    else:
        o, lse = out
        _want(o, "out", torch.bfloat16, q.shape, dev)
        _want(lse, "lse", torch.float32, (cache.B, M, Hq), dev)
    ws = on.workspace(0 if workspace is not None else paged_workspace_size(cache, G, M), workspace)
    _check(lib.sgd_paged_attn(q.data_ptr(), G, M, cache._ref, None if parent is None else parent.data_ptr(),
                              None if n_nodes is None else n_nodes.data_ptr(), _int32(window),
                              _int32(sinks), o.data_ptr(), lse.data_ptr(), ws.data_ptr(), _nbytes(ws), on.raw), "sgd_paged_attn")
    return o, lse, ws


def verify_tree(p: torch.Tensor, tokens: torch.Tensor, parent: torch.Tensor, u_accept: torch.Tensor,
                u_sample: torch.Tensor, q=None, n_nodes=None, out=None, workspace=None, stream=None):
    """Drafted tokens against the target's distributions p [B, M, V] (f32 or bf16; ``q`` the draft's, None
    for chosen drafts), tokens and parent int32 [B, M], random numbers u_accept [B, M] and u_sample [B].
    Returns (n_path [B], path [B, M], next_token [B], ws), int32."""
    if p.dim() != 3 or p.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("p must be a float32 or bfloat16 [B, M, V] tensor")
    (B, M, V), dev, i32 = p.shape, p.device, torch.int32
    _want(p, "p", p.dtype, p.shape, dev)
    _want(tokens, "tokens", i32, (B, M), dev)
    _want(parent, "parent", i32, (B, M), dev)
    _want(u_accept, "u_accept", torch.float32, (B, M), dev)
    _want(u_sample, "u_sample", torch.float32, (B,), dev)
    if q is not None:
        _want(q, "q", p.dtype, p.shape, dev)
    if n_nodes is not None:
        _want(n_nodes, "n_nodes", i32, (B,), dev)
    on = _On(dev, stream)
    if out is None:
        n_path, path, token = on.empty((B,), i32), on.empty((B, M), i32), on.empty((B,), i32)
    else:
        n_path, path, token = out
        _want(n_path, "n_path", i32, (B,), dev)
        _want(path, "path", i32, (B, M), dev)
        _want(token, "next_token", i32, (B,), dev)
    ws = on.workspace(256, workspace)
    _check(lib.sgd_verify_tree(p.data_ptr(), _DT[p.dtype], None if q is None else q.data_ptr(), B, M, V,
                               tokens.data_ptr(), parent.data_ptr(), None if n_nodes is None else n_nodes.data_ptr(),
                               u_accept.data_ptr(), u_sample.data_ptr(), n_path.data_ptr(), path.data_ptr(),
                               token.data_ptr(), ws.data_ptr(), _nbytes(ws), on.raw), "sgd_verify_tree")
    return n_path, path, token, ws


def _new_lens(on: _On, cache: PagedKv, out):
    if out is None:
        return on.empty((cache.B,), torch.int32)
    _want(out, "new_lens", torch.int32, (cache.B,), cache.device)
    return out


def _paged_ws(on: _On, cache: PagedKv, workspace):
    return on.workspace(0 if workspace is not None else paged_workspace_size(cache), workspace)


def pages_reserve(cache: PagedKv, add: torch.Tensor, out=None, workspace=None, stream=None):
    """Pages for ``add`` int32 [B] more tokens of each row.  Returns (new_lens [B], ws); new_lens is cache.lens where
    the call was refused (its status says why), so that new_lens - cache.lens is what was granted."""
    _want(add, "add", torch.int32, (cache.B,), cache.device)
    on = _On(cache.device, stream)
    new, ws = _new_lens(on, cache, out), _paged_ws(on, cache, workspace)
    _check(lib.sgd_pages_reserve(cache._ref, add.data_ptr(), new.data_ptr(), ws.data_ptr(), _nbytes(ws), on.raw),
           "sgd_pages_reserve")
    return new, ws


def pages_append(cache: PagedKv, k_new: torch.Tensor, v_new: torch.Tensor, cu_new: torch.Tensor, workspace=None,
                 stream=None):
    """Writes k_new, v_new [Hkv, T_new, D] (bf16; row b's tokens cu_new[b] .. cu_new[b+1] - 1) as the last
    entries of each row; an int8 cache takes their codes under its scales.  Returns ws."""
    if k_new.dim() != 3:
        raise ValueError("k_new must be [Hkv, T_new, D]")
    shape = (cache.Hkv, k_new.shape[1], cache.D)
    _want(k_new, "k_new", torch.bfloat16, shape, cache.device)
    _want(v_new, "v_new", torch.bfloat16, shape, cache.device)
    _want(cu_new, "cu_new", torch.int32, (cache.B + 1,), cache.device)
    on = _On(cache.device, stream)
    ws = on.workspace(256, workspace)
    _check(lib.sgd_pages_append(cache._ref, k_new.data_ptr(), v_new.data_ptr(), cu_new.data_ptr(), k_new.shape[1],
                                ws.data_ptr(), _nbytes(ws), on.raw), "sgd_pages_append")
    return ws


def pages_fork(cache: PagedKv, src: torch.Tensor, dst: torch.Tensor, workspace=None, stream=None):
    """Row dst[i] becomes a copy of row src[i] (int32 [n]).  Returns ws."""
    if src.dim() != 1:
        raise ValueError("src must be [n]")
    _want(src, "src", torch.int32, src.shape, cache.device)
    _want(dst, "dst", torch.int32, src.shape, cache.device)
    on = _On(cache.device, stream)
    ws = _paged_ws(on, cache, workspace)
    _check(lib.sgd_pages_fork(cache._ref, src.data_ptr(), dst.data_ptr(), src.shape[0], ws.data_ptr(), _nbytes(ws),
                              on.raw), "sgd_pages_fork")
    return ws


def pages_release(cache: PagedKv, keep: torch.Tensor, workspace=None, stream=None):
    """Every row gives back the pages behind its first ``keep`` int32 [B] tokens.  Returns ws."""
    _want(keep, "keep", torch.int32, (cache.B,), cache.device)
    on = _On(cache.device, stream)
    ws = on.workspace(256, workspace)
    _check(lib.sgd_pages_release(cache._ref, keep.data_ptr(), ws.data_ptr(), _nbytes(ws), on.raw), "sgd_pages_release")
    return ws


def pages_accept(cache: PagedKv, path: torch.Tensor, n_path: torch.Tensor, n_nodes: torch.Tensor, out=None,
                 workspace=None, stream=None):
    """Of each row's last n_nodes entries those of ``path`` [B, M] (its first n_path) stay, as verify_tree
    returns them.  Returns (new_lens [B], ws)."""
    if path.dim() != 2:
        raise ValueError("path must be [B, M]")
    M = path.shape[1]
    _want(path, "path", torch.int32, (cache.B, M), cache.device)
    _want(n_path, "n_path", torch.int32, (cache.B,), cache.device)
    _want(n_nodes, "n_nodes", torch.int32, (cache.B,), cache.device)
    on = _On(cache.device, stream)
    new, ws = _new_lens(on, cache, out), on.workspace(256, workspace)
    _check(lib.sgd_pages_accept(cache._ref, path.data_ptr(), n_path.data_ptr(), n_nodes.data_ptr(), M, new.data_ptr(),
                                ws.data_ptr(), _nbytes(ws), on.raw), "sgd_pages_accept")
    return new, ws


def pages_keep(cache: PagedKv, idx: torch.Tensor, cu_kept: torch.Tensor, out=None, workspace=None, stream=None):
    """Each row and KV head keeps the tokens ``idx`` [Hkv, kept_total], cu_kept [B + 1] (as oam_select
    returns them) as its first ones.  Returns (new_lens [B], ws)."""
    if idx.dim() != 2:
        raise ValueError("idx must be [Hkv, kept_total]")
    _want(idx, "idx", torch.int32, (cache.Hkv, idx.shape[1]), cache.device)
    _want(cu_kept, "cu_kept", torch.int32, (cache.B + 1,), cache.device)
    on = _On(cache.device, stream)
    new, ws = _new_lens(on, cache, out), on.workspace(256, workspace)
    _check(lib.sgd_pages_keep(cache._ref, idx.data_ptr(), cu_kept.data_ptr(), idx.shape[1], new.data_ptr(),
                              ws.data_ptr(), _nbytes(ws), on.raw), "sgd_pages_keep")
    return new, ws
