"""ctypes binding of libqsa.so (the C ABI declared in include/qsa.h).

Argument marshalling only: every function checks dtypes, devices and
contiguity of torch tensors, fills the C params struct and calls the entry
point of the same name; all computation happens in the library's kernels.
A non-QSA_OK status raises ``QsaError`` with the library's message.  There is
no CPU fallback: a missing library raises ``RuntimeError`` on first use.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqsa.so")

QSA_OK, QSA_ERR_INVALID_ARG, QSA_ERR_UNSUPPORTED, QSA_ERR_WORKSPACE, QSA_ERR_CUDA = range(5)

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_f64 = ctypes.c_double
_f32 = ctypes.c_float
_sz = ctypes.c_size_t


class QsaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_status_names.get(status, status)}: {message}")
        self.status = status


_status_names = {0: "QSA_OK", 1: "QSA_ERR_INVALID_ARG", 2: "QSA_ERR_UNSUPPORTED", 3: "QSA_ERR_WORKSPACE",
                 4: "QSA_ERR_CUDA"}


class QsaIndexerPrefillParams(ctypes.Structure):
    _fields_ = [("idxQ", _vp), ("idxK", _vp), ("qNormW", _vp), ("kNormW", _vp), ("contextLengths", _vp),
                ("indices", _vp), ("workspace", _vp), ("workspaceBytes", _sz), ("batchSize", _i32),
                ("seqLen", _i32), ("numHeads", _i32), ("headDim", _i32), ("rotDim", _i32),
                ("compressRatio", _i32), ("budget", _i32), ("topK", _i32), ("ropeTheta", _f32),
                ("rmsNormEps", _f32), ("stream", _vp)]


class QsaIndexerDecodeParams(ctypes.Structure):
    _fields_ = [("idxQ", _vp), ("idxK", _vp), ("qNormW", _vp), ("kNormW", _vp), ("kvPool", _vp),
                ("pageTable", _vp), ("contextLengths", _vp), ("indices", _vp), ("workspace", _vp),
                ("workspaceBytes", _sz), ("batchSize", _i32), ("numKVHeads", _i32), ("kvHeadDim", _i32),
                ("poolHeadDim", _i32), ("numFlatPages", _i32), ("maxPagesPerSeq", _i32), ("numHeads", _i32),
                ("headDim", _i32), ("rotDim", _i32), ("compressRatio", _i32), ("budget", _i32), ("topK", _i32),
                ("ropeTheta", _f32), ("rmsNormEps", _f32), ("stream", _vp)]


class QsaIndexerHandoffParams(ctypes.Structure):
    _fields_ = [("idxK", ctypes.c_void_p), ("contextLengths", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspaceBytes", ctypes.c_size_t), ("kvPool", ctypes.c_void_p), ("pageTable", ctypes.c_void_p),
                ("batchSize", _i32), ("seqLen", _i32), ("headDim", _i32), ("compressRatio", _i32),
                ("numKVHeads", _i32), ("kvHeadDim", _i32), ("poolHeadDim", _i32), ("numFlatPages", _i32),
                ("maxPagesPerSeq", _i32), ("stream", ctypes.c_void_p)]


class QsaRopeQkvParams(ctypes.Structure):
    _fields_ = [("qkv", ctypes.c_void_p), ("qNormW", ctypes.c_void_p), ("kNormW", ctypes.c_void_p),
                ("contextLengths", ctypes.c_void_p), ("qOut", ctypes.c_void_p), ("kOut", ctypes.c_void_p),
                ("vOut", ctypes.c_void_p), ("kvPool", ctypes.c_void_p), ("pageTable", ctypes.c_void_p),
                ("batchSize", _i32), ("seqLen", _i32), ("numQHeads", _i32), ("numKVHeads", _i32),
                ("headDim", _i32), ("rotDim", _i32), ("poolHeadDim", _i32), ("numFlatPages", _i32),
                ("maxPagesPerSeq", _i32), ("ropeTheta", ctypes.c_float), ("rmsNormEps", ctypes.c_float),
                ("stream", ctypes.c_void_p)]


class QsaSparsePrefillParams(ctypes.Structure):
    _fields_ = [("qPtr", _vp), ("kPtr", _vp), ("vPtr", _vp), ("oPtr", _vp), ("indices", _vp),
                ("contextLengths", _vp), ("batchSize", _i32), ("seqLen", _i32), ("numQHeads", _i32),
                ("numKVHeads", _i32), ("headDim", _i32), ("topK", _i32), ("attentionScale", _f32),
                ("stream", _vp), ("status", _vp)]


class QsaSparseDecodeParams(ctypes.Structure):
    _fields_ = [("qPtr", _vp), ("kvPoolPtr", _vp), ("pageTable", _vp), ("indices", _vp),
                ("contextLengths", _vp), ("oPtr", _vp), ("partialO", _vp), ("partialStats", _vp),
                ("splitCounters", _vp), ("batchSize", _i32), ("numQHeads", _i32), ("numKVHeads", _i32),
                ("headDim", _i32), ("poolHeadDim", _i32), ("numFlatPages", _i32), ("maxPagesPerSeq", _i32),
                ("topK", _i32), ("attentionScale", _f32), ("stream", _vp), ("status", _vp)]


class QsaGatherParams(ctypes.Structure):
    _fields_ = [("kvPool", _vp), ("pageTable", _vp), ("indices", _vp), ("contextLengths", _vp), ("scratch", _vp),
                ("scratchPageTable", _vp), ("scratchIndices", _vp), ("scratchLengths", _vp), ("batchSize", _i32),
                ("numKVHeads", _i32), ("headDim", _i32), ("poolHeadDim", _i32), ("numFlatPages", _i32),
                ("maxPagesPerSeq", _i32), ("topK", _i32), ("stream", _vp)]


class QsaAppendKvParams(ctypes.Structure):
    _fields_ = [("qkv", _vp), ("qNormW", _vp), ("kNormW", _vp), ("contextLengths", _vp), ("newLengths", _vp),
                ("qOut", _vp), ("kOut", _vp), ("vOut", _vp), ("kvPool", _vp), ("kvScale", _vp), ("pageTable", _vp),
                ("status", _vp), ("batchSize", _i32), ("seqLen", _i32), ("numQHeads", _i32), ("numKVHeads", _i32),
                ("headDim", _i32), ("rotDim", _i32), ("poolHeadDim", _i32), ("numFlatPages", _i32),
                ("maxPagesPerSeq", _i32), ("scaleBlock", _i32), ("ropeTheta", _f32), ("rmsNormEps", _f32),
                ("stream", _vp)]


class QsaSparsePagedKv8Params(ctypes.Structure):
    _fields_ = [("qPtr", _vp), ("kvPool", _vp), ("kvScale", _vp), ("pageTable", _vp), ("indices", _vp),
                ("contextLengths", _vp), ("newLengths", _vp), ("oPtr", _vp), ("batchSize", _i32), ("seqLen", _i32),
                ("numQHeads", _i32), ("numKVHeads", _i32), ("headDim", _i32), ("poolHeadDim", _i32),
                ("numFlatPages", _i32), ("maxPagesPerSeq", _i32), ("topK", _i32), ("scaleBlock", _i32),
                ("attentionScale", _f32), ("stream", _vp), ("status", _vp)]


class QsaRotaryParams(ctypes.Structure):
    _fields_ = [("x", _vp), ("y", _vp), ("positions", _vp), ("invFreq", _vp), ("xTokenStride", _i64),
                ("xHeadStride", _i64), ("yTokenStride", _i64), ("yHeadStride", _i64), ("numTokens", _i32),
                ("numHeads", _i32), ("headDim", _i32), ("rotDim", _i32), ("interleaved", _i32), ("inverse", _i32),
                ("magnitude", _f32), ("stream", _vp)]


class QsaStoreKv4Params(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("contextLengths", _vp), ("newLengths", _vp), ("kOut", _vp), ("vOut", _vp),
                ("kvPool", _vp), ("pageTable", _vp), ("status", _vp), ("kTokenStride", _i64), ("vTokenStride", _i64),
                ("batchSize", _i32), ("seqLen", _i32), ("numKVHeads", _i32), ("headDim", _i32), ("poolRowBytes", _i32),
                ("numFlatPages", _i32), ("maxPagesPerSeq", _i32), ("stream", _vp)]


class QsaSparsePagedKv4Params(ctypes.Structure):
    _fields_ = [("qPtr", _vp), ("kvPool", _vp), ("pageTable", _vp), ("indices", _vp), ("contextLengths", _vp),
                ("newLengths", _vp), ("oPtr", _vp), ("lse", _vp), ("status", _vp), ("batchSize", _i32), ("seqLen", _i32),
                ("numQHeads", _i32), ("numKVHeads", _i32), ("headDim", _i32), ("poolRowBytes", _i32),
                ("numFlatPages", _i32), ("maxPagesPerSeq", _i32), ("topK", _i32), ("attentionScale", _f32),
                ("stream", _vp)]


class QsaSparseWeightsKv4Params(ctypes.Structure):
    _fields_ = [("qPtr", _vp), ("kvPool", _vp), ("pageTable", _vp), ("indices", _vp), ("contextLengths", _vp),
                ("newLengths", _vp), ("lse", _vp), ("weights", _vp), ("total", _vp), ("status", _vp), ("batchSize", _i32),
                ("seqLen", _i32), ("numQHeads", _i32), ("numKVHeads", _i32), ("headDim", _i32), ("poolRowBytes", _i32),
                ("numFlatPages", _i32), ("maxPagesPerSeq", _i32), ("topK", _i32), ("totalLen", _i32),
                ("attentionScale", _f32), ("stream", _vp)]


class QsaEvictKv4Params(ctypes.Structure):
    _fields_ = [("kvPool", _vp), ("pageTable", _vp), ("contextLengths", _vp), ("total", _vp), ("kept", _vp),
                ("keptLengths", _vp), ("totalOut", _vp), ("status", _vp), ("batchSize", _i32), ("numKVHeads", _i32),
                ("headDim", _i32), ("poolRowBytes", _i32), ("numFlatPages", _i32), ("maxPagesPerSeq", _i32),
                ("totalLen", _i32), ("budget", _i32), ("sinks", _i32), ("recent", _i32), ("stream", _vp)]


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises RuntimeError when it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libqsa.so is missing ({LIB_PATH}); build it with "
                                   "`python -m block_sparse_gqa_qsa_gb300.build` -- there is no fallback")
            L = ctypes.CDLL(LIB_PATH)
            for name, st in (("qsa_indexer_prefill", QsaIndexerPrefillParams),
                             ("qsa_indexer_decode", QsaIndexerDecodeParams),
                             ("qsa_sparse_prefill", QsaSparsePrefillParams),
                             ("qsa_sparse_decode", QsaSparseDecodeParams),
                             ("qsa_sparse_decode_noalloc", QsaSparseDecodeParams),
                             ("qsa_indexer_prefill_handoff", QsaIndexerHandoffParams),
                             ("qsa_sparse_prefill_bf16", QsaSparsePrefillParams),
                             ("qsa_sparse_prefill_tcgen05", QsaSparsePrefillParams),
                             ("qsa_sparse_prefill_tcgen05_bf16", QsaSparsePrefillParams),
                             ("qsa_sparse_decode_bf16", QsaSparseDecodeParams),
                             ("qsa_rope_qkv", QsaRopeQkvParams),
                             ("qsa_gather_selected", QsaGatherParams),
                             ("qsa_append_kv", QsaAppendKvParams),
                             ("qsa_append_kv_bf16", QsaAppendKvParams),
                             ("qsa_append_kv8", QsaAppendKvParams),
                             ("qsa_append_kv8_bf16", QsaAppendKvParams),
                             ("qsa_sparse_paged_kv8", QsaSparsePagedKv8Params),
                             ("qsa_sparse_paged_kv8_bf16", QsaSparsePagedKv8Params),
                             ("qsa_rotary", QsaRotaryParams),
                             ("qsa_rotary_bf16", QsaRotaryParams),
                             ("qsa_rotary_f32", QsaRotaryParams),
                             ("qsa_store_kv4", QsaStoreKv4Params),
                             ("qsa_store_kv4_bf16", QsaStoreKv4Params),
                             ("qsa_sparse_paged_kv4", QsaSparsePagedKv4Params),
                             ("qsa_sparse_paged_kv4_bf16", QsaSparsePagedKv4Params),
                             ("qsa_sparse_weights_kv4", QsaSparseWeightsKv4Params),
                             ("qsa_sparse_weights_kv4_bf16", QsaSparseWeightsKv4Params),
                             ("qsa_evict_kv4", QsaEvictKv4Params)):
                f = getattr(L, name)
                f.argtypes = [ctypes.POINTER(st)]
                f.restype = ctypes.c_int
            L.qsa_indexer_prefill_workspace_size.argtypes = [_i32] * 4
            L.qsa_indexer_prefill_workspace_size.restype = _sz
            L.qsa_indexer_decode_workspace_size.argtypes = [_i32] * 4
            L.qsa_indexer_decode_workspace_size.restype = _sz
            L.qsa_sparse_decode_partial_o_elems.argtypes = [_i32] * 3
            L.qsa_sparse_decode_partial_o_elems.restype = _sz
            L.qsa_sparse_decode_partial_stats_elems.argtypes = [_i32] * 2
            L.qsa_sparse_decode_partial_stats_elems.restype = _sz
            L.qsa_sparse_decode_counter_elems.argtypes = [_i32] * 2
            L.qsa_sparse_decode_counter_elems.restype = _sz
            L.qsa_gather_scratch_elems.argtypes = [_i32] * 4
            L.qsa_gather_scratch_elems.restype = _sz
            L.qsa_gather_scratch_pages.argtypes = [_i32]
            L.qsa_gather_scratch_pages.restype = _i32
            for n in ("qsa_sparse_decode_max_splits", "qsa_sparse_decode_partial_rows",
                      "qsa_indexer_prefill_max_blocks", "qsa_indexer_prefill_max_seq_len"):
                getattr(L, n).argtypes = []
                getattr(L, n).restype = _i32
            L.qsa_sparse_prefill_can_implement.argtypes = [_i32] * 3
            L.qsa_sparse_prefill_can_implement.restype = _i32
            L.qsa_sparse_decode_can_implement.argtypes = [_i32] * 4
            L.qsa_sparse_decode_can_implement.restype = _i32
            L.qsa_status_string.argtypes = [ctypes.c_int]
            L.qsa_status_string.restype = ctypes.c_char_p
            L.qsa_last_error_message.argtypes = []
            L.qsa_last_error_message.restype = ctypes.c_char_p
            L.qsa_last_device_error.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(_i32)]
            L.qsa_last_device_error.restype = ctypes.c_int
            L.qsa_rotary_frequencies.argtypes = [_i32, _i32] + [_f64] * 5 + [_vp]
            L.qsa_rotary_frequencies.restype = ctypes.c_int
            L.qsa_debug_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
            L.qsa_debug_set_wait_limit_ns.restype = None
            _lib = L
    return _lib


def _check(status: int) -> None:
    if status != QSA_OK:
        raise QsaError(status, lib().qsa_last_error_message().decode())


def _ptr(t: torch.Tensor | None, dtype=None, name: str = "tensor") -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# ------------------------------------------------------------------ sizes
def indexer_prefill_workspace_size(B: int, S: int, di: int, ratio: int) -> int:
    return lib().qsa_indexer_prefill_workspace_size(B, S, di, ratio)


def indexer_decode_workspace_size(B: int, max_pages_per_seq: int, ratio: int, budget: int) -> int:
    return lib().qsa_indexer_decode_workspace_size(B, max_pages_per_seq, ratio, budget)


def sparse_decode_workspace_elems(B: int, Hkv: int, D: int) -> tuple[int, int, int]:
    L = lib()
    return (L.qsa_sparse_decode_partial_o_elems(B, Hkv, D), L.qsa_sparse_decode_partial_stats_elems(B, Hkv),
            L.qsa_sparse_decode_counter_elems(B, Hkv))


def debug_set_wait_limit_ns(ns: int) -> None:
    """qsa_debug_set_wait_limit_ns: a test bound on the decode scorer's progress waits (0 restores 0.2 s)."""
    lib().qsa_debug_set_wait_limit_ns(int(ns))


def last_device_error(workspace: torch.Tensor, stream=None) -> int:
    """The status word of an indexer workspace (device-side error bits); waits for `stream`."""
    out = _i32(0)
    _check(lib().qsa_last_device_error(_ptr(workspace, name="workspace"), _stream(stream), ctypes.byref(out)))
    st = stream if stream is not None else torch.cuda.current_stream()
    if hasattr(st, "synchronize"):
        st.synchronize()
    else:
        torch.cuda.synchronize()
    return int(out.value)


def alloc_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """Zero-filled byte buffer (torch allocations are 256-byte aligned)."""
    return torch.zeros(max(nbytes, 1), dtype=torch.uint8, device=device)


# ------------------------------------------------------------- entry points
def indexer_prefill(idxQ, idxK, wq, wk, ctx, indices, workspace, *, rot, ratio, budget, topK, theta, eps,
                    stream=None):
    """qsa_indexer_prefill: idxQ fp16 [B,S,Hi,di], idxK fp16 [B,S,di] -> indices int32 [B,S,topK]."""
    B, S, Hi, di = idxQ.shape
    p = QsaIndexerPrefillParams(
        idxQ=_ptr(idxQ, torch.float16, "idxQ"), idxK=_ptr(idxK, torch.float16, "idxK"),
        qNormW=_ptr(wq, torch.float32, "qNormW"), kNormW=_ptr(wk, torch.float32, "kNormW"),
        contextLengths=_ptr(ctx, torch.int32, "contextLengths"), indices=_ptr(indices, torch.int32, "indices"),
        workspace=_ptr(workspace, None, "workspace"), workspaceBytes=workspace.numel() * workspace.element_size(),
        batchSize=B, seqLen=S, numHeads=Hi, headDim=di, rotDim=rot, compressRatio=ratio, budget=budget,
        topK=topK, ropeTheta=theta, rmsNormEps=eps, stream=_stream(stream))
    if tuple(idxK.shape) != (B, S, di) or tuple(indices.shape[-1:]) != (topK,) or indices.numel() != B * S * topK:
        raise ValueError("indexer_prefill: shape mismatch")
    _check(lib().qsa_indexer_prefill(ctypes.byref(p)))


def indexer_decode(idxQ, idxK, wq, wk, pool, page_table, ctx, indices, workspace, *, D, rot, ratio, budget,
                   topK, theta, eps, stream=None):
    """qsa_indexer_decode: one new token per sequence; updates the pool's tail state in place."""
    B, Hi, di = idxQ.shape
    nflat, tpp, Hkv, phd = pool.shape
    p = QsaIndexerDecodeParams(
        idxQ=_ptr(idxQ, torch.float16, "idxQ"), idxK=_ptr(idxK, torch.float16, "idxK"),
        qNormW=_ptr(wq, torch.float32, "qNormW"), kNormW=_ptr(wk, torch.float32, "kNormW"),
        kvPool=_ptr(pool, torch.float16, "kvPool"), pageTable=_ptr(page_table, torch.int32, "pageTable"),
        contextLengths=_ptr(ctx, torch.int32, "contextLengths"), indices=_ptr(indices, torch.int32, "indices"),
        workspace=_ptr(workspace, None, "workspace"), workspaceBytes=workspace.numel() * workspace.element_size(),
        batchSize=B, numKVHeads=Hkv, kvHeadDim=D, poolHeadDim=phd, numFlatPages=nflat,
        maxPagesPerSeq=page_table.shape[-1], numHeads=Hi, headDim=di, rotDim=rot, compressRatio=ratio,
        budget=budget, topK=topK, ropeTheta=theta, rmsNormEps=eps, stream=_stream(stream))
    if tpp != 128 or tuple(page_table.shape[:2]) != (B, 2) or indices.numel() != B * topK:
        raise ValueError("indexer_decode: shape mismatch")
    _check(lib().qsa_indexer_decode(ctypes.byref(p)))


def indexer_prefill_handoff(idxK, ctx, workspace, pool, page_table, *, D, ratio, stream=None):
    """qsa_indexer_prefill_handoff: the prefill call's block keys and trailing raw keys into the pool tails."""
    B, S, di = idxK.shape
    nflat, tpp, Hkv, phd = pool.shape
    if tpp != 128 or tuple(page_table.shape[:2]) != (B, 2):
        raise ValueError("indexer_prefill_handoff: shape mismatch")
    p = QsaIndexerHandoffParams(
        idxK=_ptr(idxK, torch.float16, "idxK"), contextLengths=_ptr(ctx, torch.int32, "contextLengths"),
        workspace=_ptr(workspace, None, "workspace"), workspaceBytes=workspace.numel() * workspace.element_size(),
        kvPool=_ptr(pool, torch.float16, "kvPool"), pageTable=_ptr(page_table, torch.int32, "pageTable"),
        batchSize=B, seqLen=S, headDim=di, compressRatio=ratio, numKVHeads=Hkv, kvHeadDim=D, poolHeadDim=phd,
        numFlatPages=nflat, maxPagesPerSeq=page_table.shape[-1], stream=_stream(stream))
    _check(lib().qsa_indexer_prefill_handoff(ctypes.byref(p)))


def rope_qkv(qkv, wq, wk, ctx, q_out, *, Hq, Hkv, rot, theta, eps, k_out=None, v_out=None, pool=None,
             page_table=None, stream=None):
    """qsa_rope_qkv: packed qkv fp16 [B,S,Hq+2Hkv,D] -> q_out [B,S,Hq,D]; optional dense k_out / v_out
    [B,S,Hkv,D] and pool K/V rows through the page table."""
    B, S, NH, D = qkv.shape
    if NH != Hq + 2 * Hkv or tuple(q_out.shape) != (B, S, Hq, D):
        raise ValueError("rope_qkv: shape mismatch")
    for t in (k_out, v_out):
        if t is not None and tuple(t.shape) != (B, S, Hkv, D):
            raise ValueError("rope_qkv: k_out/v_out shape mismatch")
    nflat = phd = mpp = 0
    if pool is not None:
        nflat, tpp, ph, phd = pool.shape
        if tpp != 128 or ph != Hkv or page_table is None or tuple(page_table.shape[:2]) != (B, 2):
            raise ValueError("rope_qkv: pool/page table shape mismatch")
        mpp = page_table.shape[-1]
    p = QsaRopeQkvParams(
        qkv=_ptr(qkv, torch.float16, "qkv"), qNormW=_ptr(wq, torch.float32, "qNormW"),
        kNormW=_ptr(wk, torch.float32, "kNormW"), contextLengths=_ptr(ctx, torch.int32, "contextLengths"),
        qOut=_ptr(q_out, torch.float16, "q_out"), kOut=_ptr(k_out, torch.float16, "k_out"),
        vOut=_ptr(v_out, torch.float16, "v_out"), kvPool=_ptr(pool, torch.float16, "kvPool"),
        pageTable=_ptr(page_table, torch.int32, "pageTable"), batchSize=B, seqLen=S, numQHeads=Hq,
        numKVHeads=Hkv, headDim=D, rotDim=rot, poolHeadDim=phd, numFlatPages=nflat, maxPagesPerSeq=mpp,
        ropeTheta=theta, rmsNormEps=eps, stream=_stream(stream))
    _check(lib().qsa_rope_qkv(ctypes.byref(p)))


def sparse_prefill(q, k, v, indices, ctx, out, scale, stream=None, status=None, impl="mma"):
    """qsa_sparse_prefill (fp16 tensors) or qsa_sparse_prefill_bf16 (bfloat16 tensors):
    q/out [B,S,Hq,D], k/v [B,S,Hkv,D], indices int32 [B,S,topK]; status: optional int32 device
    tensor whose first word collects the error bits.  impl="tcgen05" calls the tensor-core
    variants qsa_sparse_prefill_tcgen05(_bf16) with the same arguments."""
    if impl not in ("mma", "tcgen05"):
        raise ValueError("sparse_prefill: impl must be 'mma' or 'tcgen05'")
    et = q.dtype
    if et not in (torch.float16, torch.bfloat16):
        raise ValueError("sparse_prefill: q must be float16 or bfloat16")
    B, S, Hq, D = q.shape
    Hkv = k.shape[2]
    topK = indices.shape[-1]
    if tuple(k.shape) != (B, S, Hkv, D) or tuple(v.shape) != (B, S, Hkv, D) or tuple(out.shape) != (B, S, Hq, D) \
            or indices.numel() != B * S * topK:
        raise ValueError("sparse_prefill: shape mismatch")
    p = QsaSparsePrefillParams(
        qPtr=_ptr(q, et, "q"), kPtr=_ptr(k, et, "k"), vPtr=_ptr(v, et, "v"),
        oPtr=_ptr(out, et, "out"), indices=_ptr(indices, torch.int32, "indices"),
        contextLengths=_ptr(ctx, torch.int32, "contextLengths"), batchSize=B, seqLen=S, numQHeads=Hq,
        numKVHeads=Hkv, headDim=D, topK=topK, attentionScale=scale, stream=_stream(stream),
        status=None if status is None else _ptr(status, torch.int32, "status"))
    name = "qsa_sparse_prefill" + ("_tcgen05" if impl == "tcgen05" else "") + ("_bf16" if et == torch.bfloat16 else "")
    _check(getattr(lib(), name)(ctypes.byref(p)))


def sparse_decode(q, pool, page_table, indices, ctx, out, partial_o, partial_stats, counters, *, D, scale,
                  stream=None, status=None):
    """qsa_sparse_decode (fp16) or qsa_sparse_decode_bf16 (bfloat16 q/pool/out): q/out [B,1,Hq,D]; split-K
    over the pool through the page table."""
    et = q.dtype
    if et not in (torch.float16, torch.bfloat16):
        raise ValueError("sparse_decode: q must be float16 or bfloat16")
    B = q.shape[0]
    Hq = q.shape[-2]
    nflat, tpp, Hkv, phd = pool.shape
    topK = indices.shape[-1]
    if q.numel() != B * Hq * D or out.numel() != B * Hq * D or indices.numel() != B * topK or tpp != 128:
        raise ValueError("sparse_decode: shape mismatch")
    p = QsaSparseDecodeParams(
        qPtr=_ptr(q, et, "q"), kvPoolPtr=_ptr(pool, et, "kvPool"),
        pageTable=_ptr(page_table, torch.int32, "pageTable"), indices=_ptr(indices, torch.int32, "indices"),
        contextLengths=_ptr(ctx, torch.int32, "contextLengths"), oPtr=_ptr(out, et, "out"),
        partialO=_ptr(partial_o, torch.float32, "partialO"),
        partialStats=_ptr(partial_stats, torch.float32, "partialStats"),
        splitCounters=_ptr(counters, torch.int32, "splitCounters"), batchSize=B, numQHeads=Hq, numKVHeads=Hkv,
        headDim=D, poolHeadDim=phd, numFlatPages=nflat, maxPagesPerSeq=page_table.shape[-1], topK=topK,
        attentionScale=scale, stream=_stream(stream),
        status=None if status is None else _ptr(status, torch.int32, "status"))
    fn = lib().qsa_sparse_decode_bf16 if et == torch.bfloat16 else lib().qsa_sparse_decode
    _check(fn(ctypes.byref(p)))


def gather_scratch(B: int, Hkv: int, D: int, topK: int, dtype=torch.float16, device="cuda"):
    """Buffers for gather_selected: (scratch [2*B*P, 128, Hkv, D], page table int32 [B, 2, P],
    indices int32 [B, 1, topK], lengths int32 [B]), P = ceil(topK / 128)."""
    P = int(lib().qsa_gather_scratch_pages(topK))
    n = int(lib().qsa_gather_scratch_elems(B, Hkv, D, topK))
    if P < 1 or n != 2 * B * P * 128 * Hkv * D:
        raise ValueError("gather_scratch: invalid sizes")
    return (torch.empty((2 * B * P, 128, Hkv, D), dtype=dtype, device=device),
            torch.empty((B, 2, P), dtype=torch.int32, device=device),
            torch.empty((B, 1, topK), dtype=torch.int32, device=device),
            torch.empty((B,), dtype=torch.int32, device=device))


def gather_selected(pool, page_table, indices, ctx, scratch, scratch_pt, scratch_idx, scratch_len, *, D,
                    stream=None):
    """qsa_gather_selected: the K/V rows a decode list names, from the pool [numFlat, 128, Hkv, poolHeadDim]
    into contiguous scratch described as a paged pool (see gather_scratch)."""
    et = pool.dtype
    if et not in (torch.float16, torch.bfloat16) or scratch.dtype != et:
        raise ValueError("gather_selected: pool and scratch must share a float16 or bfloat16 dtype")
    nflat, tpp, Hkv, phd = pool.shape
    B, topK = ctx.shape[0], indices.shape[-1]
    P = scratch_pt.shape[-1]
    if tpp != 128 or tuple(page_table.shape[:2]) != (B, 2) or indices.numel() != B * topK \
            or tuple(scratch.shape) != (2 * B * P, 128, Hkv, D) or tuple(scratch_pt.shape) != (B, 2, P) \
            or scratch_idx.numel() != B * topK or scratch_len.numel() != B:
        raise ValueError("gather_selected: shape mismatch")
    p = QsaGatherParams(
        kvPool=_ptr(pool, et, "pool"), pageTable=_ptr(page_table, torch.int32, "pageTable"),
        indices=_ptr(indices, torch.int32, "indices"), contextLengths=_ptr(ctx, torch.int32, "contextLengths"),
        scratch=_ptr(scratch, et, "scratch"), scratchPageTable=_ptr(scratch_pt, torch.int32, "scratchPageTable"),
        scratchIndices=_ptr(scratch_idx, torch.int32, "scratchIndices"),
        scratchLengths=_ptr(scratch_len, torch.int32, "scratchLengths"), batchSize=B, numKVHeads=Hkv, headDim=D,
        poolHeadDim=phd, numFlatPages=nflat, maxPagesPerSeq=page_table.shape[-1], topK=topK,
        stream=_stream(stream))
    _check(lib().qsa_gather_selected(ctypes.byref(p)))


def sparse_decode_noalloc(q, pool, page_table, indices, ctx, out, *, D, scale, stream=None):
    """qsa_sparse_decode_noalloc: sparse_decode with the library's own fixed scratch (no workspace
    arguments; batch * KV heads <= 256).  Concurrent calls on one GPU race on that scratch."""
    B = q.shape[0]
    Hq = q.shape[-2]
    nflat, tpp, Hkv, phd = pool.shape
    topK = indices.shape[-1]
    if q.numel() != B * Hq * D or out.numel() != B * Hq * D or indices.numel() != B * topK or tpp != 128:
        raise ValueError("sparse_decode_noalloc: shape mismatch")
    p = QsaSparseDecodeParams(
        qPtr=_ptr(q, torch.float16, "q"), kvPoolPtr=_ptr(pool, torch.float16, "kvPool"),
        pageTable=_ptr(page_table, torch.int32, "pageTable"), indices=_ptr(indices, torch.int32, "indices"),
        contextLengths=_ptr(ctx, torch.int32, "contextLengths"), oPtr=_ptr(out, torch.float16, "out"),
        partialO=None, partialStats=None, splitCounters=None, batchSize=B, numQHeads=Hq, numKVHeads=Hkv,
        headDim=D, poolHeadDim=phd, numFlatPages=nflat, maxPagesPerSeq=page_table.shape[-1], topK=topK,
        attentionScale=scale, stream=_stream(stream))
    _check(lib().qsa_sparse_decode_noalloc(ctypes.byref(p)))


# -------------------------------------------------------------- paged cache
# A decode step calls these once per layer, and its kernels take a few microseconds, so the host side is kept
# short: the checks of all tensors in one expression (`_arg` names the culprit when it fails), the params packed
# in one go (same layout as the ctypes structs above).
_APPEND_PACK = struct.Struct("@12P10i2fP")
_PAGED_PACK = struct.Struct("@8P10ifPP")
_packed_calls = {}
_F32, _I32, _F16, _BF16, _E4M3 = torch.float32, torch.int32, torch.float16, torch.bfloat16, torch.float8_e4m3fn


def _packed(name: str):
    """The entry point as a function of packed params bytes."""
    f = _packed_calls.get(name)
    if f is None:
        f = lib()._FuncPtr((name, lib()))
        f.argtypes = [_vp]
        f.restype = ctypes.c_int
        _packed_calls[name] = f
    return f


def _arg(t: torch.Tensor | None, dtype, name: str, device: int) -> int:
    """The address of a contiguous tensor of `dtype` on the current device (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
        _ptr(t, dtype, name)
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{device}")
    return t.data_ptr()


def _raw_stream(stream, device: int) -> int:
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)


def _current_device(t: torch.Tensor) -> int:
    """The current CUDA device; refuses a CPU tensor before anything touches CUDA."""
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    return torch._C._cuda_getDevice()


def _append(name, fn, qkv, wq, wk, ctx, q_out, pool, scale, page_table, Hq, Hkv, rot, theta, eps, new_lengths, k_out,
            v_out, status, stream):
    et = qkv.dtype
    bf16 = et is _BF16
    if not bf16 and et is not _F16:
        raise ValueError(f"{name}: qkv must be float16 or bfloat16")
    try:
        B, S, NH, D = qkv.shape
        nflat, tpp, ph, phd = pool.shape
        ptb, two, pages = page_table.shape
    except ValueError:
        raise ValueError(f"{name}: qkv and pool have 4 dimensions, page_table 3") from None
    if NH != Hq + 2 * Hkv or q_out.shape != (B, S, Hq, D) or wq.shape != (D,) or wk.shape != (D,) or \
            ctx.shape != (B,) or tpp != 128 or ph != Hkv or ptb != B or two != 2:
        raise ValueError(f"{name}: shape mismatch")
    if (k_out is not None and k_out.shape != (B, S, Hkv, D)) or (v_out is not None and v_out.shape != (B, S, Hkv, D)):
        raise ValueError(f"{name}: k_out/v_out shape mismatch")
    if new_lengths is not None and new_lengths.shape != (B,):
        raise ValueError(f"{name}: new_lengths must have shape ({B},)")
    block, pt = 0, et
    if scale is not None:
        if scale.dim() != 3 or scale.shape[0] != nflat or scale.shape[2] != Hkv or scale.shape[1] < 1 or \
                128 % scale.shape[1]:
            raise ValueError(f"{name}: scale must be [{nflat}, 128 / block, {Hkv}]")
        block, pt = 128 // scale.shape[1], _E4M3
    dev = _current_device(qkv)
    if wq.dtype is not _F32 or wk.dtype is not _F32 or ctx.dtype is not _I32 or q_out.dtype is not et or \
            pool.dtype is not pt or page_table.dtype is not _I32 or \
            not (qkv.get_device() == wq.get_device() == wk.get_device() == ctx.get_device() == q_out.get_device() ==
                 pool.get_device() == page_table.get_device() == dev) or \
            not (qkv.is_contiguous() and wq.is_contiguous() and wk.is_contiguous() and ctx.is_contiguous() and
                 q_out.is_contiguous() and pool.is_contiguous() and page_table.is_contiguous()):
        for t, d, n in ((qkv, et, "qkv"), (wq, _F32, "qNormW"), (wk, _F32, "kNormW"), (ctx, _I32, "contextLengths"),
                        (q_out, et, "q_out"), (pool, pt, "pool"), (page_table, _I32, "pageTable")):
            _arg(t, d, n, dev)
    packed = _APPEND_PACK.pack(
        qkv.data_ptr(), wq.data_ptr(), wk.data_ptr(), ctx.data_ptr(),
        0 if new_lengths is None else _arg(new_lengths, _I32, "new_lengths", dev), q_out.data_ptr(),
        0 if k_out is None else _arg(k_out, et, "k_out", dev), 0 if v_out is None else _arg(v_out, et, "v_out", dev),
        pool.data_ptr(), 0 if scale is None else _arg(scale, _F32, "scale", dev), page_table.data_ptr(),
        0 if status is None else _arg(status, _I32, "status", dev), B, S, Hq, Hkv, D, rot, phd, nflat, pages, block, theta,
        eps, _raw_stream(stream, dev))
    r = _packed(fn[bf16])(packed)
    if r:
        _check(r)


_APPEND_KV = ("qsa_append_kv", "qsa_append_kv_bf16")
_APPEND_KV8 = ("qsa_append_kv8", "qsa_append_kv8_bf16")


def append_kv(qkv, wq, wk, ctx, q_out, pool, page_table, *, Hq, Hkv, rot, theta, eps, new_lengths=None, k_out=None,
              v_out=None, status=None, stream=None):
    """qsa_append_kv (fp16) or qsa_append_kv_bf16: the new tokens of packed qkv [B,S,Hq+2Hkv,D], normed and rotated
    at their positions: q_out [B,S,Hq,D], the K/V rows of pool [numFlat,128,Hkv,poolHeadDim] (qkv's type) through
    page_table [B,2,pages], and optional dense mirrors k_out / v_out [B,S,Hkv,D].  ctx int32 [B] holds total lengths,
    new_lengths int32 [B] how many of them are new (None: min(S, ctx))."""
    _append("append_kv", _APPEND_KV, qkv, wq, wk, ctx, q_out, pool, None, page_table, Hq, Hkv, rot, theta, eps, new_lengths, k_out,
            v_out, status, stream)


def append_kv8(qkv, wq, wk, ctx, q_out, pool, scale, page_table, *, Hq, Hkv, rot, theta, eps, new_lengths=None,
               k_out=None, v_out=None, status=None, stream=None):
    """qsa_append_kv8 (fp16) or qsa_append_kv8_bf16: append_kv into a float8_e4m3fn pool
    [numFlat,128,Hkv,poolHeadDim] with scale float32 [numFlat,128/block,Hkv], one per block of tokens and head."""
    if scale is None:
        raise ValueError("append_kv8: scale is missing")
    _append("append_kv8", _APPEND_KV8, qkv, wq, wk, ctx, q_out, pool, scale, page_table, Hq, Hkv, rot, theta, eps, new_lengths,
            k_out, v_out, status, stream)


def sparse_paged_kv8(q, pool, kv_scale, page_table, indices, ctx, out, *, scale, new_lengths=None, status=None,
                     stream=None):
    """qsa_sparse_paged_kv8 (fp16) or qsa_sparse_paged_kv8_bf16: q/out [B,S,Hq,D], pool float8_e4m3fn
    [numFlat,128,Hkv,poolHeadDim], kv_scale float32 [numFlat,128/block,Hkv], indices int32 [B,S,topK], ctx int32 [B]
    total lengths, new_lengths int32 [B] query rows (None: min(S, ctx)); scale multiplies q . k."""
    et = q.dtype
    bf16 = et is _BF16
    if not bf16 and et is not _F16:
        raise ValueError("sparse_paged_kv8: q must be float16 or bfloat16")
    try:
        B, S, Hq, D = q.shape
        nflat, tpp, Hkv, phd = pool.shape
        sf, nblk, sh = kv_scale.shape
        ptb, two, pages = page_table.shape
        ib, is_, topK = indices.shape
    except ValueError:
        raise ValueError("sparse_paged_kv8: q and pool have 4 dimensions, kv_scale, page_table and indices 3") from None
    if out.shape != (B, S, Hq, D) or tpp != 128 or ptb != B or two != 2 or ib != B or is_ != S or ctx.shape != (B,) or \
            sf != nflat or sh != Hkv or nblk < 1 or 128 % nblk or \
            (new_lengths is not None and new_lengths.shape != (B,)):
        raise ValueError("sparse_paged_kv8: shape mismatch")
    dev = _current_device(q)
    if pool.dtype is not _E4M3 or kv_scale.dtype is not _F32 or page_table.dtype is not _I32 or \
            indices.dtype is not _I32 or ctx.dtype is not _I32 or out.dtype is not et or \
            not (q.get_device() == pool.get_device() == kv_scale.get_device() == page_table.get_device() ==
                 indices.get_device() == ctx.get_device() == out.get_device() == dev) or \
            not (q.is_contiguous() and pool.is_contiguous() and kv_scale.is_contiguous() and page_table.is_contiguous() and
                 indices.is_contiguous() and ctx.is_contiguous() and out.is_contiguous()):
        for t, d, n in ((q, et, "q"), (pool, _E4M3, "pool"), (kv_scale, _F32, "kv_scale"), (page_table, _I32, "pageTable"),
                        (indices, _I32, "indices"), (ctx, _I32, "contextLengths"), (out, et, "out")):
            _arg(t, d, n, dev)
    packed = _PAGED_PACK.pack(
        q.data_ptr(), pool.data_ptr(), kv_scale.data_ptr(), page_table.data_ptr(), indices.data_ptr(), ctx.data_ptr(),
        0 if new_lengths is None else _arg(new_lengths, _I32, "new_lengths", dev), out.data_ptr(), B, S, Hq, Hkv, D, phd,
        nflat, pages, topK, 128 // nblk, scale, _raw_stream(stream, dev),
        0 if status is None else _arg(status, _I32, "status", dev))
    r = _packed("qsa_sparse_paged_kv8_bf16" if bf16 else "qsa_sparse_paged_kv8")(packed)
    if r:
        _check(r)


# --------------------------------------------------------- rotary positions
_ROTARY_PACK = struct.Struct("@4P4q6ifP")
ROTARY_SCALINGS = {"plain": 0, "linear": 1, "base": 2, "blend": 3, "ramp": 4}
_ROTARY_FN = {_F16: "qsa_rotary", _BF16: "qsa_rotary_bf16", torch.float32: "qsa_rotary_f32"}


def rotary_frequencies(rot, *, theta, scaling="plain", factor=1.0, original_length=0.0, low_turns=1.0, high_turns=32.0):
    """qsa_rotary_frequencies: the rot/2 angles per position of `rotary`, a float64 tensor on the host.  scaling: "plain",
    "linear", "base", "blend" or "ramp" (QSA_ROTARY_*)."""
    if scaling not in ROTARY_SCALINGS:
        raise ValueError(f"rotary_frequencies: scaling must be one of {sorted(ROTARY_SCALINGS)}")
    out = torch.empty(max(rot, 0) // 2, dtype=torch.float64)
    _check(lib().qsa_rotary_frequencies(ROTARY_SCALINGS[scaling], rot, theta, factor, original_length, low_turns, high_turns,
                                        out.data_ptr() or None))
    return out


def _token_stride(shape, strides, name: str) -> int:
    """Elements between tokens of [tokens, heads, D], or of [B, S, heads, D] whose tokens are evenly spaced."""
    if len(shape) == 3 or shape[1] == 1:
        return strides[0]
    if shape[0] > 1 and strides[0] != shape[1] * strides[1]:
        raise ValueError(f"{name}: sequences must follow each other evenly (stride {shape[1] * strides[1]}, got {strides[0]})")
    return strides[1]


def rotary(x, positions, out, inv_freq, *, interleaved=False, inverse=False, magnitude=1.0, stream=None):
    """qsa_rotary (fp16), qsa_rotary_bf16 or qsa_rotary_f32: the heads of x [tokens, heads, D] or [B, S, heads, D] turned
    by positions int32 [tokens] or [B, S] (negative: padding, left alone) into out, which may be x.  inv_freq: rot/2
    angles per position, float64 on the host (see rotary_frequencies).  x and out may be views whose rows are contiguous.
    The gradient is the same call with inverse=True.  The call itself records nothing for autograd: with gradients enabled,
    an x or out that requires one is refused (an autograd.Function around the two calls is what a model uses); out counts as
    changed in place, so that a backward pass that had saved it raises."""
    et = x.dtype
    fn = _ROTARY_FN.get(et)
    if fn is None:
        raise ValueError("rotary: x must be float16, bfloat16 or float32")
    if torch.is_grad_enabled() and (x.requires_grad or out.requires_grad):
        raise ValueError("rotary: no gradient flows through the call: x and out must not require one (the gradient of x is "
                         "the call with inverse=True on that of out)")
    shape, xs, ys, pairs = x.shape, x.stride(), out.stride(), inv_freq.shape
    if len(shape) not in (3, 4) or out.shape != shape or positions.shape != shape[:-2]:
        raise ValueError("rotary: x and out are [tokens, heads, D] or [B, S, heads, D], positions [tokens] or [B, S]")
    if len(pairs) != 1 or inv_freq.dtype is not torch.float64 or not inv_freq.is_cpu or not inv_freq.is_contiguous():
        raise ValueError("rotary: inv_freq must be a contiguous float64 vector on the host")
    dev = _current_device(x)
    if out.dtype is not et or not (x.get_device() == out.get_device() == dev):
        raise ValueError(f"rotary: out must be {et}, and x and out on the current device cuda:{dev}")
    heads, D = shape[-2:]
    tokens = shape[0] if len(shape) == 3 else shape[0] * shape[1]
    if D > 1 and not (xs[-1] == ys[-1] == 1):
        raise ValueError("rotary: the rows of x and out must be contiguous")
    if not (tokens and heads and D):
        raise ValueError("rotary: x is empty")
    r = _packed(fn)(_ROTARY_PACK.pack(
        x.data_ptr(), out.data_ptr(), _arg(positions, _I32, "positions", dev), inv_freq.data_ptr(),
        _token_stride(shape, xs, "x"), xs[-2], _token_stride(shape, ys, "out"), ys[-2], tokens, heads, D, 2 * pairs[0],
        interleaved, inverse, magnitude, _raw_stream(stream, dev)))
    if r:
        _check(r)
    if not out.is_inference():
        torch.autograd.graph.increment_version(out)


# -------------------------------------------------------------- 4-bit cache
_STORE4_PACK = struct.Struct("@9P2q7iP")
_PAGED4_PACK = struct.Struct("@9P9ifP")
_WEIGHTS4_PACK = struct.Struct("@10P10ifP")
_EVICT4_PACK = struct.Struct("@8P10iP")
KV4_ROW_BYTES = 80
_U8 = torch.uint8


def _pool4(pool, page_table, name):
    """(flat pages, KV heads, row bytes, B, pages per sequence) of a 4-bit pool uint8 [flat, 128, heads, bytes] and its table."""
    try:
        flat, tpp, heads, row = pool.shape
        B, two, pages = page_table.shape
    except ValueError:
        raise ValueError(f"{name}: pool has 4 dimensions, page_table 3") from None
    if tpp != 128 or two != 2:
        raise ValueError(f"{name}: pool is uint8 [pages, 128, heads, bytes], page_table [B, 2, pages]")
    return flat, heads, row, B, pages


def store_kv4(k, v, ctx, pool, page_table, *, new_lengths=None, k_out=None, v_out=None, status=None, stream=None):
    """qsa_store_kv4 (fp16) or qsa_store_kv4_bf16: the new tokens of k and v [B,S,Hkv,128] (views of packed projections
    will do) into pool uint8 [numFlat,128,Hkv,rowBytes >= 80] through page_table [B,2,pages].  ctx int32 [B] holds cached
    lengths, new_lengths int32 [B] how many of them are new (None: min(S, ctx)); k_out / v_out [B,S,Hkv,128] get the values
    that the rows stand for."""
    et = k.dtype
    if et is not _F16 and et is not _BF16:
        raise ValueError("store_kv4: k must be float16 or bfloat16")
    nflat, Hkv, row, ptb, pages = _pool4(pool, page_table, "store_kv4")
    shape, ks, vs = k.shape, k.stride(), v.stride()
    if len(shape) != 4 or v.shape != shape or shape[2] != Hkv or ptb != shape[0] or ctx.shape != (ptb,) or \
            (new_lengths is not None and new_lengths.shape != (ptb,)) or \
            (k_out is not None and k_out.shape != shape) or (v_out is not None and v_out.shape != shape):
        raise ValueError("store_kv4: shape mismatch")
    B, S, _, D = shape
    dev = _current_device(k)
    if v.dtype is not et or not (k.get_device() == v.get_device() == dev):
        raise ValueError(f"store_kv4: v must be {et}, and k and v on the current device cuda:{dev}")
    if not (ks[3] == vs[3] == 1) or (Hkv > 1 and not (ks[2] == vs[2] == D)):
        raise ValueError("store_kv4: the heads of a token of k and v must lie together")
    r = _packed("qsa_store_kv4_bf16" if et is _BF16 else "qsa_store_kv4")(_STORE4_PACK.pack(
        k.data_ptr(), v.data_ptr(), _arg(ctx, _I32, "contextLengths", dev),
        0 if new_lengths is None else _arg(new_lengths, _I32, "new_lengths", dev),
        0 if k_out is None else _arg(k_out, et, "k_out", dev), 0 if v_out is None else _arg(v_out, et, "v_out", dev),
        _arg(pool, _U8, "pool", dev), _arg(page_table, _I32, "pageTable", dev),
        0 if status is None else _arg(status, _I32, "status", dev), _token_stride(shape, ks, "k"),
        _token_stride(shape, vs, "v"), B, S, Hkv, D, row, nflat, pages, _raw_stream(stream, dev)))
    if r:
        _check(r)


def _lists4(q, pool, page_table, indices, ctx, new_lengths, name):
    """The sizes and addresses that the two readers of a 4-bit pool by lists share."""
    et = q.dtype
    if et is not _F16 and et is not _BF16:
        raise ValueError(f"{name}: q must be float16 or bfloat16")
    nflat, Hkv, row, ptb, pages = _pool4(pool, page_table, name)
    try:
        B, S, Hq, D = q.shape
        ib, is_, topK = indices.shape
    except ValueError:
        raise ValueError(f"{name}: q has 4 dimensions, indices 3") from None
    if ib != B or is_ != S or ctx.shape != (B,) or ptb != B or (new_lengths is not None and new_lengths.shape != (B,)):
        raise ValueError(f"{name}: shape mismatch")
    dev = _current_device(q)
    if pool.dtype is not _U8 or page_table.dtype is not _I32 or indices.dtype is not _I32 or ctx.dtype is not _I32 or \
            not (q.get_device() == pool.get_device() == page_table.get_device() == indices.get_device() ==
                 ctx.get_device() == dev) or \
            not (q.is_contiguous() and pool.is_contiguous() and page_table.is_contiguous() and indices.is_contiguous() and
                 ctx.is_contiguous()):
        for t, d, n in ((q, et, "q"), (pool, _U8, "pool"), (page_table, _I32, "pageTable"), (indices, _I32, "indices"),
                        (ctx, _I32, "contextLengths")):
            _arg(t, d, n, dev)
    ptrs = (q.data_ptr(), pool.data_ptr(), page_table.data_ptr(), indices.data_ptr(), ctx.data_ptr(),
            0 if new_lengths is None else _arg(new_lengths, _I32, "new_lengths", dev))
    return et, dev, ptrs, (B, S, Hq, Hkv, D, row, nflat, pages, topK)


def sparse_paged_kv4(q, pool, page_table, indices, ctx, out, *, scale, new_lengths=None, lse=None, status=None, stream=None):
    """qsa_sparse_paged_kv4 (fp16) or qsa_sparse_paged_kv4_bf16: q/out [B,S,Hq,128], pool uint8
    [numFlat,128,Hkv,rowBytes >= 80], indices int32 [B,S,topK], ctx int32 [B] cached lengths, new_lengths int32 [B] query
    rows (None: min(S, ctx)); scale multiplies q . k; lse float32 [B,S,Hq] gets the log-sum-exp of the scaled logits."""
    et, dev, ptrs, sizes = _lists4(q, pool, page_table, indices, ctx, new_lengths, "sparse_paged_kv4")
    if out.shape != sizes[:3] + (sizes[4],) or (lse is not None and lse.shape != sizes[:3]):
        raise ValueError("sparse_paged_kv4: shape mismatch")
    r = _packed("qsa_sparse_paged_kv4_bf16" if et is _BF16 else "qsa_sparse_paged_kv4")(_PAGED4_PACK.pack(
        *ptrs, _arg(out, et, "out", dev), 0 if lse is None else _arg(lse, _F32, "lse", dev),
        0 if status is None else _arg(status, _I32, "status", dev), *sizes, scale, _raw_stream(stream, dev)))
    if r:
        _check(r)


def sparse_weights_kv4(q, pool, page_table, indices, ctx, lse, weights, total=None, *, scale, new_lengths=None, status=None,
                       stream=None):
    """qsa_sparse_weights_kv4 (fp16) or qsa_sparse_weights_kv4_bf16: behind sparse_paged_kv4 with the same q, lists and
    lengths and the lse it left: weights float32 [B,S,Hkv,topK] gets every list entry's attention weight, summed over the
    query heads of a KV head, and total float32 [B,Hkv,tokens] (None: no totals) gathers them by token."""
    et, dev, ptrs, sizes = _lists4(q, pool, page_table, indices, ctx, new_lengths, "sparse_weights_kv4")
    B, S, Hq, Hkv = sizes[:4]
    counted = None if total is None else total.shape
    if lse.shape != (B, S, Hq) or weights.shape != (B, S, Hkv, sizes[8]) or \
            (counted is not None and (len(counted) != 3 or counted[:2] != (B, Hkv))):
        raise ValueError("sparse_weights_kv4: shape mismatch")
    r = _packed("qsa_sparse_weights_kv4_bf16" if et is _BF16 else "qsa_sparse_weights_kv4")(_WEIGHTS4_PACK.pack(
        *ptrs, _arg(lse, _F32, "lse", dev), _arg(weights, _F32, "weights", dev),
        0 if total is None else _arg(total, _F32, "total", dev), 0 if status is None else _arg(status, _I32, "status", dev),
        *sizes, 0 if counted is None else counted[2], scale, _raw_stream(stream, dev)))
    if r:
        _check(r)


def evict_kv4(pool, page_table, ctx, total, kept, kept_lengths, total_out=None, *, sinks=0, recent=0, status=None,
              stream=None):
    """qsa_evict_kv4: cuts every sequence of pool uint8 [numFlat,128,Hkv,rowBytes >= 80] back to budget = kept.shape[2]
    tokens per KV head, by total float32 [B,Hkv,tokens]; the first `sinks` and the last `recent` always stay.  kept int32
    [B,Hkv,budget] gets the tokens now in each slot (-1 behind the last), kept_lengths int32 [B] the new lengths, total_out
    (may be total) their totals, zeros behind them.  Tokens that total is too short for are discarded.  A sequence that has
    been cut can no longer be indexed: its lists name slots and are the caller's own."""
    nflat, Hkv, row, B, pages = _pool4(pool, page_table, "evict_kv4")
    shape, slots = total.shape, kept.shape
    if len(shape) != 3 or shape[:2] != (B, Hkv) or len(slots) != 3 or slots[:2] != (B, Hkv) or \
            ctx.shape != (B,) or kept_lengths.shape != (B,) or (total_out is not None and total_out.shape != shape):
        raise ValueError("evict_kv4: shape mismatch")
    dev = _current_device(pool)
    r = _packed("qsa_evict_kv4")(_EVICT4_PACK.pack(
        _arg(pool, _U8, "pool", dev), _arg(page_table, _I32, "pageTable", dev), _arg(ctx, _I32, "contextLengths", dev),
        _arg(total, _F32, "total", dev), _arg(kept, _I32, "kept", dev), _arg(kept_lengths, _I32, "kept_lengths", dev),
        0 if total_out is None else _arg(total_out, _F32, "total_out", dev),
        0 if status is None else _arg(status, _I32, "status", dev), B, Hkv, 128, row, nflat, pages, shape[2], slots[2], sinks,
        recent, _raw_stream(stream, dev)))
    if r:
        _check(r)
