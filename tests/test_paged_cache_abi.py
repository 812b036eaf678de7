"""The paged-cache entry points without a GPU: params layouts, refusals before any launch, and the binding's checks."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest
import torch

from conftest import ROOT

FAKE = 1 << 20  # never dereferenced: every call below is refused first
APPEND16, APPEND8 = ("qsa_append_kv", "qsa_append_kv_bf16"), ("qsa_append_kv8", "qsa_append_kv8_bf16")
ATTEND = ("qsa_sparse_paged_kv8", "qsa_sparse_paged_kv8_bf16")


@pytest.fixture(scope="module")
def qb():
    from block_sparse_gqa_qsa_gb300 import _binding, build
    build.build()
    _binding.lib()
    return _binding


def append_params(qb, **kw):
    p = dict(qkv=FAKE, qNormW=FAKE, kNormW=FAKE, contextLengths=FAKE, newLengths=FAKE, qOut=FAKE, kOut=FAKE, vOut=FAKE,
             kvPool=FAKE, kvScale=FAKE, pageTable=FAKE, status=FAKE, batchSize=2, seqLen=16, numQHeads=8, numKVHeads=2,
             headDim=128, rotDim=64, poolHeadDim=128, numFlatPages=8, maxPagesPerSeq=4, scaleBlock=16, ropeTheta=1e4,
             rmsNormEps=1e-6)
    p.update(kw)
    return qb.QsaAppendKvParams(**p)


def attend_params(qb, **kw):
    p = dict(qPtr=FAKE, kvPool=FAKE, kvScale=FAKE, pageTable=FAKE, indices=FAKE, contextLengths=FAKE, newLengths=FAKE,
             oPtr=FAKE, batchSize=2, seqLen=16, numQHeads=8, numKVHeads=2, headDim=128, poolHeadDim=128, numFlatPages=8,
             maxPagesPerSeq=4, topK=67, scaleBlock=16, attentionScale=0.1)
    p.update(kw)
    return qb.QsaSparsePagedKv8Params(**p)


def test_params_layouts(qb, tmp_path):
    structs = {"QsaAppendKvParams": qb.QsaAppendKvParams, "QsaSparsePagedKv8Params": qb.QsaSparsePagedKv8Params}
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{os.path.join(ROOT, "include", "qsa.h")}"',
             "int main(void) {"]
    for s, cls in structs.items():
        lines.append(f'printf("{s} size %zu\\n", sizeof({s}));')
        lines += [f'printf("{s} {f} %zu\\n", offsetof({s}, {f}));' for f, _ in cls._fields_]
    lines.append("return 0; }")
    c, exe = tmp_path / "layout.c", tmp_path / "layout"
    c.write_text("\n".join(lines))
    subprocess.run(["gcc", str(c), "-o", str(exe)], check=True)
    for line in filter(None, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")):
        s, f, v = line.split()
        assert int(v) == (ctypes.sizeof(structs[s]) if f == "size" else getattr(structs[s], f).offset), line


INVALID, UNSUPPORTED = 1, 2


@pytest.mark.parametrize("change,want", [
    (dict(qkv=None), INVALID), (dict(qNormW=None), INVALID), (dict(kNormW=None), INVALID),
    (dict(contextLengths=None), INVALID), (dict(qOut=None), INVALID), (dict(kvPool=None), INVALID),
    (dict(pageTable=None), INVALID), (dict(batchSize=0), INVALID), (dict(seqLen=0), INVALID),
    (dict(numQHeads=0), INVALID), (dict(numKVHeads=-1), INVALID), (dict(headDim=0), INVALID),
    (dict(numFlatPages=0), INVALID), (dict(maxPagesPerSeq=0), INVALID), (dict(rotDim=33), INVALID),
    (dict(rotDim=-2), INVALID), (dict(rotDim=144), INVALID), (dict(ropeTheta=0.0), INVALID),
    (dict(ropeTheta=float("nan")), INVALID), (dict(rmsNormEps=-1.0), INVALID), (dict(poolHeadDim=112), INVALID),
    (dict(headDim=96, rotDim=32), UNSUPPORTED), (dict(rotDim=24), UNSUPPORTED), (dict(poolHeadDim=132), UNSUPPORTED),
    (dict(numQHeads=1025), UNSUPPORTED), (dict(numKVHeads=1025), UNSUPPORTED), (dict(qkv=FAKE + 8), UNSUPPORTED),
    (dict(qOut=FAKE + 2), UNSUPPORTED), (dict(kOut=FAKE + 8), UNSUPPORTED), (dict(vOut=FAKE + 4), UNSUPPORTED),
    (dict(kvPool=FAKE + 8), UNSUPPORTED), (dict(status=FAKE + 2), UNSUPPORTED), (dict(pageTable=FAKE + 1), UNSUPPORTED),
    (dict(batchSize=1 << 16, seqLen=1 << 15), UNSUPPORTED), (dict(maxPagesPerSeq=1 << 24), UNSUPPORTED),
    (dict(numFlatPages=1 << 24), UNSUPPORTED)])
def test_append_refusals(qb, change, want):
    for fn in APPEND8:
        assert getattr(qb.lib(), fn)(ctypes.byref(append_params(qb, **change))) == want, fn
        assert fn.encode() in qb.lib().qsa_last_error_message()
    for fn in APPEND16:
        assert getattr(qb.lib(), fn)(ctypes.byref(append_params(qb, **{"kvScale": None, "scaleBlock": 0, **change}))) == want


def test_append_scale_refusals(qb):
    L = qb.lib()
    for fn in APPEND8:
        assert getattr(L, fn)(None) == INVALID
        for change in (dict(kvScale=None), dict(scaleBlock=0), dict(scaleBlock=-4), dict(scaleBlock=24),
                       dict(scaleBlock=256)):
            assert getattr(L, fn)(ctypes.byref(append_params(qb, **change))) == INVALID, (fn, change)
        assert getattr(L, fn)(ctypes.byref(append_params(qb, poolHeadDim=136))) == UNSUPPORTED  # 8-byte rows
        assert getattr(L, fn)(ctypes.byref(append_params(qb, kvScale=FAKE + 2))) == UNSUPPORTED
    for fn in APPEND16:
        assert getattr(L, fn)(None) == INVALID
        for change in (dict(scaleBlock=0), dict(kvScale=None)):
            assert getattr(L, fn)(ctypes.byref(append_params(qb, **change))) == INVALID, (fn, change)


@pytest.mark.parametrize("change,want", [
    (dict(qPtr=None), INVALID), (dict(kvPool=None), INVALID), (dict(kvScale=None), INVALID),
    (dict(pageTable=None), INVALID), (dict(indices=None), INVALID), (dict(contextLengths=None), INVALID),
    (dict(oPtr=None), INVALID), (dict(batchSize=0), INVALID), (dict(seqLen=0), INVALID), (dict(topK=0), INVALID),
    (dict(numQHeads=7), INVALID), (dict(numFlatPages=0), INVALID), (dict(maxPagesPerSeq=0), INVALID),
    (dict(poolHeadDim=112), INVALID), (dict(scaleBlock=0), INVALID), (dict(scaleBlock=12), INVALID),
    (dict(scaleBlock=256), INVALID), (dict(headDim=64), UNSUPPORTED), (dict(numQHeads=34), UNSUPPORTED),
    (dict(poolHeadDim=136), UNSUPPORTED), (dict(topK=(1 << 24) + 1), UNSUPPORTED), (dict(qPtr=FAKE + 8), UNSUPPORTED),
    (dict(kvPool=FAKE + 4), UNSUPPORTED), (dict(oPtr=FAKE + 2), UNSUPPORTED), (dict(kvScale=FAKE + 2), UNSUPPORTED),
    (dict(indices=FAKE + 1), UNSUPPORTED), (dict(batchSize=1 << 16, seqLen=1 << 15), UNSUPPORTED),
    (dict(batchSize=1 << 15, seqLen=1 << 15), UNSUPPORTED), (dict(maxPagesPerSeq=1 << 24), UNSUPPORTED),
    (dict(numFlatPages=1 << 24), UNSUPPORTED)])
def test_attend_refusals(qb, change, want):
    for fn in ATTEND:
        assert getattr(qb.lib(), fn)(None) == INVALID
        assert getattr(qb.lib(), fn)(ctypes.byref(attend_params(qb, **change))) == want, fn
        assert fn.encode() in qb.lib().qsa_last_error_message()


def test_binding_refuses(qb):
    h = torch.float16
    qkv, w, i = torch.zeros(2, 3, 4, 128, dtype=h), torch.zeros(128), torch.zeros(2, dtype=torch.int32)
    q, pool16 = torch.zeros(2, 3, 2, 128, dtype=h), torch.zeros(4, 128, 1, 128, dtype=h)
    pool8, scale = torch.zeros(4, 128, 1, 128).to(torch.float8_e4m3fn), torch.ones(4, 8, 1)
    pt = torch.zeros(2, 2, 2, dtype=torch.int32)
    kw = dict(Hq=2, Hkv=1, rot=32, theta=1e4, eps=1e-6)
    with pytest.raises(ValueError, match="CUDA tensor"):
        qb.append_kv(qkv, w, w, i, q, pool16, pt, **kw)
    with pytest.raises(ValueError, match="CUDA tensor"):
        qb.append_kv8(qkv, w, w, i, q, pool8, scale, pt, **kw)
    with pytest.raises(ValueError, match="scale"):
        qb.append_kv8(qkv, w, w, i, q, pool8, None, pt, **kw)
    with pytest.raises(ValueError, match="scale"):
        qb.append_kv8(qkv, w, w, i, q, pool8, torch.ones(4, 3, 1), pt, **kw)  # 3 does not divide a page
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        qb.append_kv(qkv.float(), w, w, i, q, pool16, pt, **kw)
    with pytest.raises(ValueError, match="shape"):
        qb.append_kv(qkv, w, w, i, q, pool16, pt, **{**kw, "Hq": 3})
    with pytest.raises(ValueError, match="shape"):
        qb.append_kv(qkv, w[:64], w, i, q, pool16, pt, **kw)
    with pytest.raises(ValueError, match="new_lengths"):
        qb.append_kv(qkv, w, w, i, q, pool16, pt, new_lengths=i[:1], **kw)
    with pytest.raises(ValueError, match="k_out"):
        qb.append_kv(qkv, w, w, i, q, pool16, pt, k_out=q, **kw)
    lists = torch.zeros(2, 3, 5, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        qb.sparse_paged_kv8(q, pool8, scale, pt, lists, i, q.clone(), scale=0.1)
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        qb.sparse_paged_kv8(q.float(), pool8, scale, pt, lists, i, q.clone(), scale=0.1)
    with pytest.raises(ValueError, match="shape"):
        qb.sparse_paged_kv8(q, pool8, scale, pt, lists[:, :2], i, q.clone(), scale=0.1)
    with pytest.raises(ValueError, match="shape"):
        qb.sparse_paged_kv8(q, pool8, scale[:, :5], pt, lists, i, q.clone(), scale=0.1)
    with pytest.raises(ValueError, match="dimensions"):
        qb.sparse_paged_kv8(q, pool8, scale, pt, lists[0], i, q.clone(), scale=0.1)


def test_packed_params_are_the_structs(qb):
    """The binding packs the params in one go: field for field what the ctypes structs (checked against C above) hold."""
    for pack, cls in ((qb._APPEND_PACK, qb.QsaAppendKvParams), (qb._PAGED_PACK, qb.QsaSparsePagedKv8Params)):
        values = [i + 1 for i in range(len(cls._fields_))]
        got = cls.from_buffer_copy(pack.pack(*values))
        assert pack.size == ctypes.sizeof(cls) and [getattr(got, f) for f, _ in cls._fields_] == values


def test_append_refuses_an_infinite_eps(qb):
    """x / sqrt(mean + inf) is 0 and inf * 0 is not: no such norm is computed."""
    for fn in APPEND16 + APPEND8:
        kw = dict(kvScale=None, scaleBlock=0) if fn in APPEND16 else {}
        assert getattr(qb.lib(), fn)(ctypes.byref(append_params(qb, rmsNormEps=float("inf"), **kw))) == INVALID
        assert b"eps" in qb.lib().qsa_last_error_message()
