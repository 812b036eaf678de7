"""Rotary positions and the 4-bit cache without a GPU: params layouts, refusals before any launch, the frequencies, and the
binding's checks."""
from __future__ import annotations

import ctypes
import math
import os
import subprocess

import pytest
import torch

from conftest import ROOT

FAKE = 1 << 20  # never dereferenced: every call below is refused first
INVALID, UNSUPPORTED = 1, 2
ROTARY = ("qsa_rotary", "qsa_rotary_bf16", "qsa_rotary_f32")
STORE = ("qsa_store_kv4", "qsa_store_kv4_bf16")
ATTEND = ("qsa_sparse_paged_kv4", "qsa_sparse_paged_kv4_bf16")
WEIGHTS = ("qsa_sparse_weights_kv4", "qsa_sparse_weights_kv4_bf16")


@pytest.fixture(scope="module")
def qb():
    from block_sparse_gqa_qsa_gb300 import _binding, build
    build.build()
    _binding.lib()
    return _binding


FREQ = (ctypes.c_double * 32)(*([0.5] * 32))
READERS = dict(qPtr=FAKE, kvPool=FAKE, pageTable=FAKE, indices=FAKE, contextLengths=FAKE, newLengths=FAKE, lse=FAKE,
               status=FAKE, batchSize=2, seqLen=16, numQHeads=8, numKVHeads=2, headDim=128, poolRowBytes=80, numFlatPages=8,
               maxPagesPerSeq=4, topK=67, attentionScale=0.1)
DEFAULTS = {
    "QsaRotaryParams": dict(x=FAKE, y=FAKE + (1 << 16), positions=FAKE, invFreq=ctypes.addressof(FREQ), xTokenStride=1024,
                            xHeadStride=128, yTokenStride=1024, yHeadStride=128, numTokens=4, numHeads=8, headDim=128,
                            rotDim=64, magnitude=1.0),
    "QsaStoreKv4Params": dict(k=FAKE, v=FAKE, contextLengths=FAKE, newLengths=FAKE, kOut=FAKE, vOut=FAKE, kvPool=FAKE,
                              pageTable=FAKE, status=FAKE, kTokenStride=256, vTokenStride=256, batchSize=2, seqLen=16,
                              numKVHeads=2, headDim=128, poolRowBytes=80, numFlatPages=8, maxPagesPerSeq=4),
    "QsaSparsePagedKv4Params": dict(READERS, oPtr=FAKE),
    "QsaSparseWeightsKv4Params": dict(READERS, weights=FAKE, total=FAKE, totalLen=512),
    "QsaEvictKv4Params": dict(kvPool=FAKE, pageTable=FAKE, contextLengths=FAKE, total=FAKE, kept=FAKE, keptLengths=FAKE + 64,
                              totalOut=FAKE, status=FAKE, batchSize=2, numKVHeads=2, headDim=128, poolRowBytes=80,
                              numFlatPages=8, maxPagesPerSeq=4, totalLen=512, budget=64, sinks=4, recent=8),
}


def refuses(qb, struct, names, change, want):
    for name in names:
        assert getattr(qb.lib(), name)(None) == INVALID
        p = getattr(qb, struct)(**{**DEFAULTS[struct], **change})
        assert getattr(qb.lib(), name)(ctypes.byref(p)) == want, (name, change, qb.lib().qsa_last_error_message())
        assert name.encode() in qb.lib().qsa_last_error_message()


def test_params_layouts(qb, tmp_path):
    structs = {s: getattr(qb, s) for s in DEFAULTS}
    lines = ['#include <stdio.h>', '#include <stddef.h>', f'#include "{os.path.join(ROOT, "include", "qsa.h")}"',
             "int main(void) {"]
    for s, cls in structs.items():
        lines.append(f'printf("{s} size %zu\\n", sizeof({s}));')
        lines += [f'printf("{s} {f} %zu\\n", offsetof({s}, {f}));' for f, _ in cls._fields_]
    lines.append('printf("row bytes %d\\n", QSA_KV4_ROW_BYTES); return 0; }')
    c, exe = tmp_path / "layout.c", tmp_path / "layout"
    c.write_text("\n".join(lines))
    subprocess.run(["gcc", str(c), "-o", str(exe)], check=True)
    out = [line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()]
    assert out.pop() == ["row", "bytes", str(qb.KV4_ROW_BYTES)]
    for s, f, v in out:
        assert int(v) == (ctypes.sizeof(structs[s]) if f == "size" else getattr(structs[s], f).offset), (s, f)


def test_packed_params_are_the_structs(qb):
    for pack, s in ((qb._ROTARY_PACK, "QsaRotaryParams"), (qb._STORE4_PACK, "QsaStoreKv4Params"),
                    (qb._PAGED4_PACK, "QsaSparsePagedKv4Params"), (qb._WEIGHTS4_PACK, "QsaSparseWeightsKv4Params"),
                    (qb._EVICT4_PACK, "QsaEvictKv4Params")):
        cls = getattr(qb, s)
        values = [i + 1 for i in range(len(cls._fields_))]
        got = cls.from_buffer_copy(pack.pack(*values))
        assert pack.size == ctypes.sizeof(cls) and [getattr(got, f) for f, _ in cls._fields_] == values, s


NAN_FREQ = (ctypes.c_double * 32)(*([float("nan")] * 32))


@pytest.mark.parametrize("change,want", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(positions=None), INVALID), (dict(invFreq=None), INVALID),
    (dict(numTokens=0), INVALID), (dict(numHeads=0), INVALID), (dict(headDim=-1), INVALID), (dict(rotDim=0), INVALID),
    (dict(rotDim=63), INVALID), (dict(rotDim=130), INVALID), (dict(xTokenStride=-1024), INVALID),
    (dict(yTokenStride=1023), INVALID), (dict(yHeadStride=127), INVALID), (dict(yHeadStride=0), INVALID),
    (dict(yTokenStride=128, yHeadStride=128), INVALID), (dict(yTokenStride=1 << 62, yHeadStride=1 << 62), INVALID),
    (dict(y=FAKE, xTokenStride=2048), INVALID), (dict(magnitude=float("inf")), INVALID),
    (dict(invFreq=ctypes.addressof(NAN_FREQ)), INVALID), (dict(headDim=320, rotDim=320, yTokenStride=2560, yHeadStride=320), UNSUPPORTED),
    (dict(x=FAKE + 1), UNSUPPORTED), (dict(y=FAKE + 1), UNSUPPORTED), (dict(positions=FAKE + 2), UNSUPPORTED),
    (dict(numTokens=1, numHeads=1 << 16), UNSUPPORTED),
    (dict(numTokens=1, numHeads=1, headDim=1 << 16), UNSUPPORTED), (dict(numTokens=1 << 21), UNSUPPORTED), (dict(numTokens=1 << 30, numHeads=1 << 30, yHeadStride=1 << 8, yTokenStride=1 << 38), UNSUPPORTED)])
def test_rotary_refusals(qb, change, want):
    refuses(qb, "QsaRotaryParams", ROTARY, change, want)


@pytest.mark.parametrize("change,want", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(contextLengths=None), INVALID), (dict(kvPool=None), INVALID),
    (dict(pageTable=None), INVALID), (dict(batchSize=0), INVALID), (dict(seqLen=0), INVALID), (dict(numKVHeads=0), INVALID),
    (dict(numFlatPages=0), INVALID), (dict(maxPagesPerSeq=0), INVALID), (dict(kTokenStride=248), INVALID),
    (dict(vTokenStride=0), INVALID), (dict(poolRowBytes=64), INVALID), (dict(headDim=64, kTokenStride=128), UNSUPPORTED),
    (dict(poolRowBytes=88), UNSUPPORTED), (dict(kTokenStride=260), UNSUPPORTED), (dict(k=FAKE + 8), UNSUPPORTED),
    (dict(v=FAKE + 2), UNSUPPORTED), (dict(kOut=FAKE + 8), UNSUPPORTED), (dict(vOut=FAKE + 4), UNSUPPORTED),
    (dict(kvPool=FAKE + 8), UNSUPPORTED), (dict(status=FAKE + 2), UNSUPPORTED), (dict(newLengths=FAKE + 1), UNSUPPORTED),
    (dict(batchSize=1 << 16, seqLen=1 << 15), UNSUPPORTED), (dict(batchSize=1 << 13, seqLen=1 << 13), UNSUPPORTED),
    (dict(maxPagesPerSeq=1 << 24), UNSUPPORTED), (dict(numFlatPages=1 << 24), UNSUPPORTED),
    (dict(poolRowBytes=1 << 30), UNSUPPORTED)])
def test_store_refusals(qb, change, want):
    refuses(qb, "QsaStoreKv4Params", STORE, change, want)


READER_REFUSALS = [
    (dict(qPtr=None), INVALID), (dict(kvPool=None), INVALID), (dict(pageTable=None), INVALID), (dict(indices=None), INVALID),
    (dict(contextLengths=None), INVALID), (dict(batchSize=0), INVALID), (dict(seqLen=0), INVALID), (dict(topK=0), INVALID),
    (dict(numQHeads=7), INVALID), (dict(numFlatPages=0), INVALID), (dict(maxPagesPerSeq=0), INVALID),
    (dict(poolRowBytes=64), INVALID), (dict(headDim=64), UNSUPPORTED), (dict(numQHeads=34), UNSUPPORTED),
    (dict(poolRowBytes=88), UNSUPPORTED), (dict(topK=(1 << 24) + 1), UNSUPPORTED), (dict(qPtr=FAKE + 8), UNSUPPORTED),
    (dict(kvPool=FAKE + 4), UNSUPPORTED), (dict(lse=FAKE + 2), UNSUPPORTED), (dict(indices=FAKE + 1), UNSUPPORTED),
    (dict(batchSize=1 << 16, seqLen=1 << 15), UNSUPPORTED), (dict(batchSize=1 << 15, seqLen=1 << 15), UNSUPPORTED),
    (dict(maxPagesPerSeq=1 << 24), UNSUPPORTED), (dict(numFlatPages=1 << 24), UNSUPPORTED)]


@pytest.mark.parametrize("change,want", READER_REFUSALS + [(dict(oPtr=None), INVALID), (dict(oPtr=FAKE + 2), UNSUPPORTED)])
def test_attend_refusals(qb, change, want):
    refuses(qb, "QsaSparsePagedKv4Params", ATTEND, change, want)


@pytest.mark.parametrize("change,want", READER_REFUSALS + [
    (dict(lse=None), INVALID), (dict(weights=None), INVALID), (dict(total=None), INVALID), (dict(totalLen=0), INVALID),
    (dict(totalLen=-1), INVALID), (dict(weights=FAKE + 2), UNSUPPORTED), (dict(total=FAKE + 1), UNSUPPORTED),
    (dict(totalLen=(1 << 24) + 1), UNSUPPORTED)])
def test_weights_refusals(qb, change, want):
    refuses(qb, "QsaSparseWeightsKv4Params", WEIGHTS, change, want)


@pytest.mark.parametrize("change,want", [
    (dict(kvPool=None), INVALID), (dict(pageTable=None), INVALID), (dict(contextLengths=None), INVALID),
    (dict(total=None), INVALID), (dict(kept=None), INVALID), (dict(keptLengths=None), INVALID),
    (dict(keptLengths=FAKE), INVALID), (dict(batchSize=0), INVALID), (dict(numKVHeads=0), INVALID), (dict(totalLen=0), INVALID),
    (dict(budget=0), INVALID), (dict(sinks=-1), INVALID), (dict(recent=-1), INVALID), (dict(sinks=60), INVALID),
    (dict(sinks=1 << 30, recent=1 << 30), INVALID), (dict(poolRowBytes=64), INVALID), (dict(headDim=64), UNSUPPORTED),
    (dict(poolRowBytes=90), UNSUPPORTED), (dict(kvPool=FAKE + 8), UNSUPPORTED), (dict(kept=FAKE + 2), UNSUPPORTED),
    (dict(totalOut=FAKE + 1), UNSUPPORTED), (dict(batchSize=1 << 27), UNSUPPORTED), (dict(maxPagesPerSeq=1 << 24), UNSUPPORTED),
    (dict(numFlatPages=1 << 24), UNSUPPORTED), (dict(totalLen=(1 << 24) + 1), UNSUPPORTED),
    (dict(budget=(1 << 24) + 1), UNSUPPORTED)])
def test_evict_refusals(qb, change, want):
    refuses(qb, "QsaEvictKv4Params", ("qsa_evict_kv4",), change, want)


def test_frequencies(qb):
    """Each scaling against its formula, pair by pair."""
    rot, theta, factor, length = 64, 1e4, 8.0, 8192.0
    plain = [theta ** (-2.0 * i / rot) for i in range(rot // 2)]
    turns = [length * f / (2 * math.pi) for f in plain]
    low, high = 1.0, 32.0
    # pair at which n turns are made: length theta^(-2i/rot) / (2 pi) = n
    pair = [rot / 2 * math.log(length / (2 * math.pi * n)) / math.log(theta) for n in (high, low)]
    first, last = math.floor(pair[0]), math.ceil(pair[1])

    def mean(s, f):
        s = min(1.0, max(0.0, s))
        return s * f + (1 - s) * f / factor

    want = {"plain": plain, "linear": [f / factor for f in plain],
            "base": [(theta * factor ** (rot / (rot - 2))) ** (-2.0 * i / rot) for i in range(rot // 2)],
            "blend": [mean((n - low) / (high - low), f) for n, f in zip(turns, plain)],
            "ramp": [mean((last - i) / (last - first), f) for i, f in enumerate(plain)]}
    for s, w in want.items():
        got = qb.rotary_frequencies(rot, theta=theta, scaling=s, factor=factor, original_length=length, low_turns=low,
                                    high_turns=high).tolist()
        assert got == pytest.approx(w, rel=1e-13), s
    assert want["base"][0] == 1.0 and want["base"][-1] == pytest.approx(plain[-1] / factor, rel=1e-12)
    assert qb.rotary_frequencies(2, theta=1e4).tolist() == [1.0]


@pytest.mark.parametrize("change", [
    dict(rot=0), dict(rot=7), dict(rot=2, scaling="base"), dict(theta=1.0), dict(theta=float("inf")), dict(theta=float("nan")),
    dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=float("nan")), dict(scaling="blend", original_length=0.0),
    dict(scaling="ramp", low_turns=0.0), dict(scaling="ramp", low_turns=32.0), dict(scaling="blend", high_turns=float("inf"))])
def test_frequency_refusals(qb, change):
    kw = dict(rot=16, theta=1e4, scaling="plain", factor=2.0, original_length=4096.0, low_turns=1.0, high_turns=32.0)
    kw.update(change)
    with pytest.raises(qb.QsaError):
        qb.rotary_frequencies(kw.pop("rot"), **kw)
    with pytest.raises(ValueError):
        qb.rotary_frequencies(16, theta=1e4, scaling="other")
    assert qb.lib().qsa_rotary_frequencies(9, 16, 1e4, 2.0, 1.0, 1.0, 2.0, ctypes.addressof(FREQ)) == INVALID


def test_binding_refuses(qb):
    h, i32 = torch.float16, torch.int32
    x, pos, f = torch.zeros(5, 3, 64, dtype=h), torch.zeros(5, dtype=i32), torch.ones(16, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        qb.rotary(x, pos, x, f)
    with pytest.raises(ValueError, match="float16, bfloat16 or float32"):
        qb.rotary(x.double(), pos, x, f)
    with pytest.raises(ValueError, match="positions"):
        qb.rotary(x, pos[:4], x, f)
    with pytest.raises(ValueError, match="float64"):
        qb.rotary(x, pos, x, f.float())
    with pytest.raises(ValueError, match="float64"):
        qb.rotary(x, pos, x, torch.ones(32, dtype=torch.float64)[::2])
    kv, ctx, pt = torch.zeros(2, 3, 2, 128, dtype=h), torch.zeros(2, dtype=i32), torch.zeros(2, 2, 4, dtype=i32)
    pool, q = torch.zeros(16, 128, 2, 80, dtype=torch.uint8), torch.zeros(2, 3, 8, 128, dtype=h)
    lists, lse, w = torch.zeros(2, 3, 5, dtype=i32), torch.zeros(2, 3, 8), torch.zeros(2, 3, 2, 5)
    total, kept = torch.zeros(2, 2, 512), torch.zeros(2, 2, 64, dtype=i32)
    calls = {
        "store": (lambda **k: qb.store_kv4(**{**dict(k=kv, v=kv, ctx=ctx, pool=pool, page_table=pt), **k}),
                  [dict(k=kv.float()), dict(v=kv[:, :2]), dict(ctx=ctx[:1]), dict(page_table=pt[:1]),
                   dict(pool=pool[:, :64]), dict(k_out=q), dict(new_lengths=ctx[:1]), dict(page_table=pt[:, :1])]),
        "attend": (lambda **k: qb.sparse_paged_kv4(**{**dict(q=q, pool=pool, page_table=pt, indices=lists, ctx=ctx, out=q,
                                                            scale=0.1), **k}),
                   [dict(q=q.float()), dict(out=kv), dict(lse=lse[:, :2]), dict(indices=lists[:, :2]), dict(indices=lists[0]),
                    dict(ctx=ctx[:1]), dict(pool=pool[0])]),
        "weights": (lambda **k: qb.sparse_weights_kv4(**{**dict(q=q, pool=pool, page_table=pt, indices=lists, ctx=ctx, lse=lse,
                                                               weights=w, total=total, scale=0.1), **k}),
                    [dict(q=q.float()), dict(lse=lse[..., :4]), dict(weights=w[..., :4]), dict(total=total[:, :1])]),
        "evict": (lambda **k: qb.evict_kv4(**{**dict(pool=pool, page_table=pt, ctx=ctx, total=total, kept=kept,
                                                    kept_lengths=ctx), **k}),
                  [dict(total=total[:1]), dict(kept=kept[0]), dict(total_out=total[..., :4]), dict(kept_lengths=ctx[:1])]),
    }
    for call, bad in calls.values():
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
        for change in bad:
            with pytest.raises(ValueError):
                call(**change)


def test_rotary_refuses_what_autograd_would_lose(qb):
    """The call records nothing: a tensor whose gradient would be dropped without a word is refused, in place or not; with
    gradients disabled it goes on (here to the next check, the device's)."""
    x, pos, f = torch.zeros(5, 3, 64), torch.zeros(5, dtype=torch.int32), torch.ones(16, dtype=torch.float64)
    leaf = x.clone().requires_grad_()
    computed = leaf * 2
    for a, out in ((leaf, x), (computed, x), (computed, computed), (computed[:, :2], x[:, :2]), (x, leaf), (x, computed)):
        with pytest.raises(ValueError, match="gradient"):
            qb.rotary(a, pos, out, f)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA tensor"):
            qb.rotary(a, pos, out, f)
    with pytest.raises(ValueError, match="CUDA tensor"):
        qb.rotary(computed.detach(), pos, x, f)
