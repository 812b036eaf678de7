"""qsa_append_kv / qsa_append_kv8 (fp16 and bf16) against plain 64-bit forms.

Bars.  A dense output or 16-bit pool value is the fp32 evaluation rounded once: within one step of its type of the
64-bit value's rounding, plus the evaluation's own error, 2^-18 for normalised values up to about 6 (a few units of
2^-24 of each operand).  V values are copies.  A scale is amax / 448 within 2^-18 / 448 plus two fp32 roundings; a code
times its scale is within half an e4m3 step of the value (2^-4 relative, 2^-10 scales absolute) plus the same 2^-18."""
from __future__ import annotations

import pytest
import torch

import paged_cache_ref as ref
from block_sparse_gqa_qsa_gb300 import _binding as qb

pytestmark = pytest.mark.gpu
DEV = "cuda"
EVAL = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_gqa_qsa_gb300 import build
    build.build()
    qb.lib()


def make(dtype, D, Hq, Hkv, S, ctx, new, block, extra=0, tail=0, seed=0):
    """Inputs on the CPU; padding rows are NaN, the cache holds random values."""
    g = torch.Generator().manual_seed(100 + seed)
    B = len(ctx)
    n = ref.new_rows(ctx, new, S)
    qkv = torch.randn((B, S, Hq + 2 * Hkv, D), generator=g).to(dtype)
    for b in range(B):
        qkv[b, n[b]:] = float("nan")
    pt, flat = ref.page_tables(ctx, 7 + seed, extra)
    c = dict(qkv=qkv, wq=0.1 * torch.randn(D, generator=g), wk=0.1 * torch.randn(D, generator=g),
             ctx=torch.tensor(ctx, dtype=torch.int32), pt=pt, n=n,
             new=None if new is None else torch.tensor(new, dtype=torch.int32), Hq=Hq, Hkv=Hkv, S=S, D=D, block=block)
    if block:
        c["pool"] = ref.random_codes((flat, 128, Hkv, D + tail), 9 + seed)
        c["scale"] = 0.0078 * torch.exp(0.3 * torch.randn((flat, 128 // block, Hkv), generator=g))
    else:
        c["pool"] = torch.randn((flat, 128, Hkv, D + tail), generator=g).to(dtype)
    return c


def run(c, rot, dense=True, status=None, stream=None, eps=ref.EPS):
    """The call on the GPU; returns q, k, v, pool, scale on the CPU."""
    B, S, D, Hq, Hkv = len(c["n"]), c["S"], c["D"], c["Hq"], c["Hkv"]
    et = c["qkv"].dtype
    q = torch.full((B, S, Hq, D), float("nan"), dtype=et, device=DEV)
    k, v = (torch.full((B, S, Hkv, D), float("nan"), dtype=et, device=DEV) if dense else None for _ in range(2))
    pool = c["pool"].to(DEV)
    new = None if c["new"] is None else c["new"].to(DEV)
    kw = dict(Hq=Hq, Hkv=Hkv, rot=rot, theta=ref.THETA, eps=eps, new_lengths=new, k_out=k, v_out=v, status=status,
              stream=stream)
    a = (c["qkv"].to(DEV), c["wq"].to(DEV), c["wk"].to(DEV), c["ctx"].to(DEV), q, pool)
    if c["block"]:
        scale = c["scale"].to(DEV)
        qb.append_kv8(*a, scale, c["pt"].to(DEV), **kw)
    else:
        scale = None
        qb.append_kv(*a, c["pt"].to(DEV), **kw)
    torch.cuda.synchronize()
    return [None if t is None else t.cpu() for t in (q, k, v, pool, scale)]


def step_of(x, dtype):
    """One step of a 16-bit type at |x| (float64)."""
    bits, low = (11, -24) if dtype == torch.float16 else (8, -133)
    _, e = torch.frexp(x.abs())
    return torch.ldexp(torch.ones_like(x), (e - bits).clamp(min=low))


def check_dense(got, want, dtype):
    bar = step_of(want, dtype) + EVAL
    err = (got.double() - want).abs()
    assert bool((err <= bar).all()), float((err - bar).max())


def check(c, rot, out, dense=True, skip=()):
    """Every output of a call against 64 bits; `skip`: (b, plane, page index) whose rows must not be written."""
    q, k, v, pool, scale = out
    B, S, D, Hq, Hkv, blk = len(c["n"]), c["S"], c["D"], c["Hq"], c["Hkv"], c["block"]
    et = c["qkv"].dtype
    bytes_before, bytes_after = c["pool"].view(torch.uint8).flatten(-1), pool.view(torch.uint8)
    allowed = torch.zeros(pool.shape, dtype=torch.bool)  # elements a call may write
    scales_allowed = torch.zeros(c["scale"].shape, dtype=torch.bool) if blk else None
    for b in range(B):
        n, L = c["n"][b], int(c["ctx"][b])
        start = L - n
        for t in (q, k, v) if dense else (q,):
            assert not t[b, n:].view(torch.int16).any(), "padding rows are zeros"
        if n == 0:
            continue
        x = c["qkv"][b, :n]
        pos = torch.arange(start, L)
        wantq = ref.normed_rotated(x[:, :Hq], c["wq"], pos, rot)
        wantk = ref.normed_rotated(x[:, Hq:Hq + Hkv], c["wk"], pos, rot)
        check_dense(q[b, :n], wantq, et)
        if dense:
            check_dense(k[b, :n], wantk, et)
            assert torch.equal(v[b, :n].view(torch.int16), x[:, Hq + Hkv:].contiguous().view(torch.int16))
        for plane, want in ((0, wantk), (1, x[:, Hq + Hkv:].double())):
            live = [i for i in range(n) if (b, plane, (start + i) // 128) not in skip]
            if not live:
                continue
            live = torch.tensor(live)
            p = pos[live]
            page, off = c["pt"][b, plane, p // 128].long(), p % 128
            allowed[page, off, :, :D] = True
            rows = pool[page, off, :, :D] if not blk else None
            if not blk:
                if plane:
                    assert torch.equal(rows.view(torch.int16), x[live][:, Hq + Hkv:].contiguous().view(torch.int16))
                else:
                    check_dense(rows, want[live], et)
                    if dense:
                        assert torch.equal(rows.view(torch.int16), k[b, live].view(torch.int16))
                continue
            s = scale[page, off // blk].double()
            codes = ref.E4M3[bytes_after[page, off][..., :D].long()]
            err = (codes * s[..., None] - want[live]).abs()
            bar = torch.maximum(2.0 ** -4 * want[live].abs(), 2.0 ** -10 * s[..., None].expand_as(err)) + EVAL
            assert bool((err <= bar).all()), float((err - bar).max())
            first = start // blk
            for i in sorted({int(y) // blk for y in p}):
                mine = live[(p // blk) == i]
                amax = want[mine].abs().amax((0, 2))
                pg, at = int(c["pt"][b, plane, i * blk // 128]), (i * blk % 128) // blk
                scales_allowed[pg, at] = True
                got, had = scale[pg, at].double(), c["scale"][pg, at].double()
                if i > first or start % blk == 0:
                    expect = (amax / 448).clamp(2.0 ** -48, 2.0 ** 48)
                    assert bool(((got - expect).abs() <= EVAL / 448 + 2.0 ** -22 * expect).all())
                    continue
                up = torch.log2(got / had)
                assert torch.equal(up, up.round()) and bool((up >= 0).all()), "older blocks grow by powers of two"
                assert bool((amax <= 448 * got * (1 + 2.0 ** -20) + EVAL).all()), "the new tokens fit"
                assert bool(((up == 0) | (amax > 224 * got * (1 - 2.0 ** -20) - EVAL)).all()), "no more than needed"
                old = torch.arange(i * blk, start) % 128
                if old.numel():
                    allowed[pg, old, :, :D] = True
                    was = ref.E4M3[c["pool"].view(torch.uint8)[pg, old][..., :D].long()] * (had / got)[:, None]
                    is_ = ref.E4M3[bytes_after[pg, old][..., :D].long()]
                    exact = was.abs() >= 2.0 ** -6
                    assert torch.equal(was[exact], is_[exact]), "a power of two is exact in e4m3's normal range"
                    assert bool(((was - is_).abs() <= 2.0 ** -10).all())
    same = c["pool"].view(torch.uint8) == bytes_after if blk else c["pool"].view(torch.int16) == pool.view(torch.int16)
    assert bool(same[~allowed].all()), "only the new tokens' rows and their blocks change"
    if blk:
        assert torch.equal(scale[~scales_allowed], c["scale"][~scales_allowed])


ONE = dict(S=1, ctx=(1, 16, 17, 128, 5000, 0), new=None)
CHUNK = dict(S=41, ctx=(41, 140, 1033, 300, 12, 0, 77), new=(41, 37, 1, 0, 41, 5, -3))  # page ends inside, n > ctx, n < 0
WHOLE = dict(S=301, ctx=(301, 1, 150), new=None)


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("rows", (ONE, CHUNK, WHOLE), ids=("one", "chunk", "whole"))
@pytest.mark.parametrize("block", (0, 1, 16, 128))
def test_append(dtype, rows, block):
    c = make(dtype, 128, 8, 2, rows["S"], rows["ctx"], rows["new"], block, extra=2, tail=32, seed=block)
    check(c, 64, run(c, 64))


@pytest.mark.parametrize("block", (0, 2, 4, 8, 32, 64))
@pytest.mark.parametrize("D,rot,Hq,Hkv", [(64, 32, 7, 1), (64, 0, 1, 1), (128, 128, 24, 2), (128, 16, 33, 3),
                                          (128, 0, 16, 16), (64, 64, 64, 8)])
def test_append_heads(block, D, rot, Hq, Hkv):
    c = make(torch.float16, D, Hq, Hkv, 70, (70, 133, 700), (33, 70, 70), block, seed=D + rot + block)
    out = run(c, rot, dense=False)
    check(c, rot, out, dense=False)


@pytest.mark.parametrize("S", (2, 5, 15, 16, 17))
@pytest.mark.parametrize("D,block", [(128, 0), (64, 16), (128, 8), (64, 64)])
def test_append_short_chunks(S, D, block):
    """Chunks shorter than a warp's group of rows, at every offset of a block."""
    ctx = tuple(200 + 3 * i for i in range(12))
    c = make(torch.bfloat16, D, 5, 1, S, ctx, (S,) * 12, block, tail=16, seed=S + D)
    check(c, 32, run(c, 32))


def test_append_many_sequences():
    """More sequences than CTAs at once, one token each."""
    c = make(torch.float16, 128, 2, 1, 1, tuple(1 + (7 * i) % 100 for i in range(1500)), None, 16, seed=6)
    check(c, 64, run(c, 64))


@pytest.mark.parametrize("block", (0, 16, 32))
def test_append_many_heads(block):
    """More K and V heads than a CTA shares a wide block's maxima of."""
    c = make(torch.float16, 64, 3, 270, 3, (3, 37), (3, 2), block, seed=7)
    check(c, 32, run(c, 32, dense=False), dense=False)


@pytest.mark.parametrize("block", (0, 16, 64))
def test_append_again(block):
    """The same tokens a second time, as after a rejected draft, leave the same cache and scales."""
    c = make(torch.float16, 128, 8, 2, 20, (20, 75), (20, 20), block, seed=13)
    c["qkv"][:, :, 10:] *= 50  # V outgrows the older tokens' scale
    first = run(c, 64)
    c["pool"] = first[3]
    if block:
        c["scale"] = first[4]
    again = run(c, 64)
    for a, b in zip(first, again):
        assert (a is None and b is None) or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_append_many_tiles():
    """More tiles than the GPU holds at once, and a whole prompt far from position 0."""
    c = make(torch.bfloat16, 128, 8, 1, 2100, (2100, 65536, 1999, 2100), (2100, 2100, 1999, 700), 16, seed=5)
    check(c, 64, run(c, 64))


@pytest.mark.parametrize("block", (4, 16, 64))
def test_growing_blocks(block):
    """Tokens one at a time, each three times larger than the one before: every block's scale grows as it fills."""
    c = make(torch.float16, 128, 4, 2, 1, (1, 60), None, block, extra=4, seed=3)
    for i in range(11):
        check(c, 32, (out := run(c, 32)))
        c["pool"], c["scale"] = out[3], out[4]
        c["ctx"] = c["ctx"] + 1
        c["qkv"] = torch.randn(c["qkv"].shape, generator=torch.Generator().manual_seed(i)).half()
        c["qkv"][:, :, 6:] *= min(3.0 ** i, 8000.0)  # V; K is normed, so its scales hardly grow


def test_zeros_then_values():
    """A block of zeros has the smallest scale; the first real token in it grows it and leaves the zeros zero."""
    c = make(torch.float16, 128, 4, 1, 3, (3,), None, 16)
    c["qkv"][:, :, 4:] = 0
    out = run(c, 0)
    check(c, 0, out)
    assert float(out[4][int(c["pt"][0, 1, 0]), 0, 0]) == 2.0 ** -48
    c["pool"], c["scale"], c["ctx"] = out[3], out[4], torch.tensor([4], dtype=torch.int32)
    c["new"], c["n"] = torch.tensor([1], dtype=torch.int32), [1]
    c["qkv"] = torch.randn(c["qkv"].shape, generator=torch.Generator().manual_seed(1)).half()
    c["qkv"][:, 1:] = float("nan")
    out = run(c, 0)
    check(c, 0, out)
    assert not ref.E4M3[out[3].view(torch.uint8)[int(c["pt"][0, 1, 0]), :3].long()].any()


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
def test_values_that_are_no_numbers(dtype):
    """NaN and infinite V values are stored as NaN and do not enter the scale; their neighbours are unharmed."""
    c = make(dtype, 128, 4, 2, 20, (20,), None, 16)
    clean = run(c, 64)
    c["qkv"][0, 3, 6, 5], c["qkv"][0, 9, 7, 0] = float("inf"), float("nan")
    c["qkv"][0, 17, 6, 127] = float("-inf")
    q, k, v, pool, scale = run(c, 64)
    page = int(c["pt"][0, 1, 0])
    codes = pool.view(torch.uint8)[page, :20, :, :128] & 0x7f
    bad = torch.zeros(20, 2, 128, dtype=torch.bool)
    bad[3, 0, 5] = bad[9, 1, 0] = bad[17, 0, 127] = True
    assert bool((codes[bad] == 0x7f).all()) and not bool((codes[~bad] == 0x7f).any())
    finite = torch.where(torch.isfinite(c["qkv"][0, :, 6:].float()), c["qkv"][0, :, 6:].float().abs(), torch.zeros(()))
    want = torch.stack([finite[:16].amax((0, 2)), finite[16:].amax((0, 2))]) / 448
    assert torch.equal(scale[page, :2], want)
    assert torch.equal(k.view(torch.int16), clean[1].view(torch.int16))


def test_large_bf16_values():
    """Squares past fp32's range: the norm of rows of 1e30 is that of rows of 1."""
    c = make(torch.bfloat16, 128, 4, 1, 5, (5,), None, 0)
    small = run(c, 64)
    c["qkv"] = (c["qkv"].float() * 2.0 ** 100).bfloat16()
    big = run(c, 64)
    # eps is 1e-6 of a mean square near 1: 5e-7 relative, under a quarter of which rounds differently
    err = (big[0].double() - small[0].double()).abs()
    assert bool((err <= step_of(small[0].double(), torch.bfloat16)).all())


@pytest.mark.parametrize("e,eps", [(-110, 0.0), (-60, 1e-37)])
@pytest.mark.parametrize("block", (0, 16))
def test_small_bf16_values(block, e, eps):
    """Squares below fp32's range without an eps, and near its end with one of their size."""
    c = make(torch.bfloat16, 128, 4, 1, 9, (9,), None, block)
    rows = c["qkv"][0].double()
    c["qkv"] = (c["qkv"].float() * 2.0 ** e).bfloat16()  # exact
    q, k = run(c, 64, eps=eps)[:2]
    # the same numbers from rows scaled so that EPS is to them what eps is to these (for 0: 2^-100 of their mean square)
    f = 2.0 ** e * (ref.EPS / eps) ** 0.5 if eps else 2.0 ** 40
    for got, want in ((q, ref.normed_rotated(rows[:, :4] * f, c["wq"], torch.arange(9), 64)),
                      (k, ref.normed_rotated(rows[:, 4:5] * f, c["wk"], torch.arange(9), 64))):
        check_dense(got[0], want, torch.bfloat16)


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("block", (0, 16))
def test_rows_that_are_no_numbers(block, dtype):
    """A q or k row with an infinity or a NaN comes out as NaN; its neighbours are unharmed, in an 8-bit block too."""
    c = make(dtype, 128, 4, 2, 20, (20,), None, block)
    clean = run(c, 64)
    c["qkv"][0, 3, 1, 100], c["qkv"][0, 9, 4, 7] = float("inf"), float("nan")
    q, k, v, pool, scale = run(c, 64)
    assert bool(q[0, 3, 1].isnan().all()) and bool(k[0, 9, 0].isnan().all())
    for got, was, at in ((q, clean[0], (0, 3, 1)), (k, clean[1], (0, 9, 0))):
        got[at], was = 0, was.clone()
        was[at] = 0
        assert torch.equal(got.view(torch.int16), was.view(torch.int16))
    page = int(c["pt"][0, 0, 0])
    row = pool.view(torch.uint8)[page, 9, 0, :128] & 0x7f if block else pool[page, 9, 0, :128]
    assert bool((row == 0x7f).all()) if block else bool(row.isnan().all())
    if block:
        amax = k[0, :16, 0].double().abs().amax()  # the NaN row was set to zeros above
        assert abs(float(scale[page, 0, 0]) - float(amax) / 448) <= step_of(amax, dtype) / 448


def test_calls_from_many_threads():
    """Calls whose kernels need different amounts of shared memory, from several threads at once."""
    import ctypes
    import threading
    cases = [(make(torch.float16, 128, 4, 2, 140, (140,), None, 128, seed=20), 128),
             (make(torch.float16, 128, 4, 2, 40, (140,), None, 16, seed=21), 16)]
    want = [run(c, rot, dense=False)[0] for c, rot in cases]
    fn = qb.lib().qsa_append_kv8
    bad = []

    def loop(i):
        c, rot = cases[i % 2]
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            t = {n: c[n].to(DEV) for n in ("qkv", "wq", "wk", "ctx", "pool", "scale", "pt")}
            q = torch.empty((1, c["S"], 4, 128), dtype=torch.float16, device=DEV)
        st.synchronize()
        p = qb.QsaAppendKvParams(
            qkv=t["qkv"].data_ptr(), qNormW=t["wq"].data_ptr(), kNormW=t["wk"].data_ptr(),
            contextLengths=t["ctx"].data_ptr(), qOut=q.data_ptr(), kvPool=t["pool"].data_ptr(),
            kvScale=t["scale"].data_ptr(), pageTable=t["pt"].data_ptr(), batchSize=1, seqLen=c["S"], numQHeads=4,
            numKVHeads=2, headDim=128, rotDim=rot, poolHeadDim=128, numFlatPages=c["pool"].shape[0],
            maxPagesPerSeq=c["pt"].shape[2], scaleBlock=c["block"], ropeTheta=ref.THETA, rmsNormEps=ref.EPS,
            stream=st.cuda_stream)
        errors = sum(fn(ctypes.byref(p)) != 0 for _ in range(10000))
        st.synchronize()
        if errors or not torch.equal(q.cpu().view(torch.int16), want[i % 2].view(torch.int16)):
            bad.append((i, errors))

    threads = [threading.Thread(target=loop, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


@pytest.mark.parametrize("block", (0, 16, 64))
def test_bad_pages(block):
    """Page ids outside the pool and positions behind the table: skipped, reported, the rest written."""
    c = make(torch.float16, 128, 4, 2, 300, (300, 200), None, block, seed=8)
    flat = c["pool"].shape[0]
    c["pt"][0, 0, 1], c["pt"][1, 1, 0] = -1, flat
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = run(c, 64, status=status)
    assert int(status) == 2
    check(c, 64, out, skip={(0, 0, 1), (1, 1, 0)})
    c = make(torch.float16, 128, 4, 2, 300, (300, 200), None, block, seed=9)
    c["pt"] = c["pt"][:, :, :2].contiguous()  # tokens 256 .. 299 have no entry
    status.zero_()
    out = run(c, 64, status=status)
    assert int(status) == 2
    check(c, 64, out, skip={(0, 0, 2), (0, 1, 2)})
    status.zero_()
    c = make(torch.float16, 128, 4, 2, 30, (30, 20), None, block, seed=9)
    check(c, 64, run(c, 64, status=status))
    assert int(status) == 0


def test_pool_beyond_4_gib():
    """Rows past 2^32 bytes."""
    flat, Hkv, D = 34000, 8, 128  # 4.46e9 bytes
    pool = torch.zeros((flat, 128, Hkv, D), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    scale = torch.ones((flat, 8, Hkv), device=DEV)
    g = torch.Generator().manual_seed(4)
    qkv = torch.randn((1, 4, 8 + 2 * Hkv, D), generator=g).half()
    pt = torch.tensor([[[5], [flat - 1]]], dtype=torch.int32)
    ctx = torch.tensor([4], dtype=torch.int32)
    q = torch.empty((1, 4, 8, D), dtype=torch.float16, device=DEV)
    w = torch.zeros(D, device=DEV)
    qb.append_kv8(qkv.to(DEV), w, w, ctx.to(DEV), q, pool, scale, pt.to(DEV), Hq=8, Hkv=Hkv, rot=64, theta=1e4, eps=1e-6)
    v = qkv[0, :, 8 + Hkv:].double()
    s = scale[flat - 1, 0].cpu().double()
    got = ref.E4M3[pool[flat - 1, :4].view(torch.uint8).cpu().long()] * s[:, None]
    assert torch.equal(s.float(), (v.abs().amax((0, 2)) / 448).float())
    assert bool(((got - v).abs() <= torch.maximum(2.0 ** -4 * v.abs(), 2.0 ** -10 * s[:, None].expand_as(v)) + 2.0 ** -22 * v.abs()).all())
    assert int(pool.view(torch.uint8)[6:flat - 1].max()) == 0


def test_append_equals_rope():
    """Where qsa_rope_qkv applies (fp16, from position 0 or one token) the 16-bit append writes what it writes, within
    the two kernels' evaluation errors."""
    c = make(torch.float16, 128, 8, 2, 200, (200, 77), None, 0, seed=12)
    q, k, v, pool, _ = run(c, 64)
    rq, rk, rv = (torch.empty_like(t, device=DEV) for t in (q, k, v))
    rpool = c["pool"].to(DEV)
    qb.rope_qkv(c["qkv"].to(DEV), c["wq"].to(DEV), c["wk"].to(DEV), c["ctx"].to(DEV), rq, Hq=8, Hkv=2, rot=64, theta=1e4,
                eps=1e-6, k_out=rk, v_out=rv, pool=rpool, page_table=c["pt"].to(DEV))
    for a, r in ((q, rq), (k, rk), (v, rv), (pool, rpool)):
        bar = step_of(a.double(), torch.float16) + EVAL
        assert bool(((a.double() - r.cpu().double()).abs() <= bar).all())


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("block", (1, 4, 16, 32, 128))
def test_values_halfway_between_codes(dtype, block):
    """Values that lie exactly halfway between two codes of their block take the even one, for scales that have no exact
    reciprocal.  Head h has the scale s = k 2^-6, k = 3, 5, 7 .., in every block: its largest value is 7 k = 448 s.  The
    others are k t 2^(e - 6), in units of s the odd t = 17 .. 31 (5 bits where a code has 4) times 2^e.  All are exact in
    the input's type, and so is the quotient."""
    bits = 11 if dtype == torch.float16 else 8
    ks = (3, 5, 7, 9, 11, 13, 15) if dtype == torch.float16 else (3, 5, 7)
    c = make(dtype, 128, 2, len(ks), 20, (40,), (20,), block, seed=30)  # tokens 20 .. 39, some behind older ones of a block
    c["scale"][:] = torch.tensor(ks) * 2.0 ** -6
    for h, k in enumerate(ks):
        odd = [t for t in range(17, 32, 2) if k * t < 2 ** bits]
        units = torch.tensor([t * 2.0 ** e for t in odd for e in range(-9, 5) if t * 2.0 ** e < 448], dtype=torch.float64)
        pick = torch.randint(len(units), (20, 128), generator=torch.Generator().manual_seed(h))
        v = units[pick] * torch.where(pick % 2 == 0, 1.0, -1.0) * k * 2.0 ** -6
        v[:, 5] = 7.0 * k
        assert torch.equal(v.to(dtype).double(), v)
        c["qkv"][0, :, 2 + len(ks) + h] = v.to(dtype)
    out = run(c, 64)
    check(c, 64, out)
    pos = torch.arange(20, 40)
    s = out[4][c["pt"][0, 1, 0].long(), pos // block].double()  # [token, head]
    assert torch.equal(s, torch.tensor(ks).double().expand(20, -1) * 2.0 ** -6)
    got = ref.E4M3[out[3].view(torch.uint8)[int(c["pt"][0, 1, 0]), pos].long()]
    x = c["qkv"][0, :, 2 + len(ks):].double() / s[..., None]  # exact
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), e - 4)  # every value lies in the normal range
    assert torch.equal(got, torch.round(x / step) * step)


@pytest.mark.parametrize("D", (64, 128))
@pytest.mark.parametrize("block", (0, 16, 32))
def test_largest_bf16_values(D, block):
    """q and k rows of bf16's largest values: all of a row, half of it, one element, and rows at 2^64 and 2^120 beside
    them.  The sum of the squares passes fp32's range by far, the norm does not."""
    c = make(torch.bfloat16, D, 4, 2, 40, (40,), None, block, seed=31)
    top = float(torch.finfo(torch.bfloat16).max)
    g = torch.Generator().manual_seed(32)
    x = c["qkv"][0, :, :6]
    sign = torch.where(torch.rand(x.shape, generator=g) < 0.5, -1.0, 1.0)
    big = sign * top * (1 - torch.rand(x.shape, generator=g) / 2)
    big[0:4] = sign[0:4] * top
    big[4:8, :, ::2] = 1.0
    big[8:12, :, 1:] = x[8:12, :, 1:].float()
    big[12:16] = x[12:16].float() * 2.0 ** 64
    big[16:20] = x[16:20].float() * 2.0 ** 120
    c["qkv"][0, :, :6] = big.bfloat16()
    assert bool(torch.isfinite(c["qkv"]).all())
    check(c, 32, run(c, 32))
