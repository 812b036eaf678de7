"""qsa_sparse_paged_kv8 (fp16 and bf16) against plain 64-bit attention over the dequantised cache, and the append,
indexer and attention calls together.  The bar of every output is `paged_cache_ref.attend_bar`."""
from __future__ import annotations

import math

import pytest
import torch

import paged_cache_ref as ref
from block_sparse_gqa_qsa_gb300 import _binding as qb
from block_sparse_gqa_qsa_gb300 import synthetic as syn

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 128
SCALE = float(torch.tensor(1 / math.sqrt(D), dtype=torch.float32))


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_gqa_qsa_gb300 import build
    build.build()
    qb.lib()


def make(dtype, Hq, Hkv, S, ctx, new, topK, block, tail=0, seed=0, fill=1.0):
    g = torch.Generator().manual_seed(300 + seed)
    B = len(ctx)
    n = ref.new_rows(ctx, new, S)
    pt, flat = ref.page_tables(ctx, 17 + seed, extra=1)
    q = torch.randn((B, S, Hq, D), generator=g).to(dtype)
    lists = torch.full((B, S, topK), -1, dtype=torch.int32)
    for b in range(B):
        q[b, n[b]:] = float("nan")
        for t in range(n[b]):
            span = int(ctx[b]) - n[b] + t + 1
            m = min(span, max(1, round(fill * topK)))
            lists[b, t, :m] = torch.randperm(span, generator=g)[:m].to(torch.int32)
    return dict(q=q, pool=ref.random_codes((flat, 128, Hkv, D + tail), 19 + seed),
                scale=0.0078 * torch.exp(0.3 * torch.randn((flat, 128 // block, Hkv), generator=g)), pt=pt, lists=lists,
                ctx=torch.tensor(ctx, dtype=torch.int32), n=n,
                new=None if new is None else torch.tensor(new, dtype=torch.int32))


def run(c, scale=SCALE, status=None):
    out = torch.full(c["q"].shape, float("nan"), dtype=c["q"].dtype, device=DEV)
    qb.sparse_paged_kv8(c["q"].to(DEV), c["pool"].to(DEV), c["scale"].to(DEV), c["pt"].to(DEV), c["lists"].to(DEV),
                        c["ctx"].to(DEV), out, scale=scale, new_lengths=None if c["new"] is None else c["new"].to(DEV),
                        status=status)
    torch.cuda.synchronize()
    return out.cpu()


def check(c, out, scale=SCALE, lists=None):
    lists = c["lists"] if lists is None else lists
    for b, n in enumerate(c["n"]):
        assert not out[b, n:].view(torch.int16).any(), "padding rows are zeros"
        if n == 0:
            continue
        L = int(c["ctx"][b])
        k, v = (ref.dequantised(c["pool"], c["scale"], c["pt"][b, i], L) for i in (0, 1))
        want, mean_abs, dots = ref.attend(c["q"][b, :n], k, v, lists[b, :n], scale)
        bar = ref.attend_bar(want, mean_abs, dots, lists[b, 0], c["scale"], out.dtype)
        err = (out[b, :n].double() - want).abs()
        assert bool((err <= bar).all()), (b, float((err / bar).max()))


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 1), (8, 2), (14, 2), (24, 2), (64, 4), (16, 16)])
@pytest.mark.parametrize("topK,block", [(67, 16), (1, 1), (333, 4), (2051, 128)])
def test_decode(dtype, Hq, Hkv, topK, block):
    c = make(dtype, Hq, Hkv, 1, (1, 2, 130, 2500, 0), None, topK, block, tail=16, seed=Hq + topK)
    check(c, run(c))


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("Hq,Hkv,block", [(16, 2, 16), (20, 2, 32), (32, 4, 2)])
def test_chunk(dtype, Hq, Hkv, block):
    c = make(dtype, Hq, Hkv, 9, (9, 700, 40, 5, 0, 200), (9, 7, 0, 9, 9, -1), 130, block, seed=Hq)
    check(c, run(c))


def test_whole_prompt():
    """Rows of every length up to 301 from position 0, more (row, head) pairs than CTAs at once."""
    c = make(torch.float16, 8, 2, 301, (301, 150, 1), None, 301, 16, seed=2)
    check(c, run(c))


@pytest.mark.parametrize("dtype,Hq,Hkv,S,topK", [
    (torch.float16, 32, 4, 2600, 131), (torch.bfloat16, 8, 8, 1300, 300), (torch.float16, 14, 2, 2600, 70),
    (torch.bfloat16, 24, 2, 1400, 129), (torch.float16, 64, 4, 1300, 128), (torch.float16, 12, 6, 1700, 40),
    (torch.bfloat16, 3, 3, 900, 257)])
def test_many_rows(dtype, Hq, Hkv, S, topK):
    """Enough rows that a CTA takes four or two KV heads of one (or, for 3 heads, one), with padded and empty rows."""
    c = make(dtype, Hq, Hkv, S, (S + 50, 200), (S - 3, 150), topK, 16, tail=16, seed=Hq + S)
    c["lists"][0, 7] = -1
    c["lists"][0, 11, :-1] = -1
    c["lists"][0, 12:40, 3::5] = -1
    c["lists"][1, 0, topK // 2] = -1
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = run(c, status=status)
    check(c, out)
    assert int(status) == 0 and torch.equal(out, run(c))
    want = out
    c["lists"][0, 7, topK - 1], c["lists"][1, 0, topK // 2] = S + 50, -5  # from naming nothing to naming no token
    assert torch.equal(run(c, status=status), want) and int(status) == 4


@pytest.mark.parametrize("dtype,Hq,Hkv", [(torch.float16, 16, 2), (torch.bfloat16, 30, 2), (torch.float16, 6, 6)])
def test_odd_number_of_rows(dtype, Hq, Hkv):
    """Two KV heads of two rows per CTA, an odd number of rows (the last CTA has one), some CTAs with one live row."""
    c = make(dtype, Hq, Hkv, 1301, (1400, 700, 1300), (1300, 501, 1301), 97, 8, seed=Hq)
    c["lists"][2, 5], c["lists"][2, 8, :96] = -1, -1
    out = run(c)
    check(c, out)
    assert torch.equal(out, run(c))


@pytest.mark.parametrize("B", (1, 2, 9, 20, 40, 60, 114, 160))
def test_cluster_sizes(B):
    """4 KV heads x B pairs: 8 down to 1 CTAs per pair; two runs give the same bits."""
    c = make(torch.float16, 32, 4, 1, tuple(700 + 13 * b for b in range(B)), None, 1031, 16, seed=B)
    out = run(c)
    assert torch.equal(out, run(c))
    for b in {0, B // 2, B - 1}:
        one = dict(c, q=c["q"][b:b + 1], lists=c["lists"][b:b + 1], ctx=c["ctx"][b:b + 1], pt=c["pt"][b:b + 1], n=[1])
        check(one, out[b:b + 1])


def test_lists():
    """Holes, an empty list, an entry twice, entries outside [0, L) and any order."""
    c = make(torch.float16, 8, 2, 6, (500,), (6,), 200, 16, seed=4)
    lists = c["lists"]
    lists[0, 0] = -1                       # nothing
    lists[0, 1, ::3] = -1                  # holes
    lists[0, 2, 1:] = -1                   # one entry
    lists[0, 3, 100:] = lists[0, 3, :100]  # every entry twice
    lists[0, 4, :100] = -1                 # nothing in the first steps
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = run(c, status=status)
    check(c, out)
    assert int(status) == 0 and not out[0, 0].view(torch.int16).any()
    want = run(c)
    broken = dict(c, lists=lists.clone())
    broken["lists"][0, 0, 5], broken["lists"][0, 1, 0], broken["lists"][0, 4, 0] = 500, -7, 2 ** 31 - 1
    got = run(broken, status=status)
    assert int(status) == 4 and torch.equal(got, want)


def test_bad_pages():
    """Entries on pages outside the pool are skipped in K and V alike."""
    c = make(torch.bfloat16, 8, 2, 2, (600,), (2,), 300, 16, seed=5)
    c["pt"][0, 0, 1], c["pt"][0, 1, 3] = c["pool"].shape[0], -1
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = run(c, status=status)
    assert int(status) == 2
    dropped = c["lists"].clone()
    dropped[(dropped // 128 == 1) | (dropped // 128 == 3)] = -1
    c["pt"][0, 0, 1] = c["pt"][0, 1, 3] = 0
    check(c, out, lists=dropped)


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
def test_scales_far_apart(dtype):
    """V scales that differ by 2^20 from block to block, K scales of 2^-30 and 2^3, queries of any size."""
    c = make(dtype, 16, 2, 3, (900,), (3,), 400, 4, seed=6)
    g = torch.Generator().manual_seed(1)
    flat = c["scale"].shape[0]
    k, v = c["scale"][:flat // 2], c["scale"][flat // 2:]
    k.copy_(torch.where(torch.rand(k.shape, generator=g) < 0.5, torch.full_like(k, 2.0 ** -30), torch.full_like(k, 0.02)))
    v.copy_(2.0 ** torch.randint(-16, 5, v.shape, generator=g).float())
    if dtype == torch.bfloat16:  # heads of 2^60 and 2^-60 against K scales that undo it
        c["q"][:, :, 0] *= 2.0 ** -60
        c["q"][:, :, 1] *= 2.0 ** 9
    check(c, run(c))


def test_scale_bounds():
    """Scales of 0, NaN and infinity are read as the nearest bound; a block of scale 0 weighs but adds nothing."""
    c = make(torch.float16, 8, 1, 1, (64,), None, 64, 16, seed=7)
    page_v = int(c["pt"][0, 1, 0])
    c["scale"][page_v, 1] = 0.0
    c["scale"][page_v, 2] = float("nan")
    out = run(c)
    c["scale"][page_v, 1:3] = 2.0 ** -48
    assert torch.equal(out, run(c))
    check(c, out)


def test_codes_that_are_no_numbers():
    """A NaN code reaches exactly the outputs that use it; one behind the list or on an unnamed row none."""
    c = make(torch.float16, 8, 2, 2, (400,), (2,), 100, 16, seed=8)
    clean = run(c)
    codes = c["pool"].view(torch.uint8)
    named = set(c["lists"][0].flatten().tolist())
    free = next(j for j in range(399) if j not in named)
    for plane in (0, 1):
        codes[int(c["pt"][0, plane, free // 128]), free % 128] = 0x7f
    assert torch.equal(run(c), clean)
    j = int(c["lists"][0, 0, 50])
    codes[int(c["pt"][0, 1, j // 128]), j % 128, 1, 77] = 0xff
    out = run(c)
    rows = [t for t in (0, 1) if j in c["lists"][0, t].tolist()]
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[0, rows, 4:, 77] = True
    assert torch.equal(out.isnan(), bad) and torch.equal(out[~bad], clean[~bad])


def test_attention_scales():
    for scale in (0.0, -0.3, 2.0):
        c = make(torch.float16, 8, 2, 1, (300, 40), None, 150, 16, seed=9)
        check(c, run(c, scale=scale), scale=scale)


def test_pool_beyond_4_gib():
    flat, Hkv = 34000, 8
    c = make(torch.float16, 8 * Hkv, Hkv, 1, (128,), None, 100, 16, seed=10)
    pool = torch.zeros((flat, 128, Hkv, D), dtype=torch.uint8, device=DEV)
    scale = torch.ones((flat, 8, Hkv), device=DEV)
    for plane, page in ((0, flat - 1), (1, flat - 2)):
        src = int(c["pt"][0, plane, 0])
        pool[page] = c["pool"][src].view(torch.uint8).to(DEV)
        scale[page] = c["scale"][src].to(DEV)
    pt = torch.tensor([[[flat - 1], [flat - 2]]], dtype=torch.int32, device=DEV)
    out = torch.empty(c["q"].shape, dtype=torch.float16, device=DEV)
    qb.sparse_paged_kv8(c["q"].to(DEV), pool.view(torch.float8_e4m3fn), scale, pt, c["lists"].to(DEV), c["ctx"].to(DEV), out,
                        scale=SCALE)
    assert torch.equal(out.cpu(), run(c))


def test_streams_and_graphs():
    """Two calls at once on two streams, and a captured append + attention replayed on new inputs."""
    c = make(torch.float16, 8, 2, 1, (300, 900), None, 260, 16, seed=11)
    other = make(torch.float16, 8, 2, 1, (700, 20), None, 260, 16, seed=12)
    want, want2 = run(c), run(other)
    dev = [{k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in x.items()} for x in (c, other)]
    outs = [torch.empty_like(x["q"]) for x in dev]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, o, s in zip(dev, outs, streams):
            qb.sparse_paged_kv8(x["q"], x["pool"], x["scale"], x["pt"], x["lists"], x["ctx"], o, scale=SCALE, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0].cpu(), want) and torch.equal(outs[1].cpu(), want2)

    x = dev[0]
    B, Hq, Hkv = 2, 8, 2
    w = torch.zeros(D, device=DEV)
    qkv = torch.randn((B, 1, Hq + 2 * Hkv, D), device=DEV).half()
    q, out = torch.empty_like(x["q"]), torch.empty_like(x["q"])
    start = {k: x[k].clone() for k in ("pool", "scale")}

    def step(stream=None):
        qb.append_kv8(qkv, w, w, x["ctx"], q, x["pool"], x["scale"], x["pt"], Hq=Hq, Hkv=Hkv, rot=64, theta=1e4, eps=1e-6,
                      stream=stream)
        qb.sparse_paged_kv8(q, x["pool"], x["scale"], x["pt"], x["lists"], x["ctx"], out, scale=SCALE, stream=stream)

    def reset():
        for k, v in start.items():
            x[k].copy_(v)

    step()
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        qkv.copy_(torch.randn(qkv.shape, generator=torch.Generator().manual_seed(i)).half())
        reset()
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (q, out, x["pool"].view(torch.uint8), x["scale"])]
        reset()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (q, out, x["pool"].view(torch.uint8), x["scale"])):
            assert torch.equal(a, b)


@pytest.mark.parametrize("shared", (True, False), ids=("widened rows", "pool of its own"))
def test_serving_run(shared):
    """A layer's calls as a server makes them on an 8-bit cache: a ragged prompt batch (append, indexer, attention,
    hand-off), then single tokens (append, indexer, attention).  The indexer's fp16 state lives behind the codes of
    widened rows (the byte pool read as fp16), or in a one-head fp16 pool on the same page table."""
    cfg = syn.PREFILL_TINY
    B, S, Hq, Hkv, di, rot, ratio, budget, topK = 2, 333, 8, 2, cfg.di, cfg.rot, cfg.ratio, cfg.budget, cfg.topK
    steps, block = 6, 16
    g = torch.Generator().manual_seed(77)
    ctx = torch.tensor([333, 130], dtype=torch.int32)
    pt, flat = ref.page_tables([int(x) + steps for x in ctx], 5)
    pt_d = pt.to(DEV)
    phd = D + (2 * di if shared else 0)
    pool = torch.zeros((flat, 128, Hkv, phd), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    scale = torch.zeros((flat, 128 // block, Hkv), device=DEV)
    index_pool = pool.view(torch.float16) if shared else torch.zeros((flat, 128, 1, 8 + di), dtype=torch.float16, device=DEV)
    index_D = D // 2 if shared else 8
    w, wi = (0.1 * torch.randn(D, generator=g)).to(DEV), (0.1 * torch.randn(di, generator=g)).to(DEV)
    kw = dict(rot=rot, ratio=ratio, budget=budget, topK=topK, theta=1e4, eps=1e-6)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def attention(q, lists, ctx_d, rows):
        out = torch.empty_like(q)
        qb.sparse_paged_kv8(q, pool, scale, pt_d, lists, ctx_d, out, scale=SCALE, status=status)
        c = dict(q=q.cpu(), pool=pool.cpu(), scale=scale.cpu(), pt=pt, lists=lists.cpu(), ctx=ctx_d.cpu(), n=rows)
        check(c, out.cpu())

    ctx_d = ctx.to(DEV)
    qkv = torch.randn((B, S, Hq + 2 * Hkv, D), generator=g).half().to(DEV)
    idxQ, idxK = (torch.randn(s, generator=g).half().to(DEV) for s in ((B, S, cfg.Hi, di), (B, S, di)))
    q = torch.empty((B, S, Hq, D), dtype=torch.float16, device=DEV)
    lists = torch.empty((B, S, topK), dtype=torch.int32, device=DEV)
    ws = qb.alloc_workspace(qb.indexer_prefill_workspace_size(B, S, di, ratio))
    qb.append_kv8(qkv, w, w, ctx_d, q, pool, scale, pt_d, Hq=Hq, Hkv=Hkv, rot=rot, theta=1e4, eps=1e-6, status=status)
    qb.indexer_prefill(idxQ, idxK, wi, wi, ctx_d, lists, ws, **kw)
    qb.indexer_prefill_handoff(idxK, ctx_d, ws, index_pool, pt_d, D=index_D, ratio=ratio)
    attention(q, lists, ctx_d, [333, 130])

    wsd = qb.alloc_workspace(qb.indexer_decode_workspace_size(B, pt.shape[2], ratio, budget))
    for i in range(steps):
        ctx_d = ctx_d + 1
        qkv1 = torch.randn((B, 1, Hq + 2 * Hkv, D), generator=g).half().to(DEV)
        iq, ik = (torch.randn(s, generator=g).half().to(DEV) for s in ((B, cfg.Hi, di), (B, di)))
        q1 = torch.empty((B, 1, Hq, D), dtype=torch.float16, device=DEV)
        lists1 = torch.empty((B, 1, topK), dtype=torch.int32, device=DEV)
        qb.append_kv8(qkv1, w, w, ctx_d, q1, pool, scale, pt_d, Hq=Hq, Hkv=Hkv, rot=rot, theta=1e4, eps=1e-6, status=status)
        qb.indexer_decode(iq, ik, wi, wi, index_pool, pt_d, ctx_d, lists1, wsd, D=index_D, **kw)
        assert qb.last_device_error(wsd) == 0
        attention(q1, lists1, ctx_d, [1, 1])
        for b in range(B):  # a token of an incomplete block is always named, one that completes its block only if scored
            L = int(ctx_d[b])
            assert set(range(L - L % ratio, L)) <= set(lists1[b, 0].tolist())
    assert int(status) == 0


def test_chunked_prompt_16bit():
    """A prompt appended in chunks to a 16-bit pool gives the cache and the decode of one appended at once."""
    Hq, Hkv, L, rot = 8, 2, 300, 64
    g = torch.Generator().manual_seed(6)
    for dtype in (torch.float16, torch.bfloat16):
        qkv = torch.randn((1, L, Hq + 2 * Hkv, D), generator=g).to(dtype).to(DEV)
        w = (0.1 * torch.randn(D, generator=g)).to(DEV)
        pt, flat = ref.page_tables([L], 3)
        pt = pt.to(DEV)
        pools = []
        for cuts in ((0, L), (0, 1, 17, 130, 131, 299, L)):
            pool = torch.zeros((flat, 128, Hkv, D), dtype=dtype, device=DEV)
            for a, b in zip(cuts, cuts[1:]):
                q = torch.empty((1, b - a, Hq, D), dtype=dtype, device=DEV)
                qb.append_kv(qkv[:, a:b].contiguous(), w, w, torch.tensor([b], dtype=torch.int32, device=DEV), q, pool, pt,
                             Hq=Hq, Hkv=Hkv, rot=rot, theta=1e4, eps=1e-6,
                             new_lengths=torch.tensor([b - a], dtype=torch.int32, device=DEV))
            pools.append((pool, q[:, -1:].contiguous()))
        assert torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1])
        lists = torch.arange(L, dtype=torch.int32, device=DEV).view(1, 1, L)
        po, ps, pc = qb.sparse_decode_workspace_elems(1, Hkv, D)
        parts = (torch.zeros(po, device=DEV), torch.zeros(ps, device=DEV), torch.zeros(pc, dtype=torch.int32, device=DEV))
        pool, q = pools[0]
        out = torch.empty_like(q)
        qb.sparse_decode(q, pool, pt, lists, torch.tensor([L], dtype=torch.int32, device=DEV), out, *parts, D=D, scale=SCALE)
        k, v = (pool[pt[0, i].long()].flatten(0, 1)[:L].double().cpu() for i in (0, 1))
        want = ref.attend(q[0].cpu(), k, v, lists[0].cpu(), SCALE)[0]
        assert float((out[0].cpu().double() - want).abs().max()) <= (2e-3 if dtype == torch.float16 else 2e-2)


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("Hq,Hkv,S", [(8, 1, 1), (16, 1, 1), (32, 4, 1300), (12, 2, 2500), (48, 4, 700)])
def test_one_key_decides(dtype, Hq, Hkv, S):
    """Two listed keys with the same values, in different steps of a warp, the second heavier by 2^0.5 to 2^7.9.  Whatever
    the weights, the output is the values themselves, which the output's type holds exactly: numerator and denominator
    have to use the same weights (fp32 leaves 2^-20, an output's half step is 2^-12 at least)."""
    gap, topK = (1024, 1100) if S == 1 else (32, 60)  # a warp's next step (one pair: 8 CTAs share a list)
    c = make(dtype, Hq, Hkv, S, (max(S, 300),), None, topK, 16, seed=40 + Hq)
    c["lists"][:] = -1
    c["lists"][:, :, 0], c["lists"][:, :, gap + 8] = 3, 200
    c["scale"][:] = 1.0
    codes = c["pool"].view(torch.uint8)
    k = [int(c["pt"][0, 0, j // 128]) for j in (3, 200)]
    v = [int(c["pt"][0, 1, j // 128]) for j in (3, 200)]
    codes[k[0], 3] = 0
    codes[k[1], 200 - 128] = 0
    codes[k[1], 200 - 128, :, 0] = 0x38  # 1.0
    codes[v[1], 200 - 128] = codes[v[0], 3]
    c["scale"][v[0]] = c["scale"][v[1]] = 2.0 ** -7
    g = torch.Generator().manual_seed(Hq)
    c["q"][..., 0] = (0.5 + 7.4 * torch.rand(c["q"].shape[:-1], generator=g)).to(dtype)
    out = run(c, scale=math.log(2.0))  # q[0] is the heavier key's weight in powers of two
    want = (ref.E4M3[codes[v[0], 3].long()] * 2.0 ** -7).to(dtype)[None, None].repeat_interleave(Hq // Hkv, 2)
    n = c["n"][0]
    assert torch.equal(out[:, :n], want.expand(1, n, -1, -1))


@pytest.mark.parametrize("e,kscale,scale", [
    (60, 2.0 ** -48, 2.0 ** -23), (118, 2.0 ** -48, 2.0 ** -81), (118, 2.0 ** -7, 2.0 ** -122), (120, 2.0 ** -20, 2.0 ** -111),
    (-110, 2.0 ** 48, 2.0 ** 51), (-110, 2.0 ** -7, 2.0 ** 106), (0, 2.0 ** -48, 2.0 ** 37)])
@pytest.mark.parametrize("Hkv,S", [(2, 2), (4, 1300)])
def test_bf16_queries_of_any_size(e, kscale, scale, Hkv, S):
    """Queries of about 2^e against K scales and an attentionScale that bring the logits back near 1."""
    c = make(torch.bfloat16, 8 * Hkv, Hkv, S, (max(S, 400),), None, 140, 16, seed=50 + S)
    c["q"] = (c["q"].float() * 2.0 ** e).bfloat16()
    half = c["scale"].shape[0] // 2  # K pages, then V pages
    c["scale"][:half] = kscale
    out = run(c, scale=scale)
    L = int(c["ctx"][0])
    k, v = (ref.dequantised(c["pool"], c["scale"], c["pt"][0, i], L) for i in (0, 1))
    rows = list(range(2)) if S == 2 else list(range(0, S, 97)) + [S - 1]
    want, mean_abs, dots = ref.attend(c["q"][0, rows], k, v, c["lists"][0, rows], scale)
    assert 0.1 < float(dots.max()) < 1e4
    bar = ref.attend_bar(want, mean_abs, dots, c["lists"][0, 0], c["scale"][half:], out.dtype)
    err = (out[0, rows].double() - want).abs()
    assert bool((err <= bar).all()), float((err / bar).max())


@pytest.mark.parametrize("Hq,Hkv,S,L,new,pages", [(8, 2, 300, 300, None, 2), (8, 2, 20, 300, (20,), 2),
                                                  (16, 4, 1300, 1300, None, 5), (8, 2, 1, 300, None, 1)])
def test_rows_behind_the_page_table(Hq, Hkv, S, L, new, pages):
    """A length past the page table: every live row is computed from the entries that the table holds, as the append
    writes every live row's dense output; entries behind the table are skipped and reported."""
    c = make(torch.float16, Hq, Hkv, S, (L,), new, 90, 16, seed=60 + S)
    c["pt"] = c["pt"][:, :, :pages].contiguous()
    named = torch.where(c["lists"] < 128 * pages, c["lists"], torch.full_like(c["lists"], -1))
    named[0, -1, 0] = 5
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = run(dict(c, lists=named), status=status)
    check(c, want, lists=named)
    assert int(status) == 0 and bool(want[0, -1].view(torch.int16).any())
    behind = named.clone()
    behind[0, -1, 1:4] = torch.tensor([128 * pages, L - 1, -1], dtype=torch.int32)
    named[0, -1, 1:4] = -1
    assert torch.equal(run(dict(c, lists=behind), status=status), run(dict(c, lists=named)))
    assert int(status) == 4


@pytest.mark.parametrize("dtype", (torch.float16, torch.bfloat16))
@pytest.mark.parametrize("Hq,Hkv,S,topK", [(8, 2, 1, 2051), (24, 2, 1, 2051), (16, 4, 1300, 400), (12, 6, 900, 400),
                                           (24, 2, 1300, 400)])
def test_every_entry_counts_once(dtype, Hq, Hkv, S, topK):
    """Each entry of a long list by itself: in sequence b the token 128 b + d has one nonzero value, in dim d, so an output
    is one entry's probability times that value.  Relative bar: fp16 weights in numerator and denominator (2^-11 each),
    logits off by D 2^-23 of their terms, twice, the output's half step, and 2^-18 for the rest; a missing or doubled
    entry is off by 1.  Weights stay in fp16's normal range and outputs too (logits within 1.5 of each other)."""
    L = topK - 40  # the rest of the list is holes
    B = -(-L // 128)
    if S > 1:
        B = min(B, 3)
    c = make(dtype, Hq, Hkv, S, (max(L, S),) * B, None, topK, 16, seed=70 + Hq + S)
    g = torch.Generator().manual_seed(Hq)
    order = torch.rand((B, S, topK), generator=g).argsort(-1).to(torch.int32)
    c["lists"] = torch.where(order < L, order, torch.full_like(order, -1))
    half = c["scale"].shape[0] // 2
    c["scale"][:half] = 2.0 ** -7
    c["scale"][half:] = 1.0
    codes = c["pool"].view(torch.uint8)
    codes[half:] = 0
    for b in range(B):
        d = torch.arange(min(128, L - 128 * b))
        codes[int(c["pt"][b, 1, b]), d, :, d] = 0x7e  # 448
    out = run(c, scale=0.004).double()
    G = Hq // Hkv
    for b in range(B):
        k = ref.dequantised(c["pool"], c["scale"], c["pt"][b, 0], L)
        z = 0.004 * torch.einsum("thgd,lhd->thgl", c["q"][b].double().view(S, Hkv, G, D), k)
        assert float((z.amax(-1) - z.amin(-1)).max()) < 1.5
        m = min(128, L - 128 * b)
        want = 448 * torch.softmax(z, -1)[..., 128 * b:128 * b + m].reshape(S, Hq, m)
        terms = 0.004 * (c["q"][b].double().abs().sum(-1).max() * k.abs().max())
        bar = 2 * 2.0 ** -11 + 2 * D * 2.0 ** -23 * float(terms) + torch.finfo(dtype).eps / 2 + 2.0 ** -18
        assert bar < 0.02 and float(((out[b, :, :, :m] - want).abs() / want).max()) <= bar
        assert not out[b, :, :, m:].any()
