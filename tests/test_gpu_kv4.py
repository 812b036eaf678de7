"""qsa_store_kv4, qsa_sparse_paged_kv4 and qsa_sparse_weights_kv4 against their 64-bit forms.

A stored row is exact: every byte equals the reference's.  Bars of the attention: `paged_cache_ref.attend_bar`'s terms with a
row's largest value 2688 times its scale.  lse and weights: a logit is off by D 2^-23 of the largest sum of its terms'
magnitudes (fp32 tensor-core sums) and 2^-22 of itself for its scale and the units of the exponent; lse adds the exponentials'
2^-22 and its own rounding (2^-23 of it, of the maximum and of the logarithm); a weight exp(x - lse) takes both, relative."""
from __future__ import annotations

import math

import pytest
import torch

import kv4_ref as ref

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
PAGE, ROW, D = ref.PAGE, ref.ROW, ref.D


@pytest.fixture(scope="module")
def qb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_gqa_qsa_gb300 import _binding, build
    build.build()
    _binding.lib()
    return _binding


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


# ------------------------------------------------------------------- store
def store_case(B, S, Hkv, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, S, 2 * Hkv, D), generator=g)
    x[..., ::31] *= 9.0
    return x.to(DT[dtype])


def check_store(qb, kv, ctx, new, pt, flat, row=ROW, outs=True):
    B, S, H2, _ = kv.shape
    Hkv = H2 // 2
    g = torch.Generator().manual_seed(99)
    before = torch.randint(0, 256, (flat, PAGE, Hkv, row), generator=g, dtype=torch.int32).to(torch.uint8)
    n = ref.new_rows(ctx, new, S)
    want, dense, bad = before.clone(), torch.zeros((2, B, S, Hkv, D), dtype=torch.float64), False
    for b in range(B):
        for t in range(n[b]):
            p = max(ctx[b], 0) - n[b] + t
            r = ref.rows_of(kv[b, t])
            for plane in (0, 1):
                mine = r[plane * Hkv:(plane + 1) * Hkv]
                dense[plane, b, t] = ref.values_of(mine)
                page = int(pt[b, plane, p // PAGE]) if p // PAGE < pt.shape[2] else -1
                if 0 <= page < flat:
                    want[page, p % PAGE, :, :ROW] = mine
                else:
                    bad = True
    pool, gk = before.cuda(), kv.cuda()
    out = [torch.full((B, S, Hkv, D), 5.0, dtype=kv.dtype, device="cuda") if outs else None for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qb.store_kv4(gk[:, :, :Hkv], gk[:, :, Hkv:], i32(ctx).cuda(), pool, pt.cuda(),
                 new_lengths=None if new is None else i32(new).cuda(), k_out=out[0], v_out=out[1], status=status)
    assert torch.equal(pool.cpu(), want)
    assert int(status) == (2 if bad else 0)
    for o, d in zip(out, dense):
        if o is not None:
            top = torch.finfo(kv.dtype).max
            w = torch.where(torch.isnan(d), d, d.clamp(-top, top)).to(kv.dtype)
            assert torch.equal(torch.nan_to_num(o.cpu().float(), nan=-12345.0), torch.nan_to_num(w.float(), nan=-12345.0))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("B,S,Hkv,ctx,new,row", [
    (1, 1, 1, [1], None, 80), (3, 1, 2, [0, 129, 4000], None, 80), (2, 17, 3, [17, 300], [17, 5], 96),
    (4, 9, 4, [9, 4, 0, 131], [0, 9, 3, 7], 80), (2, 130, 1, [500, 128], None, 336), (2, 3, 8, [256, 3], [3, 3], 80)])
def test_store(qb, dtype, B, S, Hkv, ctx, new, row):
    pt, flat = ref.page_tables(ctx, B + S, extra=1)
    check_store(qb, store_case(B, S, Hkv, dtype, S), ctx, new, pt, flat, row)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_store_borders(qb, dtype):
    """Quotients on the borders between codes and between scales, zeros of both signs, the type's largest and smallest values,
    infinities and NaN, in rows of every magnitude."""
    x = torch.zeros((1, 24, 2, D))
    grid = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, -0.0])
    both = torch.cat([grid, -grid]).repeat(4)  # every group reaches 6: scale 448 of the row's scale
    for t in range(8):
        x[0, t, 0], x[0, t, 1] = both * 2.0 ** (t - 4), both * (1 + t / 8) * 2.0 ** -3
    # group maxima on the borders between scales: 6 (1 + (2 i + 1) / 16) and next to them
    for t in range(8, 12):
        x[0, t] = 0.01
        x[0, t, :, 0] = 48.0
        x[0, t, 0, 16::16] = torch.tensor([6 * (1 + (2 * i + 1) / 16) for i in range(7)]) * 2.0 ** -(t - 8)
        x[0, t, 1, 16::16] = torch.tensor([6 * (1 + (2 * i + 1) / 16) * (1 + 2.0 ** -7) for i in range(7)])
    top, low = torch.finfo(DT[dtype]).max, torch.finfo(DT[dtype]).tiny
    x[0, 12] = top
    x[0, 13] = -top
    x[0, 14] = low
    x[0, 15, 0, 5] = low / 4
    x[0, 16, 0], x[0, 16, 1, 3] = torch.randn(D, generator=torch.Generator().manual_seed(1)) * low, 1.0
    x[0, 17, 0, 17], x[0, 17, 1, 127] = float("inf"), float("nan")
    x[0, 18] = float("nan")
    x[0, 19, 0, ::16] = -float("inf")
    x[0, 20, :, 0], x[0, 20, :, 64] = 2688.0 * 2 ** 4, 1e-4  # a scale of 0
    x[0, 21] = -0.0
    x[0, 22, :, 3], x[0, 23, :, 3] = 21.0, 21.125  # at and above a power of two of the row scale
    pt, flat = ref.page_tables([24], 5)
    check_store(qb, x.to(DT[dtype]), [24], None, pt, flat)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_codes_keep_their_signs(qb, dtype):
    """Under a zero scale, and where a quotient rounds to 0, a code is 0 or 8 by its value's sign; next to a NaN all are 0."""
    x = torch.zeros((1, 1, 2, D))
    x[..., 0] = 2688.0 * 16  # t = 16: 1e-4 / 96 is nothing of a scale
    x[..., 16:32:3], x[..., 17:32:3], x[..., 18:32:3] = -1e-4, 1e-4, -0.0
    x[..., 32], x[..., 33:48:2], x[..., 34:48:2] = 96.0, -1e-4, 1e-4
    x[..., 64:80], x[..., 70] = -3.0, float("nan")
    x = x.to(DT[dtype])
    pt, flat = ref.page_tables([1], 2)
    check_store(qb, x, [1], None, pt, flat)
    pool = torch.full((flat, PAGE, 1, ROW), 255, dtype=torch.uint8, device="cuda")
    qb.store_kv4(x[:, :, :1].cuda(), x[:, :, 1:].cuda(), i32([1]).cuda(), pool, pt.cuda())
    for plane in (0, 1):
        row = pool[pt[0, plane, 0], 0, 0].cpu()
        code = torch.stack([row[:64] & 15, row[:64] >> 4], -1).flatten()
        assert row[64:72].tolist() == [0x7e, 0, 0x38, 0, 0x7f, 0, 0, 0]
        assert torch.equal(code[16:32], 8 * torch.signbit(x[0, 0, plane, 16:32].float()).to(torch.uint8))
        assert torch.equal(code[33:48], 8 * (torch.arange(33, 48) % 2).to(torch.uint8)) and code[32] == 7
        assert not bool(code[64:80].any())


def test_store_bad_pages_views_and_no_outputs(qb):
    ctx = [300, 140]
    pt, flat = ref.page_tables(ctx, 3)
    pt[0, 0, 2], pt[0, 1, 1], pt[1, 1, 1] = flat, -1, 2 ** 31 - 1
    check_store(qb, store_case(2, 140, 2, "fp16", 1), ctx, None, pt, flat)
    check_store(qb, store_case(2, 3, 2, "bf16", 1), [386, 130], None, pt[:, :, :2].contiguous(), flat, outs=False)  # past the table
    # the same tokens from views with other strides, in pieces: the same bytes
    kv = store_case(1, 40, 3, "bf16", 7).cuda()
    pt, flat = ref.page_tables([200], 1)
    pools = []
    for pieces in ([40], [1, 13, 26]):
        pool = torch.zeros((flat, PAGE, 3, ROW), dtype=torch.uint8, device="cuda")
        wide = torch.full((1, 40, 11, D), float("nan"), dtype=kv.dtype, device="cuda")
        wide[:, :, 1:4], wide[:, :, 5:8] = kv[:, :, :3], kv[:, :, 3:]
        at = 0
        for m in pieces:
            qb.store_kv4(wide[:, at:at + m, 1:4], wide[:, at:at + m, 5:8], i32([160 + at + m]).cuda(), pool, pt.cuda())
            at += m
        pools.append(pool)
    assert torch.equal(pools[0], pools[1]) and bool(pools[0].any())
    with pytest.raises(ValueError, match="heads"):
        qb.store_kv4(wide[:, :, 1:7:2], wide[:, :, 5:8], i32([160]).cuda(), pool, pt.cuda())


# --------------------------------------------------- attention and weights
def make(B, S, Hq, Hkv, ctx, new, topk, dtype, seed, row=ROW, keep=None, bad=False):
    n = ref.new_rows(ctx, new, S)
    pt, flat = ref.page_tables(ctx, seed)
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((B, S, Hq, D), generator=g).to(DT[dtype])
    for b in range(B):
        q[b, n[b]:] = float("nan")  # padding is never read
    pool = ref.random_pool(flat, Hkv, seed, row)
    lists = ref.lists_of(ctx, n, S, topk, seed, keep, bad)
    return dict(q=q, pool=pool, pt=pt, ctx=ctx, new=new, n=n, lists=lists, scale=1 / math.sqrt(D))


def run_attend(qb, c, lse=True, stream=None, out=None):
    q = c["q"].cuda()
    o = torch.full_like(q, 3.0) if out is None else out
    l = torch.full(q.shape[:3], 3.0, device="cuda") if lse else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qb.sparse_paged_kv4(q, c["pool"].cuda(), c["pt"].cuda(), c["lists"].cuda(), i32(c["ctx"]).cuda(), o, scale=c["scale"],
                        new_lengths=None if c["new"] is None else i32(c["new"]).cuda(), lse=l, status=status, stream=stream)
    return o, l, int(status)


def exact(c):
    B, S, Hq, _ = c["q"].shape
    Hkv = c["pool"].shape[2]
    o, mean = torch.zeros((2, B, S, Hq, D), dtype=torch.float64)
    lse = torch.full((B, S, Hq), -math.inf, dtype=torch.float64)
    w = torch.zeros((B, S, Hkv, c["lists"].shape[-1]), dtype=torch.float64)
    dots = torch.zeros((B, S, Hq), dtype=torch.float64)
    vmax = torch.zeros((B,), dtype=torch.float64)
    for b in range(B):
        L, n = max(c["ctx"][b], 0), c["n"][b]
        if L == 0 or n == 0:
            continue
        k, v = ref.cached(c["pool"], c["pt"][b, 0], L), ref.cached(c["pool"], c["pt"][b, 1], L)
        vmax[b] = 2688 * c["pool"][c["pt"][b, 1, :-(-L // PAGE)].long()][..., 72:76].contiguous().view(torch.float32).max()
        o[b, :n], lse[b, :n], w[b, :n], mean[b, :n], dots[b, :n] = ref.attend(c["q"][b, :n], k, v, c["lists"][b, :n], c["scale"])
    return dict(o=o, lse=lse, w=w, mean=mean, dots=dots, vmax=vmax)


def logit_error(x):
    return (D * 2.0 ** -23 + 2.0 ** -22) * x["dots"]


def check_attend(c, x, o, lse):
    topk, dtype = c["lists"].shape[-1], o.dtype
    sub = topk * 2.0 ** -25 * x["vmax"][:, None, None, None]
    bar = (2.0 ** -11 + 2.0 ** -18 + 2 * logit_error(x)[..., None]) * x["mean"] + sub + \
        torch.finfo(dtype).eps / 2 * x["o"].abs() + 1e-7
    err = (o.double().cpu() - x["o"]).abs()
    assert bool((err <= bar).all()), float((err / bar).max())
    for b, n in enumerate(c["n"]):
        assert not bool(o[b, n:].view(torch.int16).any())  # exact zeros
    if lse is not None:
        got, want = lse.double().cpu(), x["lse"]
        none = torch.isinf(want)
        assert torch.equal(torch.isinf(got) & (got < 0), none)
        bar = logit_error(x) + 2.0 ** -20 + 2.0 ** -22 * want.abs().nan_to_num(posinf=0)
        assert bool(((got - want).abs()[~none] <= bar[~none]).all()), float((got - want).abs()[~none].max())


def run_weights(qb, c, lse, total, stream=None):
    q = c["q"].cuda()
    w = torch.full((q.shape[0], q.shape[1], c["pool"].shape[2], c["lists"].shape[-1]), 3.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qb.sparse_weights_kv4(q, c["pool"].cuda(), c["pt"].cuda(), c["lists"].cuda(), i32(c["ctx"]).cuda(), lse, w, total,
                          scale=c["scale"], new_lengths=None if c["new"] is None else i32(c["new"]).cuda(), status=status,
                          stream=stream)
    return w, int(status)


def check_weights(c, x, lse, w, before, total):
    """Every weight; and the totals as the fp32 sum of the weights, row by row."""
    B, S, Hkv, topk = w.shape
    G = c["q"].shape[2] // Hkv
    rel = (logit_error(x) + 2.0 ** -20 + 2.0 ** -21 * lse.double().cpu().abs().nan_to_num(posinf=0)).unflatten(2, (Hkv, G)).amax(-1)
    err = (w.double().cpu() - x["w"]).abs()
    assert bool((err <= 2 * rel[..., None] * x["w"] + 1e-37).all()), float((err / x["w"].clamp(min=1e-30)).max())
    if total is None:
        return
    want, size = before.double().cpu().clone(), before.double().cpu().abs()
    for b in range(B):
        for t in range(c["n"][b]):
            j = c["lists"][b, t].long()
            ok = (j >= 0) & (j < min(max(c["ctx"][b], 0), total.shape[2]))
            for h in range(Hkv):
                want[b, h].index_add_(0, j[ok], w[b, t, h].double().cpu()[ok])
    adds = max(c["n"]) + 2
    bar = adds * 2.0 ** -24 * want.abs() * (1 + 2.0 ** -10)
    assert bool(((total.double().cpu() - want).abs() <= bar).all()), float((total.double().cpu() - want).abs().max())


CASES = [
    # few pairs, one token: one entry; two partly filled steps; every group size; wide rows
    dict(B=1, S=1, Hq=1, Hkv=1, ctx=[1], new=None, topk=1),
    dict(B=1, S=1, Hq=7, Hkv=1, ctx=[512], new=None, topk=67, keep=50),
    dict(B=3, S=1, Hq=24, Hkv=2, ctx=[0, 33, 700], new=None, topk=131, bad=True),
    dict(B=2, S=1, Hq=16, Hkv=1, ctx=[1500, 900], new=None, topk=1003, row=96),
    dict(B=2, S=1, Hq=40, Hkv=8, ctx=[2200, 2048], new=None, topk=2051, keep=2048, row=160),
    # drafted tokens, rows that are padding, a sequence without new tokens
    dict(B=4, S=5, Hq=12, Hkv=3, ctx=[3, 260, 0, 900], new=[5, 2, 1, 0], topk=259, bad=True),
    dict(B=2, S=33, Hq=18, Hkv=2, ctx=[40, 500], new=[33, 20], topk=96, keep=64),
    # many rows: four heads of a row to a CTA, and two heads of two rows (an odd number of rows)
    dict(B=1, S=1301, Hq=16, Hkv=4, ctx=[1301], new=None, topk=70, keep=64, bad=True),
    dict(B=1, S=2551, Hq=4, Hkv=2, ctx=[2560], new=None, topk=35),
    dict(B=1, S=650, Hq=48, Hkv=4, ctx=[700], new=None, topk=131, keep=128),
    dict(B=1, S=1225, Hq=2 * 13, Hkv=2, ctx=[1300], new=None, topk=40),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_attend_and_weights(qb, dtype, i):
    c = make(**CASES[i], dtype=dtype, seed=i + 1)
    x = exact(c)
    o, lse, status = run_attend(qb, c)
    assert status == (4 if CASES[i].get("bad") else 0)
    check_attend(c, x, o, lse)
    o2, none, _ = run_attend(qb, c, lse=False)
    check_attend(c, x, o2, none)
    o3, lse3, _ = run_attend(qb, c)
    assert torch.equal(o3, o) and torch.equal(lse3, lse)  # bit for bit
    T = max(1, max(c["ctx"]))
    before = torch.rand((o.shape[0], c["pool"].shape[2], T), generator=torch.Generator().manual_seed(i)).cuda()
    total = before.clone()
    w, status = run_weights(qb, c, lse, total)
    assert status == (4 if CASES[i].get("bad") else 0)
    check_weights(c, x, lse, w, before, total)
    again = before.clone()
    w2, _ = run_weights(qb, c, lse, again)
    assert torch.equal(w2, w) and torch.equal(again, total)
    w3, _ = run_weights(qb, c, lse, None)
    assert torch.equal(w3, w)


def test_totals_are_added_row_by_row(qb):
    """The totals of several rows are, bit for bit, fp32 additions in the order of the rows, and what a call per row gives;
    an entry named twice adds twice."""
    c = make(B=2, S=24, Hq=12, Hkv=2, ctx=[3000, 900], new=[24, 17], topk=900, dtype="bf16", seed=13)
    c["lists"][0, 5, 100:120] = c["lists"][0, 5, 0:20]
    _, lse, _ = run_attend(qb, c)
    before = torch.rand((2, 2, 3000), generator=torch.Generator().manual_seed(3))
    total = before.cuda()
    w, _ = run_weights(qb, c, lse, total)
    want, one = before.clone(), before.cuda()
    for t in range(24):
        for b in range(2):
            j = c["lists"][b, t].long()
            for e in ((j >= 0) & (j < c["ctx"][b])).nonzero().flatten().tolist() if t < c["n"][b] else []:
                for h in range(2):
                    want[b, h, j[e]] += w[b, t, h, e].cpu()
        row = dict(c, q=c["q"][:, t:t + 1], lists=c["lists"][:, t:t + 1], new=[int(t < n) for n in c["n"]])
        run_weights(qb, row, lse[:, t:t + 1].contiguous(), one)
    assert torch.equal(total.cpu(), want)
    assert torch.equal(one, total)


def test_totals_shorter_than_the_cache(qb):
    """Tokens at or past totalLen are not counted; nothing behind the array is written."""
    for S in (1, 6):
        c = make(B=2, S=S, Hq=8, Hkv=2, ctx=[700, 640], new=None, topk=300, dtype="fp16", seed=3)
        _, lse, _ = run_attend(qb, c)
        room = torch.zeros((2 * 2 * 200 + 64,), device="cuda")
        total = room[:800].view(2, 2, 200)
        w, status = run_weights(qb, c, lse, total)
        assert status == 0
        check_weights(c, exact(c), lse, w, torch.zeros(2, 2, 200), total)
        assert not bool(room[800:].any())


def test_long_lists_and_many_ranges(qb):
    """A list of every token of a long cache (as after an eviction), and window rows whose totals span several CTAs."""
    c = make(B=1, S=1, Hq=8, Hkv=1, ctx=[20011], new=None, topk=20011, dtype="bf16", seed=5)
    x = exact(c)
    o, lse, _ = run_attend(qb, c)
    check_attend(c, x, o, lse)
    total = torch.zeros((1, 1, 20011), device="cuda")
    w, _ = run_weights(qb, c, lse, total)
    check_weights(c, x, lse, w, torch.zeros_like(total), total)
    c = make(B=1, S=3, Hq=4, Hkv=1, ctx=[20011], new=[3], topk=6000, dtype="fp16", seed=6)
    x = exact(c)
    o, lse, _ = run_attend(qb, c)
    total = torch.ones((1, 1, 20011), device="cuda")
    w, _ = run_weights(qb, c, lse, total)
    check_weights(c, x, lse, w, torch.ones_like(total), total)


def test_an_entry_named_twice_counts_twice(qb):
    for S in (1, 3):
        c = make(B=1, S=S, Hq=8, Hkv=2, ctx=[300], new=None, topk=90, dtype="fp16", seed=7, keep=60)
        for t in range(S):
            c["lists"][0, t, 64:] = c["lists"][0, t, :26]
        x = exact(c)
        o, lse, _ = run_attend(qb, c)
        check_attend(c, x, o, lse)
        total = torch.zeros((1, 2, 300), device="cuda")
        w, _ = run_weights(qb, c, lse, total)
        check_weights(c, x, lse, w, torch.zeros_like(total), total)
        again = torch.zeros_like(total)
        run_weights(qb, c, lse, again)
        assert torch.equal(again, total)


def test_bad_pages_are_skipped(qb):
    """An entry whose K or V page lies outside the pool names nothing, for the attention and for the weights."""
    for S, Hkv in ((1, 2), (700, 4)):
        c = make(B=1, S=S, Hq=4 * Hkv, Hkv=Hkv, ctx=[900], new=None, topk=120, dtype="bf16", seed=8)
        good = c["pt"].clone()
        c["pt"][0, 0, 1], c["pt"][0, 1, 4] = c["pool"].shape[0], -1
        y = dict(c, pt=good, lists=torch.where((c["lists"] // PAGE == 1) | (c["lists"] // PAGE == 4),
                                               torch.full_like(c["lists"], -1), c["lists"]))
        x = exact(y)
        o, lse, status = run_attend(qb, c)
        assert status == 2
        check_attend(y, x, o, lse)
        w, status = run_weights(qb, c, lse, None)
        assert status == 2
        check_weights(y, x, lse, w, None, None)


@pytest.mark.parametrize("S,Hkv", [(1, 1), (1400, 4)])
def test_what_lists_do_not_name_is_not_used(qb, S, Hkv):
    """NaN scales in every row that no list names (and behind the 80 bytes of a row) show nowhere; in a named row they do."""
    c = make(B=1, S=S, Hq=8 * Hkv, Hkv=Hkv, ctx=[1600], new=[S], topk=60, dtype="fp16", seed=9, row=96)
    keep = torch.arange(0, 1600, 3)
    g = torch.Generator().manual_seed(1)
    c["lists"] = torch.where(c["lists"] >= 0, keep[torch.randint(0, 60, c["lists"].shape, generator=g)].to(torch.int32), c["lists"])
    x = exact(c)
    dirty = torch.ones(1600, dtype=torch.bool)
    dirty[keep] = False
    tok = dirty.nonzero().flatten()
    for plane in (0, 1):
        c["pool"][c["pt"][0, plane, tok // PAGE].long(), tok % PAGE, :, 64:76] = 0xff
    c["pool"][..., 80:] = 0xff
    o, lse, _ = run_attend(qb, c)
    check_attend(c, x, o, lse)
    w, _ = run_weights(qb, c, lse, None)
    check_weights(c, x, lse, w, None, None)
    j = int(c["lists"][0, 0, 0])
    c["pool"][c["pt"][0, 1, j // PAGE], j % PAGE, 0, 64 + 3] = 0x7f  # group 3 of one V row
    o2, lse2, _ = run_attend(qb, c)
    assert bool(torch.isnan(o2[0, 0, :8, 48:64]).all()) and torch.equal(o2[0, 0, :8, :48], o[0, 0, :8, :48])
    assert torch.equal(lse2, lse)


def test_scales_of_every_size(qb):
    """Row scales from 2^-48 to 2^48 side by side in V, and of K as far as logits allow."""
    c = make(B=1, S=2, Hq=8, Hkv=1, ctx=[256], new=None, topk=128, dtype="bf16", seed=10)
    g = torch.Generator().manual_seed(4)
    e = torch.randint(-48, 49, (c["pool"].shape[0], PAGE, 1, 1), generator=g).float()
    c["pool"][..., 72:76] = torch.exp2(e).view(torch.uint8)
    kp = c["pt"][0, 0].long()
    c["pool"][kp, ..., 72:76] = torch.exp2(torch.randint(-48, -9, (2, PAGE, 1, 1), generator=g).float()).view(torch.uint8)
    x = exact(c)
    o, lse, _ = run_attend(qb, c)
    check_attend(c, x, o, lse)
    assert float(x["o"].abs().max()) > 2.0 ** 40
    for big in (2.0 ** 100, 2.0 ** -100):  # bf16 queries of any size, with a scale to match
        y = dict(c, q=(c["q"].double() * big).to(torch.bfloat16), scale=c["scale"] / big)
        o2, lse2, _ = run_attend(qb, y)
        assert torch.equal(o2, o) and float((lse2 - lse).abs().max()) <= 2.0 ** -18


def test_another_stream_graph_replays_and_concurrent_calls(qb):
    c = make(B=2, S=1, Hq=16, Hkv=2, ctx=[1700, 900], new=None, topk=1030, dtype="fp16", seed=11)
    x = exact(c)
    o, lse, _ = run_attend(qb, c)
    t = {k: c[k].cuda() for k in ("q", "pool", "pt", "lists")}
    ctx = i32(c["ctx"]).cuda()
    total = torch.zeros((2, 2, 1700), device="cuda")
    w1, _ = run_weights(qb, c, lse, total)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [(torch.zeros_like(o), torch.zeros_like(lse), torch.zeros_like(w1), torch.zeros_like(total)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        for st, (a, l, w, tot) in zip(streams, outs):
            with torch.cuda.stream(st):
                tot.zero_()
                qb.sparse_paged_kv4(t["q"], t["pool"], t["pt"], t["lists"], ctx, a, scale=c["scale"], lse=l)
                qb.sparse_weights_kv4(t["q"], t["pool"], t["pt"], t["lists"], ctx, l, w, tot, scale=c["scale"])
    torch.cuda.synchronize()
    for a, l, w, tot in outs:
        assert torch.equal(a, o) and torch.equal(l, lse) and torch.equal(w, w1) and torch.equal(tot, total)
    a, l, w, tot = outs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qb.sparse_paged_kv4(t["q"], t["pool"], t["pt"], t["lists"], ctx, a, scale=c["scale"], lse=l)
        qb.sparse_weights_kv4(t["q"], t["pool"], t["pt"], t["lists"], ctx, l, w, tot, scale=c["scale"])
    for _ in range(2):
        for v in (a, l, w, tot):
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, o) and torch.equal(l, lse) and torch.equal(w, w1) and torch.equal(tot, total)
    check_attend(c, x, o, lse)


def test_pool_past_32_bit_offsets(qb):
    """Rows more than 2^32 bytes into a pool are stored, read and weighed as the first ones are."""
    Hkv, row = 8, 1024
    pages = 2 ** 32 // (PAGE * Hkv * row) + 3
    pool = torch.empty((pages, PAGE, Hkv, row), dtype=torch.uint8, device="cuda")
    small = torch.zeros((4, PAGE, Hkv, ROW), dtype=torch.uint8, device="cuda")
    kv = store_case(1, 200, Hkv, "fp16", 3).cuda()
    far = torch.tensor([[[pages - 1, pages - 3], [pages - 2, pages - 4]]], dtype=torch.int32)
    near = torch.tensor([[[0, 1], [2, 3]]], dtype=torch.int32)
    c = make(B=1, S=1, Hq=16, Hkv=Hkv, ctx=[200], new=None, topk=200, dtype="fp16", seed=12)
    got = []
    for p, pt in ((pool, far.cuda()), (small, near.cuda())):
        qb.store_kv4(kv[:, :, :Hkv], kv[:, :, Hkv:], i32([200]).cuda(), p, pt)
        o, lse = torch.empty_like(c["q"].cuda()), torch.empty((1, 1, 16), device="cuda")
        w = torch.empty((1, 1, Hkv, 200), device="cuda")
        qb.sparse_paged_kv4(c["q"].cuda(), p, pt, c["lists"].cuda(), i32([200]).cuda(), o, scale=0.1, lse=lse)
        qb.sparse_weights_kv4(c["q"].cuda(), p, pt, c["lists"].cuda(), i32([200]).cuda(), lse, w, scale=0.1)
        got.append((o, lse, w))
    for x, y in zip(*got):
        assert torch.equal(x, y)
