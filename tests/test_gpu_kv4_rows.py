"""qsa_sparse_paged_kv4's form for many rows (a CTA takes four KV heads of a row, a warp each): several groups of heads,
several sequences, padding rows, bad pages, pools past 2^32 bytes.  The form is taken from 1.6 waves of CTAs on, four on an SM
(two for groups of more than 8 heads), so the sizes go by the device's SMs.  Bars as in test_gpu_kv4."""
from __future__ import annotations

import pytest
import torch

import kv4_ref as ref
import test_gpu_kv4 as kv4
from test_gpu_kv4 import qb  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu
PAGE, D = ref.PAGE, ref.D


def rows_for(Hkv, G, B=1):
    """Rows per sequence with which every GPU of this size takes the form: 1.7 waves."""
    slots = torch.cuda.get_device_properties(0).multi_processor_count * (4 if G <= 8 else 2)
    return -(-17 * slots * 4 // (10 * Hkv * B))


# heads, and of every sequence the rows that are padding and the tokens before its new ones (None: no new tokens)
CASES = [
    dict(Hkv=8, G=8, sequences=[(0, 0)], topk=70),                      # two groups of heads to a row
    dict(Hkv=8, G=3, sequences=[(5, 300), (0, 0), (17, 40)], topk=67),  # and several sequences, padding behind two of them
    dict(Hkv=12, G=1, sequences=[(0, 130), (None, 50)], topk=40),       # three groups; a sequence without new tokens
    dict(Hkv=4, G=8, sequences=[(1, 200), (130, 0)], topk=131),         # lists of more than a chunk
    dict(Hkv=4, G=13, sequences=[(3, 0), (None, 0), (40, 77)], topk=70),
    dict(Hkv=8, G=16, sequences=[(2, 10), (9, 500)], topk=35),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_heads_sequences_and_padding(qb, dtype, i):  # noqa: F811
    c = CASES[i]
    B = len(c["sequences"])
    S = rows_for(c["Hkv"], c["G"], B)
    new = [0 if pad is None else S - pad for pad, _ in c["sequences"]]
    ctx = [n + before for n, (_, before) in zip(new, c["sequences"])]
    c = kv4.make(B, S, c["Hkv"] * c["G"], c["Hkv"], ctx, new, c["topk"], dtype, 20 + i, keep=c["topk"] - 5, bad=True)
    x = kv4.exact(c)
    o, lse, status = kv4.run_attend(qb, c)
    assert status == 4
    kv4.check_attend(c, x, o, lse)  # (zeros and -infinity in the rows that are padding, too)
    o2, none, _ = kv4.run_attend(qb, c, lse=False)
    kv4.check_attend(c, x, o2, none)
    o3, lse3, _ = kv4.run_attend(qb, c)
    assert torch.equal(o3, o) and torch.equal(lse3, lse)
    total = torch.zeros((B, o.shape[2] // (c["q"].shape[2] // c["pool"].shape[2]), max(ctx)), device="cuda")
    w, status = kv4.run_weights(qb, c, lse, total)
    assert status == 4
    kv4.check_weights(c, x, lse, w, torch.zeros_like(total), total)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("Hkv,G", [(4, 4), (8, 12)])
def test_bad_pages(qb, dtype, Hkv, G):  # noqa: F811
    """An entry whose K or V page lies outside the pool names nothing, in every head and row that lists it."""
    S = rows_for(Hkv, G)
    c = kv4.make(1, S, G * Hkv, Hkv, [S + 100], [S], 100, dtype, 8, keep=90)
    good, flat, last = c["pt"].clone(), c["pool"].shape[0], (S + 99) // PAGE
    for page, plane, value in ((1, 0, flat), (2, 1, -1), (last, 0, 2 ** 31 - 1), (last, 1, -2 ** 31)):
        c["pt"][0, plane, page] = value
    broken = torch.isin(c["lists"] // PAGE, torch.tensor([1, 2, last], dtype=torch.int32)) & (c["lists"] >= 0)
    y = dict(c, pt=good, lists=torch.where(broken, torch.full_like(c["lists"], -1), c["lists"]))
    x = kv4.exact(y)
    o, lse, status = kv4.run_attend(qb, c)
    assert status == 2
    kv4.check_attend(y, x, o, lse)
    w, status = kv4.run_weights(qb, c, lse, None)
    assert status == 2
    kv4.check_weights(y, x, lse, w, None, None)


def test_pool_past_32_bit_offsets(qb):  # noqa: F811
    """Rows more than 2^32 bytes into a pool are read as the first ones are."""
    Hkv, G, row = 8, 2, 1024
    S = rows_for(Hkv, G)
    n = -(-S // PAGE)  # pages a plane
    pages = 2 ** 32 // (PAGE * Hkv * row) + 2 * n
    pool = torch.empty((pages, PAGE, Hkv, row), dtype=torch.uint8, device="cuda")
    small = torch.zeros((2 * n, PAGE, Hkv, ref.ROW), dtype=torch.uint8, device="cuda")
    near = torch.arange(2 * n, dtype=torch.int32).view(1, 2, n)
    kv = kv4.store_case(1, S, Hkv, "fp16", 3).cuda()
    c = kv4.make(1, S, G * Hkv, Hkv, [S], None, 67, "fp16", 12)
    ctx, lists, q = kv4.i32([S]).cuda(), c["lists"].cuda(), c["q"].cuda()
    got = []
    for p, pt in ((pool, (pages - 1 - near).cuda()), (small, near.cuda())):
        qb.store_kv4(kv[:, :, :Hkv], kv[:, :, Hkv:], ctx, p, pt)
        o, lse = torch.empty_like(q), torch.empty((1, S, G * Hkv), device="cuda")
        w = torch.empty((1, S, Hkv, 67), device="cuda")
        qb.sparse_paged_kv4(q, p, pt, lists, ctx, o, scale=0.1, lse=lse)
        qb.sparse_weights_kv4(q, p, pt, lists, ctx, lse, w, scale=0.1)
        got.append((o, lse, w))
    for x, y in zip(*got):
        assert torch.equal(x, y)
    assert bool(got[0][0].any())
