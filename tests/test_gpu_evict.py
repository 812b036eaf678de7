"""qsa_evict_kv4 against a plain selection and move: every output and every byte of the pool is exact.  And the 4-bit cache's
operators as a server runs them, one behind the other."""
from __future__ import annotations

import math

import pytest
import torch

import kv4_ref as ref

pytestmark = pytest.mark.gpu
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


def totals(B, Hkv, T, seed, kind):
    g = torch.Generator().manual_seed(seed)
    if kind == "ties":
        return torch.randint(0, 4, (B, Hkv, T), generator=g).float() / 4
    if kind == "equal":
        return torch.full((B, Hkv, T), 0.25)
    w = torch.exp(2.0 * torch.randn((B, Hkv, T), generator=g) - 3)
    if kind == "odd":  # what no attention leaves, but a caller may
        w[..., ::7] = float("nan")
        w[..., 1::11] = float("inf")
        w[..., 2::5] *= -1
        w[..., 3::13] = -0.0
        w[..., 4::13] = 0.0
    return w


def check(qb, ctx, Hkv, budget, sinks, recent, kind="weights", T=None, row=ROW, seed=1, break_pages=False, inplace=False):
    B, T = len(ctx), T or max(1, max(ctx))
    pt, flat = ref.page_tables(ctx, seed, extra=1)
    g = torch.Generator().manual_seed(seed)
    pool = torch.randint(0, 256, (flat, PAGE, Hkv, row), generator=g, dtype=torch.int32).to(torch.uint8)
    if break_pages:
        pt[0, 0, 1], pt[0, 1, 0] = -5, flat
    total = totals(B, Hkv, T, seed, kind)
    want, kept = pool.clone(), torch.full((B, Hkv, budget), -1, dtype=torch.int32)
    moved, lengths, bad = torch.zeros_like(total), [], False
    for b in range(B):
        L = min(max(ctx[b], 0), T, PAGE * pt.shape[2])
        lengths.append(min(L, budget))
        for h in range(Hkv):
            keep = ref.evict(total[b, h], L, budget, sinks, recent)
            kept[b, h, :len(keep)] = torch.tensor(keep, dtype=torch.int32)
            moved[b, h, :len(keep)] = total[b, h, torch.tensor(keep, dtype=torch.long)]
            for i, j in enumerate(keep):
                for plane in (0, 1):
                    if i == j:
                        continue
                    src, dst = int(pt[b, plane, j // PAGE]), int(pt[b, plane, i // PAGE])
                    if 0 <= src < flat and 0 <= dst < flat:
                        want[dst, i % PAGE, h, :ROW] = pool[src, j % PAGE, h, :ROW]
                    else:
                        bad = True
    gp, gt = pool.cuda(), total.cuda()
    gk = torch.full((B, Hkv, budget), 9, dtype=torch.int32, device="cuda")
    gl = torch.full((B,), 9, dtype=torch.int32, device="cuda")
    out = gt if inplace else torch.full_like(gt, 9.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qb.evict_kv4(gp, pt.cuda(), i32(ctx).cuda(), gt, gk, gl, out, sinks=sinks, recent=recent, status=status)
    assert torch.equal(gk.cpu(), kept)
    assert gl.tolist() == lengths
    assert torch.equal(out.cpu().view(torch.int32), moved.view(torch.int32))
    assert torch.equal(gp.cpu(), want)
    assert int(status) == (2 if bad else 0)
    if not inplace:
        assert torch.equal(gt.cpu().view(torch.int32), total.view(torch.int32))


@pytest.mark.parametrize("ctx,Hkv,budget,sinks,recent", [
    ([2], 1, 1, 0, 0), ([2], 1, 1, 1, 0), ([2], 1, 1, 0, 1), ([1], 1, 1, 0, 0), ([0, 5], 2, 4, 1, 1), ([700], 2, 699, 0, 0),
    ([700, 64, 65, 63], 3, 64, 4, 20), ([1500, 1100], 1, 300, 0, 300), ([1500], 2, 300, 300, 0), ([1300], 4, 500, 100, 400),
    ([5000, 2047, 2048, 2049], 2, 2048, 4, 129), ([9001], 1, 4000, 16, 512), ([600] * 40, 8, 100, 2, 30)])
@pytest.mark.parametrize("kind", ["weights", "ties"])
def test_evict(qb, ctx, Hkv, budget, sinks, recent, kind):
    check(qb, ctx, Hkv, budget, sinks, recent, kind, seed=len(ctx) + budget)


@pytest.mark.parametrize("kind", ["equal", "odd"])
def test_equal_and_odd_totals(qb, kind):
    check(qb, [3000, 900], 2, 777, 3, 50, kind)


def test_totals_in_place(qb):
    check(qb, [3000, 100, 2500], 2, 640, 4, 64, inplace=True)
    check(qb, [20000], 1, 9000, 0, 1000, inplace=True)


def test_wide_rows_keep_their_tails(qb):
    check(qb, [1000, 700], 2, 300, 4, 64, row=112)


def test_lengths_past_the_totals_and_the_table(qb):
    check(qb, [1000, 300], 2, 200, 4, 64, T=517)
    check(qb, [400, 90], 1, 1000, 4, 64, T=2000)  # a budget above every length


def test_bad_pages_do_not_move(qb):
    check(qb, [900, 500], 2, 200, 4, 64, break_pages=True)


def test_long_caches(qb):
    """Clusters of 16, many rounds (the reference selects with sorts on the GPU)."""
    for B, Hkv, L, budget, sinks, recent in ((1, 2, 131072, 65536, 16, 2048), (2, 1, 70001, 1000, 4, 100), (1, 1, 40000, 39999, 0, 0)):
        ctx = [L - 17 * b for b in range(B)]
        pt, flat = ref.page_tables(ctx, 3)
        g = torch.Generator(device="cuda").manual_seed(5)
        pool = torch.randint(0, 256, (flat, PAGE, Hkv, ROW), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
        total = torch.randint(0, 100000, (B, Hkv, L), generator=g, device="cuda").float()
        before = pool.clone()
        kept = torch.empty((B, Hkv, budget), dtype=torch.int32, device="cuda")
        lengths, out = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty_like(total)
        qb.evict_kv4(pool, pt.cuda(), i32(ctx).cuda(), total, kept, lengths, out, sinks=sinks, recent=recent)
        assert lengths.tolist() == [budget] * B
        want = before.clone().view(-1, Hkv, ROW)
        for b in range(B):
            for h in range(Hkv):
                key = total[b, h, :ctx[b]].clone()
                key[:sinks] = math.inf
                key[ctx[b] - recent:] = math.inf
                order = torch.sort(key, descending=True, stable=True).indices[:budget].sort().values
                assert torch.equal(kept[b, h].long(), order)
                assert torch.equal(out[b, h, :budget], total[b, h, order]) and not bool(out[b, h, budget:].any())
                slot = torch.arange(budget, device="cuda")
                for plane in (0, 1):
                    row = pt[b, plane].long().cuda()
                    want[row[slot // PAGE] * PAGE + slot % PAGE, h] = \
                        before.view(-1, Hkv, ROW)[row[order // PAGE] * PAGE + order % PAGE, h]
        assert torch.equal(pool.view(-1, Hkv, ROW), want)


def test_graph_replay_and_another_stream(qb):
    ctx, Hkv, budget = [900, 1200], 2, 256
    pt, flat = ref.page_tables(ctx, 3)
    pool = ref.random_pool(flat, Hkv, 3).cuda()
    total = totals(2, Hkv, 1200, 4, "weights").cuda()
    args = (pt.cuda(), i32(ctx).cuda(), total)
    first = pool.clone()
    kept = torch.zeros((2, Hkv, budget), dtype=torch.int32, device="cuda")
    lengths = torch.zeros(2, dtype=torch.int32, device="cuda")
    qb.evict_kv4(first, *args, kept, lengths, recent=32)
    again, k2, l2 = pool.clone(), torch.zeros_like(kept), torch.zeros_like(lengths)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qb.evict_kv4(again, *args, k2, l2, recent=32)
    for _ in range(2):
        again.copy_(pool)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, first) and torch.equal(k2, kept) and torch.equal(l2, lengths)
    st = torch.cuda.Stream()
    again.copy_(pool)
    st.wait_stream(torch.cuda.current_stream())
    qb.evict_kv4(again, *args, k2, l2, recent=32, stream=st)
    st.synchronize()
    assert torch.equal(again, first)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_server_run(qb, dtype):
    """Two sequences: a prompt is rotated, stored and attended to; its last rows' weights decide an eviction; decoding goes
    on in the freed slots at the tokens' own positions, with totals that keep counting, and evicts once more.  Each step is
    compared with the 64-bit form of the same step on the cache as it is: stored bytes, kept tokens and moved rows exactly,
    outputs within the bars of the operators' own tests."""
    import test_gpu_kv4 as kv4
    import test_gpu_rotary as rot
    B, S, Hq, Hkv, budget, sinks, recent, window = 2, 300, 8, 2, 160, 4, 32, 16
    plen, scale = [300, 217], 1 / math.sqrt(D)
    freq = qb.rotary_frequencies(64, theta=1e4, scaling="blend", factor=4.0, original_length=128.0, low_turns=1.0, high_turns=4.0)
    pt, flat = ref.page_tables([384, 384], 2)
    pool = torch.zeros((flat, PAGE, Hkv, ROW), dtype=torch.uint8, device="cuda")
    gpt = pt.cuda()
    total = torch.zeros((B, Hkv, 384), device="cuda")
    g = torch.Generator().manual_seed(8)

    def step(x, pos, cache, new, lists, rows=slice(None)):
        """Rotates, stores, attends and weighs packed projections x [B, S, Hq + 2 Hkv, D]; rows: those that are weighed."""
        nonlocal pool
        turned, size = rot.turned(x[:, :, :Hq + Hkv], pos.clamp(min=0), freq)
        gx = x.cuda()
        qb.rotary(gx[:, :, :Hq + Hkv], pos.cuda(), gx[:, :, :Hq + Hkv], freq)
        live = pos >= 0
        rot.check(gx[:, :, :Hq + Hkv].cpu()[live], turned[live], size[live], dtype)
        before = pool.clone()
        qb.store_kv4(gx[:, :, Hq:Hq + Hkv], gx[:, :, Hq + Hkv:], i32(cache).cuda(), pool, gpt, new_lengths=i32(new).cuda())
        want = before.cpu()
        for b in range(B):
            for t in range(new[b]):
                p = cache[b] - new[b] + t
                r = ref.rows_of(gx[b, t, Hq:])
                want[pt[b, 0, p // PAGE], p % PAGE], want[pt[b, 1, p // PAGE], p % PAGE] = r[:Hkv], r[Hkv:]
        assert torch.equal(pool.cpu(), want)
        q = gx[:, :, :Hq].contiguous()
        c = dict(q=q.cpu(), pool=pool.cpu(), pt=pt, ctx=cache, new=new, n=new, lists=lists, scale=scale)
        x64 = kv4.exact(c)
        o, lse, status = kv4.run_attend(qb, c)
        assert status == 0
        kv4.check_attend(c, x64, o, lse)
        n = [max(0, min(m, window)) for m in new]
        last = dict(c, q=torch.stack([c["q"][b, max(0, new[b] - window):][:window] if new[b] >= window else c["q"][b, :window]
                                      for b in range(B)]))
        W = last["q"].shape[1]
        last.update(lists=torch.stack([lists[b, max(0, new[b] - W):][:W] for b in range(B)]), new=n, n=n)
        wl = torch.stack([lse[b, max(0, new[b] - W):][:W] for b in range(B)]).contiguous()
        y = kv4.exact(last)
        kept_total = total.clone()
        w, _ = kv4.run_weights(qb, last, wl, total)
        kv4.check_weights(last, y, wl, w, kept_total, total)

    def evict(cache):
        nonlocal pool
        before, tot = pool.cpu(), total.cpu()
        kept = torch.empty((B, Hkv, budget), dtype=torch.int32, device="cuda")
        lengths = torch.empty(B, dtype=torch.int32, device="cuda")
        qb.evict_kv4(pool, gpt, i32(cache).cuda(), total, kept, lengths, total, sinks=sinks, recent=recent)
        after = pool.cpu()
        for b in range(B):
            for h in range(Hkv):
                keep = ref.evict(tot[b, h], cache[b], budget, sinks, recent)
                assert kept[b, h, :len(keep)].tolist() == keep
                for plane in (0, 1):
                    old, new = ref.cached(before, pt[b, plane], cache[b])[:, h], ref.cached(after, pt[b, plane], len(keep))[:, h]
                    assert torch.equal(new, old[keep])
        return lengths.tolist()

    every = torch.arange(384, dtype=torch.int32)
    x = torch.randn((B, S, Hq + 2 * Hkv, D), generator=g).to(dtype)
    pos = torch.stack([torch.where(torch.arange(S) < n, torch.arange(S), torch.tensor(-1)) for n in plen]).to(torch.int32)
    lists = torch.where(every[None, None, :S] <= pos[..., None], every[None, None, :S], torch.tensor(-1, dtype=torch.int32))
    step(x, pos, plen, plen, lists.contiguous())
    cache = evict(plen)
    assert cache == [budget, budget]
    positions = list(plen)
    for turn in range(40):
        x = torch.randn((B, 1, Hq + 2 * Hkv, D), generator=g).to(dtype)
        pos = i32(positions).view(B, 1)
        cache = [c + 1 for c in cache]
        lists = torch.where(every[None, None, :256] < i32(cache).view(B, 1, 1), every[None, None, :256], torch.tensor(-1, dtype=torch.int32))
        step(x, pos, cache, [1, 1], lists.contiguous())
        positions = [p + 1 for p in positions]
        if turn == 24:
            cache = evict(cache)
    assert cache == [budget + 15] * 2


def test_workload_steps_on_a_4_bit_cache(qb, capsys):
    """run_case's 4-bit steps: finite outputs, weights that sum to the heads of a group, lengths cut to the budget."""
    import dataclasses
    from block_sparse_gqa_qsa_gb300 import run_case, synthetic as syn
    dec = dataclasses.replace(next(c for c in syn.BENCH_CONFIGS if c.name.startswith("decode_B32")), B=3, ctx_lo=5000,
                              ctx_hi=9000, max_ctx=9000)
    out, weights, kept, lengths = run_case._kv4_decode_steps(dec, 2)
    assert bool(torch.isfinite(out).all()) and lengths.tolist() == [run_case.KV4_BUDGET] * 3 and int(kept.min()) >= 0
    # (a weight is off by at most 2^-15 here: logits of at most 2^5, their sums, and the exponent's units)
    assert bool(((weights.sum(-1) - dec.Hq / dec.Hkv).abs() < 2.0 ** -10 * dec.Hq / dec.Hkv).all())
    run_case.main(["prefill_S8192", "--op", "kv4", "--steps", "1"])
    assert "ok: 1 steps" in capsys.readouterr().out


FIRST_CALL = """
import sys; sys.path[:0] = [{root!r}, {tests!r}]
import torch, kv4_ref as ref
from block_sparse_gqa_qsa_gb300 import _binding as qb
G = {group}
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
pt, flat = ref.page_tables([500, 300], 1)
pool, pt = ref.random_pool(flat, 2, 1).cuda(), pt.cuda()
kv = torch.randn(2, 1, 4, 128, device="cuda").half()
q = torch.randn(2, 1, 2 * G, 128, device="cuda").half()
ctx, pos, freq = i32([500, 300]), i32([[499], [299]]), qb.rotary_frequencies(64, theta=1e4)
lists = torch.arange({width}, dtype=torch.int32, device="cuda").expand(2, 1, {width}).contiguous()
out, lse, w = torch.zeros_like(q), torch.zeros(2, 1, 2 * G, device="cuda"), torch.zeros(2, 1, 2, {width}, device="cuda")
total, kept, length = torch.zeros(2, 2, 500, device="cuda"), torch.zeros(2, 2, 200, dtype=torch.int32, device="cuda"), i32([0, 0])
def step():
    qb.rotary(q, pos, q, freq)
    qb.store_kv4(kv[:, :, :2], kv[:, :, 2:], ctx, pool, pt)
    qb.sparse_paged_kv4(q, pool, pt, lists, ctx, out, scale=0.09, lse=lse)
    qb.sparse_weights_kv4(q, pool, pt, lists, ctx, lse, w, total, scale=0.09)
    qb.evict_kv4(pool, pt, ctx, total, kept, length, recent=16)
state = (q, pool, total)
saved = [t.clone() for t in state]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay(); torch.cuda.synchronize()
first = [t.clone() for t in (q, pool, out, lse, w, total, kept, length)]
for t, s in zip(state, saved): t.copy_(s)
step(); torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(first, (q, pool, out, lse, w, total, kept, length)))
assert length.tolist() == [200, 200] and bool(out.any()) and bool((w.sum(-1) - G).abs().max() < 1e-2 * G)
"""


@pytest.mark.parametrize("group,width", [(4, 100), (12, 100), (8, 290)])
def test_first_calls_of_a_process_may_be_captured(qb, group, width):
    """Nothing is set up by a first call that a capture would not allow."""
    import subprocess
    import sys
    from conftest import ROOT
    code = FIRST_CALL.format(root=ROOT, tests=ROOT + "/tests", group=group, width=width)
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_steps_of_a_workload_do_not_depend_on_their_number(qb):
    """run_case's 4-bit steps give the same outputs and the same cache after one step as after three: each turns the
    projections as they were.  (Totals add equal weights up, which keeps their order: the same tokens stay.)"""
    import dataclasses
    from block_sparse_gqa_qsa_gb300 import run_case, synthetic as syn
    pre = dataclasses.replace(next(c for c in syn.BENCH_CONFIGS if c.name == "prefill_S8192"), B=2, S=600)
    dec = dataclasses.replace(next(c for c in syn.BENCH_CONFIGS if c.name.startswith("decode_B32")), B=3, ctx_lo=5000,
                              ctx_hi=9000, max_ctx=9000)
    for run, cfg in ((run_case._kv4_prefill_steps, pre), (run_case._kv4_decode_steps, dec)):
        got = []
        for steps in (1, 3):
            torch.manual_seed(3)
            got.append(run(cfg, steps))
        for a, b in zip(*got):
            assert torch.equal(a, b)
