"""Runs a few steps of one named workload on cuda:0 through the C ABI.

A step is the whole path for that workload: qsa_indexer_prefill +
qsa_sparse_prefill for a prefill workload, qsa_indexer_decode +
qsa_sparse_decode for a decode workload.  Inputs come from the seeded
generators of `synthetic`.  The sizes can be overridden to get a case small
enough for a profiler's multi-pass capture (a decode pool of a few GB instead
of tens).

    python -m block_sparse_gqa_qsa_gb300.run_case prefill_S8192 --steps 2
    python -m block_sparse_gqa_qsa_gb300.run_case decode_long_B8_L512k --B 1 --steps 2
    python -m block_sparse_gqa_qsa_gb300.run_case prefill_S8192 --op rope --steps 2
    python -m block_sparse_gqa_qsa_gb300.run_case prefill_S8192 --impl tcgen05 --steps 1

`--op rope` runs qsa_rope_qkv on the workload's packed QKV instead (prefill
workloads: dense q/k/v outputs).  `--op handoff` (prefill workloads) runs the
indexer once, then qsa_indexer_prefill_handoff into a paged pool per step.
`--op gather` (decode workloads) runs one decode step for its lists, then
qsa_gather_selected into contiguous scratch per step.  `--op kv8` runs a
workload's steps on an 8-bit cache: qsa_append_kv8 (the whole prompts, or one
token per sequence), the indexer, and qsa_sparse_paged_kv8 over its lists; a
decode keeps the indexer's fp16 state in a one-head pool on the same page table.
`--op kv4` runs them on a 4-bit cache: qsa_rotary of the packed projections,
qsa_store_kv4, the indexer and qsa_sparse_paged_kv4; a decode step also gathers
its tokens' attention weights (qsa_sparse_weights_kv4), and behind the last step
qsa_evict_kv4 cuts every sequence back to 4096 tokens.

    python -m block_sparse_gqa_qsa_gb300.run_case prefill_S8192 --op kv8 --steps 2
    python -m block_sparse_gqa_qsa_gb300.run_case decode_B32_L2k-64k --op kv8 --steps 2
    python -m block_sparse_gqa_qsa_gb300.run_case decode_B32_L2k-64k --op kv4 --steps 2
"""
from __future__ import annotations

import argparse
import dataclasses
import math

import torch

from . import _binding as qb
from . import synthetic as syn


def _prefill_steps(cfg, steps, impl="mma"):
    t = {k: v.cuda() for k, v in syn.make_prefill(cfg).items()}
    ws = qb.alloc_workspace(qb.indexer_prefill_workspace_size(cfg.B, cfg.S, cfg.di, cfg.ratio))
    ind = torch.empty((cfg.B, cfg.S, cfg.topK), dtype=torch.int32, device="cuda")
    out = torch.empty((cfg.B, cfg.S, cfg.Hq, cfg.D), dtype=torch.float16, device="cuda")
    scale = float(torch.tensor(1.0 / math.sqrt(cfg.D), dtype=torch.float32))
    for _ in range(steps):
        qb.indexer_prefill(t["idxQ"], t["idxK"], t["wq"], t["wk"], t["ctx"], ind, ws, rot=cfg.rot, ratio=cfg.ratio,
                           budget=cfg.budget, topK=cfg.topK, theta=cfg.theta, eps=cfg.eps)
        qb.sparse_prefill(t["q"], t["k"], t["v"], ind, t["ctx"], out, scale, impl=impl)


def _rope_steps(cfg, steps):
    t = syn.make_prefill(cfg)
    qkv = torch.cat([t["q"], t["k"], t["v"]], dim=2).contiguous().cuda()
    wq, wk, ctx = t["wq"].cuda(), t["wk"].cuda(), t["ctx"].cuda()
    qo = torch.empty((cfg.B, cfg.S, cfg.Hq, cfg.D), dtype=torch.float16, device="cuda")
    ko = torch.empty((cfg.B, cfg.S, cfg.Hkv, cfg.D), dtype=torch.float16, device="cuda")
    vo = torch.empty_like(ko)
    for _ in range(steps):
        qb.rope_qkv(qkv, wq, wk, ctx, qo, Hq=cfg.Hq, Hkv=cfg.Hkv, rot=cfg.rot, theta=cfg.theta, eps=cfg.eps,
                    k_out=ko, v_out=vo)


def _handoff_steps(cfg, steps):
    t = {k: v.cuda() for k, v in syn.make_prefill(cfg).items()}
    ws = qb.alloc_workspace(qb.indexer_prefill_workspace_size(cfg.B, cfg.S, cfg.di, cfg.ratio))
    ind = torch.empty((cfg.B, cfg.S, cfg.topK), dtype=torch.int32, device="cuda")
    qb.indexer_prefill(t["idxQ"], t["idxK"], t["wq"], t["wk"], t["ctx"], ind, ws, rot=cfg.rot, ratio=cfg.ratio,
                       budget=cfg.budget, topK=cfg.topK, theta=cfg.theta, eps=cfg.eps)
    npg = -(-(cfg.S + 1) // syn.TOKENS_PER_PAGE)  # pages for S tokens and the next one, per sequence
    pool = torch.zeros((2 * cfg.B * npg, syn.TOKENS_PER_PAGE, cfg.Hkv, cfg.D + cfg.di), dtype=torch.float16,
                       device="cuda")
    ids = torch.arange(cfg.B * npg, dtype=torch.int32, device="cuda").view(cfg.B, npg)
    pt = torch.stack([ids, ids + cfg.B * npg], dim=1).contiguous()
    for _ in range(steps):
        qb.indexer_prefill_handoff(t["idxK"], t["ctx"], ws, pool, pt, D=cfg.D, ratio=cfg.ratio)


def _gather_steps(cfg, steps):
    d, ind = _decode_steps(cfg, 1)
    sc = qb.gather_scratch(cfg.B, cfg.Hkv, cfg.D, cfg.topK, device="cuda")
    for _ in range(steps):
        qb.gather_selected(d["pool"], d["page_table"], ind, d["ctx"], *sc, D=cfg.D)


KV8_BLOCK = 16  # tokens per scale of the 8-bit workloads


def _kv8_pool(flat, cfg):
    pool = torch.zeros((flat, syn.TOKENS_PER_PAGE, cfg.Hkv, cfg.D), dtype=torch.uint8, device="cuda")
    return (pool.view(torch.float8_e4m3fn),
            torch.ones((flat, syn.TOKENS_PER_PAGE // KV8_BLOCK, cfg.Hkv), device="cuda"))


def _kv8_weights(cfg):
    """Norm weights of the attention's q and k heads."""
    g = torch.Generator().manual_seed(cfg.seed)
    return [(0.1 * torch.randn(cfg.D, generator=g)).cuda() for _ in range(2)]


def _kv8_prefill_steps(cfg, steps):
    t = {k: v.cuda() for k, v in syn.make_prefill(cfg).items()}
    qkv = torch.cat([t["q"], t["k"], t["v"]], dim=2).contiguous()
    npg = -(-cfg.S // syn.TOKENS_PER_PAGE)
    ids = torch.randperm(cfg.B * npg, generator=torch.Generator().manual_seed(cfg.seed)).int().cuda().view(cfg.B, npg)
    pt = torch.stack([ids, ids + cfg.B * npg], dim=1).contiguous()
    pool, scale = _kv8_pool(2 * cfg.B * npg, cfg)
    wq, wk = _kv8_weights(cfg)
    ws = qb.alloc_workspace(qb.indexer_prefill_workspace_size(cfg.B, cfg.S, cfg.di, cfg.ratio))
    ind = torch.empty((cfg.B, cfg.S, cfg.topK), dtype=torch.int32, device="cuda")
    q = torch.empty((cfg.B, cfg.S, cfg.Hq, cfg.D), dtype=torch.float16, device="cuda")
    out = torch.empty_like(q)
    for _ in range(steps):
        qb.append_kv8(qkv, wq, wk, t["ctx"], q, pool, scale, pt, Hq=cfg.Hq, Hkv=cfg.Hkv, rot=cfg.rot, theta=cfg.theta,
                      eps=cfg.eps)
        qb.indexer_prefill(t["idxQ"], t["idxK"], t["wq"], t["wk"], t["ctx"], ind, ws, rot=cfg.rot, ratio=cfg.ratio,
                           budget=cfg.budget, topK=cfg.topK, theta=cfg.theta, eps=cfg.eps)
        qb.sparse_paged_kv8(q, pool, scale, pt, ind, t["ctx"], out, scale=cfg.scale)


def _kv8_decode_steps(cfg, steps):
    d = syn.make_decode(dataclasses.replace(cfg, Hkv=1), device="cuda")  # its one-head pool holds the indexer's state
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    pool, scale = _kv8_pool(d["pool"].shape[0], cfg)
    wq, wk = _kv8_weights(cfg)
    qkv = torch.randn((cfg.B, 1, cfg.Hq + 2 * cfg.Hkv, cfg.D), device="cuda").half()
    ws = qb.alloc_workspace(qb.indexer_decode_workspace_size(cfg.B, cfg.maxPagesPerSeq, cfg.ratio, cfg.budget))
    ind = torch.empty((cfg.B, 1, cfg.topK), dtype=torch.int32, device="cuda")
    q = torch.empty((cfg.B, 1, cfg.Hq, cfg.D), dtype=torch.float16, device="cuda")
    out = torch.empty_like(q)
    for _ in range(steps):
        qb.append_kv8(qkv, wq, wk, d["ctx"], q, pool, scale, d["page_table"], Hq=cfg.Hq, Hkv=cfg.Hkv, rot=cfg.rot,
                      theta=cfg.theta, eps=cfg.eps)
        qb.indexer_decode(d["idxQ"], d["idxK"], d["wq"], d["wk"], d["pool"], d["page_table"], d["ctx"], ind, ws, D=cfg.D,
                          rot=cfg.rot, ratio=cfg.ratio, budget=cfg.budget, topK=cfg.topK, theta=cfg.theta, eps=cfg.eps)
        qb.sparse_paged_kv8(q, pool, scale, d["page_table"], ind, d["ctx"], out, scale=cfg.scale)


KV4_BUDGET, KV4_SINKS, KV4_RECENT = 4096, 4, 256  # what the eviction behind the 4-bit decode steps keeps


def _kv4_prefill_steps(cfg, steps):
    t = {k: v.cuda() for k, v in syn.make_prefill(cfg).items()}
    qkv = torch.cat([t["q"], t["k"], t["v"]], dim=2).contiguous()
    npg = -(-cfg.S // syn.TOKENS_PER_PAGE)
    ids = torch.randperm(cfg.B * npg, generator=torch.Generator().manual_seed(cfg.seed)).int().cuda().view(cfg.B, npg)
    pt = torch.stack([ids, ids + cfg.B * npg], dim=1).contiguous()
    pool = torch.zeros((2 * cfg.B * npg, syn.TOKENS_PER_PAGE, cfg.Hkv, qb.KV4_ROW_BYTES), dtype=torch.uint8, device="cuda")
    row = torch.arange(cfg.S, dtype=torch.int32, device="cuda")
    pos = torch.where(row < t["ctx"][:, None], row, torch.full_like(row, -1))
    freq = qb.rotary_frequencies(cfg.rot, theta=cfg.theta)
    # every step turns the projections as they were (in place, a second step would turn them twice)
    turned = torch.zeros_like(qkv[:, :, :cfg.Hq + cfg.Hkv])
    qk, k, v = qkv[:, :, :cfg.Hq + cfg.Hkv], turned[:, :, cfg.Hq:], qkv[:, :, cfg.Hq + cfg.Hkv:]
    ws = qb.alloc_workspace(qb.indexer_prefill_workspace_size(cfg.B, cfg.S, cfg.di, cfg.ratio))
    ind = torch.empty((cfg.B, cfg.S, cfg.topK), dtype=torch.int32, device="cuda")
    out = torch.empty((cfg.B, cfg.S, cfg.Hq, cfg.D), dtype=torch.float16, device="cuda")
    for _ in range(steps):
        qb.rotary(qk, pos, turned, freq)
        qb.store_kv4(k, v, t["ctx"], pool, pt)
        qb.indexer_prefill(t["idxQ"], t["idxK"], t["wq"], t["wk"], t["ctx"], ind, ws, rot=cfg.rot, ratio=cfg.ratio,
                           budget=cfg.budget, topK=cfg.topK, theta=cfg.theta, eps=cfg.eps)
        qb.sparse_paged_kv4(turned[:, :, :cfg.Hq].contiguous(), pool, pt, ind, t["ctx"], out, scale=cfg.scale)
    return out, pool


def _kv4_decode_steps(cfg, steps):
    d = syn.make_decode(dataclasses.replace(cfg, Hkv=1), device="cuda")  # its one-head pool holds the indexer's state
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    ctx, pt = d["ctx"], d["page_table"]
    pool = torch.zeros((d["pool"].shape[0], syn.TOKENS_PER_PAGE, cfg.Hkv, qb.KV4_ROW_BYTES), dtype=torch.uint8, device="cuda")
    qkv = torch.randn((cfg.B, 1, cfg.Hq + 2 * cfg.Hkv, cfg.D), device="cuda").half()
    pos = (ctx - 1).view(cfg.B, 1)
    freq = qb.rotary_frequencies(cfg.rot, theta=cfg.theta)
    # every step turns the projections as they were (in place, a second step would turn them twice)
    turned = torch.zeros_like(qkv[:, :, :cfg.Hq + cfg.Hkv])
    qk, k, v = qkv[:, :, :cfg.Hq + cfg.Hkv], turned[:, :, cfg.Hq:], qkv[:, :, cfg.Hq + cfg.Hkv:]
    ws = qb.alloc_workspace(qb.indexer_decode_workspace_size(cfg.B, cfg.maxPagesPerSeq, cfg.ratio, cfg.budget))
    ind = torch.empty((cfg.B, 1, cfg.topK), dtype=torch.int32, device="cuda")
    out = torch.empty((cfg.B, 1, cfg.Hq, cfg.D), dtype=torch.float16, device="cuda")
    lse = torch.empty((cfg.B, 1, cfg.Hq), device="cuda")
    weights = torch.empty((cfg.B, 1, cfg.Hkv, cfg.topK), device="cuda")
    total = torch.zeros((cfg.B, cfg.Hkv, syn.TOKENS_PER_PAGE * cfg.maxPagesPerSeq), device="cuda")
    for _ in range(steps):
        qb.rotary(qk, pos, turned, freq)
        qb.store_kv4(k, v, ctx, pool, pt)
        qb.indexer_decode(d["idxQ"], d["idxK"], d["wq"], d["wk"], d["pool"], pt, ctx, ind, ws, D=cfg.D,
                          rot=cfg.rot, ratio=cfg.ratio, budget=cfg.budget, topK=cfg.topK, theta=cfg.theta, eps=cfg.eps)
        q = turned[:, :, :cfg.Hq].contiguous()
        qb.sparse_paged_kv4(q, pool, pt, ind, ctx, out, scale=cfg.scale, lse=lse)
        qb.sparse_weights_kv4(q, pool, pt, ind, ctx, lse, weights, total, scale=cfg.scale)
    kept = torch.empty((cfg.B, cfg.Hkv, KV4_BUDGET), dtype=torch.int32, device="cuda")
    lengths = torch.empty_like(ctx)
    qb.evict_kv4(pool, pt, ctx, total, kept, lengths, total, sinks=KV4_SINKS, recent=KV4_RECENT)
    return out, weights, kept, lengths


def _decode_steps(cfg, steps):
    d = syn.make_decode(cfg, device="cuda")
    d = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
    ws = qb.alloc_workspace(qb.indexer_decode_workspace_size(cfg.B, cfg.maxPagesPerSeq, cfg.ratio, cfg.budget))
    po, ps, pc = qb.sparse_decode_workspace_elems(cfg.B, cfg.Hkv, cfg.D)
    parts = (torch.zeros(po, device="cuda"), torch.zeros(ps, device="cuda"),
             torch.zeros(pc, dtype=torch.int32, device="cuda"))
    ind = torch.empty((cfg.B, 1, cfg.topK), dtype=torch.int32, device="cuda")
    out = torch.empty((cfg.B, 1, cfg.Hq, cfg.D), dtype=torch.float16, device="cuda")
    scale = float(torch.tensor(1.0 / math.sqrt(cfg.D), dtype=torch.float32))
    for _ in range(steps):
        qb.indexer_decode(d["idxQ"], d["idxK"], d["wq"], d["wk"], d["pool"], d["page_table"], d["ctx"], ind, ws,
                          D=cfg.D, rot=cfg.rot, ratio=cfg.ratio, budget=cfg.budget, topK=cfg.topK, theta=cfg.theta,
                          eps=cfg.eps)
        qb.sparse_decode(d["q"], d["pool"], d["page_table"], ind, d["ctx"], out, *parts, D=cfg.D, scale=scale)
    return d, ind


def main(argv=None):
    names = {c.name: c for c in syn.BENCH_CONFIGS + (syn.PREFILL_28K, syn.PREFILL_64K)}
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("workload", choices=sorted(names))
    ap.add_argument("--steps", type=int, default=2)
    ap.add_argument("--B", type=int, default=None, help="override the batch size")
    ap.add_argument("--ctx", type=int, default=None, help="decode: every sequence gets this total length")
    ap.add_argument("--Hkv", type=int, default=None,
                    help="decode: KV heads of the pool (Hq becomes 8 * Hkv); fewer heads make the pool smaller with "
                         "the same block-key stream per sequence")
    ap.add_argument("--impl", choices=("mma", "tcgen05"), default="mma",
                    help="prefill attention: qsa_sparse_prefill (mma.sync) or qsa_sparse_prefill_tcgen05")
    ap.add_argument("--op", choices=("path", "rope", "handoff", "gather", "kv8", "kv4"), default="path",
                    help="rope / handoff: qsa_rope_qkv / qsa_indexer_prefill_handoff of a prefill workload; "
                         "gather: qsa_gather_selected of a decode workload; kv8 / kv4: the workload's steps on an 8-bit / 4-bit "
                         "cache")
    args = ap.parse_args(argv)
    cfg = names[args.workload]
    if args.B is not None:
        cfg = dataclasses.replace(cfg, B=args.B)
    qb.lib()
    if args.op in ("rope", "handoff"):
        if isinstance(cfg, syn.DecodeConfig):
            ap.error(f"--op {args.op} takes a prefill workload")
        (_rope_steps if args.op == "rope" else _handoff_steps)(cfg, args.steps)
    elif args.op == "gather":
        if not isinstance(cfg, syn.DecodeConfig):
            ap.error("--op gather takes a decode workload")
        _gather_steps(cfg, args.steps)
    elif isinstance(cfg, syn.DecodeConfig):
        if args.ctx is not None:
            cfg = dataclasses.replace(cfg, ctx_lo=args.ctx, ctx_hi=args.ctx, max_ctx=max(args.ctx, 1), ctx_list=None)
        if args.Hkv is not None:
            cfg = dataclasses.replace(cfg, Hkv=args.Hkv, Hq=8 * args.Hkv)
        {"kv8": _kv8_decode_steps, "kv4": _kv4_decode_steps}.get(args.op, _decode_steps)(cfg, args.steps)
    elif args.op in ("kv8", "kv4"):
        (_kv8_prefill_steps if args.op == "kv8" else _kv4_prefill_steps)(cfg, args.steps)
    else:
        _prefill_steps(cfg, args.steps, args.impl)
    torch.cuda.synchronize()
    print(f"ok: {args.steps} steps of {cfg.name} (B={cfg.B})")


if __name__ == "__main__":
    main()
