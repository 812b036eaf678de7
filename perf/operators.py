"""The paged-cache operators as measurable cases: appending keys and values
(16-bit pool and 8-bit pool with block scales) and sparse GQA attention over
the 8-bit pool.

`run` computes a case either in plain torch (`own` false) or with the library's
entry points (`own` true), on the state that `prepare` makes.  `exact` gives
the same outputs from the definitions in 64 bits.

What the operators compute
--------------------------
A sequence b has L_b tokens, the last n_b of them new; its row t < n_b is the
token at position p = L_b - n_b + t.  The page of token p is p // 128.

append:  q and k heads: y = x / sqrt(mean(x^2) + eps) * (1 + w), then dims i and
         i + rot/2 (i < rot/2) rotated by p * theta^(-2 i / rot); v heads as they
         are.  q rows go to q_out (zeros for rows t >= n_b), k and v rows to the
         pool rows of token p.
8 bits:  a block is `block` consecutive tokens of a page and one KV head; its
         values are code * s with an e4m3 code and one fp32 s per block.  A block
         whose first token is among the new ones gets s = amax / 448 over its new
         tokens; one that holds older tokens keeps its s, or takes s * 2^k with
         the smallest k that makes the new tokens fit (|x| <= 448 s 2^k), and the
         older tokens' codes are divided by 2^k.  s stays in [2^-48, 2^48].
attend:  o = sum_j softmax_j(scale * q . k_j) v_j over the list entries j of a
         row inside [0, L_b); zeros for rows t >= n_b and for empty lists.
"""
from __future__ import annotations

import math

import torch

own = False

PAGE = 128
THETA = 1.0e4
EPS = 1.0e-6
RATIO = 4  # tokens per list block
E4M3_MAX = 448.0
SCALE_LO, SCALE_HI = 2.0 ** -48, 2.0 ** 48
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one new token per sequence of a serving batch, 16-bit cache
        dict(name="append16_step_B32", op="append16", dtype="fp16", B=32, S=1, Hq=32, Hkv=4, D=128, rot=64,
             ctx_lo=2048, ctx_hi=65536, new_lo=1, new_hi=1, block=0),
        # chunks of prompts that continue at odd positions, bf16, smaller heads
        dict(name="append16_chunk_B3_S517", op="append16", dtype="bf16", B=3, S=517, Hq=8, Hkv=2, D=64, rot=32,
             ctx_lo=700, ctx_hi=9001, new_lo=101, new_hi=517, block=0),
        # the smallest call: one token of one sequence, where only latency counts
        dict(name="append8_step_B1", op="append8", dtype="fp16", B=1, S=1, Hq=8, Hkv=2, D=128, rot=32,
             ctx_lo=515, ctx_hi=515, new_lo=1, new_hi=1, block=16),
        # one new token per sequence of a serving batch, 8-bit cache
        dict(name="append8_step_B32", op="append8", dtype="bf16", B=32, S=1, Hq=32, Hkv=4, D=128, rot=64,
             ctx_lo=2048, ctx_hi=65536, new_lo=1, new_hi=1, block=16),
        # prompt chunks appended behind what is cached, blocks that straddle the old end
        dict(name="append8_chunk_B4_S1000", op="append8", dtype="fp16", B=4, S=1000, Hq=16, Hkv=2, D=128, rot=64,
             ctx_lo=2500, ctx_hi=6000, new_lo=333, new_hi=1000, block=32),
        # whole prompts of a ragged batch
        dict(name="append8_prefill_B4_S16384", op="append8", dtype="bf16", B=4, S=16384, Hq=32, Hkv=4, D=128, rot=64,
             ctx_lo=4096, ctx_hi=16384, new_lo=16384, new_hi=16384, block=16),
        # decode of one short sequence with a small list
        dict(name="attend8_step_B1_L512", op="attend8", dtype="fp16", B=1, S=1, Hq=8, Hkv=2, D=128, ctx_lo=512,
             ctx_hi=512, new_lo=1, new_hi=1, budget=16, block=16),
        # decode of a serving batch
        dict(name="attend8_step_B32", op="attend8", dtype="fp16", B=32, S=1, Hq=32, Hkv=4, D=128, ctx_lo=2048,
             ctx_hi=65536, new_lo=1, new_hi=1, budget=512, block=16),
        # decode of very long sequences
        dict(name="attend8_step_B8_L512k", op="attend8", dtype="bf16", B=8, S=1, Hq=64, Hkv=8, D=128, ctx_lo=524288,
             ctx_hi=524288, new_lo=1, new_hi=1, budget=512, block=64),
        # a few drafted tokens per sequence verified at once, a head group that is no power of two
        dict(name="attend8_verify_B6_S5", op="attend8", dtype="bf16", B=6, S=5, Hq=24, Hkv=2, D=128, ctx_lo=3,
             ctx_hi=6000, new_lo=1, new_hi=5, budget=128, block=4),
        # prompt chunks against a long cache
        dict(name="attend8_chunk_B2_S700", op="attend8", dtype="bf16", B=2, S=700, Hq=32, Hkv=4, D=128, ctx_lo=12000,
             ctx_hi=20000, new_lo=500, new_hi=700, budget=512, block=128),
        # a whole prompt, every row with its own list
        dict(name="attend8_prefill_S8192", op="attend8", dtype="fp16", B=1, S=8192, Hq=32, Hkv=4, D=128, ctx_lo=8192,
             ctx_hi=8192, new_lo=8192, new_hi=8192, budget=512, block=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append16", "append8", "append8", "attend8", "attend8", "attend8"))
    dtype = rng.choice(("fp16", "bf16"))
    Hkv = rng.choice((1, 2, 4, 8))
    Hq = Hkv * rng.choice((1, 4, 7, 8, 12, 16))
    step = rng.random() < 0.5
    B = _log_int(rng, 1, 32)
    if step:
        S = 1
    elif op == "attend8":
        S = _log_int(rng, 2, max(2, 6000 // B))
    else:
        S = _log_int(rng, 2, 12000 // B)
    S = max(S, 1)
    cap = 1200000 // (B * max(1, Hkv // 2)) if step else 24000
    hi = max(S, _log_int(rng, 5, min(cap, 400000)))
    lo = min(hi, max(1, _log_int(rng, 1, hi)))
    c = dict(op=op, dtype=dtype, B=B, S=S, Hq=Hq, Hkv=Hkv, D=128, ctx_lo=lo, ctx_hi=hi,
             new_lo=rng.randint(0 if S > 1 else 1, S), new_hi=S,
             block=0 if op == "append16" else rng.choice((1, 4, 16, 32, 64, 128)))
    if op == "attend8":
        while S > 1 and B * S * Hq > 32 * 6000:
            S = c["S"] = c["new_hi"] = max(1, S // 2)
            c["new_lo"] = min(c["new_lo"], S)
        c["budget"] = _log_int(rng, 16, 512)
    else:
        c["D"] = rng.choice((64, 128))
        c["rot"] = rng.choice((16, 32, 64))
    return c


# ------------------------------------------------------------- the lengths
def _spread(lo, hi, B, mult):
    """B values over [lo, hi], the ends among them, in no sorted order; they go by the case alone."""
    if B == 1:
        return [hi]
    return [lo + (hi - lo) * ((i * mult) % B) // (B - 1) for i in range(B)]


def _coprime(B, m):
    while math.gcd(m, B) != 1:
        m += 1
    return m


def _lengths(case):
    B, S = case["B"], case["S"]
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], B, _coprime(B, 5))
    new = [min(n, S, L) for n, L in zip(_spread(case["new_lo"], case["new_hi"], B, _coprime(B, 3)), ctx)]
    return ctx, new


def _entries(case):
    """Valid list entries of every live row, over the batch."""
    total = 0
    for L, n in zip(*_lengths(case)):
        for p in range(L - n, L):
            nc = (p + 1) // RATIO
            total += min(nc, case["budget"]) * RATIO + (p + 1 - nc * RATIO)
    return total


def work(case):
    B, S, Hq, Hkv, D = (case[k] for k in ("B", "S", "Hq", "Hkv", "D"))
    ctx, new = _lengths(case)
    N = sum(new)
    if case["op"] == "attend8":
        ent = _entries(case)
        # a cached row that several lists name is read once
        rows = sum(min(L, sum(min((p + 1) // RATIO, case["budget"]) * RATIO + (p + 1) % RATIO
                              for p in range(L - n, L))) for L, n in zip(ctx, new))
        nbytes = rows * 2 * Hkv * D + rows * 2 * Hkv * 4 // case["block"] + ent * 4 + N * Hq * D * 2 + B * S * Hq * D * 2
        return {"bytes": nbytes, "flops": 4 * ent * Hq * D}
    kv = 1 if case["op"] == "append8" else 2
    nbytes = N * (Hq + 2 * Hkv) * D * 2 + B * S * Hq * D * 2 + N * 2 * Hkv * D * kv
    if kv == 1:
        nbytes += 2 * Hkv * 4 * sum((L - 1) // case["block"] - (L - n) // case["block"] + 1 for L, n in zip(ctx, new) if n)
    return {"bytes": nbytes, "flops": N * (Hq + Hkv) * D * 8}


# ------------------------------------------------------------------ inputs
def _tables(case, ctx, g):
    """K pages are a random permutation of [0, n), a V page is its K page + n; tables as wide as the longest needs."""
    pages = [max(1, -(-L // PAGE)) for L in ctx]
    n = sum(pages)
    perm = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    pt = torch.zeros((len(ctx), 2, max(pages)), dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(pages):
        pt[b, 0, :m] = perm[at:at + m]
        pt[b, 1, :m] = perm[at:at + m] + n
        at += m
    return pt, 2 * n


def _codes(shape, g):
    """e4m3 codes as a quantiser leaves them: normal values scaled to reach about 448."""
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        m = min(step, flat.numel() - i)
        x = torch.randn(m, generator=g, dtype=torch.float16, device="cuda")
        flat[i:i + m].copy_(x.mul_(128).clamp_(-E4M3_MAX, E4M3_MAX))
    return out


def _lists(case, ctx_t, new_t, g):
    """Lists as the block indexer gives them: `budget` blocks of RATIO tokens, then the causal tail, ascending, -1 behind."""
    B, S, budget = case["B"], case["S"], case["budget"]
    topk = budget * RATIO + RATIO - 1
    nb = max(1, max(_lengths(case)[0]) // RATIO)
    out = torch.full((B, S, topk), -1, dtype=torch.int32, device="cuda")
    big = 1 << 30
    step = max(1, (1 << 26) // nb)
    for b in range(B):
        for t0 in range(0, S, step):
            t = torch.arange(t0, min(S, t0 + step), device="cuda")
            live = t < new_t[b]
            p = ctx_t[b] - new_t[b] + t
            nc = torch.where(live, (p + 1) // RATIO, torch.zeros_like(p))
            key = torch.rand((t.numel(), nb), generator=g, device="cuda")
            key = torch.where(torch.arange(nb, device="cuda")[None] < nc[:, None], key, torch.full_like(key, -1.0))
            top = torch.topk(key, min(budget, nb), dim=1)
            tok = top.indices[:, :, None] * RATIO + torch.arange(RATIO, device="cuda")
            tok = torch.where((top.values >= 0)[:, :, None], tok, torch.full_like(tok, big)).flatten(1)
            tail = nc[:, None] * RATIO + torch.arange(RATIO - 1, device="cuda")
            tail = torch.where(live[:, None] & (tail <= p[:, None]), tail, torch.full_like(tail, big))
            ids = torch.sort(torch.cat([tok, tail], dim=1), dim=1).values
            out[b, t0:t0 + t.numel(), :ids.shape[1]] = torch.where(ids == big, torch.full_like(ids, -1), ids).to(torch.int32)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    B, S, Hq, Hkv, D = (case[k] for k in ("B", "S", "Hq", "Hkv", "D"))
    dt = DTYPES[case["dtype"]]
    ctx, new = _lengths(case)
    s = {"case": case}
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    s["new"] = torch.tensor(new, dtype=torch.int32, device="cuda")
    s["pt"], flat = _tables(case, ctx, g)
    if case["op"] == "append16":
        s["pool"] = torch.randn((flat, PAGE, Hkv, D), generator=g, dtype=torch.float16, device="cuda").to(dt)
    else:
        s["pool"] = _codes((flat, PAGE, Hkv, D), g)
        nblk = PAGE // case["block"]
        s["scale"] = 0.0078 * torch.exp(0.3 * torch.randn((flat, nblk, Hkv), generator=g, device="cuda"))
    if case["op"] == "attend8":
        s["q"] = torch.randn((B, S, Hq, D), generator=g, device="cuda").to(dt)
        s["lists"] = _lists(case, s["ctx"].long(), s["new"].long(), g)
        s["out"] = torch.empty((B, S, Hq, D), dtype=dt, device="cuda")
        return s
    s["qkv"] = torch.randn((B, S, Hq + 2 * Hkv, D), generator=g, device="cuda", dtype=torch.float16).to(dt)
    s["wq"] = 0.1 * torch.randn(D, generator=g, device="cuda")
    s["wk"] = 0.1 * torch.randn(D, generator=g, device="cuda")
    s["q_out"] = torch.empty((B, S, Hq, D), dtype=dt, device="cuda")
    # the live rows, and for each its position, and its rows of the pool: a program that keeps the lengths has these
    b = torch.repeat_interleave(torch.arange(B, device="cuda"), s["new"].long(), output_size=sum(new))
    first = torch.cumsum(s["new"].long(), 0) - s["new"].long()
    t = torch.arange(sum(new), device="cuda") - first[b]
    s["rows"] = b * S + t
    s["pos"] = (s["ctx"].long() - s["new"].long())[b] + t
    pt = s["pt"].long()
    s["slot"] = torch.stack([pt[b, i, s["pos"] // PAGE] * PAGE + s["pos"] % PAGE for i in (0, 1)])
    if case["op"] == "append8":
        blk = case["block"]
        # blocks that get new tokens: [plane][pool block], which block each row is in, and the older rows of the blocks
        ids, inv = torch.unique(s["slot"] // blk, return_inverse=True)
        s["blocks"], s["block_of"] = ids, inv
        start = (s["ctx"] - s["new"]).tolist()
        old = [(i, c, p) for i, (c, n) in enumerate(zip(start, new)) if n for p in range(c - c % blk, c)]
        o = torch.tensor(old, dtype=torch.long, device="cuda").reshape(-1, 3)
        slot = torch.cat([pt[o[:, 0], i, o[:, 2] // PAGE] * PAGE + o[:, 2] % PAGE for i in (0, 1)])
        s["old"] = slot
        s["old_block"] = torch.searchsorted(ids, slot // blk)
        has = torch.zeros(ids.numel(), dtype=torch.bool, device="cuda")
        has[s["old_block"]] = True
        s["has_old"] = has
    return s


# -------------------------------------------------------------- plain forms
def _rotated(x, w, pos, rot):
    """RMSNorm * (1 + w), then the rotation, of x [N, H, D] at positions pos [N], in 32 bits (angles in 64)."""
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * (1.0 + w)
    h = rot // 2
    freq = THETA ** (-2.0 * torch.arange(h, dtype=torch.float64, device=x.device) / rot)
    ang = pos.double()[:, None] * freq
    c, s = ang.cos().float()[:, None], ang.sin().float()[:, None]
    a, b = y[..., :h], y[..., h:rot]
    return torch.cat([a * c - b * s, b * c + a * s, y[..., rot:]], dim=-1)


def _append(s):
    case = s["case"]
    B, S, Hq, Hkv, D = (case[k] for k in ("B", "S", "Hq", "Hkv", "D"))
    x = s["qkv"].view(B * S, Hq + 2 * Hkv, D)[s["rows"]]
    q = s["q_out"].view(B * S, Hq, D)
    q.zero_()
    q[s["rows"]] = _rotated(x[:, :Hq], s["wq"], s["pos"], case["rot"]).to(q.dtype)
    k = _rotated(x[:, Hq:Hq + Hkv], s["wk"], s["pos"], case["rot"])
    v = x[:, Hq + Hkv:]
    rows = s["pool"].view(-1, Hkv, D)
    if case["op"] == "append16":
        rows[s["slot"][0]] = k.to(rows.dtype)
        rows[s["slot"][1]] = v
        return {"q": s["q_out"], "pool": s["pool"]}
    kv = torch.stack([k, v.float()])
    scale = s["scale"].view(-1, Hkv)
    amax = torch.zeros((s["blocks"].numel(), Hkv), device=kv.device)
    at = s["block_of"].flatten()[:, None].expand(-1, Hkv)
    amax.scatter_reduce_(0, at, kv.abs().amax(-1).flatten(0, 1), "amax")
    kept = scale[s["blocks"]]
    m, e = torch.frexp(amax / (E4M3_MAX * kept))
    up = torch.where(m == 0.5, e - 1, e).clamp(min=0)  # smallest k >= 0 with amax <= 448 kept 2^k
    grown = torch.ldexp(kept, up).clamp(SCALE_LO, SCALE_HI)
    fresh = (amax / E4M3_MAX).clamp(SCALE_LO, SCALE_HI)
    now = torch.where(s["has_old"][:, None], grown, fresh)
    scale[s["blocks"]] = now
    rows8 = rows.view(torch.uint8)
    before = rows8[s["old"]].view(torch.float8_e4m3fn).float() * (kept / now)[s["old_block"]][..., None]
    rows8[s["old"]] = before.to(torch.float8_e4m3fn).view(torch.uint8)
    code = (kv / now[s["block_of"]][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    rows8[s["slot"].flatten()] = code.view(torch.uint8).flatten(0, 1)
    return {"q": s["q_out"], "pool": s["pool"], "scale": s["scale"]}


def _attend(s):
    case = s["case"]
    B, S, Hq, Hkv, D, blk = (case[k] for k in ("B", "S", "Hq", "Hkv", "D", "block"))
    topk = s["lists"].shape[-1]
    lists, q = s["lists"].view(B * S, topk), s["q"].view(B * S, Hkv, Hq // Hkv, D)
    out = s["out"].view(B * S, Hkv, Hq // Hkv, D)
    rows, scale = s["pool"].view(torch.uint8).view(-1, Hkv, D), s["scale"].view(-1, Hkv)
    step = max(1, (1 << 28) // (topk * Hkv * D))
    for r0 in range(0, B * S, step):
        r = torch.arange(r0, min(B * S, r0 + step), device=q.device)
        b = r // S
        j = lists[r0:r0 + step].long()
        valid = (j >= 0) & (j < s["ctx"][b][:, None]) & (r % S < s["new"][b])[:, None]
        j = torch.where(valid, j, torch.zeros_like(j))

        def cached(plane):  # [rows, Hkv, topk, D] in 32 bits
            at = s["pt"][b[:, None], plane, j // PAGE].long() * PAGE + j % PAGE
            x = rows[at].view(torch.float8_e4m3fn).float() * scale[at // blk][..., None]
            return torch.where(valid[..., None, None], x, torch.zeros_like(x)).transpose(1, 2)

        logit = torch.matmul(q[r0:r0 + step].float(), cached(0).transpose(2, 3)) / math.sqrt(D)
        logit = logit.masked_fill(~valid[:, None, None, :], -math.inf)
        top = logit.amax(-1, keepdim=True)
        p = torch.exp(logit - torch.where(top == -math.inf, torch.zeros_like(top), top))
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p, cached(1)) / torch.where(total == 0, torch.ones_like(total), total)
        out[r0:r0 + step] = o.to(out.dtype)
    return s["out"]


def run(s):
    case = s["case"]
    if own:
        from block_sparse_gqa_qsa_gb300 import _binding as qb
        if case["op"] == "attend8":
            qb.sparse_paged_kv8(s["q"], s["pool"], s["scale"], s["pt"], s["lists"], s["ctx"], s["out"],
                                scale=1.0 / math.sqrt(case["D"]), new_lengths=s["new"])
            return s["out"]
        heads = dict(Hq=case["Hq"], Hkv=case["Hkv"], rot=case["rot"], theta=THETA, eps=EPS, new_lengths=s["new"])
        if case["op"] == "append16":
            qb.append_kv(s["qkv"], s["wq"], s["wk"], s["ctx"], s["q_out"], s["pool"], s["pt"], **heads)
            return {"q": s["q_out"], "pool": s["pool"]}
        qb.append_kv8(s["qkv"], s["wq"], s["wk"], s["ctx"], s["q_out"], s["pool"], s["scale"], s["pt"], **heads)
        return {"q": s["q_out"], "pool": s["pool"], "scale": s["scale"]}
    return _attend(s) if case["op"] == "attend8" else _append(s)


# ------------------------------------------------------- 64-bit definitions
def _grid_e4m3(x):
    """x (64-bit, |x| <= 448) rounded to the nearest e4m3 value, ties to even: 4 significant bits, steps of 2^-9 at least."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 4).clamp(min=-9))
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_head(x, w, p, rot):
    """One token's heads [H, D] at position p, in 64 bits."""
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * (1.0 + w)
    h = rot // 2
    i = torch.arange(h, dtype=torch.float64, device=x.device)
    turn = torch.exp(1j * p[:, None] * torch.exp(i * (-2.0 * math.log(THETA) / rot)))[:, None]
    z = torch.complex(y[..., :h].contiguous(), y[..., h:rot].contiguous()) * turn
    return torch.cat([z.real, z.imag, y[..., rot:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    B, S, Hq, Hkv, D = (case[k] for k in ("B", "S", "Hq", "Hkv", "D"))
    ctx, new = _lengths(case)
    if case["op"] == "attend8":
        return _exact_attend(s, ctx, new)
    q = torch.zeros((B, S, Hq, D), dtype=torch.float64, device="cuda")
    wq, wk = s["wq"].double(), s["wk"].double()
    small = case["op"] == "append16"
    pool = s["pool"].to(torch.float64)
    scale = None if small else s["scale"].double()
    for b in range(B):
        n, c = new[b], ctx[b] - new[b]
        if n == 0:
            continue
        x = s["qkv"][b, :n].double()
        p = torch.arange(c, c + n, device="cuda", dtype=torch.float64)
        q[b, :n] = _exact_head(x[:, :Hq], wq, p, case["rot"])
        for plane, val in ((0, _exact_head(x[:, Hq:Hq + Hkv], wk, p, case["rot"])), (1, x[:, Hq + Hkv:])):
            pages = s["pt"][b, plane].long()
            pi = p.long()
            if small:
                pool[pages[pi // PAGE], pi % PAGE] = val
                continue
            blk = case["block"]
            # the blocks from the one that holds token c to the one that holds token c + n - 1, as a dense [m, blk] array
            lo, hi = c // blk, (c + n - 1) // blk
            m = hi - lo + 1
            dense = torch.zeros((m * blk, Hkv, D), dtype=torch.float64, device="cuda")
            dense[c - lo * blk:c - lo * blk + n] = val
            tok = torch.arange(lo * blk, (hi + 1) * blk, device="cuda")
            page, off = pages[(tok // PAGE).clamp(max=pages.numel() - 1)], tok % PAGE
            amax = dense.view(m, blk, Hkv, D).abs().amax((1, 3))
            want = (amax / E4M3_MAX).clamp(SCALE_LO, SCALE_HI)
            if c % blk:
                had = scale[page[0], off[0] // blk]
                k = torch.ceil(torch.log2((amax[0] / (E4M3_MAX * had)).clamp(min=1e-300))).clamp(min=0)
                want[0] = (had * 2.0 ** k).clamp(SCALE_LO, SCALE_HI)
                oldrow = tok < c
                before = pool[page[oldrow], off[oldrow]] * (had / want[0])[:, None]
                pool[page[oldrow], off[oldrow]] = _grid_e4m3(before)
            scale[page.view(m, blk)[:, 0], off.view(m, blk)[:, 0] // blk] = want
            isnew = (tok >= c) & (tok < c + n)
            code = _grid_e4m3(dense / want.repeat_interleave(blk, 0)[:, :, None])
            pool[page[isnew], off[isnew]] = code[isnew]
    return {"q": q, "pool": pool} if small else {"q": q, "pool": pool, "scale": scale}


def _exact_attend(s, ctx, new):
    case = s["case"]
    B, S, Hq, Hkv, D, blk = (case[k] for k in ("B", "S", "Hq", "Hkv", "D", "block"))
    G = Hq // Hkv
    out = torch.zeros((B, S, Hq, D), dtype=torch.float64, device="cuda")
    for b in range(B):
        n, L = new[b], ctx[b]
        if n == 0 or L == 0:
            continue
        step = max(1, min(n, (1 << 26) // (L * G)))
        for h in range(Hkv):
            whole = []
            for plane in (0, 1):
                pg = s["pt"][b, plane, :-(-L // PAGE)].long()
                x = s["pool"][:, :, h].view(torch.uint8)[pg].view(torch.float8_e4m3fn).double()
                x = x.view(pg.numel(), PAGE // blk, blk, D) * s["scale"][pg][:, :, h].double()[:, :, None, None]
                whole.append(x.view(-1, D)[:L])
            for t0 in range(0, n, step):
                t1 = min(n, t0 + step)
                idx = s["lists"][b, t0:t1].long()
                ok = (idx >= 0) & (idx < L)
                count = torch.zeros((t1 - t0, L), dtype=torch.float64, device="cuda")
                count.scatter_add_(1, idx.clamp(0, L - 1), ok.double())
                z = s["q"][b, t0:t1, h * G:(h + 1) * G].double() @ whole[0].T / math.sqrt(D)
                z = torch.where(count[:, None] > 0, z, torch.full_like(z, -math.inf))
                w = torch.softmax(z, -1) * count[:, None]
                w = torch.nan_to_num(w)
                den = w.sum(-1, keepdim=True)
                out[b, t0:t1, h * G:(h + 1) * G] = (w @ whole[1]) / torch.where(den == 0, torch.ones_like(den), den)
    return out
