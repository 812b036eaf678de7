"""Operators around a cache held in 4 bits, as measurable cases: rotary positions in both layouts, storing keys and
values in 4 bits, sparse GQA attention over the 4-bit pool, the attention weight that its tokens gather, and eviction by
that weight.

`run` computes a case either in plain torch (`own` false) or with the library's entry points (`own` true), on the state
that `prepare` makes.  `exact` gives the same outputs from the definitions in 64 bits.

What the operators compute
--------------------------
rotary:   dims (i, i + rot/2) (halves) or (2 i, 2 i + 1) (interleaved), i < rot/2, of every head of a token at position p
          turn by p f_i (back by it: inverse, the gradient), times a magnitude; the other dims stay; tokens at negative
          positions are left alone.  f_i = theta^(-2 i / rot), or scaled for long contexts: "linear" f_i / factor,
          "blend" (f_i / factor where the pair turns less than `low` times in the original length, f_i where it turns
          more than `high` times, in between a mean that is linear in the turns), "base" (theta raised so that the
          slowest pair slows down by the factor).
4 bits:   a cached row (one token, one KV head, K or V) is 80 bytes: 128 codes (e2m1: 0 0.5 1 1.5 2 3 4 6 and a sign; dim
          2 i in the low half of byte i), 8 scales s_j (e4m3) of 16 dims each, a row scale t (fp32, a power of two), 4
          zero bytes.  It stands for code * s_j * t.  t is the smallest power of two in [2^-48, 2^48] with
          amax <= 2688 t, s_j = amax_j / (6 t) and code = x / (s_j t), each to the nearest (ties to even), saturating; a
          code has its value's sign even where it is 0.
store:    the last n_b of sequence b's L_b tokens: row t of k and v goes to the pool rows of token L_b - n_b + t; k_out and
          v_out get the values the rows stand for (zeros for rows t >= n_b).
attend:   o = sum_j softmax_j(scale q . k_j) v_j over the entries j of a row's list inside [0, L_b); zeros for rows
          t >= n_b and for empty lists.  lse: log sum_j exp(scale q . k_j), -inf where there is no j.
weights:  w[e] = sum over the query heads of a KV head of exp(scale q . k_e - lse) for every list entry e (0 for one that
          names nothing), and total[j] += the sum of w over the entries that name token j.
evict:    keeps min(L_b, budget) tokens of every KV head: the first `sinks`, the last `recent`, and of the others those with
          the largest total (ties: the lowest).  They move up in order to the first slots of the sequence.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

PAGE = 128
D = 128
ROW = 80      # bytes of a cached row
AT_SCALE = 64  # its 8 group scales
AT_ROW = 72   # its row scale
RATIO = 4     # tokens per list block
THETA = 1.0e4
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of each sequence of a serving batch, in place in the packed projections
        dict(name="rotary_step_B32", op="rotary", dtype="bf16", T=32, H=36, X=40, D=128, rot=64, interleaved=False,
             scaling="none", factor=1.0, magnitude=1.0, inverse=False, inplace=True, pos_lo=2048, pos_hi=65536, pad=0),
        # a long prompt past the trained length, interleaved pairs, padding behind it
        dict(name="rotary_prompt_T16384", op="rotary", dtype="fp16", T=16384, H=36, X=36, D=128, rot=128,
             interleaved=True, scaling="blend", factor=8.0, magnitude=1.2, inverse=False, inplace=False, pos_lo=0,
             pos_hi=131072, pad=111),
        # the gradient's way back in 32 bits, a part of odd width of heads of another size
        dict(name="rotary_grad_T5003", op="rotary", dtype="fp32", T=5003, H=24, X=24, D=96, rot=36, interleaved=False,
             scaling="base", factor=4.0, magnitude=1.0, inverse=True, inplace=False, pos_lo=0, pos_hi=20000, pad=0),
        # one new token of each sequence of a serving batch
        dict(name="store4_step_B32", op="store", dtype="bf16", B=32, S=1, Hkv=4, ctx_lo=2048, ctx_hi=65536, new_lo=1,
             new_hi=1),
        # whole prompts of a ragged batch
        dict(name="store4_prompt_B4_S16384", op="store", dtype="fp16", B=4, S=16384, Hkv=4, ctx_lo=4096, ctx_hi=16384,
             new_lo=16384, new_hi=16384),
        # decode of one short sequence with a small list: the smallest call, where only latency counts
        dict(name="attend4_step_B1_L512", op="attend", dtype="fp16", B=1, S=1, Hq=14, Hkv=2, ctx_lo=512, ctx_hi=512,
             new_lo=1, new_hi=1, budget=16, lse=False),
        # decode of a serving batch that goes on to count its tokens' weights
        dict(name="attend4_step_B32", op="attend", dtype="bf16", B=32, S=1, Hq=32, Hkv=4, ctx_lo=2048, ctx_hi=65536,
             new_lo=1, new_hi=1, budget=512, lse=True),
        # a whole prompt, every row with its own list
        dict(name="attend4_prompt_S8192", op="attend", dtype="fp16", B=1, S=8192, Hq=32, Hkv=4, ctx_lo=8192, ctx_hi=8192,
             new_lo=8192, new_hi=8192, budget=512, lse=False),
        # weights of a decode step of a serving batch
        dict(name="weights4_step_B32", op="weights", dtype="bf16", B=32, S=1, Hq=32, Hkv=4, ctx_lo=2048, ctx_hi=65536,
             new_lo=1, new_hi=1, budget=512),
        # weights of the last rows of ragged prompts, before a first eviction; a head group that is no power of two
        dict(name="weights4_window_B3_S37", op="weights", dtype="fp16", B=3, S=37, Hq=24, Hkv=2, ctx_lo=5000,
             ctx_hi=24001, new_lo=20, new_hi=37, budget=512),
        # a serving batch whose caches are cut back to their budget
        dict(name="evict4_B32_to_4096", op="evict", B=32, Hkv=4, ctx_lo=3000, ctx_hi=9001, budget=4096, sinks=4,
             recent=512),
        # long prompts cut to half
        dict(name="evict4_B2_L131072", op="evict", B=2, Hkv=4, ctx_lo=120001, ctx_hi=131072, budget=65536, sinks=16,
             recent=2048),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rotary", "store", "attend", "attend", "weights", "evict"))
    if op == "rotary":
        dtype = rng.choice(("fp16", "bf16", "fp32"))
        dim = rng.choice((64, 96, 128, 256))
        H = rng.choice((1, 5, 12, 36))
        T = _log_int(rng, 1, 64000000 // (H * dim * (2 if dtype == "fp32" else 1)))
        scaling = rng.choice(("none", "linear", "blend", "base"))
        inplace = rng.random() < 0.5
        return dict(op=op, dtype=dtype, T=min(T, 40000), H=H, X=H + rng.choice((0, 1, 4)), D=dim,
                    rot=2 * rng.randint(1, dim // 2) if rng.random() < 0.3 else rng.choice((dim, dim // 2, 32)),
                    interleaved=rng.random() < 0.5, scaling=scaling, factor=1.0 if scaling == "none" else rng.choice((2.0, 8.0)),
                    magnitude=1.0 if inplace else rng.choice((1.0, 0.9)), inverse=rng.random() < 0.3, inplace=inplace,
                    pos_lo=0, pos_hi=_log_int(rng, 10, 1000000), pad=rng.choice((0, 0, min(T, 40000) // 9)))
    B = _log_int(rng, 1, 32)
    Hkv = rng.choice((1, 2, 3, 4, 8))
    if op == "evict":
        hi = _log_int(rng, 10, min(131072, 1000000 // (B * Hkv)))
        budget = _log_int(rng, 4, hi + hi // 4)
        recent = rng.randint(0, budget // 2)
        return dict(op=op, B=B, Hkv=Hkv, ctx_lo=max(1, hi - rng.randint(0, hi - 1)), ctx_hi=hi, budget=budget,
                    sinks=rng.randint(0, min(8, budget - recent)), recent=recent)
    dtype = rng.choice(("fp16", "bf16"))
    step = rng.random() < 0.5
    if op == "store":
        S = 1 if step else _log_int(rng, 2, 48000 // (B * max(1, Hkv // 4)))
        hi = max(S, _log_int(rng, 5, 800000 // (B * Hkv) if step else 16384))
        return dict(op=op, dtype=dtype, B=B, S=S, Hkv=Hkv, ctx_lo=max(1, hi - rng.randint(0, hi - 1)), ctx_hi=hi,
                    new_lo=rng.randint(0 if S > 1 else 1, S), new_hi=S)
    G = rng.choice((1, 4, 7, 8, 12, 16))
    if op == "weights":
        S = 1 if step else _log_int(rng, 2, max(2, 120 // B))
    else:
        S = 1 if step else _log_int(rng, 2, max(2, 6000 // B))
        while S > 1 and B * S * G * Hkv > 32 * 6000:
            S = max(1, S // 2)
    hi = max(S, _log_int(rng, 5, min(24000 if S > 1 else 400000, 1200000 // (B * max(1, Hkv // 2)))))
    c = dict(op=op, dtype=dtype, B=B, S=S, Hq=Hkv * G, Hkv=Hkv, ctx_lo=max(1, hi - rng.randint(0, hi - 1)), ctx_hi=hi,
             new_lo=rng.randint(0 if S > 1 else 1, S), new_hi=S, budget=_log_int(rng, 16, 512))
    if op == "attend":
        c["lse"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------- the lengths
def _spread(lo, hi, B, mult):
    """B values over [lo, hi], the ends among them, in no sorted order; they go by the case alone."""
    while math.gcd(mult, B) != 1:
        mult += 1
    return [hi] if B == 1 else [lo + (hi - lo) * ((i * mult) % B) // (B - 1) for i in range(B)]


def _lengths(case):
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], case["B"], 5)
    if case["op"] == "evict":
        return ctx, [0] * case["B"]
    return ctx, [min(n, case["S"], L) for n, L in zip(_spread(case["new_lo"], case["new_hi"], case["B"], 3), ctx)]


def _entries(case, p):
    """Valid list entries of the row at position p."""
    nc = (p + 1) // RATIO
    return min(nc, case["budget"]) * RATIO + (p + 1 - nc * RATIO)


def _width(case):
    return case["budget"] * RATIO + RATIO - 1


def work(case):
    op = case["op"]
    if op == "rotary":
        size, T = (4 if case["dtype"] == "fp32" else 2), case["T"] - case["pad"]
        dims = case["rot"] if case["inplace"] else case["D"]
        return {"bytes": 2 * T * case["H"] * dims * size + T * 4, "flops": 3 * T * case["H"] * case["rot"]}
    B, Hkv = case["B"], case["Hkv"]
    ctx, new = _lengths(case)
    if op == "evict":
        kept = sum(min(L, case["budget"]) for L in ctx)
        moved = sum(case["budget"] for L in ctx if L > case["budget"])
        return {"bytes": Hkv * (4 * sum(ctx) + 8 * kept + 2 * 2 * moved * 76), "flops": Hkv * sum(ctx)}
    S, N = case["S"], sum(new)
    if op == "store":
        return {"bytes": N * 2 * Hkv * D * 2 + N * 2 * Hkv * ROW + B * S * 2 * Hkv * D * 2, "flops": N * 2 * Hkv * D * 4}
    Hq = case["Hq"]
    ent = sum(_entries(case, p) for L, n in zip(ctx, new) for p in range(L - n, L))
    # a cached row that several lists name is read once
    rows = sum(min(L, sum(_entries(case, p) for p in range(L - n, L))) for L, n in zip(ctx, new))
    if op == "attend":
        return {"bytes": rows * 2 * Hkv * 76 + ent * 4 + N * Hq * D * 2 + B * S * Hq * (D * 2 + (4 if case["lse"] else 0)),
                "flops": 4 * ent * Hq * D}
    return {"bytes": rows * Hkv * (76 + 8) + ent * 4 + N * Hq * (D * 2 + 4) + B * S * Hkv * _width(case) * 4,
            "flops": 2 * ent * Hq * D}


# ------------------------------------------------------------------ inputs
def _tables(ctx, g):
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


def _pool(flat, Hkv, g):
    """Rows as a quantiser leaves normal values of about unit size: codes with a normal's frequencies (16 values of a
    group reach 6 about once), scales of 1/4 to 1 of the largest, row scales of a few powers of two."""
    x = 3.0 * torch.randn((1 << 16, 2), generator=g, device="cuda")
    c = torch.bucketize(x.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")) + 8 * (x < 0)
    pairs = (c[:, 0] + 16 * c[:, 1]).to(torch.uint8)
    pool = torch.zeros((flat, PAGE, Hkv, ROW), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (PAGE * Hkv * AT_SCALE))
    for i in range(0, flat, step):
        part = pool[i:i + step]
        lead = part.shape[:3]
        part[..., :AT_SCALE] = pairs[torch.randint(0, 1 << 16, (*lead, AT_SCALE), generator=g, device="cuda", dtype=torch.int32)]
        part[..., AT_SCALE:AT_ROW] = torch.randint(0x6e, 0x7f, (*lead, 8), generator=g, device="cuda", dtype=torch.uint8)
        t = torch.exp2(torch.randint(-11, -8, (*lead, 1), generator=g, device="cuda").float())
        part[..., AT_ROW:AT_ROW + 4] = t.view(torch.uint8)
    return pool


def _lists(case, ctx_t, new_t, g):
    """Lists as the block indexer gives them: `budget` blocks of RATIO tokens, then the causal tail, ascending, -1 behind."""
    B, S, budget = case["B"], case["S"], case["budget"]
    nb = max(1, max(_lengths(case)[0]) // RATIO)
    out = torch.full((B, S, _width(case)), -1, dtype=torch.int32, device="cuda")
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


def _frequencies(case):
    """rot/2 angles per position, in 64 bits on the host: a program keeps these with its model."""
    rot, factor = case["rot"], case["factor"]
    theta = THETA * factor ** (rot / max(rot - 2, 1)) if case["scaling"] == "base" else THETA
    f = theta ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot)
    if case["scaling"] == "linear":
        f = f / factor
    elif case["scaling"] == "blend":
        low, high, length = 1.0, 4.0, 8192.0
        share = ((length * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f / factor * (1 - share) + f * share
    return f


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": case}
    op = case["op"]
    if op == "rotary":
        dt, T = DTYPES[case["dtype"]], case["T"]
        s["x"] = torch.randn((T, case["X"], case["D"]), generator=g, device="cuda").to(dt)
        s["out"] = s["x"] if case["inplace"] else torch.zeros((T, case["H"], case["D"]), dtype=dt, device="cuda")
        s["pos"] = torch.randint(case["pos_lo"], case["pos_hi"], (T,), generator=g, device="cuda", dtype=torch.int32)
        s["pos"][T - case["pad"]:] = -1
        s["freq"] = _frequencies(case)
        s["freq_gpu"] = s["freq"].cuda()
        return s
    B, Hkv = case["B"], case["Hkv"]
    ctx, new = _lengths(case)
    s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    s["new"] = torch.tensor(new, dtype=torch.int32, device="cuda")
    s["pt"], flat = _tables(ctx, g)
    s["pool"] = _pool(flat, Hkv, g)
    if op == "evict":
        # most tokens gather little, a few a lot, some nothing at all
        T = max(ctx)
        w = torch.exp(2.0 * torch.randn((B, Hkv, T), generator=g, device="cuda") - 4.0)
        s["total"] = torch.where(torch.rand((B, Hkv, T), generator=g, device="cuda") < 0.1, torch.zeros_like(w), w)
        s["total_out"] = torch.empty_like(s["total"])
        s["kept"] = torch.empty((B, Hkv, case["budget"]), dtype=torch.int32, device="cuda")
        s["length"] = torch.empty((B,), dtype=torch.int32, device="cuda")
        return s
    S, dt = case["S"], DTYPES[case["dtype"]]
    # the live rows and their positions: a program that keeps the lengths has these
    b = torch.repeat_interleave(torch.arange(B, device="cuda"), s["new"].long(), output_size=sum(new))
    t = torch.arange(sum(new), device="cuda") - (torch.cumsum(s["new"].long(), 0) - s["new"].long())[b]
    s["rows"] = b * S + t
    if op == "store":
        pos = (s["ctx"].long() - s["new"].long())[b] + t
        pt = s["pt"].long()
        s["slot"] = torch.stack([pt[b, i, pos // PAGE] * PAGE + pos % PAGE for i in (0, 1)])
        # normed keys with a few channels that carry more; k and v lie side by side in the packed projections
        s["kv"] = torch.randn((B, S, 2 * Hkv, D), generator=g, device="cuda")
        s["kv"][:, :, :Hkv, ::29] *= 6.0
        s["kv"] = s["kv"].to(dt)
        s["k_out"], s["v_out"] = (torch.empty((B, S, Hkv, D), dtype=dt, device="cuda") for _ in range(2))
        return s
    s["q"] = torch.randn((B, S, case["Hq"], D), generator=g, device="cuda").to(dt)
    s["lists"] = _lists(case, s["ctx"].long(), s["new"].long(), g)
    s["lse"] = torch.empty((B, S, case["Hq"]), device="cuda")
    if op == "attend":
        s["out"] = torch.empty((B, S, case["Hq"], D), dtype=dt, device="cuda")
        return s
    # the step's attention has left its log-sum-exp
    for r, logit, _ in _logits(s):
        s["lse"].view(B * S, Hkv, -1)[r] = torch.logsumexp(logit.double(), -1).float()
    s["weights"] = torch.empty((B, S, Hkv, _width(case)), device="cuda")
    s["total"] = 0.1 * torch.rand((B, Hkv, max(ctx)), generator=g, device="cuda")
    return s


# -------------------------------------------------------------- plain forms
def _rotary(s):
    case = s["case"]
    H, rot, h = case["H"], case["rot"], case["rot"] // 2
    pos = s["pos"]
    angle = pos.double()[:, None] * s["freq_gpu"]
    c = (angle.cos() * case["magnitude"]).float()[:, None]
    sn = (angle.sin() * (-case["magnitude"] if case["inverse"] else case["magnitude"])).float()[:, None]
    x = s["x"][:, :H].float()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, h), slice(h, rot))
    y = x.clone()
    y[..., first] = x[..., first] * c - x[..., second] * sn
    y[..., second] = x[..., second] * c + x[..., first] * sn
    out = s["out"][:, :H]
    out.copy_(torch.where((pos >= 0)[:, None, None], y.to(out.dtype), out))
    return s["out"]


def _quantised(x):
    """x [..., 128] as rows of bytes [..., 80] and as the values they stand for, in 32 bits.  (Quotients in 64 bits: a value
    may lie next to a border.)"""
    x = x.double()
    groups = x.unflatten(-1, (8, 16))
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax / 2688.0)
    t = torch.ldexp(torch.ones_like(amax), torch.where(m == 0.5, e - 1, e).clamp(-48, 48))
    t = torch.where(amax == 0, torch.full_like(t, 2.0 ** -48), t).float().double()  # (a power function's is off by 2^-53)
    want = groups.abs().amax(-1) / (6.0 * t)[..., None]
    scale = want.clamp(max=448.0).float().to(torch.float8_e4m3fn)
    unit = scale.double() * t[..., None]
    q = (groups.abs() / unit[..., None]).flatten(-2)
    code = ((q > 0.25).to(torch.uint8) + (q >= 0.75) + (q > 1.25) + (q >= 1.75) + (q > 2.5) + (q >= 3.5) + (q > 5.0))
    code = code * (unit > 0).repeat_interleave(16, -1) + 8 * torch.signbit(x)
    row = torch.zeros((*x.shape[:-1], ROW), dtype=torch.uint8, device=x.device)
    row[..., :AT_SCALE] = code[..., 0::2] + 16 * code[..., 1::2]
    row[..., AT_SCALE:AT_ROW] = scale.view(torch.uint8)
    row[..., AT_ROW:AT_ROW + 4] = t.float()[..., None].view(torch.uint8)
    return row, _values(row)


def _values(row):
    """The values [..., 128] that rows of bytes [..., >= 80] stand for, in 32 bits."""
    codes = torch.tensor(E2M1 + [-v for v in E2M1], device=row.device)
    b = row[..., :AT_SCALE].to(torch.int32)
    v = codes[torch.stack([b & 15, b >> 4], -1).flatten(-2)]
    scale = row[..., AT_SCALE:AT_ROW].contiguous().view(torch.float8_e4m3fn).float()
    t = row[..., AT_ROW:AT_ROW + 4].contiguous().view(torch.float32).clamp(2.0 ** -48, 2.0 ** 48)
    return (v.unflatten(-1, (8, 16)) * (scale * t)[..., None]).flatten(-2)


def _store(s):
    case = s["case"]
    Hkv = case["Hkv"]
    x = s["kv"].flatten(0, 1)[s["rows"]]
    row, value = _quantised(x)
    pool = s["pool"].view(-1, Hkv, ROW)
    pool[s["slot"][0]] = row[:, :Hkv]
    pool[s["slot"][1]] = row[:, Hkv:]
    for out, v in ((s["k_out"], value[:, :Hkv]), (s["v_out"], value[:, Hkv:])):
        out.zero_()
        out.view(-1, Hkv, D)[s["rows"]] = v.to(out.dtype)
    return {"k": s["k_out"], "v": s["v_out"], "pool": s["pool"]}


def _named(s, r):
    """The tokens that the list rows r (of all B S) name, 0 for entries that name none, and which do."""
    case = s["case"]
    S = case["S"]
    b = r // S
    j = s["lists"].view(case["B"] * S, -1)[r].long()
    valid = (j >= 0) & (j < s["ctx"][b][:, None]) & (r % S < s["new"][b])[:, None]
    return b, torch.where(valid, j, torch.zeros_like(j)), valid


def _cached(s, b, j, valid, plane):
    """Values [rows, Hkv, topk, D] of the tokens j of sequences b, in 32 bits; zeros where not valid."""
    at = s["pt"][b[:, None], plane, j // PAGE].long() * PAGE + j % PAGE
    x = _values(s["pool"].view(-1, s["case"]["Hkv"], ROW)[at])
    return torch.where(valid[..., None, None], x, torch.zeros_like(x)).transpose(1, 2)


def _logits(s):
    """Rows of the call, a part at a time, with their logits [rows, Hkv, G, topk] in 32 bits (-inf: names nothing) and tokens."""
    case = s["case"]
    B, S, Hq, Hkv = (case[k] for k in ("B", "S", "Hq", "Hkv"))
    q = s["q"].view(B * S, Hkv, Hq // Hkv, D)
    step = max(1, (1 << 28) // (_width(case) * Hkv * D))
    for r0 in range(0, B * S, step):
        r = torch.arange(r0, min(B * S, r0 + step), device=q.device)
        b, j, valid = _named(s, r)
        logit = torch.matmul(q[r].float(), _cached(s, b, j, valid, 0).transpose(2, 3)) / math.sqrt(D)
        yield r, logit.masked_fill(~valid[:, None, None, :], -math.inf), (b, j, valid)


def _attend(s):
    case = s["case"]
    B, S, Hq, Hkv = (case[k] for k in ("B", "S", "Hq", "Hkv"))
    out, lse = s["out"].view(B * S, Hkv, Hq // Hkv, D), s["lse"].view(B * S, Hkv, Hq // Hkv)
    for r, logit, (b, j, valid) in _logits(s):
        top = logit.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        p = torch.exp(logit - top)
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p, _cached(s, b, j, valid, 1)) / torch.where(total == 0, torch.ones_like(total), total)
        out[r] = o.to(out.dtype)
        lse[r] = (top + torch.log(total))[..., 0]
    return {"out": s["out"], "lse": s["lse"]} if case["lse"] else {"out": s["out"]}


def _weights(s):
    case = s["case"]
    B, S, Hkv = (case[k] for k in ("B", "S", "Hkv"))
    T = s["total"].shape[-1]
    lse, weights = s["lse"].view(B * S, Hkv, -1), s["weights"].view(B * S, Hkv, -1)
    add = torch.zeros((B * Hkv * T,), dtype=torch.float64, device=lse.device)  # (64 bits: no order of additions shows)
    for r, logit, (b, j, valid) in _logits(s):
        w = torch.exp(logit - lse[r][..., None]).masked_fill(~valid[:, None, None, :], 0.0).sum(2)
        weights[r] = w
        at = (b[:, None] * Hkv + torch.arange(Hkv, device=w.device))[..., None] * T + j[:, None, :]
        add.index_add_(0, at.flatten(), w.double().flatten())
    s["total"] += add.view_as(s["total"]).float()
    return {"weights": s["weights"], "total": s["total"]}


def _evict(s):
    case = s["case"]
    B, Hkv, budget = (case[k] for k in ("B", "Hkv", "budget"))
    total, L = s["total"], s["ctx"].long()[:, None, None]
    T = total.shape[-1]
    j = torch.arange(T, device=total.device)
    key = torch.where((j < case["sinks"]) | (j >= L - case["recent"]), torch.full_like(total, math.inf), total)
    key = torch.where(j < L, key, torch.full_like(key, -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :budget]
    order = torch.nn.functional.pad(order, (0, budget - order.shape[-1]))
    keep = torch.clamp(L, max=budget)
    i = torch.arange(budget, device=total.device)
    src = torch.sort(torch.where(i < keep, order, torch.full_like(order, T)), dim=-1).values  # ascending, T behind the last
    s["kept"].copy_(torch.where(i < keep, src, torch.full_like(src, -1)))
    s["length"].copy_(keep.flatten())
    s["total_out"].zero_()
    m = min(budget, T)
    picked = torch.gather(total, 2, src[..., :m].clamp(max=T - 1))
    s["total_out"][..., :m] = torch.where(i[:m] < keep, picked, torch.zeros_like(picked))
    b, h, at = ((i < keep) & (src != i)).nonzero(as_tuple=True)  # the rows that move
    old = src[b, h, at]
    pool, pt = s["pool"].view(-1, Hkv, ROW), s["pt"].long()
    to = torch.stack([pt[b, p, at // PAGE] * PAGE + at % PAGE for p in (0, 1)])
    row = pool[torch.stack([pt[b, p, old // PAGE] * PAGE + old % PAGE for p in (0, 1)]), h]
    pool[to, h] = row
    return {"kept": s["kept"], "length": s["length"], "total": s["total_out"], "pool": s["pool"]}


PLAIN = {"rotary": _rotary, "store": _store, "attend": _attend, "weights": _weights, "evict": _evict}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return PLAIN[op](s)
    from block_sparse_gqa_qsa_gb300 import _binding as qb
    if op == "rotary":
        qb.rotary(s["x"][:, :case["H"]], s["pos"], s["out"][:, :case["H"]], s["freq"], interleaved=case["interleaved"],
                  inverse=case["inverse"], magnitude=case["magnitude"])
        return s["out"]
    if op == "store":
        Hkv = case["Hkv"]
        qb.store_kv4(s["kv"][:, :, :Hkv], s["kv"][:, :, Hkv:], s["ctx"], s["pool"], s["pt"], new_lengths=s["new"],
                     k_out=s["k_out"], v_out=s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"], "pool": s["pool"]}
    if op == "evict":
        qb.evict_kv4(s["pool"], s["pt"], s["ctx"], s["total"], s["kept"], s["length"], s["total_out"],
                     sinks=case["sinks"], recent=case["recent"])
        return {"kept": s["kept"], "length": s["length"], "total": s["total_out"], "pool": s["pool"]}
    scale = 1.0 / math.sqrt(D)
    if op == "attend":
        lse = s["lse"] if case["lse"] else None
        qb.sparse_paged_kv4(s["q"], s["pool"], s["pt"], s["lists"], s["ctx"], s["out"], scale=scale, new_lengths=s["new"],
                            lse=lse)
        return {"out": s["out"], "lse": s["lse"]} if case["lse"] else {"out": s["out"]}
    qb.sparse_weights_kv4(s["q"], s["pool"], s["pt"], s["lists"], s["ctx"], s["lse"], s["weights"], s["total"], scale=scale,
                          new_lengths=s["new"])
    return {"weights": s["weights"], "total": s["total"]}


# ------------------------------------------------------- 64-bit definitions
def _nearest(x, grid):
    """x >= 0 to the nearest of an ascending 64-bit grid whose entries' codes count up from 0: ties to the even code."""
    i = torch.searchsorted(grid, x.contiguous()).clamp(1, grid.numel() - 1)
    below, above = x - grid[i - 1], grid[i] - x
    up = (above < below) | ((above == below) & (i % 2 == 0))
    return torch.where(up, grid[i], grid[i - 1])


def _exact_rows(x):
    """The values that rows x [..., 128] are held as, in 64 bits."""
    x = x.double().unflatten(-1, (8, 16))
    amax = x.abs().amax((-1, -2), keepdim=True)
    k = torch.ceil(torch.log2((amax / 2688.0).clamp(min=1e-300)) - 1e-14).clamp(-48, 48)
    t = torch.exp2(k).float().double()
    e4m3 = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    e2m1 = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    scale = _nearest(x.abs().amax(-1, keepdim=True) / 6.0 / t, e4m3)
    unit = torch.where(scale > 0, scale * t, torch.full_like(scale, math.inf))
    return (_nearest(x.abs() / unit, e2m1) * torch.sign(x) * scale * t).flatten(-2)


def _exact_cache(s, b, h, plane, L):
    """The first L tokens of a sequence and head, [L, D] in 64 bits."""
    pages = s["pt"][b, plane, :-(-L // PAGE)].long()
    row = s["pool"][pages, :, h].reshape(-1, ROW)[:L]
    b4 = row[:, :AT_SCALE].long()
    sign = torch.tensor([1.0, -1.0], dtype=torch.float64, device=row.device)
    mag = torch.tensor(E2M1, dtype=torch.float64, device=row.device)
    x = torch.empty((L, D), dtype=torch.float64, device=row.device)
    x[:, 0::2] = mag[b4 % 8] * sign[b4 // 8 % 2]
    x[:, 1::2] = mag[b4 // 16 % 8] * sign[b4 // 128]
    e4m3 = torch.arange(256, dtype=torch.int32, device=row.device).to(torch.uint8).view(torch.float8_e4m3fn).double()
    x *= e4m3[row[:, AT_SCALE:AT_ROW].long()].repeat_interleave(16, 1)
    return x * row[:, AT_ROW:AT_ROW + 4].contiguous().view(torch.float32).double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        H, rot = case["H"], case["rot"]
        y = s["out"].double()
        x = s["x"][:, :H].double()
        pairs = x[..., :rot].unflatten(-1, (rot // 2, 2)) if case["interleaved"] else \
            x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        turn = (-1j if case["inverse"] else 1j) * s["pos"].double()[:, None] * s["freq_gpu"]
        z = torch.view_as_complex(pairs.contiguous()) * (case["magnitude"] * torch.exp(turn))[:, None]
        z = torch.view_as_real(z)
        x[..., :rot] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        live = s["pos"] >= 0
        y[:, :H][live] = x[live]
        return y
    ctx, new = _lengths(case)
    if op == "evict":  # (the other outputs are whole numbers)
        total, moved = s["total"].double().cpu().numpy(), torch.zeros_like(s["total"], dtype=torch.float64)
        for b, L in enumerate(ctx):
            first, last = (L, L) if L <= case["budget"] else (case["sinks"], L - case["recent"])
            for h in range(case["Hkv"]):
                middle = np.arange(first, last)
                best = middle[np.lexsort((middle, -total[b, h, first:last]))][:case["budget"] - (first + L - last)]
                kept = np.concatenate([np.arange(first), np.sort(best), np.arange(last, L)])
                moved[b, h, :len(kept)] = torch.from_numpy(total[b, h, kept]).cuda()
        return {"kept": None, "length": None, "total": moved, "pool": None}
    B, S, Hkv = (case[k] for k in ("B", "S", "Hkv"))
    if op == "store":
        value = _exact_rows(s["kv"])
        for b, n in enumerate(new):
            value[b, n:] = 0.0
        return {"k": value[:, :, :Hkv], "v": value[:, :, Hkv:], "pool": None}
    Hq = case["Hq"]
    G = Hq // Hkv
    out = torch.zeros((B, S, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, S, Hq), -math.inf, dtype=torch.float64, device="cuda")
    weights = torch.zeros((B, S, Hkv, _width(case)), dtype=torch.float64, device="cuda") if op == "weights" else None
    total = s["total"].double() if op == "weights" else None
    for b in range(B):
        n, L = new[b], ctx[b]
        step = max(1, (1 << 26) // (L * G))
        for h in range(Hkv):
            hs = slice(h * G, (h + 1) * G)
            k = _exact_cache(s, b, h, 0, L)
            v = _exact_cache(s, b, h, 1, L) if op == "attend" else None
            for t0 in range(0, n, step):
                ts = slice(t0, min(n, t0 + step))
                idx = s["lists"][b, ts].long()
                ok = (idx >= 0) & (idx < L)
                at = idx.clamp(0, L - 1)
                z = s["q"][b, ts, hs].double() @ k.T / math.sqrt(D)  # [t, G, L]
                if op == "weights":
                    p = torch.exp(z - s["lse"][b, ts, hs].double()[..., None]).sum(1)
                    w = torch.where(ok, torch.gather(p, 1, at), torch.zeros((), dtype=torch.float64, device="cuda"))
                    weights[b, ts, h] = w
                    total[b, h].scatter_add_(0, at.flatten(), w.flatten())
                    continue
                count = torch.zeros((idx.shape[0], L), dtype=torch.float64, device="cuda")
                count.scatter_add_(1, at, ok.double())
                z = z + torch.log(count)[:, None]
                lse[b, ts, hs] = torch.logsumexp(z, -1)
                out[b, ts, hs] = torch.softmax(z, -1) @ v
    if op == "weights":
        return {"weights": weights, "total": total}
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
