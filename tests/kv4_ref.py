"""Plain 64-bit forms of the 4-bit cache's operators, and the caches their tests use."""
from __future__ import annotations

import math

import torch

from paged_cache_ref import PAGE, new_rows, page_tables  # noqa: F401  (the tests take them from here)

ROW, D = 80, 128
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E4M3 = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double()


def nearest_code(x, grid):
    """Codes of x >= 0 on an ascending grid whose codes count up from 0: the nearest, ties to the even code, saturating."""
    i = torch.searchsorted(grid, x.contiguous()).clamp(1, grid.numel() - 1)
    below, above = x - grid[i - 1], grid[i] - x
    up = (above < below) | ((above == below) & (i % 2 == 0))
    return torch.where(up, i, i - 1)


def rows_of(x):
    """Bytes [..., 80] of values x [..., 128]."""
    x = x.double().cpu()
    finite = torch.isfinite(x)
    mag = torch.where(finite, x.abs(), torch.zeros_like(x))
    k = torch.full(x.shape[:-1], -48, dtype=torch.int64)
    for e in range(-48, 48):  # the smallest power of two that reaches amax / 2688
        k = torch.where(mag.amax(-1) > 2688.0 * 2.0 ** e, e + 1, k)
    t = torch.tensor([2.0 ** e for e in range(-48, 49)], dtype=torch.float64)[k + 48]
    g = mag.unflatten(-1, (8, 16))
    sc = nearest_code(g.amax(-1) / (6.0 * t[..., None]), E4M3[:127])
    ok = finite.unflatten(-1, (8, 16)).all(-1)
    s = E4M3[sc]
    unit = torch.where(s > 0, s * t[..., None], torch.full_like(s, math.inf))
    code = nearest_code(g / unit[..., None], E2M1) + 8 * torch.signbit(x).unflatten(-1, (8, 16))
    code = torch.where(ok[..., None], code, torch.zeros_like(code)).flatten(-2).to(torch.uint8)
    row = torch.zeros((*x.shape[:-1], ROW), dtype=torch.uint8)
    row[..., :64] = code[..., 0::2] | (code[..., 1::2] << 4)
    row[..., 64:72] = torch.where(ok, sc, torch.full_like(sc, 0x7f)).to(torch.uint8)
    row[..., 72:76] = t.float().unsqueeze(-1).contiguous().view(torch.uint8)
    return row


def values_of(row):
    """float64 [..., 128] of bytes [..., >= 80]."""
    row = row.cpu()
    b = row[..., :64].long()
    code = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    v = E2M1[code & 7] * torch.where(code >= 8, -1.0, 1.0)
    t = row[..., 72:76].contiguous().view(torch.float32).double()
    t = torch.where(torch.isnan(t), torch.full_like(t, 2.0 ** -48), t.clamp(2.0 ** -48, 2.0 ** 48))
    return v * E4M3[row[..., 64:72].long()].repeat_interleave(16, -1) * t


def random_pool(flat, Hkv, seed, row=ROW, spread=2):
    """uint8 [flat, 128, Hkv, row]: random codes, scales of 1/16 to 1 of the largest, row scales around 2^-10; junk behind."""
    g = torch.Generator().manual_seed(seed)
    pool = torch.randint(0, 256, (flat, PAGE, Hkv, row), generator=g, dtype=torch.int32).to(torch.uint8)
    pool[..., 64:72] = torch.randint(0x60, 0x7f, (flat, PAGE, Hkv, 8), generator=g, dtype=torch.int32).to(torch.uint8)
    t = torch.exp2(torch.randint(-10 - spread, -9, (flat, PAGE, Hkv, 1), generator=g).float())
    pool[..., 72:76] = t.view(torch.uint8)
    pool[..., 76:80] = 0
    return pool


def cached(pool, pt_row, L):
    """[L, Hkv, 128] float64 of one plane's pages of a sequence."""
    pages = pt_row[:-(-L // PAGE)].long().cpu()
    return values_of(pool.cpu()[pages][..., :ROW]).flatten(0, 1)[:L]


def lists_of(ctx, new, S, topk, seed, keep=None, bad=False):
    """int32 [B, S, topk]: up to `keep` random distinct tokens of the causal ones per row, in random order and places, -1
    elsewhere; bad: entries outside [0, L) among them."""
    g = torch.Generator().manual_seed(seed)
    out = torch.full((len(ctx), S, topk), -1, dtype=torch.int32)
    for b, (L, n) in enumerate(zip(ctx, new)):
        for t in range(n):
            p = L - n + t
            m = min(p + 1, topk if keep is None else keep)
            tok = torch.randperm(p + 1, generator=g)[:m].to(torch.int32)
            at = torch.randperm(topk, generator=g)[:m]
            out[b, t, at] = tok
            if bad and topk > m:
                free = (out[b, t] == -1).nonzero().flatten()
                out[b, t, free[0]] = L + 5
                out[b, t, free[-1]] = -7
    return out


def attend(q, keys, values, lists, scale):
    """One sequence, everything float64: o, log-sum-exp, weights [n, Hkv, topk], mean of |v|, largest sum of |q k| terms."""
    n, Hq, _ = q.shape
    L, Hkv, _ = keys.shape
    G, topk = Hq // Hkv, lists.shape[1]
    o, mean = torch.zeros((2, n, Hq, D), dtype=torch.float64)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64)
    w = torch.zeros((n, Hkv, topk), dtype=torch.float64)
    dots = torch.zeros((n, Hq), dtype=torch.float64)
    for t in range(n):
        at = ((lists[t] >= 0) & (lists[t] < L)).nonzero().flatten()
        if at.numel() == 0:
            continue
        j = lists[t, at].long()
        for h in range(Hkv):
            hs = slice(h * G, (h + 1) * G)
            z = scale * q[t, hs].double() @ keys[j, h].T
            lse[t, hs] = torch.logsumexp(z, -1)
            p = torch.softmax(z, -1)
            w[t, h, at] = p.sum(0)
            o[t, hs], mean[t, hs] = p @ values[j, h], p @ values[j, h].abs()
            dots[t, hs] = abs(scale) * (q[t, hs].double().abs() @ keys[j, h].abs().T).amax(-1)
    return o, lse, w, mean, dots


def evict(total, L, budget, sinks, recent):
    """Tokens kept of one (sequence, head), ascending."""
    if L <= budget:
        return list(range(L))
    key = [0.0 if x == 0 else x for x in total[:L].tolist()]
    middle = [j for j in range(sinks, L - recent)]
    middle.sort(key=lambda j: (-(key[j] if key[j] == key[j] else -math.inf), key[j] != key[j], j))
    best = sorted(middle[:budget - sinks - recent])
    return list(range(sinks)) + best + list(range(L - recent, L))
