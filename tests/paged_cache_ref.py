"""Plain 64-bit forms of the paged-cache operators, and the caches their tests use."""
from __future__ import annotations

import math

import torch

PAGE = 128
THETA, EPS = 1.0e4, 1.0e-6
E4M3 = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double()


def page_tables(ctx, seed, extra=0):
    """(page_table int32 [B, 2, P], flat pages): shuffled K pages, V page = K page + n, `extra` spare pages per plane."""
    g = torch.Generator().manual_seed(seed)
    pages = [max(1, -(-int(L) // PAGE)) for L in ctx]
    n = sum(pages) + extra
    perm = torch.randperm(n, generator=g).to(torch.int32)
    pt = torch.zeros((len(pages), 2, max(pages)), dtype=torch.int32)
    at = 0
    for b, m in enumerate(pages):
        pt[b, 0, :m] = perm[at:at + m]
        pt[b, 1, :m] = perm[at:at + m] + n
        at += m
    return pt, 2 * n


def random_codes(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return (128.0 * torch.randn(shape, generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn)


def new_rows(ctx, new, S):
    """Rows per sequence as the operators count them."""
    return [max(0, min(S if new is None else int(new[b]), S, max(int(L), 0))) for b, L in enumerate(ctx)]


def normed_rotated(x, w, pos, rot):
    """x [N, H, D] float64, pos [N]: RMSNorm * (1 + w), then the half-split rotation."""
    x, w = x.double(), w.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * (1 + w)
    h = rot // 2
    ang = pos.double()[:, None, None] * THETA ** (-2.0 * torch.arange(h, dtype=torch.float64) / max(rot, 1))
    c, s = torch.cos(ang), torch.sin(ang)
    out = y.clone()
    out[..., :h] = y[..., :h] * c - y[..., h:rot] * s
    out[..., h:rot] = y[..., h:rot] * c + y[..., :h] * s
    return out


def attend(q, keys, values, lists, scale):
    """One sequence: q [n, Hq, D], keys / values [L, Hkv, D] (float64), lists [n, topK].  Returns the output, the
    probability-weighted mean of |v|, and the largest logit magnitude sum, all float64 [n, Hq, ...]."""
    n, Hq, D = q.shape
    L, Hkv, _ = keys.shape
    G = Hq // Hkv
    out = torch.zeros((n, Hq, D), dtype=torch.float64)
    mean_abs = torch.zeros_like(out)
    dots = torch.zeros((n, Hq), dtype=torch.float64)
    for t in range(n):
        j = lists[t].long()
        j = j[(j >= 0) & (j < L)]
        if j.numel() == 0:
            continue
        for h in range(Hkv):
            qq = q[t, h * G:(h + 1) * G].double()
            p = torch.softmax(scale * qq @ keys[j, h].T, -1)
            out[t, h * G:(h + 1) * G] = p @ values[j, h]
            mean_abs[t, h * G:(h + 1) * G] = p @ values[j, h].abs()
            dots[t, h * G:(h + 1) * G] = abs(scale) * (qq.abs() @ keys[j, h].abs().T).amax(-1)
    return out, mean_abs, dots


def attend_bar(out, mean_abs, dots, values, scales, dtype, D=128):
    """How far an output may be from the 64-bit one: probabilities rounded to fp16 (half a step, 2^-11 of each, and
    2^-25 of the largest probability times V scale below fp16's normal range), logits off by the fp32 sums (2^-23 per
    term: a tensor-core sum drops bits below its largest term) and their effect on every weight, and the output's own
    half step."""
    logit = D * 2.0 ** -23 * dots[..., None]
    n = values.shape[0]
    sub = n * 2.0 ** -25 * 448 * float(scales.max())  # every entry's fp16 underflow, against the largest V scale
    return (2.0 ** -11 + 2.0 ** -18 + 2 * logit) * mean_abs + sub + torch.finfo(dtype).eps / 2 * out.abs() + 1e-7


def dequantised(pool, scale, pt_row, L, D=128):
    """[L, Hkv, D] float64 of one plane's pages of a sequence."""
    pages = pt_row[:-(-L // PAGE)].long()
    x = E4M3[pool.view(torch.uint8)[pages][..., :D].long()]
    s = scale[pages].double().repeat_interleave(PAGE // scale.shape[1], 1)
    return (x * s[..., None]).flatten(0, 1)[:L]
