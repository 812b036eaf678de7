"""perf/operators.py: its plain forms and the library's calls against its 64-bit definitions, on listed and drawn cases.

Bars.  q of an append and the values of a 16-bit pool: one step of the type plus 2^-18, as in test_gpu_append; a scale:
2^-18 / 448 plus 2^-22 of it, and a block that grew may have grown by one power of two less or more where its largest
value meets 448 scales within that; a code: one e4m3 step (2^-3 of the value, 2^-9 at least) where its scale is the
64-bit form's, half a step for each of two roundings.  Attention: `paged_cache_ref.attend_bar`, with the weighted mean of
|v| from the 64-bit form over the codes' magnitudes, and 2^5 for the terms of a logit (unit normals: 7 on average, K
scales up to 4 times theirs)."""
from __future__ import annotations

import importlib.util
import os
import random

import pytest
import torch

import paged_cache_ref as ref
from conftest import ROOT

pytestmark = pytest.mark.gpu
EVAL = 2.0 ** -18


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_gqa_qsa_gb300 import _binding, build
    build.build()
    _binding.lib()
    spec = importlib.util.spec_from_file_location("operator_cases", os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def step_of(x, dtype):
    bits, low = (11, -24) if dtype == torch.float16 else (8, -133)
    _, e = torch.frexp(x.abs())
    return torch.ldexp(torch.ones_like(x), (e - bits).clamp(min=low))


def mean_magnitude(ops, case, seed):
    """Probability-weighted mean of |v| of every output, in 64 bits."""
    s = ops.prepare(case, seed)
    codes = s["pool"].view(torch.uint8)
    codes[codes.shape[0] // 2:] &= 0x7f  # V pages are the second half
    return ops._exact_attend(s, *ops._lengths(case))


def check_attend(case, out, want, mean_abs):
    bar = ref.attend_bar(want, mean_abs, torch.full(want.shape[:-1], 2.0 ** 5, dtype=torch.float64, device=want.device),
                         torch.empty(4 * case["budget"] + 3), torch.tensor(2.0 ** -5), out.dtype)
    err = (out.double() - want).abs()
    assert bool((err <= bar).all()), float((err / bar).max())


def check_append(case, out, want):
    dt = out["q"].dtype
    assert bool(((out["q"].double() - want["q"]).abs() <= step_of(want["q"], dt) + EVAL).all())
    pool = out["pool"].double()
    if case["op"] == "append16":
        assert bool(((pool - want["pool"]).abs() <= step_of(want["pool"], dt) + EVAL).all())
        return
    got, s = out["scale"].double(), want["scale"]
    same = (got - s).abs() <= EVAL / 448 + 2.0 ** -22 * s
    grown = ~same & (((got / 2 - s).abs() <= 2.0 ** -20 * s) | ((got * 2 - s).abs() <= 2.0 ** -20 * s))
    assert bool((same | grown).all()) and int(grown.sum()) <= 2
    ok = same.repeat_interleave(ref.PAGE // s.shape[1], 1)[..., None]
    floor = torch.full((), 2.0 ** -9, dtype=torch.float64, device=s.device)
    # (the 64-bit form multiplies by a step from a power function: its codes are off by a rounding or two, 2^-52)
    bar = (1 + 2.0 ** -48) * torch.maximum(2.0 ** -3 * want["pool"].abs(), floor)
    assert bool((((pool - want["pool"]).abs() <= bar) | ~ok).all())




def both_forms(ops, case, seed):
    want = ops.exact(case, seed)
    mean_abs = mean_magnitude(ops, case, seed) if case["op"] == "attend8" else None
    for own in (False, True):
        ops.own = own
        try:
            out = ops.run(ops.prepare(case, seed))
            torch.cuda.synchronize()
        finally:
            ops.own = False
        if case["op"] == "attend8":
            check_attend(case, out, want, mean_abs)
        else:
            check_append(case, out, want)


@pytest.mark.parametrize("name", [
    "append16_step_B32", "append16_chunk_B3_S517", "append8_step_B1", "append8_step_B32", "append8_chunk_B4_S1000",
    "append8_prefill_B4_S16384", "attend8_step_B1_L512", "attend8_step_B32", "attend8_step_B8_L512k",
    "attend8_verify_B6_S5", "attend8_chunk_B2_S700"])
def test_listed_case(ops, name):
    """(A whole prompt's attention has its own tests: its plain form takes a quarter of a second, its 64-bit one far more.)"""
    both_forms(ops, next(c for c in ops.listed() if c["name"] == name), 11)


@pytest.mark.parametrize("seed", range(6))
def test_drawn_case(ops, seed):
    """Drawn cases, cut to what the 64-bit form does quickly."""
    rng = random.Random(seed)
    case = ops.draw(rng)
    while case["B"] * case["S"] * case["Hq"] * case["ctx_hi"] > 1 << 31:
        case = ops.draw(rng)
    both_forms(ops, case, seed)


def test_work_is_counted_from_the_lengths(ops):
    """bytes and flops of the listed cases: positive, and of the largest at least 16 times the smallest's."""
    work = [ops.work(c) for c in ops.listed()]
    assert all(w["bytes"] > 0 and w["flops"] > 0 for w in work)
    assert max(w["bytes"] for w in work) >= 16 * min(w["bytes"] for w in work)
