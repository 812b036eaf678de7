"""perf/more_operators.py: its plain forms and the library's calls against its 64-bit definitions, on listed and drawn cases.

Bars.  rotary: as in test_gpu_rotary, with 64-bit angles of positions up to 2^20 (2^-30) for the plain form.  store, evict:
every byte and value equal.  attend: as in test_gpu_kv4, with 2^5 for the terms of a logit (unit normals), for an output the
mean of |v| bounded by the 64-bit form's over all |v|, at most 2^3 here.  weights: relative 2^-12 (2^-23 D 2^5 and the
exponent's units), totals by the fp32 additions of at most 40 rows, 2^-18 of them."""
from __future__ import annotations

import importlib.util
import os
import random

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_gqa_qsa_gb300 import _binding, build
    build.build()
    _binding.lib()
    spec = importlib.util.spec_from_file_location("more_operator_cases", os.path.join(ROOT, "perf", "more_operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def within(got, want, rel, floor):
    got = got.double()
    same = (got == want) | (torch.isinf(got) & torch.isinf(want) & (got.sign() == want.sign()))
    err = torch.where(same, torch.zeros_like(want), (got - want).abs())
    bar = rel * want.abs().nan_to_num(posinf=0) + floor
    assert bool((err <= bar).all()), float((err - bar).max())


def check(case, out, want):
    op = case["op"]
    if op == "rotary":
        eps = torch.finfo(out.dtype).eps / 2
        # |x_a| + |x_b| of normal inputs stays below 2^4; fp16's smallest half step is 2^-25
        within(out, want, eps * (1 + 2.0 ** -9), 2.0 ** -17 * case["magnitude"] + 2.0 ** -25)
    elif op == "store":
        within(out["k"], want["k"], 0.0, 0.0)
        within(out["v"], want["v"], 0.0, 0.0)
    elif op == "evict":
        within(out["total"], want["total"], 0.0, 0.0)
    elif op == "attend":
        o = out["out"]
        # probabilities to 11 bits, 2^-25 of the largest weight times scale an entry, logits' sums; |v| below 2^4
        width = 4 * case["budget"] + 3
        floor = (2.0 ** -11 + 2.0 ** -18 + 2.0 ** -16 * 2.0 ** 5) * 2.0 ** 3 + width * 2.0 ** -25 * 2688 * 2.0 ** -9
        within(o, want["out"], torch.finfo(o.dtype).eps / 2, floor)
        if case["lse"]:
            within(out["lse"], want["lse"], 2.0 ** -21, 2.0 ** -11)
    else:
        within(out["weights"], want["weights"], 2.0 ** -11, 1e-30)
        within(out["total"], want["total"], 2.0 ** -11, 1e-30)


def both_forms(ops, case, seed):
    want = ops.exact(case, seed)
    got = []
    for own in (False, True):
        ops.own = own
        try:
            got.append(ops.run(ops.prepare(case, seed)))
            torch.cuda.synchronize()
        finally:
            ops.own = False
        check(case, got[-1], want)
    if isinstance(got[0], dict):  # whole numbers and bytes are the same in both
        for name, x in got[0].items():
            if not x.is_floating_point():
                assert torch.equal(x, got[1][name]), name


@pytest.mark.parametrize("name", [
    "rotary_step_B32", "rotary_prompt_T16384", "rotary_grad_T5003", "store4_step_B32", "store4_prompt_B4_S16384",
    "attend4_step_B1_L512", "attend4_step_B32", "weights4_step_B32", "weights4_window_B3_S37", "evict4_B32_to_4096",
    "evict4_B2_L131072"])
def test_listed_case(ops, name):
    """(A whole prompt's attention has its own tests: its plain form takes half a second, its 64-bit one far more.)"""
    both_forms(ops, next(c for c in ops.listed() if c["name"] == name), 11)


@pytest.mark.parametrize("seed", range(12))
def test_drawn_case(ops, seed):
    """Drawn cases, cut to what the 64-bit form does quickly."""
    rng = random.Random(seed)
    case = ops.draw(rng)
    while case["op"] in ("attend", "weights") and case["B"] * case["S"] * case["Hq"] * case["ctx_hi"] > 1 << 31:
        case = ops.draw(rng)
    both_forms(ops, case, seed)


def test_work_is_counted_from_the_lengths(ops):
    work = [ops.work(c) for c in ops.listed()]
    assert all(w["bytes"] > 0 and w["flops"] > 0 for w in work)
    assert max(w["bytes"] for w in work) >= 16 * min(w["bytes"] for w in work)


@pytest.mark.parametrize("name", ["weights4_step_B32", "weights4_window_B3_S37"])
def test_weights_and_totals_within_their_derived_bars(ops, name):
    """A logit is off by D 2^-23 + 2^-22 of the sum of its terms' magnitudes, at most |q| |k| scale; the log-sum-exp's
    product and the exponential add 2^-21 of its magnitude and 2^-20: e, so that a weight is off by e (1 + e) of itself.  A
    total is off by that much of what it was given, and by 2^-24 of itself for each of at most S additions and a rounding."""
    case, seed = next(c for c in ops.listed() if c["name"] == name), 12
    s = ops.prepare(case, seed)
    ctx, new = ops._lengths(case)
    G, scale = case["Hq"] // case["Hkv"], ops.D ** -0.5
    e = torch.zeros((case["B"], case["S"], case["Hkv"]), dtype=torch.float64, device="cuda")
    for b, (L, n) in enumerate(zip(ctx, new)):
        for h in range(case["Hkv"]):
            longest = ops._exact_cache(s, b, h, 0, L).norm(dim=-1).max()
            q = s["q"][b, :n, h * G:(h + 1) * G].double().norm(dim=-1)
            lse = s["lse"][b, :n, h * G:(h + 1) * G].double().abs()
            e[b, :n, h] = ((ops.D * 2.0 ** -23 + 2.0 ** -22) * scale * longest * q + 2.0 ** -21 * lse + 2.0 ** -20).amax(-1)
    before, want = s["total"].double(), ops.exact(case, seed)
    rel = (e * (1 + e))[..., None]
    most = rel.amax((1, 3))[..., None]
    added = want["total"] - before
    bar = most * added + (max(new) + 1) * 2.0 ** -24 * want["total"] * (1 + 2.0 ** -10)
    for own in (False, True):
        ops.own = own
        try:
            out = ops.run(ops.prepare(case, seed))
        finally:
            ops.own = False
        assert bool(((out["weights"].double() - want["weights"]).abs() <= rel * want["weights"] + 1e-37).all())
        assert bool(((out["total"].double() - want["total"]).abs() <= bar).all())
