"""qsa_rotary against the rotation in 64 bits.

Bar: an angle is a fraction of a turn cut to 32 bits (2^-32 turns, 2^-29.3 in radians) and rounded to fp32 (2^-25 of half a
turn, 2^-23.3), its sine and cosine are off by at most 2 units of 2^-24 more, the products and the sum by 3 roundings of
2^-24 of |x_a| + |x_b|: together below 2^-21 (|x_a| + |x_b|) times the magnitude; then half a step of the type (fp16: 2^-25 at
least)."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def qb():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_gqa_qsa_gb300 import _binding, build
    build.build()
    _binding.lib()
    return _binding


def turned(x, pos, freq, interleaved=False, inverse=False, magnitude=1.0):
    """(y, |x_a| + |x_b| of every element's pair) in 64 bits, on the host."""
    x, rot = x.double().cpu(), 2 * freq.numel()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    ang = pos.cpu().double()[..., None] * freq
    c, s = magnitude * torch.cos(ang)[..., None, :], magnitude * torch.sin(ang)[..., None, :] * (-1 if inverse else 1)
    y, size = x.clone(), torch.zeros_like(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, size


def check(got, y, size, dtype, magnitude=1.0):
    bar = 2.0 ** -21 * abs(magnitude) * size + torch.finfo(dtype).eps / 2 * y.abs()
    if dtype == torch.float16:
        bar = torch.maximum(bar, 2.0 ** -21 * abs(magnitude) * size + 2.0 ** -25)
    bar = bar * (1 + 2.0 ** -9)  # half a step of a value that lies across a power of two from the exact one
    err = (got.double().cpu() - y).abs()
    assert bool((err <= bar).all()), float((err - bar).max())


def inputs(dtype, T, H, D, seed, hi=70000):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H, D), generator=g).to(DT[dtype]).cuda()
    pos = torch.randint(0, hi, (T,), generator=g, dtype=torch.int32).cuda()
    return x, pos


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 64, 64), (37, 5, 128, 64), (3, 40, 96, 36), (130, 3, 128, 128), (7, 2, 256, 256),
                                       (11, 4, 80, 2), (9, 3, 66, 34), (5, 2, 20, 12), (600, 36, 128, 64),
                                       (6, 3, 65, 64), (400, 9, 81, 20), (5, 65, 84, 20)])
def test_rotary(qb, dtype, interleaved, T, H, D, rot):
    freq = qb.rotary_frequencies(rot, theta=1e4)
    x, pos = inputs(dtype, T, H, D, T + H)
    for inverse, magnitude in ((False, 1.0), (True, 1.25)):
        y, size = turned(x, pos, freq, interleaved, inverse, magnitude)
        out = torch.full_like(x, 7.0)
        qb.rotary(x, pos, out, freq, interleaved=interleaved, inverse=inverse, magnitude=magnitude)
        check(out, y, size, DT[dtype], magnitude)
        assert torch.equal(out[..., rot:], x[..., rot:])  # what does not turn is copied
        same = x.clone()
        qb.rotary(same, pos, same, freq, interleaved=interleaved, inverse=inverse, magnitude=magnitude)
        assert torch.equal(same, out)


def test_long_positions(qb):
    """Angles of positions up to 2^31 - 1 keep an absolute error, whatever the number of turns.  (The frequency's own
    rounding to 64 bits of a turn and the reference's are 2^31 2^-52 radians apart.)"""
    freq = qb.rotary_frequencies(64, theta=1e4, scaling="blend", factor=32.0, original_length=8192.0)
    x, _ = inputs("fp32", 64, 2, 64, 3)
    pos = torch.tensor([0, 1, 2 ** 20, 2 ** 24 + 1, 2 ** 31 - 1] + list(range(59)), dtype=torch.int32).cuda()
    y, size = turned(x, pos, freq)
    out = torch.empty_like(x)
    qb.rotary(x, pos, out, freq)
    check(out, y, size * (1 + 2.0 ** 21 * 2.0 ** -20), torch.float32)
    assert torch.equal(out[0], x[0])  # position 0 turns nothing


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_views_padding_and_neighbours(qb, dtype):
    """Heads of a packed projection in place; odd strides and offsets; head-major tensors; broadcast rows; rows at negative
    positions and everything between the rows stay as they are."""
    freq = qb.rotary_frequencies(64, theta=5e5)
    g = torch.Generator().manual_seed(1)
    packed = torch.randn((2, 6, 12, 128), generator=g).to(DT[dtype]).cuda()
    pos = torch.randint(0, 9000, (2, 6), generator=g, dtype=torch.int32).cuda()
    pos[0, 4:] = -1
    pos[1, 2] = -2 ** 31
    before = packed.clone()
    y, size = turned(packed[:, :, :9], pos.clamp(min=0), freq)
    qb.rotary(packed[:, :, :9], pos, packed[:, :, :9], freq)
    live = (pos >= 0).cpu()
    check(packed[:, :, :9].cpu()[live], y[live], size[live], DT[dtype])
    assert torch.equal(packed.cpu()[~live], before.cpu()[~live]) and torch.equal(packed[:, :, 9:], before[:, :, 9:])
    # rows one element off any vector, an odd token stride
    wide = torch.randn((5 * 901 + 1,), generator=g).to(DT[dtype]).cuda()
    x = wide[1:].as_strided((5, 3, 128), (901, 300, 1))
    x = wide.as_strided((5, 3, 128), (901, 300, 1), 1)
    p5 = pos.flatten()[:5].clamp(min=0).contiguous()
    y, size = turned(x, p5, freq, True)
    keep = wide.clone()
    qb.rotary(x, p5, x, freq, interleaved=True)
    check(x, y, size, DT[dtype])
    touched = torch.zeros_like(wide, dtype=torch.bool)
    touched.as_strided((5, 3, 64), (901, 300, 1), 1).fill_(True)
    assert torch.equal(wide[~touched], keep[~touched])
    # head-major in and out, and a broadcast input
    x = torch.randn((4, 7, 128), generator=g).to(DT[dtype]).cuda()
    p7 = torch.arange(7, dtype=torch.int32).cuda() * 1000
    y, size = turned(x.transpose(0, 1), p7, freq)
    out = torch.zeros_like(x)
    qb.rotary(x.transpose(0, 1), p7, out.transpose(0, 1), freq)
    check(out.transpose(0, 1), y, size, DT[dtype])
    row = x[:1, :1].expand(7, 4, 128)
    y, size = turned(row, p7, freq)
    out = torch.zeros((7, 4, 128), dtype=x.dtype, device="cuda")
    qb.rotary(row, p7, out, freq)
    check(out, y, size, DT[dtype])
    with pytest.raises(qb.QsaError, match="overlap"):
        qb.rotary(row, p7, out[:1, :1].expand(7, 4, 128), freq)


def test_infinities_and_nans_stay_in_their_pairs(qb):
    freq = qb.rotary_frequencies(64, theta=1e4)
    x, pos = inputs("fp16", 4, 2, 128, 9)
    x[1, 0, 3], x[2, 1, 40] = float("inf"), float("nan")
    out = torch.empty_like(x)
    qb.rotary(x, pos, out, freq)
    bad = torch.zeros_like(x, dtype=torch.bool)
    bad[1, 0, [3, 35]] = bad[2, 1, [8, 40]] = True
    assert bool(torch.isfinite(out[~bad]).all()) and not bool(torch.isfinite(out[bad]).any())


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient(qb, interleaved):
    """The inverse call is the transposed map: against the formula's, and against differences.  (The map is linear: a central
    difference of step 1 has no truncation, only the fp32 errors of its two ends, 2^-21 (|x_a| + |x_b| + 2) each, times dy.)"""
    freq = qb.rotary_frequencies(48, theta=1e4)
    x, pos = inputs("fp32", 6, 2, 64, 4)
    dy, _ = inputs("fp32", 6, 2, 64, 5)
    want, size = turned(dy, pos, freq, interleaved, inverse=True, magnitude=0.75)
    dx = torch.empty_like(dy)
    qb.rotary(dy, pos, dx, freq, interleaved=interleaved, inverse=True, magnitude=0.75)
    check(dx, want, size, torch.float32, 0.75)
    g = torch.Generator().manual_seed(6)
    for _ in range(8):
        d = torch.randint(-1, 2, x.shape, generator=g).float().cuda()
        ends = []
        for sign in (1.0, -1.0):
            y = torch.empty_like(x)
            qb.rotary(x + sign * d, pos, y, freq, interleaved=interleaved, magnitude=0.75)
            ends.append(float((y.double() * dy.double()).sum()))
        slope = (ends[0] - ends[1]) / 2
        bar = float(((x.double().abs().amax() * 2 + 2) * 2.0 ** -21 * dy.double().abs()).sum()) + \
            float((size * 2.0 ** -21).sum())
        assert abs(slope - float((dx.double() * d.double()).sum())) <= bar


def test_another_stream_and_a_graph(qb):
    freq = qb.rotary_frequencies(64, theta=1e4)
    x, pos = inputs("bf16", 33, 4, 128, 8)
    y, size = turned(x, pos, freq)
    st = torch.cuda.Stream()
    out = torch.zeros_like(x)
    st.wait_stream(torch.cuda.current_stream())
    qb.rotary(x, pos, out, freq, stream=st)
    st.synchronize()
    check(out, y, size, torch.bfloat16)
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qb.rotary(x, pos, out, freq)
    freq.zero_()  # read when the call was made, not when it runs
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(out, y, size, torch.bfloat16)


def test_autograd(qb):
    """A Function around the call and its inverse has the formula's gradient; a tensor that a backward pass has saved and the
    call overwrites makes that pass raise, whether the call was made with gradients enabled or not."""
    freq = qb.rotary_frequencies(48, theta=1e4)
    x, pos = inputs("fp32", 6, 2, 64, 4)
    dy, _ = inputs("fp32", 6, 2, 64, 5)

    class Rotary(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            y = torch.empty_like(x)
            qb.rotary(x, pos, y, freq, magnitude=0.75)
            return y

        @staticmethod
        def backward(ctx, dy):
            dx = torch.empty_like(dy)
            qb.rotary(dy, pos, dx, freq, inverse=True, magnitude=0.75)
            return dx

    leaf = x.clone().requires_grad_()
    y = Rotary.apply(leaf)
    check(y.detach(), *turned(x, pos, freq, magnitude=0.75), torch.float32, 0.75)
    y.backward(dy)
    check(leaf.grad, *turned(dy, pos, freq, inverse=True, magnitude=0.75), torch.float32, 0.75)
    with pytest.raises(ValueError, match="gradient"):
        qb.rotary(leaf, pos, torch.empty_like(x), freq)
    for enabled in (True, False):
        w, seen = torch.ones_like(x).requires_grad_(), x.clone()
        loss = (w * seen).sum()
        with torch.set_grad_enabled(enabled):
            qb.rotary(seen[:, :1], pos, seen[:, :1], freq)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    with torch.inference_mode():  # such tensors have no version
        frozen = x.clone()
    qb.rotary(frozen, pos, frozen, freq)
    qb.rotary(x, pos, x, freq)
    assert torch.equal(frozen, x)
