"""Rotary positions and the append to the 8-bit cache that applies them, against
their formulas in 64 bits.

Tolerances.  A turned element y = a cos t - b sin t is formed in fp32 from a cosine
and a sine whose angle is off by at most 2^-25 pi (its fraction of a half turn,
rounded to fp32) + 2^-31 pi and which are themselves off by at most an ulp (2^-23 for
values up to 1): (|a| + |b|) (2^-23.3 + 2^-23) in all, two products and a sum add at
most 2^-23 (|a| + |b|); together below TURN = 2^-20 (|a| + |b|).  Rounding to bf16
adds 2^-8 of the result, to e4m3 half a step of the code.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

from tests.gpu_util import assert_no_device_error, f64, gpu, require_gpu
from tests.test_gpu_cache8 import bits, e4m3, make_table, needed_scale, random_cache, store_formula, values

pytestmark = gpu

TURN = 2.0 ** -20
ERR_PAGE = 12
PI = Fraction(3141592653589793238462643383279502884197, 10 ** 39)


def freqs(pairs, base=10000.0):
    return [base ** (-i / pairs) for i in range(pairs)]


def angles(positions, freq, axis):
    """Exact angles reduced to [0, 2 pi): [T, pairs]; positions [axes, T] integers."""
    turn = [Fraction(f) / (2 * PI) for f in freq]
    out = np.zeros((positions.shape[1], len(freq)))
    for j, f in enumerate(turn):
        for t in range(positions.shape[1]):
            x = int(positions[axis[j], t]) * f
            out[t, j] = float(x - (x.numerator // x.denominator)) * 2 * np.pi
    return out


def turned(x, angle, interleaved, back=False):
    """(x turned, |a| + |b| of each element's pair), in 64 bits; x [T, heads, d]."""
    m = angle.shape[1]
    ia, ib = (np.arange(0, 2 * m, 2), np.arange(1, 2 * m, 2)) if interleaved else (np.arange(m), np.arange(m, 2 * m))
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None] * (-1 if back else 1)
    out, size = x.copy(), np.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = np.abs(a) + np.abs(b)
    return out, size


def held_to(got, want, size):
    assert (np.abs(f64(got) - want) <= 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -10) + TURN * size).all()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def spread_axis(pairs, axes):
    return [(7 * j) % axes for j in range(pairs)]


# ---------------------------------------------------------------- the turn and its gradient
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,pairs", [(64, 32), (64, 8), (64, 24), (128, 64), (128, 48), (128, 16)])
@pytest.mark.parametrize("T,H,Hk", [(1, 1, 1), (5, 6, 2), (37, 3, 3), (9, 71, 1)])
def test_turn_and_gradient(T, H, Hk, d, pairs, interleaved):
    fa = require_gpu()
    gen = torch.Generator().manual_seed(T + d + pairs)
    positions = torch.randint(0, 5000, (1, T), generator=gen, dtype=torch.int32)
    plan = fa.rotary_plan(freqs(pairs), interleaved=interleaved)
    q, k, dq, dk = (torch.randn(T, h, d, generator=gen).bfloat16().cuda() for h in (H, Hk, H, Hk))
    q.requires_grad_(), k.requires_grad_()
    out = fa.rotary_embedding(q, k, positions[0].cuda(), plan)
    grads = torch.autograd.grad(out, (q, k), (dq, dk))
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    angle = angles(positions.numpy(), freqs(pairs), [0] * pairs)
    for x, y, dy, dx in zip((q, k), out, (dq, dk), grads):
        held_to(y, *turned(f64(x), angle, interleaved))
        held_to(dx, *turned(f64(dy), angle, interleaved, back=True))
        assert torch.equal(y[..., 2 * pairs:], x[..., 2 * pairs:]) and torch.equal(dx[..., 2 * pairs:], dy[..., 2 * pairs:])
    # against differences: the loss <dy, y> along a direction v, by its values at x + v and x - v
    v = torch.randn(T, H, d, generator=gen).bfloat16().cuda()
    up, down = (fa.rotary_forward((q.detach().float() + f * v.float()).bfloat16(), k.detach(), positions[0].cuda(), plan)[0]
                for f in (1, -1))
    step = (f64((q.detach().float() + v.float()).bfloat16()) - f64((q.detach().float() - v.float()).bfloat16()))
    by_difference = (f64(dq) * (f64(up) - f64(down))).sum()
    by_gradient = (f64(grads[0]) * step).sum()
    # each rounding at most 2^-8 of its value
    slack = 2.0 ** -8 * (np.abs(f64(dq)) * (np.abs(f64(up)) + np.abs(f64(down)))).sum() + 2.0 ** -8 * np.abs(f64(grads[0]) * step).sum()
    assert abs(by_difference - by_gradient) <= slack * 1.01


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes", [2, 3])
@pytest.mark.parametrize("d,pairs", [(64, 32), (128, 48)])
def test_several_axes_and_far_positions(d, pairs, axes, interleaved):
    """Positions up to the ends of int32, negative ones, frequencies above a turn a step."""
    fa = require_gpu()
    T = 12
    gen = torch.Generator().manual_seed(axes)
    far = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, 2 ** 30, 99, -70000, 7, 2 ** 24 + 1, 5])
    positions = torch.stack([far.roll(a) for a in range(axes)]).int()
    freq = [f * 9.7 if j % 5 == 0 else -f if j % 5 == 1 else f for j, f in enumerate(freqs(pairs, 500000.0))]
    axis = spread_axis(pairs, axes)
    plan = fa.rotary_plan(freq, axis=axis, interleaved=interleaved)
    assert plan.axes == axes
    q, k = (torch.randn(T, h, d, generator=gen).bfloat16().cuda() for h in (3, 1))
    out = fa.rotary_forward(q, k, positions.cuda(), plan)
    back = fa.rotary_backward(*out, positions.cuda(), plan)
    angle = angles(positions.numpy(), freq, axis)
    for x, y, z in zip((q, k), out, back):
        held_to(y, *turned(f64(x), angle, interleaved))
        held_to(z, *turned(f64(y), angle, interleaved, back=True))
    assert_no_device_error(fa)


def test_slices_streams_graph_and_python_path(monkeypatch):
    fa = require_gpu()
    gen = torch.Generator().manual_seed(3)
    H, Hk, d, T = 6, 2, 128, 50
    qkv = torch.randn(T, H + 2 * Hk, d, generator=gen).bfloat16().cuda().requires_grad_()
    q, k = qkv[:, :H], qkv[:, H:H + Hk]
    plan, at = fa.rotary_plan(freqs(64)), torch.arange(T, dtype=torch.int32, device="cuda") + 7
    want = fa.rotary_forward(q.detach().contiguous(), k.detach().contiguous(), at, plan)
    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))  # noqa: E731
    assert same(want, fa.rotary_forward(q, k, at, plan)) and same(want, fa.rotary_embedding(q, k, at, plan))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = fa.rotary_forward(q.detach(), k.detach(), at, plan, stream=side)
    side.synchronize()
    assert same(want, other)
    do = [torch.randn(T, h, d, generator=gen).bfloat16().cuda() for h in (H, Hk)]
    grad = torch.autograd.grad(fa.rotary_embedding(q, k, at, plan), qkv, do)[0]
    assert not grad[:, H + Hk:].any()
    # an expanded gradient, and an output that is not used
    one = torch.autograd.grad(fa.rotary_embedding(q, k, at, plan)[0].sum(), qkv)[0]
    assert not one[:, H:].any() and same([one[:, :H]], fa.rotary_backward(torch.ones_like(q), torch.zeros_like(k), at, plan)[:1])
    at2 = at.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = fa.rotary_forward(q.detach(), k.detach(), at2, plan)
    at2.add_(5)
    graph.replay()
    assert same(cap, fa.rotary_forward(q, k, at + 5, plan))
    with pytest.raises(RuntimeError, match="once"):
        g = torch.autograd.grad(fa.rotary_embedding(q, k, at, plan), qkv, do, create_graph=True)[0]
        g.float().square().sum().backward()
    monkeypatch.setattr(fa._binding, "_native", fa._binding._NoNative())
    assert same(want, fa.rotary_forward(q, k, at, plan))
    assert torch.equal(grad, torch.autograd.grad(fa.rotary_embedding(q, k, at, plan), qkv, do)[0])
    torch.cuda.synchronize()
    assert_no_device_error(fa)


def test_training_step_with_attention():
    """Rotary positions in front of the grouped attention, gradients through both,
    against 64 bits.  The turned queries and keys are rounded to bf16 (2^-8 of each),
    as are P, dS and the results: held to 2^-6 of the gradient's norm."""
    fa = require_gpu()
    gen = torch.Generator().manual_seed(5)
    H, Hk, d, lens = 4, 2, 64, [40, 1, 90]
    T, cu = sum(lens), i32(np.cumsum([0] + lens).tolist())
    q, k, v, do = (torch.randn(T, h, d, generator=gen).bfloat16().cuda() for h in (H, Hk, Hk, H))
    at = torch.cat([torch.arange(n) for n in lens]).int()
    plan = fa.rotary_plan(freqs(32))
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    qt, kt = fa.rotary_embedding(leaves[0], leaves[1], at.cuda(), plan)
    got = torch.autograd.grad(fa.flash_attention_grouped(qt, kt, leaves[2], cu, max(lens), causal=True), leaves, do)
    angle = torch.tensor(angles(at.numpy()[None], freqs(32), [0] * 32))[:, None]
    wide = [t.cpu().double().requires_grad_() for t in (q, k, v)]

    def turn(x):
        a, b = x[..., :32], x[..., 32:]
        return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1)

    qs, ks, vs = turn(wide[0]), turn(wide[1]).repeat_interleave(H // Hk, 1), wide[2].repeat_interleave(H // Hk, 1)
    outs = []
    for a, n in zip(np.cumsum([0] + lens).tolist(), lens):
        s = torch.einsum("ihd,jhd->hij", qs[a:a + n], ks[a:a + n]) * d ** -0.5
        s = s.masked_fill(torch.ones(n, n).triu(1).bool(), -float("inf"))
        outs.append(torch.einsum("hij,jhd->ihd", s.softmax(-1), vs[a:a + n]))
    want = torch.autograd.grad(torch.cat(outs), wide, do.cpu().double())
    for a, b in zip(got, want):
        assert np.linalg.norm(f64(a) - b.numpy()) <= 2.0 ** -6 * np.linalg.norm(b.numpy())
    assert_no_device_error(fa)


# ---------------------------------------------------------------- append
def append(fa, q, k, v, cache, table, cu, start, max_new, plan, positions=None, **kw):
    out = fa.cache8_store_rotary(q, k, v, cache, table.cuda(), i32(cu), i32(start), max_new, plan, positions, **kw)
    torch.cuda.synchronize()
    return out


LENS = lambda block: [1, 0, 5, block, 2 * block + 3, 1, 33, 7]  # noqa: E731
STARTS = lambda block: [0, 9, 3, 0, block - 1, block, 2 * block + 5, block - 7]  # noqa: E731


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("d,pairs", [(64, 32), (128, 64), (128, 24)])
@pytest.mark.parametrize("H,Hk", [(1, 1), (10, 5)])
def test_append_at_position_zero_is_the_store(H, Hk, d, pairs, block, interleaved):
    """Turned by nothing: pages, held tokens, scales and codes equal to the store's,
    bit for bit; queries as they came, zeros behind the last sequence."""
    fa = require_gpu()
    lens, start = LENS(block), STARTS(block)
    cols = max(-(-(a + n) // block) for a, n in zip(start, lens))
    caches = [random_cache(fa, len(lens) * cols + 2, Hk, block, d, seed=block + d) for _ in range(2)]
    table, cu = make_table(len(lens) * cols + 2, len(lens), cols, 2), [0] + np.cumsum(lens).tolist()
    gen = torch.Generator().manual_seed(1)
    T = cu[-1] + 5
    q = torch.randn(T, H, d, generator=gen).bfloat16().cuda()
    k, v = ((torch.randn(T, Hk, d, generator=gen) * torch.exp(2 * torch.randn(T, 1, 1, generator=gen))).bfloat16().cuda()
            for _ in range(2))
    plan = fa.rotary_plan(freqs(pairs), interleaved=interleaved)
    got = append(fa, q, k, v, caches[0], table, cu, start, max(lens), plan, torch.zeros(T, dtype=torch.int32, device="cuda"))
    fa.cache8_store(k, v, caches[1], table.cuda(), i32(cu), i32(start), max(lens))
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    for a, b in zip(*caches):
        assert torch.equal(bits(a), bits(b))
    assert torch.equal(got[:cu[-1]], q[:cu[-1]]) and not got[cu[-1]:].any()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("block", [16, 128])
@pytest.mark.parametrize("d,pairs,axes", [(64, 32, 1), (128, 64, 1), (128, 40, 3)])
def test_append_turns(d, pairs, axes, block, interleaved):
    """Keys turned by their positions (a token's place, or given ones): scales are
    those of the turned keys, codes the nearest to them."""
    fa = require_gpu()
    H, Hk = 6, 3
    lens, start = LENS(block), STARTS(block)
    cols = max(-(-(a + n) // block) for a, n in zip(start, lens))
    pages = len(lens) * cols + 2
    cache = random_cache(fa, pages, Hk, block, d, seed=7)
    before = values(cache)
    table, cu = make_table(pages, len(lens), cols, 3), [0] + np.cumsum(lens).tolist()
    gen = torch.Generator().manual_seed(4)
    T = cu[-1]
    q, k, v = (torch.randn(T, h, d, generator=gen).bfloat16().cuda() for h in (H, Hk, Hk))
    axis = spread_axis(pairs, axes)
    plan = fa.rotary_plan(freqs(pairs), axis=axis, interleaved=interleaved)
    place = np.concatenate([np.arange(a, a + n) for a, n in zip(start, lens)])[None].repeat(axes, 0)
    given = None
    if axes > 1:
        place = place * 3 + np.arange(axes)[:, None] * 11 - 50
        given = torch.tensor(place, dtype=torch.int32, device="cuda")
    got = append(fa, q, k, v, cache, table, cu, start, max(lens), plan, given)
    assert_no_device_error(fa)
    angle = angles(place, freqs(pairs), axis)
    held_to(got, *turned(f64(q), angle, interleaved))
    kt, size = turned(f64(k), angle, interleaved)
    ck, cv, sk, sv = values(cache)
    ref_v, ref_sv = before[1].copy(), before[3].copy()
    store_formula(f64(v), ref_v, ref_sv, table.tolist(), cu, start)
    assert np.array_equal(cv, ref_v) and np.array_equal(sv, ref_sv)
    for b, n in enumerate(lens):
        for j in range(start[b] // block, -(-(start[b] + n) // block) if n else 0):
            lo, hi = max(start[b], j * block), min(start[b] + n, (j + 1) * block)
            page, old = int(table[b, j]), max(0, start[b] - j * block)
            rows = slice(cu[b] + lo - start[b], cu[b] + hi - start[b])
            for h in range(Hk):
                y, e = kt[rows, h], TURN * size[rows, h]
                top = np.abs(y).max()
                fits = {needed_scale(y * f) for f in (1.0, 1 - e.max() / top, 1 + e.max() / top)}
                assert len(fits) == 1  # (the largest is not at a scale's border)
                s = max(fits.pop(), before[2][page, h] if old else 0.0)
                assert sk[page, h] == s
                assert np.array_equal(ck[page, h, :old], e4m3(before[0][page, h, :old] * before[2][page, h] / s))
                _, ex = np.frexp(np.abs(y) / s)
                half = np.exp2(np.maximum(ex - 4, -9) - 1.0)
                assert (np.abs(ck[page, h, lo - j * block:hi - j * block] * s - y) <= half * s * (1 + 2.0 ** -20) + e).all()
                assert np.array_equal(ck[page, h, hi - j * block:], before[0][page, h, hi - j * block:])


@pytest.mark.parametrize("d", [64, 128])
def test_append_borders_infinities_and_nan(d):
    """Scales and codes at their borders, infinities and NaN, as the store takes them:
    in dimensions that are not turned and, at position 0, in turned pairs of finite
    values."""
    fa = require_gpu()
    pairs, block = 8, 16
    x = torch.zeros(6 * block, 1, d)
    for i, top in enumerate((448.0, 450.0, 2.0 ** -70, 3.3e38, 0.0, 1.0)):
        x[i * block, 0, i] = top
        x[i * block + 1, 0, :40] = top / 448 * torch.cat([torch.arange(1, 21) / 16, 2.0 ** -torch.arange(0.0, 20.0)])
    x[5 * block + 2, 0, 2 * pairs], x[5 * block + 3, 0, 2 * pairs + 1], x[5 * block + 4, 0, 2 * pairs + 2] = (
        float("inf"), float("-inf"), float("nan"))
    x = x.bfloat16().cuda()
    caches = [fa.cache8_alloc(6, 1, block, d) for _ in range(2)]
    table, cu = torch.arange(6, dtype=torch.int32)[:, None], [i * block for i in range(7)]
    append(fa, x, x, x, caches[0], table, cu, [0] * 6, block, fa.rotary_plan(freqs(pairs)), torch.zeros_like(i32([0] * 6 * block)))
    fa.cache8_store(x, x, caches[1], table.cuda(), i32(cu), i32([0] * 6), block)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    for a, b in zip(*caches):
        assert torch.equal(bits(a), bits(b))


def test_append_indexes_out_of_range_touch_nothing():
    fa = require_gpu()
    cache = random_cache(fa, 4, 1, 16, 64, seed=11)
    plan = fa.rotary_plan(freqs(32))
    x = torch.randn(20, 1, 64).bfloat16().cuda()
    for table, cu, start in (([[-1]], [0, 5], [0]), ([[4]], [0, 5], [3]), ([[2 ** 31 - 1]], [0, 5], [0]),
                             ([[0]], [0, 5], [16]), ([[0]], [0, 5], [2 ** 31 - 1]), ([[0]], [0, 5], [-1])):
        before = [t.clone() for t in cache]
        append(fa, x, x, x, cache, torch.tensor(table, dtype=torch.int32), cu, start, 5, plan)
        assert fa.fa_get_device_error() == ERR_PAGE
        for a, b in zip(before, cache):
            assert torch.equal(bits(a), bits(b))
    # rows that do not exist are not read, tokens past max_new are dropped
    other = fa.Cache8(*(t.clone() for t in cache))
    zero = torch.zeros(20, dtype=torch.int32, device="cuda")
    append(fa, x, x, x, cache, torch.tensor([[0, 1]], dtype=torch.int32), [0, 400], [0], 18, plan, zero)
    fa.cache8_store(x, x, other, i32([[0, 1]]), i32([0, 400]), i32([0]), 18)
    assert_no_device_error(fa)
    for a, b in zip(cache, other):
        assert torch.equal(bits(a), bits(b))


def test_append_slices_stream_graph_and_tail():
    fa = require_gpu()
    H, Hk, d, block, T = 4, 2, 128, 32, 53
    gen = torch.Generator().manual_seed(8)
    qkv = torch.randn(T, H + 2 * Hk, d, generator=gen).bfloat16().cuda()
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    table, cu, start = make_table(8, 2, 4, 9), [0, 20, 50], [5, 0]
    plan = fa.rotary_plan(freqs(64))
    first = random_cache(fa, 8, Hk, block, d, seed=10)
    caches = [first] + [fa.Cache8(*(t.clone() for t in first)) for _ in range(4)]
    want = append(fa, q.contiguous(), k.contiguous(), v.contiguous(), caches[0], table, cu, start, 30, plan)
    assert not want[50:].any()
    got = [append(fa, q, k, v, caches[1], table, cu, start, 30, plan)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got.append(append(fa, q, k, v, caches[2], table, cu, start, 30, plan, stream=side))
    args = (table.cuda(), i32(cu), i32(start), 30, plan)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = fa.cache8_store_rotary(q, k, v, caches[3], *args)
    graph.replay()
    graph.replay()  # storing the same tokens again changes nothing
    got.append(cap)
    # rows behind the last sequence as they were
    out = torch.full_like(want, 3.0)
    fa.fa_cache8_store_rotary(q, k, v, out, caches[4], *args)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    assert torch.equal(out[:50], want[:50]) and (out[50:] == 3).all()
    assert all(torch.equal(want, g) for g in got)
    for c in caches[1:]:
        for a, b in zip(caches[0], c):
            assert torch.equal(bits(a), bits(b))


def test_refusals():
    fa = require_gpu()
    plan = fa.rotary_plan(freqs(32))
    q, k = torch.randn(3, 4, 64).bfloat16().cuda(), torch.randn(3, 2, 64).bfloat16().cuda()
    at = torch.arange(3, dtype=torch.int32, device="cuda")
    for bad in ([], [1.0] * 7, [float("nan")] * 8, [float("inf")] * 8):
        with pytest.raises(ValueError):
            fa.rotary_plan(bad)
    for bad in ([0] * 7, [-1] * 8, [8] * 8):
        with pytest.raises(ValueError):
            fa.rotary_plan([1.0] * 8, axis=bad)
    for f in (fa.rotary_forward, fa.rotary_backward, fa.rotary_embedding):
        with pytest.raises(TypeError):
            f(q.float(), k, at, plan)
        for bad in ((q, k[:2], at, plan), (q, k, at.long(), plan), (q, k, at[:2], plan), (q, k, at[None].repeat(2, 1), plan),
                    (q, k, at.cpu(), plan), (q, k, at, plan._replace(turns=plan.turns.int())),
                    (q, k, at, plan._replace(axis=plan.axis[:8])), (q, k, at, plan._replace(axes=2)),
                    (q, k, at, plan._replace(axes=0)), (q, k, at, fa.rotary_plan(freqs(40))),
                    (q, k, at, plan._replace(turns=plan.turns[:4], axis=plan.axis[:4]))):
            with pytest.raises(ValueError):
                f(*bad)
    with pytest.raises(TypeError):
        fa.rotary_forward(q, k, None, plan)
    with pytest.raises(fa.FaError):
        x = torch.randn(3, 4, 32).bfloat16().cuda()
        fa.rotary_forward(x, x, at, fa.rotary_plan(freqs(16)))
    cache = fa.cache8_alloc(4, 2, 16, 64)
    table, cu, start = i32([[0, 1]]), i32([0, 3]), i32([0])
    s = fa.cache8_store_rotary
    for bad in ((q, k[:, :1], k, cu, start, plan, None), (q, k, k[:2], cu, start, plan, None), (q[:2], k, k, cu, start, plan, None),
                (q, k, k, i32([0, 3, 3]), start, plan, None), (q, k, k, cu, start.long(), plan, None),
                (q, k, k, cu, start, fa.rotary_plan(freqs(40)), None), (q, k, k, cu, start, plan, at.long()),
                (q, k, k, cu, start, plan, at[None].repeat(3, 1))):
        with pytest.raises(ValueError):
            s(*bad[:3], cache, table, bad[3], bad[4], 3, *bad[5:])
    with pytest.raises(fa.FaError):
        s(q, k, k, cache, table, cu, start, 0, plan)
    with pytest.raises(ValueError):
        s(q, k, k, cache, table, cu, start, 2 ** 32 + 1, plan)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
