"""Grouped heads over packed batches: forward and backward against the formulas
in 64 bits, rows behind the last sequence, rows of other sequences, strides,
streams and graphs.

Tolerances.  u = 2^-9 bounds bf16's relative rounding error as the kernels use
it twice (a probability, an output; half a step is 2^-9 of the value's binade
top, at most 2^-8 of the value).
  O: each P_ij is rounded to bf16 (at most 2^-8 P_ij), so Σ P_ij |v_j| <= max|v|
     moves by at most 2^-8 max|v|, and the output's own rounding adds
     2^-8 |O| <= 2^-8 max|v|: |dO| <= 2^-7 max|v|.
  LSE: fp32 sums of fp32 exponentials of scores whose products are exact in
     fp32 and summed over d terms: 2^-23 · d · Σ|q||k| scale is far below 1e-3;
     held to 1e-4.
  dQ, dK, dV: sums of products of a rounded factor (P or dS, 2^-8) with exact
     ones, dS moreover from D formed of the rounded O (2^-8 again); as relative
     Frobenius norms the independent roundings (uniform: a 3^-1/2 of their
     bound, 2^-8 · 0.58 = 2.3e-3 each, four of them in dQ and dK: P, O in D,
     dS, the output) add to at most 2 · 2.3e-3 in the root of squares; held
     to 1e-2.
"""
import numpy as np
import pytest
import torch

from io_aware_attention_flash_gb300 import workloads as wl
from tests.gpu_util import assert_no_device_error, f64, gpu, rel_fro, require_gpu

pytestmark = gpu

LSE_TOL = 1e-4
GRAD_TOL = 1e-2


def make(lengths, H, Hk, d, seed, pad=0, amplitude=1.0):
    gen = torch.Generator().manual_seed(seed)
    cu = wl.cu_seqlens_from_lengths(lengths)
    T = max(int(cu[-1]) + pad, 1)
    draw = lambda h: (torch.randn(T, h, d, generator=gen) * amplitude).to(torch.bfloat16)  # noqa: E731
    return cu, draw(H), draw(Hk), draw(Hk), draw(H)


def formula(cu, q, k, v, do, scale, causal):
    """O, LSE, dQ, dK, dV of every sequence and head in 64 bits; zeros (LSE -inf)
    in rows of no sequence."""
    q, k, v, do = (f64(x) for x in (q, k, v, do))
    T, H, d = q.shape
    G = H // k.shape[1]
    o, dq, dk, dv = np.zeros_like(q), np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    lse = np.full((H, T), -np.inf)
    for a, b in zip(cu[:-1].tolist(), cu[1:].tolist()):
        if a == b:
            continue
        n = b - a
        hidden = np.triu(np.ones((n, n), bool), 1) if causal else np.zeros((n, n), bool)
        for h in range(H):
            kh, vh = k[a:b, h // G], v[a:b, h // G]
            s = np.where(hidden, -np.inf, scale * q[a:b, h] @ kh.T)
            m = s.max(1, keepdims=True)
            e = np.exp(s - m)
            l = e.sum(1, keepdims=True)
            p = e / l
            lse[h, a:b] = (m + np.log(l))[:, 0]
            o[a:b, h] = p @ vh
            dp = do[a:b, h] @ vh.T
            ds = p * (dp - (p * dp).sum(1, keepdims=True))
            dq[a:b, h] = scale * ds @ kh
            dk[a:b, h // G] += scale * ds.T @ q[a:b, h]
            dv[a:b, h // G] += p.T @ do[a:b, h]
    return o, lse, dq, dk, dv


def check(fa, cu, q, k, v, do, causal, max_len, scale=None, dev=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    qd, kd, vd, dod = dev if dev is not None else (x.cuda() for x in (q, k, v, do))
    cu_d = cu.cuda()
    o, lse = fa.attention_forward_grouped(qd, kd, vd, cu_d, max_len, causal, scale)
    grads = fa.attention_backward_grouped(qd, kd, vd, o, dod, lse, cu_d, max_len, causal, scale)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    O, L, *G = formula(cu, q, k, v, do, scale, causal)
    end = int(cu[-1])
    assert np.abs(f64(o) - O).max() <= 2.0 ** -7 * np.abs(f64(v)[:max(end, 1)]).max()
    assert not f64(o)[end:].any()
    seen = np.isfinite(L)
    got = f64(lse)
    assert np.array_equal(np.isfinite(got), seen) and (got[~seen] == -np.inf).all()
    assert not seen.any() or np.abs(got[seen] - L[seen]).max() <= LSE_TOL
    for name, g, ref in zip(("dq", "dk", "dv"), grads, G):
        g = f64(g)
        assert np.isfinite(g).all(), name
        assert not g[end:].any(), name
        # a single visible key has dS = 0: what is left is rounding, next to |do||v|
        floor = 1e-2 * np.sqrt(g.size) if name != "dv" else 0.0
        assert np.linalg.norm(g - ref) <= GRAD_TOL * max(np.linalg.norm(ref), floor), (name, rel_fro(g, ref))
    return o, lse, grads


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(4, 1), (6, 2), (3, 3), (14, 2)])
def test_ragged_lengths(H, Hk, d, causal):
    fa = require_gpu()
    lengths = [1, 0, 5, 127, 128, 129, 0, 300, 64, 257, 1]
    check(fa, *make(lengths, H, Hk, d, seed=d + H, pad=19), causal, max(lengths))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 31, 33, 255, 256, 257, 511, 513, 700])
def test_one_sequence(n, d):
    fa = require_gpu()
    check(fa, *make([n], 8, 2, d, seed=n), True, n)


@pytest.mark.parametrize("d", [64, 128])
def test_longer_sequences(d):
    """Several query and key tiles a head, the group in parts (few sequences)
    and one CTA a group (many sequences)."""
    fa = require_gpu()
    check(fa, *make([1000, 1100], 4, 2, d, seed=3), True, 1100)
    check(fa, *make([300] * 40, 4, 2, d, seed=4), False, 300)
    check(fa, *make([300] * 80, 4, 2, d, seed=5), False, 300)
    check(fa, *make([300] * 2, 4, 2, d, seed=6), False, 300)
    sizes = [fa.fa_bwd_grouped_workspace_bytes(n, 300, 300 * n, 4, 2, d, False) / (300 * n) for n in (2, 80)]
    assert sizes[0] > sizes[1] + 2 * 2 * 2 * d * 4 - 64, "the two calls were meant to split and not to split the group"


def test_only_empty_sequences():
    """No row belongs to a sequence: zeros, -infinity, and nothing left running
    that later calls on the same memory would meet."""
    fa = require_gpu()
    for d in (64, 128):
        _, q, k, v, do = (t.cuda() for t in make([0, 0], 4, 2, d, seed=1, pad=300))
        cu = torch.zeros(3, dtype=torch.int32, device="cuda")
        for _ in range(20):
            o, lse = fa.attention_forward_grouped(q, k, v, cu, 50, True)
            grads = fa.attention_backward_grouped(q, k, v, o, do, lse, cu, 50, True)
            filled = [torch.full_like(t, 3.0) for t in (q, k, v, o)]
            torch.cuda.synchronize()
            assert not o.any() and (lse == -np.inf).all() and not any(g.any() for g in grads)
            assert all((t == 3.0).all() for t in filled)
            del o, lse, grads, filled
        assert_no_device_error(fa)


def test_max_seqlen_above_the_longest_and_large_scores():
    fa = require_gpu()
    cu, q, k, v, do = make([200, 77], 4, 2, 128, seed=8)
    check(fa, cu, q, k, v, do, True, 1000)
    check(fa, cu, (q.float() * 20).bfloat16(), k, v, do, True, 200)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3e38])
def test_what_stands_in_other_rows_does_not_matter(bad, d, causal):
    """Rows behind the last sequence and a whole neighbouring sequence hold NaN
    or infinities: every other sequence's results are bit for bit what they are
    with zeros there (dQ up to the order of its fp32 sums)."""
    fa = require_gpu()
    lengths = [130, 50, 70, 33]
    cu, *ts = make(lengths, 4, 2, d, seed=5, pad=40)
    cu_d = cu.cuda()
    runs = []
    for fill in (0.0, bad):
        q, k, v, do = (t.clone().cuda() for t in ts)
        for t in (q, k, v, do):
            t[130:180] = fill        # the second sequence
            t[int(cu[-1]):] = fill   # behind the last
        o, lse = fa.attention_forward_grouped(q, k, v, cu_d, max(lengths), causal)
        grads = fa.attention_backward_grouped(q, k, v, o, do, lse, cu_d, max(lengths), causal)
        torch.cuda.synchronize()
        assert_no_device_error(fa)
        runs.append((o, lse.T, *grads))
    keep = torch.cat([torch.arange(0, 130), torch.arange(180, int(cu[-1]))]).cuda()
    for i, (a, b) in enumerate(zip(*runs)):
        assert torch.isfinite(b[keep].float()).all()
        if i == 2:
            assert rel_fro(f64(b[keep]), f64(a[keep])) < 2.0 ** -8
        else:
            assert torch.equal(a[keep], b[keep]), i
        if i != 1:
            assert not b[int(cu[-1]):].float().any()


def test_caller_buffers_behind_the_last_sequence_are_left():
    fa = require_gpu()
    cu, q, k, v, do = (t.cuda() for t in make([40, 90], 4, 2, 64, seed=6, pad=50))
    T, end = q.shape[0], 130
    o, dq, dk, dv = (torch.full_like(t, 7.0) for t in (q, q, k, v))
    lse = torch.full((4, T), 7.0, device="cuda")
    ws = torch.empty(fa.fa_bwd_grouped_workspace_bytes(2, 90, T, 4, 2, 64, True), dtype=torch.uint8, device="cuda")
    fa.fa_fwd_grouped(q, k, v, o, lse, cu, 90, True)
    fa.fa_bwd_grouped(q, k, v, o, do, lse, dq, dk, dv, ws, cu, 90, True)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    assert (lse[:, end:] == 7.0).all() and not (lse[:, :end] == 7.0).any()
    for t in (o, dq, dk, dv):
        assert (t[end:] == 7.0).all() and not (t[:end] == 7.0).all(-1).any()


def test_offsets_that_lie_are_clamped():
    """cu_seqlens past the tensors or decreasing: nothing outside is touched
    (guard rows around every output stay), nothing hangs."""
    fa = require_gpu()
    H, Hk, d, T = 4, 2, 64, 150
    for offsets in ([0, 100, 400], [0, 120, 60, 150], [-5, 70, 2 ** 31 - 1]):
        cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        full = [torch.randn(T + 256, h, d, device="cuda").bfloat16() for h in (H, Hk, Hk, H)]
        outs = [torch.full((T + 256, h, d), 7.0, device="cuda", dtype=torch.bfloat16) for h in (H, H, Hk, Hk)]
        lse = torch.full((H * T + 1024,), 7.0, device="cuda")
        q, k, v, do = (t[128:128 + T] for t in full)
        o, dq, dk, dv = (t[128:128 + T] for t in outs)
        stat = lse[512:512 + H * T].view(H, T)
        n = fa.fa_bwd_grouped_workspace_bytes(len(offsets) - 1, 130, T, H, Hk, d, True)
        ws = torch.zeros(n + 512, dtype=torch.uint8, device="cuda")
        fa.fa_fwd_grouped(q, k, v, o, stat, cu, 130, True)
        fa.fa_bwd_grouped(q, k, v, o, do, stat, dq, dk, dv, ws[:n], cu, 130, True)
        torch.cuda.synchronize()
        assert_no_device_error(fa)
        for t in outs:
            assert (t[:128] == 7.0).all() and (t[128 + T:] == 7.0).all()
        assert (lse[:512] == 7.0).all() and (lse[512 + H * T:] == 7.0).all() and not ws[n:].any()


@pytest.mark.parametrize("d", [64, 128])
def test_slices_of_one_projection(d):
    fa = require_gpu()
    H, Hk, lengths = 6, 2, [150, 64, 3]
    cu, q, k, v, do = make(lengths, H, Hk, d, seed=7)
    qkv = torch.cat([q, k, v], 1).cuda()
    dev = (qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:], do.cuda())
    assert not dev[0].is_contiguous()
    check(fa, cu, q, k, v, do, True, 150, dev=dev)


@pytest.mark.parametrize("d", [64, 128])
def test_autograd_and_differences(d):
    """The autograd function's gradients against the formula's, and the loss's
    change along a direction against the gradients in it."""
    fa = require_gpu()
    cu, q, k, v, do = make([70, 200], 4, 2, d, seed=9)
    leaves = [t.cuda().requires_grad_() for t in (q, k, v)]
    cu_d = cu.cuda()
    o = fa.flash_attention_grouped(*leaves, cu_d, 200, causal=True)
    o.backward(do.cuda())
    O, L, *ref = formula(cu, q, k, v, do, d ** -0.5, True)
    for t, r in zip(leaves, ref):
        assert rel_fro(f64(t.grad), r) <= GRAD_TOL
    # central difference in 64 bits of the same loss along the gradients' signs
    steps = [np.sign(r) for r in ref]
    eps = 1e-4
    up, down = (formula(cu, *(torch.from_numpy(f64(t) + s * eps * e) for t, e in zip((q, k, v), steps)), do, d ** -0.5,
                        True)[0] for s in (1, -1))
    slope = ((up - down) * f64(do)).sum() / (2 * eps)
    got = sum((f64(t.grad) * e).sum() for t, e in zip(leaves, steps))
    assert abs(got - slope) <= 1e-2 * abs(slope)
    with pytest.raises(RuntimeError):
        o = fa.flash_attention_grouped(*leaves, cu_d, 200, causal=True)
        (g,) = torch.autograd.grad(o, leaves[0], do.cuda(), create_graph=True)
        g.sum().backward()


def test_only_some_leaves_need_gradients():
    fa = require_gpu()
    cu, q, k, v, do = (t.cuda() for t in make([70], 4, 1, 64, seed=10))
    k.requires_grad_()
    o = fa.flash_attention_grouped(q, k, v, cu, 70, causal=True)
    o.backward(do)
    assert q.grad is None and v.grad is None and torch.isfinite(k.grad.float()).all()
    # a gradient that arrives expanded from one value
    k.grad = None
    fa.flash_attention_grouped(q, k, v, cu, 70, causal=True).sum().backward()
    assert torch.isfinite(k.grad.float()).all()


def test_own_stream_and_captured_training_step():
    fa = require_gpu()
    cu, q, k, v, do = (t.cuda() for t in make([190, 5, 400], 4, 2, 128, seed=11, pad=3))
    o, lse = fa.attention_forward_grouped(q, k, v, cu, 400, True)
    want = (o, lse, *fa.attention_backward_grouped(q, k, v, o, do, lse, cu, 400, True))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, lse2 = fa.attention_forward_grouped(q, k, v, cu, 400, True, stream=side)
    got = (o2, lse2, *fa.attention_backward_grouped(q, k, v, o2, do, lse2, cu, 400, True, stream=side))
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, lse3 = fa.attention_forward_grouped(q, k, v, cu, 400, True)
        cap = (o3, lse3, *fa.attention_backward_grouped(q, k, v, o3, do, lse3, cu, 400, True))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    for i, (a, b, c) in enumerate(zip(want, got, cap)):
        if i == 2:  # dQ: fp32 sums in another order
            assert rel_fro(f64(b), f64(a)) < 2.0 ** -8 and rel_fro(f64(c), f64(a)) < 2.0 ** -8
        else:
            assert torch.equal(a, b) and torch.equal(a, c), i
    # new lengths in the captured buffers
    cu.copy_(torch.tensor([0, 100, 300, 310], dtype=torch.int32))
    graph.replay()
    o, lse = fa.attention_forward_grouped(q, k, v, cu, 400, True)
    assert torch.equal(o, cap[0]) and torch.equal(lse, cap[1])


def test_more_than_two_to_the_31_elements():
    """1200 sequences of 500 tokens, 32 heads of 128: q holds 2.4e9 elements.
    The first and the last sequence against the formula, one head of each group."""
    fa = require_gpu()
    n, nseq, H, Hk, d = 500, 1200, 32, 2, 128
    T = n * nseq
    assert T * H * d > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(33)
    q, do = (torch.empty(T, H, d, device="cuda", dtype=torch.bfloat16).normal_(generator=g) for _ in range(2))
    k, v = (torch.empty(T, Hk, d, device="cuda", dtype=torch.bfloat16).normal_(generator=g) for _ in range(2))
    cu = torch.arange(0, T + 1, n, dtype=torch.int32, device="cuda")
    o, lse = fa.attention_forward_grouped(q, k, v, cu, n, True)
    grads = fa.attention_backward_grouped(q, k, v, o, do, lse, cu, n, True)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    for a in (0, T - n):
        rows = [t[a:a + n].cpu() for t in (q, k, v, do)]
        O, L, *ref = formula(torch.tensor([0, n]), *rows, d ** -0.5, True)
        assert np.abs(f64(o[a:a + n]) - O).max() <= 2.0 ** -7 * np.abs(f64(rows[2])).max()
        assert np.abs(f64(lse[:, a:a + n]) - L).max() <= LSE_TOL
        for t, r in zip(grads, ref):
            assert rel_fro(f64(t[a:a + n]), r) <= GRAD_TOL


def test_two_calls_at_once():
    """Two training steps of different shapes on two streams, queued in turn,
    each with a workspace of its own."""
    fa = require_gpu()
    jobs = []
    for lengths, H, Hk, d, seed in (([700, 90, 300], 8, 2, 128, 31), ([513, 40], 4, 4, 64, 32)):
        cu, q, k, v, do = (t.cuda() for t in make(lengths, H, Hk, d, seed=seed, pad=7))
        n = max(lengths)
        o, lse = fa.attention_forward_grouped(q, k, v, cu, n, True)
        want = (o, lse, *fa.attention_backward_grouped(q, k, v, o, do, lse, cu, n, True))
        ws = torch.empty(fa.fa_bwd_grouped_workspace_bytes(len(lengths), n, q.shape[0], H, Hk, d, True), dtype=torch.uint8,
                         device="cuda")
        jobs.append((torch.cuda.Stream(), (q, k, v, cu, n), do, ws, want))
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for side, (q, k, v, cu, n), do, ws, want in jobs:
            o, lse = fa.attention_forward_grouped(q, k, v, cu, n, True, stream=side)
            got.append(((o, lse, *fa.attention_backward_grouped(q, k, v, o, do, lse, cu, n, True, stream=side, workspace=ws)),
                        want))
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    for a, b in got:
        for i, (x, y) in enumerate(zip(a, b)):
            assert rel_fro(f64(x), f64(y)) < 2.0 ** -8 if i == 2 else torch.equal(x, y), i


def test_single_heads_match_the_packed_entry_points():
    """H = Hk: the outputs of the packed entry points; dK (and dQ) up to the
    rows that see few keys, whose row statistic is exact here: each side's own
    error is at most GRAD_TOL."""
    fa = require_gpu()
    lengths = [100, 257]
    cu, q, k, v, do = (t.cuda() for t in make(lengths, 3, 3, 128, seed=12))
    o, lse = fa.attention_forward_grouped(q, k, v, cu, 257, True)
    o1, lse1 = fa.attention_forward_varlen(q, k, v, cu, 257, True)
    assert torch.equal(o, o1)
    assert torch.equal(lse[:, :100], lse1[0, :, :100]) and torch.equal(lse[:, 100:], lse1[1])
    _, dk, dv = fa.attention_backward_grouped(q, k, v, o, do, lse, cu, 257, True)
    _, dk1, dv1 = fa.attention_backward_varlen(q, k, v, o1, do, lse1, cu, 257, True)
    assert torch.equal(dv, dv1) and rel_fro(f64(dk), f64(dk1)) <= 2 * GRAD_TOL
    assert torch.equal(dk[16:100], dk1[16:100]) or rel_fro(f64(dk[16:100]), f64(dk1[16:100])) <= 2.0 ** -8


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 7, 16, 17, 30])
def test_gradients_of_short_sequences(n, d, causal):
    """Rows that see few keys, where dP - D is a small difference of large
    numbers: dS = 0 exactly for one key; else the roundings of dS and of the
    output (each at most 2^-8 of a value, as independent errors 2.3e-3 in the
    norm, 3.3e-3 together) are all that is left: held to 5e-3."""
    fa = require_gpu()
    cu, q, k, v, do = make([n] * 12, 6, 2, d, seed=20 + n)
    dev = [t.cuda() for t in (q, k, v, do, cu)]
    o, lse = fa.attention_forward_grouped(*dev[:3], dev[4], n, causal)
    grads = fa.attention_backward_grouped(*dev[:3], o, dev[3], lse, dev[4], n, causal)
    _, _, *ref = formula(cu, q, k, v, do, d ** -0.5, causal)
    for g, r in zip(grads, ref):
        if n == 1 and not r.any():
            assert not g.float().any()
        else:
            assert rel_fro(f64(g), r) <= 5e-3
    assert_no_device_error(fa)


def test_refusals():
    fa = require_gpu()
    cu, q, k, v, do = (t.cuda() for t in make([40], 4, 2, 64, seed=13))
    f = fa.attention_forward_grouped
    with pytest.raises(TypeError):
        f(q.float(), k, v, cu, 40)
    with pytest.raises(ValueError):
        f(q, k, v[:, :1], cu, 40)
    with pytest.raises(ValueError):
        f(q, k.transpose(0, 1).contiguous().transpose(0, 1), v, cu, 40)
    with pytest.raises(ValueError):
        f(q, k, v, cu.long(), 40)
    with pytest.raises(ValueError):
        f(q, k, v, cu.cpu(), 40)
    with pytest.raises(fa.FaError):
        f(q[:, :3].contiguous(), k, v, cu, 40)  # 3 heads over 2
    with pytest.raises(fa.FaError):
        f(q, k, v, cu, 0)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(fa.FaError):
            f(q, k, v, cu, 40, scale=scale)
    o, lse = f(q, k, v, cu, 40)
    with pytest.raises(fa.FaError):
        fa.attention_backward_grouped(q, k, v, o, do, lse, cu, 40, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert_no_device_error(fa)


def test_compiled_and_python_calls_agree():
    """The helpers' compiled calls do what their Python paths do, and hand over
    what is not in order."""
    fa = require_gpu()
    from io_aware_attention_flash_gb300 import _binding
    n = _binding.native()
    cu, q, k, v, do = (t.cuda() for t in make([40, 200], 4, 2, 64, seed=14, pad=5))
    o, lse = n.forward_grouped(q, k, v, cu, 200, True, None)
    checked = _binding._grouped(q, k, v, cu)
    o1, lse1 = fa._forward_grouped(checked, q, k, v, cu, 200, True, None)
    assert torch.equal(o, o1) and torch.equal(lse, lse1)
    _, dk, dv = n.backward_grouped(q, k, v, cu, 200, True, 0.3, o, do, lse)
    _, dk1, dv1 = fa._backward_grouped(checked, q, k, v, o, do, lse, cu, 200, True, 0.3, None)
    assert torch.equal(dk, dk1) and torch.equal(dv, dv1)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    o2 = n.flash_attention_grouped(*leaves, cu, 200, True, None)
    o3 = fa._FlashAttentionGrouped.apply(*leaves, cu, 200, True, None)
    assert torch.equal(o2, o3) and o2.requires_grad
    for a, b in zip(torch.autograd.grad(o2, leaves[1:], do), torch.autograd.grad(o3, leaves[1:], do)):
        assert torch.equal(a, b)
    with pytest.raises(RuntimeError):
        o2 = n.flash_attention_grouped(*leaves, cu, 200, True, None)
        (g,) = torch.autograd.grad(o2, leaves[0], do, create_graph=True)
        g.sum().backward()
    for bad in ((q.float(), k, v, cu, 200, True, None), (q, k, v, cu.cpu(), 200, True, None), (q, k, v, cu, 0, True, None),
                (q, k, v, cu, 2 ** 32 + 200, True, None), (q, k, v, cu, 200, True, -1.0), (q, k, v, cu, 200, True, "1"),
                (q, k, 3, cu, 200, True, None), (q, k, v, cu)):
        assert n.forward_grouped(*bad) is None and n.flash_attention_grouped(*bad) is None
    with pytest.raises(ValueError):
        fa.attention_forward_grouped(q, k, v, cu, 2 ** 32 + 200)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
