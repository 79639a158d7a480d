"""Rotary positions, the append and the chunk attention as programs call them: directly
behind one another, from several threads, under PyTorch's modes and hooks, captured,
and at the ends of what they take."""
import threading
import time

import numpy as np
import pytest
import torch

from tests.gpu_util import assert_no_device_error, f64, gpu, require_gpu
from tests.test_gpu_cache8 import bits, make_table, random_cache
from tests.test_gpu_chunk8 import check

pytestmark = gpu

I32 = dict(dtype=torch.int32, device="cuda")


def i32(v):
    return torch.tensor(v, **I32)


def draw(gen, *shape):
    return torch.randn(*shape, generator=gen).bfloat16().cuda()


def assert_same(got, want):
    assert len(got) == len(want)
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(bits(a), bits(b)), i


def plan_of(fa, pairs, axes=1):
    return fa.rotary_plan([10000.0 ** (-j / pairs) for j in range(pairs)], axis=[j % axes for j in range(pairs)])


@pytest.mark.parametrize("B,H,Hk,d,block,piece,held", [(2, 8, 2, 128, 16, 40, 3000), (5, 4, 4, 64, 64, 1, 50), (3, 16, 1, 64, 32, 130, 0)])
def test_calls_directly_behind_one_another(B, H, Hk, d, block, piece, held):
    """Append and attend in turn, each token twice the size of those before, so that
    pages' scales change under the attention that follows at once: the results are, bit
    for bit, those of the same calls with a synchronisation after each.  How far two
    kernels overlap differs from run to run, so the run is repeated, and captured."""
    fa = require_gpu()
    steps, gen = 8, torch.Generator().manual_seed(B + d)
    cols = -(-(held + steps * piece) // block)
    table = make_table(B * cols, B, cols, d).cuda()
    plan = plan_of(fa, d // 2)
    first = random_cache(fa, B * cols, Hk, block, d, seed=B)
    x = [(draw(gen, B * piece, H + 2 * Hk, d) * 2.0 ** i).bfloat16() for i in range(steps)]
    cu = torch.arange(B + 1, **I32) * piece
    starts = [torch.full((B,), held + i * piece, **I32) for i in range(steps)]
    lens = [torch.full((B,), held + (i + 1) * piece, **I32) for i in range(steps)]

    def run(cache, pause):
        out = []
        for i in range(steps):
            q = fa.cache8_store_rotary(x[i][:, :H], x[i][:, H:H + Hk], x[i][:, H + Hk:], cache, table, cu, starts[i], piece, plan)
            pause()
            out += [q, *fa.attention_chunk_cache8(q, cache, table, cu, lens[i], piece, held + steps * piece, True, 2.0 ** (-2 * i) / d)]
            pause()
        return out

    cache = fa.Cache8(*[t.clone() for t in first])
    torch.cuda.synchronize()
    want = run(cache, torch.cuda.synchronize)
    want_cache = [t.clone() for t in cache]

    def reset():
        for t, e in zip(cache, first):
            bits(t).copy_(bits(e))
        torch.cuda.synchronize()

    for _ in range(5):
        reset()
        got = run(cache, lambda: None)
        torch.cuda.synchronize()
        assert_same(got, want)
        assert_same(cache, want_cache)
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = run(cache, lambda: None)
    for _ in range(3):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert_same(cap, want)
        assert_same(cache, want_cache)
    assert_no_device_error(fa)


def small(fa, seed=0):
    """Small calls of each kind, with their results."""
    gen = torch.Generator().manual_seed(seed)
    q, k = draw(gen, 70, 4, 64), draw(gen, 70, 2, 64)
    cu, start, lens, table, at = i32([0, 30, 70]), i32([0, 5]), i32([30, 45]), i32([[0, 1, 2], [3, 4, 5]]), torch.arange(70, **I32)
    plan = plan_of(fa, 32)
    cache = random_cache(fa, 6, 2, 16, 64, seed)
    mine = fa.Cache8(*[t.clone() for t in cache])
    leaf = q.clone().requires_grad_()
    return {
        "rotary": lambda: fa.rotary_forward(q, k, at, plan),
        "autograd": lambda: torch.autograd.grad(fa.rotary_embedding(leaf, k, at, plan), leaf, (q, k)),
        "append": lambda: [fa.cache8_store_rotary(q, k, k, mine, table, cu, start, 40, plan)],
        "chunk": lambda: fa.attention_chunk_cache8(q, cache, table, cu, lens, 40, 45, True),
    }


def test_the_python_path_gives_the_same(monkeypatch):
    fa = require_gpu()
    want = {n: f() for n, f in small(fa).items()}
    monkeypatch.setattr(fa._binding, "_native", fa._binding._NoNative())
    for n, f in small(fa).items():
        assert_same(f(), want[n])
    assert_no_device_error(fa)


def test_two_threads_at_once():
    fa = require_gpu()
    wrong, sides = [], [torch.cuda.Stream() for _ in range(2)]
    wants = [{n: f() for n, f in small(fa, i).items()} for i in range(2)]
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(sides[i]):
            calls = small(fa, i)
            for _ in range(100):
                for n, f in calls.items():
                    got = f()
                    sides[i].synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, wants[i][n])):
                        wrong.append((i, n))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong
    assert_no_device_error(fa)


@pytest.mark.parametrize("name", ["rotary", "autograd", "append", "chunk"])
def test_a_full_launch_queue_stops_no_other_thread(name):
    """More calls are queued behind a bounded spin than the driver takes: the call that
    blocks must not hold the interpreter (another thread notes the time)."""
    fa = require_gpu()
    call = small(fa)[name]
    for _ in range(10):
        call()
    torch.cuda.synchronize()
    gap, done = [0.0], threading.Event()

    def clock():
        last = time.perf_counter()
        while not done.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gap[0] = max(gap[0], now - last)
            last = now

    t = threading.Thread(target=clock)
    t.start()
    begin = time.perf_counter()
    torch.cuda._sleep(2_000_000_000)
    for _ in range(2000):
        call()
    blocked = time.perf_counter() - begin
    done.set()
    t.join()
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    assert blocked > 0.5, "the queue was meant to fill"
    assert gap[0] < 0.25, f"another thread stood still for {gap[0]:.2f} s of {blocked:.2f} s"


@pytest.mark.parametrize("compiled", [True, False])
@pytest.mark.parametrize("mode", ["anomaly", "dispatch", "hooks", "save_on_cpu", "inference"])
def test_modes_and_hooks(mode, compiled, monkeypatch):
    from torch.utils._python_dispatch import TorchDispatchMode

    fa = require_gpu()
    if not compiled:
        monkeypatch.setattr(fa._binding, "_native", fa._binding._NoNative())
    seen = []

    class Log(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            seen.append(str(func))
            return func(*args, **(kwargs or {}))

    gen = torch.Generator().manual_seed(72)
    q, k, dq, dk = (draw(gen, 150, h, 64) for h in (4, 2, 4, 2))
    at = torch.stack([torch.arange(150, **I32), 3 * torch.arange(150, **I32)])
    plan = plan_of(fa, 16, 2)

    def step():
        leaves = [t.clone().requires_grad_() for t in (q, k)]
        out = fa.rotary_embedding(*leaves, at, plan)
        return list(out) if torch.is_inference_mode_enabled() else [*out, *torch.autograd.grad(out, leaves, (dq, dk))]

    want = step()
    scope = {"anomaly": lambda: torch.autograd.detect_anomaly(check_nan=True), "dispatch": Log,
             "hooks": lambda: torch.autograd.graph.saved_tensors_hooks(lambda t: seen.append(1) or t.clone(), lambda t: t),
             "save_on_cpu": torch.autograd.graph.save_on_cpu, "inference": torch.inference_mode}[mode]
    with scope():
        got = step()
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    assert mode not in ("dispatch", "hooks") or seen
    assert_same(got, want[:len(got)])


def test_saved_positions_are_watched():
    """What the gradient needs may not be changed before it, nor come back as another type."""
    fa = require_gpu()
    q = torch.randn(9, 2, 64).bfloat16().cuda().requires_grad_()
    at, plan = torch.arange(9, **I32), plan_of(fa, 32)
    out, _ = fa.rotary_embedding(q, q.detach(), at, plan)
    at.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        out.sum().backward()
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: t.long() if t.shape == (9,) else t):
        out, _ = fa.rotary_embedding(q, q.detach(), at, plan)
        with pytest.raises(RuntimeError, match="saved tensors"):
            out.sum().backward()
    torch.cuda.synchronize()
    assert_no_device_error(fa)


def test_captured_training_step():
    """Rotary positions in front of the attention, forward and backward in one graph,
    replayed with other inputs: the eager step's gradients (dQ, whose sums' order
    differs from run to run, to 2^-8 of its norm; a turn does not change it)."""
    fa = require_gpu()
    gen = torch.Generator().manual_seed(9)
    T, cu, at, plan = 200, i32([0, 60, 200]), torch.arange(200, **I32), plan_of(fa, 32)
    q, k, v, do = (draw(gen, T, h, 64) for h in (4, 2, 2, 4))

    def step(q, k, v):
        leaves = [t.detach().requires_grad_() for t in (q, k, v)]
        o = fa.flash_attention_grouped(*fa.rotary_embedding(*leaves[:2], at, plan), leaves[2], cu, 140, causal=True)
        return [o.detach(), *torch.autograd.grad(o, leaves, do)]

    step(q, k, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = step(q, k, v)
    for t in (q, k, v):
        t.copy_(draw(gen, *t.shape))
    at.add_(1000)
    graph.replay()
    want = step(q, k, v)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    for i, (a, b) in enumerate(zip(cap, want)):
        if i == 1:
            assert np.linalg.norm(f64(a) - f64(b)) <= 2.0 ** -8 * np.linalg.norm(f64(b))
        else:
            assert torch.equal(a, b), i


@pytest.mark.parametrize("d,pairs,axes", [(64, 32, 1), (128, 64, 3), (128, 24, 2)])
def test_gradient_against_differences(d, pairs, axes):
    """The turn is linear: <f(x + u) - f(x), w> = <u, f'(w)>, whatever u.  x and u are
    multiples of 2^-3 below 8, so that x + u is exact in bf16.  Each element of the three
    results is off by at most 2^-8 of itself (its rounding) and 2^-20 of its pair's
    magnitudes; no element exceeds its pair's two magnitudes together, so the sides differ
    by at most 2^-7 times the sum of the products of those magnitudes."""
    fa = require_gpu()
    gen = torch.Generator().manual_seed(pairs)
    T, H = 40, 3
    x, u = ((torch.randint(-31, 32, (T, H, d), generator=gen) / 8).bfloat16().cuda() for _ in range(2))
    w = draw(gen, T, H, d)
    at = torch.randint(-9999, 9999, (axes, T), generator=gen).int().cuda()
    plan = plan_of(fa, pairs, axes)
    f = lambda a: f64(fa.rotary_forward(a, a, at, plan)[0])  # noqa: E731
    assert torch.equal((x + u).double(), x.double() + u.double())

    def size(a):  # of the pair that each element is in
        a = np.abs(f64(a))
        a[..., :pairs] = a[..., pairs:2 * pairs] = a[..., :pairs] + a[..., pairs:2 * pairs]
        return a

    left = ((f(x + u) - f(x)) * f64(w)).sum()
    right = (f64(u) * f64(fa.rotary_backward(w, w, at, plan)[0])).sum()
    assert abs(left - right) <= 2.0 ** -7 * (((size(x + u) + size(x)) * np.abs(f64(w))).sum() + (size(w) * np.abs(f64(u))).sum())
    # and u alone, whose difference to zero has no cancellation
    assert abs((f(u) * f64(w)).sum() - right) <= 2.0 ** -7 * ((size(u) * np.abs(f64(w))).sum() + (size(w) * np.abs(f64(u))).sum())


# ---------------------------------------------------------------- ends of the ranges
def test_pages_past_four_gigabytes():
    """The last pages of a cache of 4.6 GB of codes each for K and V: what a small cache
    with the same pages gives, bit for bit."""
    fa = require_gpu()
    pages, Hk, block, d, H = 140000, 2, 128, 128, 8
    cache = fa.cache8_alloc(pages, Hk, block, d)
    assert cache.k.numel() > 2 ** 32
    few = random_cache(fa, 4, Hk, block, d, seed=5)
    for big, part in zip(cache, few):
        bits(big)[-4:] = bits(part)
    gen = torch.Generator().manual_seed(6)
    x, cu, start, plan = draw(gen, 150, H + 2 * Hk, d), i32([0, 150]), i32([300]), plan_of(fa, 64)
    got = []
    for c, first in ((few, 0), (cache, pages - 4)):
        table = i32([[first, first + 1, first + 2, first + 3]])
        q = fa.cache8_store_rotary(x[:, :H], x[:, H:H + Hk], x[:, H + Hk:], c, table, cu, start, 150, plan)
        got.append([q, *fa.attention_chunk_cache8(q, c, table, cu, i32([450]), 150, 450, True)])
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    assert_same(*got)
    assert_same([t[-4:] for t in cache], few)
    assert not bits(cache.k)[:-4].any() and not bits(cache.v)[:-4].any()


def test_more_than_two_to_the_31_elements():
    """q of 2.4e9 elements: turned, and over the cache; the first and the last sequence."""
    fa = require_gpu()
    n, nseq, H, Hk, d, block = 500, 1200, 32, 2, 128, 64
    T, cols = n * nseq, -(-n // block)
    g = torch.Generator(device="cuda").manual_seed(34)
    q, k = (torch.empty(T, h, d, device="cuda", dtype=torch.bfloat16).normal_(generator=g) for h in (H, Hk))
    at, plan = torch.arange(T, **I32) % n, plan_of(fa, 64)
    qt, kt = fa.rotary_forward(q, k, at, plan)
    for a in (0, T - n):
        assert_same((qt[a:a + n], kt[a:a + n]), fa.rotary_forward(q[a:a + n], k[a:a + n], at[a:a + n], plan))
    cache = random_cache(fa, 16, Hk, block, d, seed=35)
    table = (torch.arange(nseq * cols) % 16).reshape(nseq, cols).int()
    cu = torch.arange(0, T + 1, n, **I32)
    o, lse = fa.attention_chunk_cache8(qt, cache, table.cuda(), cu, torch.full((nseq,), n, **I32), n, n, True)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    for b in (0, nseq - 1):
        rows = slice(b * n, b * n + n)
        check(o[rows], lse[:, rows], qt[rows], cache, table[b:b + 1], [n], [n], d ** -0.5, True)


@pytest.mark.parametrize("d,block,n,new", [(64, 64, 2 ** 31 - 1, 1), (128, 128, 2 ** 31 - 130, 2)])
def test_lengths_up_to_the_largest_int(d, block, n, new):
    """A table of 2^31 tokens over eight pages, each shared millions of times.  A CTA's
    run is 2^24 / 152 = 110,377 tiles, every other one of them a half's: 55,189.  A row's
    sum adds one partial sum a tile, of positive terms, in fp32: off by at most 55,189 ·
    2^-24 = 3.3e-3 of itself.  O takes eight steps of 16 keys a tile: 441,512 additions
    of at most 2^-23 of Σ P |v| so far (the tensor core may cut instead of round), 5.3e-2.
    With the rounding of P (2^-8) and of O (2^-8), the scores' 1e-4, and the joining of
    152 parts (2^-16): 5.3e-2 + 2^-7 + 4e-3 of Σ P |v|; 4e-3 of the LSE, whose own
    rounding is 22 · 2^-24."""
    fa = require_gpu()
    pages = 8
    g = torch.Generator(device="cuda").manual_seed(d)
    cache = fa.cache8_alloc(pages, 1, block, d)
    cache.k.copy_(torch.randn(pages, 1, block, d, device="cuda", generator=g))
    cache.v.copy_(torch.randn(pages, 1, block, d, device="cuda", generator=g))
    table = (torch.arange(-(-n // block), **I32) % pages)[None]
    q = torch.randn(new, 1, d, device="cuda", generator=g).bfloat16()
    o, lse = fa.attention_chunk_cache8(q, cache, table, i32([0, new]), i32([n]), new, 2 ** 31 - 1, True)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    k, v = (f64(t).reshape(-1, d) for t in cache[:2])
    for i in range(new):
        count = np.zeros((pages, block))
        full, rest = divmod(n - new + i + 1, block)
        count += np.bincount(np.arange(full % pages), minlength=pages)[:, None] + full // pages
        count[full % pages, :rest] += 1
        p = count.reshape(-1) * np.exp(d ** -0.5 * k @ f64(q)[i, 0])
        assert abs(f64(lse)[0, i] - np.log(p.sum())) <= 4e-3
        p /= p.sum()
        assert (np.abs(f64(o)[i, 0] - p @ v) <= (5.3e-2 + 2.0 ** -7 + 4e-3) * (p @ np.abs(v))).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,lens", [([200, 3], [300, 900]), ([40], [30000]), ([300], [30000])])
def test_infinite_and_nan_queries_stay_in_their_rows(new, lens, d):
    """Rows with an infinity or NaN become NaN, whole items and those that many CTAs share
    alike; the others are as the formula has them, and a row that sees no key is empty."""
    fa = require_gpu()
    H, Hk, block, T = 6, 2, 64, sum(new)
    cols = -(-max(lens) // block)
    B = len(new)
    cache = random_cache(fa, B * cols, Hk, block, d, seed=d)
    table = make_table(B * cols, B, cols, 8)
    q = draw(torch.Generator().manual_seed(d), T, H, d)
    bad = torch.zeros(T, H, dtype=torch.bool, device="cuda")
    for i, (tok, h, x) in enumerate(((0, 0, np.nan), (3, 2, np.inf), (17, 5, -np.inf), (T - 1, 3, np.nan))):
        q[tok, h, 11 * i] = x
        bad[tok, h] = True
    cu = i32([0] + np.cumsum(new).tolist())
    o, lse = fa.attention_chunk_cache8(q, cache, table.cuda(), cu, i32(lens), max(new), max(lens), True)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    assert torch.isnan(o[bad]).all() and torch.isnan(lse.T[bad]).all()
    clean = q.clone()
    clean[bad] = 0  # (these rows' results are of their own)
    want, want_lse = fa.attention_chunk_cache8(clean, cache, table.cuda(), cu, i32(lens), max(new), max(lens), True)
    o, lse = torch.where(bad[..., None], want, o), torch.where(bad.T, want_lse, lse)
    check(o, lse, clean, cache, table, new, lens, d ** -0.5, True)
    # no key to see: empty all the same
    o, lse = fa.attention_chunk_cache8(q[:20], cache, table.cuda()[:1], i32([0, 20]), i32([0]), 20, 10, True)
    torch.cuda.synchronize()
    assert not o.any() and (lse == -np.inf).all()


def test_capacities_far_above_what_is_there():
    """max_new and max_seqlen are upper limits: the largest int gives what the tight ones do."""
    fa = require_gpu()
    x, cu, start = draw(torch.Generator().manual_seed(12), 150, 12, 64), i32([0, 30, 150]), i32([0, 33])
    table, plan = i32([[0, 1, 2, 3, 4], [5, 6, 7, 8, 9]]), plan_of(fa, 32)
    first = random_cache(fa, 10, 2, 32, 64, seed=13)
    got = []
    for max_new, max_seqlen in ((120, 153), (2 ** 31 - 1, 2 ** 31 - 1)):
        cache = fa.Cache8(*[t.clone() for t in first])
        q = fa.cache8_store_rotary(x[:, :8], x[:, 8:10], x[:, 10:], cache, table, cu, start, max_new, plan)
        got.append([q, *cache, *fa.attention_chunk_cache8(q, cache, table, cu, i32([30, 153]), max_new, max_seqlen, True)])
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    o = [g.pop(-2) for g in got]  # (tiles may be shared out otherwise: two of the formula's tolerances)
    lse = [g.pop(-1) for g in got]
    assert_same(*got)
    vmax = float((got[0][2].float() * got[0][4][..., None, None]).abs().max())
    assert float((o[0] - o[1]).abs().max()) <= 2.0 ** -6 * vmax and float((lse[0] - lse[1]).abs().max()) <= 2e-4
