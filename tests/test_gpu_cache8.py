"""The 8-bit paged cache: storing against the definition in 64 bits (codes and
scales equal, not near), attention over it against the formula in 64 bits on
the stored values, indexes out of range, and prompts, stores and decoding steps
together.

Tolerances of the attention.  The cache's values are the inputs, so the
quantisation is no error.  A probability is split into two e4m3 factors with 8
significant bits together (at most 2^-9 of it is lost), so sum P_j |v_j| moves
by at most 2^-9 max|v|; the output's rounding to bf16 adds 2^-8 |O|: held to
2^-7 max|v|.  LSE: fp32 sums of fp32 exponentials, the query exact to 2^-24 of
its largest element over d terms; held to 1e-4 for scores of order 1, and to that
times the largest score S where it is larger: d <= 128 products summed in fp32
are off by at most 128 · 2^-24 S = 7.7e-6 S, the LSE's own rounding adds
2^-24 S.
"""
import numpy as np
import pytest
import torch

from tests.gpu_util import assert_no_device_error, f64, gpu, require_gpu

pytestmark = gpu

FLOOR = -64
LSE_TOL = 1e-4
ERR_PAGE = 12


# ---------------------------------------------------------------- the definition
def e4m3(x):
    """Nearest e4m3 value (ties to even), saturating; x in 64 bits."""
    a = np.abs(x)
    _, e = np.frexp(np.where(np.isfinite(a), a, 1.0))
    step = np.exp2(np.maximum(e - 4, -9).astype(np.float64))
    with np.errstate(invalid="ignore"):
        r = np.minimum(np.round(a / step) * step, 448.0)
    return np.copysign(r, x)


def needed_scale(x):
    a = np.abs(x[np.isfinite(x)])
    m = a.max() if a.size else 0.0
    if m == 0:
        return 2.0 ** FLOOR
    half, e = np.frexp(m / 448.0)
    return 2.0 ** max(int(e) - (half == 0.5), FLOOR)


def store_formula(x, codes, scale, table, cu, start):
    """x [T, Hk, d] into codes [pages, Hk, block, d] (values) and scale, in place."""
    block = codes.shape[2]
    for b in range(len(start)):
        n = cu[b + 1] - cu[b]
        for j in range(start[b] // block, -(-(start[b] + n) // block) if n else 0):
            lo, hi = max(start[b], j * block), min(start[b] + n, (j + 1) * block)
            page, old = table[b][j], max(0, start[b] - j * block)
            for h in range(x.shape[1]):
                new = x[cu[b] + lo - start[b]:cu[b] + hi - start[b], h]
                s = needed_scale(new)
                if old:
                    s = max(s, scale[page, h])
                    codes[page, h, :old] = e4m3(codes[page, h, :old] * scale[page, h] / s)
                codes[page, h, lo - j * block:hi - j * block] = e4m3(new / s)
                scale[page, h] = s


def attend_formula(q, cache, table, lens, scale, causal):
    k, v, ks, vs = cache
    B, Nq, H, d = q.shape
    Hk, block = k.shape[1:3]
    o, lse = np.zeros(q.shape), np.full((B, H, Nq), -np.inf)
    vmax = 0.0
    for b in range(B):
        n = int(lens[b])
        if not n:
            continue
        pages = table[b][:-(-n // block)]
        kk, vv = ((c[pages] * s[pages][..., None, None]).transpose(1, 0, 2, 3).reshape(Hk, -1, d)[:, :n]
                  for c, s in ((k, ks), (v, vs)))
        vmax = max(vmax, np.abs(vv).max())
        for h in range(H):
            s = scale * q[b, :, h] @ kk[h // (H // Hk)].T
            if causal:
                s = np.where(np.arange(n)[None] > n - Nq + np.arange(Nq)[:, None], -np.inf, s)
            live = np.isfinite(s.max(1))
            s = s[live]
            m = s.max(1, keepdims=True)
            e = np.exp(s - m)
            l = e.sum(1, keepdims=True)
            lse[b, h, live] = (m + np.log(l))[:, 0]
            o[b, live, h] = e / l @ vv[h // (H // Hk)]
    return o, lse, vmax


def values(cache):
    return [f64(t) for t in cache]


def make_table(pages, rows, cols, seed):
    """Distinct pages anywhere in the pool; -1 is never read."""
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))[:rows * cols]
    return order.reshape(rows, cols).to(torch.int32)


def random_cache(fa, pages, Hk, block, d, seed, spread=0.5):
    """A pool of filled pages, uneven scales among them."""
    gen = torch.Generator().manual_seed(seed)
    cache = fa.cache8_alloc(pages, Hk, block, d)
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = torch.randn(pages, Hk, block, d, generator=gen) * torch.exp(spread * torch.randn(pages, Hk, 1, 1, generator=gen))
        want = torch.tensor([[needed_scale(x[i, h].double().numpy()) for h in range(Hk)] for i in range(pages)])
        c.copy_((x / want[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn))
        s.copy_(want)
    return cache


def bits(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


# ---------------------------------------------------------------- store
def run_store(fa, x, cache, table, cu, start, max_new, ref, **kw):
    kd, vd = (t.cuda() for t in x) if not x[0].is_cuda else x
    fa.cache8_store(kd, vd, cache, table.cuda(), torch.tensor(cu, dtype=torch.int32, device="cuda"),
                    torch.tensor(start, dtype=torch.int32, device="cuda"), max_new, **kw)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    for t, c, s in zip(x, (0, 1), (2, 3)):
        store_formula(f64(t), ref[c], ref[s], table.tolist(), cu, start)
    for got, want in zip(values(cache), ref):
        assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hk", [1, 3])
def test_store_ragged(Hk, d, block):
    fa = require_gpu()
    lens, start = [1, 0, 5, block, 2 * block + 3, 1, 33, 7], [0, 9, 3, 0, block - 1, block, 2 * block + 5, block - 7]
    cols = max(-(-(a + n) // block) for a, n in zip(start, lens))
    pages = len(lens) * cols + 2
    cache = random_cache(fa, pages, Hk, block, d, seed=block + d)
    ref = values(cache)
    cu = [0] + np.cumsum(lens).tolist()
    gen = torch.Generator().manual_seed(1)
    # magnitudes from token to token, so that held pages are rounded again and others are not
    x = [(torch.randn(cu[-1], Hk, d, generator=gen) * torch.exp(2 * torch.randn(cu[-1], 1, 1, generator=gen))).bfloat16()
         for _ in range(2)]
    run_store(fa, x, cache, make_table(pages, len(lens), cols, 2), cu, start, max(lens), ref)


@pytest.mark.parametrize("block", [16, 128])
def test_store_token_by_token(block):
    """300 single tokens of two sequences, of growing and shrinking size."""
    fa = require_gpu()
    cols = -(-300 // block)
    cache = random_cache(fa, 2 * cols + 1, 2, block, 64, seed=3)
    ref = values(cache)
    table = make_table(2 * cols + 1, 2, cols, 4)
    gen = torch.Generator().manual_seed(5)
    table_d, cu = table.cuda(), torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    for t in range(300):
        x = [(torch.randn(2, 2, 64, generator=gen) * 2.0 ** ((t * 7) % 23 - 11)).bfloat16() for _ in range(2)]
        fa.cache8_store(x[0].cuda(), x[1].cuda(), cache, table_d, cu, torch.tensor([t, t], dtype=torch.int32, device="cuda"), 1)
        for i in (0, 1):
            store_formula(f64(x[i]), ref[i], ref[2 + i], table.tolist(), [0, 1, 2], [t, t])
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    for got, want in zip(values(cache), ref):
        assert np.array_equal(got, want)


def test_store_borders_of_the_scale_and_of_the_codes():
    fa = require_gpu()
    block, d = 16, 64
    rows = []
    for top in (448.0, 450.0, 446.0, 1.75, 1.7578125, 2.0 ** -70, 2.0 ** -56, 3.3e38, 2.0 ** 127, 0.0):
        x = torch.zeros(block, 1, d)
        x[0, 0, 0] = top
        # ties, steps below the normal codes, and what rounds to zero
        steps = torch.cat([torch.arange(1, 33) / 16, 2.0 ** -torch.arange(0.0, 30.0)])
        x[1, 0, :62] = top / 448 * steps
        x[2, 0] = -top * torch.rand(d, generator=torch.Generator().manual_seed(7))
        rows.append(x)
    x = torch.cat(rows).bfloat16()
    n = len(rows)
    cache = fa.cache8_alloc(n, 1, block, d)
    run_store(fa, [x, x.clone()], cache, torch.arange(n, dtype=torch.int32)[:, None], [i * block for i in range(n + 1)],
              [0] * n, block, values(cache))


def test_store_infinities_and_nan():
    fa = require_gpu()
    x = torch.randn(16, 1, 64).bfloat16()
    x[3, 0, 5], x[4, 0, 6], x[5, 0, 7] = float("inf"), float("-inf"), float("nan")
    cache = fa.cache8_alloc(1, 1, 16, 64)
    run_store(fa, [x, x.clone()], cache, torch.zeros(1, 1, dtype=torch.int32), [0, 16], [0], 16, values(cache))
    assert f64(cache.k)[0, 0, 3, 5] == 448 and f64(cache.k)[0, 0, 4, 6] == -448 and np.isnan(f64(cache.k)[0, 0, 5, 7])


def test_store_slices_stream_and_graph():
    fa = require_gpu()
    Hk, d, block = 2, 128, 32
    gen = torch.Generator().manual_seed(8)
    qkv = torch.randn(50, 3 * Hk, d, generator=gen).bfloat16().cuda()
    k, v = qkv[:, Hk:2 * Hk], qkv[:, 2 * Hk:]
    table, cu, start = make_table(8, 2, 4, 9), [0, 20, 50], [5, 0]
    cache = random_cache(fa, 8, Hk, block, d, seed=10)
    before = [t.clone() for t in cache]
    run_store(fa, [k, v], cache, table, cu, start, 30, values(cache))
    args = (table.cuda(), torch.tensor(cu, dtype=torch.int32, device="cuda"), torch.tensor(start, dtype=torch.int32, device="cuda"), 30)
    other, captured = (fa.Cache8(*(t.clone() for t in before)) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fa.cache8_store(k, v, other, *args, stream=side)
    graph = torch.cuda.CUDAGraph()
    side.synchronize()
    with torch.cuda.graph(graph):
        fa.cache8_store(k, v, captured, *args)
    graph.replay()
    graph.replay()  # storing the same tokens again changes nothing
    torch.cuda.synchronize()
    for a, b, c in zip(cache, other, captured):
        assert torch.equal(bits(a), bits(b)) and torch.equal(bits(a), bits(c))


def test_store_indexes_out_of_range_touch_nothing():
    fa = require_gpu()
    cache = random_cache(fa, 4, 1, 16, 64, seed=11)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.randn(20, 1, 64).bfloat16().cuda()
    for table, cu, start in (([[-1]], [0, 5], [0]), ([[4]], [0, 5], [3]), ([[2 ** 31 - 1]], [0, 5], [0]),
                             ([[0]], [0, 5], [16]), ([[0]], [0, 5], [2 ** 31 - 1]), ([[0]], [0, 5], [-1])):
        before = [t.clone() for t in cache]
        fa.cache8_store(x, x, cache, i32(table), i32(cu), i32(start), 5)
        assert fa.fa_get_device_error() == ERR_PAGE
        for a, b in zip(before, cache):
            assert torch.equal(bits(a), bits(b))
    # rows that do not exist are not read, tokens past max_new are dropped
    ref = values(cache)
    fa.cache8_store(x, x, cache, i32([[0, 1]]), i32([0, 400]), i32([0]), 18)
    assert_no_device_error(fa)
    for c, s in ((0, 2), (1, 3)):
        store_formula(f64(x)[:18], ref[c], ref[s], [[0, 1]], [0, 18], [0])
    for got, want in zip(values(cache), ref):
        assert np.array_equal(got, want)
    assert fa.fa_get_device_error() == 0


# ---------------------------------------------------------------- attention
def poison(cache, table, lens):
    """NaN codes in every slot that no token holds, NaN scales in unused pages."""
    block = cache.k.shape[2]
    used = set()
    for b, n in enumerate(lens):
        for j in range(-(-n // block)):
            page = int(table[b, j])
            used.add(page)
            rest = n - j * block
            if rest < block:
                for c in cache[:2]:
                    c.view(torch.uint8)[page, :, rest:] = 0x7F
    for page in range(cache.k.shape[0]):
        if page not in used:
            for c in cache[:2]:
                c.view(torch.uint8)[page] = 0x7F
            cache.k_scale[page] = cache.v_scale[page] = float("nan")


def check_attend(fa, H, Hk, d, block, lens, Nq, causal, seed, max_seqlen=None, cache=None, amplitude=1.0, scale=None):
    B, cols = len(lens), max(1, max(-(-n // block) for n in lens))
    pages = B * cols + 1
    cache = random_cache(fa, pages, Hk, block, d, seed) if cache is None else cache
    table = make_table(pages, B, cols, seed)
    poison(cache, table, lens)
    for b, n in enumerate(lens):
        table[b, -(-n // block):] = -7  # entries behind the last token are never read
    q = (torch.randn(B, Nq, H, d, generator=torch.Generator().manual_seed(seed)) * amplitude).bfloat16()
    scale = d ** -0.5 if scale is None else scale
    o, lse = fa.attention_decode_cache8(q.cuda(), cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                        max(lens) if max_seqlen is None else max_seqlen, causal, scale)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    O, L, vmax = attend_formula(f64(q), values(cache), table.numpy(), lens, scale, causal)
    assert np.isfinite(f64(o)).all()
    assert np.abs(f64(o) - O).max() <= 2.0 ** -7 * vmax
    seen = np.isfinite(L)
    got = f64(lse)
    assert np.array_equal(np.isfinite(got), seen) and (got[~seen] == -np.inf).all()
    assert not f64(o).transpose(0, 2, 1, 3)[~seen].any()
    big = max(1.0, np.abs(L[seen]).max()) if seen.any() else 1.0
    assert not seen.any() or np.abs(got[seen] - L[seen]).max() <= LSE_TOL * big
    return o, lse


LENS = [1, 0, 127, 128, 129, 17, 300, 1000, 15, 640]


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_attend_ragged(d, block):
    fa = require_gpu()
    check_attend(fa, 8, 2, d, block, LENS, 1, True, seed=d + block)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (2, 2), (6, 3), (3, 1), (14, 2), (8, 1), (16, 1), (40, 2), (71, 1)])
def test_attend_heads(H, Hk, d):
    fa = require_gpu()
    check_attend(fa, H, Hk, d, 32, [5, 200, 333], 1, False, seed=H)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [2, 3, 4, 5, 8])
def test_attend_several_tokens(Nq, d, causal):
    """Sequences shorter than the new tokens leave rows that see nothing."""
    fa = require_gpu()
    check_attend(fa, 8, 2, d, 16, [1, 0, 3, 128, 130, 257, 700], Nq, causal, seed=Nq)


def test_attend_many_sequences_and_empty_batch():
    fa = require_gpu()
    check_attend(fa, 4, 1, 64, 16, [(i * 37) % 90 for i in range(700)], 1, True, seed=12)
    check_attend(fa, 4, 1, 128, 16, [0, 0, 0], 1, True, seed=13, max_seqlen=50)


@pytest.mark.parametrize("d", [64, 128])
def test_attend_long_sequences(d):
    """Items that many CTAs share, and items that one CTA runs through."""
    fa = require_gpu()
    check_attend(fa, 4, 2, d, 128, [20000], 1, True, seed=14)
    check_attend(fa, 2, 1, d, 64, [9000, 130, 40, 5000, 77], 1, True, seed=15, max_seqlen=10000)


@pytest.mark.parametrize("d", [64, 128])
def test_attend_very_long_sequence(d):
    """300,001 tokens whose weight lies on the first one and, as small parts, on
    all others: what a running maximum would lose must still count."""
    fa = require_gpu()
    n, block = 300001, 128
    pages = -(-n // block)
    g = torch.Generator(device="cuda").manual_seed(34)
    cache = fa.cache8_alloc(pages, 1, block, d)
    cache.k.copy_(torch.randn(pages, 1, block, d, device="cuda", generator=g) * 0.02)
    cache.v.copy_(torch.randn(pages, 1, block, d, device="cuda", generator=g) + 1.0)
    q = torch.randn(1, 1, 4, d, device="cuda", generator=g).bfloat16()
    scale = d ** -0.5
    first = q[0, 0, 0].double() / (q[0, 0, 0].double().square().sum() * scale)
    cache.k[0, 0, 0] = (first * 12.0).to(torch.float8_e4m3fn)  # a score near 12: e^12 against 300,000
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    o, lse = fa.attention_decode_cache8(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), n, True)
    k, v = (t.reshape(-1, d)[:n].double() for t in cache[:2])
    s = scale * q[0, 0].double() @ k.T
    want = torch.softmax(s, 1) @ v
    assert_no_device_error(fa)
    # values near 1 of one sign: what of the tail's weight is lost shows in full
    assert (o[0, 0].double() - want).abs().max() <= 2.0 ** -7 * want.abs().max()
    assert (lse[0, :, 0].double() - torch.logsumexp(s, 1)).abs().max() <= LSE_TOL * 15


def test_attend_uneven_scales_and_peaked_scores():
    """V scales 2^40 apart from page to page; scores of which one key takes all,
    found late; scores that fall and rise by hundreds."""
    fa = require_gpu()
    for d in (64, 128):
        cache = random_cache(fa, 40, 1, 16, d, seed=16)
        f = 2.0 ** (torch.arange(40) % 5 * 10.0 - 20)
        cache.v_scale.mul_(f[:, None].cuda())
        check_attend(fa, 4, 1, d, 16, [600], 1, True, seed=17, cache=cache)
        check_attend(fa, 4, 1, d, 16, [2000, 513], 1, True, seed=18, amplitude=30.0)
        cache = random_cache(fa, 130, 1, 16, d, seed=19)
        cache.k_scale.mul_(2.0 ** (torch.arange(130, device="cuda") % 7 - 3.0)[:, None])
        check_attend(fa, 8, 1, d, 16, [2000], 1, False, seed=20, cache=cache, amplitude=8.0)


def test_attend_small_query_elements_count():
    """Queries whose elements span many powers of two: the split keeps the small ones."""
    fa = require_gpu()
    d, n = 128, 400
    cache = random_cache(fa, 30, 1, 16, d, seed=21)
    q = torch.randn(1, 1, 4, d) * torch.exp2(-torch.arange(d) % 16.0)
    q = q.bfloat16()
    table = torch.arange(25, dtype=torch.int32)[None]
    o, lse = fa.attention_decode_cache8(q.cuda(), cache, table.cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), n)
    O, L, vmax = attend_formula(f64(q), values(cache), table.numpy(), [n], d ** -0.5, False)
    # the LSE here is the largest score, some 5e4: the header's bound
    assert np.abs(f64(o) - O).max() <= 2.0 ** -7 * vmax and np.abs(f64(lse) - L).max() <= LSE_TOL * np.abs(L).max()
    assert_no_device_error(fa)


def test_attend_shared_pages():
    """Two sequences with a common beginning in the same pages."""
    fa = require_gpu()
    cache = random_cache(fa, 12, 2, 32, 128, seed=22)
    table = torch.tensor([[3, 4, 5, 6], [3, 4, 9, 1]], dtype=torch.int32)
    q = torch.randn(2, 1, 4, 128).bfloat16()
    lens = [110, 70]
    o, lse = fa.attention_decode_cache8(q.cuda(), cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), 110)
    O, L, vmax = attend_formula(f64(q), values(cache), table.numpy(), lens, 128 ** -0.5, False)
    assert np.abs(f64(o) - O).max() <= 2.0 ** -7 * vmax and np.abs(f64(lse) - L).max() <= LSE_TOL


def test_attend_indexes_out_of_range():
    """A page out of range reads as zeros, a length out of range is clamped; both are reported."""
    fa = require_gpu()
    for d in (64, 128):
        cache = random_cache(fa, 6, 1, 16, d, seed=23)
        q = torch.randn(1, 1, 2, d).bfloat16()
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        for bad in (-1, 6, 2 ** 31 - 1, -2 ** 31):
            o, lse = fa.attention_decode_cache8(q.cuda(), cache, i32([[0, bad, 2]]), i32([40]), 48)
            assert fa.fa_get_device_error() == ERR_PAGE
            k, v, ks, vs = (np.concatenate([t, np.zeros_like(t[:1])]) for t in values(cache))
            O, L, vmax = attend_formula(f64(q), (k, v, ks, vs), np.array([[0, 6, 2]]), [40], d ** -0.5, False)
            assert np.abs(f64(o) - O).max() <= 2.0 ** -7 * vmax and np.abs(f64(lse) - L).max() <= LSE_TOL
        for n, held in ((-3, 0), (1000, 48), (2 ** 31 - 1, 48)):
            o, lse = fa.attention_decode_cache8(q.cuda(), cache, i32([[0, 1, 2]]), i32([n]), 48)
            assert fa.fa_get_device_error() == ERR_PAGE
            O, L, vmax = attend_formula(f64(q), values(cache), np.array([[0, 1, 2]]), [held], d ** -0.5, False)
            assert np.abs(f64(o) - O).max() <= 2.0 ** -7 * vmax
            assert (f64(lse) == -np.inf).all() if not held else np.abs(f64(lse) - L).max() <= LSE_TOL


@pytest.mark.parametrize("d", [64, 128])
def test_attend_repeatable_streams_and_graph(d):
    fa = require_gpu()
    H, Hk, block, lens = 8, 2, 32, [3000, 5, 700]
    cols = -(-max(lens) // block)
    cache = random_cache(fa, 3 * cols, Hk, block, d, seed=24)
    table = make_table(3 * cols, 3, cols, 25).cuda()
    q = torch.randn(3, 1, H, d).bfloat16().cuda()
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    f = lambda **kw: fa.attention_decode_cache8(q, cache, table, n, 3200, True, **kw)  # noqa: E731
    size = fa.fa_decode_cache8_workspace_bytes(3, 1, H, Hk, 3200, d)
    ws = [torch.full((size,), fill, dtype=torch.uint8, device="cuda") for fill in (0xFF, 0x7F)]
    want = f()
    assert all(torch.equal(a, b) for a, b in zip(want, f(workspace=ws[0])))
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):  # two calls at once, each with a workspace of its own
        for side, w in zip(sides, ws):
            side.wait_stream(torch.cuda.current_stream())
            got.append(f(stream=side, workspace=w))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(want, g))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = f()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, cap))
    # other lengths in the captured buffers; 3100 is past the page table's end
    for new, error in (([12, 3100, 0], ERR_PAGE), ([12, cols * block, 0], 0)):
        n.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        want = f()
        torch.cuda.synchronize()
        assert fa.fa_get_device_error() == error
        assert all(torch.equal(a, b) for a, b in zip(want, cap))


def test_cache_past_four_gigabytes():
    """Pages whose bytes lie past 2^32 in the pool, stored and attended to."""
    fa = require_gpu()
    Hk, block, d, n = 8, 128, 128, 300
    pages = 2 ** 32 // (Hk * block * d) + 40
    cache = fa.cache8_alloc(pages, Hk, block, d)
    table = torch.tensor([[pages - 1, 5, pages - 7]], dtype=torch.int32)
    gen = torch.Generator().manual_seed(28)
    k, v = (torch.randn(n, Hk, d, generator=gen).bfloat16() for _ in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    fa.cache8_store(k.cuda(), v.cuda(), cache, table.cuda(), i32([0, n]), i32([0]), n)
    q = torch.randn(1, 1, 16, d, generator=gen).bfloat16()
    o, lse = fa.attention_decode_cache8(q.cuda(), cache, table.cuda(), i32([n]), n)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    used = table[0].long()
    ref = [np.zeros((3, Hk, block, d)), np.zeros((3, Hk, block, d)), np.ones((3, Hk)), np.ones((3, Hk))]
    for x, c, s in ((k, 0, 2), (v, 1, 3)):
        store_formula(f64(x), ref[c], ref[s], [[0, 1, 2]], [0, n], [0])
    for t, want in zip(cache, ref):
        assert np.array_equal(f64(t.view(torch.uint8)[used.cuda()].view(t.dtype) if t.dtype != torch.float32 else t[used.cuda()]), want)
    O, L, vmax = attend_formula(f64(q), ref, np.array([[0, 1, 2]]), [n], d ** -0.5, False)
    assert np.abs(f64(o) - O).max() <= 2.0 ** -7 * vmax and np.abs(f64(lse) - L).max() <= LSE_TOL


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("d,block", [(64, 16), (128, 64)])
def test_prompt_store_and_decoding_steps(d, block):
    """Prompts through the packed attention, their keys and values into the
    cache, then single tokens and two at once, as a serving loop runs them."""
    fa = require_gpu()
    H, Hk, prompts, steps = 8, 2, [70, 1, 200], [1, 1, 2, 1]
    gen = torch.Generator().manual_seed(26)
    B, cols = len(prompts), -(-(max(prompts) + sum(steps)) // block)
    cache = fa.cache8_alloc(B * cols, Hk, block, d)
    ref = values(cache)
    table = make_table(B * cols, B, cols, 27)
    table_d = table.cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    held = [0] * B
    for n_new in [None] + steps:
        new = prompts if n_new is None else [n_new] * B
        cu = [0] + np.cumsum(new).tolist()
        qkv = torch.randn(cu[-1], H + 2 * Hk, d, generator=gen).bfloat16()
        dev = qkv.cuda()
        q, k, v = dev[:, :H], dev[:, H:H + Hk], dev[:, H + Hk:]
        if n_new is None:
            o, _ = fa.attention_forward_grouped(q, k, v, i32(cu), max(new), causal=True)
            for b in range(B):
                s = np.einsum("ihd,jhd->hij", f64(q[cu[b]:cu[b + 1]]), f64(k[cu[b]:cu[b + 1]]).repeat(H // Hk, 1)) * d ** -0.5
                s[:, np.triu(np.ones(s.shape[1:], bool), 1)] = -np.inf
                p = np.exp(s - s.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                want = np.einsum("hij,jhd->ihd", p, f64(v[cu[b]:cu[b + 1]]).repeat(H // Hk, 1))
                assert np.abs(f64(o[cu[b]:cu[b + 1]]) - want).max() <= 2.0 ** -7 * np.abs(f64(v)).max()
        fa.cache8_store(k, v, cache, table_d, i32(cu), i32(held), max(new))
        for i, x in ((0, k), (1, v)):
            store_formula(f64(x), ref[i], ref[2 + i], table.tolist(), cu, held)
        held = [a + n for a, n in zip(held, new)]
        if n_new is not None:
            qd = q.reshape(B, n_new, H, d).contiguous()
            o, lse = fa.attention_decode_cache8(qd, cache, table_d, i32(held), max(held), causal=True)
            O, L, vmax = attend_formula(f64(qd), ref, table.numpy(), held, d ** -0.5, True)
            assert np.abs(f64(o) - O).max() <= 2.0 ** -7 * vmax and np.abs(f64(lse) - L).max() <= LSE_TOL
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    for got, want in zip(values(cache), ref):
        assert np.array_equal(got, want)


def test_refusals():
    fa = require_gpu()
    cache = fa.cache8_alloc(4, 2, 16, 64)
    q, k = torch.randn(1, 1, 4, 64).bfloat16().cuda(), torch.randn(3, 2, 64).bfloat16().cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table, n = i32([[0, 1]]), i32([20])
    f = fa.attention_decode_cache8
    for bad in ((q.float(), cache, table, n), (q, cache._replace(k=cache.k.view(torch.uint8)), table, n)):
        with pytest.raises(TypeError):
            f(*bad, 20)
    for bad in ((q, cache, table.long(), n), (q, cache, table, n.long()), (q, cache._replace(v=cache.v[:3]), table, n),
                (q, cache._replace(k_scale=cache.k_scale.double()), table, n), (q, cache, table, i32([20, 20])),
                (q[..., :32].contiguous(), cache, table, n), (q, cache, table.cpu(), n)):
        with pytest.raises(ValueError):
            f(*bad, 20)
    for bad in ((q[:, :, :3].contiguous(), 20, None), (q, 0, None), (q, 20, -1.0), (q.expand(1, 9, 4, 64).contiguous(), 20, None)):
        with pytest.raises(fa.FaError):
            f(bad[0], cache, table, n, bad[1], scale=bad[2])
    with pytest.raises(fa.FaError):
        f(q, cache, table, n, 20, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fa.FaError):
        f(q, fa.cache8_alloc(4, 2, 24, 64), table, n, 20)
    s = fa.cache8_store
    cu, start = i32([0, 3]), i32([0])
    for bad in ((k[:, :1], k, cu, start), (k, k[:2], cu, start), (k, k, i32([0, 3, 3]), start), (k, k, cu, start.long())):
        with pytest.raises(ValueError):
            s(bad[0], bad[1], cache, table, bad[2], bad[3], 3)
    with pytest.raises(fa.FaError):
        s(k, k, cache, table, cu, start, 0)
    torch.cuda.synchronize()
    assert_no_device_error(fa)


def test_compiled_and_python_calls_agree():
    fa = require_gpu()
    from io_aware_attention_flash_gb300 import _binding
    n = _binding.native()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    caches = [random_cache(fa, 6, 2, 16, 64, seed=29) for _ in range(2)]
    k, v = (torch.randn(20, 2, 64).bfloat16().cuda() for _ in range(2))
    table, cu, start = i32([[0, 1, 2], [3, 4, 5]]), i32([0, 5, 20]), i32([7, 2])
    assert n.cache8_store(k, v, caches[0], table, cu, start, 15) is True
    fa.fa_cache8_store(k, v, caches[1], table, cu, start, 15)
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(*caches))
    q, lens = torch.randn(2, 1, 6, 64).bfloat16().cuda(), i32([12, 17])
    got = n.decode_cache8(q, caches[0], table, lens, 48, True, None)
    ws = torch.empty(fa.fa_decode_cache8_workspace_bytes(2, 1, 6, 2, 48, 64), dtype=torch.uint8, device="cuda")
    want = fa.attention_decode_cache8(q, caches[0], table, lens, 48, True, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for bad in ((q.float(), caches[0], table, lens, 48, True, None), (q, caches[0][:3], table, lens, 48, True, None),
                (q, caches[0], table[:1], lens, 48, True, None), (q, caches[0], table, lens, -1, True, None),
                (q, caches[0], table, lens.long(), 48, True, None), (q, caches[0], table, lens, 48, True, 0.0)):
        assert n.decode_cache8(*bad) is None
    assert n.cache8_store(k, v[:3], caches[0], table, cu, start, 15) is None
    with pytest.raises(ValueError):
        fa.cache8_store(k, v, caches[0], table, cu, start, 2 ** 32 + 1)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
