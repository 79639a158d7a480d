"""The 8-bit cache's attention at the ends of its ranges, against the formula in
64 bits."""
import numpy as np
import pytest
import torch

from tests.gpu_util import assert_no_device_error, f64, gpu, require_gpu
from tests.test_gpu_cache8 import check_attend

pytestmark = gpu


@pytest.mark.parametrize("d,block,n", [(64, 64, 2 ** 31 - 1), (128, 128, 2 ** 31 - 1), (128, 128, 2 ** 31 - 130)])
def test_lengths_up_to_the_largest_int(d, block, n):
    """A table of 2^31 tokens over eight pages, each shared millions of times.
    Every term of a sum is one of 8 · block values, repeated.  A CTA adds 2^31 / 304
    tokens, a thread of it (128 rows) at most 2^31 / 304 / 128 = 55,189 of them in
    fp32: the sum of weights, of positive terms, is off by at most 55,189 · 2^-24 =
    3.3e-3 of itself, and so is O of Σ P |v| by its own sum over 2^31 / 304 / 128
    tiles (one term a tile); the joining of 304 parts adds 2^-16.  With the
    rounding of P (2^-9) and of O (2^-8) that is 2^-7 + 7e-3 of Σ P |v|, and 4e-3 of
    the LSE (plus 2^-24 of it, 22, for its own rounding)."""
    fa = require_gpu()
    pages = 8
    g = torch.Generator(device="cuda").manual_seed(d + n % 1000)
    cache = fa.cache8_alloc(pages, 1, block, d)
    cache.k.copy_(torch.randn(pages, 1, block, d, device="cuda", generator=g))
    cache.v.copy_(torch.randn(pages, 1, block, d, device="cuda", generator=g))
    cols = -(-n // block)
    table = (torch.arange(cols, device="cuda", dtype=torch.int32) % pages)[None]
    q = torch.randn(1, 1, 1, d, device="cuda", generator=g).bfloat16()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    o, lse = fa.attention_decode_cache8(q, cache, table, lens, 2 ** 31 - 1, True)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    count = np.zeros((pages, block))
    full, rest = divmod(n, block)
    count += np.bincount(np.arange(full % pages), minlength=pages)[:, None] + full // pages
    count[full % pages, :rest] += 1
    k, v = (f64(t).reshape(-1, d) for t in cache[:2])
    s = d ** -0.5 * k @ f64(q)[0, 0, 0]
    p = count.reshape(-1) * np.exp(s)
    assert abs(f64(lse)[0, 0, 0] - np.log(p.sum())) <= 4e-3
    p /= p.sum()
    assert (np.abs(f64(o)[0, 0, 0] - p @ v) <= (2.0 ** -7 + 7e-3) * (p @ np.abs(v))).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_exp,k_exp", [(110, -60), (125, -70), (-100, 60), (-115, 90), (-60, 30), (0, 0)])
def test_queries_of_any_size(q_exp, k_exp, d):
    """Queries up to bf16's largest and down to its smallest normal numbers, over
    keys (by their scales) and a softmax scale that make the scores of order 1.  A
    query element is off by at most 2^-17 of its row's largest (half of e4m3's least
    step, 2^-10, where the largest is at least 224), so a score by
    e = scale 2^-17 max|q| max_j Σ|k_j|, the LSE by e and P by 2e of itself; the
    rest as everywhere: 2^-7 Σ P |v| for O, 1e-4 for the LSE."""
    fa = require_gpu()
    H, Hk, block, n = 8, 2, 16, 300
    pages = -(-n // block)
    g = torch.Generator(device="cuda").manual_seed(q_exp + 200)
    cache = fa.cache8_alloc(pages, Hk, block, d)
    cache.k.copy_(torch.randn(pages, Hk, block, d, device="cuda", generator=g))
    cache.v.copy_(torch.randn(pages, Hk, block, d, device="cuda", generator=g))
    cache.k_scale.fill_(2.0 ** k_exp)
    table = torch.arange(pages, device="cuda", dtype=torch.int32)[None]
    # (2^q_exp in two steps: neither factor leaves fp32)
    q = (torch.randn(1, 2, H, d, device="cuda", generator=g) * 2.0 ** (q_exp // 2) * 2.0 ** (q_exp - q_exp // 2)).bfloat16()
    scale = d ** -0.5 * 2.0 ** -(q_exp + k_exp)
    o, lse = fa.attention_decode_cache8(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), n, True, scale)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    Q = f64(q)
    assert np.isfinite(Q).all() and np.abs(Q).max() > 2.0 ** q_exp
    for h in range(H):
        k, v = ((f64(c)[:, h // (H // Hk)] * f64(s)[:, h // (H // Hk), None, None]).reshape(-1, d)[:n]
                for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        for i in range(2):
            seen = slice(0, n - 1 + i)
            s = scale * (k[seen] @ Q[0, i, h])
            e = scale * 2.0 ** -17 * np.abs(Q[0, i, h]).max() * np.abs(k).sum(1).max()
            assert e < 1e-3
            p = np.exp(s - s.max())
            assert abs(f64(lse)[0, h, i] - (s.max() + np.log(p.sum()))) <= 1e-4 + e
            p /= p.sum()
            bound = p @ np.abs(v[seen])
            assert (np.abs(f64(o)[0, i, h] - p @ v[seen]) <= (2.0 ** -7 + 2 * e) * bound).all()


@pytest.mark.parametrize("spread", [0, 40, 90, 130, 184])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [200, 700, 5000])
def test_values_of_very_different_sizes(n, d, spread):
    """V's scales up to the 2^184 apart that a store can write (pages of zeros beside
    bf16's largest values) from page to page, within tiles, from tile to
    tile and from CTA to CTA.  All values are positive, so that O is Σ P |v| and a
    relative bound on it can be held: 2^-7 of it, and what the two e4m3 terms of
    P s_V lose where P s_V is below its tile's largest, M: at most 2^-18 M a key,
    times the key's code.  A dropped page's weight, or the folding of a scale left
    out, changes every element by far more: the bound is asserted to be a small
    part of O."""
    fa = require_gpu()
    H, Hk, block = 6, 2, 16
    pages = -(-n // block)
    g = torch.Generator(device="cuda").manual_seed(n + spread)
    cache = fa.cache8_alloc(pages, Hk, block, d)
    cache.k.copy_(torch.randn(pages, Hk, block, d, device="cuda", generator=g))
    cache.v.copy_(64.0 + 128.0 * torch.rand(pages, Hk, block, d, device="cuda", generator=g))
    at = torch.arange(pages * Hk, device="cuda").reshape(pages, Hk)
    cache.v_scale.copy_(2.0 ** (torch.floor(spread * ((at * 7) % 5) / 4.0) - min(spread // 2, 64)))
    table = torch.arange(pages, device="cuda", dtype=torch.int32)[None]
    q = torch.randn(1, 1, H, d, device="cuda", generator=g).bfloat16()
    o, lse = fa.attention_decode_cache8(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), n)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    tile = 128 * 128 // d
    for h in range(H):
        hk = h // (H // Hk)
        k, codes = (f64(c)[:, hk].reshape(-1, d)[:n] for c in (cache.k, cache.v))
        sv = f64(cache.v_scale)[:, hk].repeat(block)[:n]
        s = d ** -0.5 * k @ f64(q)[0, 0, h]
        p = np.exp(s - s.max())
        assert abs(f64(lse)[0, h, 0] - (s.max() + np.log(p.sum()))) <= 1e-4
        p = p / p.sum() * sv
        want = p @ codes
        lost = sum(2.0 ** -18 * p[a:a + tile].max() * codes[a:a + tile].sum(0) for a in range(0, n, tile))
        bound = 2.0 ** -7 * want + lost
        assert (bound <= 2.0 ** -5 * want).all()
        assert (np.abs(f64(o)[0, 0, h] - want) <= bound).all()


@pytest.mark.parametrize("B", [63, 64, 65, 128, 129])
def test_batches_on_both_sides_of_the_scan(B):
    """Few sequences are found by every warp by itself, more by all together: ragged
    lengths, empty sequences among them, first, last and in between."""
    fa = require_gpu()
    check_attend(fa, 4, 2, 64, 16, [0] + [(i * 53) % 300 for i in range(1, B - 1)] + [0], 1, True, seed=B)
    check_attend(fa, 2, 1, 128, 32, [(i * 29) % 400 for i in range(B)], 2, True, seed=B + 1)
