"""The 8-bit cache's attention at the ends of its ranges, against the formula in
64 bits."""
import numpy as np
import pytest
import torch

from tests.gpu_util import assert_no_device_error, f64, gpu, require_gpu

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
