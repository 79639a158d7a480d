"""The chunk attention where a call's rows are not those of the tight case: more new
tokens than max_new, rows in front of the first sequence, batches without a new token,
many empty places of a batch, values stored as NaN.  Tolerances as in
tests/test_gpu_chunk8.py, whose check of the formula is used."""
import numpy as np
import pytest
import torch

from tests.gpu_util import assert_no_device_error, gpu, require_gpu
from tests.test_gpu_cache8 import make_table, random_cache
from tests.test_gpu_chunk8 import ERR_PAGE, check, i32

pytestmark = gpu


def batch(fa, H, Hk, d, block, lens, T, seed):
    cols = max(1, max(-(-n // block) for n in lens))
    cache = random_cache(fa, len(lens) * cols, Hk, block, d, seed)
    table = make_table(len(lens) * cols, len(lens), cols, seed)
    q = torch.randn(T, H, d, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
    return cache, table, q


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,Hk,d,block,max_new", [(4, 2, 64, 16, 7), (8, 1, 128, 64, 33), (6, 2, 128, 32, 1), (16, 2, 64, 128, 100)])
def test_more_new_tokens_than_max_new(H, Hk, d, block, max_new, causal):
    """The first max_new rows of a sequence are those of the whole one, and that there
    are more is reported; sequences within the limit, and rows behind the last, are as
    ever.  Lengths below the number of new tokens too."""
    fa = require_gpu()
    new, lens = [max_new, max_new + 1, 150, 0, 1, 200, 180, max_new], [max_new, 400, 150, 9, 300, 160, 1000, 130]
    cache, table, q = batch(fa, H, Hk, d, block, lens, sum(new) + 3, seed=max_new + d)
    cu = np.cumsum([0] + new).tolist()
    args = (q, cache, table.cuda(), i32(cu), i32(lens))
    whole = fa.attention_chunk_cache8(*args, max(new), max(lens), causal)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    check(*whole, q, cache, table, new, lens, d ** -0.5, causal)
    o, lse = fa.attention_chunk_cache8(*args, max_new, max(lens), causal)
    torch.cuda.synchronize()
    assert fa.fa_get_device_error() == ERR_PAGE
    for a, n in zip(cu, new):  # rows past the limit are unspecified
        o[a + max_new:a + n], lse[:, a + max_new:a + n] = whole[0][a + max_new:a + n], whole[1][:, a + max_new:a + n]
    check(o, lse, q, cache, table, new, lens, d ** -0.5, causal)
    assert not o[cu[-1]:].any() and (lse[:, cu[-1]:] == -np.inf).all()


def test_a_replayed_step_outgrows_max_new():
    fa = require_gpu()
    H, Hk, d, block = 8, 2, 128, 16
    cache, table, q = batch(fa, H, Hk, d, block, [200, 300], 60, seed=4)
    cu, lens = i32([0, 8, 16]), i32([100, 300])
    f = lambda: fa.attention_chunk_cache8(q, cache, table.cuda(), cu, lens, 8, 300, True)  # noqa: E731
    f()
    graph = torch.cuda.CUDAGraph()
    held = table.cuda()
    with torch.cuda.graph(graph):
        o, lse = fa.attention_chunk_cache8(q, cache, held, cu, lens, 8, 300, True)
    for new, n, error in (([8, 8], [100, 300], 0), ([30, 5], [120, 300], ERR_PAGE), ([3, 8], [200, 8], 0)):
        cu.copy_(torch.tensor(np.cumsum([0] + new), dtype=torch.int32))
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert fa.fa_get_device_error() == error
        whole = fa.attention_chunk_cache8(q, cache, held, cu, lens, 60, 300, True)
        got = [t.clone() for t in (o, lse)]
        for a, m in zip(np.cumsum([0] + new), new):
            got[0][a + 8:a + m], got[1][:, a + 8:a + m] = whole[0][a + 8:a + m], whole[1][:, a + 8:a + m]
        check(*got, q, cache, table, new, n, d ** -0.5, True)
    assert_no_device_error(fa)


@pytest.mark.parametrize("d", [64, 128])
def test_rows_in_front_of_the_first_sequence(d):
    """They belong to no sequence, as those behind the last: zeros from the call that
    allocates, left as they were by the one that does not."""
    fa = require_gpu()
    H, Hk, block, new, lens = 4, 2, 16, [7, 0, 30], [90, 3, 30]
    for first, tail in ((0, 4), (1, 0), (13, 4), (200, 1)):
        cu = np.cumsum([first] + new).tolist()
        T = cu[-1] + tail
        cache, table, q = batch(fa, H, Hk, d, block, lens, T, seed=first + d)
        q[:first] = q[cu[-1]:] = float("nan")
        args = (q, cache, table.cuda(), i32(cu), i32(lens))
        ws = torch.empty(fa.fa_chunk_cache8_workspace_bytes(3, 30, T, H, Hk, 90, d), dtype=torch.uint8, device="cuda")
        for zero_tail in (True, False):
            o, lse = torch.full((T, H, d), 3.0, device="cuda").bfloat16(), torch.full((H, T), 3.0, device="cuda")
            fa.fa_fwd_chunk_cache8(*args, o, lse, ws, 30, 90, True, zero_tail=zero_tail)
            torch.cuda.synchronize()
            outside = torch.ones(T, dtype=torch.bool, device="cuda")
            outside[first:cu[-1]] = False
            assert (o[outside] == (0 if zero_tail else 3)).all() and (lse.T[outside] == (-np.inf if zero_tail else 3)).all()
            check(o[first:], lse[:, first:], q[first:], cache, table, new, lens, d ** -0.5, True)
    # a batch of rows, none of them a sequence's
    o, lse = fa.attention_chunk_cache8(q, cache, table.cuda(), i32([5, 5, 5, 5]), i32([0, 3, 0]), 30, 90, True)
    torch.cuda.synchronize()
    assert not o.any() and (lse == -np.inf).all()
    assert_no_device_error(fa)


def test_lengths_are_reported_without_new_tokens():
    fa = require_gpu()
    cache, table, q = batch(fa, 2, 1, 64, 16, [40, 40], 5, seed=3)
    for lens, error in (([40, 0], 0), ([41, 48], 0), ([40, 49], ERR_PAGE), ([-1, 3], ERR_PAGE), ([0, 2 ** 31 - 1], ERR_PAGE)):
        o, lse = fa.attention_chunk_cache8(q, cache, table.cuda(), i32([0, 0, 0]), i32(lens), 5, 1000, True)
        torch.cuda.synchronize()
        assert fa.fa_get_device_error() == error
        assert not o.any() and (lse == -np.inf).all()


@pytest.mark.parametrize("H,d,total,B", [(64, 64, 4096, 32768), (8, 128, 1024, 5000)])
def test_many_places_without_new_tokens(H, d, total, B):
    """A batch of many places, of which a few have a token, in a buffer of many rows: the
    places between two of them times the row blocks that the buffer could hold (2^25 at
    the most here) are passed within the waits' limit."""
    fa = require_gpu()
    at = {0: (1, 700), 1: (2, 90), B // 2: (3, 1000), B - 1: (1, 400)}
    new, lens = [0] * B, [0] * B
    for b, (n, L) in at.items():
        new[b], lens[b] = n, L
    block, cols = 128, 8
    cache = random_cache(fa, len(at) * cols, 1, block, d, seed=d)
    few = make_table(len(at) * cols, len(at), cols, d)
    table = torch.full((B, cols), -5, dtype=torch.int32)
    for row, b in enumerate(at):
        table[b] = few[row]
    q = torch.randn(total, H, d, generator=torch.Generator().manual_seed(d)).bfloat16().cuda()
    o, lse = fa.attention_chunk_cache8(q, cache, table.cuda(), i32(np.cumsum([0] + new).tolist()), i32(lens), 2 ** 31 - 1, 1000, True)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    check(o, lse, q, cache, few, [n for n, _ in at.values()], [L for _, L in at.values()], d ** -0.5, True)
    assert not o[7:].any() and (lse[:, 7:] == -np.inf).all()


@pytest.mark.parametrize("what", ["v", "k"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,Hk,d,block,new,lens", [
    (8, 2, 128, 16, [40, 1, 300, 9], [700, 513, 300, 5000]), (4, 1, 64, 64, [33, 600, 2], [64, 1500, 9000]),
    (2, 2, 64, 16, [130, 3], [130, 384]), (16, 1, 128, 128, [20, 100], [3000, 260])])
def test_stored_nan_reaches_the_rows_that_see_it(H, Hk, d, block, new, lens, causal, what):
    """A key or value stored as NaN makes the results of the rows that see it NaN, and no
    others'; NaN codes behind a sequence's last token reach none."""
    fa = require_gpu()
    G, T = H // Hk, sum(new)
    clean, table, q = batch(fa, H, Hk, d, block, lens, T, seed=H + d)
    cache = fa.Cache8(*(t.clone() for t in clean))
    for b, L in enumerate(lens):
        if L % block:
            for c in cache[:2]:
                c.view(torch.uint8)[int(table[b, L // block]), :, L % block:] = 0x7F
    bad = torch.zeros(T, H, dtype=torch.bool, device="cuda")
    first = 0
    for b, (n, L) in enumerate(zip(new, lens)):
        # the last token, one inside the new ones, one long before them, by head
        places = [(0, L - 1, d - 1, 0x7F), (Hk - 1, max(0, L - n) + n // 3, 5, 0xFF)]
        if b == 1:
            places = [(Hk - 1, L // 7, 0, 0x7F)] if Hk > 1 else []
        for hk, at, dim, code in places:
            getattr(cache, what).view(torch.uint8)[int(table[b, at // block]), hk, at % block, dim] = code
            seen = L - n + np.arange(n) + 1 if causal else np.full(n, L)
            for i in np.flatnonzero(seen > at):
                bad[first + i, hk * G:(hk + 1) * G] = True
        first += n
    args = (table.cuda(), i32(np.cumsum([0] + new).tolist()), i32(lens), max(new), max(lens), causal)
    o, lse = fa.attention_chunk_cache8(q, cache, *args)
    want, want_lse = fa.attention_chunk_cache8(q, clean, *args)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    assert bad.any() and not bad.all()
    assert torch.isnan(o[bad]).all() and torch.isnan(lse.T[bad]).all()
    o, lse = torch.where(bad[..., None], want, o), torch.where(bad.T, want_lse, lse)
    check(o, lse, q, clean, table, new, lens, d ** -0.5, causal)


@pytest.mark.parametrize("d", [64, 128])
def test_pages_out_of_range_beside_stored_nan(d):
    """What a page out of range leaves in its place from tiles before it counts as zeros,
    a NaN too."""
    fa = require_gpu()
    block, cols = 16, 60
    cache = random_cache(fa, cols + 1, 1, block, d, seed=d)
    cache.v.view(torch.uint8)[cols] = 0x7F
    table = torch.arange(cols, dtype=torch.int32)[None].repeat(3, 1)
    q = torch.randn(12, 2, d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    clean = fa.Cache8(*(t.clone() for t in cache))
    for c in clean[:2]:
        c.view(torch.uint8)[cols] = 0
    sent, read = table.clone(), table.clone()
    sent[0, ::2] = read[0, ::2] = cols          # sequence 0: every other page all NaN
    sent[1, 1::3], read[1, 1::3] = cols + 1, cols  # sequence 1: out of range
    new, lens = [4, 4, 4], [900, 950, 960]
    args = (i32([0, 4, 8, 12]), i32(lens), 4, 960, True)
    o, lse = fa.attention_chunk_cache8(q, cache, sent.cuda(), *args)
    torch.cuda.synchronize()
    assert fa.fa_get_device_error() == ERR_PAGE
    assert torch.isnan(o[:4]).all() and torch.isfinite(o[4:]).all()
    want = fa.attention_chunk_cache8(q, clean, read.cuda(), *args)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    o[:4], lse[:, :4] = want[0][:4], want[1][:, :4]
    clean.k_scale[cols] = clean.v_scale[cols] = 1.0
    check(o, lse, q, clean, read, new, lens, d ** -0.5, True)
