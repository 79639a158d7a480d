"""Attention of chunks of new tokens over the 8-bit paged cache, against the formula
in 64 bits on the stored values.

Tolerances, element by element.  Keys and values are code times a power of two,
exact in bf16.  A probability is rounded to bf16, by at most 2^-8 of it, and the
output by 2^-8 of itself, which is at most sum P |v|: 2^-7 sum P |v| together.  A
score is a sum of d products in fp32, off by at most d 2^-24 scale sum |q| |k|, of
queries in two e4m3 terms, each element off by at most 2^-17 of its row's largest:
another scale 2^-17 max |q| sum |k|.  The two together, E, move the LSE by E and each
P by 2 E of itself.  The fp32 sums over the keys add
2^-14 of sum P |v| and the exponentials 2^-20: both within 2^-7 * 2^-5.  LSE: 1e-4 + E.
"""
import numpy as np
import pytest
import torch

from tests.gpu_util import assert_no_device_error, f64, gpu, require_gpu
from tests.test_gpu_cache8 import make_table, poison, random_cache

pytestmark = gpu

ERR_PAGE = 12


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check(o, lse, q, cache, table, new, lens, scale, causal):
    """o, lse of the call against the formula; table without entries out of range."""
    H, d = q.shape[1:]
    Hk, block = cache.k.shape[1:3]
    G, first = H // Hk, 0
    ids = table.long().cuda()
    for b, (n, L) in enumerate(zip(new, lens)):
        got, got_lse, qs = (x[first:first + n].double() for x in (o, lse.T, q))
        first += n
        seen = L - n + torch.arange(n, device="cuda") + 1 if causal else torch.full((n,), L, device="cuda")
        live = seen > 0
        assert not got[~live].any() and (got_lse[~live] == -np.inf).all()
        if not live.any():
            continue
        pages = ids[b, :-(-L // block)]
        for h in range(H):
            k, v = ((c[pages, h // G].double() * s[pages, h // G].double()[:, None, None]).reshape(-1, d)[:L]
                    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
            x = qs[live, h]
            s = scale * x @ k.T
            s = s.masked_fill(torch.arange(L, device="cuda") >= seen[live][:, None], -np.inf)
            e = scale * (d * 2.0 ** -24 * float((x.abs() @ k.abs().T).max())
                         + 2.0 ** -17 * float(x.abs().max() * k.abs().sum(1).max()))
            p = torch.softmax(s, 1)
            bound = (2.0 ** -7 * (1 + 2.0 ** -5) + 2 * e) * (p @ v.abs())
            assert ((got[live, h] - p @ v).abs() <= bound).all(), (b, h)
            assert float((got_lse[live, h] - torch.logsumexp(s, 1)).abs().max()) <= 1e-4 + e, (b, h)


def run(fa, H, Hk, d, block, new, lens, causal, seed, cache=None, amplitude=1.0, scale=None, tail=0, max_seqlen=None,
        max_new=None, cols=None):
    B = len(new)
    cols = cols or max(1, max(-(-n // block) for n in lens))
    pages = B * cols + 1
    cache = random_cache(fa, pages, Hk, block, d, seed) if cache is None else cache
    table = make_table(pages, B, cols, seed)
    poison(cache, table, lens)
    sent = table.clone()
    for b, n in enumerate(lens):
        sent[b, -(-n // block):] = -7  # entries behind the last token are never read
    T = sum(new) + tail
    q = (torch.randn(T, H, d, generator=torch.Generator().manual_seed(seed)) * amplitude).bfloat16().cuda()
    q[T - tail:] = float("nan")
    scale = d ** -0.5 if scale is None else scale
    o, lse = fa.attention_chunk_cache8(q, cache, sent.cuda(), i32([0] + np.cumsum(new).tolist()), i32(lens),
                                       max_new or max(1, max(new)), max_seqlen or max(1, max(lens)), causal, scale)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    assert torch.isfinite(o).all()
    check(o, lse, q, cache, table, new, lens, scale, causal)
    assert not o[T - tail:].any() and (lse[:, T - tail:] == -np.inf).all()
    return o, lse


NEW = [1, 0, 5, 128, 70, 3, 33, 300, 2]
LENS = [1, 9, 5, 128, 199, 1, 500, 1000, 0]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_one_short_sequence(d, causal):
    fa = require_gpu()
    run(fa, 4, 2, d, 16, [3], [20], causal, seed=1)
    run(fa, 4, 2, d, 16, [40], [200], causal, seed=2)


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged(causal, d, block):
    """Single tokens, whole prompts, pieces of prompts, empty sequences, sequences with
    fewer cached than new tokens, rows behind the last sequence."""
    fa = require_gpu()
    run(fa, 8, 2, d, block, NEW, LENS, causal, seed=d + block, tail=5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (2, 2), (6, 2), (3, 1), (7, 1), (8, 1), (40, 1), (130, 1), (300, 1)])
def test_heads(H, Hk, d):
    fa = require_gpu()
    run(fa, H, Hk, d, 32, [5, 1, 41], [200, 333, 41], True, seed=H)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 31, 32, 33, 63, 64, 65, 127, 129])
def test_row_blocks_and_tile_borders(n, d):
    """Rows on both sides of the row tiles' borders (4 heads a group), lengths on both
    sides of the key tiles'."""
    fa = require_gpu()
    for L in (n, 127 + n, 128 + n, 256, 257):
        run(fa, 4, 1, d, 64, [n], [max(L, n)], True, seed=n + L)


@pytest.mark.parametrize("d", [64, 128])
def test_long_sequences_shared_by_many_ctas(d):
    fa = require_gpu()
    run(fa, 4, 2, d, 128, [9], [20000], True, seed=14)
    run(fa, 4, 1, d, 64, [300, 1, 64, 700], [9000, 130, 5000, 700], True, seed=15, max_seqlen=10000)
    run(fa, 8, 1, d, 16, [1000], [1300], True, seed=16)


def test_many_sequences():
    """More (sequence, row block) pairs than a block has threads; most of them empty."""
    fa = require_gpu()
    new = [(i * 5) % 4 for i in range(700)]
    run(fa, 2, 1, 64, 16, new, [n + (i * 37) % 90 for i, n in enumerate(new)], True, seed=12)
    run(fa, 2, 1, 128, 16, [1] * 513, [(i * 29) % 50 + 1 for i in range(513)], True, seed=13, max_new=600)
    run(fa, 4, 1, 128, 16, [0, 0, 0], [0, 5, 0], True, seed=13, tail=3)
    run(fa, 4, 1, 128, 16, [2, 1, 0], [0, 0, 0], True, seed=13, tail=3, max_seqlen=50)


@pytest.mark.parametrize("d", [64, 128])
def test_peaked_scores_and_uneven_scales(d):
    """Scores of which one key takes all, found late; scales 2^40 apart; scores that
    rise and fall by hundreds."""
    fa = require_gpu()
    run(fa, 4, 1, d, 16, [50], [2000], True, seed=18, amplitude=30.0)
    for seed, f in ((19, 2.0 ** (torch.arange(130) % 5 * 10.0 - 20)), (20, 2.0 ** (torch.arange(130) % 7 * 20.0 - 60))):
        cache = random_cache(fa, 130, 1, 16, d, seed=seed)
        cache.v_scale.mul_(f[:, None].cuda())
        cache.k_scale.mul_(2.0 ** (torch.arange(130, device="cuda") % 7 - 3.0)[:, None])
        run(fa, 4, 1, d, 16, [30], [2000], True, seed=seed, cache=cache, amplitude=4.0, cols=129)
    # rising scores: the reference of the first tile is left behind by far
    cache = random_cache(fa, 65, 1, 16, d, seed=21)
    cache.k_scale.copy_(torch.exp2(torch.arange(65, device="cuda") / 8).round().log2().round().exp2()[:, None])
    run(fa, 4, 1, d, 16, [30], [1024], False, seed=22, cache=cache, amplitude=3.0, cols=64)


@pytest.mark.parametrize("d", [64, 128])
def test_every_code_and_scale(d):
    """Each of the codes, subnormal ones among them, and scales from 2^-64 to 2^119:
    the values themselves, read back through rows that see one key (O is that key's V,
    rounded to bf16: exact, for a code times a power of two)."""
    fa = require_gpu()
    codes = torch.arange(256, dtype=torch.uint8)
    codes = codes[(codes & 127) != 127]
    n = codes.numel()
    for e in (-64, -30, -1, 0, 7, 8, 60, 118, 119):
        cache = fa.cache8_alloc(n, 1, 16, d)
        cache.v.view(torch.uint8).copy_(codes[:, None, None, None].expand(n, 1, 16, d))
        cache.v_scale.fill_(2.0 ** e)
        q = torch.randn(n, 1, d).bfloat16().cuda()
        table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None]
        cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
        o, _ = fa.attention_chunk_cache8(q, cache, table, cu, torch.ones(n, dtype=torch.int32, device="cuda"), 1, 1, True)
        want = cache.v.float()[:, :, 0] * 2.0 ** e
        assert torch.equal(o.float(), want.bfloat16().float()), e
    # keys: a query of one dimension reads a key's dimension as the score of an only key
    for e in (-64, 0, 7, 9, 60):
        cache = fa.cache8_alloc(n, 1, 16, d)
        cache.k.view(torch.uint8).copy_(codes[:, None, None, None].expand(n, 1, 16, d))
        cache.k_scale.fill_(2.0 ** e)
        for dim in (0, 1, 2, 3, d - 1):
            q = torch.zeros(n, 1, d)
            q[:, :, dim] = 1.0
            _, lse = fa.attention_chunk_cache8(q.bfloat16().cuda(), cache, table, cu, torch.ones(n, dtype=torch.int32, device="cuda"),
                                               1, 1, True, 1.0)
            want = cache.k.double()[:, 0, 0, dim] * 2.0 ** e
            # lse = (score · log2 e + log2 1) ln 2 in fp32: three roundings of 2^-24
            assert ((lse[0].double() - want).abs() <= 2.0 ** -22 * want.abs()).all(), (e, dim)
    assert_no_device_error(fa)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_exp,k_exp", [(110, -60), (125, -70), (-100, 60), (-115, 90), (-60, 30), (0, 119)])
def test_queries_of_any_size(q_exp, k_exp, d):
    """Queries up to bf16's largest and down to its smallest normal numbers, keys over
    the range of their scales, with a softmax scale that makes the scores of order 1."""
    fa = require_gpu()
    cache = random_cache(fa, 20, 2, 16, d, seed=40)
    cache.k_scale.fill_(2.0 ** k_exp)
    q = (torch.randn(21, 8, d, generator=torch.Generator().manual_seed(41)) * 2.0 ** (q_exp // 2) * 2.0 ** (q_exp - q_exp // 2)).bfloat16().cuda()
    assert torch.isfinite(q).all()
    table, scale = torch.arange(19, dtype=torch.int32)[None], d ** -0.5 * 2.0 ** -(q_exp + k_exp) / 8
    o, lse = fa.attention_chunk_cache8(q, cache, table.cuda(), i32([0, 21]), i32([300]), 21, 300, True, scale)
    assert_no_device_error(fa)
    check(o, lse, q, cache, table, [21], [300], scale, True)


@pytest.mark.parametrize("d", [64, 128])
def test_large_values_under_rising_scores(d):
    """Values up to bf16's largest while the scores climb past their first tile's by
    far: what is summed before the last division must not leave fp32."""
    fa = require_gpu()
    cache = random_cache(fa, 40, 1, 16, d, seed=42)
    cache.v.copy_((cache.v.float() / 2).to(torch.float8_e4m3fn))
    cache.v_scale.fill_(2.0 ** 119)
    cache.k_scale.copy_(2.0 ** (torch.arange(40, device="cuda") // 5 - 2.0)[:, None])
    q = torch.randn(9, 4, d, generator=torch.Generator().manual_seed(43)).bfloat16().cuda()
    table = torch.arange(40, dtype=torch.int32)[None]
    o, lse = fa.attention_chunk_cache8(q, cache, table.cuda(), i32([0, 9]), i32([640]), 9, 640, False)
    assert_no_device_error(fa)
    check(o, lse, q, cache, table, [9], [640], d ** -0.5, False)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,block,B", [(64, 32, 5), (128, 16, 3), (64, 128, 130), (128, 64, 70)])
def test_sequences_of_a_few_tiles(d, block, B, causal):
    """Up to 384 keys, the limit under which no item is cut: fewer items than CTAs and
    more, of one half and of both, and empty ones; and one key above the limit."""
    fa = require_gpu()
    for most in (384, 385):
        lens = [(37 * i * i + 11) % (most - 1) + 1 for i in range(B - 2)] + [0, most]
        new = [min(n, (53 * i + 1) % 200) for i, n in enumerate(lens)]
        run(fa, 6, 2, d, block, new, lens, causal, seed=B + d)


def test_indexes_out_of_range():
    """A page out of range reads as zeros, a length out of range is clamped; both are reported."""
    fa = require_gpu()
    for d in (64, 128):
        cache = random_cache(fa, 6, 1, 16, d, seed=23)
        zeros = fa.Cache8(*(torch.cat([t.view(torch.uint8), torch.zeros_like(t[:1].view(torch.uint8))]).view(t.dtype)
                            if t.dtype != torch.float32 else torch.cat([t, torch.ones_like(t[:1])]) for t in cache))
        q = torch.randn(7, 2, d).bfloat16().cuda()
        for bad in (-1, 6, 2 ** 31 - 1, -2 ** 31):
            o, lse = fa.attention_chunk_cache8(q, cache, i32([[0, bad, 2]]), i32([0, 7]), i32([40]), 7, 48, True)
            assert fa.fa_get_device_error() == ERR_PAGE
            check(o, lse, q, zeros, torch.tensor([[0, 6, 2]]), [7], [40], d ** -0.5, True)
        for n, held in ((-3, 0), (1000, 48), (2 ** 31 - 1, 48)):
            o, lse = fa.attention_chunk_cache8(q, cache, i32([[0, 1, 2]]), i32([0, 7]), i32([n]), 7, 48, True)
            assert fa.fa_get_device_error() == ERR_PAGE
            check(o, lse, q, cache, torch.tensor([[0, 1, 2]]), [7], [held], d ** -0.5, True)
        # rows that do not exist are neither read nor written; tokens past max_new are not computed
        o, lse = fa.attention_chunk_cache8(q, cache, i32([[0, 1, 2]]), i32([-5, 400]), i32([40]), 7, 48, True)
        check(o, lse, q, cache, torch.tensor([[0, 1, 2]]), [7], [40], d ** -0.5, True)
        assert_no_device_error(fa)


@pytest.mark.parametrize("d", [64, 128])
def test_repeatable_streams_and_graph(d):
    fa = require_gpu()
    H, Hk, block, new, lens = 8, 2, 32, [70, 1, 200], [3000, 5, 700]
    cols = -(-max(lens) // block)
    cache = random_cache(fa, 3 * cols, Hk, block, d, seed=24)
    table = make_table(3 * cols, 3, cols, 25).cuda()
    wide = torch.randn(sum(new) + 4, H + 3, d).bfloat16().cuda()
    q = wide[:, 1:H + 1]
    n, cu = i32(lens), i32([0] + np.cumsum(new).tolist())
    f = lambda **kw: fa.attention_chunk_cache8(q, cache, table, cu, n, 300, 3200, True, **kw)  # noqa: E731
    size = fa.fa_chunk_cache8_workspace_bytes(3, 300, q.shape[0], H, Hk, 3200, d)
    ws = [torch.full((size,), fill, dtype=torch.uint8, device="cuda") for fill in (0xFF, 0x7F)]
    want = f()
    check(*want, q, cache, table.cpu(), new, lens, d ** -0.5, True)
    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))  # noqa: E731
    assert same(want, f(workspace=ws[0]))
    assert same(want, fa.attention_chunk_cache8(q.contiguous(), cache, table, cu, n, 300, 3200, True))
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):  # two calls at once, each with a workspace of its own
        for side, w in zip(sides, ws):
            side.wait_stream(torch.cuda.current_stream())
            got.append(f(stream=side, workspace=w))
    torch.cuda.synchronize()
    assert all(same(want, g) for g in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = f()
    graph.replay()
    torch.cuda.synchronize()
    assert same(want, cap)
    # other lengths in the captured buffers; 3100 is past the page table's end
    for lens2, new2, error in (([3100, 0, 12], [300, 0, 1], ERR_PAGE), ([cols * block, 0, 12], [300, 0, 1], 0), ([0, 0, 0], [0, 0, 0], 0)):
        n.copy_(torch.tensor(lens2, dtype=torch.int32))
        new2 = [min(x, 271) for x in new2]
        cu.copy_(torch.tensor([0] + np.cumsum(new2).tolist(), dtype=torch.int32))
        graph.replay()
        want = f()
        torch.cuda.synchronize()
        assert fa.fa_get_device_error() == error
        assert same(want, cap)
        check(*cap, q, cache, table.cpu(), new2, [min(x, cols * block) for x in lens2], d ** -0.5, True)
    # rows behind the last sequence as they were
    o, lse = torch.full_like(want[0], 3.0), torch.full_like(want[1], 3.0)
    fa.fa_fwd_chunk_cache8(q, cache, table, cu, n, o, lse, ws[0], 300, 3200, True)
    torch.cuda.synchronize()
    assert (o == 3).all() and (lse == 3).all()


def test_agrees_with_the_other_attentions():
    """A whole prompt against the grouped attention over the same values, and single
    tokens against the cache's decode: each within its own bounds of 64 bits (2^-7
    sum P |v|, twice)."""
    fa = require_gpu()
    H, Hk, d, block, L = 8, 2, 128, 64, 300
    cache = random_cache(fa, 6, Hk, block, d, seed=31)
    table = torch.arange(5, dtype=torch.int32)[None].cuda()
    k, v = ((c[:5].float() * s[:5, :, None, None]).transpose(1, 2).reshape(-1, Hk, d)[:L].bfloat16() for c, s in
            ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    q = torch.randn(L, H, d).bfloat16().cuda()
    vmax = float(v.abs().max())
    o, lse = fa.attention_chunk_cache8(q, cache, table, i32([0, L]), i32([L]), L, L, True)
    og, lg = fa.attention_forward_grouped(q, k, v, i32([0, L]), L, True)
    assert float((o - og).abs().max()) <= 2.0 ** -6 * vmax and float((lse - lg).abs().max()) <= 2e-4
    o, lse = fa.attention_chunk_cache8(q[-1:], cache, table, i32([0, 1]), i32([L]), 1, L, True)
    od, ld = fa.attention_decode_cache8(q[-1:, None].contiguous(), cache, table, i32([L]), L, True)
    assert float((o - od[:, 0]).abs().max()) <= 2.0 ** -6 * vmax and float((lse - ld[0]).abs().max()) <= 2e-4
    assert_no_device_error(fa)


@pytest.mark.parametrize("d,block,axes", [(64, 16, 1), (128, 64, 3)])
def test_serving_loop(d, block, axes):
    """Prompts in pieces (turned and stored, then attended to), then single tokens with
    the decode, as a serving loop runs them: each step against the formula on what the
    cache holds, and what it holds against the whole prompts stored at once."""
    fa = require_gpu()
    H, Hk = 8, 2
    steps = [[70, 1, 200], [0, 130, 33], [64, 0, 5], [1, 1, 1], [1, 1, 1]]
    total = [sum(s) for s in zip(*steps)]
    B, cols = 3, -(-max(total) // block)
    gen = torch.Generator().manual_seed(26)
    plan = fa.rotary_plan([10000.0 ** (-j / (d // 2)) for j in range(d // 2)], axis=[j % axes for j in range(d // 2)])
    cache = fa.cache8_alloc(B * cols, Hk, block, d)
    table = make_table(B * cols, B, cols, 27)
    held = [0] * B
    for new in steps:
        cu = [0] + np.cumsum(new).tolist()
        qkv = torch.randn(cu[-1], H + 2 * Hk, d, generator=gen).bfloat16().cuda()
        q = fa.cache8_store_rotary(qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:], cache, table.cuda(), i32(cu), i32(held),
                                   max(new), plan)
        place = torch.cat([torch.arange(a, a + n) for a, n in zip(held, new)]).int().cuda()
        want, _ = fa.rotary_forward(qkv[:, :H], qkv[:, H:H + Hk], place if axes == 1 else place.expand(axes, -1).contiguous(), plan)
        assert torch.equal(q, want)
        held = [a + n for a, n in zip(held, new)]
        o, lse = fa.attention_chunk_cache8(q, cache, table.cuda(), i32(cu), i32(held), max(new), max(held), True)
        check(o, lse, q, cache, table, new, held, d ** -0.5, True)
        if new == [1, 1, 1]:
            od, _ = fa.attention_decode_cache8(q.reshape(B, 1, H, d), cache, table.cuda(), i32(held), max(held), True)
            vmax = float((cache.v.float() * cache.v_scale[..., None, None]).abs().max())
            assert float((od[:, 0] - o).abs().max()) <= 2.0 ** -6 * vmax
    assert_no_device_error(fa)


def test_refusals():
    fa = require_gpu()
    cache = fa.cache8_alloc(4, 2, 16, 64)
    q = torch.randn(3, 4, 64).bfloat16().cuda()
    table, cu, n = i32([[0, 1]]), i32([0, 3]), i32([20])
    f = fa.attention_chunk_cache8
    for bad in ((q.float(), cache, table, cu, n), (q, cache._replace(k=cache.k.view(torch.uint8)), table, cu, n)):
        with pytest.raises(TypeError):
            f(*bad, 3, 20)
    for bad in ((q, cache, table.long(), cu, n), (q, cache, table, cu, n.long()), (q, cache, table, cu.long(), n),
                (q, cache, table, i32([0, 1, 3]), n), (q, cache._replace(v=cache.v[:3]), table, cu, n),
                (q, cache._replace(k_scale=cache.k_scale.double()), table, cu, n), (q, cache, table, cu, i32([20, 20])),
                (q[..., :32].contiguous(), cache, table, cu, n), (q[..., ::2], cache, table, cu, n), (q, cache, table.cpu(), cu, n),
                (q[None], cache, table, cu, n)):
        with pytest.raises(ValueError):
            f(*bad, 3, 20)
    for bad in ((q[:, :3].contiguous(), 3, 20, None), (q, 3, 0, None), (q, 0, 20, None), (q, 3, 20, -1.0), (q, 3, 20, 0.0),
                (q, 3, 20, float("nan"))):
        with pytest.raises(fa.FaError):
            f(bad[0], cache, table, cu, n, bad[1], bad[2], scale=bad[3])
    for bad in ((2 ** 32 + 1, 20), (3, 2 ** 32 + 1)):
        with pytest.raises(ValueError):
            f(q, cache, table, cu, n, *bad)
    with pytest.raises(fa.FaError):
        f(q, cache, table, cu, n, 3, 20, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(fa.FaError):
        f(q, fa.cache8_alloc(4, 2, 24, 64), table, cu, n, 3, 20)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
