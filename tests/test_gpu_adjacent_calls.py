"""Calls queued directly behind one another: each kernel may be scheduled while
the one before it finishes, so what a call reads (codes, scales, queries, row
statistics) may have been written a moment before it.  All tensors are on the
device before the first call and nothing comes in between; the results are, bit
for bit, those of the same calls with a synchronisation after each."""
import pytest
import torch

from tests.gpu_util import assert_no_device_error, gpu, require_gpu

pytestmark = gpu


def bits(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def assert_same(got, want):
    assert len(got) == len(want)
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(bits(a), bits(b)), i


@pytest.mark.parametrize("B,d,block,H,Hk,Nq", [(3, 128, 16, 8, 2, 1), (2, 64, 64, 4, 4, 1), (64, 128, 32, 16, 8, 1),
                                               (5, 64, 16, 16, 2, 4), (1, 128, 128, 16, 1, 8)])
def test_store_and_attend_in_turn(B, d, block, H, Hk, Nq):
    """Every store appends Nq tokens twice the size of the ones before, so that
    pages' scales change under the attention that follows at once.  How far two
    kernels overlap differs from run to run, so the run is repeated."""
    fa = require_gpu()
    steps, held = 12, 37
    gen = torch.Generator().manual_seed(B + d)
    cols = -(-(held + steps * Nq) // block)
    table = torch.randperm(B * cols, generator=gen).reshape(B, cols).int().cuda()
    draw = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    prompt = [draw(B * held, Hk, d).bfloat16().cuda() for _ in range(2)]
    new = [[(draw(B * Nq, Hk, d) * 2.0 ** i).bfloat16().cuda() for _ in range(2)] for i in range(steps)]
    # scores of order 1 at every step
    q = [(draw(B, Nq, H, d) * 2.0 ** -i).bfloat16().cuda() for i in range(steps)]
    i32 = dict(dtype=torch.int32, device="cuda")
    cu0, cu = torch.arange(B + 1, **i32) * held, torch.arange(B + 1, **i32) * Nq
    zero = torch.zeros(B, **i32)
    starts = [torch.full((B,), held + i * Nq, **i32) for i in range(steps)]
    lens = [torch.full((B,), held + (i + 1) * Nq, **i32) for i in range(steps)]
    empty = [t.clone() for t in fa.cache8_alloc(B * cols, Hk, block, d)]

    def run(cache, pause):
        out = []
        fa.cache8_store(*prompt, cache, table, cu0, zero, held)
        for i in range(steps):
            pause()
            fa.cache8_store(*new[i], cache, table, cu, starts[i], Nq)
            pause()
            out += fa.attention_decode_cache8(q[i], cache, table, lens[i], held + steps * Nq, True)
        pause()
        return out

    cache = fa.cache8_alloc(B * cols, Hk, block, d)
    torch.cuda.synchronize()
    want = run(cache, torch.cuda.synchronize)
    want_cache = [t.clone() for t in cache]

    def reset():
        for t, e in zip(cache, empty):
            bits(t).copy_(bits(e))
        torch.cuda.synchronize()

    for _ in range(10):
        reset()
        got = run(cache, lambda: None)
        torch.cuda.synchronize()
        assert_same(got, want)
        assert_same(cache, want_cache)
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = run(cache, lambda: None)
    for _ in range(5):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert_same(cap, want)
        assert_same(cache, want_cache)
    assert_no_device_error(fa)


@pytest.mark.parametrize("d", [64, 128])
def test_a_layers_outputs_are_the_next_calls_inputs(d):
    """A prompt's attention, whose output is taken as the keys and values that the
    store writes and as the queries that then attend to them; and a forward whose
    gradients are the next forward's inputs."""
    fa = require_gpu()
    H, Hk, block, lengths = 8, 2, 16, [64, 130, 5, 300]
    B, T = len(lengths), sum(lengths)
    gen = torch.Generator().manual_seed(d)
    q, do = ((torch.randn(T, H, d, generator=gen)).bfloat16().cuda() for _ in range(2))
    k, v = ((torch.randn(T, Hk, d, generator=gen)).bfloat16().cuda() for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + lengths, **i32).cumsum(0, dtype=torch.int32)
    cols = -(-max(lengths) // block)
    table = torch.arange(B * cols, **i32).reshape(B, cols)
    zero, lens = torch.zeros(B, **i32), torch.tensor(lengths, **i32)
    n = max(lengths)
    cache = fa.cache8_alloc(B * cols, Hk, block, d)
    torch.cuda.synchronize()

    def run(pause):
        o, lse = fa.attention_forward_grouped(q, k, v, cu, n, True)
        pause()
        fa.cache8_store(o[:, :Hk], o[:, Hk:2 * Hk], cache, table, cu, zero, n)
        pause()
        o2, lse2 = fa.attention_decode_cache8(o[:B].view(B, 1, H, d), cache, table, lens, n)
        pause()
        _, dk, dv = fa.attention_backward_grouped(q, k, v, o, do, lse, cu, n, True)
        pause()
        o3, lse3 = fa.attention_forward_grouped(o, dk, dv, cu, n, True)
        pause()
        _, dk2, dv2 = fa.attention_backward_grouped(o, dk, dv, o3, do, lse3, cu, n, True)
        pause()
        return [o, lse, o2, lse2, dk, dv, o3, lse3, dk2, dv2, *(t.clone() for t in cache)]

    want = run(torch.cuda.synchronize)
    for _ in range(10):
        got = run(lambda: None)
        torch.cuda.synchronize()
        assert_same(got, want)
    assert_no_device_error(fa)
