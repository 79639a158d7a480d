"""torch.jit.trace and make_fx record PyTorch's operations, not a kernel that a C
call launches: a recorded call has to become an operation of its own (the autograd
function) or be refused, else the recorded graph returns memory that nothing has
written.  Host side on CPU tensors, which the compiled calls hand to the Python
paths; that the compiled calls leave a recorder to those, on the GPU."""
import pytest
import torch

import io_aware_attention_flash_gb300 as fa
from tests.gpu_util import f64, gpu, rel_fro, require_gpu


@pytest.fixture(autouse=True)
def built():
    from io_aware_attention_flash_gb300 import build
    build.build()


def calls(cu, cache, table, lens):
    """Calls of x [5, 4, 64] that have no operation to record."""
    return [lambda x: fa.attention_forward_grouped(x, x, x, cu, 5)[0],
            lambda x: fa.attention_backward_grouped(x, x, x, x, x, x[..., 0].float().T.contiguous(), cu, 5)[0],
            lambda x: fa.attention_decode_cache8(x[:1, None].contiguous(), cache, table, lens, 5)[0],
            lambda x: fa.cache8_store(x, x, cache, table, cu, lens, 5) or x]


def cpu_calls():
    cu = torch.tensor([0, 5], dtype=torch.int32)
    return calls(cu, fa.Cache8(*[torch.zeros(1)] * 4), cu[None], cu[1:])


def test_a_traced_call_is_recorded_as_an_operation(monkeypatch):
    monkeypatch.setattr(fa._binding, "_grouped", lambda *a: None)
    monkeypatch.setattr(fa, "_forward_grouped", lambda checked, q, *a: (q * 2, q.sum()))
    q, k = torch.randn(5, 4, 64), torch.randn(5, 2, 64)
    cu = torch.tensor([0, 5], dtype=torch.int32)
    traced = torch.jit.trace(lambda q, k, cu: fa.flash_attention_grouped(q, k, k, cu, 5), (q, k, cu), check_trace=False)
    other = torch.randn(5, 4, 64)
    assert torch.equal(traced(other, k, cu), other * 2)


def refused(f, x):
    from torch.fx.experimental.proxy_tensor import make_fx

    with pytest.raises(RuntimeError, match="cannot be recorded"):
        make_fx(f)(x)


def test_calls_that_cannot_be_recorded_are_refused():
    x = torch.randn(5, 4, 64)
    cu = torch.tensor([0, 5], dtype=torch.int32)
    for f in cpu_calls():
        with pytest.raises(RuntimeError, match="cannot be recorded"):
            torch.jit.trace(f, (x,), check_trace=False)
    for f in (*cpu_calls(), lambda x: fa.flash_attention_grouped(x, x, x, cu, 5)):
        refused(f, x)


@gpu
def test_the_compiled_calls_leave_a_recorder_to_the_python_paths():
    require_gpu()
    x = torch.randn(5, 4, 64, device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, lens, table = torch.tensor([0, 5], **i32), torch.tensor([5], **i32), torch.zeros(1, 1, **i32)
    cache = fa.cache8_alloc(1, 4, 16, 64)
    for f in calls(cu, cache, table, lens):
        f(x)  # in order outside
        with pytest.raises(RuntimeError, match="cannot be recorded"):
            torch.jit.trace(f, (x,), check_trace=False)
        refused(f, x)
    refused(lambda x: fa.flash_attention_grouped(x, x, x, cu, 5), x)


@gpu
def test_traced_on_the_gpu():
    """The traced function on other inputs: the eager call's outputs and gradients."""
    require_gpu()
    gen = torch.Generator().manual_seed(41)
    cu = torch.tensor([0, 70, 200], dtype=torch.int32, device="cuda")

    def inputs():
        return [torch.randn(200, h, 64, generator=gen).bfloat16().cuda().requires_grad_() for h in (4, 2, 2)]

    traced = torch.jit.trace(lambda q, k, v, cu: fa.flash_attention_grouped(q, k, v, cu, 130, causal=True),
                             (*inputs(), cu), check_trace=False)
    q, k, v = inputs()
    do = torch.randn(200, 4, 64, generator=gen).bfloat16().cuda()
    want = fa.flash_attention_grouped(q, k, v, cu, 130, causal=True)
    got = traced(q, k, v, cu)
    assert torch.equal(got, want)
    a, b = (torch.autograd.grad(o, (q, k, v), do) for o in (got, want))
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    assert rel_fro(f64(a[0]), f64(b[0])) < 2.0 ** -8  # dQ: fp32 sums in another order
