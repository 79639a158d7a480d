"""torch.jit.trace records PyTorch's operations, not a kernel that a C call
launches: a traced call has to become an operation of its own (the autograd
function) or be refused, else the recorded graph returns memory that nothing has
written.  Host side, with the launches replaced; the calls themselves are traced
in the GPU test below."""
import pytest
import torch

import io_aware_attention_flash_gb300 as fa
from tests.gpu_util import f64, gpu, rel_fro, require_gpu


class CompiledCalls:
    """Stands for the compiled calls: outputs that no recorded operation fills."""

    def __getattr__(self, name):
        def call(*args):
            out = torch.empty_like(args[0])
            out.detach().numpy()[:] = 3.0
            return out if name == "flash_attention_grouped" else (out, out, out)

        return call


def test_a_traced_call_is_recorded_as_an_operation(monkeypatch):
    def forward(checked, q, k, v, cu, max_seqlen, causal, scale):
        return q * 2, q.sum()

    monkeypatch.setattr(fa._binding, "native", lambda: CompiledCalls())
    monkeypatch.setattr(fa._binding, "_grouped", lambda *a: None)
    monkeypatch.setattr(fa, "_forward_grouped", forward)
    q, k = torch.randn(5, 4, 64), torch.randn(5, 2, 64)
    cu = torch.tensor([0, 5], dtype=torch.int32)
    assert (fa.flash_attention_grouped(q, k, k, cu, 5) == 3.0).all()  # not traced: the compiled call
    traced = torch.jit.trace(lambda q, k, cu: fa.flash_attention_grouped(q, k, k, cu, 5), (q, k, cu), check_trace=False)
    other = torch.randn(5, 4, 64)
    assert torch.equal(traced(other, k, cu), other * 2)


def test_calls_that_cannot_be_recorded_refuse_a_trace(monkeypatch):
    monkeypatch.setattr(fa._binding, "native", lambda: CompiledCalls())
    x = torch.randn(5, 4, 64)
    cu = torch.tensor([0, 5], dtype=torch.int32)
    cache = fa.Cache8(x, x, x, x)
    for f in (lambda x: fa.attention_forward_grouped(x, x, x, cu, 5)[0],
              lambda x: fa.attention_backward_grouped(x, x, x, x, x, x, cu, 5)[0],
              lambda x: fa.attention_decode_cache8(x, cache, cu, cu, 5)[0],
              lambda x: fa.cache8_store(x, x, cache, cu, cu, cu, 5) or x):
        with pytest.raises(RuntimeError, match="trace"):
            torch.jit.trace(f, (x,), check_trace=False)


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


def test_a_proxy_graph_is_refused(monkeypatch):
    """torch.fx's make_fx records operations below the autograd function: none of the
    calls has one to record."""
    from torch.fx.experimental.proxy_tensor import make_fx

    monkeypatch.setattr(fa._binding, "native", lambda: CompiledCalls())
    x = torch.randn(5, 4, 64)
    cu = torch.tensor([0, 5], dtype=torch.int32)
    cache = fa.Cache8(x, x, x, x)
    for f in (lambda x: fa.flash_attention_grouped(x, x, x, cu, 5),
              lambda x: fa.attention_forward_grouped(x, x, x, cu, 5)[0],
              lambda x: fa.attention_backward_grouped(x, x, x, x, x, x, cu, 5)[0],
              lambda x: fa.attention_decode_cache8(x, cache, cu, cu, 5)[0],
              lambda x: fa.cache8_store(x, x, cache, cu, cu, cu, 5) or x):
        with pytest.raises(RuntimeError, match="make_fx"):
            make_fx(f)(x)
    assert (fa.flash_attention_grouped(x, x, x, cu, 5) == 3.0).all()
