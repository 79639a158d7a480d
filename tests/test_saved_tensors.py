"""What the autograd function saves may come back laid out otherwise (hooks that
keep saved tensors elsewhere, as torch.autograd.graph.save_on_cpu, return slices of
a projection as tensors of their own): the backward goes by what it gets."""
import pytest
import torch

import io_aware_attention_flash_gb300 as fa
from tests.gpu_util import assert_no_device_error, f64, gpu, rel_fro, require_gpu


def test_the_backward_goes_by_the_tensors_it_gets(monkeypatch):
    """Host side: the row strides handed on are those of the tensors handed on."""
    seen = []

    def grouped(q, k, v, cu):
        return tuple(t.stride(0) for t in (q, k, v))

    def backward(checked, q, k, v, o, do, lse, cu, *rest):
        seen.append((checked, tuple(t.stride(0) for t in (q, k, v))))
        return tuple(torch.zeros_like(t) for t in (q, k, v))

    monkeypatch.setattr(fa._binding, "_grouped", grouped)
    monkeypatch.setattr(fa, "_forward_grouped", lambda checked, q, k, v, *a: (q.clone(), q.sum()))
    monkeypatch.setattr(fa, "_backward_grouped", backward)
    qkv = torch.randn(10, 8, 64, requires_grad=True)
    cu = torch.tensor([0, 10], dtype=torch.int32)
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.detach().clone(memory_format=torch.contiguous_format), lambda t: t):
        o = fa._FlashAttentionGrouped.apply(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], cu, 10, True, None)
    o.sum().backward()
    (checked, strides), = seen
    assert strides == (256, 128, 128) and checked == strides


@gpu
@pytest.mark.parametrize("compiled", [True, False])
def test_save_on_cpu(compiled, monkeypatch):
    require_gpu()
    if not compiled:
        monkeypatch.setattr(fa._binding, "_native", fa._binding._NoNative())
    gen = torch.Generator().manual_seed(61)
    qkv = torch.randn(210, 10, 64, generator=gen).bfloat16().cuda().requires_grad_()
    do = torch.randn(210, 6, 64, generator=gen).bfloat16().cuda()
    cu = torch.tensor([0, 130, 200], dtype=torch.int32, device="cuda")

    def step():
        return fa.flash_attention_grouped(qkv[:, :6], qkv[:, 6:8], qkv[:, 8:], cu, 130, causal=True)

    (want,) = torch.autograd.grad(step(), qkv, do)
    with torch.autograd.graph.save_on_cpu():
        o = step()
    (got,) = torch.autograd.grad(o, qkv, do)
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    assert torch.equal(got[:, 6:], want[:, 6:])
    assert rel_fro(f64(got[:, :6]), f64(want[:, :6])) < 2.0 ** -8  # dQ: fp32 sums in another order


@gpu
def test_saved_tensors_of_another_type_are_refused():
    require_gpu()
    q = torch.randn(20, 4, 64, device="cuda").bfloat16().requires_grad_()
    k = torch.randn(20, 2, 64, device="cuda").bfloat16()
    cu = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    # o and lse, which are the kernel's own, come back in half the bytes
    with torch.autograd.graph.saved_tensors_hooks(
            lambda t: t, lambda t: t.to(torch.float8_e4m3fn) if t.shape == (20, 4, 64) and t.grad_fn is not None else t):
        o = fa.flash_attention_grouped(q, k, k, cu, 20, causal=True)
    with pytest.raises(RuntimeError, match="saved tensors"):
        o.sum().backward()
    torch.cuda.synchronize()
    assert_no_device_error(fa)
