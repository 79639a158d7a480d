"""The compiled calls from PyTorch belong to the PyTorch and the Python they were
built against: with another one they are rebuilt, and never loaded as they are."""
import pytest
import torch

from io_aware_attention_flash_gb300 import _binding
from io_aware_attention_flash_gb300 import build as fabuild


@pytest.fixture()
def unloaded(monkeypatch):
    """As in a process that has not loaded the compiled calls yet."""
    fabuild.build()
    monkeypatch.setattr(_binding, "_native", None)
    return monkeypatch


def test_another_pytorch_makes_the_build_out_of_date(unloaded):
    assert fabuild.up_to_date()
    unloaded.setattr(torch, "__version__", "0.0.1+other")
    assert not fabuild.up_to_date()


def test_another_compiler_abi_makes_the_build_out_of_date(unloaded):
    unloaded.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    assert not fabuild.up_to_date()


def test_a_module_built_for_another_pytorch_is_not_loaded(unloaded):
    """The helpers' Python paths, which need libfa_gb300.so alone, take every call."""
    unloaded.setattr(torch, "__version__", "0.0.1+other")
    with pytest.warns(RuntimeWarning, match="built for another"):
        n = _binding.native()
    assert type(n) is not type(_binding)
    assert n.forward_grouped() is None and n.decode_cache8(1, 2) is None
    assert _binding.native() is n  # said once


def test_without_the_module_the_python_paths_take_every_call(unloaded, tmp_path):
    unloaded.setattr(_binding, "TORCH_LIB_PATH", str(tmp_path / "none.so"))
    with pytest.warns(RuntimeWarning, match="is missing"):
        n = _binding.native()
    calls = ("forward_grouped", "backward_grouped", "flash_attention_grouped", "cache8_store", "decode_cache8")
    assert all(getattr(n, name)(None) is None for name in calls)


def test_the_module_built_here_loads(unloaded):
    assert _binding.native().forward_grouped() is None


@pytest.mark.gpu
def test_the_python_paths_alone(unloaded):
    """Prompt, training step, store and decode without the compiled calls: what they give with them."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    import io_aware_attention_flash_gb300 as fa
    i32 = dict(dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(51)
    q, k, v, do = (torch.randn(90, h, 64, device="cuda", generator=gen).bfloat16() for h in (4, 2, 2, 4))
    cu, zero, lens = torch.tensor([0, 60, 90], **i32), torch.zeros(2, **i32), torch.tensor([60, 30], **i32)
    table = torch.arange(8, **i32).reshape(2, 4)

    def run():
        cache = fa.cache8_alloc(8, 2, 16, 64)
        leaves = [t.clone().requires_grad_() for t in (q, k, v)]
        o = fa.flash_attention_grouped(*leaves, cu, 60, causal=True)
        _, dk, dv = torch.autograd.grad(o, leaves, do)
        o1, lse = fa.attention_forward_grouped(q, k, v, cu, 60, True)
        _, dk1, dv1 = fa.attention_backward_grouped(q, k, v, o1, do, lse, cu, 60, True)
        fa.cache8_store(k, v, cache, table, cu, zero, 60)
        return (o, dk, dv, o1, lse, dk1, dv1, *fa.attention_decode_cache8(q[:2, None], cache, table, lens, 60),
                cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale)

    want = run()
    unloaded.setattr(_binding, "_native", _binding._NoNative())
    for a, b in zip(run(), want):
        assert torch.equal(a, b)
