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
    unloaded.setattr(torch, "__version__", "0.0.1+other")
    with pytest.raises(RuntimeError, match="built for another"):
        _binding.native()


def test_the_module_built_here_loads(unloaded):
    assert _binding.native().forward_grouped() is None
