"""A recorder (torch.jit.trace, make_fx) would not see the kernels that the rotary, the
append and the chunk calls launch: they refuse it, on the compiled and on the Python
path."""
import pytest
import torch

import io_aware_attention_flash_gb300 as fa
from tests.gpu_util import gpu, require_gpu


@pytest.fixture(autouse=True)
def built():
    from io_aware_attention_flash_gb300 import build
    build.build()


def calls(cache, cu, start, lens, table, at, plan):
    """Calls of x [5, 4, 64]."""
    return [lambda x: fa.rotary_forward(x, x, at, plan)[0], lambda x: fa.rotary_backward(x, x, at, plan)[0],
            lambda x: fa.rotary_embedding(x, x, at, plan)[0],
            lambda x: fa.cache8_store_rotary(x, x, x, cache, table, cu, start, 5, plan),
            lambda x: fa.attention_chunk_cache8(x, cache, table, cu, lens, 5, 5)[0]]


def assert_refused(f, x):
    from torch.fx.experimental.proxy_tensor import make_fx

    with pytest.raises(RuntimeError, match="cannot be recorded"):
        torch.jit.trace(f, (x,), check_trace=False)
    with pytest.raises(RuntimeError, match="cannot be recorded"):
        make_fx(f)(x)


def test_refused_on_the_host():
    cu = torch.tensor([0, 5], dtype=torch.int32)
    plan = fa.rotary_plan([1.0] * 8, device="cpu")
    for f in calls(fa.Cache8(*[torch.zeros(1)] * 4), cu, cu[:1], cu[1:], cu[None], torch.arange(5).int(), plan):
        assert_refused(f, torch.randn(5, 4, 64))


@gpu
def test_refused_by_the_compiled_calls():
    require_gpu()
    i32 = dict(dtype=torch.int32, device="cuda")
    args = (fa.cache8_alloc(1, 4, 16, 64), torch.tensor([0, 5], **i32), torch.zeros(1, **i32), torch.tensor([5], **i32),
            torch.zeros(1, 1, **i32), torch.arange(5, **i32), fa.rotary_plan([1.0] * 8))
    x = torch.randn(5, 4, 64, device="cuda").bfloat16()
    for f in calls(*args):
        f(x)  # in order outside
        assert_refused(f, x)
