"""Other Python threads run on while a call waits for room in the launch queue."""
import threading
import time

import pytest
import torch

from tests.gpu_util import assert_no_device_error, gpu, require_gpu

pytestmark = gpu


def calls(fa):
    i32 = dict(dtype=torch.int32, device="cuda")
    k = torch.randn(4, 2, 64, device="cuda").bfloat16()
    q = torch.randn(4, 4, 64, device="cuda").bfloat16()
    cu, zero, lens = torch.tensor([0, 4], **i32), torch.zeros(1, **i32), torch.tensor([4], **i32)
    cache = fa.cache8_alloc(1, 2, 16, 64)
    table = torch.zeros(1, 1, **i32)
    o, lse = fa.attention_forward_grouped(q, k, k, cu, 4, True)
    leaf = q.clone().requires_grad_()
    q1 = q[:1, None].contiguous()
    return {
        "store": lambda: fa.cache8_store(k, k, cache, table, cu, zero, 4),
        "decode": lambda: fa.attention_decode_cache8(q1, cache, table, lens, 4),
        "forward": lambda: fa.attention_forward_grouped(q, k, k, cu, 4, True),
        "backward": lambda: fa.attention_backward_grouped(q, k, k, o, q, lse, cu, 4, True),
        "autograd": lambda: fa.flash_attention_grouped(leaf, k, k, cu, 4, True),
    }


@pytest.mark.parametrize("name", ["store", "decode", "forward", "backward", "autograd"])
def test_a_full_launch_queue_stops_no_other_thread(name):
    """The GPU is kept busy for about a second (a bounded spin) and more calls are
    queued than the driver takes: the call that blocks must not hold the
    interpreter.  Another thread notes the time every millisecond; were it stopped
    for the length of the block (checked to be over half a second in all), its
    largest gap would show it."""
    fa = require_gpu()
    call = calls(fa)[name]
    for _ in range(10):
        call()
    torch.cuda.synchronize()
    gap, done = [0.0], threading.Event()

    def clock():
        last = time.perf_counter()
        while not done.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gap[0] = max(gap[0], now - last)
            last = now

    t = threading.Thread(target=clock)
    t.start()
    begin = time.perf_counter()
    torch.cuda._sleep(2_000_000_000)
    for _ in range(2000):
        call()
    blocked = time.perf_counter() - begin
    done.set()
    t.join()
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    assert blocked > 0.5, "the queue was meant to fill"
    assert gap[0] < 0.25, f"another thread stood still for {gap[0]:.2f} s of {blocked:.2f} s"


@pytest.mark.parametrize("mode", ["anomaly", "dispatch", "hooks", "inference"])
def test_modes_that_call_python_while_the_lock_is_free(mode):
    """What PyTorch calls back into Python for during a compiled call takes the
    interpreter's lock itself: the call's outputs and gradients are the plain ones."""
    from torch.utils._python_dispatch import TorchDispatchMode

    fa = require_gpu()
    seen = []

    class Log(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            seen.append(str(func))
            return func(*args, **(kwargs or {}))

    gen = torch.Generator(device="cuda").manual_seed(71)
    q, k, v, do = (torch.randn(150, h, 64, device="cuda", generator=gen).bfloat16() for h in (4, 2, 2, 4))
    cu = torch.tensor([0, 100, 150], dtype=torch.int32, device="cuda")

    def step():
        leaves = [t.clone().requires_grad_() for t in (q, k, v)]
        o = fa.flash_attention_grouped(*leaves, cu, 100, causal=True)
        if torch.is_inference_mode_enabled():
            return [o]
        return [o, *torch.autograd.grad(o, leaves[1:], do)]

    want = step()
    scope = {"anomaly": lambda: torch.autograd.detect_anomaly(check_nan=True), "dispatch": Log,
             "hooks": lambda: torch.autograd.graph.saved_tensors_hooks(lambda t: seen.append(1) or t.clone(), lambda t: t),
             "inference": torch.inference_mode}[mode]
    with scope():
        got = step()
    torch.cuda.synchronize()
    assert_no_device_error(fa)
    assert mode not in ("dispatch", "hooks") or seen
    for a, b in zip(got, want):
        assert torch.equal(a, b)
