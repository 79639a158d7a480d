"""Rows of the append that belong to no sequence."""
import numpy as np
import pytest
import torch

from tests.gpu_util import assert_no_device_error, gpu, require_gpu
from tests.test_gpu_cache8 import bits, make_table, random_cache

pytestmark = gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("d,block,H,Hk", [(64, 16, 4, 2), (128, 64, 10, 5)])
def test_rows_in_front_of_the_first_sequence(d, block, H, Hk, given):
    """They belong to no sequence, as those behind the last: zeros from the call that
    allocates, left as they were by the one that does not; the others as without them."""
    fa = require_gpu()
    new, start = [7, 0, 30, 1], [3, 9, 0, block]
    cols = max(-(-(a + n) // block) for a, n in zip(start, new))
    plan = fa.rotary_plan([10000.0 ** (-j / (d // 2)) for j in range(d // 2)])
    for first, tail in ((0, 5), (1, 0), (2, 3), (6, 1), (203, 2)):
        cu = np.cumsum([first] + new).tolist()
        T, gen = cu[-1] + tail, torch.Generator().manual_seed(first + d)
        q, k, v = (torch.randn(T, h, d, generator=gen).bfloat16().cuda() for h in (H, Hk, Hk))
        at = torch.randint(0, 5000, (T,), dtype=torch.int32, generator=gen).cuda() if given else None
        pool = random_cache(fa, len(new) * cols, Hk, block, d, seed=first)
        caches = [fa.Cache8(*(t.clone() for t in pool)) for _ in range(3)]
        table = make_table(len(new) * cols, len(new), cols, first).cuda()
        inner = slice(first, cu[-1])
        want = fa.cache8_store_rotary(q[inner], k[inner], v[inner], caches[0], table, i32(np.cumsum([0] + new).tolist()), i32(start),
                                      30, plan, at[inner].contiguous() if given else None)
        args = (table, i32(cu), i32(start), 30, plan, at)
        outs = [torch.full((T, H, d), 3.0, device="cuda").bfloat16() for _ in range(2)]
        for zero_tail in (True, False):
            fa.fa_cache8_store_rotary(q, k, v, outs[zero_tail], caches[1 + zero_tail], *args, zero_tail=zero_tail)
        torch.cuda.synchronize()
        assert_no_device_error(fa)
        outside = torch.ones(T, dtype=torch.bool, device="cuda")
        outside[inner] = False
        for zero_tail in (True, False):
            assert torch.equal(outs[zero_tail][inner], want)
            assert (outs[zero_tail][outside] == (0 if zero_tail else 3)).all()
        for c in caches[1:]:
            assert all(torch.equal(bits(a), bits(b)) for a, b in zip(caches[0], c))
