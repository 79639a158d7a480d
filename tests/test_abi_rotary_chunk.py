"""Refusals of the rotary, append and chunk entry points, on the host: bad arguments
are errors before anything touches a GPU, and frequencies become fractions of a turn."""
import math
from fractions import Fraction

import pytest
import torch

import io_aware_attention_flash_gb300 as fa
from io_aware_attention_flash_gb300 import _binding
from io_aware_attention_flash_gb300 import build as fabuild

P = 0x10000  # aligned; arguments are refused before it is used
NULL, ALIGN, HEAD_DIM, SHAPE, WORKSPACE, SCALE, NOT_DEVICE = 1, 2, 3, 4, 8, 9, 10


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return _binding.lib()


def rotary(lib, q=P, k=P, q_out=P, k_out=P, positions=P, turns=P, axis=P, total=5, H=4, Hk=2, d=64, pairs=32, axes=1, il=0,
           inverse=0, ldq=256, ldk=128):
    return lib.fa_rotary(q, k, q_out, k_out, positions, turns, axis, total, H, Hk, d, pairs, axes, il, inverse, ldq, ldk, None)


def append(lib, q=P, k=P, v=P, q_out=P, kc=P, vc=P, ks=P, vs=P, table=P, cu=P, start=P, positions=None, turns=P, axis=None, B=2,
           max_new=3, total=5, num_blocks=4, cols=2, H=4, Hk=2, block=16, d=64, pairs=32, axes=1, il=0, ldq=256, ldk=128, ldv=128):
    return lib.fa_cache8_store_rotary(q, k, v, q_out, kc, vc, ks, vs, table, cu, start, positions, turns, axis, B, max_new, total,
                                      num_blocks, cols, H, Hk, block, d, pairs, axes, il, ldq, ldk, ldv, 0, None)


def chunk(lib, q=P, kc=P, vc=P, ks=P, vs=P, table=P, cu=P, lens=P, o=P, lse=P, ws=P, nbytes=1 << 40, B=2, max_new=3, total=5, H=4,
          Hk=2, num_blocks=4, cols=2, block=16, max_seqlen=32, d=64, ldq=256, scale=0.125):
    return lib.fa_fwd_chunk_cache8(q, kc, vc, ks, vs, table, cu, lens, o, lse, ws, nbytes, B, max_new, total, H, Hk, num_blocks, cols,
                                   block, max_seqlen, d, ldq, scale, 1, 0, None)


@pytest.mark.parametrize("bad,status", [
    (dict(d=32, pairs=8), HEAD_DIM), (dict(pairs=0), SHAPE), (dict(pairs=12), SHAPE), (dict(pairs=40), SHAPE), (dict(axes=0), SHAPE),
    (dict(axes=33), SHAPE), (dict(turns=None), NULL), (dict(axes=2, axis=None), NULL), (dict(total=0), SHAPE), (dict(H=0), SHAPE),
    (dict(Hk=0), SHAPE), (dict(positions=None), NULL), (dict(q=None), NULL), (dict(k_out=None), NULL), (dict(q=P + 8), ALIGN),
    (dict(k_out=P + 2), ALIGN), (dict(ldq=255), SHAPE), (dict(ldq=260), SHAPE), (dict(ldk=120), SHAPE), (dict(H=65535, total=2 ** 31 - 1), SHAPE)])
def test_rotary(lib, bad, status):
    assert rotary(lib, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(d=32), HEAD_DIM), (dict(block=24), SHAPE), (dict(B=0), SHAPE), (dict(num_blocks=0), SHAPE), (dict(cols=0), SHAPE),
    (dict(Hk=0), SHAPE), (dict(pairs=36), SHAPE), (dict(axes=3), NULL), (dict(turns=None), NULL), (dict(total=0), SHAPE),
    (dict(max_new=0), SHAPE), (dict(B=2 ** 30, max_new=2 ** 20), SHAPE), (dict(q_out=None), NULL), (dict(start=None), NULL),
    (dict(kc=P + 8), ALIGN), (dict(ldv=64), SHAPE), (dict(H=0), SHAPE)])
def test_append(lib, bad, status):
    assert append(lib, **bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(d=32), HEAD_DIM), (dict(block=8), SHAPE), (dict(H=5), SHAPE), (dict(Hk=3), SHAPE), (dict(B=0), SHAPE), (dict(max_new=0), SHAPE),
    (dict(total=0), SHAPE), (dict(max_seqlen=0), SHAPE), (dict(ldq=192), SHAPE), (dict(scale=0.0), SCALE), (dict(scale=-1.0), SCALE),
    (dict(scale=math.nan), SCALE), (dict(scale=math.inf), SCALE), (dict(nbytes=16), WORKSPACE), (dict(ws=None), NULL), (dict(cu=None), NULL),
    (dict(q=P + 8), ALIGN), (dict(ws=P + 8), ALIGN), (dict(total=2 ** 29, H=8), SHAPE), (dict(B=2 ** 30, max_new=2 ** 20, total=2 ** 20), SHAPE),
    (dict(B=2 ** 23 + 1, max_new=2 ** 14, total=2 ** 14), SHAPE)])
def test_chunk(lib, bad, status):
    assert chunk(lib, **bad) == status


def test_in_order_fails_only_for_the_pointers(lib):
    # (host memory: found out without a launch; on a machine without a GPU the query itself fails)
    for call in (rotary, append, chunk):
        assert call(lib) == NOT_DEVICE


def test_workspace(lib):
    f = lib.fa_chunk_cache8_workspace_bytes
    assert f(2, 3, 5, 4, 2, 0, 64) == f(2, 3, 5, 4, 3, 32, 64) == f(2, 3, 5, 4, 2, 32, 80) == 0
    # two partials a CTA of 256 rows (O and two statistics), and a record of each
    one = 2 * 256 * (64 + 2) * 4
    assert f(1, 1, 1, 4, 1, 100, 64) == one + 256
    assert f(4, 1, 4, 4, 1, 10000, 64) == f(2, 700, 1400, 32, 8, 2 ** 31 - 1, 64) == 152 * one + 152 * 32 // 256 * 256
    assert f(2 ** 20, 2 ** 9, 2 ** 12, 65535, 65535, 2 ** 31 - 1, 128) == 2 * 152 * 256 * 130 * 4 + 152 * 32


@pytest.mark.parametrize("f", [1.0, 1e-4, 0.1, 2 * math.pi, 7.5, -1.0, 1e9, 1e-30, 0.0])
def test_frequencies_as_fractions_of_a_turn(f):
    plan = fa.rotary_plan([f] * 8, axis=[0, 1, 2, 0, 1, 2, 0, 1], interleaved=True, device="cpu")
    assert plan.turns.shape == (8,) and plan.axes == 3 and plan.interleaved is True and plan.axis.tolist() == [0, 1, 2, 0, 1, 2, 0, 1]
    pi = Fraction(3141592653589793238462643383279502884197, 10 ** 39)
    turn = Fraction(f) / (2 * pi)
    got = Fraction(int(plan.turns[0]) % 2 ** 64, 2 ** 64)
    off = (got - turn) % 1
    assert min(off, 1 - off) <= Fraction(1, 2 ** 65) + abs(turn) / 2 ** 120


def test_plan_refusals():
    for bad in ([], [1.0] * 7, [float("nan")] * 8, [float("inf")] * 8):
        with pytest.raises(ValueError):
            fa.rotary_plan(bad, device="cpu")
    for bad in ([0] * 7, [-1] * 8, [8] * 8):
        with pytest.raises(ValueError):
            fa.rotary_plan([1.0] * 8, axis=bad, device="cpu")


def test_calls_on_the_host_are_refused(lib):
    plan = fa.rotary_plan([1.0] * 8, device="cpu")
    q, at = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.arange(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        fa.rotary_forward(q, q, at, plan)
    with pytest.raises(TypeError):
        fa.rotary_embedding(q, q, at, plan)
    with pytest.raises(TypeError):
        fa.cache8_store_rotary(q, q, q, fa.Cache8(*[q] * 4), at, at, at, 1, plan)
    with pytest.raises(TypeError):
        fa.attention_chunk_cache8(q, fa.Cache8(*[q] * 4), at, at, at, 1, 1)
