"""The order of waits between the roles of the cache attention, explored in full
on the host: the barrier and phase of every wait come from the header that the
kernel is compiled with, the roles' sequences are those of the kernel, and every
interleaving of them is followed.  None may end in a wait that nothing can
complete, and no wait may pass on another phase than the awaited one (a parity
tells neighbouring phases apart, no more)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "io_aware_attention_flash_gb300", "csrc", "cache8_phases.h")

DUMP = """
#include <cstdio>
#include "%s"
using namespace fa::cache8;
int main() {
  std::printf("bars %%d %%d %%d\\n", kSBars, kPBars, kPvBars);
  for (int t = 0; t < 16; ++t) {
    const Phase p[5] = {s_full(t), p_full(t), pv_done(t), ring(t, 2), ring(t, 3)};
    for (const Phase& x : p) std::printf("%%d %%u ", x.index, x.parity);
    std::printf("\\n");
  }
}
"""


@pytest.fixture(scope="module")
def phases(tmp_path_factory):
    """kind -> list over tiles of (barrier index, parity)"""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("phases")
    (d / "dump.cpp").write_text(DUMP % HEADER)
    subprocess.run([cxx, "-std=c++17", "-o", str(d / "dump"), str(d / "dump.cpp")], check=True)
    lines = subprocess.run([str(d / "dump")], check=True, capture_output=True, text=True).stdout.splitlines()
    bars = [int(x) for x in lines[0].split()[1:]]
    rows = [[int(x) for x in line.split()] for line in lines[1:]]
    kinds = {n: [(r[2 * i], r[2 * i + 1]) for r in rows] for i, n in enumerate(("S", "P", "PV", "ring2", "ring3"))}
    for n, count in zip(("S", "P", "PV"), bars):
        assert {i for i, _ in kinds[n]} == set(range(count)), n
    return kinds


def scripts(phases, items, stages, threads):
    """The roles as lists of ("wait" | "arrive" | "mma", barrier, parity or arrivals, nth phase of the barrier).
    A barrier is (kind, index); an "mma" is queued on the tensor core, which arrives in order, at any later time."""
    ring = phases[f"ring{stages}"]

    def nth(kind, t, table):  # the how-manieth phase of its barrier tile t stands for
        return sum(table[u][0] == table[t][0] for u in range(t))

    def at(op, kind, t, table):
        return op, (kind, table[t][0]), table[t][1], nth(kind, t, table)

    n_tiles = sum(items)
    load = []
    for t in range(n_tiles):
        if t >= stages:
            load.append(at("wait", "EMPTY", t - stages, ring))
        load.append(("arrive", ("FULL", ring[t][0]), 0, 0))
    mma, soft = [], []
    t = 0
    for i, n in enumerate(items):
        q = ("Q", 0)
        mma.append(("wait", q, i & 1, i))

        def scores(u):
            mma.append(at("wait", "FULL", u, ring))
            mma.append(("mma", (("S", phases["S"][u][0]),), 0, 0))

        scores(t)
        soft += [("arrive", q, 0, 0), ("wait", q, i & 1, i)]
        for k in range(n):
            u = t + k
            if k + 1 < n:
                scores(u + 1)
            mma.append(at("wait", "P", u, phases["P"]))
            mma.append(("mma", (("PV", phases["PV"][u][0]), ("EMPTY", ring[u][0])), 0, 0))
            soft += [at("wait", "FULL", u, ring), at("wait", "S", u, phases["S"]),
                     ("arrive", ("P", phases["P"][u][0]), 0, 0)]
            if k > 0:
                soft.append(at("wait", "PV", u - 1, phases["PV"]))
        soft.append(at("wait", "PV", t + n - 1, phases["PV"]))
        t += n
    return [load, mma] + [soft] * threads


def explore(roles, threads):
    """Follows every interleaving; returns what can go wrong (None if nothing)."""
    need = {"Q": threads, "P": threads}
    bars = sorted({b for r in roles for op in r for b in ([op[1]] if op[0] != "mma" else op[1])})
    slot = {b: i for i, b in enumerate(bars)}

    def arrive(state, b):
        done, pending = state[slot[b]]
        pending += 1
        return state[:slot[b]] + (((done + 1, 0) if pending == need.get(b[0], 1) else (done, pending)),) + state[slot[b] + 1:]

    start = (tuple(0 for _ in roles), 0, tuple((0, 0) for _ in bars))  # places, products completed, barriers
    queue = [op for op in roles[1] if op[0] == "mma"]
    issued_at = [sum(op[0] == "mma" for op in roles[1][:i]) for i in range(len(roles[1]) + 1)]
    todo, known = [start], {start}
    while todo:
        pcs, completed, state = todo.pop()
        after = []
        if completed < issued_at[pcs[1]]:  # the tensor core finishes its oldest product
            s = state
            for b in queue[completed][1]:
                s = arrive(s, b)
            after.append((pcs, completed + 1, s))
        for i, role in enumerate(roles):
            if pcs[i] == len(role):
                continue
            op, b, parity, nth = role[pcs[i]]
            s = state
            if op == "wait":
                done = state[slot[b]][0]
                if done & 1 == parity:
                    continue  # not complete, as far as a parity tells
                if done != nth + 1:
                    return f"role {i} passes phase {nth} of {b} when {done} are complete"
            elif op == "arrive":
                s = arrive(state, b)
            after.append((pcs[:i] + (pcs[i] + 1,) + pcs[i + 1:], completed, s))
        if not after and (any(pc < len(r) for pc, r in zip(pcs, roles)) or completed < len(queue)):
            return f"stuck at {[r[pc] if pc < len(r) else 'end' for pc, r in zip(pcs, roles)]}"
        for x in after:
            if x not in known:
                known.add(x)
                todo.append(x)
    return None


@pytest.mark.parametrize("stages", [2, 3])
@pytest.mark.parametrize("items", [(1,), (2,), (7,), (1, 1, 1, 1), (3, 1, 4), (2, 5)])
def test_no_order_of_the_roles_gets_stuck(phases, items, stages):
    assert explore(scripts(phases, items, stages, 2), 2) is None


def test_the_exploration_finds_a_phase_that_is_passed_by(phases):
    """One barrier for P with the scores issued a tile ahead: the second phase can complete before the first is awaited."""
    one = dict(phases, P=[(0, t & 1) for t in range(16)])
    assert "stuck" in explore(scripts(one, (3,), 3, 2), 2)
