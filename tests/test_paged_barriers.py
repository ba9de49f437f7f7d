"""The hand-over of the Q buffers of the attention over pages (CPU): a model of the barriers' phases
under every order in which the copying warp and the two chains can advance, with the releases of the
kernel's own header.

A wait by parity cannot tell a phase from the next but one: it passes when the phase after the one
that it names is the current one, so a waiter that two phases have passed stands still."""
import ctypes as C
import itertools
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HOST_SRC = r"""
#include "paged_work.cuh"
using namespace fg;
extern "C" int h_at_once(int chain, int single) { return q_given_at_once(chain, single); }
extern "C" int h_after_use(int chain, int single) { return q_given_after_use(chain, single); }
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("barriers")
    src, so = d / "b.cpp", d / "b.so"
    src.write_text(HOST_SRC)
    inc = os.path.join(ROOT, "bit_compressed_throughput_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", inc, str(src), "-o",
                    str(so)], check=True)
    dll = C.CDLL(str(so))
    return dll.h_at_once, dll.h_after_use


def stuck(singles, at_once, after_use):
    """A state from which nothing advances, or None.  singles: per segment, whether its block has one
    row tile.  at_once(chain, single): arrivals at buffer 0's barrier right behind the chain's wait for
    the segment's Q; after_use(chain, single): those at the barrier of the buffer that it multiplies."""
    n = len(singles)
    two_before = [sum(not s for s in singles[:i]) for i in range(n + 1)]
    # (loads issued, (segment, step) of either chain, arrivals at either buffer's barrier).  Steps: 0
    # waits for buffer 0, 1 for buffer 1 (chain 1 of two row tiles), 2 multiplies.
    start = (0, (0, 0), (0, 0), 0, 0)
    seen, todo = {start}, [start]
    while todo:
        loads, *chains, free0, free1 = todo.pop()
        full = (loads, two_before[loads])                    # phases that the loads have completed
        nexts = []
        # the copying warp: buffer 0, and with two row tiles buffer 1, given back by both arrivals
        if loads < n and (loads == 0 or (free0 // 2) % 2 != (loads - 1) % 2) and (
                singles[loads] or full[1] == 0 or (free1 // 2) % 2 != (full[1] - 1) % 2):
            assert free0 >= 2 * loads and (singles[loads] or free1 >= 2 * full[1]), "loaded over"
            nexts.append((loads + 1, *chains, free0, free1))
        for t, (seg, step) in enumerate(chains):
            if seg == n:
                continue
            single, f0, f1 = singles[seg], free0, free1
            if step < 2:
                phase = seg if step == 0 else two_before[seg]
                if full[step] % 2 == phase % 2:              # the named phase is the current one
                    continue
                assert full[step] == phase + 1, "passed too early"
                more = step == 0 and t == 1 and not single
                if not more:
                    f0 += at_once(t, single)
                to = (seg, 1 if more else 2)
            else:
                if t == 0 or single:
                    f0 += after_use(t, single)
                else:
                    f1 += after_use(t, single)
                to = (seg + 1, 0)
            moved = list(chains)
            moved[t] = to
            nexts.append((loads, *moved, f0, f1))
        if not nexts and any(seg < n for seg, _ in chains):
            return loads, chains
        for s in nexts:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return None


@pytest.mark.parametrize("n", [1, 2, 3, 4, 6])
def test_no_order_of_the_chains_stands_still(rules, n):
    for singles in itertools.product((True, False), repeat=n):
        assert stuck(singles, *rules) is None, singles


def test_the_model_finds_a_release_without_the_other_chain():
    """Both arrivals of chain 0 where there are two row tiles: chain 1 may still wait for the buffer
    when the next segment's rows come."""
    at_once = lambda t, single: 0
    after_use = lambda t, single: 1 if single else 2
    assert stuck((True, True, True), at_once, after_use) is None
    assert stuck((False, False), at_once, after_use) is None
    assert stuck((False, True), at_once, after_use) is not None
