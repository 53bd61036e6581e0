"""What the tree kernel's producers wait for before their CTA may exit: the last
load of every ring slot, whichever producer warp issued it (csrc/ring.h, compiled
here as host code and run on the states that a given-up wait leaves)."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_attention_fp8_gb300", "csrc")


@pytest.fixture(scope="module")
def last_load(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    src, lib = d / "ring.cpp", d / "ring.so"
    src.write_text('#include "ring.h"\nextern "C" int last_load(const int* next, int warps, int stages, int slot) {\n'
                   "    return pafp8::ring_last_load(next, warps, stages, slot);\n}\n")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).last_load
    return lambda nxt, stages, slot: f((ctypes.c_int * 3)(*(nxt + [0] * (3 - len(nxt)))), len(nxt), stages, slot)


def stalled(seed, stages):
    """A ring some of whose waits gave up: (one past the last tile of each warp
    for K and for V).  All loads have landed: what a wait asks for
    has to be there."""
    r = random.Random(seed)
    warps, total = min(3, stages), r.choice([0, 1, 2, 3, 5, 9, 20, 60])
    qk, pv = r.randint(0, total), 0          # tiles whose products freed their K and V slots
    pv = r.randint(max(0, qk - 3), qk)
    k, v = [0] * warps, [0] * warps
    for w in range(warps):
        stop = r.choice([total, total, r.randint(0, total)])
        n = w
        while n < total and n < stop and n < qk + stages:  # K(n) waits for QK(n - stages)
            k[w] = n + 1
            if n >= pv + stages:                            # V(n) gives up
                break
            v[w] = n + 1
            n += warps
    return k, v


def loads(nxt, stages, slot):
    return [n for n in range(max(nxt + [0])) if n % stages == slot and n < nxt[n % len(nxt)]]


@pytest.mark.parametrize("stages", range(2, 9))
def test_the_last_load_of_a_slot_is_the_one_waited_for(last_load, stages):
    for seed in range(400):
        for nxt in stalled(seed, stages):
            for slot in range(stages):
                have = loads(nxt, stages, slot)
                got = last_load(nxt, stages, slot)
                assert got == (have[-1] if have else -1), (seed, nxt, slot)


@pytest.mark.parametrize("stages", range(2, 9))
def test_a_parity_wait_for_it_ends(last_load, stages):
    """Slots are filled in turn, so the load numbered n of a slot completes phase
    n / stages; a wait for its parity passes when that is the last completed."""
    for seed in range(400):
        for nxt in stalled(seed, stages):
            for slot in range(stages):
                have = loads(nxt, stages, slot)
                n = last_load(nxt, stages, slot)
                if n >= 0 and have == list(range(slot, n + 1, stages)):
                    assert (len(have) - 1) & 1 == (n // stages) & 1


def test_a_warps_own_tiles_do_not_tell():
    """Why the warps have to look at each other's loads: a warp that gave up at
    V(n) would wait for its own K(n - 3), whose slot K(n + 1) has filled since."""
    stuck = set()
    for stages in range(3, 9):
        n, warps = 30, 3
        k = [n + 1 if n % 3 == w else max(m for m in (n + 1, n + 2) if m % 3 == w) + 1 for w in range(3)]
        x = n - warps
        while x >= 0 and x + stages >= n + 1:
            if loads(k, stages, x % stages)[-1] != x:
                stuck.add(stages)
            x -= warps
    assert stuck == {4, 5, 7, 8}
