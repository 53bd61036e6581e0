"""The tree kernel's K / V ring on the CPU: random interleavings of its roles
over barriers whose waits name a phase by parity, as the hardware's do.  Loads
land independently of each other, and a softmax group waits for V only at the
tile that holds its request's end, whose value rows behind the end it zeroes."""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_attention_fp8_gb300", "csrc", "tree.cuh")


class Bar:
    def __init__(self, count=1):
        self.count = self.pending = count
        self.phases = 0  # completed ones

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.phases += 1
            self.pending = self.count

    def wait(self, parity):
        """Passes when the last completed phase has this parity, whichever phase it is."""
        while (self.phases & 1) == (parity & 1):
            yield


class Hazard(AssertionError):
    pass


def expect(ok, *what):
    if not ok:
        raise Hazard(what)


def simulate(seed, stages, lines, guard):
    """One CTA over `lines`, each a list of its segments' tile counts; the last
    tile of a line is its request's end.  guard: the group first waits for the
    slot's previous use."""
    R = random.Random(seed)
    segs = [n for line in lines for n in line]
    ends, at = set(), 0
    for line in lines:
        at += sum(line)
        ends.add(at - 1)
    total = sum(segs)
    k_full, k_empty, v_full, v_empty = ([Bar() for _ in range(stages)] for _ in range(4))
    s_full, p_full = [Bar() for _ in range(3)], [Bar() for _ in range(3)]
    K, V = [None] * stages, [None] * stages  # the tile that landed
    owner = [None] * stages                  # the tile whose load V's slot was last given to
    cleared = set()                          # tiles whose tail rows are zero
    queue, qk_done, pv_done, p_given = [], set(), set(), set()
    tasks = {}

    def load(kv, n):
        slot = n % stages
        for _ in range(R.choice([0, 1, 5, 40])):
            yield
        (V if kv else K)[slot] = n
        (v_full if kv else k_full)[slot].arrive()

    def producer(w, step):
        for n in range(w, total, step):
            slot, odd = n % stages, (n // stages) & 1
            for kv in (0, 1):
                yield from (v_empty if kv else k_empty)[slot].wait(odd ^ 1)
                expect(n < stages or n - stages in (pv_done if kv else qk_done), "slot in use", n, kv)
                (V if kv else K)[slot] = None
                if kv:
                    owner[slot] = n
                tasks[("load", kv, n)] = load(kv, n)
                yield

    def tensor():
        while len(pv_done) < total:
            if queue:
                op = queue.pop(0)
                for _ in range(R.randint(0, 3)):
                    yield
                op()
            yield

    def mma():
        qn, seg_of = 0, [i for i, n in enumerate(segs) for _ in range(n)]
        for n in range(total):
            while qn < total and qn <= n + 2 and seg_of[qn] <= seg_of[n] + 1:
                yield from k_full[qn % stages].wait((qn // stages) & 1)
                expect(K[qn % stages] == qn, "K", qn)

                def qk(j=qn):
                    expect(K[j % stages] == j, "K overwritten", j)
                    qk_done.add(j)
                    s_full[j % 3].arrive()
                    k_empty[j % stages].arrive()
                queue.append(qk)
                qn += 1
                yield
            yield from v_full[n % stages].wait((n // stages) & 1)
            yield from p_full[n % 3].wait((n // 3) & 1)
            expect(V[n % stages] == n and n in p_given, "V or P", n)

            def pv(j=n):
                expect(V[j % stages] == j, "V overwritten", j)
                expect(j not in ends or j in cleared, "tail of V not zero", j)
                pv_done.add(j)
                v_empty[j % stages].arrive()
            queue.append(pv)
            yield

    def softmax(group):
        for j in range(group, total, 2):
            slot, odd = j % stages, (j // stages) & 1
            yield from s_full[j % 3].wait((j // 3) & 1)
            expect(j in qk_done, "S", j)
            for _ in range(R.choice([0, 2, 8])):
                yield
            if j in ends:
                if guard:
                    yield from v_empty[slot].wait(odd ^ 1)
                yield from v_full[slot].wait(odd)
                # Zeros in another tile's slot, or under a load still to land.
                expect(owner[slot] == j and V[slot] == j, "zeroed", owner[slot], "for", j)
                cleared.add(j)
            p_given.add(j)
            p_full[j % 3].arrive()
            yield

    step = min(3, stages)
    tasks.update({("producer", w): producer(w, step) for w in range(step)})
    tasks.update(tensor=tensor(), mma=mma(), even=softmax(0), odd=softmax(1))
    weight = {}
    for _ in range(400000):
        names = list(tasks)
        for x in names:
            weight.setdefault(x, R.choice([1, 1, 5, 20]))
        name = R.choices(names, [weight[x] for x in names])[0]
        try:
            next(tasks[name])
        except StopIteration:
            del tasks[name]
        if not tasks:
            break
    expect(len(pv_done) == total, "hang", sorted(map(str, tasks)))


def lines_of(seed):
    r = random.Random(seed)
    return [[r.choice([1, 1, 2, 3, 5, 9]) for _ in range(r.choice([1, 1, 2]))] for _ in range(r.randint(2, 5))]


def guarded():
    """Whether the kernel's softmax role, with two stages, waits for the slot's previous use before it waits for V."""
    with open(SOURCE) as f:
        return re.search(r"if constexpr \(two_stages<D, R, NP>\(\)\) dead \|= !wait_all\(tVEmpty \+ stage, vphase \^ 1u\);\s+"
                         r"dead \|= !wait_all\(tVFull \+ stage, vphase\);", f.read()) is not None


@pytest.mark.parametrize("stages", range(2, 9))
def test_value_rows_are_zeroed_in_their_own_tile(stages):
    guard = stages == 2 and guarded()
    for seed in range(40):
        simulate(seed, stages, lines_of(seed), guard)


def test_the_model_sees_a_wait_that_does_not_name_its_phase():
    """Without the wait for the slot's previous use, two stages do not hold."""
    seen = 0
    for seed in range(40):
        try:
            simulate(seed, 2, lines_of(seed), False)
        except Hazard:
            seen += 1
    assert seen >= 5
