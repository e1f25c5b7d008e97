"""The barriers of the prefill kernel as a model: its roles run in random orders, each
with a random slowness, over random lists of runs, and every product's operands are
checked.  An mbarrier wait knows a phase by its parity alone, so a wait that comes a lap
early passes at once; the model shows that the order in which the MMA warps wait rules
that out, and that the order without the first tile's P in front does not."""
import random

import pytest


class Bar:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self, times=1):
        for _ in range(times):
            self.left -= 1
            if self.left == 0:
                self.left, self.phase = self.count, self.phase + 1

    def passed(self, parity):
        return (self.phase & 1) != parity


def simulate(runs, seed, p_first=True):
    """runs: (tiles, narrow) each.  Returns (operands read too early, all roles ended)."""
    rng = random.Random(seed)
    k_full, v_full, q_full, o_full = ([Bar(1), Bar(1)] for _ in range(4))
    k_empty, v_empty = ([Bar(2), Bar(2)] for _ in range(2))
    s_full, p_full = ([[Bar(1), Bar(1)] for _ in range(2)] for _ in range(2))
    q_empty, both = Bar(2), [0]
    k_slot, v_slot, q_slot, bad = [None, None], [None, None], [None, None], []
    total = sum(n for n, _ in runs)

    def unpack(full, empty, slot):
        for t in range(total):
            s, lap = t & 1, t >> 1
            yield lambda: empty[s].passed((lap & 1) ^ 1)
            slot[s] = None  # being written
            yield lambda: True
            slot[s] = t
            full[s].arrive()
            yield lambda: True

    def loads_q(m, r):
        return r < len(runs) and (m == 0 or not runs[r][1])

    def softmax(m):
        s_ph = o_ph = e_ph = 0
        if loads_q(m, 0):
            q_slot[m] = 0
            q_full[m].arrive()
        for r, (n, narrow) in enumerate(runs):
            mine = len(range(m, n, 2)) if narrow else n
            for _ in range(mine):
                for sub in (0, 1):
                    yield lambda: s_full[m][sub].passed(s_ph)
                    yield lambda: True
                    p_full[m][sub].arrive()
                s_ph ^= 1
            if loads_q(m, r + 1):
                yield lambda: q_empty.passed(e_ph)
                q_slot[m] = r + 1
                q_full[m].arrive()
            e_ph ^= 1
            if mine:
                yield lambda: o_full[m].passed(o_ph)
                o_ph ^= 1
            if narrow:
                for _ in range(2):
                    both[0] += 1
                    target = (both[0] + 1) // 2 * 2
                    yield lambda: both[0] >= target

    def mma(m):
        p_ph, q_ph, t0 = 0, [0, 0], 0
        for r, (n, narrow) in enumerate(runs):
            first, step = (m, 2) if narrow else (0, 1)
            yield lambda: q_full[0].passed(q_ph[0])
            q_ph[0] ^= 1
            if not narrow:
                if m == 1:
                    yield lambda: q_full[1].passed(q_ph[1])
                q_ph[1] ^= 1

            def slot(k):
                return (t0 + k) & 1

            def phase(k):
                return ((t0 + k) >> 1) & 1

            def scores(k, sub):
                if k_slot[slot(k)] != t0 + k:
                    bad.append("K")
                if q_slot[0 if narrow else m] != r:
                    bad.append("Q")
                s_full[m][sub].arrive()
                if sub:
                    k_empty[slot(k)].arrive(2 if narrow else 1)
                    if k + step >= n:
                        q_empty.arrive()

            if first < n:
                yield lambda: k_full[slot(first)].passed(phase(first))
                scores(first, 0)
                scores(first, 1)
            else:
                q_empty.arrive()
            for k in range(first, n, step):
                again = k + step < n
                if p_first and k == first:
                    yield lambda: p_full[m][0].passed(p_ph)
                yield lambda: v_full[slot(k)].passed(phase(k))
                if again:
                    yield lambda: k_full[slot(k + step)].passed(phase(k + step))
                for sub in (0, 1):
                    yield lambda: p_full[m][sub].passed(p_ph)
                    if v_slot[slot(k)] != t0 + k:
                        bad.append("V")
                    if sub:
                        v_empty[slot(k)].arrive(2 if narrow else 1)
                    if again:
                        scores(k + step, sub)
                if not again:
                    o_full[m].arrive()
                p_ph ^= 1
            t0 += n

    roles = [unpack(k_full, k_empty, k_slot), unpack(v_full, v_empty, v_slot), softmax(0),
             softmax(1), mma(0), mma(1)]
    slow = [rng.choice([1, 1, 3, 30, 300]) for _ in roles]
    waits = [next(x, None) for x in roles]
    while True:
        ready = [i for i, w in enumerate(waits) if w is not None and w()]
        if not ready:
            return bad, not any(waits)
        i = rng.choices(ready, [1 / slow[j] for j in ready])[0]
        waits[i] = next(roles[i], None)


def lists(n, seed):
    rng = random.Random(seed)
    for k in range(n):
        yield k, [(rng.choice([1, 1, 2, 3, 4, 5, 7]), rng.random() < 0.6)
                  for _ in range(rng.randint(1, 9))]


def test_every_product_reads_its_own_tiles():
    for seed, runs in lists(1500, 1):
        assert simulate(runs, seed) == ([], True), runs


def test_the_model_sees_a_wait_that_passes_a_lap_early():
    wrong = sum(simulate(runs, seed, p_first=False) != ([], True) for seed, runs in lists(600, 2))
    assert wrong > 0


@pytest.mark.parametrize("runs", [[(3, True), (4, True)], [(1, True), (1, True), (2, True)],
                                  [(5, False), (1, True), (3, False), (2, True)]])
def test_short_lists_in_many_orders(runs):
    for seed in range(300):
        assert simulate(runs, seed) == ([], True)
