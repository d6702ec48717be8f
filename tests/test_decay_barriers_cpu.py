"""The barriers of the decayed attention's tensor-core kernels under random
schedules of their warps, copies and products.  A wait for a phase of a barrier
that has run two phases on never ends, which a run on a GPU shows only now and
then.  Roles, barriers and the order of waits are those of csrc/decay_tc.cu."""

import os
import random
import re

import pytest

import linear_softmax_attention_gb300 as favor


class Bar:
    """An mbarrier: `count` arrivals end a phase; a wait asks whether the last phase of a parity has ended."""

    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.phase += 1
            self.left = self.count

    def ended(self, parity):
        return (self.phase & 1) != (parity & 1)


def finishes(roles, queues, rng):
    """Runs the roles (generators of waits) and the queues' events in random order; False: stuck."""
    waits = dict.fromkeys(range(len(roles)))
    speed = [rng.choice([1, 1, 1, 0.05]) for _ in roles]
    while waits:
        acts = [(i, None, speed[i]) for i, w in waits.items() if w is None or w[0].ended(w[1])]
        acts += [(None, q, rng.choice([1, 0.3])) for q in queues if q]
        if not acts:
            return False
        i, queue, _ = rng.choices(acts, [a[2] for a in acts])[0]
        if queue is not None:
            queue.pop(0)()
            continue
        try:
            waits[i] = next(roles[i])
        except StopIteration:
            del waits[i]
    return True


def pass_kernel(rng, live, slots, epi=4):
    full = [Bar(1) for _ in range(slots)]
    scores, out, gain, gain_free = Bar(1), Bar(1), Bar(1), [Bar(1), Bar(1)]
    weights, faded, rows, copy, rows_free = Bar(epi), Bar(epi), Bar(epi), Bar(epi), [Bar(epi), Bar(epi)]
    tma, mma, holds = [[] for _ in range(slots)], [], [None] * slots

    def slot(i, kind):
        return (3 * i + kind) % slots

    def ready(i, kind):
        return full[slot(i, kind)], (3 * i + kind) // slots & 1

    def load(i, kind):
        if i < live:
            holds[slot(i, kind)] = None

            def landed():
                holds[slot(i, kind)] = i, kind
                full[slot(i, kind)].arrive()

            tma[slot(i, kind)].append(landed)

    def product(i, kinds, *bars):
        def ended():
            assert all(holds[slot(i, k)] == (i, k) for k in kinds)       # what it reads is still there
            for b in bars:
                b.arrive()

        mma.append(ended)

    def products():
        for i in range(live):
            yield ready(i, 0)
            yield ready(i, 1)
            product(i, (0, 1), scores)
            yield copy, i & 1
            yield ready(i, 2)
            yield weights, i & 1
            product(i, (1, 2), out)
            if i + 1 < live:
                yield faded, i & 1
                product(i, (0, 2), gain, gain_free[i & 1])
            yield rows, i & 1

    def copies():
        for i, kind in [(0, 0), (0, 1), (0, 2), (1, 0), (1, 1)] + [(1, 2)] * (slots == 6):
            load(i, kind)
        for i in range(live):
            yield rows_free[i & 1], i >> 1 & 1
            if i + 1 == live:
                break
            yield gain_free[i & 1], i >> 1 & 1
            for j, kind in [(i + 2, 0), (i + 2, 2), (i + 2, 1)] if slots == 6 else [(i + 1, 2), (i + 2, 1), (i + 2, 0)]:
                load(j, kind)

    def registers():
        copy.arrive()
        for i in range(live):
            yield scores, i & 1
            weights.arrive()
            if i + 1 < live:
                faded.arrive()
            yield out, i & 1
            rows.arrive()
            rows_free[i & 1].arrive()
            if i + 1 < live:
                yield gain, i & 1
                copy.arrive()

    return finishes([products(), copies()] + [registers() for _ in range(epi)], tma + [mma], rng)


def gain_kernel(rng, n, depth_b, depth_c, splits=3, takes=2):
    b_full, b_free = [Bar(1) for _ in range(depth_b)], [Bar(splits) for _ in range(depth_b)]
    c_full, c_free = [Bar(1) for _ in range(depth_c)], [Bar(1) for _ in range(depth_c)]
    split, done, taken = ([Bar(k), Bar(k)] for k in (splits, 1, takes))
    tma_b, tma_c, mma = [[] for _ in range(depth_b)], [[] for _ in range(depth_c)], []

    def products():
        for j in range(n):
            yield c_full[j % depth_c], j // depth_c & 1
            yield split[j & 1], j >> 1 & 1
            if j >= 2:
                yield taken[j & 1], (j - 2) >> 1 & 1

            def ended(j=j):
                done[j & 1].arrive()
                c_free[j % depth_c].arrive()

            mma.append(ended)

    def copies():
        for j in range(n):
            if j >= depth_b:
                yield b_free[j % depth_b], j // depth_b - 1 & 1
            tma_b[j % depth_b].append(b_full[j % depth_b].arrive)
            if j >= depth_c:
                yield c_free[j % depth_c], j // depth_c - 1 & 1
            tma_c[j % depth_c].append(c_full[j % depth_c].arrive)

    def splitting():
        for j in range(n):
            yield b_full[j % depth_b], j // depth_b & 1
            if j >= 2:
                yield done[j & 1], (j - 2) >> 1 & 1
            split[j & 1].arrive()
            b_free[j % depth_b].arrive()

    def taking():
        for j in range(n):
            yield done[j & 1], j >> 1 & 1
            taken[j & 1].arrive()

    roles = [products(), copies()] + [splitting() for _ in range(splits)] + [taking() for _ in range(takes)]
    return finishes(roles, tma_b + tma_c + [mma], rng)


@pytest.mark.parametrize("slots", [5, 6])
def test_a_pass_ends_under_any_schedule(slots):
    rng = random.Random(slots)
    assert all(pass_kernel(rng, rng.randint(0, 9), slots) for _ in range(400))


@pytest.mark.parametrize("depths", [(4, 4), (2, 3)])
def test_the_gains_end_under_any_schedule(depths):
    rng = random.Random(sum(depths))
    assert all(gain_kernel(rng, rng.randint(0, 14), *depths) for _ in range(400))


def test_the_copies_wait_for_barriers_of_their_own():
    # the waits of the model above, in the source
    text = open(os.path.join(os.path.dirname(favor.__file__), "csrc", "decay_tc.cu")).read()
    for section in re.findall(r"// ---- copies.*?\n  \} else", text, re.S):
        waits = re.findall(r"mbar_wait\((\w+)", section)
        assert waits in (["rows_free", "gain_free"], ["b_free", "c_free"]), waits
    assert len(re.findall(r"// ---- copies", text)) == 2
