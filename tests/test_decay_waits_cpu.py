"""Models of the decayed attention's tensor-core kernels under random schedules, with
the paths of rare inputs (rows behind a sequence's end, products done again after
infinities) and with waits that run out.  Which barrier and parity each wait asks
for, and which barrier each arrival goes to, are read out of csrc/decay_tc.cu; the
roles' order is written down here.

Held at every step: what a product or a copy reads is what it should be.  Held at
the end, whatever has run out: every role ends, and nothing is in flight when the
CTA's memory goes."""

import os
import random
import re

import pytest

import linear_softmax_attention_gb300 as favor

SOURCE = open(os.path.join(os.path.dirname(favor.__file__), "csrc", "decay_tc.cu")).read()
CALLS = ("mbar_wait", "mbar_arrive", "mbar_arrive_expect_tx", "mma_commit", "drain", "named_bar", "named_bar_or")


def arguments(text, at):
    """The arguments of the call whose parenthesis opens at `at`."""
    depth, args, start = 0, [], at + 1
    for i in range(at, len(text)):
        depth += (text[i] in "([{") - (text[i] in ")]}")
        if depth == 0:
            return args + [text[start:i].strip()]
        if depth == 1 and text[i] == ",":
            args.append(text[start:i].strip())
            start = i + 1
    raise AssertionError("no end")


def expression(c):
    """C as Python"""
    c = re.sub(r"\s+", " ", c).replace("C::", "C.").replace("/", "//")
    return compile(c, c, "eval")


def section(kernel, start, end):
    """The calls from one mark of a kernel to another, in the text's order."""
    text = SOURCE[SOURCE.index(kernel):]
    text = text[text.index(start):]
    text = text[:text.index(end, 1)]
    text = re.sub(r"//[^\n]*", "", text)
    return [(m[1], [a for a in arguments(text, m.end() - 1)])
            for m in re.finditer(r"\b(" + "|".join(CALLS) + r")\(", text)]


PASS, GAIN = "void pass_body(", "decay_tc_gain_kernel(const"
SECTIONS = {
    ("pass", "products"): section(PASS, "// ---- products", "// ---- copies"),
    ("pass", "copies"): section(PASS, "// ---- copies", "const int q = warp & 3"),
    ("pass", "start"): section(PASS, "// The state's copy for I = A M", "// ---- the weights"),
    ("pass", "weights"): section(PASS, "// ---- the weights", "// ---- b's faded rows"),
    ("pass", "faded"): section(PASS, "// ---- b's faded rows", "// ---- rows out"),
    ("pass", "rows"): section(PASS, "// ---- rows out", "// ---- the next chunk's copy"),
    ("pass", "next"): section(PASS, "// ---- the next chunk's copy", "// rows of chunks behind"),
    ("gain", "products"): section(GAIN, "// ---- products", "// ---- copies"),
    ("gain", "copies"): section(GAIN, "// ---- copies", "// ---- b's rows in three parts"),
    ("gain", "split"): section(GAIN, "// ---- b's rows in three parts", "// ---- the sums"),
    ("gain", "sums"): section(GAIN, "// ---- the sums", "tmem_dealloc"),
}
# the calls that the roles below make, in the text's order
ORDER = {
    ("pass", "products"): "mbar_wait mbar_wait mma_commit mbar_wait mbar_wait mbar_wait mma_commit mbar_wait mma_commit "
                          "mma_commit mbar_wait mma_commit drain",
    ("pass", "copies"): "mbar_arrive_expect_tx mbar_wait mbar_wait drain",
    ("pass", "start"): "mbar_arrive named_bar named_bar",
    ("pass", "weights"): "mbar_wait mbar_wait named_bar mbar_arrive",
    ("pass", "faded"): "mbar_arrive",
    ("pass", "rows"): "mbar_wait named_bar_or mbar_wait named_bar named_bar mma_commit mbar_wait drain mbar_arrive "
                      "mbar_arrive",
    ("pass", "next"): "mbar_wait",
    ("gain", "products"): "mbar_wait mbar_wait mbar_wait mma_commit mma_commit mma_commit drain",
    ("gain", "copies"): "mbar_wait mbar_arrive_expect_tx mbar_wait mbar_arrive_expect_tx drain drain",
    ("gain", "split"): "mbar_wait mbar_wait mbar_wait mbar_arrive mbar_arrive",
    ("gain", "sums"): "mbar_wait mbar_arrive",
}


@pytest.mark.parametrize("where", sorted(SECTIONS))
def test_the_roles_make_the_sources_calls(where):
    assert " ".join(name for name, _ in SECTIONS[where]) == ORDER[where]


def test_the_barriers_counts():
    text = re.sub(r"\s+", " ", SOURCE)
    assert ("for (int i = 0; i < 10; ++i) mbar_init(full + i, 1); for (int i = 10; i < 14; ++i) mbar_init(full + i, "
            "C::kEpiWarps); mbar_init(end_bar, 1); for (int i = 0; i < 2; ++i) { mbar_init(rows_free + i, C::kEpiWarps); "
            "mbar_init(gain_free + i, 1); }") in text
    assert ("for (int i = 0; i < 23; ++i) { const bool splits = (i >= 8 && i < 12) || i == 16 || i == 17; mbar_init("
            "b_full + i, splits ? kSplitWarps : i == 20 || i == 21 ? kTakeWarps : 1); }") in text


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


class Bars:
    """Neighbouring barriers, of which + picks one."""

    def __init__(self, n, count):
        self.bars = [Bar(count) for _ in range(n)]

    def __add__(self, i):
        return self.bars[i]

    __getitem__ = __add__


class Kernel:
    """Roles (generators of waits) and queues of what is in flight."""

    def __init__(self, rng, name, expire):
        self.rng, self.name, self.expire = rng, name, expire
        self.abort = False
        self.env = {}
        self.queues, self.compiled = [], {}

    def code(self, where, n, arg):
        key = (where, n, arg)
        if key not in self.compiled:
            self.compiled[key] = expression(SECTIONS[self.name, where][n][1][arg])
        return self.compiled[key]

    def bar(self, where, n, **local):
        """The barrier of the n-th call of a section"""
        return eval(self.code(where, n, 0), {**self.env, **local})

    def wait(self, where, n, **local):
        """(barrier, parity, may run out) of the n-th call of a section"""
        assert SECTIONS[self.name, where][n][0] in ("mbar_wait", "drain")
        return (self.bar(where, n, **local), eval(self.code(where, n, 1), {**self.env, **local}),
                SECTIONS[self.name, where][n][0] == "mbar_wait")

    def queue(self):
        self.queues.append([])
        return self.queues[-1]

    def expect(self, ok, *what):
        assert ok or self.abort, what

    def run(self, roles):
        """False: stuck, or something was in flight at the end"""
        rng, waits, answers = self.rng, dict.fromkeys(range(len(roles))), {}
        speed = [rng.choice([1, 1, 1, 0.05]) for _ in roles]
        slow = [rng.choice([1, 0.3, 0.003]) for _ in self.queues]
        while waits:
            acts = []
            for i, w in waits.items():
                if w is None or w[0].ended(w[1]):
                    acts.append((i, True, speed[i]))
                elif w[2] and self.abort:
                    acts.append((i, False, speed[i]))
                elif w[2] and self.expire:
                    acts.append((i, False, 0.002))
            acts += [(None, q, s) for q, s in zip(self.queues, slow) if q]
            if not acts:
                return False
            i, what, _ = rng.choices(acts, [a[2] for a in acts])[0]
            if i is None:
                what.pop(0)()
                continue
            if not what:
                self.abort = True
            try:
                waits[i] = roles[i].send(None if waits[i] is None else what)
            except StopIteration:
                del waits[i]
        return not any(self.queues)


class Namespace:
    def __init__(self, **kw):
        self.__dict__.update(kw)


def pass_kernel(rng, live, slots, expire, drains=True, epi=4):
    """drains=False: what is in flight is waited for only by roles whose own waits have run out."""
    k = Kernel(rng, "pass", expire)
    again_of = {i for i in range(live) if rng.random() < 0.15}
    cleared_of = rng.choice([None, 0, live - 1])
    full = Bars(slots, 1)
    one = {n: Bar(1) for n in ("scores", "out_bar", "gain_bar", "again_bar", "end_bar")}
    many = {n: Bar(epi) for n in ("weights_done", "faded_done", "rows_done", "copy_done")}
    named = {5: Bar(epi)}
    tma, mma, mma_again, store = [k.queue() for _ in range(slots)], k.queue(), k.queue(), k.queue()
    stores = Bar(1)                                       # stands for bulk_wait_read0 and bulk_wait0
    holds, tm, issued = [None] * slots, {"image": None, "P": None, "O": None, "M": 0}, {}

    def slot(i, kind):
        return (3 * i + kind) % slots

    def slot_phase(i, kind):
        return (3 * i + kind) // slots & 1

    k.env = dict(full=full, rows_free=Bars(2, epi), gain_free=Bars(2, 1), slot_phase=slot_phase,
                 slot_full=lambda i, kind: full[slot(i, kind)], phases=0, **one, **many)

    def landed(i, kind):
        holds[slot(i, kind)] = i, kind
        full[slot(i, kind)].arrive()

    def load(i, kind):
        if i < live:
            issued[slot(i, kind)] = slot_phase(i, kind)
            holds[slot(i, kind)] = None
            tma[slot(i, kind)].append(lambda: landed(i, kind))

    def product(reads, writes, *bars):
        def ended():
            for where, what in reads:
                have = holds[where] if isinstance(where, int) else tm[where]
                k.expect(have == what, where, have, what)
            tm.update(writes)
            for b in bars:
                b.arrive()
        return ended

    def products():
        ok = True
        for i in range(live):
            w = lambda n: k.wait("products", n, i=i)
            ok = (yield w(0)) and (yield w(1))
            if not ok:
                break
            mma.append(product([(slot(i, 0), (i, 0)), (slot(i, 1), (i, 1))], {"P": ("scores", i)}, k.bar("products", 2)))
            ok = yield w(3)
            if not ok:
                break
            mma.append(product([(slot(i, 1), (i, 1)), ("image", i)], {"I": i}))
            ok = (yield w(4)) and (yield w(5))
            if not ok:
                break
            mma.append(product([("P", ("weights", i)), (slot(i, 2), ("clean", i) if i == cleared_of else (i, 2))],
                               {"O": i}, k.bar("products", 6)))
            if i + 1 < live:
                ok = yield w(7)
                if not ok:
                    break
                # the whole state for the next chunk; b's rows are faded by all warps
                mma.append(product([(slot(i, 0), ("faded", i)), (slot(i, 2), ("clean", i) if i == cleared_of else (i, 2))],
                                   {"M": i + 1}, k.bar("products", 8), k.bar("products", 9, i=i)))
            ok = yield w(10)
            if not ok:
                break
        if not ok or (drains and k.abort):
            mma.append(k.bar("products", 11).arrive)
            yield k.wait("products", 12)

    def copies():
        for i, kind in [(0, 0), (0, 1), (0, 2), (1, 0), (1, 1)] + [(1, 2)] * (slots == 6):
            load(i, kind)
        ok, out = True, 0
        for i in range(live):
            ok = yield k.wait("copies", 1, i=i)
            if not ok:
                break

            def left(i=i):
                k.expect(holds[slot(i, 1)] == ("rows", i), "store", i, holds[slot(i, 1)])
                stores.arrive()

            store.append(left)
            out += 1
            if i + 1 == live:
                break
            ok = yield k.wait("copies", 2, i=i)
            if not ok:
                break
            for j, kind in [(i + 2, 0), (i + 2, 2)] if slots == 6 else [(i + 1, 2), (i + 2, 1)]:
                load(j, kind)
            while stores.phase < out:
                yield stores, stores.phase & 1, False
            load(i + 2, 1 if slots == 6 else 0)
        while stores.phase < out:
            yield stores, stores.phase & 1, False
        if not ok or (drains and k.abort):
            for x, phase in issued.items():
                yield k.bar("copies", 3, x=x), eval(k.code("copies", 3, 1), {"phases": phase << x, "x": x}), False

    def together(n):
        """bar.sync among the warps that share the registers' work"""
        b = named[n]
        parity = b.phase & 1
        b.arrive()
        yield b, parity, False

    count = {}

    def all_warps(what):
        """True for the last warp that comes here"""
        count[what] = count.get(what, 0) + 1
        return count[what] == epi

    def registers(warp):
        again = 0

        def copy_state(i):
            k.expect(tm["M"] == i, "state", i, tm["M"])
            tm["image"] = i if all_warps(("image", i)) else None
            k.bar("start", 0).arrive()

        if live:
            yield from together(5)
            yield from together(5)
            copy_state(0)
        for i in range(live):
            if i == cleared_of:
                yield k.wait("weights", 0, i=i)
                k.expect(holds[slot(i, 2)] in ((i, 2), ("clean", i)), "clear", i)
                if all_warps(("clear", i)):
                    holds[slot(i, 2)] = "clean", i
            yield k.wait("weights", 1, i=i)
            k.expect(tm["P"] == ("scores", i) or warp != 0 or count.get(("P", i), 0) > 0, "scores", i)
            # (the bar of the warps of the same lanes, named 1 + q, lies between their loads and their stores)
            if all_warps(("P", i)):
                tm["P"] = "weights", i
            k.bar("weights", 3).arrive()
            if i + 1 < live:
                k.expect(holds[slot(i, 0)] in ((i, 0), ("faded", i)), "fade", i)
                if all_warps(("fade", i)):
                    holds[slot(i, 0)] = "faded", i
                k.bar("faded", 0).arrive()
            yield k.wait("rows", 0, i=i)
            patch = False
            while True:
                k.expect(tm["O"] == (("again", i) if patch else i), "rows", i, tm["O"])
                k.expect(tm["P"] == ("weights", i), "weights", i)
                if all_warps(("rows", i, patch)):
                    holds[slot(i, 1)] = "rows", i
                yield from together(5)
                if patch or i not in again_of:
                    break
                if i + 1 < live:
                    yield k.wait("rows", 2, i=i)
                yield from together(5)
                if all_warps(("c", i)):
                    k.expect(holds[slot(i, 2)] in ((i, 2), ("clean", i)), "patched", i)
                    holds[slot(i, 2)] = "patched", i
                yield from together(5)
                made = warp == 0 and not k.abort
                if made:
                    mma_again.append(product([("P", ("weights", i)), (slot(i, 2), ("patched", i))], {"O": ("again", i)},
                                             k.bar("rows", 5)))
                if not (yield k.wait("rows", 6, again=again)) and made and drains:
                    yield k.wait("rows", 7, again=again)
                again += 1
                patch = True
            k.bar("rows", 8).arrive()
            k.bar("rows", 9, i=i).arrive()
            if i + 1 < live:
                yield k.wait("next", 0, i=i)
                copy_state(i + 1)

    return k.run([products(), copies()] + [registers(w) for w in range(epi)])


def gain_kernel(rng, n, depth_b, depth_c, expire, drains=True, splits=3, takes=2):
    k = Kernel(rng, "gain", expire)
    cleared_of = {j for j in range(n) if rng.random() < 0.2}
    b_full, c_full, c_free = Bars(depth_b, 1), Bars(depth_c, 1), Bars(depth_c, 1)
    k.env = dict(b_full=b_full, c_full=c_full, b_free=Bars(depth_b, splits), c_free=c_free, split=Bars(2, splits),
                 done=Bars(2, 1), taken=Bars(2, takes), end_bar=Bar(1), C=Namespace(kDepthB=depth_b, kDepthC=depth_c))
    tma_b, tma_c, mma = [k.queue() for _ in range(depth_b)], [k.queue() for _ in range(depth_c)], k.queue()
    tile_b, tile_c, parts, acc, count = [None] * depth_b, [None] * depth_c, [None] * 2, [None] * 2, {}
    m = re.search(r"uint64_t\* const waits\[3\] = \{(.*?)\};", SOURCE)
    waits = expression("[" + m[1] + "]")

    def all_warps(what, of):
        count[what] = count.get(what, 0) + 1
        return count[what] == of

    def products():
        ok = True
        for j in range(n):
            k.env["waits"] = eval(waits, {**k.env, "j": j})
            local = dict(waits=k.env["waits"], j=j)
            ok = (yield k.wait("products", 0, **local)) and (yield k.wait("products", 1, **local))
            if ok and j >= 2:
                ok = yield k.wait("products", 2, **local)
            if not ok:
                break

            def ended(j=j, done=k.bar("products", 3, j=j), free=k.bar("products", 4, j=j)):
                k.expect(parts[j & 1] == j and tile_c[j % depth_c] == (("clean", j) if j in cleared_of else j), "product", j)
                acc[j & 1] = j
                done.arrive()
                free.arrive()

            mma.append(ended)
        if drains or not ok:
            mma.append(k.bar("products", 5).arrive)
            yield k.wait("products", 6)

    def landed(tile, x, j, bar):
        tile[x] = j
        bar.arrive()

    def copies():
        ok, j, jc = True, 0, 0
        for _ in range(n):
            nb, nc = j // depth_b, jc // depth_c
            if nb > 0:
                ok = yield k.wait("copies", 0, j=j, nb=nb)
                if not ok or (drains and k.abort):
                    ok = False
                    break
            tile_b[j % depth_b] = None
            tma_b[j % depth_b].append(lambda j=j, bar=k.bar("copies", 1, j=j): landed(tile_b, j % depth_b, j, bar))
            j += 1
            if nc > 0:
                ok = yield k.wait("copies", 2, jc=jc, nc=nc)
                if not ok:
                    break
            tile_c[jc % depth_c] = None
            tma_c[jc % depth_c].append(lambda j=jc, bar=k.bar("copies", 3, jc=jc): landed(tile_c, j % depth_c, j, bar))
            jc += 1
        if drains or not ok:
            for x in range(min(depth_b, j)):
                yield k.wait("copies", 4, k=x, j=j)
            for x in range(min(depth_c, jc)):
                yield k.wait("copies", 5, k=x, jc=jc)

    def splitting():
        for j in range(n):
            yield k.wait("split", 0, j=j)
            if j >= 2:
                yield k.wait("split", 1, j=j)
            k.expect(tile_b[j % depth_b] == j and acc[j & 1] in ((None,) if j < 2 else (j - 2, j)), "split", j)
            if all_warps(("split", j), splits):
                parts[j & 1] = j
            if j in cleared_of:
                yield k.wait("split", 2, j=j)
                k.expect(tile_c[j % depth_c] in (j, ("clean", j)), "clear", j)
                if all_warps(("clear", j), splits):
                    tile_c[j % depth_c] = "clean", j
            k.bar("split", 3, j=j).arrive()
            k.bar("split", 4, j=j).arrive()

    def sums():
        for j in range(n):
            yield k.wait("sums", 0, j=j)
            k.expect(acc[j & 1] == j, "sum", j)
            k.bar("sums", 1, j=j).arrive()

    return k.run([products(), copies()] + [splitting() for _ in range(splits)] + [sums() for _ in range(takes)])


@pytest.mark.parametrize("slots", [5, 6])
def test_passes_read_what_they_should(slots):
    rng = random.Random(slots)
    assert all(pass_kernel(rng, rng.randint(0, 9), slots, False) for _ in range(300))


@pytest.mark.parametrize("depths", [(4, 4), (2, 3)])
def test_gains_read_what_they_should(depths):
    rng = random.Random(sum(depths))
    assert all(gain_kernel(rng, rng.randint(0, 14), *depths, False) for _ in range(300))


@pytest.mark.parametrize("slots", [5, 6])
def test_passes_whose_waits_run_out_leave_nothing_in_flight(slots):
    rng = random.Random(slots + 10)
    assert all(pass_kernel(rng, rng.randint(0, 4), slots, True) for _ in range(1500))
    # the last waits are what it takes
    assert not all(pass_kernel(rng, rng.randint(0, 4), slots, True, drains=False) for _ in range(1500))


@pytest.mark.parametrize("depths", [(4, 4), (2, 3)])
def test_gains_whose_waits_run_out_leave_nothing_in_flight(depths):
    rng = random.Random(sum(depths) + 10)
    assert all(gain_kernel(rng, rng.randint(0, 7), *depths, True) for _ in range(1500))
    assert not all(gain_kernel(rng, rng.randint(0, 7), *depths, True, drains=False) for _ in range(1500))


def test_the_last_waits_of_the_source():
    text = re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", SOURCE))
    assert "if (!ok || *abort_flag) { mma_commit(end_bar); drain(end_bar, 0); }" in text
    assert "bulk_wait0(); if (!ok || *abort_flag) for (int x = 0; x < C::kSlots; ++x) if (issued >> x & 1) drain(" in text
    assert "} mma_commit(end_bar); drain(end_bar, 0); } __syncwarp();" in text
    assert "} for (int k = 0; k < C::kDepthB && k < j; ++k) drain(" in text
    assert "(nb - 1) & 1, wctx) && !*abort_flag)) break;" in text
