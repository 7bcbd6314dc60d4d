"""The roles of shared_kernel (two producers, two MMA issuers, two softmax warpgroups) as a model on the CPU: the shares of random
batches are walked as the kernel walks them, the roles' waits and arrivals run against barriers that know a phase by its parity
alone, and whoever may go next is chosen against them.  Every wait must end with the use of the slot that it asked for, and every
product must find its own tile.  The order of the waits in question is read from the source."""
import os
import random
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_io_aware_75_b200", "csrc", "shared_sm100.cu")
S_BUFS = 4


def source_of(name):
    """A function's text in the kernel's source, comments taken out."""
    text = re.sub(r"//[^\n]*", "", open(SRC).read())
    at = re.search(r"__device__ \w+ " + name + r"\(", text).start()
    return text[at:text.index("\n}\n", at)]


def ceil_div(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ the plan
def shares(items, n, d):
    """Of each CTA, its shares in order: (few, warpgroup, pair, blocks, ring).  items: (rows, keys)."""
    few_c, one_c, pair_c = (3, 3, 5) if d == 128 else (3, 4, 8)

    def block(rows):
        return pair_c if rows > 128 else one_c if rows > 16 else few_c
    start, total = [], 0
    for rows, keys in items:
        start.append(total)
        if keys > 0:
            total += ceil_div(keys, 128) * block(rows) + (5 if rows > 32 else 1)
    most = pair_c if any(rows > 128 for rows, _ in items) else one_c
    span = max(most, ceil_div(total, n))
    out = []
    for c in range(n):
        lo, hi, turn, ring, mine = c * span, (c + 1) * span, 0, 0, []
        for (rows, keys), st in zip(items, start):
            nb = ceil_div(keys, 128)
            b0 = 0 if st >= lo else min(nb, ceil_div(lo - st, block(rows)))
            b1 = min(nb, ceil_div(hi - st, block(rows))) if st < hi else 0
            if b0 >= b1:
                continue
            mine.append((rows <= 32, turn, rows > 128, b1 - b0, ring))
            turn ^= rows <= 32
            ring += 2 * (b1 - b0)
        out.append(mine)
    assert sum(s[3] for c in out for s in c) == sum(ceil_div(k, 128) for _, k in items)
    return out


# ----------------------------------------------------------------- the model
class Barrier:
    def __init__(self, count=1):
        self.count, self.pending, self.done = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.done = self.count, self.done + 1

    def passes(self, parity):
        return (self.done & 1) != parity


class Model:
    """One CTA.  Roles are generators; they yield (barrier, parity, uses that must be over) to wait, or None after a step."""

    def __init__(self, work, stages, pv_first, both_q):
        self.work, self.stages, self.pv_first, self.both_q = work, stages, pv_first, both_q
        two = range(2)
        self.kv_full = [Barrier() for _ in range(stages)]
        self.kv_empty = [Barrier(1 if s & 1 else 2) for s in range(stages)]
        self.q_full, self.s_full, self.p_full, self.o_full = ([Barrier() for _ in two] for _ in range(4))
        self.st_full, self.st_empty = ([[Barrier() for _ in range(S_BUFS)] for _ in two] for _ in two)
        self.pt_full, self.pt_empty = ([[Barrier() for _ in two] for _ in two] for _ in two)
        self.join = Barrier(2)
        self.tile = [None] * stages          # (kind, ring position) that a slot holds
        self.loads = {"K": [], "V": []}      # issued, not yet arrived
        self.products = []                   # issued, not yet executed: (slot, tile it must hold) or a barrier to arrive on

    def producer(self, kind):
        it = 0 if kind == "K" else 1
        for *_, nb, _ in self.work:
            for _ in range(nb):
                use = it // self.stages
                yield self.kv_empty[it % self.stages], (use & 1) ^ 1, use
                self.loads[kind].append(it)
                yield None
                it += 2

    def arrivals(self, kind):
        while True:
            if self.loads[kind]:
                it = self.loads[kind].pop(0)
                self.tile[it % self.stages] = (kind, it)
                self.kv_full[it % self.stages].arrive()
                yield None
            else:
                yield "idle"

    def tensor_core(self):
        while True:
            if self.products:
                x = self.products.pop(0)
                if isinstance(x, Barrier):
                    x.arrive()
                else:
                    slot, want = x
                    assert self.tile[slot] == want, f"a product read {self.tile[slot]}, not {want}"
                yield None
            else:
                yield "idle"

    def wait_kv(self, it):
        use = it // self.stages
        return self.kv_full[it % self.stages], use & 1, use + 1

    def product(self, it, *commits):
        self.products.append((it % self.stages, ("V" if it & 1 else "K", it)))
        self.products += commits

    def issuer_s(self):
        q, st, p = [0, 0], [0, 0], [0, 0]

        def wait_q(t):
            q[t] += 1
            return self.q_full[t], (q[t] - 1) & 1, q[t]

        def wait_p(t):
            p[t] += 1
            return self.p_full[t], (p[t] - 1) & 1, p[t]
        for few, wg, pair, nb, it in self.work:
            if few:
                yield wait_q(wg)
                for _ in range(nb):
                    n = st[wg]
                    st[wg] += 1
                    yield self.wait_kv(it)
                    yield self.st_empty[wg][n % S_BUFS], ((n // S_BUFS) & 1) ^ 1, n // S_BUFS
                    self.product(it, self.st_full[wg][n % S_BUFS])
                    yield None
                    it += 2
                continue
            one = not pair and nb == 1
            yield wait_q(0)
            if not one:
                yield wait_q(1)
            prev = None
            for j in range(nb):
                yield self.wait_kv(it)
                v, it = it + 1, it + 2
                if pair:
                    self.product(v - 1, self.s_full[0])
                    if j > 0:
                        yield wait_p(1)
                        self.product(prev, self.kv_empty[prev % self.stages])
                    self.product(v - 1, self.s_full[1])
                    yield self.wait_kv(v)
                    yield wait_p(0)
                    self.product(v, *([self.o_full[0]] if j == nb - 1 else []))
                else:
                    t = j & 1
                    self.product(v - 1, self.s_full[t])
                    if j > 0:
                        yield self.wait_kv(prev)
                        yield wait_p(t ^ 1)
                        self.product(prev, self.kv_empty[prev % self.stages], *([self.o_full[t ^ 1]] if j == nb - 1 else []))
                prev = v
            if one and self.both_q:
                yield wait_q(1)
            t = 1 if pair else (nb - 1) & 1
            if not pair:
                yield self.wait_kv(prev)
            yield wait_p(t)
            self.product(prev, self.kv_empty[prev % self.stages], self.o_full[t])
            yield None

    def issuer_pv(self):
        cnt = [0, 0]
        for few, wg, _, nb, ring in self.work:
            if not few:
                continue
            for j in range(nb):
                it, c = ring + 1 + 2 * j, cnt[wg]
                cnt[wg] += 1
                waits = [(self.pt_full[wg][c & 1], (c >> 1) & 1, (c >> 1) + 1), self.wait_kv(it)]
                yield from waits if self.pv_first else waits[::-1]
                self.product(it, self.kv_empty[it % self.stages], self.pt_empty[wg][c & 1])
                yield None

    def softmax(self, t):
        s = o = n = joins = 0
        for few, wg, pair, nb, ring in self.work:
            if few:
                if wg != t:
                    continue
                self.q_full[t].arrive()
                yield None
                for j in range(nb):
                    yield self.st_full[t][n % S_BUFS], (n // S_BUFS) & 1, n // S_BUFS + 1
                    self.st_empty[t][n % S_BUFS].arrive()
                    for _ in range(2):
                        self.kv_empty[(ring + 2 * j) % self.stages].arrive()
                    yield None
                    yield self.pt_empty[t][n & 1], ((n >> 1) & 1) ^ 1, n >> 1
                    self.pt_full[t][n & 1].arrive()
                    yield None
                    n += 1
                yield self.pt_empty[t][(n - 1) & 1], ((n - 1) >> 1) & 1, ((n - 1) >> 1) + 1
                continue
            j0, step = (0, 1) if pair else (t, 2)
            if j0 < nb or self.both_q:
                self.q_full[t].arrive()
                yield None
            for j in range(j0, nb, step):
                yield self.s_full[t], s & 1, s + 1
                s += 1
                for _ in range(1 if pair else 2):
                    self.kv_empty[(ring + 2 * j) % self.stages].arrive()
                self.p_full[t].arrive()
                yield None
            if j0 < nb:
                yield self.o_full[t], o & 1, o + 1
                o += 1
            joins += 1
            self.join.arrive()
            yield self.join, (joins - 1) & 1, joins

    def run(self, order):
        """Lets the first in `order` that can go make a step, until all roles are done."""
        roles = {"K": self.producer("K"), "V": self.producer("V"), "S": self.issuer_s(), "PV": self.issuer_pv(),
                 "0": self.softmax(0), "1": self.softmax(1), "kin": self.arrivals("K"), "vin": self.arrivals("V"),
                 "mma": self.tensor_core()}
        waits = {}
        while set(roles) & {"K", "V", "S", "PV", "0", "1"}:
            for name in order:
                if name not in roles:
                    continue
                if name in waits:
                    barrier, parity, uses = waits[name]
                    if not barrier.passes(parity):
                        continue
                    assert barrier.done >= uses, f"{name} went on at use {barrier.done} of {uses}"
                    del waits[name]
                try:
                    got = next(roles[name])
                except StopIteration:
                    del roles[name]
                    break
                if got == "idle":
                    continue
                if got is not None:
                    waits[name] = got
                break
            else:
                raise AssertionError(f"nobody can go on: {sorted(waits)}")
        while any(self.loads.values()) or self.products:
            for name in ("kin", "vin", "mma"):
                next(roles[name])


NAMES = ["K", "V", "S", "PV", "0", "1", "kin", "vin", "mma"]


def orders(rng, many):
    """Each one held back in turn (all others go first), and some at random."""
    for last in NAMES:
        rest = [x for x in NAMES if x != last]
        rng.shuffle(rest)
        yield rest + [last]
    for _ in range(many):
        yield rng.sample(NAMES, len(NAMES))


def from_source():
    """(whether P V of few rows waits for P before it waits for V, whether one block of many rows waits for both Q)"""
    pv, s = source_of("mma_issuer_pv"), source_of("mma_issuer")
    return pv.index("sh.pt_full") < pv.index("sh.kv_full"), "sh.q_full[1]" in s


def random_items(rng):
    items, G = [], rng.choice([1, 3, 4, 8, 16, 40])
    for _ in range(rng.randint(0, 3)):                 # groups on their shared pages
        rows = rng.randint(2, 12) * G
        keys = 16 * rng.randint(1, rng.choice([8, 90]))
        items += [(min(256, rows - r), keys) for r in range(0, rows, 256)]
    rng.shuffle(items)
    return items + [(G, rng.choice([0, 1, 128, 129, rng.randint(1, 900)])) for _ in range(rng.randint(1, 10))]


def check(items, n, d, order, pv_first, both_q):
    for mine in shares(items, n, d):
        Model(mine, 4 if d == 128 else 8, pv_first, both_q).run(order)


def test_products_wait_for_their_tiles():
    """Random batches, d = 64 and 128, every role and every arrival late in turn."""
    pv_first, both_q = from_source()
    rng = random.Random(1)
    for _ in range(150):
        items, n, d = random_items(rng), rng.choice([1, 1, 2, 3]), rng.choice([64, 128])
        for order in orders(rng, 4):
            check(items, n, d, order, pv_first, both_q)


def test_few_rows_after_many():
    """Sequences' own pages behind their group's shared ones, V late: the place of a wait that passed a phase too early."""
    pv_first, both_q = from_source()
    late = ["K", "kin", "S", "PV", "0", "1", "mma", "V", "vin"]
    for d in (64, 128):
        for blocks in range(1, 12):
            items = [(48, 128 * blocks)] + [(3, 128)] * 6 + [(200, 128 * blocks), (3, 300), (3, 1)]
            check(items, 1, d, late, pv_first, both_q)


def test_one_block_of_many_rows_after_few():
    """One block of many rows while the other warpgroup still has few rows whose V is late."""
    pv_first, both_q = from_source()
    late = ["K", "kin", "S", "0", "1", "mma", "PV", "V", "vin"]
    for d in (64, 128):
        for keys in range(100, 1500, 100):
            check([(8, 90), (8, keys), (48, 100)], 1, d, late, pv_first, both_q)


def test_the_model_finds_a_wait_too_early():
    """V asked for before P: the model has to show it."""
    rng = random.Random(2)
    with pytest.raises(AssertionError, match="went on at use|a product read"):
        for order in orders(rng, 10):
            check([(48, 128 * 5)] + [(3, 128)] * 6, 1, 128, order, False, True)
