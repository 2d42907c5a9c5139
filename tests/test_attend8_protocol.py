"""The barrier protocol of the 8-bit cache's prefill kernel (csrc/attend8_tc.cu) under random schedules (CPU).

Roles are generators that yield the condition they wait on, copies and products complete after random delays (one issuer's
products in order), and a parity wait succeeds, as the hardware's does, when the barrier's current parity differs from the
waited one: a waiter two phases off would pass early.  Every buffer access is checked: key and byte-value slots, S and P
buffers and f16-value slots hold the pair that their reader expects and are not overwritten before they were read."""
import random

import pytest

from attention_protocol import Bar


class Model:
    def __init__(self, n_union, seed, v16_wait=True):
        self.n, self.pairs = n_union, (n_union + 1) // 2
        self.v16_wait = v16_wait                            # the widening warps wait for PV_DONE of pair p - 2
        self.r = random.Random(seed)
        self.B = {}
        for s in range(2):
            for name, count in (("K_LAND", 1), ("S_FREE", 8), ("QK_DONE", 1), ("V8_LAND", 1), ("V8_FREE", 4), ("V16_READY", 4),
                                ("PV_READY", 8), ("PV_DONE", 1)):
                self.B[name, s] = Bar("%s%d" % (name, s), count)
        self.B["O_FULL", 0] = Bar("O_FULL", 1)
        self.k, self.v8, self.s, self.p, self.v16 = ([None, None] for _ in range(5))
        self.s_reads, self.v8_reads, self.v16_parts = [0, 0], [0, 0], [set(), set()]
        self.p_parts = [set(), set()]
        self.events, self.queues, self.now, self.products = [], {"qk": [], "pv": []}, 0, []

    def later(self, fn):
        self.events.append((self.now + self.r.randint(1, 40), self.r.random(), fn))

    def product(self, who, fn):
        q = self.queues[who]
        q.append(fn)
        self.later(lambda: q.pop(0)())

    def done(self, name, s, phase):
        return lambda: self.B[name, s].done(phase & 1)

    def loader(self, slots, land, freed):
        for p in range(self.pairs):
            s = p & 1
            if p >= 2:
                yield self.done(freed, s, (p >> 1) - 1)
            assert slots[s] is None, "%s slot overwritten" % land
            slots[s] = ("loading", p)
            self.B[land, s].expect_tx(1)

            def landed(s=s, p=p):
                slots[s] = p
                self.B[land, s].complete_tx(1)
            self.later(landed)
            yield None

    def key_issuer(self):
        for p in range(self.pairs):
            s = p & 1
            yield self.done("K_LAND", s, p >> 1)
            if p >= 2:
                yield self.done("S_FREE", s, (p >> 1) - 1)
            assert self.k[s] == p, "key product without its keys"
            assert self.s[s] is None, "S overwritten before it was read"

            def complete(s=s, p=p):
                self.s[s], self.s_reads[s], self.k[s] = p, 0, None
                self.B["QK_DONE", s].arrive()
            self.product("qk", complete)
            yield None

    def value_issuer(self):
        for p in range(self.pairs):
            s = p & 1
            yield self.done("V16_READY", s, p >> 1)
            yield self.done("PV_READY", s, p >> 1)
            want = {2 * p, 2 * p + 1} & set(range(self.n))
            assert self.v16[s] == p and len(self.v16_parts[s]) == 4, "value product without its values"
            assert {c for c, _ in self.p_parts[s]} == want and len(self.p_parts[s]) == 4 * len(want), "value product without its P"

            def complete(s=s, p=p):
                self.products.append(p)
                self.v16[s], self.p_parts[s] = None, set()
                self.B["PV_DONE", s].arrive()
            self.product("pv", complete)
            yield None
        self.product("pv", lambda: self.B["O_FULL", 0].arrive())

    def widen(self, w):
        for p in range(self.pairs):
            s = p & 1
            yield self.done("V8_LAND", s, p >> 1)
            if p >= 2 and self.v16_wait:
                yield self.done("PV_DONE", s, (p >> 1) - 1)
            assert self.v8[s] == p, "widening another pair"
            assert self.v16[s] in (None, p), "f16 values overwritten before their product"
            if self.v16[s] is None:
                self.v16[s], self.v16_parts[s] = p, set()
            self.v16_parts[s].add(w)
            self.v8_reads[s] += 1
            if self.v8_reads[s] == 4:
                self.v8[s], self.v8_reads[s] = None, 0
            yield None
            self.B["V8_FREE", s].arrive()
            self.B["V16_READY", s].arrive()

    def softmax(self, w):
        for t in range(w // 4, self.n, 3):
            p, s = t >> 1, (t >> 1) & 1
            lone = t == self.n - 1 and not t & 1
            yield self.done("QK_DONE", s, p >> 1)
            assert self.s[s] == p, "softmax reads another pair's scores"
            self.s_reads[s] += 2 if lone else 1
            if self.s_reads[s] == 8:
                self.s[s] = None
            self.B["S_FREE", s].arrive()
            yield None
            if p >= 2:
                yield self.done("PV_DONE", s, (p >> 1) - 1)
            assert all(c >> 1 == p for c, _ in self.p_parts[s]), "P overwritten before its product"
            self.p_parts[s].add((t, w % 4))
            yield None
            self.B["PV_READY", s].arrive()
            if lone:
                self.B["PV_READY", s].arrive()
        yield self.done("O_FULL", 0, 0)
        assert self.products == list(range(self.pairs)), "the result is read before every product is done"

    def run(self):
        roles = {"k": self.loader(self.k, "K_LAND", "QK_DONE"), "v": self.loader(self.v8, "V8_LAND", "V8_FREE"),
                 "qk": self.key_issuer(), "pv": self.value_issuer()}
        roles.update({"w%d" % w: self.widen(w) for w in range(4)})
        roles.update({"s%d" % w: self.softmax(w) for w in range(12)})
        waiting = dict.fromkeys(roles)
        for _ in range(200000):
            if not roles:
                return
            ready = [x for x in roles if waiting[x] is None or waiting[x]()]
            if self.events and (not ready or self.r.random() < 0.3):
                self.events.sort(key=lambda e: e[:2])
                t, _, fn = self.events.pop(self.r.randrange(min(3, len(self.events))))
                self.now = max(self.now, t)
                fn()
                continue
            assert ready, "deadlock: %s" % sorted(roles)
            x = self.r.choice(ready)
            self.now += 1
            try:
                waiting[x] = next(roles[x])
            except StopIteration:
                del roles[x]
        raise AssertionError("no completion within the step limit")


@pytest.mark.parametrize("n_union", list(range(1, 20)) + [40])
def test_no_schedule_races_or_stops(n_union):
    for seed in range(12):
        Model(n_union, 1000 * n_union + seed).run()


def test_the_model_sees_a_missing_wait():
    bad = 0
    for seed in range(60):
        try:
            Model(9 + seed % 8, seed, v16_wait=False).run()
        except AssertionError:
            bad += 1
    assert bad > 0
