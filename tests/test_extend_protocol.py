"""Event model of the chunk-attention kernel's barriers (CPU).

The kernel's roles (feed, key and value decoders, product, softmax groups by
turns) meet at mbarriers and wait by phase parity, which tells only two neighbouring phases
of a barrier apart.  Here the roles run in random order, copies land in random
order and products finish in issue order; every use of a buffer checks that it
holds what its user expects.  As controls, barriers shared by keys and values
(with an odd number of places), one barrier for both logit buffers and a wait for
the last product by the group that has not seen the one two before it fail."""
import random

import pytest


class Bar:
    def __init__(self, count):
        self.count = self.left = count
        self.done = 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.done, self.left = self.done + 1, self.count

    def ready(self, parity):                   # what a try_wait on that parity answers
        return (self.done & 1) != parity


def run(mode, groups, n_raw, n, seed, slots=4, shared=False, one_done=False, all_wait=False):
    """mode 0: accumulators with rows of their own; 1: on alternate tiles; 2: one step a tile."""
    r = random.Random(seed)
    per = 1 if mode == 2 else 2                # softmax steps of a tile
    k_raw, k_slot = (n_raw, slots) if shared else (2 * n_raw, 2 * slots)
    raw_full, raw_empty = [Bar(1) for _ in range(k_raw)], [Bar(4) for _ in range(n_raw)]
    kv_full, kv_empty = [Bar(4) for _ in range(slots)], [Bar(1) for _ in range(k_slot)]
    s_full, p_full, o_done = ([[Bar(1), Bar(1)] for _ in range(2)] for _ in range(3))
    turn, settled = [Bar(1), Bar(1)], [-1, -1]  # the last step whose reference is known
    raw, slot = [None] * n_raw, [(None, 0)] * slots
    logits = [[None, None], [None, None]]      # what each buffer holds: ("S" or "P", step)
    flying, queue = [], []
    products = [set(), set()]
    uses = {i: (per if i & 1 else 1) * (groups if mode == 0 else 1) for i in range(2 * n)}
    steps = [((n - s + 1) // 2 if mode == 1 else n) * per for s in range(groups)]

    def tile(s, k):
        return 2 * (k // per) + s if mode == 1 else k // per

    def feed():
        for i in range(2 * n):
            while not raw_empty[i % n_raw].ready(((i // n_raw) & 1) ^ 1):
                yield
            flying.append(i)
            yield

    def decoder(kind):
        for i in range(kind, 2 * n, 2):
            while not raw_full[i % k_raw].ready((i // k_raw) & 1):
                yield
            assert raw[i % n_raw] == i, "codes"
            b = i - slots
            while b >= 0 and not kv_empty[b % k_slot].ready((b // k_slot) & 1):
                yield
            held, done = slot[i % slots]
            if held != i:
                assert held is None or (held == b and uses[b] == 0), "slot still in use"
                slot[i % slots] = (i, 1)
            else:
                slot[i % slots] = (i, done + 1)
            yield
            assert raw[i % n_raw] == i, "codes overwritten"
            raw_empty[i % n_raw].arrive()
            kv_full[i % slots].arrive()
            yield

    def product():
        ahead = 2 if per == 1 else 1
        for i in range(steps[0] // per + ahead):
            for s in range(groups):
                tiles = steps[s] // per
                if i >= ahead and i - ahead < tiles:
                    for h in range(per):
                        v = (i - ahead) * per + h
                        n_ = 2 * tile(s, v) + 1
                        while h == 0 and not kv_full[n_ % slots].ready((n_ // slots) & 1):
                            yield
                        assert slot[n_ % slots] == (n_, 4), "values"
                        while not p_full[s][v & 1].ready((v >> 1) & 1):
                            yield
                        assert logits[s][v & 1] == ("P", v), "weights"
                        last = h == per - 1 and (mode != 0 or s == groups - 1)
                        queue.append(("pv", s, v, n_, last))
                        yield
                if i < tiles:
                    n_ = 2 * tile(s, i * per)
                    while not kv_full[n_ % slots].ready((n_ // slots) & 1):
                        yield
                    assert slot[n_ % slots] == (n_, 4), "keys"
                    queue.append(("qk", s, i, n_, mode != 0 or s == groups - 1))
                    yield

    def softmax(s, side):
        def done(k):
            return o_done[s][0].ready(k & 1) if one_done else o_done[s][k & 1].ready((k >> 1) & 1)

        for k in range(side, steps[s], 2):
            while not s_full[s][side].ready((k >> 1) & 1):
                yield
            assert logits[s][side] == ("S", k), "logits"
            while k and not turn[s].ready((k - 1) & 1):
                yield
            assert settled[s] == k - 1, "reference"
            if k and r.random() < 0.5:         # the maximum moves: the accumulator is rescaled
                while not done(k - 1):
                    yield
                assert k - 1 in products[s], "accumulator not ready"
                assert max(products[s]) == k - 1, "accumulator moved on"
            yield
            settled[s] = k
            turn[s].arrive()
            yield
            assert logits[s][side] == ("S", k), "logits"
            logits[s][side] = ("P", k)
            p_full[s][side].arrive()
            yield
        if steps[s] and (all_wait or (steps[s] - 1) & 1 == side):
            while not done(steps[s] - 1):
                yield
            assert steps[s] - 1 in products[s], "result read too early"

    roles = [feed(), product()] + [softmax(s, side) for s in range(groups) for side in (0, 1)] + [decoder(k) for k in (0, 1) for _ in range(4)]
    idle = 0
    while roles:
        x = r.random()
        if x < 0.15 and flying:
            i = flying.pop(r.randrange(len(flying)))
            raw[i % n_raw] = i
            raw_full[i % k_raw].arrive()
            idle = 0
            continue
        if x < 0.3 and queue:
            what, s, u, i, last = queue.pop(0)
            assert slot[i % slots][0] == i, "operand overwritten"
            uses[i] -= 1
            if what == "qk":
                for v in range(u * per, (u + 1) * per):
                    logits[s][v & 1] = ("S", v)
                    s_full[s][v & 1].arrive()
            else:
                assert logits[s][u & 1] == ("P", u), "weights overwritten"
                products[s].add(u)
                o_done[s][0 if one_done else u & 1].arrive()
            if last:
                kv_empty[i % k_slot].arrive()
            idle = 0
            continue
        g = r.choice(roles)
        try:
            next(g)
        except StopIteration:
            roles.remove(g)
        idle += 1
        assert idle < 100000, "stuck"


# two row tiles; one of them empty; alternate key tiles; heads of 256
@pytest.mark.parametrize("mode,groups", [(0, 2), (0, 1), (1, 2), (2, 1)])
@pytest.mark.parametrize("n_raw", [2, 3, 7])
def test_roles_never_meet_a_wrong_buffer(mode, groups, n_raw):
    for n in (1, 2, 3, 5, 17):
        for seed in range(12):
            run(mode, groups, n_raw, n, seed)


@pytest.mark.parametrize("kw", [{"shared": True, "slots": 3}, {"shared": True, "n_raw": 3}, {"one_done": True}, {"all_wait": True}])
def test_controls_fail(kw):
    failed, n_raw = 0, kw.get("n_raw", 3)
    for seed in range(200):
        try:
            run(2, 1, n_raw, 17, seed, **{k: v for k, v in kw.items() if k != "n_raw"})
        except AssertionError:
            failed += 1
    assert failed > 0
