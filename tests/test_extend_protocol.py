"""Event model of the chunk-attention kernel's barriers (CPU).

The kernel's roles (feed, key and value decoders, product, softmax) meet at
mbarriers and wait by phase parity, which tells only two neighbouring phases of
a barrier apart.  Here the roles run in random order, copies land in random
order and products finish in issue order; every use of a buffer checks that it
holds what its user expects.  As controls, the layouts with one barrier per place
(shared by keys and values) and with one barrier for two logit buffers fail."""
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


def run(mode, lag, slots, n_raw, n, seed, shared=False, one_done=False):
    r = random.Random(seed)
    k_raw, k_slot = (n_raw, slots) if shared else (2 * n_raw, 2 * slots)
    raw_full, raw_empty = [Bar(1) for _ in range(k_raw)], [Bar(4) for _ in range(n_raw)]
    kv_full, kv_empty = [Bar(4) for _ in range(slots)], [Bar(1) for _ in range(k_slot)]
    s_full, p_full, o_done = ([Bar(1) for _ in range(2)] for _ in range(3))
    raw, slot = [None] * n_raw, [(None, 0)] * slots
    flying, queue, products = [], [], []
    uses = {i: lag if mode == 0 else 1 for i in range(2 * n)}
    units = n * (lag if mode == 0 else 1)

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
        for u in range(units + lag):
            if u >= lag:
                v = u - lag
                i = 2 * (v // lag if mode == 0 else v) + 1
                while not kv_full[i % slots].ready((i // slots) & 1):
                    yield
                assert slot[i % slots] == (i, 4), "values"
                while not p_full[v % lag].ready((v // lag) & 1):
                    yield
                queue.append(("pv", v, i))
                yield
            if u < units:
                i = 2 * (u // lag if mode == 0 else u)
                while not kv_full[i % slots].ready((i // slots) & 1):
                    yield
                assert slot[i % slots] == (i, 4), "keys"
                queue.append(("qk", u, i))
                yield

    def softmax(st):
        steps = n if mode != 1 else (n - st + 1) // 2

        def unit(k):
            return k if mode == 2 else (lag * k + st if mode == 0 else 2 * k + st)

        def done(k):
            if mode == 2 and not one_done:
                return o_done[k & 1].ready((k >> 1) & 1)
            return o_done[st].ready(k & 1)

        for k in range(steps):
            buf, phase = (k & 1, k >> 1) if mode == 2 else (st, k)
            while not s_full[buf].ready(phase & 1):
                yield
            if k and r.random() < 0.5:         # the maximum moves: the accumulator is rescaled
                while not done(k - 1):
                    yield
                assert unit(k - 1) in products, "accumulator not ready"
            yield
            p_full[buf].arrive()
            yield
        while steps and not done(steps - 1):
            yield
        assert not steps or unit(steps - 1) in products, "result read too early"

    roles = [feed(), product(), softmax(0)] + [decoder(k) for k in (0, 1) for _ in range(4)]
    if mode == 1 or (mode == 0 and lag == 2):
        roles.append(softmax(1))
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
            what, u, i = queue.pop(0)
            assert slot[i % slots][0] == i, "operand overwritten"
            uses[i] -= 1
            if what == "qk":
                s_full[u % lag].arrive()
            else:
                products.append(u)
                o_done[0 if mode == 2 and one_done else u % lag].arrive()
            if mode != 0 or u % lag == lag - 1:
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


# mode, logit buffers, decoded tiles: two row tiles; two of them with one empty;
# alternating key tiles; heads of 256
SHAPES = [(0, 2, 3), (0, 1, 3), (1, 2, 4), (2, 2, 3)]


@pytest.mark.parametrize("mode,lag,slots", SHAPES)
@pytest.mark.parametrize("n_raw", [3, 7])
def test_roles_never_meet_a_wrong_buffer(mode, lag, slots, n_raw):
    for n in (1, 2, 3, 5, 17):
        for seed in range(12):
            run(mode, lag, slots, n_raw, n, seed)


@pytest.mark.parametrize("kw,shape", [({"shared": True}, (2, 2, 3)), ({"one_done": True}, (2, 2, 3))])
def test_controls_fail(kw, shape):
    failed = 0
    for seed in range(60):
        try:
            run(*shape, 3, 17, seed, **kw)
        except AssertionError:
            failed += 1
    assert failed > 0
