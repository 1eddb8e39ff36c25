"""Event model of a chunk-attention block whose waits give up (CPU).

A wait that runs out sets the block's abort flag, and from then on every wait
returns at once: the roles walk their loops to the end over buffers that may hold
anything.  What they take from shared memory must still lead nowhere but into
the pool, and copies and products in flight must have ended before the block reuses
their places.  Here the roles run in random order and any wait may give up.  As
controls, a ring entry that holds width and index in two words that nothing
initialises leads a decoder out of the pool, and roles that look at the flag once, at
the end of their own loops, leave work in flight when a later wait gives up."""
import random

N4, N8, N2 = 9, 3, 2                           # blocks of a pool, by width
N = N4 + N8 + N2


def width(block):
    return 4 if block < N4 else 8 if block < N4 + N8 else 2


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


class Block:
    """What the roles share, and their wait."""

    def __init__(self, seed, give_up):
        self.r = random.Random(seed)
        self.give_up, self.abort = give_up, False

    def wait(self, bar, parity):
        while not bar.ready(parity):
            if self.abort:
                return
            if self.r.random() < self.give_up:
                self.abort = True
                return
            yield

    def play(self, roles, land):
        while roles:
            if self.r.random() < 0.2 and land():
                continue
            g = self.r.choice(roles)
            try:
                next(g)
            except StopIteration:
                roles.remove(g)


def decode(seed, two_words, n_raw=3, n=9):
    """Width and place among the blocks of that width of every tile a decoder worked on."""
    blk = Block(seed, 0.02)
    r = blk.r
    raw_full, raw_empty = [Bar(1) for _ in range(2 * n_raw)], [Bar(4) for _ in range(n_raw)]
    left_over = [(r.choice((0, 2, 4, 8)), r.randrange(-50, 50)) for _ in range(n_raw)]     # of whatever ran before
    entry = left_over if two_words else [-1] * n_raw
    flying, seen = [], []

    def feed():
        for i in range(2 * n):
            yield from blk.wait(raw_empty[i % n_raw], ((i // n_raw) & 1) ^ 1)
            if blk.abort:
                return
            b = r.randrange(-1, N)
            if two_words:
                index = b if width(b) == 4 else b - N4 if width(b) == 8 else b - N4 - N8
                entry[i % n_raw] = (width(b) if b >= 0 else 0, entry[i % n_raw][1])
                yield
                if b >= 0:
                    entry[i % n_raw] = (width(b), index)
            else:
                entry[i % n_raw] = b
            flying.append(i)
            yield

    def decoder(kind):
        for i in range(kind, 2 * n, 2):
            yield from blk.wait(raw_full[i % (2 * n_raw)], (i // (2 * n_raw)) & 1)
            if two_words:
                seen.append(entry[i % n_raw])
            else:
                b = entry[i % n_raw]
                seen.append((0, 0) if b < 0 else (width(b), b if width(b) == 4 else b - N4 if width(b) == 8 else b - N4 - N8))
            yield
            raw_empty[i % n_raw].arrive()

    def land():
        if flying:
            raw_full[flying.pop(r.randrange(len(flying))) % (2 * n_raw)].arrive()
        return False

    blk.play([feed()] + [decoder(k) for k in (0, 1) for _ in range(4)], land)
    return blk.abort, seen


def inside(seen):
    return all(0 <= index < {0: 1, 4: N4, 8: N8, 2: N2}[bits] for bits, index in seen)


def test_decoders_stay_inside_the_pool_when_waits_give_up():
    gave_up = 0
    for seed in range(300):
        abort, seen = decode(seed, two_words=False)
        gave_up += abort
        assert inside(seen)
    assert gave_up > 100


def test_two_words_lead_out_of_the_pool():
    assert not all(inside(decode(seed, two_words=True)[1]) for seed in range(300))


def leave(seed, own_end, n_raw=3, n=6):
    """Copies and products in flight when the block's result is written."""
    blk = Block(seed, 0.01)
    r = blk.r
    raw_full, raw_empty = [Bar(1) for _ in range(2 * n_raw)], [Bar(2) for _ in range(n_raw)]
    kv_full, done = [Bar(2) for _ in range(2 * n)], [Bar(1) for _ in range(n)]
    landed, flying, queue, issued = set(), [], [], [0]

    def drain_copies():
        for c in range(max(0, issued[0] - n_raw), issued[0]):
            while not raw_full[c % (2 * n_raw)].ready((c // (2 * n_raw)) & 1):
                yield

    def drain_products():
        while queue:                           # (products of one thread end in order)
            yield

    def feed():
        for i in range(2 * n):
            yield from blk.wait(raw_empty[i % n_raw], ((i // n_raw) & 1) ^ 1)
            if blk.abort:
                break
            assert i < n_raw or i - n_raw in landed, "a place still being filled"
            flying.append(i)
            issued[0] = i + 1
            yield
        if own_end and blk.abort:
            yield from drain_copies()

    def decoder(kind):
        for i in range(kind, 2 * n, 2):
            yield from blk.wait(raw_full[i % (2 * n_raw)], (i // (2 * n_raw)) & 1)
            raw_empty[i % n_raw].arrive()
            kv_full[i].arrive()
            yield

    def product():
        for j in range(n):
            for i in (2 * j, 2 * j + 1):
                yield from blk.wait(kv_full[i], 0)
            queue.append(j)
            yield
        if own_end and blk.abort:
            yield from drain_products()

    def softmax():
        for j in range(n):
            yield from blk.wait(done[j], 0)

    def land():
        if flying and r.random() < 0.5:
            c = flying.pop(r.randrange(len(flying)))
            landed.add(c)
            raw_full[c % (2 * n_raw)].arrive()
        elif queue:
            done[queue.pop(0)].arrive()
        else:
            return False
        return True

    blk.play([feed(), product(), softmax()] + [decoder(k) for k in (0, 1) for _ in range(2)], land)
    if blk.abort and not own_end:              # after the block's barrier, where the flag is final
        blk.play([drain_copies(), drain_products()], land)
    return blk.abort, len(flying), len(queue)


def test_nothing_is_in_flight_when_the_result_is_written():
    gave_up = 0
    for seed in range(400):
        abort, copies, products = leave(seed, own_end=False)
        gave_up += abort
        assert copies == 0 and products == 0
    assert 100 < gave_up


def test_a_look_at_the_flag_at_the_end_of_a_role_is_too_early():
    left = [leave(seed, own_end=True) for seed in range(400)]
    assert any(copies for _, copies, _ in left) and any(products for _, _, products in left)
