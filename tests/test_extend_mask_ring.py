"""Event model of the chunk-attention kernel's ring of remap masks (CPU).

The key decoders write a tile's mask before they wait for the tile's slot, and the
softmax reads it with the tile's logits.  No barrier belongs to the ring: a writer
is kept off by what it has waited for, the slot of the tile before.  Values' tiles,
the rings of packed tiles and the running reference hold the roles back further and
are left out.  As a control, shorter rings are overwritten too early."""
import random

import pytest


def run(mode, groups, ring, n, seed):
    """mode 0: accumulators with rows of their own; 1: on alternate tiles; 2: one step a tile."""
    r = random.Random(seed)
    per = 1 if mode == 2 else 2                # softmax steps of a tile
    steps = [((n - s + 1) // 2 if mode == 1 else n) * per for s in range(groups)]
    mask, used_up, decoded = [None] * ring, set(), set()
    logits, weights, queue = set(), set(), []

    def tile(s, k):
        return 2 * (k // per) + s if mode == 1 else k // per

    def decoder():
        for j in range(n):
            mask[j % ring] = j
            yield
            while j >= 2 and j - 2 not in used_up:     # keys have two of the four slots
                yield
            decoded.add(j)
            yield

    def product():
        ahead = 2 if per == 1 else 1
        for i in range(steps[0] // per + ahead):
            for s in range(groups):
                tiles = steps[s] // per
                if i >= ahead and i - ahead < tiles:
                    for h in range(per):
                        while (s, (i - ahead) * per + h) not in weights:
                            yield
                if i < tiles:
                    while tile(s, i * per) not in decoded:
                        yield
                    queue.append((s, i))
                    yield

    def softmax(s, side):
        for k in range(side, steps[s], 2):
            while (s, k) not in logits:
                yield
            yield
            assert mask[tile(s, k) % ring] == tile(s, k), "mask overwritten"
            yield
            weights.add((s, k))
            yield

    roles = [decoder(), product()] + [softmax(s, side) for s in range(groups) for side in (0, 1)]
    slow = r.choice(roles)                     # one role runs seldom
    idle = 0
    while roles:
        if queue and r.random() < 0.3:
            s, i = queue.pop(0)
            logits.update((s, v) for v in range(i * per, (i + 1) * per))
            if mode != 0 or s == groups - 1:
                used_up.add(tile(s, i * per))
            idle = 0
            continue
        g = r.choice(roles)
        if g is slow and r.random() < 0.9:
            continue
        try:
            next(g)
        except StopIteration:
            roles.remove(g)
        idle += 1
        assert idle < 100000, "stuck"


# two row tiles; one of them empty; alternate key tiles; heads of 256
SHAPES = [(0, 2), (0, 1), (1, 2), (2, 1)]


@pytest.mark.parametrize("mode,groups", SHAPES)
def test_eight_masks_are_enough(mode, groups):
    for seed in range(150):
        run(mode, groups, 8, 23, seed)


@pytest.mark.parametrize("mode,groups,ring", [(0, 2, 3), (0, 1, 3), (1, 2, 3), (2, 1, 4)])
def test_shorter_rings_fail(mode, groups, ring):
    with pytest.raises(AssertionError, match="overwritten"):
        for seed in range(600):
            run(mode, groups, ring, 23, seed)
