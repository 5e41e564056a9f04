"""How paged attention divides its work, in plain integers: the weights of the
items, the CTAs' shares, the key tiles of a share, the workspace slots its
partial results take and the parts the join looks for (the arithmetic of
vark_paged_attention.cu's Entry, Share, Segments and join_kernel).  Over random
batches: every key tile is done once, every item is finished by exactly one
side, no two partials share a slot, and the join reads the ones that were
written."""
import random

import pytest

CTAS, UNIT, KT = 148, 16, 128


def items_of(batch, R, G, heads, causal, cost):
    """[(weight, key tiles)] in order, head after head, row tile after row tile."""
    out = []
    for n, length in batch:
        tiles = -(-n * G // R)
        slope = R * UNIT // G if causal and tiles > 1 else 0
        seen0 = min(length, max(0, length - n) + R // G) if slope else length
        for _ in range(heads):
            for t in range(tiles):
                limit = length
                if causal:
                    limit = max(0, length - n + min(n - 1, (t * R + R - 1) // G) + 1)
                out.append((UNIT * (cost * KT + seen0) + t * slope, max(1, -(-limit // KT))))
    return out


def tile_at(u, frm, to, key_tiles, cost):
    if u >= to:
        return key_tiles
    return max(0, min(key_tiles, (u - frm) // (UNIT * KT) - cost))


def check(batch, R, G, heads, causal, cost, one_each=False):
    items = items_of(batch, R, G, heads, causal, cost)
    if one_each:                          # no more items than CTAs: every one weighs one unit
        assert len(items) <= CTAS
        items = [(1, kt) for _, kt in items]
    starts = [0]
    for w, _ in items:
        assert w > 0
        starts.append(starts[-1] + w)
    total = starts[-1]
    if total == 0:
        return
    ctas = min(CTAS, total)
    per, extra = divmod(total, CTAS) if total > CTAS else (1, 0)
    begin = [per * c + min(c, extra) for c in range(ctas + 1)]
    assert begin[-1] == total
    wide = extra * (per + 1)

    def holder(u):
        return u // (per + 1) if u < wide else extra + (u - wide) // per

    done = [[] for _ in items]            # (k0, k1, cta) of every item
    slots = {}
    i = 0
    for c in range(ctas):
        u, end = begin[c], begin[c + 1]
        assert holder(u) == c and holder(end - 1) == c
        while starts[i + 1] <= u:
            i += 1
        j = i
        while u < end:
            frm, to, kt = starts[j], starts[j + 1], items[j][1]
            stop = min(to, end)
            k0, k1 = tile_at(u, frm, to, kt, cost), tile_at(stop, frm, to, kt, cost)
            if k0 < k1:
                done[j].append((k0, k1, c))
                if not (k0 == 0 and k1 == kt):
                    key = (c, 1 if k0 == 0 else 0)
                    assert key not in slots, "two partials in a slot"
                    slots[key] = j
            u = stop
            j += 1
    for j, runs in enumerate(done):
        frm, to, kt = starts[j], starts[j + 1], items[j][1]
        at = 0
        for k0, k1, _ in runs:            # in order, without a gap
            assert k0 == at
            at = k1
        assert at == kt
        # the join: shares from the item's first unit to its last
        c0, c1 = holder(frm), holder(to - 1)
        found = []
        for c in range(c0, c1 + 1):
            k0 = tile_at(max(frm, begin[c]), frm, to, kt, cost)
            k1 = tile_at(min(to, begin[c + 1]), frm, to, kt, cost)
            if k0 < k1:
                found.append((k0, k1, c))
        assert found == runs
        finished_alone = runs[0][:2] == (0, kt)
        assert finished_alone == (len(runs) == 1)
        # every share that joins an item finds it at one of its two ends
        if not finished_alone:
            for c in range(c0, c1 + 1):
                assert frm <= begin[c] < to or frm <= begin[c + 1] - 1 < to


@pytest.mark.parametrize("seed", range(12))
def test_shares_cover_every_key_tile_once(seed):
    rng = random.Random(seed)
    for _ in range(25):
        R = rng.choice([16, 32, 256])
        G = rng.choice([1, 2, 3, 4, 5, 8, 16, 40])
        causal = rng.random() < 0.6
        batch = []
        for _ in range(rng.choice([1, 2, 7, 40])):
            n = rng.choice([0, 1, 1, rng.randint(1, 9), rng.randint(1, 600)])
            past = rng.choice([-n, -rng.randint(0, n), 0, rng.randint(0, 300), rng.randint(0, 20000)])
            batch.append((n, n + past))
        check(batch, R, G, rng.choice([1, 2, 8]), causal, rng.choice([1, 3]))


def test_smallest_and_single_items():
    check([(1, 1)], 16, 1, 1, True, 1)
    check([(1, 0)], 16, 1, 1, True, 1)
    check([(1, 1 << 20)], 16, 4, 1, True, 3)
    check([(4096, 4096)], 256, 1, 1, False, 3)
    check([(1, 1)] * 300, 32, 1, 16, False, 1)


def test_one_item_a_share():
    """Few short items are not cut: every share is one of them."""
    rng = random.Random(7)
    for _ in range(60):
        batch = [(n, n + rng.randint(0, 700)) for n in (rng.randint(0, 90) for _ in range(rng.randint(1, 18)))]
        G, heads, causal = rng.choice([1, 4, 5]), rng.choice([1, 2, 4]), rng.random() < 0.5
        items = items_of(batch, 256, G, heads, causal, 2)
        if len(items) <= CTAS:
            check(batch, 256, G, heads, causal, 2, one_each=True)
    check([(0, 5), (0, 0)], 256, 4, 8, True, 2, one_each=True)
