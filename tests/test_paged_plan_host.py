"""How paged attention divides its work, by the kernels' own arithmetic compiled
for the host: every key tile is done once, every item is finished by exactly
one side, no two partials share a slot, the join reads the ones that were
written; divisions and row tiles at the ends of their ranges."""
import random

import numpy as np
import pytest

from tests import paged_plan

pytestmark = pytest.mark.skipif(paged_plan.library() is None, reason="no C++ compiler")


def items_of(R, n, lens, heads, G, causal, KT):
    """{(entry, head, row tile): keys seen}, from the definition."""
    out = {}
    lens = np.asarray(lens)
    for e in range(lens.size):
        b, head = divmod(e, heads) if lens.ndim == 2 else (e, None)
        length = int(lens.reshape(-1)[e])
        for h in range(heads) if head is None else [head]:
            for t in range(-(-n[b] * G // R)):
                last_token = min(n[b] - 1, (t * R + R - 1) // G)
                out[e, h, t] = max(0, length - n[b] + last_token + 1) if causal else length
    return out


def check(R, n, lens, heads, G, causal):
    c = paged_plan.constants()
    KT = c["tile_keys"]
    segments, joins, total, whole, shares = paged_plan.plan(R, n, lens, heads, G, causal)
    items = items_of(R, n, lens, heads, G, causal, KT)
    assert shares == min(c["ctas"], total) and (total == 0) == (not items)
    done = {key: [] for key in items}
    slots = {}
    for cta, e, h, t, k0, k1, key_tiles, limit in segments.tolist():
        assert limit == items[e, h, t] and key_tiles == max(1, -(-limit // KT)) and 0 <= k0 < k1 <= key_tiles
        done[e, h, t].append((k0, k1, cta, key_tiles))
        if k1 - k0 < key_tiles:
            slot = 2 * cta + (k0 == 0)
            assert slot not in slots, "two partials in a slot"
            slots[slot] = (e, h, t)
    read = {}
    for cta, e, h, t, share, k0, k1, slot in joins.tolist():
        read.setdefault((e, h, t), {}).setdefault(cta, []).append((share, k0, k1, slot))
    for key, runs in done.items():
        assert runs[0][0] == 0 and runs[-1][1] == runs[0][3]
        assert all(a[1] == b[0] and a[2] < b[2] for a, b in zip(runs, runs[1:])), "in order, without a gap"
        if whole:
            assert len(runs) == 1
        by = read.get(key, {})
        if len(runs) == 1:
            # a share that finds the item cut by the plan sees that one share did all of it
            for parts in by.values():
                assert [p for p in parts if p[3] >= 0] == [(runs[0][2], 0, runs[0][3], 2 * runs[0][2] + 1)]
        else:
            # every share from the first part's to the last's joins it, and all read the same parts
            want = [(cta, k0, k1, 2 * cta + (k0 == 0)) for k0, k1, cta, _ in runs]
            assert by and all([p for p in parts if p[3] >= 0] == want for parts in by.values())
            shares_of = sorted(by)
            assert shares_of == list(range(shares_of[0], shares_of[-1] + 1)) == [p[0] for p in by[shares_of[0]]]
            assert all(slots[s] == key for _, _, _, s in want)
    return whole


@pytest.mark.parametrize("seed", range(10))
def test_shares_cover_every_key_tile_once(seed):
    rng = random.Random(seed)
    for _ in range(25):
        R, G = rng.choice([16, 32, 256]), rng.choice([1, 2, 3, 4, 5, 8, 16, 40, 300])
        B, heads = rng.choice([1, 2, 7, 40]), rng.choice([1, 2, 8])
        n = [rng.choice([0, 1, 1, rng.randint(1, 9), rng.randint(1, 600)]) for _ in range(B)]

        def length(k):
            return k + rng.choice([-k, -rng.randint(0, k), 0, rng.randint(0, 300), rng.randint(0, 20000)])

        lens = [[length(k) for _ in range(heads)] if seed % 2 else length(k) for k in n]
        check(R, n, lens, heads, G, rng.random() < 0.6)


def test_smallest_and_single_items():
    check(16, [1], [1], 1, 1, True)
    check(16, [1], [0], 1, 1, True)
    check(16, [0, 0], [5, 0], 3, 2, True)
    check(16, [1], [1 << 20], 1, 4, True)
    check(256, [4096], [4096], 1, 1, False)
    check(32, [1] * 300, [1] * 300, 16, 1, False)
    check(16, [1], [2 ** 31 - 2048], 2, 1, True)


def test_few_short_items_stay_whole():
    """Which side of the rule a batch lies on, and that none is cut on one."""
    rng = random.Random(7)
    seen = set()
    for _ in range(150):
        n = [rng.randint(0, 90) for _ in range(rng.randint(1, 18))]
        lens = [k + rng.choice([rng.randint(0, 700), rng.randint(0, 6000)]) for k in n]
        seen.add(check(256, n, lens, rng.choice([1, 2, 4]), rng.choice([1, 4, 5]), rng.random() < 0.5))
    assert seen == {True, False}
    assert check(256, [40] * 16, [500] * 16, 8, 4, False)             # 128 items of 4 tiles, 148 CTAs
    assert not check(256, [40] * 20, [500] * 20, 8, 4, False)         # 160 of them
    assert not check(256, [200], [40000], 1, 1, False)                # one long item


def test_divisions_by_products():
    rng = random.Random(3)
    lib = paged_plan.library()
    for d in [1, 2, 3, 5, 7, 40, 255, 256, 257, 1000, 32767, 32768, 65535, 65536, 5000, 6, 12]:
        xs = [0, 1, d - 1, d, d + 1, 2 ** 30, 2 ** 31 - 1, 2 ** 31 - 2]
        xs += [k * d + r for k in (1, 77, (2 ** 31 - 1) // d - 1) for r in (-1, 0, 1)]
        xs += [rng.randrange(2 ** 31) for _ in range(200)]
        for x in xs:
            if 0 <= x < 2 ** 31:
                assert lib.fast_div(x, d) == x // d, (x, d)


def test_quotients_on_both_sides_of_32_bits():
    rng = random.Random(4)
    lib = paged_plan.library()
    ends = [1, 2, 3, 2 ** 31 - 1, 2 ** 31, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 1, 2 ** 62]
    for a in [0, *ends, *(rng.randrange(2 ** rng.randint(1, 62)) for _ in range(100))]:
        for b in ends + [rng.randrange(1, 2 ** rng.randint(1, 62)) for _ in range(20)]:
            assert lib.divide(a, b) == a // b


def test_row_tiles_of_units():
    """tile_of is the inverse of the sums, at the ends of every tile and of the
    ranges that the limits of a call allow (2^26 row tiles, 2^31 keys)."""
    rng = random.Random(5)
    lib = paged_plan.library()
    for _ in range(400):
        R, G = rng.choice([16, 32, 256]), rng.choice([1, 2, 3, 5, 8, 40])
        most = 2 ** 30 // G - 1                              # tokens * query heads stay below 2^30
        n = min(most, rng.choice([1, 2, 3, rng.randint(1, 300), rng.randint(1, 1 << 22), most]))
        tiles, slope = -(-n * G // R), rng.choice([0, R * 16 // G])
        weight0 = 16 * (256 + rng.choice([0, 1, 300, rng.randint(0, 1 << 20), 2 ** 31 - 2048]))
        for t in {0, tiles - 1, tiles // 2, rng.randrange(tiles)}:
            a = lib.tile_sum(slope, weight0, t)
            assert a == t * weight0 + slope * (t * (t - 1) // 2)
            b = lib.tile_sum(slope, weight0, t + 1) - 1
            assert lib.tile_of(tiles, slope, weight0, a) == t and lib.tile_of(tiles, slope, weight0, b) == t
