"""Host model of the cache attention's work split (csrc/kv8.cu): units of
128 keys of one group (sequence, kv head, row tile),
behind two units per group that stand for its fixed cost and hold no keys;
equal contiguous ranges of them per CTA; and the hand-over of groups that
several CTAs work on to the fixup kernel. Where the block table is short, a group is
one unit and nothing is handed over. Checked on random ragged batches: every unit
is computed once, a group's rows are written once, by the CTA that computes
all of it or by the fixup, and the fixup reads exactly the slots that the
group's contributors wrote."""
import random

import pytest


COST = 2   # units of a group that hold no keys


def plan(seqs, group, heads, rows_per_tile, keys_per_unit):
    """(row_tiles, key_tiles) of every sequence (new tokens, length)."""
    return [(-(-t * group // rows_per_tile), max(-(-n // keys_per_unit), 1)) for t, n in seqs]


def simulate(seqs, group, heads, rows_per_tile, keys_per_unit, grid, whole=False):
    tiles = plan(seqs, group, heads, rows_per_tile, keys_per_unit)
    def units(k):
        return 1 if whole else k + COST

    total = sum(r * units(k) * heads for r, k in tiles)
    ctas = min(total, grid)
    owner = {}      # (group, key tile) -> CTA
    direct = set()  # groups written by the attention kernel
    slots = {}      # (cta, slot) -> group
    fix = {}        # cta -> (group, last cta)
    for c in range(ctas):
        u = total // ctas * c + total % ctas * c // ctas
        u1 = total // ctas * (c + 1) + total % ctas * (c + 1) // ctas
        b, base = 0, 0
        while u < u1:
            while u >= base + tiles[b][0] * units(tiles[b][1]) * heads:
                base += tiles[b][0] * units(tiles[b][1]) * heads
                b += 1
            rt, kt = tiles[b]
            g, v0 = divmod(u - base, units(kt))
            take = min(u1 - u, units(kt) - v0)
            tile0 = max(v0 - COST, 0)
            n = kt if whole else v0 + take - COST - tile0
            u += take
            if n <= 0:
                continue
            h, row_tile = divmod(g, rt)
            who = (b, h, row_tile)
            assert 0 <= h < heads and 0 <= row_tile < rt
            for i in range(tile0, tile0 + n):
                assert (who, i) not in owner and i < kt
                owner[who, i] = c
            if tile0 == 0 and v0 + take == units(kt):
                assert who not in direct
                direct.add(who)
            else:
                key = (c, 1 if tile0 == 0 else 0)
                assert key not in slots
                slots[key] = who
                if tile0 == 0:
                    end = base + (g + 1) * units(kt)
                    assert c not in fix
                    fix[c] = (who, (end * ctas + total - 1) // total - 1)
    assert len(owner) == sum(r * k * heads for r, k in tiles)
    fixed = set()
    for c, (who, last) in fix.items():
        assert last > c
        for i in range(c, last + 1):
            assert slots.pop((i, 1 if i == c else 0)) == who
        assert who not in fixed and who not in direct
        fixed.add(who)
    assert not slots
    assert not (whole and fix)
    groups = {(b, h, r) for b, (rt, _) in enumerate(tiles) for h in range(heads) for r in range(rt)}
    assert direct | fixed == groups


@pytest.mark.parametrize("seed", range(16))
def test_every_unit_once_and_every_group_written_once(seed):
    rng = random.Random(seed)
    for _ in range(25):
        B = rng.randint(1, 20)
        seqs = [(rng.choice([0, 1, 1, 1, rng.randint(2, 40)]), rng.choice([0, 1, rng.randint(1, 300), rng.randint(1, 9000)]))
                for _ in range(B)]
        simulate(seqs, rng.choice([1, 4, 8, 29]), rng.choice([1, 2, 8]), rng.choice([8, 16]), 128,
                 rng.choice([1, 3, 148, 296, 444]), rng.random() < 0.2)


def test_long_and_empty_batches():
    simulate([(1, 131072)], 4, 8, 8, 128, 296)
    simulate([(0, 0), (0, 50), (1, 0)], 4, 8, 8, 128, 296)
    simulate([(0, 0)], 4, 8, 8, 128, 296)
