"""Host models of index arithmetic of the cache kernels (csrc/kv8.cu) when a
batch's lists are bad, or change while the kernels read them."""
import random


def block_of(u, base, past, shift, width):
    """The append's place in a block table: item u of the batch, where its sequence's items begin at `base`. 64 bits up
    to the clamp: with bad starts there can be more than 2^31 items, and with changed ones base can be 0."""
    return min((max(past, 0) >> shift) + (u - base), width - 1)


def test_place_in_the_block_table_stays_inside_it():
    rng = random.Random(3)
    narrow = 0
    for _ in range(2000):
        width, shift = rng.choice([1, 9, 1 << 21]), rng.choice([4, 7])
        u = rng.choice([rng.randrange(1 << 12), rng.randrange(1 << 44), (1 << 31) + rng.randrange(1 << 8)])
        base, past = rng.choice([0, u, rng.randint(0, u)]), rng.choice([-5, 0, rng.randrange(width << shift)])
        assert 0 <= block_of(u, base, past, shift, width) < width
        low = (u - base) & 0xFFFFFFFF                    # what an int would keep of it
        narrow += min((max(past, 0) >> shift) + (low - (low >> 31 << 32)), width - 1) < 0
    assert narrow > 50


# How a CTA finds its first unit of work: each of 128 threads counts the units of
# its run of sequences, a scan adds them up, and then the list is read again for
# the sequence that holds the unit. Between the two readings the lists may change.
# What is handed out (a sequence's first row and rows) must come from one
# thread: a mixture of two has rows up to beyond the buffers.
THREADS = 128
ROWS = 4096


def sequence(rng):
    """(first row, rows, units) as a reading of the lists gives it, clamped to the buffers."""
    row0 = rng.randint(0, ROWS)
    return row0, rng.randint(0, ROWS - row0), rng.choice([0, 1, 3, 40, 3000])


def finders(first, second, u, by_counts):
    """What the threads find for unit u: counted in `first`, read again in `second`. by_counts: only the thread whose
    counts hold u looks; otherwise every thread goes by what it reads the second time."""
    per = -(-len(first) // THREADS)
    found, before = [], 0
    for t in range(THREADS):
        run = range(t * per, min(len(first), (t + 1) * per))
        mine = sum(first[b][2] for b in run)
        if not by_counts or before <= u < before + mine:
            at = before
            for b in run:
                if at <= u < at + second[b][2]:
                    found.append(second[b])
                    break
                at += second[b][2]
        before += mine
    return found


def outside(found):
    """Whether fields of different finders can make rows beyond the buffers."""
    return any(f[0] + g[1] > ROWS for f in found for g in found)


def test_one_thread_hands_out_the_first_unit():
    rng = random.Random(1)
    several = beyond = none = 0
    for _ in range(300):
        seqs = rng.choice([2, 60, 128, 300])
        first = [sequence(rng) for _ in range(seqs)]
        second = [sequence(rng) if rng.random() < 0.5 else s for s in first]
        total = sum(s[2] for s in first)
        for u in (rng.randrange(total) for _ in range(5) if total):
            found = finders(first, second, u, True)
            assert len(found) <= 1 and not outside(found)
            none += not found
            found = finders(first, second, u, False)
            several += len(found) > 1
            beyond += outside(found)
    assert several > 100 and beyond > 50 and none > 50   # every thread by its own reading: the fault is in the model


def test_unchanged_lists_have_one_finder():
    rng = random.Random(2)
    for _ in range(50):
        lists = [sequence(rng) for _ in range(rng.choice([1, 2, 128, 129, 300]))]
        total = sum(s[2] for s in lists)
        for u in (rng.randrange(total) for _ in range(5) if total):
            assert finders(lists, lists, u, True) == finders(lists, lists, u, False) != []
