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
