"""The cache attention where a CTA's part of a group is long: block numbers and
exponents are fetched for 16 steps of a warp at a time, sums run over many
steps and many CTAs' parts are added. The lengths of those parts come from a
host model of the split, so that the cases are known to be what they say.

Tolerance of `check_tight` (p the softmax weights, A = sum p |v|, S steps of a
warp in the longest part, P parts):
  2^-11 |y|          the fp16 result (2^-25 among the subnormals)
  2^-11 A            p rounded to fp16
  2 d A              the scores: D exact products summed in fp32 and the two
                     roundings of x in units of log2: d = (D + 4) 2^-23 scale
                     max sum |q k| + 2^-23 (max|e_v| + 64)
  (2 S + P + 40) 2^-22 A
                     fp32 sums: two products of 16 keys a step, 4 warps, the
                     parts, lanes; the special function
  2^-37 2^max(e_v) sum |code|
                     weights among the fp16 subnormals: half their spacing is
                     2^-25, the largest weight of a row is at least 2^12
It does not grow with the number of keys. The sums over keys that go wrong by a
whole unit of work are `test_every_unit_counts_once`'s."""
import math

import pytest
import torch

import weight_only_bit_awq_b200 as awq
from test_gpu_kv8 import Batch

pytestmark = pytest.mark.gpu

COST = 2        # what a group counts in the split besides its units
UNIT = 128      # keys of a unit: one step of each of four warps


def kernel_of(bt):
    """(rows of a tile, CTAs) of the kernel that the library takes."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    G, B = bt.Hq // bt.Hkv, len(bt.new)
    rows = 16 if -(-bt.R // B) * G > 8 else 8
    few = bt.Hkv * (B + bt.R * G // rows) * 8 <= 2 * sms
    return rows, sms * (2 if bt.D == 128 and few else 3), few


def segments(bt):
    """(CTA, group, units) of every part of a group, in order."""
    rows, grid, _ = kernel_of(bt)
    G = bt.Hq // bt.Hkv
    groups = [(b, max(-(-n // UNIT), 1)) for b, (t, n) in enumerate(zip(bt.new, bt.n)) for _ in range(-(-t * G // rows) * bt.Hkv)]
    total = sum(k + COST for _, k in groups)
    ctas = min(total, grid)
    out, c, end = [], 0, total // ctas
    at = 0
    for g, (_, k) in enumerate(groups):
        v = 0
        while v < k + COST:
            while at == end:
                c += 1
                end = total * (c + 1) // ctas
            take = min(end - at, k + COST - v)
            n = v + take - COST - max(v - COST, 0)
            if n > 0:
                out.append((c, g, n))
            v, at = v + take, at + take
    return out


def most_parts(segs):
    parts = {}
    for _, g, _ in segs:
        parts[g] = parts.get(g, 0) + 1
    return max(parts.values())


def mixed_exponents(bt):
    for t, lo, hi in ((bt.cache.k_exp, -9, -4), (bt.cache.v_exp, -14, 1)):
        t.copy_(torch.randint(lo, hi, t.shape, generator=bt.g, device="cuda").to(torch.int8))


def check_tight(bt, segs):
    y = bt.attend().double().unflatten(1, (bt.Hq, bt.D))
    assert bt.status() == awq.AWQ_OK
    steps, parts = max(n for _, _, n in segs), most_parts(segs)
    G, scale = bt.Hq // bt.Hkv, bt.D ** -0.5
    for b, T in enumerate(bt.new):
        n = bt.n[b]
        k, _ = bt.kept(b, "k")
        v, ev = bt.kept(b, "v")
        r = slice(bt.starts_h[b], bt.starts_h[b] + T)
        for h in range(bt.Hkv):
            kh, vh, eh = k[:, h], v[:, h], ev[:, h].double()
            q = bt.q[r, h * G:(h + 1) * G].double()
            s = (q @ kh.T) * scale
            pos = n - T + torch.arange(T, device="cuda")
            s = s.masked_fill((torch.arange(n, device="cuda")[None] > pos[:, None])[:, None], -math.inf)
            p = torch.softmax(s, dim=-1)
            ref, A = p @ vh, p @ vh.abs()
            mag = (q.abs() @ kh.abs().T).amax(dim=-1, keepdim=True) * scale
            d = (bt.D + 4) * 2.0 ** -23 * mag + 2.0 ** -23 * (float(eh.abs().max()) + 64)
            codes = (vh.abs() * torch.exp2(-eh)[:, None]).sum(dim=0)
            tol = (2.0 ** -11 * ref.abs() + 2.0 ** -25 + (2.0 ** -11 + 2 * d + (2 * steps + parts + 40) * 2.0 ** -22) * A
                   + 2.0 ** (float(eh.max()) - 37) * codes)
            err = (y[r, h * G:(h + 1) * G] - ref).abs()
            assert (err <= tol).all(), (b, h, n, float((err / tol).max()))


AROUND = [2047, 2048, 2049, 2175, 2176, 2177, 4223, 4225, 4353, 8190, 9001, 16000]   # 16, 17 and 33 steps of 128 keys

# (D, block, q heads, kv heads, new tokens, lengths, few groups)
LONG = [
    (128, 16, 32, 8, [1], [160000], True), (128, 128, 32, 8, [1], [160000], True),
    (128, 16, 32, 8, [4], [160000], True), (128, 128, 32, 8, [4], [160000], True),
    (128, 16, 32, 8, [1] * 48, AROUND * 4, False), (128, 128, 32, 8, [1] * 48, AROUND * 4, False),
    (128, 16, 64, 8, [2] * 48, AROUND * 4, False), (128, 128, 64, 8, [2] * 48, AROUND * 4, False),
    (64, 16, 32, 8, [1] * 48, AROUND * 4, False), (64, 128, 32, 8, [1] * 48, AROUND * 4, False),
    (64, 16, 64, 8, [1, 2, 3] * 16, AROUND * 4, False), (64, 128, 64, 8, [2] * 48, AROUND * 4, False),
]


@pytest.mark.parametrize("D,block,Hq,Hkv,new,lens,few", LONG)
def test_exponents_and_blocks_over_many_steps(D, block, Hq, Hkv, new, lens, few):
    bt = Batch(new, lens, Hq, Hkv, D, block, seed=40 + D + block)
    assert kernel_of(bt)[2] == few
    segs = segments(bt)
    assert max(n for _, _, n in segs) > 33     # fetched three times
    mixed_exponents(bt)
    check_tight(bt, segs)


@pytest.mark.parametrize("D,block,T", [(128, 64, 1), (64, 32, 1), (128, 16, 3), (64, 128, 3)])
def test_parts_of_sixteen_and_seventeen_steps(D, block, T):
    # most groups are taken whole by one CTA, and have 16, 17 or 18 units
    lens = [AROUND[i % 6] for i in range(300)]
    bt = Batch([T] * 300, lens, 32, 8, D, block, seed=50 + D)
    segs = segments(bt)
    for n in (16, 17, 18):
        assert sum(u == n for _, _, u in segs) > 50, n
    mixed_exponents(bt)
    check_tight(bt, segs)


@pytest.mark.parametrize("Hq,Hkv,D,block,new,lens", [
    (8, 2, 128, 64, [1], [40001]), (8, 2, 64, 64, [1], [40001]), (32, 2, 128, 16, [2, 1], [9000, 20011]),
    (32, 8, 128, 64, [1] * 48, [37 + 173 * b for b in range(48)]), (16, 2, 64, 32, [3, 1, 4] * 8, [200 + 163 * b for b in range(24)]),
    (32, 8, 128, 64, [1], [500]), (8, 8, 128, 16, [1], [1100]), (64, 8, 128, 32, [4, 1, 2], [20011, 3001, 8191])])
def test_every_unit_counts_once(Hq, Hkv, D, block, new, lens):
    # Flat weights (scale 0), one exponent, and V is 1 in one unit of 128 keys and
    # 0 in the others, another unit for every channel and head: y is the share
    # of that unit's keys among those the row sees. All sums are of powers of two and
    # exact, so y is off by its rounding and the division's: 2^-11 + 2^-20. A
    # unit left out or taken twice moves its own channels by all of their value
    # (2^-5 / 40001 at least, 25 times the smallest fp16).
    bt = Batch(new, lens, Hq, Hkv, D, block, seed=60)
    bt.cache.v_exp.fill_(-5)
    rel = 2.0 ** -11 + 2.0 ** -20
    G, units = Hq // Hkv, -(-max(lens) // UNIT)
    col = torch.arange(Hkv * D, device="cuda").view(Hkv, D)          # the unit of a channel, of each round
    for turn in range(-(-units // (Hkv * D))):
        mine = col + turn * Hkv * D
        for b, n in enumerate(lens):
            blocks = bt.table[b, :-(-n // block)].long()
            token = torch.arange(len(blocks) * block, device="cuda") // UNIT
            on = token[:, None, None] == mine[None]                              # [tokens][Hkv][D]
            codes = (on.to(torch.uint8) * 0x38).unflatten(0, (-1, block)).transpose(1, 2)
            bt.cache.v[blocks] = codes.contiguous()
        y = bt.attend(scale=0.0).double().unflatten(1, (Hkv, G, D))
        for b, T in enumerate(new):
            for i in range(T):
                seen = lens[b] - T + i + 1
                keys = (seen - mine * UNIT).clamp(0, UNIT).double()
                ref = (keys / seen * 2.0 ** -5)[:, None].expand(-1, G, -1)
                got = y[bt.starts_h[b] + i]
                assert ((got - ref).abs() <= rel * ref + 2.0 ** -25).all(), (b, i, turn)
    assert bt.status() == awq.AWQ_OK
