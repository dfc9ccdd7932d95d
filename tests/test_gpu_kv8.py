"""The 8-bit key/value cache: awq_kv8_append bit for bit against a plain
token-by-block model, awq_kv8_attention against its formula in fp64 on the
values the cache holds.

Tolerance of the attention (p the softmax weights, A = sum p |v|, N keys):
  2^-11 |y|             the fp16 result (2^-25 among the subnormals)
  2^-11 A               p rounded to fp16
  2 d A                 the scores: products of fp16 q and E4M3 codes are exact,
                        D of them are summed in fp32 (D 2^-24 of sum |q k|), then
                        two roundings of x in units of log2: d = (D + 4) 2^-24
                        scale max sum |q k| + 2^-24 max(|e_v| + 64)
  (N + 16) 2^-23 A      fp32 sums over keys, the special function (2^-22)
  N 2^-31 2^max(e_v)    weights that fall among the fp16 subnormals
"""
import math

import pytest
import torch

import weight_only_bit_awq_b200 as awq

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def values(codes, exps):
    return codes.view(E4M3).double() * torch.exp2(exps.double())[..., None, None]


class Batch:
    """A ragged batch: new[b] new tokens of lens[b], blocks drawn at random."""

    def __init__(self, new, lens, Hq, Hkv, D, block, seed=0, spare=3, q_std=1.0, empty=False):
        g = torch.Generator(device="cuda").manual_seed(seed + 11)
        self.g, self.new, self.n, self.Hq, self.Hkv, self.D, self.block = g, new, lens, Hq, Hkv, D, block
        B, R = len(new), sum(new)
        self.R = R
        width = max(1, max(-(-n // block) for n in lens))
        self.blocks = B * width + spare
        order = torch.randperm(self.blocks, generator=g, device="cuda")[:B * width]
        self.table = order.to(torch.int32).view(B, width).contiguous()
        self.starts_h = [sum(new[:b]) for b in range(B + 1)]
        self.starts = torch.tensor(self.starts_h, dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        qkv = torch.randn(max(R, 1), (Hq + 2 * Hkv) * D, generator=g, device="cuda").half()
        self.q = (qkv[:R, :Hq * D] * q_std).unflatten(1, (Hq, D)) if q_std != 1.0 else qkv[:R, :Hq * D].unflatten(1, (Hq, D))
        self.k = qkv[:R, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
        self.v = qkv[:R, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
        if empty:
            self.cache = awq.new_kv8_cache(self.blocks, Hkv, block, D, "cuda")
        else:
            shape = (self.blocks, Hkv, block, D)
            c = [(torch.randn(shape, generator=g, device="cuda") * 70).clamp(-448, 448).to(E4M3).view(torch.uint8) for _ in "kv"]
            e = [torch.randint(-8, -3, shape[:2], generator=g, device="cuda").to(torch.int8) for _ in "kv"]
            self.cache = awq.Kv8Cache(*c, *e)
        self.ws = awq.new_kv8_workspace(R, B, Hq, Hkv, D, "cuda")

    def append(self):
        awq.awq_kv8_append(self.k, self.v, self.cache, self.starts, self.lens, self.table, self.ws)

    def attend(self, **kw):
        return awq.awq_kv8_attention(self.q, self.cache, self.starts, self.lens, self.table, self.ws, **kw)

    def status(self):
        return awq.awq_get_status(self.ws)

    def kept(self, b, part):
        """fp64 [len][Hkv][D] values of sequence b, and the exponents [len][Hkv]."""
        n = self.n[b]
        rows = self.table[b, :-(-n // self.block)].long()
        codes, exps = (self.cache.k, self.cache.k_exp) if part == "k" else (self.cache.v, self.cache.v_exp)
        x = values(codes[rows], exps[rows]).permute(0, 2, 1, 3).reshape(-1, self.Hkv, self.D)[:n]
        return x, exps[rows].repeat_interleave(self.block, dim=0)[:n]

    def attention_ref(self, scale=None):
        """(y, tolerance) fp64 [R][Hq * D]."""
        scale = self.D ** -0.5 if scale is None else scale
        G = self.Hq // self.Hkv
        y = torch.zeros(self.R, self.Hq, self.D, dtype=torch.float64, device="cuda")
        tol = torch.full_like(y, 2.0 ** -25)
        for b, T in enumerate(self.new):
            if self.n[b] == 0 or T == 0:
                continue
            k, _ = self.kept(b, "k")
            v, ev = self.kept(b, "v")
            r = slice(self.starts_h[b], self.starts_h[b] + T)
            q = self.q[r].double().unflatten(1, (self.Hkv, G))                    # [T][H][G][D]
            pos = self.n[b] - T + torch.arange(T, device="cuda")
            hidden = torch.arange(self.n[b], device="cuda")[None] > pos[:, None]   # [T][N]
            s = torch.einsum("thgd,nhd->thgn", q, k) * scale
            s = s.masked_fill(hidden[:, None, None], -math.inf)
            p = torch.nan_to_num(torch.softmax(s, dim=-1), nan=0.0)                # rows that see nothing
            out = torch.einsum("thgn,nhd->thgd", p, v)
            A = torch.einsum("thgn,nhd->thgd", p, v.abs())
            mag = torch.einsum("thgd,nhd->thgn", q.abs(), k.abs()).amax(dim=-1)[..., None] * abs(scale)
            d = (self.D + 4) * 2.0 ** -24 * mag + 2.0 ** -24 * (float(ev.abs().max()) + 64)
            N = self.n[b]
            t = 2.0 ** -11 * out.abs() + (2.0 ** -11 + 2 * d + (N + 16) * 2.0 ** -23) * A
            t = t + N * 2.0 ** -31 * 2.0 ** float(ev.max())
            y[r] = out.flatten(1, 2)
            tol[r] += t.flatten(1, 2)
        return y.flatten(1), tol.flatten(1)

    def check(self, what="", scale=None):
        y = self.attend(scale=scale)
        ref, tol = self.attention_ref(scale)
        err = (y.double() - ref).abs()
        assert (err <= tol).all(), (what, float((err / tol).max()))
        assert self.status() == awq.AWQ_OK
        return y


def needed_exponent(amax):
    if amax == 0:
        return -32
    e = math.frexp(amax)[1] - 9
    while amax > 448 * 2.0 ** e:
        e += 1
    while amax <= 448 * 2.0 ** (e - 1):
        e -= 1
    return e


def append_model(bt, cache):
    """The cache after the append, on the CPU, block by block."""
    k, v, ke, ve = (t.cpu().clone() for t in cache)
    table = bt.table.cpu()
    for src, codes, exps in ((bt.k.cpu(), k, ke), (bt.v.cpu(), v, ve)):
        for b, T in enumerate(bt.new):
            past = bt.n[b] - T
            for j in range(max(past, 0) // bt.block, -(-bt.n[b] // bt.block) if T else 0):
                lo, hi = max(past, j * bt.block, 0), min(bt.n[b], (j + 1) * bt.block)
                if lo >= hi:
                    continue
                blk = int(table[b, j])
                for h in range(bt.Hkv):
                    x = src[bt.starts_h[b] + lo - past:bt.starts_h[b] + hi - past, h].float()
                    fin = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
                    e = needed_exponent(float(fin.abs().max()))
                    off = lo - j * bt.block
                    if off:
                        e_old = int(exps[blk, h])
                        e = max(e, e_old)
                        if e > e_old:
                            old = codes[blk, h, :off].view(E4M3).float() * 2.0 ** (e_old - e)
                            codes[blk, h, :off] = old.to(E4M3).view(torch.uint8)
                    exps[blk, h] = e
                    x = torch.where(torch.isfinite(x), x * 2.0 ** -e, torch.full_like(x, math.nan))
                    codes[blk, h, off:off + hi - lo] = x.to(E4M3).view(torch.uint8)
    return k, v, ke, ve


def same_cache(got, want):
    for name, a, b in zip(("k", "v", "k_exp", "v_exp"), got, want):
        a = a.cpu()
        if a.dtype == torch.uint8:   # NaN has a sign bit that the conversion may drop
            a, b = (torch.where((x & 0x7F) == 0x7F, torch.full_like(x, 0x7F), x) for x in (a, b))
        assert torch.equal(a, b), (name, int((a != b).sum()))


APPENDS = [
    # new tokens and lengths of the sequences
    ([1], [1]), ([1], [17]), ([1, 1, 1], [1, 64, 65]), ([5, 0, 1], [5, 9, 200]), ([40, 130, 1], [40, 300, 128]),
    ([0, 3], [0, 3]), ([4], [2]), ([2, 1], [0, 1]), ([33] * 7, [33, 34, 50, 64, 65, 200, 97]),
]


@pytest.mark.parametrize("new,lens", APPENDS)
@pytest.mark.parametrize("D,block", [(128, 64), (64, 16), (128, 16), (64, 128), (128, 128), (64, 32)])
def test_append_is_bit_exact(new, lens, D, block):
    bt = Batch(new, lens, 4, 2, D, block, seed=len(new) + block)
    want = append_model(bt, bt.cache)
    bt.append()
    same_cache(bt.cache, want)
    assert bt.status() == awq.AWQ_OK
    bt.append()                                     # once more: nothing changes
    same_cache(bt.cache, want)


def test_append_token_by_token_grows_the_exponent():
    # values that grow from token to token, so a block is rescaled again and
    # again; the model is applied token by token too
    n, D, block = 70, 64, 32
    bt = Batch([1], [1], 2, 2, D, block, seed=5, empty=True)
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
    cache = awq.new_kv8_cache(5, 2, block, D, "cuda")
    bt.table, bt.cache, bt.blocks = table, cache, 5
    for i in range(n):
        bt.n, bt.lens = [i + 1], torch.tensor([i + 1], dtype=torch.int32, device="cuda")
        bt.k = (torch.randn(1, 2, D, generator=bt.g, device="cuda") * 1.3 ** (i % 40)).half()
        bt.v = (torch.randn(1, 2, D, generator=bt.g, device="cuda") * 2.0 ** -(i % 20)).half()
        want = append_model(bt, bt.cache)
        bt.append()
        same_cache(bt.cache, want)
    assert bt.status() == awq.AWQ_OK


def test_append_edge_values():
    bt = Batch([6], [6], 2, 2, 64, 16, seed=1, empty=True)
    k = torch.zeros(6, 2, 64, device="cuda").half()
    k[0, 0] = 65504.0                               # exponent 8
    k[1, 0] = 2.0 ** -24
    k[2, 1, 3], k[2, 1, 4], k[2, 1, 5] = float("nan"), float("inf"), -float("inf")
    k[3, 1] = 448.0 * 2.0 ** -6                     # exactly the largest code
    v = torch.zeros(6, 2, 64, device="cuda").half()
    v[1, 1] = 2.0 ** -24                            # exponent -32
    bt.k, bt.v = k, v
    want = append_model(bt, bt.cache)
    bt.append()
    same_cache(bt.cache, want)
    blk = int(bt.table[0, 0])
    assert [int(x) for x in bt.cache.k_exp[blk]] == [8, -6] and [int(x) for x in bt.cache.v_exp[blk]] == [-32, -32]
    assert (bt.cache.k[blk, 1, 2, 3:6] & 0x7F == 0x7F).all()


HEADS = [(4, 4), (8, 2), (8, 1), (16, 2), (29, 1), (58, 2)]


@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("D,block", [(128, 64), (64, 64), (128, 16), (64, 16), (128, 128), (64, 32)])
def test_attention_single_tokens(Hq, Hkv, D, block):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 500, 0, 1031]
    Batch([1] * len(lens), lens, Hq, Hkv, D, block, seed=Hq).check((Hq, Hkv, D, block))


@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (8, 2), (29, 1)])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_several_tokens_are_causal(Hq, Hkv, D):
    new = [1, 3, 0, 8, 17, 2, 40, 5]
    lens = [30, 3, 9, 70, 17, 1, 300, 0]            # also fewer keys than new tokens: rows that see nothing
    y = Batch(new, lens, Hq, Hkv, D, 32, seed=D).check()
    assert (y[1 + 3 + 8 + 17] == 0).all() and (y[-5:] == 0).all()


def test_attention_long_sequence_is_split():
    Batch([1], [40001], 8, 2, 128, 64, seed=2).check()
    Batch([2, 1], [9000, 20011], 8, 1, 64, 128, seed=3).check()


def test_attention_many_short_sequences():
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 90, (700,), generator=g).tolist()
    Batch([1] * 700, lens, 8, 2, 128, 16, seed=4).check()


def test_attention_sharp_and_flat_softmax():
    Batch([1, 1], [700, 3000], 8, 2, 128, 64, seed=6, q_std=30.0).check("sharp")
    bt = Batch([1, 1], [700, 3000], 8, 2, 128, 64, seed=7)
    bt.check("flat", scale=0.0)
    bt.check("negative", scale=-0.2)


def test_attention_exponents_that_differ_by_block():
    # blocks of very different magnitudes: the unit of the weights follows them
    bt = Batch([1], [640], 8, 2, 128, 32, seed=8)
    bt.cache.v_exp.copy_(torch.randint(-32, 9, bt.cache.v_exp.shape, generator=bt.g, device="cuda").to(torch.int8))
    bt.cache.k_exp.copy_(torch.randint(-20, -5, bt.cache.k_exp.shape, generator=bt.g, device="cuda").to(torch.int8))
    ref, tol = bt.attention_ref()
    y = bt.attend()
    big = ref.abs() > 65000                          # beyond fp16
    err = (y.double() - ref).abs()
    assert (err[~big] <= tol[~big]).all()


def test_what_lies_behind_the_end_is_not_seen():
    # NaN codes behind each sequence's last token, in the same block and in
    # blocks that no table names
    bt = Batch([1, 2, 1], [20, 70, 64], 8, 2, 128, 64, seed=9)
    want = bt.attend().clone()
    used = torch.zeros(bt.blocks, bt.block, dtype=torch.bool, device="cuda")
    for b, n in enumerate(bt.n):
        for j in range(n):
            used[bt.table[b, j // bt.block].long(), j % bt.block] = True
    for c in (bt.cache.k, bt.cache.v):
        c.masked_fill_(~used[:, None, :, None], 0x7F)
    assert torch.equal(bt.attend(), want)
    # table entries behind the sequence's blocks are not looked at either
    wide = torch.full((3, 9), -7, dtype=torch.int32, device="cuda")
    wide[:, :bt.table.shape[1]] = bt.table
    wide[0, 1] = 1 << 30
    bt.table = wide
    assert torch.equal(bt.attend(), want) and bt.status() == awq.AWQ_OK


def test_nan_reaches_the_rows_that_see_it():
    bt = Batch([4], [50], 4, 2, 128, 16, seed=10)
    blk, place = int(bt.table[0, 47 // 16]), 47 % 16
    bt.cache.k[blk, 0, place, 5] = 0x7F              # token 47: seen by new rows 1, 2 and 3
    y = bt.attend().view(4, 4, 128)
    assert torch.isfinite(y[0]).all() and torch.isnan(y[1:, :2]).all() and torch.isfinite(y[1:, 2:]).all()
    bt.cache.k[blk, 0, place, 5] = 0
    bt.cache.v[blk, 1, place, 9] = 0x7F
    y = bt.attend().view(4, 4, 128)
    nan = torch.isnan(y)
    assert nan[1:, 2:, 9].all() and int(nan.sum()) == 6
    bt = Batch([1, 1], [50, 60], 4, 2, 128, 16, seed=12)
    bt.q = bt.q.clone()
    bt.q[0, 1, 3] = float("inf")
    y = bt.attend().view(2, 4, 128)
    assert torch.isnan(y[0, 1]).all() and torch.isfinite(y[0, 0]).all() and torch.isfinite(y[1]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,G", [(5, 4), (3, 8), (4, 1)])   # two row tiles of 16, or one of 8
def test_nan_codes_of_v_at_every_place(T, G, D):
    for n in range(33, 50):
        bt = Batch([T], [n], 2 * G, 2, D, 32, seed=n)
        token, channel, head = n - 1 - n % T, (7 * n) % D, n % 2
        want = bt.attend().view(T, 2 * G, D).clone()
        bt.cache.v[int(bt.table[0, token // 32]), head, token % 32, channel] = 0xFF if n % 3 else 0x7F
        y = bt.attend().view(T, 2 * G, D)
        hit = torch.zeros_like(y, dtype=torch.bool)
        hit[T - n + token:, head * G:(head + 1) * G, channel] = True
        assert torch.equal(torch.isnan(y), hit), (n, token, channel)
        assert torch.equal(y[~hit], want[~hit])


@pytest.mark.parametrize("n", [3, 40, 4000])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_queries_give_nan_in_their_own_row(n, sign):
    # with codes of one sign all scores of the row are +inf or all -inf: 0 / 0 either way
    bt = Batch([2], [n], 8, 2, 64, 32, seed=16)
    bt.cache.k.copy_(torch.where((bt.cache.k & 0x7F) == 0, torch.full_like(bt.cache.k, 0x38), bt.cache.k & 0x7F))
    bt.q = bt.q.clone()
    bt.q[1, 5, 0] = sign * math.inf
    y = bt.attend()
    ref, tol = bt.attention_ref()
    row = torch.zeros_like(y, dtype=torch.bool)
    row[1, 5 * 64:6 * 64] = True
    assert torch.isnan(y[row]).all()
    assert ((y.double() - ref).abs() <= tol)[~row].all()


def test_exponents_of_any_caller():
    # all 256 values of the exponents: those outside -32 .. 31 count as the nearest of them
    bt = Batch([1, 2], [128 * 16, 128 * 16], 4, 2, 64, 16, seed=17)
    bt.cache.v_exp.copy_(torch.arange(bt.cache.v_exp.numel(), device="cuda").view_as(bt.cache.v_exp).to(torch.int8))
    bt.cache.k_exp.copy_(bt.cache.v_exp.flatten().flip(0).view_as(bt.cache.k_exp))
    y = bt.attend(scale=2.0 ** -40).clone()
    for t in (bt.cache.k_exp, bt.cache.v_exp):
        t.clamp_(-32, 31)
    assert torch.equal(bt.attend(scale=2.0 ** -40), y) and not torch.isnan(y).any()


def test_rows_of_no_sequence_are_left_alone():
    bt = Batch([1, 2], [30, 40], 4, 2, 64, 32, seed=13)
    want = bt.attend()
    q = torch.cat([bt.q, torch.full_like(bt.q, math.nan)])
    y = torch.full((6, 4 * 64), 7.0, device="cuda").half()
    awq.awq_kv8_attention(q, bt.cache, bt.starts, bt.lens, bt.table, bt.ws, y=y)
    assert torch.equal(y[:3], want) and (y[3:] == 7.0).all()
    before = [t.clone() for t in bt.cache]
    bt.append()
    after = [t.clone() for t in bt.cache]
    for t, x in zip(bt.cache, before):
        t.copy_(x)
    kk, vv = (torch.cat([x, torch.full_like(x, math.nan)]) for x in (bt.k, bt.v))
    awq.awq_kv8_append(kk, vv, bt.cache, bt.starts, bt.lens, bt.table, bt.ws)
    same_cache(bt.cache, [t.cpu() for t in after])


def test_bad_contents_are_reported_and_touch_nothing():
    # every index below is checked by the kernels before it is used
    bt = Batch([1, 2], [40, 50], 4, 2, 64, 32, seed=14)
    good = bt.attend().clone()
    assert bt.status() == awq.AWQ_OK
    keep = [t.clone() for t in bt.cache]
    table = bt.table.clone()
    for bad in (-1, bt.blocks, 2 ** 31 - 1, -2 ** 31):
        bt.table = table.clone()
        bt.table[0, 1] = bad                         # the block of sequence 0's new token
        bt.append()
        assert bt.status() == awq.AWQ_ERR_BOUNDS
        y = bt.attend()
        assert bt.status() == awq.AWQ_ERR_BOUNDS and torch.isfinite(y).all()
        for t, x in zip(bt.cache, keep):
            t.copy_(x)
        assert torch.equal(bt.attend()[1:], good[1:])  # the other sequence is as it was
        bt.status()
    bt.table = table
    starts, lens = bt.starts.clone(), bt.lens.clone()
    for s, n in (([0, 9, 3], [40, 50]), ([-4, 1, 3], [40, 50]), ([0, 2, 1], [40, 50]), ([0, 1, 3], [-1, 50]),
                 ([0, 1, 3], [40, 65]), ([0, 1, 3], [2 ** 31 - 1, 50]), ([5, 6, 7], [40, 50]),
                 ([-2 ** 31, 1, 2 ** 31 - 1], [40, 50])):
        bt.starts = torch.tensor(s, dtype=torch.int32, device="cuda")
        bt.lens = torch.tensor(n, dtype=torch.int32, device="cuda")
        bt.append()
        assert bt.status() == awq.AWQ_ERR_BOUNDS, (s, n)
        bt.attend()
        assert bt.status() == awq.AWQ_ERR_BOUNDS, (s, n)
        for t, x in zip(bt.cache, keep):
            t.copy_(x)
    bt.starts, bt.lens = starts, lens
    assert torch.equal(bt.attend(), good) and bt.status() == awq.AWQ_OK


def test_attention_is_deterministic_and_replays_in_a_graph():
    bt = Batch([1] * 9, [1000 + 77 * i for i in range(9)], 32, 8, 128, 64, seed=15)
    y0 = bt.attend().clone()
    for _ in range(5):
        assert torch.equal(bt.attend(), y0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        y1 = bt.attend()
    s.synchronize()
    assert torch.equal(y1, y0)
    y = torch.zeros_like(y0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bt.append()
        bt.attend(y=y)
    # replay with contents that grow, as in generation
    for step in range(3):
        bt.k.copy_(torch.randn(bt.k.shape, generator=bt.g, device="cuda").half())
        bt.q.copy_(torch.randn(bt.q.shape, generator=bt.g, device="cuda").half())
        bt.n = [n - step for n in bt.n]
        bt.lens.copy_(torch.tensor(bt.n, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        ref, tol = bt.attention_ref()
        assert ((y.double() - ref).abs() <= tol).all()
    assert bt.status() == awq.AWQ_OK


def test_two_streams_at_once():
    # two batches over one cache, each with its own workspace, on two streams
    one = Batch([1] * 20, [300 + 90 * i for i in range(20)], 32, 8, 128, 64, seed=23)
    other = Batch([3] * 20, one.n, 32, 8, 128, 64, seed=24)
    other.cache, other.table = one.cache, one.table
    torch.cuda.synchronize()
    want = [b.attend().clone() for b in (one, other)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, b in enumerate((one, other)):
            with torch.cuda.stream(streams[i]):
                got[i].append(b.attend())
    torch.cuda.synchronize()
    for i, b in enumerate((one, other)):
        assert all(torch.equal(y, want[i]) for y in got[i])
        assert b.status() == awq.AWQ_OK


@pytest.mark.parametrize("T", [4, 5, 9])
@pytest.mark.parametrize("D,block", [(128, 64), (64, 16)])
def test_few_long_sequences_with_drafts(T, D, block):
    # 16-row tiles (4 to 9 tokens of 4 query heads), both depths of the ring
    for lens in ([20011], [9000, 77, 4100, 12345, 3, 8191]):
        bt = Batch([T] * len(lens), lens, 32, 8, D, block, seed=25)
        bt.append()
        bt.check((T, lens))


def test_strided_rows_and_binding_checks():
    bt = Batch([1, 1, 1], [40, 50, 60], 8, 2, 64, 32, seed=16)
    want = bt.attend()
    assert bt.q.stride(0) == 12 * 64
    q = bt.q.contiguous()
    assert torch.equal(awq.awq_kv8_attention(q, bt.cache, bt.starts, bt.lens, bt.table, bt.ws), want)
    with pytest.raises(ValueError):
        awq.awq_kv8_attention(q.transpose(1, 2).contiguous().transpose(1, 2), bt.cache, bt.starts, bt.lens, bt.table, bt.ws)
    with pytest.raises(ValueError):
        awq.awq_kv8_attention(q[:, :, :32], bt.cache, bt.starts, bt.lens, bt.table, bt.ws)
    with pytest.raises(ValueError):
        awq.awq_kv8_attention(q, bt.cache, bt.starts[:3], bt.lens, bt.table, bt.ws)
    with pytest.raises(ValueError):
        awq.awq_kv8_attention(q, bt.cache, bt.starts, bt.lens.long(), bt.table, bt.ws)
    with pytest.raises(ValueError):
        awq.awq_kv8_append(bt.k[:2], bt.v, bt.cache, bt.starts, bt.lens, bt.table, bt.ws)
    with pytest.raises(awq.AwqError) as e:
        awq.awq_kv8_attention(q, bt.cache, bt.starts, bt.lens, bt.table, bt.ws[:256])
    assert e.value.status == awq.AWQ_ERR_WORKSPACE
    empty = awq.awq_kv8_attention(q[:0], bt.cache, bt.starts[:1], bt.lens[:0], bt.table[:0], bt.ws)
    assert empty.shape == (0, 512)


def test_offsets_beyond_32_bits():
    # 5 GiB of codes per part; the sequence's blocks lie at the pool's end
    free, _ = torch.cuda.mem_get_info()
    assert free > 14 << 30
    Hkv, D, block = 8, 128, 128
    blocks = (5 << 30) // (Hkv * D * block)
    bt = Batch([1], [300], 16, 8, D, block, seed=17)
    old = bt.cache
    big = awq.Kv8Cache(torch.zeros(blocks, Hkv, block, D, dtype=torch.uint8, device="cuda"),
                       torch.zeros(blocks, Hkv, block, D, dtype=torch.uint8, device="cuda"),
                       torch.zeros(blocks, Hkv, dtype=torch.int8, device="cuda"),
                       torch.zeros(blocks, Hkv, dtype=torch.int8, device="cuda"))
    bt.append()
    want = bt.attend()
    rows = bt.table[0].long()
    at = torch.arange(blocks - len(rows), blocks, device="cuda")
    for t, s in zip(big, old):
        t[at] = s[rows]
    bt.cache, bt.table = big, at.to(torch.int32).view(1, -1)
    assert torch.equal(bt.attend(), want)
    bt.append()
    for t, s in zip(big, old):
        assert torch.equal(t[at], s[rows])


def test_more_sequences_than_a_grid_dimension_holds():
    # one token each: the attention returns the value that the cache holds
    B, D = 70001, 64
    g = torch.Generator(device="cuda").manual_seed(18)
    q, k, v = (torch.randn(B, 1, D, generator=g, device="cuda").half() for _ in "qkv")
    cache = awq.new_kv8_cache(B, 1, 16, D, "cuda")
    starts = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    table = torch.randperm(B, generator=g, device="cuda").to(torch.int32).view(B, 1)
    ws = awq.new_kv8_workspace(B, B, 1, 1, D, "cuda")
    awq.awq_kv8_append(k, v, cache, starts, lens, table, ws)
    y = awq.awq_kv8_attention(q, cache, starts, lens, table, ws)
    assert awq.awq_get_status(ws) == awq.AWQ_OK
    rows = table.view(-1).long()
    for src, codes, exps in ((k, cache.k, cache.k_exp), (v, cache.v, cache.v_exp)):
        amax = src.view(B, D).double().abs().amax(dim=1)
        e = exps[rows].view(B).double()
        assert (amax <= 448 * torch.exp2(e)).all() and (amax > 448 * torch.exp2(e - 1)).all()
        assert torch.equal(codes[rows, 0, 0], (src.view(B, D).double() * torch.exp2(-e)[:, None]).float().to(E4M3).view(torch.uint8))
    held = values(cache.v[rows], cache.v_exp[rows])[:, 0, 0]
    assert torch.equal(y.double(), held)


def test_a_prompt_in_pieces_equals_the_prompt_at_once():
    # attention of a prompt appended and read in pieces against all of it: the
    # same tokens see the same keys (the codes differ where a block was filled in
    # two pieces, so the pieces end on blocks)
    T, block = 704, 64
    bt = Batch([T], [T], 8, 2, 128, block, seed=19, empty=True)
    bt.append()
    bt.check("prompt")
    codes = [t.clone() for t in bt.cache]
    q, k, v = bt.q, bt.k, bt.v
    for t in bt.cache:
        t.zero_()
    at = 0
    for n in (64, 320, 128, 192):
        bt.new, bt.R, bt.starts_h = [n], n, [0, n]
        bt.starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        bt.n, bt.lens = [at + n], torch.tensor([at + n], dtype=torch.int32, device="cuda")
        bt.q, bt.k, bt.v = (x[at:at + n] for x in (q, k, v))
        bt.append()
        bt.check("piece")
        at += n
    for a, b in zip(bt.cache, codes):
        assert torch.equal(a, b)


@pytest.mark.parametrize("capacity", [512, 528])
def test_both_ways_of_sharing_out_the_work(capacity):
    # the same batch with a block table at and above the size up to which CTAs
    # take whole groups
    lens = [1, 16, 130, 512, 500]
    bt = Batch([1, 1, 2, 1, 3], lens, 16, 2, 64, 16, seed=22)
    table = torch.full((5, capacity // 16), -1, dtype=torch.int32, device="cuda")
    table[:, :bt.table.shape[1]] = bt.table
    bt.table = table
    bt.check(capacity)


def test_append_beside_exponents_of_any_caller():
    # blocks that hold tokens under each of the 256 exponents, as the attention
    # reads them (-32 .. 31), get a token more: what they held keeps its value
    for seed, std in ((26, 1.0), (27, 2e-7), (28, 2e4)):
        bt = Batch([1] * 256, [6 + b % 9 for b in range(256)], 4, 2, 64, 16, seed=seed, spare=0)
        bt.k, bt.v = bt.k * std, bt.v * std
        e = torch.arange(-128, 128, device="cuda").to(torch.int8)
        bt.cache.k_exp[bt.table[:, 0].long()] = e[:, None].expand(-1, 2)
        bt.cache.v_exp[bt.table[:, 0].long()] = e.flip(0)[:, None].expand(-1, 2)
        want = append_model(bt, [bt.cache.k, bt.cache.v, bt.cache.k_exp.clamp(-32, 31), bt.cache.v_exp.clamp(-32, 31)])
        bt.append()
        same_cache(bt.cache, want)
        assert bt.status() == awq.AWQ_OK


@pytest.mark.parametrize("D,block", [(128, 64), (64, 16), (128, 16), (64, 64), (128, 128)])
def test_append_of_many_sequences_is_bit_exact(D, block):
    # more blocks than CTAs: each takes a range of them, over empty sequences too
    g = torch.Generator().manual_seed(29)
    new = torch.tensor([0, 1, 1, 3, 40, 130])[torch.randint(0, 6, (1100,), generator=g)]
    new[100:290] = 0                                 # more than a few times 32 without new tokens
    new[-40:] = 0
    past = torch.randint(0, 90, (1100,), generator=g)
    past[300:320] = -2                               # rows without a place
    lens = (new + past).clamp(min=0)
    bt = Batch(new.tolist(), lens.tolist(), 4, 2, D, block, seed=block)
    want = append_model(bt, bt.cache)
    keep = [t.clone() for t in bt.cache]
    bt.append()
    same_cache(bt.cache, want)
    assert bt.status() == awq.AWQ_OK
    # a bad block number in the middle of a CTA's range changes nothing else
    b = 500 + int((new[500:] > 0).int().argmax())
    j = int(lens[b] - 1) // block
    good = int(bt.table[b, j])
    bt.table[b, j] = bt.blocks
    for t, x in zip(bt.cache, keep):
        t.copy_(x)
    bt.append()
    assert bt.status() == awq.AWQ_ERR_BOUNDS
    for w, x in zip(want, keep):
        w[good] = x[good].cpu()
    same_cache(bt.cache, want)


def test_append_grows_with_the_sequences_and_not_their_square():
    times = []
    for B in (4096, 32768):
        H, D, block = 8, 64, 16
        cache = awq.new_kv8_cache(B, H, block, D, "cuda")
        k, v = (torch.randn(B, H, D, device="cuda").half() for _ in "kv")
        starts = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        lens = torch.full((B,), 9, dtype=torch.int32, device="cuda")
        table = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
        ws = awq.new_kv8_workspace(B, B, H, H, D, "cuda")
        best = math.inf
        for _ in range(5):
            t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            t0.record()
            awq.awq_kv8_append(k, v, cache, starts, lens, table, ws)
            t1.record()
            torch.cuda.synchronize()
            best = min(best, t0.elapsed_time(t1))
        times.append(best)
    assert times[1] < 24 * times[0], times           # 8 times the sequences: 8, where the square would be 64


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_largest_scores(D, sign):
    # the largest q, codes, exponents and scale: every key of a row has the same
    # score of about 2^95, whose fp32 steps are far above 1, so which keys count is
    # open; y is a mean of some of them, not NaN
    bt = Batch([1, 2], [700, 1300], 8, 2, D, 64, seed=31)
    bt.q = torch.full_like(bt.q, 65504.0)
    bt.cache.k.fill_(0x7E)
    bt.cache.k_exp.fill_(31)
    y = bt.attend(scale=sign * 2.0 ** 32).double().unflatten(1, (2, 4, D))
    assert bt.status() == awq.AWQ_OK
    for b in range(2):
        v = bt.kept(b, "v")[0]
        slack = 2.0 ** -10 * v.abs().amax(dim=0)[:, None]      # the weights' rounding and y's
        r = y[bt.starts_h[b]:bt.starts_h[b + 1]]
        assert (r <= v.amax(dim=0)[:, None] + slack).all() and (r >= v.amin(dim=0)[:, None] - slack).all()
