"""Cases, plain forms and definitions of the operators between a decoder
layer's 4-bit linear layers: RMS norm with the residual's addition, the gated
SiLU, and the 8-bit key/value cache with the attention that reads it.

``run`` computes a case in elementary torch operations (``own`` False) or
through the library's entry points (``own`` True); ``exact`` computes it from
the definition in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
MIN_EXP = -32   # exponent of a cache block that holds only zeros


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm(name, M, K, residual, out):
    return {"name": name, "op": "rmsnorm", "M": M, "K": K, "residual": residual, "out": out}


def _silu(name, M, F, out):
    return {"name": name, "op": "silu_mul", "M": M, "F": F, "out": out}


def _append(name, B, new_lo, new_hi, past_lo, past_hi, Hq, Hkv, D, block):
    return {"name": name, "op": "kv8_append", "B": B, "new_lo": new_lo, "new_hi": new_hi, "past_lo": past_lo,
            "past_hi": past_hi, "Hq": Hq, "Hkv": Hkv, "D": D, "block": block}


def _attention(name, B, new_lo, new_hi, past_lo, past_hi, Hq, Hkv, D, block):
    return {**_append(name, B, new_lo, new_hi, past_lo, past_hi, Hq, Hkv, D, block), "op": "kv8_attention"}


def listed():
    return [
        # one token of LLaMA-3-8B in generation: latency
        _norm("norm_8b_token", 1, 4096, True, "fp16"),
        # a prompt batch of LLaMA-2-70B on the W4A8 path
        _norm("norm_70b_prompt_fp8", 8192, 8192, True, "fp8"),
        # the first norm of a Falcon-180B-wide layer (no residual yet), odd batch
        _norm("norm_14848_odd", 517, 14848, False, "fp16"),
        # a small generation batch, LLaMA-3-8B feed-forward
        _silu("silu_8b_batch8", 8, 14336, "fp16"),
        # a prompt batch, LLaMA-3-8B feed-forward on the W4A8 path
        _silu("silu_8b_prompt_fp8", 8192, 14336, "fp8"),
        # one generated token per sequence, 32 sequences
        _append("append_8b_batch32", 32, 1, 1, 100, 2000, 32, 8, 128, 64),
        # prompts of different lengths entering the cache, some behind a past
        _append("append_8b_prompts", 12, 30, 1500, 0, 700, 32, 8, 128, 64),
        # one short sequence: latency
        _attention("attn_8b_short", 1, 1, 1, 499, 499, 32, 8, 128, 64),
        # one long sequence: work is split along the keys
        _attention("attn_8b_long", 1, 1, 1, 131001, 131001, 32, 8, 128, 64),
        # a ragged generation batch
        _attention("attn_8b_batch48", 48, 1, 1, 37, 8190, 32, 8, 128, 64),
        # LLaMA-2-7B heads (every head with its own keys), small pages
        _attention("attn_7b_batch16", 16, 1, 1, 500, 2047, 32, 32, 128, 16),
        # several tokens at once (checking drafted tokens), 64-wide heads
        _attention("attn_d64_drafts", 24, 1, 5, 200, 4100, 64, 8, 64, 32),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rmsnorm", "silu_mul", "kv8_append", "kv8_attention", "kv8_attention"])
    if op == "rmsnorm":
        K = 8 * _log(rng, 16, 2048)
        M = _log(rng, 1, 8192)
        while M * K > 8192 * 8192:
            M //= 2
        c = _norm("", M, K, rng.random() < 0.7, rng.choice(["fp16", "fp8"]))
    elif op == "silu_mul":
        F = 8 * _log(rng, 16, 3584)
        M = _log(rng, 1, 8192)
        while M * F > 8192 * 14336:
            M //= 2
        c = _silu("", M, F, rng.choice(["fp16", "fp8"]))
    else:
        Hkv = rng.choice([1, 2, 4, 8, 8, 8, 32])
        G = 1 if Hkv == 32 else rng.choice([1, 4, 4, 7, 8])
        D, block = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
        if op == "kv8_append":
            B = _log(rng, 1, 32)
            hi = rng.choice([1, 1, _log(rng, 2, 1500)])
            while B * hi * Hkv > 12 * 1500 * 8:
                hi = max(1, hi // 2)
            past = _log(rng, 1, 2000)
            c = _append("", B, max(1, hi // rng.choice([1, 7, 30])), hi, past // 5, past, G * Hkv, Hkv, D, block)
        else:
            B = _log(rng, 1, 64)
            hi = rng.choice([1, 1, 1, rng.randint(2, 6)])
            past = _log(rng, 1, 65536)
            while B * (past + hi) * Hkv * D > 48 * 8191 * 8 * 128 // 2:
                past //= 2
            c = _attention("", B, max(1, hi - 3), hi, past // rng.choice([1, 3, 50]), past, G * Hkv, Hkv, D, block)
    del c["name"]
    return c


def _spread(lo, hi, B, turn):
    """B whole numbers from lo to hi, in an order that mixes long and short."""
    return [lo + (hi - lo) * ((b * 7 + turn) % B) // max(1, B - 1) for b in range(B)]


def _lengths(case):
    B = case["B"]
    new = _spread(case["new_lo"], case["new_hi"], B, 0)
    past = _spread(case["past_lo"], case["past_hi"], B, 3)
    return new, [p + n for p, n in zip(past, new)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float16) * std)

    s = {"case": case}
    if case["op"] == "rmsnorm":
        M, K = case["M"], case["K"]
        s["x"] = normal(M, K)
        s["x"][:, 3] *= 12.0                     # activations have outlier channels
        s["w"] = (1.0 + 0.2 * torch.randn(K, generator=g, device="cuda")).half()
        s["residual"] = normal(M, K, std=4.0) if case["residual"] else None
        return s
    if case["op"] == "silu_mul":
        s["gate_up"] = normal(case["M"], 2 * case["F"], std=2.0)
        return s

    new, lens = _lengths(case)
    B, Hq, Hkv, D, block = case["B"], case["Hq"], case["Hkv"], case["D"], case["block"]
    R = sum(new)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    # the qkv layer's output: q, k and v are column ranges of it
    qkv = normal(R, (Hq + 2 * Hkv) * D)
    s["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    s["v"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    width = max(-(-n // block) for n in lens)
    blocks = B * width + 1                       # the last block of the pool belongs to no sequence
    s["table"] = torch.randperm(blocks - 1, generator=g, device="cuda").to(torch.int32).view(B, width)
    s["new_hi"] = max(new)

    def codes(std):
        c = torch.empty(blocks, Hkv, block, D, dtype=torch.uint8, device="cuda")
        flat, step = c.view(-1), 1 << 26
        for i in range(0, flat.numel(), step):
            n = min(step, flat.numel() - i)
            v = (torch.randn(n, generator=g, device="cuda") * std).clamp_(-E4M3_MAX, E4M3_MAX)
            flat[i:i + n] = v.to(torch.float8_e4m3fn).view(torch.uint8)
        return c

    def exponents():
        return torch.randint(-7, -4, (blocks, Hkv), generator=g, device="cuda").to(torch.int8)

    s["cache"] = (codes(80.0), codes(64.0), exponents(), exponents())
    if own:
        import weight_only_bit_awq_b200 as awq
        s["cache"] = awq.Kv8Cache(*s["cache"])
        s["ws"] = awq.new_kv8_workspace(R, B, Hq, Hkv, D, "cuda")
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _to_e4m3(y):
    """fp32 rows -> (E4M3 codes, fp32 scale of each row)."""
    sx = y.abs().amax(dim=1) / E4M3_MAX
    scaled = torch.where(sx[:, None] == 0, torch.zeros_like(y), y / sx[:, None])
    return scaled.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), sx


def _plain_rmsnorm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS) * s["w"].float()
    got = {"h": h.half()} if s["residual"] is not None else {}
    if s["case"]["out"] == "fp16":
        return {**got, "y": y.half()}
    x8, sx = _to_e4m3(y)
    return {**got, "x8": x8, "sx": sx}


def _plain_silu_mul(s):
    F = s["case"]["F"]
    g, u = s["gate_up"][:, :F].float(), s["gate_up"][:, F:].float()
    y = g / (1.0 + torch.exp(-g)) * u
    if s["case"]["out"] == "fp16":
        return {"y": y.half()}
    x8, sx = _to_e4m3(y)
    return {"x8": x8, "sx": sx}


def _needed_exponent(amax):
    """Smallest e with amax <= 448 * 2^e; MIN_EXP for amax = 0."""
    m, x = torch.frexp(amax)                     # amax = m * 2^x, m in [0.5, 1)
    e = x - 9 + (m > E4M3_MAX / 512.0).int()
    return torch.where(amax == 0, torch.full_like(e, MIN_EXP), e)


def _pow2(e):
    """2^e in fp32, exactly, for whole e in the normal range."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _plain_append_one(new, codes, exps, blk, rows, is_new, is_old):
    """new [R][H][D] into the blocks blk [B][N] of one of the two caches; rows
    [B][N][T]: which new row each token of a block takes, where is_new; is_old:
    the tokens that were there before."""
    mine = is_new[:, :, None, :, None]
    old = codes[blk].view(torch.float8_e4m3fn).float()                       # [B][N][H][T][D]
    fresh = new.float()[rows].permute(0, 1, 3, 2, 4)
    amax = torch.where(mine, fresh, torch.zeros_like(fresh)).abs().amax(dim=(3, 4))
    had = is_old.any(dim=2)[:, :, None]
    e_old = torch.where(had, exps[blk].int(), torch.full_like(exps[blk], MIN_EXP).int())
    e = torch.maximum(_needed_exponent(amax), e_old)
    touched = is_new.any(dim=2)[:, :, None]
    e = torch.where(touched, e, exps[blk].int())
    moved = torch.where(is_old[:, :, None, :, None], old * _pow2(exps[blk].int() - e)[..., None, None], old)
    value = torch.where(mine, fresh * _pow2(-e)[..., None, None], moved)
    codes[blk] = value.to(torch.float8_e4m3fn).view(torch.uint8)
    exps[blk] = e.to(torch.int8)


def _plain_append(s):
    block, B = s["case"]["block"], s["case"]["B"]
    kc, vc, ke, ve = s["cache"]
    lens, starts = s["lens"].long(), s["starts"].long()
    past = lens - (starts[1:] - starts[:-1])
    N = (s["new_hi"] + block - 2) // block + 1
    j = past[:, None] // block + torch.arange(N, device="cuda")               # block of the sequence [B][N]
    there = j <= (lens[:, None] - 1) // block
    spare = kc.shape[0] - 1
    blk = torch.where(there, torch.gather(s["table"].long(), 1, j.clamp(max=s["table"].shape[1] - 1)), spare)
    pos = j[:, :, None] * block + torch.arange(block, device="cuda")          # [B][N][T]
    is_new = there[:, :, None] & (pos >= past[:, None, None]) & (pos < lens[:, None, None])
    is_old = there[:, :, None] & (pos < past[:, None, None])
    rows = (starts[:-1, None, None] + pos - past[:, None, None]).clamp(0, s["k"].shape[0] - 1)
    _plain_append_one(s["k"], kc, ke, blk, rows, is_new, is_old)
    _plain_append_one(s["v"], vc, ve, blk, rows, is_new, is_old)
    return {"k": kc.view(torch.float8_e4m3fn), "v": vc.view(torch.float8_e4m3fn), "k_exp": ke, "v_exp": ve}


def _plain_values(codes, exps, table):
    """[B][H][tokens][D] values of the sequences' blocks."""
    t = table.long()
    x = codes[t].view(torch.float8_e4m3fn).float() * _pow2(exps[t])[..., None, None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_attention(s):
    c = s["case"]
    B, Hq, Hkv, D, T = c["B"], c["Hq"], c["Hkv"], c["D"], s["new_hi"]
    R, G = s["q"].shape[0], Hq // Hkv
    kc, vc, ke, ve = s["cache"]
    lens, starts = s["lens"].long(), s["starts"].long()
    t = torch.arange(T, device="cuda")
    row = starts[:-1, None] + t                                               # [B][T]
    row = torch.where(row < starts[1:, None], row, R)
    q = s["q"].float()[row.clamp(max=R - 1)]                                  # [B][T][Hq][D]
    q = q.view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    k, v = _plain_values(kc, ke, s["table"]), _plain_values(vc, ve, s["table"])
    x = q @ k.transpose(2, 3) / math.sqrt(D)
    seen = (lens - (starts[1:] - starts[:-1]))[:, None] + t + 1               # keys a token sees [B][T]
    masked = torch.arange(k.shape[2], device="cuda") >= seen[:, :, None]      # [B][T][L]
    x = x.view(B, Hkv, T, G, -1).masked_fill(masked[:, None, :, None], -math.inf)
    top = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(dim=-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).view(B, Hkv, T, G, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    out = torch.zeros(R + 1, Hq * D, dtype=torch.float16, device="cuda")
    out[row] = o.permute(0, 2, 1, 3, 4).reshape(B, T, Hq * D).half()
    return {"y": out[:R]}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _own_run(s):
    import weight_only_bit_awq_b200 as awq
    c = s["case"]
    e4m3 = torch.float8_e4m3fn
    if c["op"] == "rmsnorm":
        if c["out"] == "fp16":
            got = awq.awq_rmsnorm(s["x"], s["w"], EPS, residual=s["residual"])
            return {"y": got} if s["residual"] is None else {"h": got[1], "y": got[0]}
        got = awq.awq_rmsnorm_fp8(s["x"], s["w"], EPS, residual=s["residual"])
        return {**({"h": got[2]} if s["residual"] is not None else {}), "x8": got[0].view(e4m3), "sx": got[1]}
    if c["op"] == "silu_mul":
        if c["out"] == "fp16":
            return {"y": awq.awq_silu_mul(s["gate_up"])}
        x8, sx = awq.awq_silu_mul_fp8(s["gate_up"])
        return {"x8": x8.view(e4m3), "sx": sx}
    if c["op"] == "kv8_append":
        awq.awq_kv8_append(s["k"], s["v"], s["cache"], s["starts"], s["lens"], s["table"], s["ws"])
        kc, vc, ke, ve = s["cache"]
        return {"k": kc.view(e4m3), "v": vc.view(e4m3), "k_exp": ke, "v_exp": ve}
    return {"y": awq.awq_kv8_attention(s["q"], s["cache"], s["starts"], s["lens"], s["table"], s["ws"])}


def run(state):
    if own:
        return _own_run(state)
    return {"rmsnorm": _plain_rmsnorm, "silu_mul": _plain_silu_mul, "kv8_append": _plain_append,
            "kv8_attention": _plain_attention}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "rmsnorm":
        n = case["M"] * case["K"]
        b = 2 * n + (4 * n if case["residual"] else 0) + 2 * case["K"]
        b += 2 * n if case["out"] == "fp16" else n + 4 * case["M"]
        return {"bytes": b, "flops": (5 if case["residual"] else 4) * n}
    if case["op"] == "silu_mul":
        n = case["M"] * case["F"]
        return {"bytes": 4 * n + (2 * n if case["out"] == "fp16" else n + 4 * case["M"]), "flops": 5 * n}
    new, lens = _lengths(case)
    R, Hq, Hkv, D, block = sum(new), case["Hq"], case["Hkv"], case["D"], case["block"]
    if case["op"] == "kv8_append":
        pages = sum((n - 1) // block - (n - t) // block + 1 for t, n in zip(new, lens))
        return {"bytes": 2 * (3 * R * Hkv * D + pages * Hkv) + 4 * (pages + 2 * case["B"]), "flops": 4 * R * Hkv * D}
    pages = sum(-(-n // block) for n in lens)
    seen = sum(t * (n - t) + t * (t + 1) // 2 for t, n in zip(new, lens))
    return {"bytes": 4 * R * Hq * D + 2 * Hkv * (sum(lens) * D + pages) + 4 * (pages + 2 * case["B"]),
            "flops": 4 * seen * Hq * D}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_scaled(y):
    """y and its E4M3 form: the values before their rounding to 8 bits, and the row scales."""
    sx = y.abs().max(dim=1).values / 448.0
    return {"x8": y / torch.where(sx > 0, sx, torch.ones_like(sx)).unsqueeze(1), "sx": sx}


def _exact_append(new, codes, exps, table, starts, lens, block):
    value, e_out = codes.view(torch.float8_e4m3fn).double(), exps.clone()
    for b in range(len(lens)):
        T = starts[b + 1] - starts[b]
        for j in range((lens[b] - T) // block, (lens[b] - 1) // block + 1):
            blk = int(table[b, j])
            p0, p1 = max(lens[b] - T, j * block), min(lens[b], (j + 1) * block)
            x = new[starts[b] + p0 - (lens[b] - T):starts[b] + p1 - (lens[b] - T)].double()    # [t][H][D]
            big = x.abs().amax(dim=(0, 2)).clamp(min=448.0 * 2.0 ** MIN_EXP)
            e = torch.ceil(torch.log2(big / 448.0)).long()
            e += (big > 448.0 * torch.exp2(e.double())).long() - (big <= 448.0 * torch.exp2(e.double() - 1)).long()
            if p0 > j * block:
                e = torch.maximum(e, exps[blk].long())
                value[blk][:, :p0 - j * block] *= torch.exp2((exps[blk].long() - e).double()).view(-1, 1, 1)
            value[blk][:, p0 - j * block:p1 - j * block] = (x * torch.exp2(-e.double()).view(1, -1, 1)).transpose(0, 1)
            e_out[blk] = e.to(torch.int8)
    return value, e_out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "rmsnorm":
        h = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
        y = h / torch.sqrt(h.square().sum(dim=1, keepdim=True) / case["K"] + EPS) * s["w"].double()
        got = {} if s["residual"] is None else {"h": h}
        return {**got, "y": y} if case["out"] == "fp16" else {**got, **_exact_scaled(y)}
    if case["op"] == "silu_mul":
        g, u = s["gate_up"].double().split(case["F"], dim=1)
        y = g * torch.sigmoid(g) * u
        return {"y": y} if case["out"] == "fp16" else _exact_scaled(y)
    starts, lens, block = s["starts"].tolist(), s["lens"].tolist(), case["block"]
    kc, vc, ke, ve = s["cache"]
    if case["op"] == "kv8_append":
        table = s["table"].cpu()
        k, k_exp = _exact_append(s["k"], kc, ke, table, starts, lens, block)
        v, v_exp = _exact_append(s["v"], vc, ve, table, starts, lens, block)
        return {"k": k, "v": v, "k_exp": k_exp, "v_exp": v_exp}
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    out = torch.zeros(s["q"].shape[0], Hq, D, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        T = starts[b + 1] - starts[b]
        pages = s["table"][b, :-(-lens[b] // block)].long()
        for h in range(Hkv):
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            k, v = (c[pages, h].view(torch.float8_e4m3fn).double() * torch.exp2(e[pages, h].double()).view(-1, 1, 1)
                    for c, e in ((kc, ke), (vc, ve)))
            k, v = k.reshape(-1, D)[:lens[b]], v.reshape(-1, D)[:lens[b]]
            for t in range(T):
                n = lens[b] - T + t + 1
                q = s["q"][starts[b] + t, heads].double()
                out[starts[b] + t, heads] = torch.softmax(q @ k[:n].T / math.sqrt(D), dim=1) @ v[:n]
    return {"y": out.flatten(1)}
