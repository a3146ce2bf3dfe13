"""The cache-compression operators as measured work: a 4-bit paged cache (written, converted, attended) and eviction by accumulated attention weight.

A case names one operator and its sizes.  `run` computes it with elementary torch operations where `own` is false, and by
the library's public calls where it is true; `exact` computes the definition in 64 bits.

The 4-bit pool (uint8 [blocks][heads][9 * head_dim], one 16-token tile per block and head):
  bytes [0, 8 D)     data [D / 32 pieces][16 tokens][16 bytes]; byte b of piece c holds dimension 32 c + 2 b in its low
                     half and 32 c + 2 b + 1 in its high half
  bytes [8 D, 9 D)   one 32-bit word per 64 dimensions, [D / 64 groups][16 tokens]: the scale s (bf16) in the upper
                     half, the zero point z (a whole number, fp16) in the lower; a value n stands for s (n - z)
Quantisation of a group of 64 values x:  s = bf16(max((max x - min x) / 15, max |x| / 2000)),  z = round(-min x / s),
n = clamp(round(x / s) + z, 0, 15); a group with s = 0 holds n = z = 0.
"""
import math

import torch

own = False

BLOCK = 16
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---- cases ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 200 requests: each appends one token, and its tail block is read back in 16 bits
        {"name": "append_step_200", "op": "append", "seqs": 200, "new": 1, "start": 500, "heads": 32, "dim": 128, "type": "f16"},
        # chunked prefill: 8 prompts bring 2045 tokens each from the middle of a block; the chunk's attention reads them back
        {"name": "append_chunk_8x2045", "op": "append", "seqs": 8, "new": 2045, "start": 7, "heads": 32, "dim": 128, "type": "f16"},
        # a shared 1000-token prefix (63 blocks) of a small model goes to 4 bits, and back for its next prompt
        {"name": "convert_prefix_63", "op": "convert", "blocks": 63, "heads": 8, "dim": 64, "type": "bf16"},
        # four 4096-token prompts go from the prefill's pool to 4 bits, and back
        {"name": "convert_prompts_1024", "op": "convert", "blocks": 1024, "heads": 32, "dim": 128, "type": "f16"},
        # four short requests of a small model: latency
        {"name": "decode4_short", "op": "decode4", "seqs": 4, "lens": "uniform", "max": 33, "heads": 2, "group": 1, "dim": 64, "type": "f16"},
        # one layer of the decode step: 200 requests, lengths exponential with mean 500 up to 2048
        {"name": "decode4_step_200", "op": "decode4", "seqs": 200, "lens": "exp", "max": 2048, "heads": 32, "group": 1, "dim": 128, "type": "f16"},
        # grouped queries, 64 requests
        {"name": "decode4_gqa8_64", "op": "decode4", "seqs": 64, "lens": "uniform", "max": 2048, "heads": 8, "group": 8, "dim": 128, "type": "bf16"},
        # long contexts
        {"name": "decode4_long_8x32768", "op": "decode4", "seqs": 8, "lens": "full", "max": 32768, "heads": 32, "group": 1, "dim": 128, "type": "f16"},
        # one layer of decode over a 16-bit cache that also gathers each token's attention weight
        {"name": "mass_64", "op": "mass", "q4": False, "seqs": 64, "lens": "uniform", "max": 2048, "heads": 32, "group": 1, "dim": 128, "type": "f16"},
        # the same over a 4-bit cache with grouped queries
        {"name": "mass4_gqa4_200", "op": "mass", "q4": True, "seqs": 200, "lens": "exp", "max": 2048, "heads": 8, "group": 4, "dim": 128, "type": "bf16"},
        # 200 requests, those over 1024 tokens go back to it
        {"name": "evict_200_to_1024", "op": "evict", "seqs": 200, "lens": "uniform", "max": 2048, "keep": 1024, "sinks": 4, "recent": 128, "heads": 8, "dim": 128, "type": "f16"},
        # long contexts to a quarter
        {"name": "evict_8x32768_to_8192", "op": "evict", "seqs": 8, "lens": "full", "max": 32768, "keep": 8192, "sinks": 4, "recent": 1000, "heads": 8, "dim": 128, "type": "bf16"},
    ]


def draw(rng):
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["append", "convert", "decode4", "mass", "evict"])
    heads, dim, kind = log_int(1, 32), rng.choice([64, 128]), rng.choice(["f16", "bf16"])
    if op == "append":
        seqs = log_int(1, 200)
        return {"op": op, "seqs": seqs, "new": log_int(1, max(1, 16360 // seqs)), "start": rng.randint(0, 500), "heads": heads, "dim": dim, "type": kind}
    if op == "convert":
        return {"op": op, "blocks": log_int(1, 1024), "heads": heads, "dim": dim, "type": kind}
    seqs = log_int(1, 200)
    if op == "evict":
        longest = log_int(16, min(32768, 262144 // seqs))
        keep = rng.randint(1, longest)
        return {"op": op, "seqs": seqs, "lens": rng.choice(["uniform", "exp", "full"]), "max": longest, "keep": keep,
                "sinks": rng.choice([0, 1, 4]), "recent": rng.randint(0, keep), "heads": min(heads, 8), "dim": dim,
                "type": rng.choice(["f32", "f16", "bf16"]) if seqs * longest <= 131072 else kind}
    group = rng.choice([1, 2, 4, 8])
    c = {"op": op, "seqs": seqs, "lens": rng.choice(["uniform", "exp", "full"]), "heads": heads, "group": group, "dim": dim, "type": kind}
    c["max"] = log_int(1, min(32768, 262144 * 8 // max(8, heads * group) // seqs))
    if op == "mass":
        c["q4"] = rng.random() < 0.5
        c["type"] = kind if c["q4"] else rng.choice(["f32", "f16", "bf16"])
        c["max"] = min(c["max"], max(1, 65536 * 8 // heads // seqs))
    return c


def lengths(c):
    """Context lengths of a case, ascending: the middle of each of `seqs` equal shares of the distribution."""
    at = [(i + 0.5) / c["seqs"] for i in range(c["seqs"])]
    if c["lens"] == "full":
        return [c["max"]] * c["seqs"]
    if c["lens"] == "uniform":
        return [min(c["max"], 1 + int(u * c["max"])) for u in at]
    return [min(c["max"], 1 + int(-c["max"] / 4.096 * math.log(1 - u))) for u in at]


# ---- the 4-bit format, elementary ------------------------------------------------------

def quantise(x, real=torch.float32):
    """x [..., D] -> whole numbers n [..., D], scales and zero points [..., D / 64]."""
    g = x.to(real).unflatten(-1, (-1, 64))
    hi, lo, top = g.amax(-1), g.amin(-1), g.abs().amax(-1)
    # quotients by tensors: by a plain number they would be products with its rounded reciprocal, and ties would fall apart
    s = torch.maximum((hi - lo) / torch.full_like(hi, 15), top / torch.full_like(hi, 2000)).to(torch.bfloat16).to(real)
    d = torch.where(s == 0, 1, s)
    z = torch.round(-lo / d)
    n = (torch.round(g / d[..., None]) + z[..., None]).clamp(0, 15)
    return n.flatten(-2), s, z


def pack(n, s, z):
    """Tokens of whole blocks [blocks, H, 16, D] as a 4-bit pool."""
    nb, h, _, dim = n.shape
    b = n.to(torch.uint8).view(nb, h, 16, dim // 32, 16, 2)
    data = (b[..., 0] | b[..., 1] << 4).transpose(2, 3)
    words = torch.stack([z.to(torch.float16).view(torch.uint8).view(nb, h, 16, -1, 2),
                         s.to(torch.bfloat16).view(torch.uint8).view(nb, h, 16, -1, 2)], -2)
    return torch.cat([data.reshape(nb, h, 8 * dim), words.transpose(2, 3).reshape(nb, h, dim)], -1)


def values(tiles, dim, real=torch.float32):
    """Tiles of a 4-bit pool [..., 9 D] -> the values that they stand for [..., 16, D]."""
    data = tiles[..., :8 * dim].unflatten(-1, (dim // 32, 16, 16))
    n = torch.stack([data & 15, data >> 4], -1).flatten(-2).transpose(-3, -2).flatten(-2)
    words = tiles[..., 8 * dim:].unflatten(-1, (dim // 64, 16, 4)).transpose(-3, -2)
    z = words[..., :2].contiguous().view(torch.float16)
    s = words[..., 2:].contiguous().view(torch.bfloat16)
    n = n.to(real).unflatten(-1, (-1, 64))
    return (s.to(real) * (n - z.to(real))).flatten(-2)


def rounded(x, kind):
    top = torch.finfo(kind).max
    return x.clamp(-top, top).to(kind)


# ---- inputs --------------------------------------------------------------------------

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind, dim, heads = DTYPES[c["type"]], c["dim"], c["heads"]
    st = {"case": c, "kind": kind}

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=kind)

    def spread(*shape):
        # keys and values of a model: channels of different size and offset
        size = torch.exp(0.5 * torch.randn((shape[-1],), generator=g, device="cuda"))
        return (torch.randn(shape, generator=g, device="cuda") * size + 0.5 * size.flip(0)).to(kind)

    def order(n):
        return torch.randperm(n, generator=g, device="cuda").to(torch.int32)

    def four(nb):
        return pack(*quantise(spread(nb, heads, BLOCK, dim)))

    if c["op"] == "append":
        first = c["start"] % BLOCK
        per = (first + c["new"] + BLOCK - 1) // BLOCK
        nb = c["seqs"] * per
        tables = order(nb).view(c["seqs"], per)
        at = first + torch.arange(c["new"], device="cuda")
        st["slots"] = (tables[:, at // BLOCK] * BLOCK + at % BLOCK).to(torch.int32).flatten()
        st["k_new"], st["v_new"] = spread(st["slots"].numel(), heads, dim), spread(st["slots"].numel(), heads, dim)
        st["k"], st["v"] = four(nb), four(nb)
        st["pairs"] = torch.stack([tables.flatten(), torch.arange(nb, device="cuda", dtype=torch.int32)], 1).contiguous()
        st["k_out"], st["v_out"] = (torch.zeros((nb, heads, BLOCK, dim), device="cuda", dtype=kind) for _ in range(2))
        return st
    if c["op"] == "convert":
        nb = c["blocks"]
        st["k16"], st["v16"] = spread(nb, heads, BLOCK, dim), spread(nb, heads, BLOCK, dim)
        st["k"], st["v"] = (torch.zeros((nb, heads, 9 * dim), device="cuda", dtype=torch.uint8) for _ in range(2))
        st["pairs"] = torch.stack([order(nb), order(nb)], 1).contiguous()
        st["back"] = torch.stack([st["pairs"][:, 1], order(nb)], 1).contiguous()
        st["k_out"], st["v_out"] = torch.zeros_like(st["k16"]), torch.zeros_like(st["v16"])
        return st
    lens = torch.tensor(lengths(c), device="cuda", dtype=torch.int32)[order(c["seqs"]).long()]
    wide = (c["max"] + BLOCK - 1) // BLOCK
    nb = c["seqs"] * wide
    st["lens"], st["tables"] = lens, order(nb).view(c["seqs"], wide).contiguous()
    if c["op"] == "evict":
        st["k"], st["v"] = normal(nb, heads, BLOCK, dim), normal(nb, heads, BLOCK, dim)
        # accumulated weight: heavy tails, and tokens that never drew any
        m = torch.exp(2.0 * torch.randn((c["seqs"], c["max"]), generator=g, device="cuda"))
        st["mass"] = torch.where(torch.rand(m.shape, generator=g, device="cuda") < 0.05, 0.0, m)
        # every second sequence was evicted before: its first slots hold scattered positions
        odd = torch.arange(c["seqs"], device="cuda") % 2
        held = torch.minimum(lens, torch.full_like(lens, c["keep"])) * odd
        st["history"] = torch.stack([held, 3 * held], 1).to(torch.int32).contiguous()
        st["positions"] = (3 * torch.arange(c["max"], device="cuda")[None] + torch.randint(0, 3, m.shape, generator=g, device="cuda")).to(torch.int32)
        st["keep"] = torch.full_like(lens, c["keep"])
        for k in ("mass", "positions", "history"):
            st[k + "_out"] = torch.zeros_like(st[k])
        return st
    st["q"] = normal(c["seqs"], heads * c["group"], dim)
    q4 = c["op"] == "decode4" or c["q4"]
    st["k"], st["v"] = (four(nb), four(nb)) if q4 else (normal(nb, heads, BLOCK, dim), normal(nb, heads, BLOCK, dim))
    st["out"] = torch.zeros_like(st["q"])
    if c["op"] == "mass":
        st["mass"] = torch.rand((c["seqs"], wide * BLOCK), generator=g, device="cuda")
        st["mass_out"] = torch.zeros_like(st["mass"])
    return st


# ---- the operators, plain and the library's ----------------------------------------------

DECAY = 0.99


def attend(q, k, v, lens, group, dim):
    """softmax(q k / sqrt(D)) v of [S, HQ, D] queries over [S, H, L, D] keys and values; also the weights."""
    s, hq, _ = q.shape
    q = q.to(k.dtype).view(s, hq // group, group, dim)
    x = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(dim)
    real = (torch.arange(k.shape[2], device=k.device) < lens[:, None])[:, None, None]
    x = x.masked_fill(~real, -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    w = e / e.sum(-1, keepdim=True)
    return torch.matmul(w, v).view(s, hq, dim), w


def of_tables(pool, tables, dim, real=torch.float32):
    """The cached rows of every sequence, [S, H, blocks * 16, D]."""
    t = pool[tables.long()]
    t = values(t, dim, real) if pool.dtype == torch.uint8 else t.to(real)
    return t.transpose(1, 2).flatten(2, 3)


def plain_append(st):
    dim, at = st["case"]["dim"], st["slots"].long()
    block, row = at // BLOCK, at % BLOCK

    def write(pool, new):
        n, s, z = quantise(new)
        h = n.shape[1]
        b = n.to(torch.uint8).view(-1, h, dim // 32, 16, 2)
        words = torch.stack([z.to(torch.float16).view(torch.uint8).view(-1, h, dim // 64, 2),
                             s.to(torch.bfloat16).view(torch.uint8).view(-1, h, dim // 64, 2)], -2).flatten(-2)
        pool[..., :8 * dim].unflatten(-1, (dim // 32, 16, 16))[block, :, :, row] = b[..., 0] | b[..., 1] << 4
        pool[..., 8 * dim:].unflatten(-1, (dim // 64, 16, 4))[block, :, :, row] = words

    def read(pool, out):
        src, dst = st["pairs"].long().unbind(1)
        out[dst] = rounded(values(pool[src], dim), st["kind"])

    write(st["k"], st["k_new"])
    write(st["v"], st["v_new"])
    read(st["k"], st["k_out"])
    read(st["v"], st["v_out"])
    return st["k_out"], st["v_out"]


def plain_convert(st):
    dim = st["case"]["dim"]
    (src, dst), (src2, dst2) = st["pairs"].long().unbind(1), st["back"].long().unbind(1)

    def there_and_back(x, pool, out):
        pool[dst] = pack(*quantise(x[src]))
        out[dst2] = rounded(values(pool[src2], dim), st["kind"])
        return out

    return there_and_back(st["k16"], st["k"], st["k_out"]), there_and_back(st["v16"], st["v"], st["v_out"])


def plain_decode(st):
    c = st["case"]
    out, w = attend(st["q"], of_tables(st["k"], st["tables"], c["dim"]), of_tables(st["v"], st["tables"], c["dim"]), st["lens"], c["group"], c["dim"])
    if c["op"] == "decode4":
        return out.to(st["kind"])
    real = torch.arange(st["mass"].shape[1], device=w.device) < st["lens"][:, None]
    return out.to(st["kind"]), torch.where(real, DECAY * st["mass"] + w.sum((1, 2)), 0.0)


def selection(st, real):
    """Which slots stay, and every slot's original position."""
    c, lens, mass = st["case"], st["lens"][:, None], st["mass"].to(real)
    t = torch.arange(mass.shape[1], device=mass.device)[None]
    held, after = st["history"][:, :1], st["history"][:, 1:]
    where = torch.where(t < held, st["positions"], after + t - held)
    seen = after + lens - held
    key = mass.masked_fill((where < c["sinks"]) | (where >= seen - c["recent"]), math.inf).masked_fill(t >= lens, -math.inf)
    place = torch.sort(key, dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(place).scatter_(1, place, t.expand_as(place))
    stays = (rank < st["keep"][:, None]) & (t < lens)
    return stays, where, t, lens, seen


def plain_evict(st):
    stays, where, t, lens, seen = selection(st, torch.float32)
    left = torch.minimum(st["keep"][:, None], lens)
    seq, hole = (~stays & (t < left)).nonzero(as_tuple=True)
    mover = (stays & (t >= left)).nonzero(as_tuple=True)[1]
    src, dst = st["tables"][seq, mover // BLOCK].long(), st["tables"][seq, hole // BLOCK].long()
    mass, place, history = torch.where(t < left, st["mass"], 0.0), torch.where(t < left, where, 0), torch.cat([left, seen], 1)
    mass[seq, hole], place[seq, hole] = st["mass"][seq, mover], where[seq, mover]
    whole = (st["keep"][:, None] >= lens) & (t < lens)
    mass, place = torch.where(whole, st["mass"], mass), torch.where(whole, st["positions"], place)
    history = torch.where(st["keep"][:, None] >= lens, st["history"], history)
    st["k"][dst, :, hole % BLOCK] = st["k"][src, :, mover % BLOCK]
    st["v"][dst, :, hole % BLOCK] = st["v"][src, :, mover % BLOCK]
    return st["k"], st["v"], mass, place.to(torch.int32), history.to(torch.int32)


def handles(st):
    """What a program keeps from call to call: the pools' descriptors and a workspace."""
    if "pool" not in st:
        import paged_kv_cache_478_b200 as pa

        c = st["case"]
        four = {"f16": pa.PA_Q4_F16, "bf16": pa.PA_Q4_BF16}.get(c["type"])
        nb = st["k"].shape[0]
        q4 = st["k"].dtype == torch.uint8
        st["pa"], st["pool"] = pa, pa.pa_pool_create(nb, BLOCK, c["heads"], c["dim"], four if q4 else st["kind"])
        need = 0
        if c["op"] in ("append", "convert"):
            st["pool16"] = pa.pa_pool_create(nb, BLOCK, c["heads"], c["dim"], st["kind"])
        elif c["op"] == "evict":
            need = pa.pa_evict_workspace_bytes(st["pool"], c["seqs"], st["tables"].shape[1], c["max"])
        else:
            pa.pa_pool_set_query_heads(st["pool"], c["heads"] * c["group"])
            size = pa.pa_decode_mass_workspace_bytes if c["op"] == "mass" else pa.pa_decode_workspace_bytes
            need = size(st["pool"], c["seqs"], st["tables"].shape[1], c["max"])
        st["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return st["pa"], st["pool"]


def own_append(st):
    pa, pool = handles(st)
    pa.pa_reshape_and_cache(pool, st["k_new"], st["v_new"], st["slots"], st["k"], st["v"])
    pa.pa_convert_blocks(pool, st["k"], st["v"], st["pool16"], st["k_out"], st["v_out"], st["pairs"])
    return st["k_out"], st["v_out"]


def own_convert(st):
    pa, pool = handles(st)
    pa.pa_convert_blocks(st["pool16"], st["k16"], st["v16"], pool, st["k"], st["v"], st["pairs"])
    pa.pa_convert_blocks(pool, st["k"], st["v"], st["pool16"], st["k_out"], st["v_out"], st["back"])
    return st["k_out"], st["v_out"]


def own_decode(st):
    pa, pool = handles(st)
    c = st["case"]
    if c["op"] == "decode4":
        pa.pa_decode_attention(pool, st["q"], st["k"], st["v"], st["tables"], st["lens"], 1 / math.sqrt(c["dim"]), st["out"], st["workspace"],
                               max_context_len=c["max"])
        return st["out"]
    pa.pa_decode_attention_mass(pool, st["q"], st["k"], st["v"], st["tables"], st["lens"], 1 / math.sqrt(c["dim"]), st["out"], st["mass"], st["mass_out"],
                                st["workspace"], decay=DECAY, max_context_len=c["max"])
    return st["out"], st["mass_out"]


def own_evict(st):
    pa, pool = handles(st)
    c = st["case"]
    track = {k: st[k] for k in ("mass", "positions", "history")}
    after = {k: st[k + "_out"] for k in ("mass", "positions", "history")}
    pa.pa_evict_tokens(pool, st["k"], st["v"], st["tables"], st["lens"], st["keep"], c["sinks"], c["recent"], track, after, st["workspace"],
                       max_context_len=c["max"])
    return st["k"], st["v"], after["mass"], after["positions"], after["history"]


PLAIN = {"append": plain_append, "convert": plain_convert, "decode4": plain_decode, "mass": plain_decode, "evict": plain_evict}
OWN = {"append": own_append, "convert": own_convert, "decode4": own_decode, "mass": own_decode, "evict": own_evict}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ---- what a pass cannot do without ---------------------------------------------------------

def work(case):
    c = case
    h, d = c["heads"], c["dim"]
    wide, narrow = h * d * (4 if c["type"] == "f32" else 2), h * d * 9 // 16  # bytes of one K or V row of a token
    if c["op"] == "append":
        new = c["seqs"] * c["new"]
        kept = c["seqs"] * ((c["start"] % BLOCK + c["new"] + BLOCK - 1) // BLOCK) * BLOCK
        # new tokens in, their 4-bit rows out; the touched blocks' other rows in, all of their rows out in 16 bits
        return {"bytes": 2 * (new * (wide + narrow) + (kept - new) * narrow + kept * wide) + 4 * new, "flops": 8 * (new + kept) * h * d}
    if c["op"] == "convert":
        return {"bytes": 2 * c["blocks"] * BLOCK * (2 * wide + narrow), "flops": 16 * c["blocks"] * BLOCK * h * d}
    lens = lengths(c)
    total = sum(lens)
    blocks = sum((n + BLOCK - 1) // BLOCK for n in lens)
    if c["op"] == "evict":
        # tokens past `keep` that stay, if weight falls evenly over the slots: they move, and the tracks go in and out
        moved = sum(min(c["recent"] + (c["keep"] - c["recent"]) * max(0, n - c["keep"] - c["recent"]) // max(1, n - c["recent"]), n - c["keep"], c["keep"])
                    for n in lens if n > c["keep"])
        return {"bytes": 4 * moved * wide + 16 * total + 8 * moved, "flops": 8 * total}
    hq = h * c["group"]
    four = c["op"] == "decode4" or c["q4"]
    b = 2 * total * (narrow if four else wide) + 2 * c["seqs"] * hq * d * (4 if c["type"] == "f32" else 2) + 4 * blocks
    if c["op"] == "mass":
        b += 8 * total
    return {"bytes": b, "flops": 4 * total * hq * d}


# ---- the definition in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    c, st = dict(case), prepare(case, seed)
    dim, f = c["dim"], torch.float64
    if c["op"] in ("append", "convert"):
        def held(x):
            # what the cache stands for once x [..., D] went in
            g = x.double().reshape(*x.shape[:-1], dim // 64, 64)
            hi, lo = g.max(-1, keepdim=True).values, g.min(-1, keepdim=True).values
            fifteen, most = torch.tensor([15.0, 2000.0], dtype=f, device=x.device)
            step = torch.maximum((hi - lo) / fifteen.expand_as(hi), torch.maximum(hi.abs(), lo.abs()) / most.expand_as(hi)).bfloat16().double()
            zero = torch.where(step > 0, -(lo / step).round(), 0.0)
            n = torch.where(step > 0, (g / step).round() + zero, 0.0).clip(0, 15)
            return (step * (n - zero)).reshape(x.shape)

        if c["op"] == "convert":
            def back(x):
                y = torch.zeros_like(x, dtype=f)
                y[st["back"][:, 1].long()] = held(x[st["pairs"][:, 0].long()])
                return y

            return back(st["k16"]), back(st["v16"])

        def after(pool, new):
            out = torch.empty(pool.shape[0], c["heads"], BLOCK, dim, dtype=f, device=pool.device)
            src, dst = st["pairs"][:, 0].long(), st["pairs"][:, 1].long()
            now = old_values(pool, dim)
            now[st["slots"].long() // BLOCK, :, st["slots"].long() % BLOCK] = held(new)
            out[dst] = now[src]
            return out

        return after(st["k"], st["k_new"]), after(st["v"], st["v_new"])
    lens = st["lens"].tolist()
    if c["op"] == "evict":
        k, v = st["k"].double(), st["v"].double()
        mass, place, history = torch.zeros_like(st["mass"], dtype=f), torch.zeros_like(st["positions"]), st["history"].clone()
        for s, n in enumerate(lens):
            keep = c["keep"]
            if n <= keep:
                mass[s, :n], place[s, :n] = st["mass"][s, :n].double(), st["positions"][s, :n]
                continue
            held, after_ = st["history"][s].tolist()
            slots = torch.arange(n, device="cuda")
            where = torch.cat([st["positions"][s, :held], torch.arange(after_, after_ + n - held, device="cuda", dtype=torch.int32)])
            seen = after_ + n - held
            safe = (where < c["sinks"]) | (where >= seen - c["recent"])
            w = st["mass"][s, :n].double()
            first = slots[safe]
            rest = slots[~safe]
            rest = rest[torch.argsort(-w[rest], stable=True)]
            stays = torch.cat([first, rest])[:keep].sort().values
            mask = torch.zeros(n, dtype=torch.bool, device="cuda")
            mask[stays] = True
            hole, mover = slots[:keep][~mask[:keep]], slots[keep:][mask[keep:]]
            origin = slots[:keep].clone()
            origin[hole] = mover
            mass[s, :keep], place[s, :keep] = w[origin], where[origin]
            history[s, 0], history[s, 1] = keep, seen
            a, b = st["tables"][s, mover // BLOCK].long(), st["tables"][s, hole // BLOCK].long()
            k[b, :, hole % BLOCK], v[b, :, hole % BLOCK] = k[a, :, mover % BLOCK], v[a, :, mover % BLOCK]
        return k, v, mass, place, history
    out = torch.zeros(st["q"].shape, dtype=f, device="cuda")
    mass = torch.zeros_like(st["mass"], dtype=f) if c["op"] == "mass" else None
    for s, n in enumerate(lens):
        t = st["tables"][s, :(n + BLOCK - 1) // BLOCK].long()
        k, v = ((old_values(p[t], dim) if p.dtype == torch.uint8 else p[t].double()).permute(1, 0, 2, 3).reshape(c["heads"], -1, dim)[:, :n] for p in (st["k"], st["v"]))
        w = torch.softmax(torch.einsum("hgd,htd->hgt", st["q"][s].double().view(c["heads"], c["group"], dim), k) * dim ** -0.5, -1)
        out[s] = torch.einsum("hgt,htd->hgd", w, v).reshape(-1, dim)
        if mass is not None:
            mass[s, :n] = DECAY * st["mass"][s, :n].double() + w.sum((0, 1))
    return out if mass is None else (out, mass)


def old_values(tiles, dim):
    """A 4-bit pool's tiles [blocks, H, 9 D] as 64-bit values [blocks, H, 16, D], dimension by dimension."""
    nb, h, _ = tiles.shape
    d = torch.arange(dim, device=tiles.device)
    t = torch.arange(BLOCK, device=tiles.device)[:, None]
    byte = tiles[:, :, (d // 32) * 256 + t * 16 + d % 32 // 2].long()
    n = torch.where(d % 2 == 1, byte >> 4, byte & 15).double()
    word = 8 * dim + (d // 64) * 64 + t * 4
    zero = (tiles[:, :, word].int() | tiles[:, :, word + 1].int() << 8).to(torch.int16).view(torch.float16).double()
    step = (tiles[:, :, word + 2].int() | tiles[:, :, word + 3].int() << 8).to(torch.int16).view(torch.bfloat16).double()
    return step * (n - zero)
