"""Workloads of the block-scaled 8-bit KV cache path: rotary positions, append,
attention, accumulated attention weight and eviction.

The cache holds int8 codes [num_blocks, kv heads, block tokens, head dim] for K
and V and one fp32 scale per (block, kv head); a block table maps the blocks of
each sequence.  Every case is one call of one operator (append and evict read
the stored values back, which is what they leave behind).
"""
import math
import random

import torch

own = False

# head dims, block sizes and head counts that the drawn cases mix
_DIMS = (64, 128, 256)
_BLOCKS = (16, 32, 64, 128, 256)
_MOST_BYTES = 6.8e8   # no drawn case moves more than the largest listed one
_MOST_FLOPS = 3.0e11  # or computes more


def listed():
    return [
        # one decode step of 64 sequences: every head of q and k, far positions
        dict(name="rope step", op="rope", tokens=64, hq=32, hkv=8, dim=128, rot=128,
             interleaved=False, scaling="none", dtype="bf16", fused=False, inverse=False,
             max_pos=131072),
        # a long prompt whose q and k are slices of one projection; a quarter of
        # the head is rotated, pairs lie next to each other, context extended
        dict(name="rope prompt", op="rope", tokens=16384, hq=32, hkv=4, dim=256, rot=64,
             interleaved=True, scaling="yarn", dtype="bf16", fused=True, inverse=False,
             max_pos=262144),
        # one new token in each of 64 sequences, in the middle of their blocks
        dict(name="append step", op="append", batch=64, t_new=1, hkv=8, dim=128, block=16,
             dtype="bf16", rope=True, interleaved=False, lo=1000, hi=8000),
        # 4096-token prompts of 8 sequences, the size of the quantize benchmark
        dict(name="append prompt", op="append", batch=8, t_new=4096, hkv=8, dim=256, block=64,
             dtype="bf16", rope=True, interleaved=False, lo=0, hi=0),
        # a short chat: one sequence, one token, full precision
        dict(name="decode short", op="attn", batch=1, nq=1, hq=32, hkv=8, dim=128, block=16,
             dtype="f32", lo=777, hi=777),
        # the long-context decode benchmark's shape
        dict(name="decode long", op="attn", batch=1, nq=1, hq=32, hkv=4, dim=256, block=256,
             dtype="bf16", lo=131072, hi=131072),
        # a full serving batch of ragged contexts over small pages
        dict(name="decode batch", op="attn", batch=32, nq=1, hq=32, hkv=8, dim=128, block=32,
             dtype="bf16", lo=2048, hi=16384),
        # chunks of prompts on top of what is cached already
        dict(name="prefill chunk", op="attn", batch=4, nq=1024, hq=32, hkv=8, dim=128, block=64,
             dtype="bf16", lo=3000, hi=8192),
        # the decode step's weights, added up for eviction
        dict(name="mass step", op="mass", batch=32, nq=1, hq=32, hkv=8, dim=128, block=32,
             dtype="bf16", lo=2048, hi=16384),
        # the last tokens of each prompt vote on the prompt's tokens
        dict(name="mass window", op="mass", batch=4, nq=32, hq=32, hkv=8, dim=128, block=16,
             dtype="bf16", lo=4000, hi=8192),
        # a batch that outgrew its budget: a quarter of the tokens stays
        dict(name="evict batch", op="evict", batch=16, hkv=8, dim=128, block=32, lo=12000,
             hi=16384, keep=4096, recent=512, sinks=4),
        # one sequence just past its budget
        dict(name="evict one", op="evict", batch=1, hkv=4, dim=256, block=64, lo=2113, hi=2113,
             keep=1024, recent=128, sinks=4),
    ]


def draw(rng):
    def logu(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(("rope", "append", "attn", "attn", "mass", "evict"))
        dim = rng.choice(_DIMS)
        hkv = rng.choice((1, 2, 3, 4, 8))
        group = rng.choice((1, 2, 3, 4, 5, 8, 16))
        block = rng.choice(_BLOCKS)
        dtype = rng.choice(("bf16", "bf16", "f32"))
        lo = logu(1, 20000)
        hi = lo + logu(1, 20000)
        if op == "rope":
            c = dict(op=op, tokens=logu(1, 16384), hq=hkv * group, hkv=hkv, dim=dim,
                     rot=rng.choice((dim, dim // 2, dim // 4)), interleaved=rng.random() < 0.5,
                     scaling=rng.choice(("none", "linear", "ntk", "yarn")), dtype=dtype,
                     fused=rng.random() < 0.5, inverse=rng.random() < 0.3,
                     max_pos=logu(100, 1000000))
        elif op == "append":
            c = dict(op=op, batch=logu(1, 64), t_new=logu(1, 4096), hkv=hkv, dim=dim, block=block,
                     dtype=dtype, rope=rng.random() < 0.5, interleaved=rng.random() < 0.5,
                     lo=lo - 1, hi=hi)
        elif op == "evict":
            keep = logu(8, 8192)
            c = dict(op=op, batch=logu(1, 32), hkv=hkv, dim=dim, block=block, lo=lo, hi=hi,
                     keep=keep, recent=rng.randint(0, keep // 2), sinks=rng.randint(0, keep // 4))
        else:
            nq = rng.choice((1, 1, rng.randint(2, 8), logu(9, 1024)))
            c = dict(op=op, batch=logu(1, 64), nq=nq, hq=hkv * group, hkv=hkv, dim=dim,
                     block=block, dtype=dtype, lo=lo, hi=hi)
        w = work(c)
        if w["bytes"] <= _MOST_BYTES and w["flops"] <= _MOST_FLOPS and _scratch(c) < 8e9:
            return c


# ------------------------------------------------------------------ sizes
def _scratch(c):
    """Bytes of the scores that the plain form holds at once."""
    if c["op"] not in ("attn", "mass"):
        return 0
    return 4.0 * c["batch"] * c["nq"] * c["hq"] * c["hi"]


def _lens(c):
    """Tokens cached per sequence (before an append), the same for every seed."""
    r = random.Random("%d/%d/%d" % (c["batch"], c["lo"], c["hi"]))
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["batch"])]


def _nq(c):
    """Query tokens per sequence: ragged where there are many."""
    r = random.Random("%d:%d" % (c["batch"], c["nq"]))
    return [c["nq"] if c["nq"] < 4 else r.randint((c["nq"] + 1) // 2, c["nq"])
            for _ in range(c["batch"])]


def _t_new(c):
    r = random.Random("%d;%d" % (c["batch"], c["t_new"]))
    return [c["t_new"] if c["t_new"] < 4 else r.randint((c["t_new"] + 1) // 2, c["t_new"])
            for _ in range(c["batch"])]


def _size(dtype):
    return 2 if dtype == "bf16" else 4


def _torch(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def work(c):
    if c["op"] == "rope":
        n = c["tokens"] * (c["hq"] + c["hkv"])
        return {"bytes": float(2 * n * c["dim"] * _size(c["dtype"]) + 4 * c["tokens"]),
                "flops": float(3 * n * c["rot"])}
    lens = _lens(c)
    if c["op"] == "append":
        new = _t_new(c)
        rows = 2 * c["hkv"] * sum(new)
        old = 2 * c["hkv"] * sum(n % c["block"] for n in lens)
        # read the new rows, write their codes; the stored rows come back as bf16
        return {"bytes": float(rows * c["dim"] * (_size(c["dtype"]) + 1)
                               + (rows + old) * c["dim"] * 3), "flops": float(4 * rows * c["dim"])}
    if c["op"] == "evict":
        kept = sum(min(n, c["keep"]) for n in lens)
        # weights in, kept codes in and out, kept values back as bf16
        return {"bytes": float(c["hkv"] * (4 * sum(lens) + kept * (2 * c["dim"] * 5 + 8))),
                "flops": float(c["hkv"] * kept * c["dim"] * 4)}
    pairs = sum(nq * n - nq * (nq - 1) // 2 if n >= nq else n * (n + 1) // 2
                for nq, n in zip(_nq(c), lens))
    q = sum(_nq(c)) * c["hq"] * c["dim"] * _size(c["dtype"])
    if c["op"] == "mass":
        return {"bytes": float(c["hkv"] * sum(lens) * (c["dim"] + 8) + q),
                "flops": float(2 * pairs * c["hq"] * c["dim"])}
    return {"bytes": float(c["hkv"] * sum(lens) * 2 * c["dim"] + 2 * q),
            "flops": float(4 * pairs * c["hq"] * c["dim"])}


# ------------------------------------------------------------------ inputs
def _values(g, shape, dtype):
    """Gaussian head vectors with the few large channels that K and V have."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    n = max(1, round(shape[-1] / 100))
    ch = torch.randperm(shape[-1], generator=g, device="cuda")[:n]
    x[..., ch] *= 16.0
    return x.to(_torch(dtype))


def _cache(g, c, blocks_per_seq, spare=0):
    """Codes and scales of filled blocks, and a shuffled block table; `spare`
    further blocks per sequence get a table of their own."""
    cols = max(blocks_per_seq + [1])
    total = sum(blocks_per_seq) + spare * c["batch"]
    nb = max(total, 1)
    shape = (nb, c["hkv"], c["block"], c["dim"])
    s = {}
    for n in ("k", "v"):
        x = torch.empty(shape, dtype=torch.int8, device="cuda")
        sc = torch.empty(shape[:2], dtype=torch.float32, device="cuda")
        step = max(1, (1 << 26) // (shape[1] * shape[2] * shape[3]))
        for i in range(0, nb, step):
            w = _values(g, (min(step, nb - i),) + shape[1:], "f32")
            a = w.abs().amax((2, 3)) / 127.0
            x[i:i + step] = torch.round(w / a[:, :, None, None]).to(torch.int8)
            sc[i:i + step] = a
        s[n + "_codes"], s[n + "_scales"] = x, sc
    perm = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["batch"], cols), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(blocks_per_seq):
        table[b, :n] = perm[at:at + n]
        at += n
    s["table"] = table
    if spare:
        s["table2"] = perm[at:at + spare * c["batch"]].view(c["batch"], spare).contiguous()
    return s


def _inv_freq(rot, scaling):
    """Radians per position of each pair, and the factor on the rotated values."""
    i = torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot
    base, factor, trained = 10000.0, 8.0, 32768.0
    if scaling == "ntk":
        base = base * factor ** (rot / max(rot - 2, 1))
    f = base ** -i
    if scaling == "linear":
        f = f / factor
    if scaling != "yarn":
        return f, 1.0
    # pairs that turn often within the trained length keep their frequency,
    # those that turn less than once are stretched, a ramp lies between
    turns = trained * f / (2 * math.pi)
    ramp = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
    return f / factor * (1 - ramp) + f * ramp, 0.1 * math.log(factor) + 1.0


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "rope":
        n, dt = c["tokens"], _torch(c["dtype"])
        heads = c["hq"] + c["hkv"] * (2 if c["fused"] else 1)
        x = torch.randn((n, heads, c["dim"]), generator=g, device="cuda").to(dt)
        if c["fused"]:  # one projection: q, k and v of a token lie next to each other
            s["q"], s["k"] = x[:, :c["hq"]], x[:, c["hq"]:c["hq"] + c["hkv"]]
        else:
            s["q"], s["k"] = x[:, :c["hq"]].contiguous(), x[:, c["hq"]:].contiguous()
        s["pos"] = torch.randint(0, c["max_pos"], (n,), generator=g, device="cuda",
                                 dtype=torch.int32)
        s["inv_freq"], s["factor"] = _inv_freq(c["rot"], c["scaling"])
        return s
    lens, blk = _lens(c), c["block"]
    if c["op"] == "append":
        new = _t_new(c)
        s |= _cache(g, c, [(n + m + blk - 1) // blk for n, m in zip(lens, new)])
        shape = (c["batch"], c["t_new"], c["hkv"], c["dim"])
        s["k"], s["v"] = _values(g, shape, c["dtype"]), _values(g, shape, c["dtype"])
        s["start"], s["new"] = _ints(lens), _ints(new)
        s["first"] = _ints([n // blk * blk for n in lens])
        s["ends"] = _ints([n + m for n, m in zip(lens, new)])
        s["span"] = max(n % blk + m for n, m in zip(lens, new))
        s["inv_freq"], s["factor"] = _inv_freq(c["dim"], "none")
    elif c["op"] == "evict":
        spare = (c["keep"] + blk - 1) // blk
        s |= _cache(g, c, [(n + blk - 1) // blk for n in lens], spare)
        m = torch.randn((c["batch"], c["hkv"], max(lens)), generator=g, device="cuda")
        m = torch.exp(2.0 * m)  # a few tokens hold most of the weight
        m[torch.rand(m.shape, generator=g, device="cuda") < 0.1] = 0.0
        s["mass"], s["lens"], s["max_len"] = m, _ints(lens), max(lens)
    else:
        nq = _nq(c)
        s |= _cache(g, c, [(n + blk - 1) // blk for n in lens])
        s["q"] = torch.randn((sum(nq), c["hq"], c["dim"]), generator=g,
                             device="cuda").to(_torch(c["dtype"]))
        s["lens"], s["max_len"], s["max_q"] = _ints(lens), max(lens), max(nq)
        at = [0]
        for n in nq:
            at.append(at[-1] + n)
        s["cu_q"] = _ints(at) if c["nq"] > 1 else None
        # where query i of the flat list sits in a padded [batch, max_q] layout
        s["slot"] = torch.tensor([b * max(nq) + i for b, n in enumerate(nq) for i in range(n)],
                                 device="cuda")
        s["nq"] = _ints(nq)
        s["scale"] = c["dim"] ** -0.5
        if c["op"] == "mass":
            s["mass"] = torch.rand((c["batch"], c["hkv"], max(lens)), generator=g, device="cuda")
            s["lse"] = _lse(s)
    if own:  # the handle over these tensors that a serving program keeps
        from hadamard_rotated_bit_fwht_b200 import kvq
        s["cache"] = kvq.B8Cache.wrap(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"],
                                      s["table"])
        if c["op"] == "evict":
            s["cache2"] = s["cache"].with_block_table(s["table2"])
    return s


# ------------------------------------------------------------------ plain forms
def _rotate(x, pos, inv_freq, factor, interleaved, inverse):
    """fp32 rotation of the leading 2 * len(inv_freq) dims; x [..., heads, D], pos [...]."""
    a = pos.double()[..., None, None] * inv_freq * (-1.0 if inverse else 1.0)
    cos, sin = (a.cos() * factor).float(), (a.sin() * factor).float()
    r = 2 * inv_freq.numel()
    x = x.float()
    u, v = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    y = (u * cos - v * sin, v * cos + u * sin)
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat((y, x[..., r:]), -1)


def _paged(s, which, table, tokens):
    """fp32 values [batch, kv heads, tokens, D] of the leading tokens."""
    t = table.long().clamp_min(0)
    x = s[which + "_codes"][t].float() * s[which + "_scales"][t][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)[:, :, :tokens]


def _scores(s):
    """Scores [batch, kv heads, group, max_q, tokens] with -inf where a query
    does not attend, in fp32."""
    c = s["case"]
    nb, tq = c["batch"], s["max_q"]
    q = torch.zeros((nb * tq, c["hq"], c["dim"]), device="cuda")
    q[s["slot"]] = s["q"].float()
    q = q.view(nb, tq, c["hkv"], -1, c["dim"]).permute(0, 2, 3, 1, 4)
    k = _paged(s, "k", s["table"], s["max_len"])
    x = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)) * s["scale"]
    x = x.view(q.shape[:4] + (s["max_len"],))
    lim = (s["lens"] - s["nq"])[:, None] + 1 + torch.arange(tq, device="cuda")
    t = torch.arange(s["max_len"], device="cuda")
    return x.masked_fill_((t >= lim[..., None])[:, None, None], -math.inf)


def _flat(s, x):
    """[batch, kv heads, group, max_q, ...] -> one row per query token."""
    x = x.flatten(1, 2).transpose(1, 2)
    return x.flatten(0, 1)[s["slot"]]


def _lse(s):
    return _flat(s, _scores(s).logsumexp(-1)).contiguous()


def _plain_attn(s):
    x = _scores(s)
    m = x.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp_(x.sub_(m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), _paged(s, "v", s["table"], s["max_len"]))
    o = torch.where(total > 0, o.view(p.shape[:4] + (-1,)) / total, 0.0)
    lse = torch.where(total > 0, m + total.log(), -math.inf)[..., 0]
    return {"out": _flat(s, o).to(s["q"].dtype), "lse": _flat(s, lse)}


def _plain_mass(s):
    c = s["case"]
    lse = torch.full((c["batch"] * s["max_q"], c["hq"]), math.inf, device="cuda")
    lse[s["slot"]] = torch.where(torch.isinf(s["lse"]), math.inf, s["lse"])
    lse = lse.view(c["batch"], s["max_q"], c["hkv"], -1).permute(0, 2, 3, 1)
    s["mass"] += torch.exp_(_scores(s).sub_(lse[..., None])).sum((2, 3))
    return s["mass"]


def _quantise(x, old_codes, old_scale, fresh):
    """Blocks of fp32 rows [n, kv heads, block, D] (zero where a block has no new
    row) into codes; blocks that are not fresh keep their older rows."""
    amax = x.abs().amax((2, 3))
    amax = torch.where(amax < 2.0 ** -100, 0.0, amax)
    need = amax / torch.full_like(amax, 127.0)
    old = torch.where(fresh[:, None], 0.0, old_scale)
    scale = torch.maximum(need, old)
    ones = torch.ones_like(scale)
    inv = torch.where(scale > 0, ones / scale, 0.0)
    ratio = torch.where(scale > old, torch.where(scale > 0, old / scale, 0.0), ones)
    codes = torch.round(x * inv[..., None, None]).clamp(-127, 127)
    kept = torch.round(old_codes.float() * ratio[..., None, None])
    return codes, kept, scale


def _plain_append(s):
    c = s["case"]
    nb, blk = c["batch"], c["block"]
    cols = s["table"].shape[1]
    i = torch.arange(c["t_new"], device="cuda")
    pos = s["start"][:, None] + i
    live = i < s["new"][:, None]
    # the new rows at their places in the sequences' blocks
    b, col = torch.nonzero(torch.zeros((nb, cols), device="cuda", dtype=torch.bool).index_put_(
        (torch.arange(nb, device="cuda")[:, None].expand_as(pos)[live], (pos // blk)[live].long()),
        torch.tensor(True, device="cuda")), as_tuple=True)
    page = s["table"][b, col].long()
    where = torch.full((nb, cols), -1, device="cuda", dtype=torch.long)
    where[b, col] = torch.arange(b.numel(), device="cuda")
    start = s["start"].long()[b]
    fresh = start <= col * blk
    row = torch.arange(blk, device="cuda")
    old = (col[:, None] * blk + row < start[:, None])[:, None, :, None]
    done = []
    for n in ("k", "v"):
        x = s[n].float()
        if n == "k" and c["rope"]:
            x = _rotate(x, pos, s["inv_freq"], s["factor"], c["interleaved"], False)
        into = torch.zeros((b.numel(), c["hkv"], blk, c["dim"]), device="cuda")
        bi = torch.arange(nb, device="cuda")[:, None].expand_as(pos)[live]
        into[where[bi, (pos // blk)[live].long()], :, (pos % blk)[live].long()] = x[live]
        new = ((col[:, None] * blk + row >= start[:, None])
               & (col[:, None] * blk + row < s["ends"].long()[b][:, None]))[:, None, :, None]
        codes, kept, scale = _quantise(into, s[n + "_codes"][page], s[n + "_scales"][page], fresh)
        codes = torch.where(new, codes, torch.where(old, kept, s[n + "_codes"][page].float()))
        s[n + "_codes"][page] = codes.to(torch.int8)
        s[n + "_scales"][page] = scale
        done.append(scale)
    return _read(s, s["table"], s["first"], s["ends"], s["span"]) | {"scales": s["k_scales"],
                                                                     "v_scales": s["v_scales"]}


def _read(s, table, first, ends, span):
    """Stored values of tokens first[b] .. first[b] + span - 1 as bf16, zero
    from ends[b] on: [batch, span, kv heads, D]."""
    blk = s["case"]["block"]
    t = first.long()[:, None] + torch.arange(span, device="cuda")
    live = t < ends[:, None]
    col = (t // blk).clamp_max(table.shape[1] - 1)
    page = table.long().gather(1, col).clamp_min(0)
    got = {}
    for n in ("k", "v"):
        x = s[n + "_codes"][page, :, t % blk].float() * s[n + "_scales"][page][..., None]
        got[n] = torch.where(live[..., None, None], x, 0.0).to(torch.bfloat16)
    return got


def _plain_evict(s):
    c = s["case"]
    n, keep, blk = s["max_len"], c["keep"], c["block"]
    t = torch.arange(n, device="cuda")
    lens = s["lens"].long()
    m = torch.where((t < c["sinks"]) | (t >= lens[:, None] - c["recent"]), math.inf, 1.0)
    m = torch.where(torch.isinf(m)[:, None], math.inf, s["mass"])
    m = torch.where((t < lens[:, None])[:, None], m, -math.inf)
    order = torch.sort(m, dim=-1, descending=True, stable=True).indices[..., :keep]
    new = lens.clamp_max(keep)
    i = torch.arange(keep, device="cuda")
    if n < keep:
        order = torch.nn.functional.pad(order, (0, keep - n), value=n)
    order = torch.where(i < new[:, None, None], order, n + 1).sort(-1).values
    live = (i < new[:, None])[:, None].expand_as(order)
    at = torch.where(live, order, 0)
    mass = torch.where(live, s["mass"].gather(-1, at.clamp_max(n - 1)), 0.0)
    # the kept rows, block by block
    page = s["table"].long().gather(1, (at // blk).flatten(1)).view(at.shape)
    h = torch.arange(c["hkv"], device="cuda")[:, None]
    pad = -keep % blk
    to = s["table2"].long()
    first = (torch.arange(to.shape[1], device="cuda") * blk < new[:, None]).flatten()
    to = to.flatten()[first]
    for w in ("k", "v"):
        x = s[w + "_codes"][page, h, at % blk].float() * s[w + "_scales"][page, h][..., None]
        x = torch.where(live[..., None], x, 0.0)
        x = torch.nn.functional.pad(x, (0, 0, 0, pad))
        x = x.unflatten(2, (-1, blk)).transpose(1, 2).flatten(0, 1)[first]
        codes, _, scale = _quantise(x, x[..., :1, :1], x[..., 0, 0],
                                    torch.ones_like(to, dtype=torch.bool))
        rows = (torch.nn.functional.pad(live, (0, pad)).unflatten(2, (-1, blk)).transpose(1, 2)
                .flatten(0, 1)[first])
        codes = torch.where(rows[..., None], codes, s[w + "_codes"][to].float())
        s[w + "_codes"][to] = codes.to(torch.int8)
        s[w + "_scales"][to] = scale
    zero = torch.zeros_like(s["lens"])
    return _read(s, s["table2"], zero, new, keep) | {
        "mass": mass, "lens": new.to(torch.int32),
        "kept": torch.where(live, order, -1).to(torch.int32)}


def run(state):
    s, c = state, state["case"]
    if not own:
        if c["op"] == "rope":
            return [_rotate(x, s["pos"], s["inv_freq"], s["factor"], c["interleaved"],
                            c["inverse"]).to(x.dtype) for x in (s["q"], s["k"])]
        return {"append": _plain_append, "attn": _plain_attn, "mass": _plain_mass,
                "evict": _plain_evict}[c["op"]](s)
    from hadamard_rotated_bit_fwht_b200 import kvq
    if c["op"] == "rope":
        return list(kvq.rope(s["q"], s["k"], s["pos"],
                             kvq.Rope(s["inv_freq"], c["interleaved"], s["factor"]),
                             inverse=c["inverse"]))
    if c["op"] == "append":
        rope = kvq.Rope(s["inv_freq"], c["interleaved"], s["factor"]) if c["rope"] else None
        kvq.b8_append(s["cache"], s["k"], s["v"], s["start"], new_lens=s["new"], rope=rope)
        k, v = kvq.b8_gather(s["cache"], s["first"], s["ends"], s["span"], torch.bfloat16)
        return {"k": k, "v": v, "scales": s["k_scales"], "v_scales": s["v_scales"]}
    if c["op"] == "attn":
        out, lse = kvq.b8_attn(s["cache"], s["q"], s["lens"], s["max_len"], s["scale"],
                               cu_q=s["cu_q"], max_q=s["max_q"], return_lse=True)
        return {"out": out, "lse": lse}
    if c["op"] == "mass":
        kvq.b8_attn_mass(s["cache"], s["q"], s["lse"], s["lens"], s["max_len"], s["scale"],
                         s["mass"], cu_q=s["cu_q"], max_q=s["max_q"])
        return s["mass"]
    lens, kept, mass = kvq.b8_evict(s["cache"], s["cache2"], s["mass"], s["lens"], s["max_len"],
                                    c["keep"], recent=c["recent"], sinks=c["sinks"])
    k, v = kvq.b8_gather(s["cache2"], torch.zeros_like(lens), lens, c["keep"], torch.bfloat16)
    return {"k": k, "v": v, "mass": mass, "lens": lens, "kept": kept}


# ------------------------------------------------------------------ 64 bits
def _rows64(s, which, table_row, n):
    """fp64 values [kv heads, n, D] of one sequence, block by block in order."""
    blocks = (n + s["case"]["block"] - 1) // s["case"]["block"]
    ids = table_row[:blocks].long()
    x = s[which + "_codes"].index_select(0, ids).double()
    x *= s[which + "_scales"].index_select(0, ids).double().reshape(blocks, -1, 1, 1)
    return torch.cat(list(x), dim=1)[:, :n] if blocks else x.new_zeros(
        (x.shape[1], 0, x.shape[3]))


def _turn64(x, pos, inv_freq, factor, interleaved, sign):
    """Rotation as a complex product, fp64: x [heads, tokens, D], pos [tokens]."""
    r = 2 * inv_freq.numel()
    w = torch.polar(torch.full((pos.numel(), r // 2), factor, dtype=torch.float64, device="cuda"),
                    sign * torch.outer(pos.double(), inv_freq))
    y = x.double().clone()
    if interleaved:
        z = torch.view_as_complex(y[..., :r].reshape(y.shape[:-1] + (r // 2, 2)).contiguous())
        y[..., :r] = torch.view_as_real(z * w).reshape(y.shape[:-1] + (r,))
    else:
        z = torch.complex(y[..., :r // 2].contiguous(), y[..., r // 2:r].contiguous()) * w
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    return y


def _block64(old, old_scale, x):
    """One block of one sequence: rows already there (codes [h, m, D] at
    old_scale [h]) and new fp64 rows [h, n, D] -> codes, scale."""
    need = x.abs().amax((1, 2)) / 127.0
    need = torch.where(need * 127.0 < 2.0 ** -100, 0.0, need)
    scale = torch.maximum(need, old_scale)
    inv = torch.where(scale > 0, 1.0 / scale, 0.0)[:, None, None]
    if old.shape[1]:
        old = torch.where((scale > old_scale)[:, None, None],
                          torch.round(old * old_scale[:, None, None] * inv), old)
    return torch.cat((old, torch.round(x * inv).clamp(-127, 127)), 1), scale


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "rope":
        sign = -1.0 if c["inverse"] else 1.0
        return [_turn64(x.transpose(0, 1), s["pos"], s["inv_freq"], s["factor"], c["interleaved"],
                        sign).transpose(0, 1) for x in (s["q"], s["k"])]
    lens, blk = s["lens"].tolist() if "lens" in s else s["start"].tolist(), c["block"]
    if c["op"] == "append":
        new, out = s["new"].tolist(), {}
        if sum((m + blk - 1) // blk + 1 for m in new) > 8000:
            return None
        for w in ("k", "v"):
            scales = s[w + "_scales"].double()
            got = torch.zeros((c["batch"], s["span"], c["hkv"], c["dim"]), dtype=torch.float64,
                              device="cuda")
            for b in range(c["batch"]):
                x = s[w][b, :new[b]].transpose(0, 1).double()
                if w == "k" and c["rope"]:
                    x = _turn64(x, lens[b] + torch.arange(new[b], device="cuda"), s["inv_freq"],
                                s["factor"], c["interleaved"], 1.0)
                t, at, end = lens[b], 0, lens[b] + new[b]
                while t < end:
                    page, o = int(s["table"][b, t // blk]), t % blk
                    n = min(end - t, blk - o)
                    was = s[w + "_scales"][page].double() * (1.0 if o else 0.0)
                    codes, scale = _block64(s[w + "_codes"][page, :, :o].double(), was,
                                            x[:, t - lens[b]:t - lens[b] + n])
                    scales[page] = scale
                    got[b, at:at + o + n] = (codes * scale[:, None, None]).transpose(0, 1)
                    t, at = t + n, at + o + n
            out[w] = got
            out["scales" if w == "k" else "v_scales"] = scales
        return out
    if c["op"] == "evict":
        if c["batch"] * c["hkv"] * ((c["keep"] + blk - 1) // blk) > 20000:
            return None
        out = {w: torch.zeros((c["batch"], c["keep"], c["hkv"], c["dim"]), dtype=torch.float64,
                              device="cuda") for w in ("k", "v")}
        out["mass"] = torch.zeros((c["batch"], c["hkv"], c["keep"]), dtype=torch.float64,
                                  device="cuda")
        out["kept"] = torch.full((c["batch"], c["hkv"], c["keep"]), -1, dtype=torch.int32,
                                 device="cuda")
        out["lens"] = _ints([min(n, c["keep"]) for n in lens])
        mass = s["mass"].cpu()
        for b, n in enumerate(lens):
            m = min(n, c["keep"])
            first = min(c["sinks"], m) if n > c["keep"] else m
            tail = min(c["recent"], m - first)
            k64, v64 = _rows64(s, "k", s["table"][b], n), _rows64(s, "v", s["table"][b], n)
            for h in range(c["hkv"]):
                w = mass[b, h].tolist()
                mid = sorted(range(first, n - tail), key=lambda t: (-w[t], t))[:m - first - tail]
                ids = sorted(list(range(first)) + mid + list(range(n - tail, n)))
                ids = torch.tensor(ids, device="cuda")
                out["kept"][b, h, :m] = ids.int()
                out["mass"][b, h, :m] = s["mass"][b, h, ids].double()
                for name, rows in (("k", k64), ("v", v64)):
                    x = rows[h].index_select(0, ids)
                    x = torch.cat((x, x.new_zeros((-m % blk, c["dim"])))).reshape(-1, blk, c["dim"])
                    none = x.new_zeros((x.shape[0], 0, c["dim"]))
                    codes, scale = _block64(none, x.new_zeros(x.shape[0]), x)
                    out[name][b, :m, h] = (codes * scale[:, None, None]).flatten(0, 1)[:m]
        return out
    at = [0] + s["cu_q"].tolist()[1:] if s["cu_q"] is not None else list(range(c["batch"] + 1))
    group = c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    mass = s["mass"].double() if c["op"] == "mass" else None
    for b, n in enumerate(lens):
        nq = at[b + 1] - at[b]
        if not n or not nq:
            continue
        k = _rows64(s, "k", s["table"][b], n)
        v = _rows64(s, "v", s["table"][b], n) if mass is None else None
        hide = torch.ones((nq, n), dtype=torch.bool, device="cuda").triu(n - nq + 1)
        dead = hide.all(1)
        for h in range(c["hq"]):
            x = (s["q"][at[b]:at[b + 1], h].double() @ k[h // group].T) * s["scale"]
            x[hide] = -math.inf
            if mass is not None:
                total = s["lse"][at[b]:at[b + 1], h, None].double()
                mass[b, h // group, :n] += torch.exp(x - total)[~dead].sum(0)
                continue
            top = torch.logsumexp(x, 1, keepdim=True)
            p = torch.where(dead[:, None], 0.0, torch.exp(x - top))
            out[at[b]:at[b + 1], h] = p @ v[h // group]
            lse[at[b]:at[b + 1], h] = top[:, 0]
    return {"out": out, "lse": lse} if mass is None else mass
