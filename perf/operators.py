"""Operators of block-sparse decoding over the paged cache: cases, plain forms and definitions.

Four operators make one decode step over a long context cheap. A new token's query and key get
their position rotation while its key and value go to their slots (``append``); the channel-wise
largest and smallest key of each touched block is brought up to date (``bounds``); each query
scores every block of its context by an upper bound on its logits and keeps the best ones
(``select``); attention reads the kept blocks only (``attend``).

With ``own`` false, :func:`run` is elementary torch code; with ``own`` true it calls the library.
Caches are ``[blocks, kv_heads, block, dim]``, key bounds ``[blocks, kv_heads, 2, dim]`` with the
largest values first.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


# ---- cases ------------------------------------------------------------------------------------
def listed():
    return [
        # Four requests decode one token each on the smallest geometry: latency of one call.
        dict(name="append-4x1-f16", op="append", seqs=4, new=1, q_heads=4, kv_heads=4, dim=64,
             rot=64, block=16, dtype="f16", cache="f16", paired=False, far=2048),
        # A serving step of 256 requests on the 13B multi-head geometry, one token each.
        dict(name="append-256x1-f16", op="append", seqs=256, new=1, q_heads=40, kv_heads=40,
             dim=128, rot=128, block=16, dtype="f16", cache="f16", paired=False, far=2048),
        # Four prompts of odd length prefilled into an 8-bit cache, neighbouring channels paired
        # and half of each head rotated.
        dict(name="append-4x4095-e4m3", op="append", seqs=4, new=4095, q_heads=32, kv_heads=8,
             dim=128, rot=64, block=16, dtype="bf16", cache="e4m3", paired=True, far=32768),
        # The same serving step's bounds: one block of each of 256 requests changes.
        dict(name="bounds-256x1-f16", op="bounds", seqs=256, new=1, lo=1, hi=2048, kv_heads=40,
             dim=128, block=16, cache="f16"),
        # Bounds of whole long prompts after their prefill: every block of 32 requests.
        dict(name="bounds-32xall-bf16", op="bounds", seqs=32, new=0, lo=16384, hi=32768,
             kv_heads=8, dim=128, block=16, cache="bf16"),
        # Selection for short contexts on the smallest geometry: some keep every block.
        dict(name="select-4-f16", op="select", seqs=4, lo=1, hi=600, q_heads=4, kv_heads=4,
             dim=64, block=16, dtype="f16", cache="f16", keep=16, sink=1, recent=2),
        # Long-context serving with grouped heads: 128 of about 1,500 blocks for each of 32.
        dict(name="select-32-bf16", op="select", seqs=32, lo=16384, hi=32768, q_heads=32,
             kv_heads=8, dim=128, block=16, dtype="bf16", cache="bf16", keep=128, sink=1,
             recent=4),
        # One very long context over an 8-bit cache: few rows, many blocks.
        dict(name="select-1-e4m3", op="select", seqs=1, lo=131072, hi=131072, q_heads=32,
             kv_heads=8, dim=128, block=16, dtype="bf16", cache="e4m3", keep=256, sink=1,
             recent=4),
        # Attention over the kept blocks: the smallest geometry.
        dict(name="attend-4-f16", op="attend", seqs=4, lo=1, hi=600, q_heads=4, kv_heads=4,
             dim=64, block=16, dtype="f16", cache="f16", keep=16),
        # Multi-head attention, one query head per KV head, 64 requests of up to 2,048 tokens.
        dict(name="attend-64-f16", op="attend", seqs=64, lo=1, hi=2048, q_heads=40, kv_heads=40,
             dim=128, block=16, dtype="f16", cache="f16", keep=32),
        # Long-context serving with grouped heads: 4,096 tokens kept of up to 32,768.
        dict(name="attend-32-bf16", op="attend", seqs=32, lo=16384, hi=32768, q_heads=32,
             kv_heads=8, dim=128, block=16, dtype="bf16", cache="bf16", keep=256),
        # Three requests of very long contexts over an 8-bit cache with blocks of 32.
        dict(name="attend-3-e4m3", op="attend", seqs=3, lo=65000, hi=131071, q_heads=32,
             kv_heads=8, dim=128, block=32, dtype="bf16", cache="e4m3", keep=500),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "bounds", "select", "attend"])
    kv_heads = rng.choice([1, 2, 4, 8, 40])
    group = rng.choice([1, 4, 8, 16]) if kv_heads <= 4 else rng.choice([1, 4]) if kv_heads == 8 else 1
    dim = rng.choice([64, 128])
    block = rng.choice([8, 16, 32])
    dtype = rng.choice(["f16", "bf16"])
    cache = "e4m3" if dim == 128 and rng.random() < 0.3 else dtype
    base = dict(op=op, kv_heads=kv_heads, dim=dim, block=block, cache=cache)
    heads = dict(q_heads=kv_heads * group, dtype=dtype)
    if op == "append":
        new = 1 if rng.random() < 0.5 else _log(rng, 2, 4096)
        most = max(1, 16384 * 48 // (new * (kv_heads * (group + 2))))
        rot = rng.choice([r for r in (16, 32, 64, 128) if r <= dim])
        return dict(base, **heads, seqs=_log(rng, 1, min(512, most)), new=new, rot=rot,
                    paired=rng.random() < 0.5, far=rng.choice([4096, 32768, 131072]))
    hi = _log(rng, 1, 131072)
    lo = max(1, int(hi * rng.uniform(0.1, 1.0)))
    if op == "bounds":
        most = max(1, 32 * 24576 * 8 * 128 // (hi * kv_heads * dim))
        return dict(base, seqs=_log(rng, 1, min(512, most)), lo=lo, hi=hi,
                    new=rng.choice([0, 1, _log(rng, 2, 300)]))
    # the pool of a case holds at most about as many values as the largest listed one's
    most = max(1, 32 * 24576 * 8 * 128 // (hi * kv_heads * dim))
    seqs = _log(rng, 1, min(256, most))
    blocks = -(-hi // block)
    if op == "select":
        keep = _log(rng, 8, 1024)
        return dict(base, **heads, seqs=seqs, lo=lo, hi=hi, keep=keep,
                    sink=rng.choice([0, 1, 4]), recent=rng.choice([1, 2, 4]))
    room = 32 * 8 * 256 * 16 * 128 // (seqs * kv_heads * block * dim)
    keep = max(1, min(_log(rng, 8, 1024), room, blocks + 3))
    return dict(base, **heads, seqs=seqs, lo=lo, hi=hi, keep=keep)


def _lens(c):
    """Context lengths spread evenly over [lo, hi], in an order that is not sorted."""
    n = c["seqs"]
    if n == 1:
        return [c["hi"]]
    even = [c["lo"] + (c["hi"] - c["lo"]) * i // (n - 1) for i in range(n)]
    step = next(s for s in (7, 5, 3, 2, 1) if math.gcd(s, n) == 1)
    return [even[(i * step) % n] for i in range(n)]


def _touched(c):
    """Blocks of each sequence that hold one of its newest tokens (new == 0: every block)."""
    bs = c["block"]
    return [-(-n // bs) - (max(0, n - (c["new"] or n)) // bs) for n in _lens(c)]


def work(c):
    size = 1 if c["cache"] == "e4m3" else 2
    heads, dim, bs = c["kv_heads"], c["dim"], c["block"]
    if c["op"] == "append":
        tokens = c["seqs"] * c["new"]
        read = tokens * (c["q_heads"] + 2 * heads) * dim * 2
        write = tokens * (c["q_heads"] * 2 + 2 * heads * size) * dim
        rows = min(tokens, c["far"])
        return {"bytes": read + write + rows * c["rot"] * 4 + tokens * 16,
                "flops": tokens * (c["q_heads"] + heads) * c["rot"] * 3}
    if c["op"] == "bounds":
        blocks = sum(_touched(c))
        tokens = sum((b - 1) * bs + ((n - 1) % bs) + 1 for b, n in zip(_touched(c), _lens(c)))
        return {"bytes": tokens * heads * dim * size + blocks * (heads * 2 * dim * 2 + 4),
                "flops": tokens * heads * dim * 2}
    blocks = sum(-(-n // bs) for n in _lens(c))
    if c["op"] == "select":
        return {"bytes": blocks * (heads * 2 * dim * 2 + 4)
                + c["seqs"] * (c["q_heads"] * dim * 2 + heads * c["keep"] * 4),
                "flops": blocks * heads * 2 * dim * 2}
    kept = sum(min(n, min(-(-n // bs), c["keep"]) * bs) for n in _lens(c))
    return {"bytes": kept * heads * dim * 2 * size + c["seqs"] * (c["q_heads"] * dim * 4
                                                                  + heads * c["keep"] * 4),
            "flops": kept * c["q_heads"] * dim * 4}


# ---- inputs -----------------------------------------------------------------------------------
def _normal(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _pool(shape, cache, gen):
    """A cache pool of keys or values, filled in pieces (a block's tokens have a common part)."""
    x = torch.empty(shape, device=DEV, dtype=TYPES[cache])
    step = max(1, (1 << 26) // max(1, math.prod(shape[1:])))
    for b in range(0, shape[0], step):
        n = min(step, shape[0] - b)
        part = torch.randn((n,) + tuple(shape[1:]), generator=gen, device=DEV)
        part += 0.5 * torch.randn((n, shape[1], 1, shape[3]), generator=gen, device=DEV)
        if cache == "e4m3":  # a scale of 1/64 uses the codes' range
            part = (part * 64).clamp_(-448, 448)
        x[b:b + n] = part.to(TYPES[cache])
    return x


def _tables(c, gen, pool=None):
    """Block tables [seqs, most blocks] over a shuffled pool, padded with -1, and the pool's size."""
    counts = torch.tensor([-(-n // c["block"]) for n in _lens(c)], device=DEV)
    total, most = sum(-(-n // c["block"]) for n in _lens(c)), -(-max(_lens(c)) // c["block"])
    pool = pool or -(-total * 5 // 4) + 1
    order = torch.randperm(pool, generator=gen, device=DEV)[:total].to(torch.int32)
    table = torch.full((c["seqs"], most), -1, dtype=torch.int32, device=DEV)
    held = torch.arange(most, device=DEV)[None] < counts[:, None]
    table[held] = order
    return table, pool


def _scales(c, gen):
    if c["cache"] != "e4m3":
        return None, None
    k, v = (torch.rand((c["kv_heads"],), generator=gen, device=DEV) * 0.01 + 0.01 for _ in range(2))
    return k, v


def prepare(c, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    heads, dim, bs = c["kv_heads"], c["dim"], c["block"]
    s = {"case": c}
    if c["op"] == "append":
        seqs, new, dt = c["seqs"], c["new"], TYPES[c["dtype"]]
        # one projection's output: queries, keys and values side by side for each token
        rows = _normal((seqs * new, (c["q_heads"] + 2 * heads) * dim), dt, gen)
        q, k, v = rows.split([c["q_heads"] * dim, heads * dim, heads * dim], dim=1)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, dim)) for x in (q, k, v))
        half = c["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) * 2 / c["rot"])
        angle = torch.arange(c["far"], device=DEV, dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        first = torch.randint(0, max(1, c["far"] - new), (seqs, 1), generator=gen, device=DEV)
        pos = first + torch.arange(new, device=DEV)
        most = -(-new // bs) + 1
        pool = seqs * most + 3
        table = torch.randperm(pool, generator=gen, device=DEV)[: seqs * most].view(seqs, most)
        block = table.gather(1, pos // bs - first // bs)
        s["positions"], s["slots"] = pos.flatten(), (block * bs + pos % bs).flatten()
        s["k_cache"], s["v_cache"] = (_pool((pool, heads, bs, dim), c["cache"], gen)
                                      for _ in range(2))
        s["k_scale"], s["v_scale"] = _scales(c, gen)
        s["q_out"] = torch.empty((seqs * new, c["q_heads"], dim), device=DEV, dtype=dt)
        return s
    s["lens"] = torch.tensor(_lens(c), dtype=torch.int32, device=DEV)
    s["table"], pool = _tables(c, gen)
    small = torch.float16 if c["cache"] == "e4m3" else TYPES[c["cache"]]
    if c["op"] == "bounds":
        s["k_cache"] = _pool((pool, heads, bs, dim), c["cache"], gen)
        s["bounds"] = torch.zeros((pool, heads, 2, dim), device=DEV, dtype=small)
        s["new"] = torch.full((c["seqs"],), c["new"], dtype=torch.int32, device=DEV) if c["new"] else None
        return s
    s["q"] = _normal((c["seqs"], c["q_heads"], dim), TYPES[c["dtype"]], gen)
    if c["op"] == "select":
        a, b = (_pool((pool, heads, 1, dim), c["cache"], gen) for _ in range(2))
        a, b = a.to(small), b.to(small)  # the two ends of each channel's range in a block
        s["bounds"] = torch.cat([torch.maximum(a, b), torch.minimum(a, b)], 2)
        return s
    s["k_cache"], s["v_cache"] = (_pool((pool, heads, bs, dim), c["cache"], gen) for _ in range(2))
    s["k_scale"], s["v_scale"] = _scales(c, gen)
    # for each KV head its own blocks, the last one always among them, ascending, -1 behind them
    most, keep = s["table"].shape[1], c["keep"]
    count = (s["lens"] + bs - 1) // bs
    luck = torch.rand((c["seqs"], heads, most), generator=gen, device=DEV)
    index = torch.arange(most, device=DEV)
    luck[(index >= count[:, None])[:, None].expand_as(luck)] = -1.0
    luck[(index == count[:, None] - 1)[:, None].expand_as(luck)] = 2.0
    value, at = luck.topk(min(keep, most), dim=2)
    at = torch.where(value < 0, most, at).sort(dim=2).values
    selected = torch.full((c["seqs"], heads, keep), -1, dtype=torch.int32, device=DEV)
    selected[:, :, : at.shape[2]] = torch.where(at >= most, -1, at)
    s["selected"] = selected
    return s


# ---- one pass ---------------------------------------------------------------------------------
def run(s):
    return {"append": _append, "bounds": _bounds, "select": _select, "attend": _attend}[s["case"]["op"]](s)


def _append(s):
    c = s["case"]
    if own:
        import paged_kv_cache_319_b200 as kvp

        kvp.rope_reshape_and_cache(s["q"], s["k"], s["v"], s["cos_sin"], s["positions"],
                                   s["k_cache"], s["v_cache"], s["slots"], s["q_out"],
                                   interleaved=c["paired"], k_scale=s["k_scale"],
                                   v_scale=s["v_scale"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    rot, half, bs = c["rot"], c["rot"] // 2, c["block"]
    row = s["cos_sin"][s["positions"]][:, None]
    cos, sin = row[..., :half], row[..., half:]

    def rotated(x):
        x = x.float()
        if c["paired"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:rot]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([turned, x[..., rot:]], -1)

    def store(pool, x, scale):
        block, off = s["slots"] // bs, s["slots"] % bs
        if c["cache"] == "e4m3":
            x = (x / scale[:, None]).clamp(-448, 448).to(pool.dtype)
            pool.view(torch.uint8)[block, :, off] = x.view(torch.uint8)
        else:
            pool[block, :, off] = x.to(pool.dtype)

    s["q_out"].copy_(rotated(s["q"]))
    store(s["k_cache"], rotated(s["k"]), s["k_scale"])
    store(s["v_cache"], s["v"].float(), s["v_scale"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _bounds(s):
    c, bounds = s["case"], s["bounds"]
    if own:
        import paged_kv_cache_319_b200 as kvp

        kvp.update_key_bounds(s["k_cache"], bounds, s["table"], s["lens"], new_tokens=s["new"],
                              max_new_tokens=c["new"] or None, max_context_len=c["hi"])
        return bounds
    bs, lens = c["block"], s["lens"][:, None]
    index = torch.arange(s["table"].shape[1], device=lens.device)[None]
    first = (lens - s["new"][:, None]).clamp(min=0) // bs if c["new"] else torch.zeros_like(lens)
    touched = (index >= first) & (index * bs < lens)
    block = s["table"][touched].long()
    room = (lens - index * bs)[touched]  # valid slots of each touched block
    keys = s["k_cache"][block].float()
    held = (torch.arange(bs, device=keys.device) < room[:, None])[:, None, :, None]
    high = torch.where(held, keys, -math.inf).amax(2)
    low = torch.where(held, keys, math.inf).amin(2)
    bounds[block] = torch.stack([high, low], 2).to(bounds.dtype)
    return bounds


def _select(s):
    c, q, bounds, table, lens = s["case"], s["q"], s["bounds"], s["table"], s["lens"]
    if own:
        import paged_kv_cache_319_b200 as kvp

        return kvp.select_blocks(q, bounds, table, lens, block_size=c["block"],
                                 num_selected=c["keep"], num_sink=c["sink"],
                                 num_recent=c["recent"], max_context_len=c["hi"])
    seqs, most, heads = *table.shape, c["kv_heads"]
    # sums in 64 bits: which of two near blocks is taken hangs on their last bits
    q = q.double().unflatten(1, (heads, -1))
    weight = torch.stack([q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)], 2)  # [S, Hkv, 2, D]
    score = (bounds[table.clamp(min=0).long()].double() * weight[:, None]).sum((3, 4))
    index = torch.arange(most, device=q.device)
    count = ((lens + c["block"] - 1) // c["block"])[:, None]
    forced = (index < c["sink"]) | (index >= count - c["recent"])
    score = torch.where(forced[..., None], math.inf, score)
    score = torch.where((index < count)[..., None], score, -math.inf)
    keep = min(c["keep"], most)
    best = score.transpose(1, 2).sort(dim=2, descending=True, stable=True).indices[..., :keep]
    best = torch.where(best < count[..., None], best, most).sort(dim=2).values
    out = torch.full((seqs, heads, c["keep"]), -1, dtype=torch.int32, device=q.device)
    out[..., :keep] = torch.where(best == most, -1, best)
    return out


def _attend(s):
    c, q, lens = s["case"], s["q"], s["lens"]
    scale = 1.0 / math.sqrt(c["dim"])
    if own:
        import paged_kv_cache_319_b200 as kvp

        return kvp.paged_attention_decode_sparse(q, s["k_cache"], s["v_cache"], s["table"], lens,
                                                 s["selected"], scale, k_scale=s["k_scale"],
                                                 v_scale=s["v_scale"], max_context_len=c["hi"])
    seqs, heads, bs = c["seqs"], c["kv_heads"], c["block"]
    kept = s["selected"].long()
    block = s["table"].long().gather(1, kept.clamp(min=0).flatten(1)).view_as(kept)
    head = torch.arange(heads, device=q.device)[None, :, None]
    k, v = (x[block, head].float().flatten(2, 3) for x in (s["k_cache"], s["v_cache"]))
    pos = kept[..., None] * bs + torch.arange(bs, device=q.device)
    held = ((kept >= 0)[..., None] & (pos < lens[:, None, None, None])).flatten(2)[:, :, None]
    z = torch.einsum("shgd,shtd->shgt", q.float().unflatten(1, (heads, -1)) * scale, k)
    if s["k_scale"] is not None:
        z = z * s["k_scale"][:, None, None]
        v = v * s["v_scale"][:, None, None]
    z = torch.where(held, z, -math.inf)
    p = (z - z.amax(-1, keepdim=True)).exp()
    out = torch.einsum("shgt,shtd->shgd", p / p.sum(-1, keepdim=True), v)
    return out.flatten(1, 2).to(q.dtype)


# ---- definitions in 64 bits -------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    bs, heads = c["block"], c["kv_heads"]
    if c["op"] == "append":
        half = c["rot"] // 2
        angles = s["cos_sin"].double()[s["positions"]]
        turn = torch.complex(angles[:, :half], angles[:, half:])[:, None]

        def rotated(x):
            x = x.double().clone()
            lo, hi = ((slice(0, c["rot"], 2), slice(1, c["rot"], 2)) if c["paired"]
                      else (slice(0, half), slice(half, c["rot"])))
            z = torch.complex(x[..., lo].contiguous(), x[..., hi].contiguous()) * turn
            x[..., lo], x[..., hi] = z.real, z.imag
            return x

        out = {"q": rotated(s["q"])}
        for name, x, scale in (("k_cache", rotated(s["k"]), s["k_scale"]),
                               ("v_cache", s["v"].double(), s["v_scale"])):
            pool = s[name].double().transpose(1, 2).contiguous()
            if scale is not None:
                x = (x / scale.double()[:, None]).clamp(-448, 448)
            pool.view(-1, heads, c["dim"])[s["slots"]] = x
            out[name] = pool.transpose(1, 2)
        return out
    lens, table = _lens(c), s["table"].long()
    if c["op"] == "bounds":
        out = s["bounds"].double()
        for i, n in enumerate(lens):
            first = max(0, n - (c["new"] or n)) // bs
            ids = table[i, first: -(-n // bs)]
            keys = s["k_cache"][ids].double()
            full = keys[:-1]
            out[ids[:-1], :, 0], out[ids[:-1], :, 1] = full.amax(2), full.amin(2)
            last = keys[-1, :, : (n - 1) % bs + 1]
            out[ids[-1], :, 0], out[ids[-1], :, 1] = last.amax(1), last.amin(1)
        return out
    if c["op"] == "select":
        out = torch.full((c["seqs"], heads, c["keep"]), -1, dtype=torch.int32, device=DEV)
        for i, n in enumerate(lens):
            count = -(-n // bs)
            high, low = s["bounds"][table[i, :count]].double().unbind(2)
            score = 0.0
            for g in range(c["q_heads"] // heads):
                q = s["q"][i, g::c["q_heads"] // heads].double()
                score = score + torch.maximum(q * high, q * low).sum(-1)
            score[: c["sink"]] = math.inf
            score[max(0, count - c["recent"]):] = math.inf
            best = score.t().sort(dim=1, descending=True, stable=True).indices[:, : c["keep"]]
            out[i, :, : best.shape[1]] = best.sort(dim=1).values
        return out
    out = torch.zeros((c["seqs"], c["q_heads"], c["dim"]), dtype=torch.float64, device=DEV)
    group = c["q_heads"] // heads
    for i, n in enumerate(lens):
        kept = s["selected"][i].long()
        kept = kept[:, : min(c["keep"], -(-n // bs))]  # the lists of one sequence are equally long
        for h in range(heads):
            token = (kept[h][:, None] * bs + torch.arange(bs, device=DEV)).flatten()
            token = token[token < n]
            at = (table[i, token // bs], h, token % bs)
            k, v = s["k_cache"][at].double(), s["v_cache"][at].double()
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            z = s["q"][i, h * group:(h + 1) * group].double() @ k.t() / math.sqrt(c["dim"])
            out[i, h * group:(h + 1) * group] = torch.softmax(z, -1) @ v
    return out
