"""Cases and plain forms of the operators around a paged cache in 8 bits.

* ``append8``: new keys and values written to a paged cache of e4m3 values with a scale for each block of tokens and
  head, keys and queries rotated by position on the way;
* ``attend8``: attention of one new token per sequence over such a cache, all rows or a window with a few first rows;
* ``sinks``: attention over a cache in 16 or 32 bits with a window and a few first rows that stay visible;
* ``resize``: page tables, offsets and slots of the new rows from the sequences' lengths: pages taken from a free list,
  and given back.

``run`` computes them with elementary torch operations in 32 bits, or, where ``own`` is true, through the
package's entry points. ``exact`` is the same from the definitions in 64 bits.

A cache in 8 bits comes back as the e4m3 tensor, whose values are in units of their block's scale, and the scales.
"""
import math

import torch

own = False

_kda = None


def _pkg():
    global _kda
    if _kda is None:
        import chunked_gated_delta_10_gb300

        _kda = chunked_gated_delta_10_gb300
    return _kda


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
_E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # One user's token: the block's other rows are there already, and may have to follow a larger scale.
        dict(name="append8_1", op="append8", N=1, T=1, ragged=False, HQ=32, HKV=8, K=128, V=128, page=16, block=16,
             rot=128, pairs=False, cached=2047, dtype="bf16"),
        # One token for each of a serving batch, half of each head rotated, a scale for a page.
        dict(name="append8_128", op="append8", N=128, T=1, ragged=False, HQ=32, HKV=8, K=128, V=128, page=64, block=64,
             rot=64, pairs=False, cached=1000, dtype="bf16"),
        # Three prompts in full precision, neighbouring channels paired, pages and blocks that divide nothing else.
        dict(name="append8_f32", op="append8", N=3, T=701, ragged=True, HQ=6, HKV=2, K=64, V=128, page=27, block=9,
             rot=64, pairs=True, cached=130, dtype="f32"),
        # Sixteen packed prompts of 1 to 4096 tokens into an empty cache.
        dict(name="append8_prompts", op="append8", N=16, T=4096, ragged=True, HQ=32, HKV=8, K=128, V=128, page=64,
             block=16, rot=128, pairs=False, cached=0, dtype="bf16"),
        # One user at 2048 tokens: latency.
        dict(name="attend8_1", op="attend8", N=1, L=2048, ragged=False, HQ=32, HKV=8, K=128, V=128, page=64, block=16,
             window=0, sinks=0, dtype="bf16"),
        # One user at the long context: few heads, the length has to be split.
        dict(name="attend8_65536", op="attend8", N=1, L=65536, ragged=False, HQ=16, HKV=2, K=128, V=128, page=16,
             block=16, window=0, sinks=0, dtype="bf16"),
        # Queries in full precision, no grouping, a window with four first rows, odd pages.
        dict(name="attend8_f32", op="attend8", N=12, L=1500, ragged=True, HQ=16, HKV=16, K=64, V=64, page=20, block=5,
             window=1024, sinks=4, dtype="f32"),
        # A serving batch of 64 at 0 to 8192 tokens.
        dict(name="attend8_64", op="attend8", N=64, L=8192, ragged=True, HQ=32, HKV=8, K=128, V=128, page=64, block=64,
             window=0, sinks=0, dtype="bf16"),
        # A full-precision batch with a window and first rows that end inside a page.
        dict(name="sinks_f32", op="sinks", N=8, L=6000, ragged=True, HQ=20, HKV=4, K=128, V=64, page=27, window=777,
             sinks=5, dtype="f32"),
        # A serving batch of 64 at 0 to 16384 tokens, of which each sees a first page and the last 4096.
        dict(name="sinks_64", op="sinks", N=64, L=16384, ragged=True, HQ=32, HKV=8, K=128, V=128, page=64, window=4096,
             sinks=64, dtype="bf16"),
        # A decoding batch of 256, one more token each, and the token taken back again.
        dict(name="resize_256", op="resize", N=256, T=1, page=16, cached=4000),
        # A thousand requests of 1 to 4096 tokens that come, and go.
        dict(name="resize_1000", op="resize", N=1000, T=4096, page=16, cached=0),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _drawn(rng):
    op = rng.choice(["append8", "attend8", "sinks", "resize"])
    if op == "resize":
        return dict(op=op, N=_log(rng, 1, 2000), T=rng.choice([1, _log(rng, 1, 4096)]), page=rng.choice([1, 5, 16, 64, 100]),
                    cached=rng.choice([0, _log(rng, 1, 8000)]))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    K, V = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64)])
    kv = rng.choice([1, 2, 3, 4, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    page, block = rng.choice([(1, 1), (5, 1), (16, 16), (16, 4), (27, 9), (32, 32), (64, 16), (64, 64), (100, 50), (128, 8)])
    heads = dict(HQ=kv * group, HKV=kv, K=K, V=V, page=page, dtype=dtype)
    if op != "sinks":
        heads["block"] = block
    if op == "append8":
        one = rng.random() < 0.5
        return dict(op=op, N=_log(rng, 1, 256) if one else _log(rng, 1, 16), T=1 if one else _log(rng, 2, 4096),
                    ragged=not one, rot=rng.choice([0, 32, 64, K]), pairs=rng.random() < 0.5, cached=_log(rng, 1, 1024),
                    **heads)
    window = _log(rng, 1, 4096) if op == "sinks" or rng.random() < 0.4 else 0
    return dict(op=op, N=_log(rng, 1, 64), L=_log(rng, 1, 65536), ragged=rng.random() < 0.6, window=window,
                sinks=_log(rng, 1, 128) if op == "sinks" or window and rng.random() < 0.5 else 0, **heads)


def _bound(case):
    """An upper bound of the work of the case (in bytes, longest lengths taken) and of its memory in the plain form."""
    if case["op"] == "resize":
        return 60.0 * case["N"] * case["T"] + 16.0 * case["N"] * (case["cached"] + case["T"]) / case["page"]
    wide = case["HKV"] * (case["K"] + case["V"])
    if case["op"] == "append8":
        return 2.0 * _BYTES[case["dtype"]] * case["N"] * case["T"] * (wide + case["HQ"] * case["K"])
    # the plain form gathers the cache in 32 bits
    return 2.0 * case["N"] * case["L"] * wide + 2.0 * case["N"] * case["L"] * case["HQ"]


def draw(rng):
    while True:
        case = _drawn(rng)
        if _bound(case) <= (2.0e8 if case["op"] == "resize" else 1.0e9):
            return case


def _lengths(case):
    """The lengths of a case's sequences, or of their new rows. They go by the case alone, so that its outputs always have
    the same shapes. A sequence of a ragged batch that attends has none."""
    N, longest = case["N"], case["L"] if "L" in case else case["T"]
    if not case.get("ragged", longest > 1):
        return torch.full((N,), longest, dtype=torch.int64)
    lens = torch.randint(1, longest + 1, (N,), generator=torch.Generator().manual_seed(1000 * N + longest))
    if "L" in case and N > 2:
        lens[N // 2] = 0
    return lens


def _pages(lens, page, width, gen, dev):
    """A table of scattered pages for sequences of these lengths, -1 where there is none, and the pool's other pages."""
    need = (lens + page - 1) // page
    pool = len(lens) * width + 2
    have = torch.arange(width, device=dev)[None, :] < need.to(dev)[:, None]
    order, used = torch.randperm(pool, generator=gen, device=dev).to(torch.int32), int(need.sum())
    table = torch.full(have.shape, -1, dtype=torch.int32, device=dev)
    table[have] = order[:used]
    return table, order[used:], pool


def _normal(gen, dev, dtype, *shape):
    return torch.randn(*shape, generator=gen, device=dev).to(dtype)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    N, page = case["N"], case["page"]
    s = dict(case)
    lens = _lengths(case)
    if case["op"] == "resize":
        cached = torch.randint(case["cached"] // 2, case["cached"] + 1, (N,), generator=torch.Generator().manual_seed(seed + 1))
        s["table"], rest, pool = _pages(cached, page, -(-(case["cached"] + case["T"]) // page), gen, dev)
        s["lens"], s["new"] = cached.to(dev, torch.int32), (cached + lens).to(dev, torch.int32)
        s["free"] = torch.full((pool,), -1, dtype=torch.int32, device=dev)
        s["free"][: len(rest)] = rest
        s["count"] = torch.tensor([len(rest)], dtype=torch.int32, device=dev)
        s["rows"] = int(lens.sum())
        return s
    dt, K, V, HQ, HKV = _TYPES[case["dtype"]], case["K"], case["V"], case["HQ"], case["HKV"]
    if case["op"] == "append8":
        rows = int(lens.sum())
        cached = torch.randint(0, case["cached"] + 1, (N,), generator=torch.Generator().manual_seed(seed + 1))
        longest = case["cached"] + case["T"]
        s["table"], _, pool = _pages(cached + lens, page, -(-longest // page), gen, dev)
        s["lens"] = cached.to(dev, torch.int32)
        s["cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(dev) if case["ragged"] else None
        s["q"] = _normal(gen, dev, dt, rows, HQ, K)
        s["k"] = _normal(gen, dev, dt, rows, HKV, K)
        s["v"] = _normal(gen, dev, dt, rows, HKV, V)
        if case["rot"]:
            half = case["rot"] // 2
            rate = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
            angle = torch.arange(longest, device=dev, dtype=torch.float64)[:, None] * rate
            s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        else:
            s["rope"] = None
    else:
        s["table"], _, pool = _pages(lens, page, -(-case["L"] // page), gen, dev)
        s["lens"] = lens.to(dev, torch.int32)
        s["q"] = (2.0 * torch.randn(N, HQ, K, generator=gen, device=dev)).to(dt)
    # a pool's pages hold the heads one after another; the tensors show [page, row, head, channel]
    if case["op"] == "sinks":
        s["kc"], s["vc"] = (_normal(gen, dev, dt, pool, HKV, page, d).transpose(1, 2) for d in (K, V))
        return s
    blocks = page // case["block"]
    for x, d in (("k", K), ("v", V)):
        top = torch.empty(pool, HKV, page, d, device=dev).normal_(0, 110.0, generator=gen).clamp_(-448, 448)
        s[x + "c"] = top.to(_E4M3).transpose(1, 2)
        # of a mean of 2^-7, as if the values had a standard deviation near 1; powers of two, as an append leaves them
        spread = torch.randint(-8, -5, (pool, HKV, blocks), generator=gen, device=dev).double()
        s[x + "s"] = torch.exp2(spread).float().transpose(1, 2)
    return s


# ------------------------------------------------------------------ plain forms


def _turn(x, cos, sin, pairs):
    """The rotation of the leading channels of x [rows, heads, K] by per-row angles [rows, r / 2]."""
    r = 2 * cos.shape[1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if pairs else (x[..., : r // 2], x[..., r // 2 : r])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _where(s):
    """Sequence and position of each new row."""
    rows, dev = s["k"].shape[0], s["k"].device
    row = torch.arange(rows, device=dev)
    if s["cu"] is None:
        n = row // s["T"]
        first = n * s["T"]
    else:
        n = torch.searchsorted(s["cu"], row, right=True) - 1
        first = s["cu"][n]
    return n, s["lens"].long()[n] + row - first


def _least_scale(top):
    """The smallest power of two, 2^-126 at least, by which values of this magnitude come to 448 at most."""
    part, power = torch.frexp(top)  # top = part 2^power, part in [0.5, 1); 448 = 0.875 2^9
    power = torch.where(part > 0.875, power - 8, power - 9)
    return torch.ldexp(torch.ones_like(top), torch.where(top > 0, power, -126).clamp_min(-126))


def _plain_append8(s):
    dt, page, block, rows = s["k"].dtype, s["page"], s["block"], torch.arange(s["block"], device=s["k"].device)
    n, pos = _where(s)
    at, off = s["table"].long()[n, pos // page], pos % page
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if s["rope"] is not None:
        cos, sin = s["rope"][pos].chunk(2, 1)
        q, k = (_turn(x, cos, sin, s["pairs"]) for x in (q, k))
    # a sequence's first new row may lie in a block that has rows: the block of old rows of each sequence
    lens = s["lens"].long()
    first = lens - lens % block
    their = s["table"].long().gather(1, (first // page)[:, None])[:, 0].clamp_min(0)
    their_block, their_rows = first % page // block, first[:, None] % page + rows
    has = lens % block > 0
    old = (rows < (lens % block)[:, None]) & has[:, None]
    for x, new in (("k", k), ("v", v)):
        cache, scales = s[x + "c"], s[x + "s"]
        flat = torch.zeros(scales.shape, device=new.device)
        key = (at * scales.shape[1] + off // block)[:, None].expand(-1, s["HKV"])
        top = flat.flatten(0, 1).scatter_reduce_(0, key, new.abs().amax(-1), "amax").view(scales.shape)
        least = _least_scale(top)
        before = scales[their, their_block]
        kept = torch.where(has[:, None], torch.maximum(before, least[their, their_block]), least[their, their_block])
        least[their, their_block] = kept
        held = cache[their[:, None], their_rows].float()
        again = (held * (before / kept)[:, None, :, None]).to(_E4M3)
        bits = cache.view(torch.uint8)
        bits[their[:, None], their_rows] = torch.where(old[:, :, None, None], again.view(torch.uint8),
                                                       bits[their[:, None], their_rows])
        bits[at, off] = (new / least[at, off // block][..., None]).to(_E4M3).view(torch.uint8)
        scales[at, off // block] = least[at, off // block]
    return dict(q=q.to(dt), k_cache=s["kc"], v_cache=s["vc"], k_scale=s["ks"], v_scale=s["vs"])


def _plain_attend(s):
    N, HKV, dt = s["N"], s["HKV"], s["q"].dtype
    table = s["table"].long().clamp_min(0)
    k, v = (s[x][table].float() for x in ("kc", "vc"))  # [N, width, page, HKV, .]
    if "ks" in s:
        k = k * s["ks"][table].repeat_interleave(s["block"], 2)[..., None]
        v = v * s["vs"][table].repeat_interleave(s["block"], 2)[..., None]
    k, v = (x.flatten(1, 2).transpose(1, 2) for x in (k, v))
    q = s["q"].float().view(N, HKV, -1, s["K"])
    scores = q @ k.transpose(2, 3) * s["K"] ** -0.5
    at, lens = torch.arange(k.shape[2], device=k.device), s["lens"].long()[:, None]
    keep = at < lens
    if s["window"]:
        keep = keep & ((at >= lens - s["window"]) | (at < s["sinks"]))
    scores = scores.masked_fill(~keep[:, None, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    e = (scores - top.clamp_min(torch.finfo(torch.float32).min)).exp()
    total = e.sum(-1, keepdim=True)
    o = (e @ v) / total.clamp_min(torch.finfo(torch.float32).tiny)  # (a row of largest score adds 1)
    return dict(o=o.flatten(1, 2).to(dt), lse=(top + total.log()).flatten(1))


def _plain_resize(s, lens, new):
    """One change of lengths: pages beyond the new length go back, in order; then the missing ones are taken, in order."""
    table, free, page, dev = s["table"], s["free"], s["page"], s["table"].device
    has, need = ((x.clamp_min(0).long() + page - 1) // page for x in (lens, new))
    col = torch.arange(table.shape[1], device=dev)
    back = (col >= need[:, None]) & (col < has[:, None])
    given = table[back]
    free[s["count"].long() + torch.arange(len(given), device=dev)] = given
    table[back] = -1
    count = s["count"] + len(given)
    end = (need - has).clamp_min(0).cumsum(0)
    served = (end <= count) | (need <= has)
    take = (col >= has[:, None]) & (col < need[:, None]) & served[:, None]
    taken = take.sum()
    table[take] = free[(count - 1).long() - (take.flatten().cumsum(0) - 1)[take.flatten()]]
    s["count"].copy_(count - taken)
    grown = (new.clamp_min(0) - lens.clamp_min(0)).clamp_min(0).long()
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), grown.cumsum(0)])
    row = torch.arange(s["rows"], device=dev)
    n = (torch.searchsorted(cu, row, right=True) - 1).clamp_max(len(lens) - 1)
    pos = (lens.clamp_min(0).long()[n] + row - cu[n]).clamp(0, page * table.shape[1] - 1)
    at = table[n, pos // page].long()
    slots = torch.where((row < cu[-1]) & (at >= 0) & served[n], at * page + pos % page, -1)
    return cu, slots, torch.where(served, new, lens)


_PLAIN = dict(append8=_plain_append8, attend8=_plain_attend, sinks=_plain_attend)


def _resized(s, there, back):
    return dict(table=s["table"], free=s["free"], count=s["count"], there=there, back=back)


def run(state):
    s = state
    if s["op"] == "resize":  # requests that come, or one more token each; and the same taken back
        if not own:
            return _resized(s, _plain_resize(s, s["lens"], s["new"]), _plain_resize(s, s["new"], s["lens"]))
        kda = _kda or _pkg()
        there, back = (kda.cache_resize(s["table"], x, y, s["free"], s["count"], s["page"], rows=s["rows"])
                       for x, y in ((s["lens"], s["new"]), (s["new"], s["lens"])))
        return _resized(s, there, back)
    if not own:
        return _PLAIN[s["op"]](s)
    kda = _kda or _pkg()
    if s["op"] == "append8":
        q = kda.cache_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"], q=s["q"], rope=s["rope"],
                             interleaved=s["pairs"], cu_seqlens=s["cu"], k_scale=s["ks"], v_scale=s["vs"])
        return dict(q=q, k_cache=s["kc"], v_cache=s["vc"], k_scale=s["ks"], v_scale=s["vs"])
    if s["op"] == "attend8":
        o, lse = kda.cache_attend(s["q"], s["kc"], s["vc"], s["table"], s["lens"], window=s["window"], sinks=s["sinks"],
                                  k_scale=s["ks"], v_scale=s["vs"])
    else:
        o, lse = kda.cache_attend(s["q"], s["kc"], s["vc"], s["table"], s["lens"], window=s["window"], sinks=s["sinks"])
    return dict(o=o, lse=lse)


def work(case):
    """Each input read once, each output written once (caches, tables and lists only where they are touched)."""
    N, page = case["N"], case["page"]
    if case["op"] == "resize":  # there and back
        rows, pages = int(_lengths(case).sum()), -(-_lengths(case) // page)
        return {"bytes": 2 * (N * 20 + 8 * rows + 8 * int(pages.sum())), "flops": 2 * (N + rows)}
    K, V, HQ, HKV, b = case["K"], case["V"], case["HQ"], case["HKV"], _BYTES[case["dtype"]]
    if case["op"] == "append8":
        rows = int(_lengths(case).sum())
        turned = case["rot"] * (HQ + HKV)
        return {"bytes": rows * (2 * b * HQ * K + (b + 1) * HKV * (K + V) + 4 * case["rot"]) + 8 * HKV * -(-rows // case["block"]),
                "flops": 3 * rows * turned + 2 * rows * HKV * (K + V)}
    read = _lengths(case)
    if case["window"]:
        read = read.clamp_max(case["window"] + case["sinks"])
    read = int(read.sum())
    row = HKV * ((K + V) * b if case["op"] == "sinks" else K + V + 8.0 / case["block"])
    return {"bytes": int(read * row) + N * HQ * ((K + V) * b + 4), "flops": 2 * read * HQ * (K + V)}


# ------------------------------------------------------------------ the definitions in 64 bits


def _exact_append8(s, case):
    """Block by block: the values that a block's rows stand for, divided by the block's scale, before they are rounded."""
    page, block = case["page"], case["block"]
    n, pos = _where(s)
    turned = {x: s[x].double() for x in ("q", "k", "v")}
    if case["rot"]:
        half = case["rot"] // 2
        z = torch.complex(s["rope"][:, :half].double(), s["rope"][:, half:].double())[pos]
        for x in (turned["q"], turned["k"]):
            for i in range(half):
                a, b = (2 * i, 2 * i + 1) if case["pairs"] else (i, i + half)
                y = torch.complex(x[..., a], x[..., b]) * z[:, i, None]
                x[..., a], x[..., b] = y.real, y.imag
    out = dict(q=turned["q"])
    for x in ("k", "v"):
        cache, scales = s[x + "c"].double(), s[x + "s"].double()
        for i in range(case["N"]):
            mine = turned[x][n == i]  # rows of positions start .. start + len(mine) - 1
            start = int(s["lens"][i])
            begin, end = start - start % block, start + len(mine)
            width = -(-end // block) * block
            at = torch.arange(begin, width, device=mine.device)
            where = s["table"][i].long()[(at // page).clamp_max(s["table"].shape[1] - 1)], at % page
            now = cache[where] * scales[where[0], where[1] // block][..., None]
            now[at >= end] = 0  # (what lies behind the rows is not theirs)
            now[start - begin: end - begin] = mine
            top = now.clone()
            top[at < start] = 0
            top = top.unflatten(0, (-1, block)).abs().amax((1, 3))  # [blocks, heads], of the new rows
            power = torch.log2(top / 448).ceil().clamp_min(-126)
            power += (top > 448 * torch.exp2(power)).double() - (top <= 224 * torch.exp2(power)).double() * (power > -126)
            if start > begin:
                was = scales[where[0][0], where[1][0] // block]
                power[0] = torch.maximum(power[0], torch.log2(was).round())
            live = at < end
            scale = torch.exp2(power)
            cache[where[0][live], where[1][live]] = (now / scale.repeat_interleave(block, 0)[..., None])[live]
            scales[where[0][::block], where[1][::block] // block] = scale
        out[x + "_cache"], out[x + "_scale"] = cache, scales
    return out


def _exact_attend(s, case):
    N, HQ, HKV, page = case["N"], case["HQ"], case["HKV"], case["page"]
    o = torch.empty(N, HQ, case["V"], dtype=torch.float64, device=s["q"].device)
    lse = torch.empty(N, HQ, dtype=torch.float64, device=s["q"].device)
    for i, end in enumerate(s["lens"].tolist()):
        begin = max(0, end - case["window"]) if case["window"] else 0
        first = min(begin, case["sinks"])
        pos = torch.cat([torch.arange(first), torch.arange(begin, end)]).to(o.device)
        at, row = s["table"][i].long()[pos // page], pos % page
        for j in range(HKV):
            mine = slice(j * HQ // HKV, (j + 1) * HQ // HKV)
            k, v = (s[c][at, row, j].double() for c in ("kc", "vc"))
            if "ks" in s:
                k, v = (x * s[c][at, row // case["block"], j].double()[:, None] for x, c in ((k, "ks"), (v, "vs")))
            x = s["q"][i, mine].double() @ k.T / math.sqrt(case["K"])
            lse[i, mine] = torch.logsumexp(x, 1)
            o[i, mine] = torch.softmax(x, 1) @ v
    return dict(o=o, lse=lse)


def exact(case, seed):
    if case["op"] == "resize":  # whole numbers
        return None
    s = prepare(case, seed)
    return _exact_append8(s, case) if case["op"] == "append8" else _exact_attend(s, case)
