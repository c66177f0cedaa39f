"""Cases and plain forms of the single-token serving operators.

Three operators that follow the chunked forward when a hybrid of KDA layers and full-attention layers
answers token by token:

* ``step``: T new tokens per sequence (one, or a few) on the fp32 KDA states, in place;
* ``append``: new keys and values written to a paged cache, keys and queries rotated by position on the way;
* ``attend``: attention of one new token per sequence over the paged cache.

``run`` computes them with elementary torch operations in 32 bits, or, where ``own`` is true, through the
package's entry points. ``exact`` is the same from the definitions in 64 bits.
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


def listed():
    return [
        # One user, 16 heads of 128 (the small training shape's layer): the latency of one KDA layer.
        dict(name="step_1", op="step", N=1, T=1, H=16, HV=16, K=128, V=128, dtype="bf16", slots=False),
        # A full-precision check run: odd batch, grouped values, unequal head dims.
        dict(name="step_f32", op="step", N=33, T=1, H=4, HV=12, K=64, V=128, dtype="f32", slots=False),
        # Four tokens at once (an accepted draft, or a short continuation), grouped values, states in slots.
        dict(name="step_4_tokens", op="step", N=16, T=4, H=16, HV=32, K=128, V=128, dtype="bf16", slots=True),
        # A serving batch of 256 on the 32-head layer, states in slots.
        dict(name="step_256", op="step", N=256, T=1, H=32, HV=32, K=128, V=128, dtype="bf16", slots=True),
        # One user's token, grouped queries, rotation of whole heads.
        dict(name="append_1", op="append", N=1, T=1, ragged=False, HQ=32, HKV=8, K=128, V=128, page=16, rot=128,
             pairs=False, cached=2047, dtype="bf16"),
        # One token for each of a serving batch, half of each head rotated.
        dict(name="append_128", op="append", N=128, T=1, ragged=False, HQ=32, HKV=8, K=128, V=128, page=64, rot=64,
             pairs=False, cached=1000, dtype="bf16"),
        # Three prompts in full precision, neighbouring channels paired, pages that do not divide anything.
        dict(name="append_f32", op="append", N=3, T=701, ragged=True, HQ=6, HKV=2, K=64, V=128, page=27, rot=64,
             pairs=True, cached=130, dtype="f32"),
        # Sixteen packed prompts of 1 to 4096 tokens into an empty cache.
        dict(name="append_prompts", op="append", N=16, T=4096, ragged=True, HQ=32, HKV=8, K=128, V=128, page=64,
             rot=128, pairs=False, cached=0, dtype="bf16"),
        # One user at 2048 tokens: latency.
        dict(name="attend_1", op="attend", N=1, L=2048, ragged=False, HQ=32, HKV=8, K=128, V=128, page=64, window=0,
             dtype="bf16"),
        # One user at the long context: few heads, the length has to be split.
        dict(name="attend_65536", op="attend", N=1, L=65536, ragged=False, HQ=16, HKV=2, K=128, V=128, page=16,
             window=0, dtype="bf16"),
        # A full-precision batch, no grouping, a window, odd pages.
        dict(name="attend_f32", op="attend", N=12, L=1500, ragged=True, HQ=16, HKV=16, K=64, V=64, page=20, window=1024,
             dtype="f32"),
        # A serving batch of 64 at 1 to 8192 tokens.
        dict(name="attend_64", op="attend", N=64, L=8192, ragged=True, HQ=32, HKV=8, K=128, V=128, page=64, window=0,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _drawn(rng):
    op = rng.choice(["step", "append", "attend"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    K, V = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64)])
    kv = rng.choice([1, 2, 3, 4, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    if op == "step":
        return dict(op=op, N=_log(rng, 1, 256), T=rng.choice([1, 1, 2, 3, 4, 7]), H=kv, HV=kv * min(group, 4), K=K, V=V,
                    dtype=dtype, slots=rng.random() < 0.5)
    heads = dict(HQ=kv * group, HKV=kv, K=K, V=V, page=rng.choice([1, 5, 16, 27, 32, 64, 100, 128]), dtype=dtype)
    if op == "append":
        one = rng.random() < 0.5
        return dict(op=op, N=_log(rng, 1, 256) if one else _log(rng, 1, 16), T=1 if one else _log(rng, 2, 4096),
                    ragged=not one, rot=rng.choice([0, 32, 64, K]), pairs=rng.random() < 0.5, cached=_log(rng, 1, 1024),
                    **heads)
    return dict(op=op, N=_log(rng, 1, 64), L=_log(rng, 1, 65536), ragged=rng.random() < 0.6,
                window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), **heads)


def _bound(case):
    """An upper bound of the work of the case (in bytes, longest lengths taken) and of its memory in the plain form."""
    b = _BYTES[case["dtype"]]
    if case["op"] == "step":
        return 8.0 * case["N"] * case["HV"] * case["K"] * case["V"] * (1 + 0.1 * case["T"])
    wide = case["HKV"] * (case["K"] + case["V"])
    if case["op"] == "append":
        return 2.0 * b * case["N"] * case["T"] * (wide + case["HQ"] * case["K"])
    # the plain form gathers the cache in 32 bits
    return 2.0 * case["N"] * case["L"] * wide + 2.0 * case["N"] * case["L"] * case["HQ"]


def draw(rng):
    while True:
        case = _drawn(rng)
        if _bound(case) <= 1.0e9:
            return case


def _lengths(case):
    """The lengths of a case's sequences. They go by the case alone, so that its outputs always have the same shapes."""
    N, longest = case["N"], case["T"] if case["op"] == "append" else case["L"]
    if not case["ragged"]:
        return torch.full((N,), longest, dtype=torch.int64)
    return torch.randint(1, longest + 1, (N,), generator=torch.Generator().manual_seed(1000 * N + longest))


def _pages(lens, page, width, gen, dev):
    """A pool of pages, some of them free, and a table of scattered pages for sequences of these lengths; -1 where there is none."""
    need = (lens + page - 1) // page
    pool = len(lens) * width + 2
    at = torch.arange(width, device=dev)[None, :]
    have = at < need.to(dev)[:, None]
    order = torch.randperm(pool, generator=gen, device=dev)[: int(need.sum())]
    table = torch.full(have.shape, -1, dtype=torch.int64, device=dev)
    table[have] = order
    return pool, table.to(torch.int32)


def _normal(gen, dev, dtype, *shape):
    return torch.randn(*shape, generator=gen, device=dev).to(dtype)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt, N, K, V = _TYPES[case["dtype"]], case["N"], case["K"], case["V"]
    s = dict(case)
    if case["op"] == "step":
        T, H, HV = case["T"], case["H"], case["HV"]
        q, k = (torch.randn(N, T, H, K, generator=gen, device=dev) for _ in range(2))
        s["q"], s["k"] = (x.div(x.norm(dim=-1, keepdim=True)).to(dt) for x in (q, k))
        s["v"] = _normal(gen, dev, dt, N, T, HV, V)
        gate = torch.randn(N, T, HV, K, generator=gen, device=dev) + 3.0
        s["g"] = torch.nn.functional.logsigmoid(gate)
        s["beta"] = torch.sigmoid(torch.randn(N, T, HV, generator=gen, device=dev)).to(dt)
        pool = N + 3 if case["slots"] else N
        s["state"] = 0.3 * torch.randn(pool, HV, K, V, generator=gen, device=dev)
        s["slot_of"] = torch.randperm(pool, generator=gen, device=dev)[:N].to(torch.int32) if case["slots"] else None
        return s
    HQ, HKV, page = case["HQ"], case["HKV"], case["page"]
    lens = _lengths(case)
    if case["op"] == "append":
        rows = int(lens.sum())
        cached = torch.randint(0, case["cached"] + 1, (N,), generator=torch.Generator().manual_seed(seed + 1))
        longest = case["cached"] + case["T"]
        pool, s["table"] = _pages(cached + lens, page, -(-longest // page), gen, dev)
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
        pool, s["table"] = _pages(lens, page, -(-case["L"] // page), gen, dev)
        s["lens"] = lens.to(dev, torch.int32)
        s["q"] = (2.0 * torch.randn(N, HQ, K, generator=gen, device=dev)).to(dt)
    # a pool's pages hold the heads one after another; the tensors show [page, row, head, channel]
    s["kc"] = _normal(gen, dev, dt, pool, HKV, page, K).transpose(1, 2)
    s["vc"] = _normal(gen, dev, dt, pool, HKV, page, V).transpose(1, 2)
    return s


# ------------------------------------------------------------------ plain forms


def _plain_step(s):
    dt, T, rep = s["q"].dtype, s["T"], s["HV"] // s["H"]
    at = slice(None) if s["slot_of"] is None else s["slot_of"].long()
    S = s["state"][at]
    q, k = (s[x].float().repeat_interleave(rep, 2) for x in ("q", "k"))
    v, beta, decay = s["v"].float(), s["beta"].float(), s["g"].exp()
    scale = s["K"] ** -0.5
    out = []
    for t in range(T):  # each token needs the state that the one before it left
        S = S * decay[:, t, :, :, None]
        d = beta[:, t, :, None] * (v[:, t] - (k[:, t, :, :, None] * S).sum(2))
        S = S + k[:, t, :, :, None] * d[:, :, None, :]
        out.append(scale * (q[:, t, :, :, None] * S).sum(2))
    s["state"][at] = S
    return dict(o=torch.stack(out, 1).to(dt), state=s["state"])


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


def _plain_append(s):
    dt = s["k"].dtype
    n, pos = _where(s)
    page = s["table"].long()[n, pos // s["page"]]
    q, k = s["q"].float(), s["k"].float()
    if s["rope"] is not None:
        cos, sin = s["rope"][pos].chunk(2, 1)
        q, k = (_turn(x, cos, sin, s["pairs"]) for x in (q, k))
    s["kc"][page, pos % s["page"]] = k.to(dt)
    s["vc"][page, pos % s["page"]] = s["v"]
    return dict(q=q.to(dt), k_cache=s["kc"], v_cache=s["vc"])


def _plain_attend(s):
    N, HKV, dt = s["N"], s["HKV"], s["q"].dtype
    table = s["table"].long().clamp_min(0)
    k, v = (s[x][table].flatten(1, 2).float().transpose(1, 2) for x in ("kc", "vc"))  # [N, HKV, width, .]
    q = s["q"].float().view(N, HKV, -1, s["K"])
    scores = q @ k.transpose(2, 3) * s["K"] ** -0.5
    at, lens = torch.arange(k.shape[2], device=k.device), s["lens"].long()[:, None]
    keep = at < lens
    if s["window"]:
        keep = keep & (at >= lens - s["window"])
    scores = scores.masked_fill(~keep[:, None, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    e = (scores - top).exp()
    total = e.sum(-1, keepdim=True)
    o = (e @ v) / total
    return dict(o=o.flatten(1, 2).to(dt), lse=(top + total.log()).flatten(1))


_PLAIN = dict(step=_plain_step, append=_plain_append, attend=_plain_attend)


def run(state):
    s = state
    if not own:
        return _PLAIN[s["op"]](s)
    kda = _kda or _pkg()
    if s["op"] == "step":
        o = kda.step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slot_of"])
        return dict(o=o, state=s["state"])
    if s["op"] == "append":
        q = kda.cache_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"], q=s["q"], rope=s["rope"],
                             interleaved=s["pairs"], cu_seqlens=s["cu"])
        return dict(q=q, k_cache=s["kc"], v_cache=s["vc"])
    o, lse = kda.cache_attend(s["q"], s["kc"], s["vc"], s["table"], s["lens"], window=s["window"])
    return dict(o=o, lse=lse)


def work(case):
    """Each input read once, each output written once (states and caches only where they are touched)."""
    b, N, K, V = _BYTES[case["dtype"]], case["N"], case["K"], case["V"]
    if case["op"] == "step":
        T, H, HV = case["T"], case["H"], case["HV"]
        token = 2 * H * K * b + 2 * HV * V * b + HV * K * 4 + HV * b
        return {"bytes": 8 * N * HV * K * V + N * T * token, "flops": 7 * N * T * HV * K * V}
    HQ, HKV = case["HQ"], case["HKV"]
    if case["op"] == "append":
        rows = int(_lengths(case).sum())
        turned = case["rot"] * (HQ + HKV)
        return {"bytes": rows * (2 * b * (HQ * K + HKV * (K + V)) + 4 * case["rot"]), "flops": 3 * rows * turned}
    read = _lengths(case)
    if case["window"]:
        read = read.clamp_max(case["window"])
    read = int(read.sum())
    return {"bytes": read * HKV * (K + V) * b + N * HQ * ((K + V) * b + 4), "flops": 2 * read * HQ * (K + V)}


# ------------------------------------------------------------------ the definitions in 64 bits


def _exact_step(s):
    rep, scale = s["HV"] // s["H"], 1.0 / math.sqrt(s["K"])
    at = torch.arange(s["N"], device=s["q"].device) if s["slot_of"] is None else s["slot_of"].long()
    state = s["state"].double()
    o = torch.empty(s["N"], s["T"], s["HV"], s["V"], dtype=torch.float64, device=state.device)
    q, k, v, g, beta = (s[x].double() for x in ("q", "k", "v", "g", "beta"))
    for h in range(s["HV"]):
        S = state[at, h]
        for t in range(s["T"]):
            kt, qt, bt = k[:, t, h // rep], q[:, t, h // rep], beta[:, t, h, None, None]
            S = torch.exp(g[:, t, h])[:, :, None] * S
            S = S - bt * torch.einsum("nk,nj,njv->nkv", kt, kt, S) + bt * torch.einsum("nk,nv->nkv", kt, v[:, t, h])
            o[:, t, h] = scale * torch.einsum("nk,nkv->nv", qt, S)
        state[at, h] = S
    return dict(o=o, state=state)


def _exact_append(s, case):
    n, pos = _where(s)
    kc, vc = s["kc"].double(), s["vc"].double()
    turned = {x: s[x].double() for x in ("q", "k")}
    if case["rot"]:
        half = case["rot"] // 2
        z = torch.complex(s["rope"][:, :half].double(), s["rope"][:, half:].double())[pos]
        for x in turned.values():
            for i in range(half):
                a, b = (2 * i, 2 * i + 1) if case["pairs"] else (i, i + half)
                y = torch.complex(x[..., a], x[..., b]) * z[:, i, None]
                x[..., a], x[..., b] = y.real, y.imag
    for i in range(case["N"]):
        mine = n == i
        at, row = s["table"][i].long()[pos[mine] // case["page"]], pos[mine] % case["page"]
        kc[at, row], vc[at, row] = turned["k"][mine], s["v"][mine].double()
    return dict(q=turned["q"], k_cache=kc, v_cache=vc)


def _exact_attend(s, case):
    N, HQ, HKV, page = case["N"], case["HQ"], case["HKV"], case["page"]
    o = torch.empty(N, HQ, case["V"], dtype=torch.float64, device=s["q"].device)
    lse = torch.empty(N, HQ, dtype=torch.float64, device=s["q"].device)
    for i, end in enumerate(s["lens"].tolist()):
        begin = max(0, end - case["window"]) if case["window"] else 0
        pos = torch.arange(begin, end, device=o.device)
        at, row = s["table"][i].long()[pos // page], pos % page
        for j in range(HKV):
            mine = slice(j * HQ // HKV, (j + 1) * HQ // HKV)
            x = s["q"][i, mine].double() @ s["kc"][at, row, j].double().T / math.sqrt(case["K"])
            lse[i, mine] = torch.logsumexp(x, 1)
            o[i, mine] = torch.softmax(x, 1) @ s["vc"][at, row, j].double()
    return dict(o=o, lse=lse)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "step":
        return _exact_step(s)
    return _exact_append(s, case) if case["op"] == "append" else _exact_attend(s, case)
