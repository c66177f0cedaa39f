"""The single-token operators on the GPU against plain implementations in 64 bits.

Bounds, from unit roundoffs u = 2^-24 (fp32, 24 significant bits) and 2^-8 (bf16, 8 significant bits):

* step: a token's state update and its two products sum K terms; its relative error is at most (K + 10) u of the sum
  of the terms' magnitudes, and T tokens add up (the recurrence contracts). By rows' norms: state 4 T (K + 10) u
  relative L2, and o, a product of the state with a unit vector that is sqrt(K) times smaller than the state's column
  norm, sqrt(K) times that, plus the rounding of o.
* append: x c - y s with one fused or two separate products: 3 u (|x c| + |y s|) per element, plus its rounding.
* attend: a score errs by (K + 4) 2u scale sum |q k| (a tensor core may truncate: 2u); a weight by twice the largest
  score error, 2^-20 for the exponential and, for bf16 inputs, 2^-16 (probabilities as a pair of bf16 values); the sum
  over n rows by 2 (n + 16) u. The output errs by the sum of these times sum p |v|, plus its rounding.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def kda():
    import chunked_gated_delta_10_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    m.build()
    m.load()
    return m


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rel(x, ref):
    return float((x.double().cpu() - ref).norm() / ref.norm().clamp_min(1e-300))


# ------------------------------------------------------------------ step


def step_inputs(seed, N, T, H, HV, K, V, dtype, slots=None):
    gen = _gen(seed)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    dt = DT[dtype]
    return dict(q=unit(rnd(N, T, H, K)).to(dt), k=unit(rnd(N, T, H, K)).to(dt), v=rnd(N, T, HV, V).to(dt),
                g=torch.nn.functional.logsigmoid(rnd(N, T, HV, K) + 3), beta=torch.sigmoid(rnd(N, T, HV)).to(dt),
                state=rnd(slots or N, HV, K, V))


def step_ref(x, scale, slots=None):
    """Token by token, head by head, as the recurrence is written: S <- (I - beta k k^T) Diag(e^g) S + beta k v^T."""
    q, k, v, g, beta, state = (x[n].double() for n in ("q", "k", "v", "g", "beta", "state"))
    state = state.clone()
    N, T, HV, V = v.shape
    rep = HV // q.shape[2]
    o = torch.zeros(N, T, HV, V, dtype=torch.float64)
    for n in range(N):
        at = n if slots is None else int(slots[n])
        if not 0 <= at < state.shape[0]:
            continue
        for h in range(HV):
            S = state[at, h]
            for t in range(T):
                kt, b = k[n, t, h // rep], beta[n, t, h]
                S = g[n, t, h].exp()[:, None] * S
                S = S - b * torch.outer(kt, kt @ S) + b * torch.outer(kt, v[n, t, h])
                o[n, t, h] = scale * (q[n, t, h // rep] @ S)
            state[at, h] = S
    return o, state


def _cuda(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def run_step(kda, x, **kw):
    y = _cuda(x)
    o = kda.step(y["q"], y["k"], y["v"], y["g"], y["beta"], y["state"], **kw)
    torch.cuda.synchronize()
    return o, y["state"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,T,H,HV,K,V", [(1, 1, 1, 1, 128, 128), (3, 1, 2, 6, 64, 128), (2, 4, 3, 3, 128, 64),
                                          (5, 7, 2, 4, 64, 64), (1, 33, 1, 2, 128, 128), (40, 1, 4, 8, 128, 128),
                                          (160, 2, 1, 1, 128, 64)])
def test_step(kda, N, T, H, HV, K, V, dtype):
    x = step_inputs(N * 100 + T, N, T, H, HV, K, V, dtype)
    o, state = run_step(kda, x)
    ro, rs = step_ref(x, K ** -0.5)
    tol = 4 * T * (K + 10) * U
    assert _rel(state, rs) <= tol
    assert _rel(o, ro) <= tol * math.sqrt(K) + ROUND[dtype]
    again = run_step(kda, x)
    assert torch.equal(o, again[0]) and torch.equal(state, again[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_step_tokens_one_by_one(kda, dtype):
    """Several tokens in a call are the same tokens in as many calls, bit for bit."""
    x = step_inputs(5, 3, 6, 2, 4, 128, 64, dtype)
    o, state = run_step(kda, x, scale=0.3)
    y = _cuda(x)
    for t in range(6):
        one = [y[n][:, t:t + 1].contiguous() for n in ("q", "k", "v", "g", "beta")]
        ot = kda.step(*one, y["state"], scale=0.3)
        assert torch.equal(ot[:, 0], o[:, t])
    assert torch.equal(y["state"], state)


def test_step_slots(kda):
    """Slots in any order, inactive rows, and a slot that does not exist: states that no row names stay as they are."""
    x = step_inputs(6, 5, 2, 2, 2, 64, 64, "bf16", slots=7)
    slots = torch.tensor([6, -1, 0, 7, 3], dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((5, 2, 2, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    o, state = run_step(kda, x, slots=slots.cuda(), status=status, out=out)
    ro, rs = step_ref(x, 64 ** -0.5, slots)
    assert o is out and int(status) == 1
    assert not o[1].any() and not o[3].any()
    assert _rel(o, ro) <= 2e-3 and _rel(state, rs) <= 8 * 74 * U
    for idle in (1, 2, 4, 5):
        assert torch.equal(state[idle].cpu(), x["state"][idle])
    status.zero_()
    run_step(kda, x, slots=torch.tensor([6, -1, 0, -5, 3], dtype=torch.int32).cuda(), status=status)
    assert int(status) == 0


def test_step_continues_the_chunked_forward(kda):
    """A prompt through chunk_fwd, then tokens one at a time on its ht: the chunked forward of the whole sequence."""
    import kda_inputs
    inp = kda_inputs.small(seed=3, B=2, T=75, H=2, HV=4, K=128, V=128, dtype="bf16", dht=False)
    y = {n: getattr(inp, n).cuda() for n in ("q", "k", "v", "g", "beta", "h0")}
    cut = lambda a, b: [y[n][:, a:b].contiguous() for n in ("q", "k", "v", "g", "beta")]  # noqa: E731
    whole, end, _ = kda.chunk_fwd(*cut(0, 75), scale=inp.scale, h0=y["h0"])
    _, state, _ = kda.chunk_fwd(*cut(0, 70), scale=inp.scale, h0=y["h0"])
    last = torch.cat([kda.step(*cut(t, t + 1), state, scale=inp.scale) for t in range(70, 75)], 1)
    # both sides are within the framework's bf16 tolerance of the exact result
    assert _rel(last, whole[:, 70:].double().cpu()) <= 1e-2
    assert _rel(state, end.double().cpu()) <= 1e-2


def test_step_extremes(kda):
    """Gates of 0 and -inf (keep all, forget all), beta 0 and 1, on states that hold large values."""
    x = step_inputs(9, 2, 1, 1, 1, 64, 64, "f32")
    x["g"][0], x["g"][1] = 0.0, -math.inf
    x["beta"][0], x["beta"][1] = 0.0, 1.0
    x["state"] *= 1e18
    o, state = run_step(kda, x)
    assert torch.equal(state[0].cpu(), x["state"][0])
    want = torch.outer(x["k"][1, 0, 0], x["v"][1, 0, 0])
    assert _rel(state[1, 0], want.double()) <= 4 * 74 * U
    assert torch.isfinite(o).all()


# ------------------------------------------------------------------ the paged cache


def make_cache(gen, pages, size, heads, K, V, dtype, layout):
    """A cache of random values in one of the layouts that strides can say (CPU tensors)."""
    dt = DT[dtype]
    rnd = lambda *s: torch.randn(*s, generator=gen).to(dt)  # noqa: E731
    if layout == "heads first":
        return rnd(pages, heads, size, K).transpose(1, 2), rnd(pages, heads, size, V).transpose(1, 2)
    if layout == "rows first":
        return rnd(pages, size, heads, K), rnd(pages, size, heads, V)
    pool = rnd(pages, size, heads, K + V + 8)  # keys and values side by side, with a gap
    return pool[..., :K], pool[..., K:K + V]


def to_gpu(t):
    """The same strides on the GPU: the storage goes over as it is."""
    base = torch.empty(0, dtype=t.dtype).set_(t.untyped_storage())
    return base.cuda().as_strided(t.shape, t.stride(), t.storage_offset())


def make_table(gen, reach, size, pages, spare=1):
    """Scattered pages for sequences that reach these many rows; -1 behind them."""
    need = [-(-max(int(x), 0) // size) for x in reach]
    order = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((len(need), max(need + [0]) + spare), -1, dtype=torch.int32)
    for n, m in enumerate(need):
        for j in range(m):
            table[n, j] = order.pop()
    return table


def turn(x, pos, rope, interleaved):
    """The rotation in 64 bits, pair by pair, and the magnitude that its error goes by."""
    y, size = x.double().clone(), x.double().abs()
    if rope is None:
        return y, 0 * size
    half = rope.shape[1] // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = rope[pos, i].double()[:, None], rope[pos, half + i].double()[:, None]
        p, q = x[..., a].double(), x[..., b].double()
        y[..., a], y[..., b] = p * c - q * s, p * s + q * c
        size[..., a], size[..., b] = (p * c).abs() + (q * s).abs(), (p * s).abs() + (q * c).abs()
    size[..., 2 * half:] = 0
    return y, size


def rope_table(positions, dim):
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(dim // 2) / (dim / 2))
    return torch.cat([angle.cos(), angle.sin()], 1).float()


APPENDS = [
    # lens, new rows, HQ, HKV, K, V, page, rot, interleaved, layout
    ([0], [1], 1, 1, 64, 64, 1, 0, False, "heads first"),
    ([5, 0, 63], [1, 1, 1], 8, 2, 128, 128, 64, 128, False, "heads first"),
    ([17, 0, 3, 9], [13, 0, 1, 200], 6, 2, 128, 64, 27, 64, False, "rows first"),
    ([17, 0, 3, 9], [130, 1, 0, 20], 5, 5, 64, 128, 16, 64, True, "shared pool"),
    ([0, 1000], [3, 5], 40, 8, 128, 128, 7, 32, True, "rows first"),
    ([2] * 70, [1] * 70, 16, 1, 64, 64, 100, 16, False, "shared pool"),
    ([300], [1500], 2, 2, 128, 128, 64, 96, False, "heads first"),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append(kda, case, dtype):
    lens, rows, HQ, HKV, K, V, size, rot, inter, layout = APPENDS[case]
    gen, dt = _gen(case), DT[dtype]
    reach = [a + b for a, b in zip(lens, rows)]
    pages = sum(-(-x // size) for x in reach) + 2
    kc, vc = make_cache(gen, pages, size, HKV, K, V, dtype, layout)
    table = make_table(gen, reach, size, pages)
    R = sum(rows)
    joint = torch.randn(R, (HQ + HKV) * K + HKV * V, generator=gen).to(dt)  # one projection's rows: strides apart
    q, k, v = joint.split([HQ * K, HKV * K, HKV * V], 1)
    q, k, v = q.unflatten(1, (HQ, K)), k.unflatten(1, (HKV, K)), v.unflatten(1, (HKV, V))
    rope = rope_table(max(reach), rot) if rot else None
    even = len(set(rows)) == 1
    cu = torch.tensor([0] + rows).cumsum(0)
    g = joint.cuda()
    gq, gk, gv = g.split([HQ * K, HKV * K, HKV * V], 1)
    gkc, gvc = to_gpu(kc), to_gpu(vc)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for use_cu in ([True, False] if even else [True]):
        out = kda.cache_append(gk.unflatten(1, (HKV, K)), gv.unflatten(1, (HKV, V)), gkc, gvc, table.cuda(),
                               torch.tensor(lens, dtype=torch.int32).cuda(), q=gq.unflatten(1, (HQ, K)),
                               rope=None if rope is None else rope.cuda(), interleaved=inter,
                               cu_seqlens=cu.cuda() if use_cu else None, status=status)
        assert int(status) == 0
        pos = torch.cat([torch.arange(a, a + b) for a, b in zip(lens, rows)])
        n = torch.repeat_interleave(torch.arange(len(rows)), torch.tensor(rows))
        wq, size_q = turn(q, pos, rope, inter)
        wk, size_k = turn(k, pos, rope, inter)
        bound = lambda want, mag: (3 * U * mag + ROUND[dtype] * want.abs() * (mag > 0)) * 1.01  # noqa: E731
        assert ((out.double().cpu() - wq).abs() <= bound(wq, size_q)).all()
        page = table[n, pos // size].long()
        got = gkc.cpu()[page, pos % size]
        assert ((got.double() - wk).abs() <= bound(wk, size_k)).all()
        assert torch.equal(gvc.cpu()[page, pos % size], v)
        # everything else is untouched
        for now, before in ((gkc.cpu(), kc), (gvc.cpu(), vc)):
            keep = torch.ones(pages, size, dtype=torch.bool)
            keep[page, pos % size] = False
            assert torch.equal(now[keep], before[keep])


def test_append_without_queries_and_in_place(kda):
    gen = _gen(1)
    k, v, q = (torch.randn(4, 2, 64, generator=gen).bfloat16().cuda() for _ in range(3))
    rope, lens = rope_table(40, 64).cuda(), torch.tensor([30, 3], dtype=torch.int32).cuda()
    table = torch.tensor([[0, 1, 2], [3, -1, -1]], dtype=torch.int32).cuda()
    caches = []
    for with_q in (False, True):
        kc, vc = kda.new_cache(4, 16, 2, 64, 64)
        out = kda.cache_append(k, v, kc, vc, table, lens, q=q.clone() if with_q else None, rope=rope)
        assert (out is not None) == with_q
        caches.append((kc, vc))
    assert torch.equal(caches[0][0], caches[1][0]) and torch.equal(caches[0][1], caches[1][1])
    same = q.clone()
    assert kda.cache_append(k, v, *caches[0], table, lens, q=same, rope=rope, q_out=same) is same
    assert torch.equal(same, out)


def test_append_drops_what_has_no_place(kda):
    """Inactive sequences silently; pages that do not exist and positions beyond the table or the rotation flagged."""
    gen = _gen(2)
    size, HKV, K = 8, 2, 64
    k, v, q = (torch.randn(6, HKV, K, generator=gen).bfloat16().cuda() for _ in range(3))
    table = torch.tensor([[0, 1], [2, -1], [3, 9], [4, 5], [6, 7], [1, 2]], dtype=torch.int32).cuda()
    lens = torch.tensor([-1, 8, 9, 16, 12, 3], dtype=torch.int32).cuda()  # row 5 alone has a place
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rope = rope_table(12, 32).cuda()  # positions 0 .. 11
    before = [torch.randn(9, size, HKV, K, generator=gen).bfloat16().cuda() for _ in range(2)]
    for who, flag in (([0], 0), ([1], 1), ([2], 1), ([3], 1), ([4], 1), ([5], 0), ([0, 1, 2, 3, 4, 5], 1)):
        kc, vc = (t.clone() for t in before)
        status.zero_()
        out = kda.cache_append(k[who], v[who], kc, vc, table[who], lens[who], q=q[who], rope=rope, status=status)
        assert int(status) == flag
        for i, n in enumerate(who):
            assert bool(out[i].any()) == (n == 5)
        changed = [int((a != b).flatten(1).any(1).sum()) for a, b in zip((kc, vc), before)]
        assert changed == ([1, 1] if 5 in who else [0, 0])
        if 5 in who:
            assert torch.equal(vc[1, 3], v[5])


def attend_ref(q, kc, vc, table, lens, scale, window, size):
    """Row by row in 64 bits: o, lse, and the bounds of their errors (that of o before its rounding)."""
    pair = 2.0 ** -16 if kc.dtype == torch.bfloat16 else 0.0
    N, HQ, K = q.shape
    HKV, V, pages = kc.shape[2], vc.shape[3], kc.shape[0]
    o, lse = torch.zeros(N, HQ, V, dtype=torch.float64), torch.full((N, HQ), -math.inf, dtype=torch.float64)
    err, err_lse = torch.zeros(N, HQ, V, dtype=torch.float64), torch.zeros(N, HQ, dtype=torch.float64)
    for n in range(N):
        end = int(lens[n])
        begin = max(0, end - window) if window else 0
        pos = torch.arange(begin, max(begin, min(end, table.shape[1] * size)))
        page = table[n, pos // size].long()
        pos, page = pos[(page >= 0) & (page < pages)], page[(page >= 0) & (page < pages)]
        if not len(pos):
            continue
        for h in range(HQ):
            j = h // (HQ // HKV)
            kk, vv, qq = kc[page, pos % size, j].double(), vc[page, pos % size, j].double(), q[n, h].double()
            s = scale * (kk @ qq)
            p = torch.softmax(s, 0)
            o[n, h], lse[n, h] = p @ vv, torch.logsumexp(s, 0)
            ds = float((scale * (kk.abs() @ qq.abs())).max()) * (K + 4) * 2 * U
            w = 2 * ds + 2.0 ** -20 + pair + 2 * (len(pos) + 16) * U
            err[n, h] = w * (p @ vv.abs())
            err_lse[n, h] = w + 4 * U * (abs(float(lse[n, h])) + 1)
    return o, lse, err, err_lse


ATTENDS = [
    # lens, HQ, HKV, K, V, page, window, layout
    ([1], 1, 1, 64, 64, 1, 0, "heads first"),
    ([0, 1, 2, 15, 16, 17, 63, 64, 65], 4, 2, 128, 128, 16, 0, "heads first"),
    ([300, 0, 1, 129], 5, 1, 128, 64, 27, 0, "rows first"),
    ([700, 33], 16, 2, 64, 128, 64, 0, "shared pool"),
    ([513, 1025, 7], 12, 4, 128, 128, 100, 0, "rows first"),
    ([900, 100, 0, 40], 8, 8, 64, 64, 20, 129, "shared pool"),
    ([70, 2, 1], 3, 3, 128, 128, 5, 1, "heads first"),
    ([400, 250], 20, 1, 128, 128, 32, 250, "heads first"),
    ([5000], 32, 1, 64, 64, 16, 0, "rows first"),
    ([6000], 2, 1, 128, 128, 64, 0, "heads first"),
    ([40] * 90, 4, 4, 64, 128, 16, 0, "heads first"),
    ([3000, 1, 2999], 6, 2, 128, 128, 128, 2000, "shared pool"),
]


def run_attend(kda, q, kc, vc, table, lens, **kw):
    o, lse = kda.cache_attend(q.cuda(), kc if kc.is_cuda else to_gpu(kc), vc if vc.is_cuda else to_gpu(vc), table.cuda(),
                              torch.as_tensor(lens, dtype=torch.int32).cuda(), **kw)
    torch.cuda.synchronize()
    return o, lse


def check_attend(dtype, got, ref):
    (o, lse), (ro, rl, err, err_lse) = got, ref
    assert ((o.double().cpu() - ro).abs() <= 1.01 * (err + ROUND[dtype] * ro.abs())).all()
    some = rl > -math.inf
    assert ((lse.double().cpu() - rl).abs()[some] <= err_lse[some]).all()
    assert (lse.cpu()[~some] == -math.inf).all() and not o.cpu()[~some].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(ATTENDS)))
def test_attend(kda, case, dtype):
    lens, HQ, HKV, K, V, size, window, layout = ATTENDS[case]
    gen = _gen(case)
    pages = sum(-(-x // size) for x in lens) + 2
    kc, vc = make_cache(gen, pages, size, HKV, K, V, dtype, layout)
    table = make_table(gen, lens, size, pages)
    # whatever no sequence owns holds NaN: the rows behind each length and the free pages
    own = torch.zeros(pages, size, dtype=torch.bool)
    for n, m in enumerate(lens):
        pos = torch.arange(max(0, m - window) if window else 0, m)
        own[table[n, pos // size].long(), pos % size] = True
    kc[~own], vc[~own] = math.nan, math.nan
    q = (2 * torch.randn(len(lens), HQ + 3, K, generator=gen)).to(DT[dtype])[:, 2:-1]  # rows apart
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_attend(kda, q, kc, vc, table, lens, window=window, status=status)
    assert int(status) == 0
    check_attend(dtype, got, attend_ref(q, kc, vc, table, lens, K ** -0.5, window, size))
    again = run_attend(kda, q, kc, vc, table, lens, window=window)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_sharp_and_flat(kda, dtype):
    """One row that outweighs all others (at either end), scores far from 0, and equal scores."""
    gen, dt = _gen(7), DT[dtype]
    kc, vc = make_cache(gen, 40, 16, 1, 64, 64, dtype, "heads first")
    table = torch.arange(40, dtype=torch.int32)[None]
    q = torch.randn(1, 4, 64, generator=gen).to(dt)
    for at, factor in ((0, 40.0), (638, 40.0), (300, -40.0)):
        kd = kc.clone()
        kd[at // 16, at % 16] = (factor * q[0, 0]).to(dt)
        check_attend(dtype, run_attend(kda, q, kd, vc, table, [639]),
                     attend_ref(q, kd, vc, table, [639], 0.125, 0, 16))
    check_attend(dtype, run_attend(kda, q, 0 * kc, vc, table, [639]),
                 attend_ref(q, 0 * kc, vc, table, [639], 0.125, 0, 16))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_infinities(kda, dtype):
    """Rows whose score is -inf weigh nothing; where all are -inf nothing is left; a NaN in the range comes out."""
    gen, dt = _gen(8), DT[dtype]
    kc, vc = make_cache(gen, 8, 16, 1, 64, 64, dtype, "rows first")
    table = torch.arange(8, dtype=torch.int32)[None]
    q = torch.randn(1, 2, 64, generator=gen).abs().to(dt)
    kd = kc.clone()
    kd[2:4, :, :, 0] = -math.inf
    ref = attend_ref(q, torch.cat([kc[:2], kc[4:]]), torch.cat([vc[:2], vc[4:]]), table[:, :6], [96], 0.125, 0, 16)
    check_attend(dtype, run_attend(kda, q, kd, vc, table, [128]), ref)
    kd[..., 0] = -math.inf
    o, lse = run_attend(kda, q, kd, vc, table, [100])
    assert not o.any() and (lse == -math.inf).all()
    kd = kc.clone()
    kd[0, 0, 0, 3] = math.nan
    o, lse = run_attend(kda, q, kd, vc, table, [100])
    assert torch.isnan(o).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_leaves_out_what_does_not_exist(kda, dtype):
    gen = _gen(9)
    size = 16
    kc, vc = make_cache(gen, 6, size, 2, 64, 64, dtype, "heads first")
    q = torch.randn(3, 4, 64, generator=gen).to(DT[dtype])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, 6, 1], [2, 3, 4], [5, -7, 0]], dtype=torch.int32)
    for lens, flag in (([16, 48, 16], 0), ([48, 48, 16], 1), ([0, 49, 0], 1), ([16, 2 ** 31 - 1, 40], 1), ([-3, -1, 5], 0)):
        status.zero_()
        got = run_attend(kda, q, kc, vc, table, lens, status=status)
        assert int(status) == flag
        check_attend(dtype, got, attend_ref(q, kc, vc, table, lens, 0.125, 0, size))


def test_attend_without_pages(kda):
    q = torch.randn(2, 4, 64).bfloat16()
    kc, vc = kda.new_cache(1, 16, 2, 64, 64)
    o, lse = run_attend(kda, q, kc, vc, torch.zeros(2, 0, dtype=torch.int32), [0, 0])
    assert not o.any() and (lse == -math.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cache_beyond_32_bits(kda, dtype):
    """Pages whose offset in the pool passes 2^32 elements."""
    gen, dt, K, size = _gen(10), DT[dtype], 128, 64
    stride = 1 << 26  # elements from page to page
    pool = torch.empty(66 * stride, dtype=dt, device="cuda")
    kc = pool.as_strided((66, size, 1, K), (stride, K, K, 1))
    vc = pool.as_strided((66, size, 1, K), (stride, K, K, 1), 2 * size * K)
    table = torch.tensor([[65, 0, 64]], dtype=torch.int32)
    k, v = (torch.randn(150, 1, K, generator=gen).to(dt) for _ in range(2))
    kda.cache_append(k.cuda(), v.cuda(), kc, vc, table.cuda(), torch.zeros(1, dtype=torch.int32).cuda())
    q = torch.randn(1, 4, K, generator=gen).to(dt)
    got = run_attend(kda, q, kc, vc, table, [150])
    pad = torch.zeros(42, 1, K, dtype=dt)
    flat = lambda x: torch.cat([x, pad]).view(3, size, 1, K)  # noqa: E731
    check_attend(dtype, got, attend_ref(q, flat(k), flat(v), torch.tensor([[0, 1, 2]]), [150], K ** -0.5, 0, size))


def test_on_another_stream(kda):
    """The kernels run on the current stream: work queued there before and after them is in order with them."""
    gen = _gen(11)
    side = torch.cuda.Stream()
    kc, vc = kda.new_cache(64, 16, 2, 128, 128)
    table = torch.randperm(64, generator=gen)[None].to(torch.int32).cuda()
    rows = [torch.randn(1000, 2, 128, generator=gen).bfloat16() for _ in range(2)]
    q = torch.randn(1, 8, 128, generator=gen).bfloat16().cuda()
    pinned = [t.pin_memory() for t in rows]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        k, v = (t.cuda(non_blocking=True) for t in pinned)
        kda.cache_append(k, v, kc, vc, table, torch.zeros(1, dtype=torch.int32, device="cuda"))
        o, _ = kda.cache_attend(q, kc, vc, table, torch.full((1,), 1000, dtype=torch.int32, device="cuda"))
        o = o + 0
    side.synchronize()
    flat = lambda x: torch.cat([x, x[:24]]).view(64, 16, 2, 128)  # noqa: E731
    ref = attend_ref(q.cpu(), flat(rows[0]), flat(rows[1]), torch.arange(64)[None], [1000], 128 ** -0.5, 0, 16)
    assert ((o.double().cpu() - ref[0]).abs() <= 1.01 * (ref[2] + ROUND["bf16"] * ref[0].abs())).all()


def test_in_a_graph(kda):
    """A captured step of all three operators replays on new contents of the same buffers."""
    gen = _gen(12)
    x = {n: t.cuda() for n, t in step_inputs(12, 2, 1, 2, 2, 64, 64, "bf16").items()}
    kc, vc = kda.new_cache(8, 16, 2, 64, 64)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn(2, 2, 64, generator=gen).bfloat16().cuda() for _ in range(3))
    rope = rope_table(64, 64).cuda()

    def token():
        kda.step(x["q"], x["k"], x["v"], x["g"], x["beta"], x["state"])
        turned = kda.cache_append(k, v, kc, vc, table, lens, q=q, rope=rope)
        lens.add_(1)
        return kda.cache_attend(turned, kc, vc, table, lens)[0]

    start = x["state"].clone()
    want = [token().clone() for _ in range(20)]
    end = x["state"].clone()
    lens.zero_()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        o = token()
    x["state"].copy_(start)
    lens.zero_()
    for w in want:
        graph.replay()
        assert torch.equal(o, w)
    assert torch.equal(x["state"], end)
