"""The paged cache in 8 bits on the GPU, against plain implementations in 64 bits.

Bounds, with u = 2^-24 (fp32), 2^-8 (bf16) and 2^-4 (e4m3, or 2^-10 of the scale below its normal values):

* append: x c - y s in fp32, each product and sum rounded: 3 u (|x c| + |y s|), then one rounding to e4m3. Values that are
  not rotated have exactly one result. A scale is exact unless the block's largest value is that near to a power of two
  times 448.
* attend: a score errs by (K + 4) 2u scale sum |q k| (a tensor core may truncate: 2u), and by 2^-23 of that more where the
  query is two fp16 values, and 4 u of itself for its factors; a weight by twice the largest score error, 2^-20 for the
  exponential, 2^-22 for its two fp16 parts and 2 u for the factors; the sum over n rows by 2 (n + 16) u. The output errs
  by the sum of these times sum p |v|, by 2^-35 of the largest p |sv| times sum |v8|, plus its rounding.
"""
import math

import pytest
import torch

from tests.test_gpu_serve import DT, ROUND, U, _gen, kda, make_table, rope_table, to_gpu, turn  # noqa: F401
from tests.test_gpu_serve_sinks import visible

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def make_cache8(gen, pages, size, heads, K, V, block, layout="heads first", spread=3):
    """Random values and scales (CPU): e4m3 values over their range, scales around 2^-7, not powers of two alone."""
    out = []
    for d in (K, V):
        x = (torch.randn(pages, heads, size, d, generator=gen) * 110).clamp(-448, 448).to(E4M3)
        s = torch.exp2(torch.randn(pages, heads, size // block, generator=gen) * spread - 7)
        s = torch.where(torch.rand(s.shape, generator=gen) < 0.5, torch.exp2(torch.log2(s).round()), s).float()
        if layout == "heads first":
            x, s = x.transpose(1, 2), s.transpose(1, 2)
        else:
            x, s = (t.transpose(1, 2).contiguous() for t in (x, s))
        out.append((x, s))
    if layout == "shared pool":  # keys and values side by side, with a gap; scales likewise
        pool = torch.zeros(pages, size, heads, K + V + 16, dtype=torch.uint8)
        pool[..., :K], pool[..., K:K + V] = out[0][0].view(torch.uint8), out[1][0].view(torch.uint8)
        scales = torch.stack([out[0][1], out[1][1]], -1)
        return pool[..., :K].view(E4M3), pool[..., K:K + V].view(E4M3), scales[..., 0], scales[..., 1]
    return out[0][0], out[1][0], out[0][1], out[1][1]


def gpu8(t):
    return to_gpu(t.view(torch.uint8)).view(E4M3) if t.dtype == E4M3 else to_gpu(t)


def bits(t):
    """What can be compared as it is: the bytes of 8-bit values."""
    return t.view(torch.uint8) if t.dtype == E4M3 else t


def least(top):
    """The smallest power of two, 2^-126 at least, by which `top` comes to 448 at most."""
    if top == 0:
        return 2.0 ** -126
    e = math.ceil(math.log2(top / 448))
    while top <= 448 * 2.0 ** (e - 1):
        e -= 1
    while top > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** max(e, -126)


def held(s):
    """The smallest power of two that is not below a scale's magnitude (0 where it says nothing; 2^126 at most)."""
    s = abs(s)
    return 0.0 if s == 0 or not math.isfinite(s) else 2.0 ** min(max(math.ceil(math.log2(s)), -126), 126)


def check_append8(new, mag, pos, n, lens, table, size, block, before, after):
    """new: the rows' values in 64 bits [R, H, D]; mag: what their error goes by; before, after: (values, scales), CPU."""
    (c0, s0), (c1, s1) = before, after
    f0, f1 = c0.float(), c1.float()  # (8-bit tensors are not indexed on every CPU)
    untouched = torch.ones(c0.shape[:2], dtype=torch.bool)
    idle = torch.ones(s0.shape[:2], dtype=torch.bool)
    blocks = {}
    for r in range(len(pos)):
        p = int(table[n[r], int(pos[r]) // size])
        blocks.setdefault((p, int(pos[r]) % size // block, int(n[r])), []).append(r)
    for (p, b, i), rows in blocks.items():
        start = int(pos[rows[0]]) // block * block  # the block's first position
        old = list(range(start, min(int(lens[i]), start + block)))
        idle[p, b] = False
        for t in old:
            untouched[p, t % size] = False
        for r in rows:
            untouched[p, int(pos[r]) % size] = False
        for h in range(new.shape[1]):
            x, m = new[rows, h], mag[rows, h]
            fine = torch.where(torch.isfinite(x), x.abs(), 0)
            top, slack = float(fine.max()), float((3.01 * U * m[torch.isfinite(x)]).max()) if torch.isfinite(x).any() else 0.0
            was = float(s0[p, b, h]) if old else 0.0
            want = {max(least(v), held(was)) for v in (max(top - slack, 0.0), top, top + slack)}
            now = float(s1[p, b, h])
            assert now in want, (now, want)
            got = f1[[p] * len(rows), [int(pos[r]) % size for r in rows], h].double()
            gone = ~torch.isfinite(x)
            assert torch.equal(torch.isnan(got), gone)
            err = torch.maximum(2.0 ** -4 * x.abs(), torch.tensor(2.0 ** -10 * now)) + 4 * U * m
            assert ((got * now - x).abs() <= 1.0001 * err)[~gone].all()
            if not m.any():
                assert torch.equal(got[~gone], (x.float() / now).to(E4M3).double()[~gone])
            for t in old:
                was_row, now_row = f0[p, t % size, h], f1[p, t % size, h]
                if now == was:
                    assert torch.equal(was_row.nan_to_num(999), now_row.nan_to_num(999))
                else:
                    again = (was_row * (torch.tensor(was) / now)).to(E4M3)
                    assert torch.equal(again.float().nan_to_num(999), now_row.nan_to_num(999))
    assert torch.equal(c1.view(torch.uint8)[untouched], c0.view(torch.uint8)[untouched])
    assert torch.equal(s1[idle], s0[idle])


APPENDS = [
    # lens, new rows, HQ, HKV, K, V, page, block, rot, interleaved, layout
    ([0], [1], 1, 1, 64, 64, 1, 1, 0, False, "heads first"),
    ([5, 0, 63], [1, 1, 1], 8, 2, 128, 128, 64, 16, 128, False, "heads first"),
    ([17, 0, 3, 9], [13, 0, 1, 200], 6, 2, 128, 64, 27, 9, 64, False, "rows first"),
    ([17, 0, 3, 9], [130, 1, 0, 20], 5, 5, 64, 128, 16, 16, 64, True, "shared pool"),
    ([0, 1000], [3, 5], 40, 8, 128, 128, 7, 7, 32, True, "rows first"),
    ([2] * 70, [1] * 70, 16, 1, 64, 64, 100, 50, 16, False, "shared pool"),
    ([300], [700], 2, 2, 128, 128, 64, 64, 96, False, "heads first"),
    ([31, 1], [450, 33], 3, 1, 64, 128, 200, 100, 16, True, "rows first"),
    ([8, 7, 0, 0], [8, 9, 0, 1], 2, 2, 64, 64, 8, 1, 64, False, "heads first"),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append8(kda, case, dtype):  # noqa: F811
    lens, rows, HQ, HKV, K, V, size, block, rot, inter, layout = APPENDS[case]
    gen, dt = _gen(case), DT[dtype]
    reach = [a + b for a, b in zip(lens, rows)]
    pages = sum(-(-x // size) for x in reach) + 2
    cache = make_cache8(gen, pages, size, HKV, K, V, block, layout)
    table = make_table(gen, reach, size, pages)
    R = sum(rows)
    big = torch.exp2(torch.randint(-6, 4, (R, 1), generator=gen))  # rows of different size: scales that have to grow
    joint = (torch.randn(R, (HQ + HKV) * K + HKV * V, generator=gen) * big).to(dt)
    q, k, v = joint.split([HQ * K, HKV * K, HKV * V], 1)
    q, k, v = q.unflatten(1, (HQ, K)), k.unflatten(1, (HKV, K)), v.unflatten(1, (HKV, V))
    rope = rope_table(max(reach), rot) if rot else None
    even = len(set(rows)) == 1
    cu = torch.tensor([0] + rows).cumsum(0)
    g = joint.cuda()
    gq, gk, gv = g.split([HQ * K, HKV * K, HKV * V], 1)
    pos = torch.cat([torch.arange(a, a + b) for a, b in zip(lens, rows)])
    n = torch.repeat_interleave(torch.arange(len(rows)), torch.tensor(rows))
    wq, size_q = turn(q, pos, rope, inter)
    wk, size_k = turn(k, pos, rope, inter)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    seen = []
    for use_cu in ([True, False] if even else [True]):
        kc, vc, ks, vs = (gpu8(t) for t in cache)
        out = kda.cache_append(gk.unflatten(1, (HKV, K)), gv.unflatten(1, (HKV, V)), kc, vc, table.cuda(),
                               torch.tensor(lens, dtype=torch.int32).cuda(), q=gq.unflatten(1, (HQ, K)),
                               rope=None if rope is None else rope.cuda(), interleaved=inter,
                               cu_seqlens=cu.cuda() if use_cu else None, status=status, k_scale=ks, v_scale=vs)
        assert int(status) == 0
        bound = (3 * U * size_q + ROUND[dtype] * wq.abs() * (size_q > 0)) * 1.01
        assert ((out.double().cpu() - wq).abs() <= bound).all()
        check_append8(wk, size_k, pos, n, lens, table, size, block, (cache[0], cache[2]), (kc.cpu(), ks.cpu()))
        check_append8(v.double(), 0 * v.double(), pos, n, lens, table, size, block, (cache[1], cache[3]), (vc.cpu(), vs.cpu()))
        seen.append((out, kc, vc, ks, vs))
    for a, b in zip(seen[0], seen[-1]):
        assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N, T", [(3, 40), (50, 1)])
def test_append8_rounds_each_product_and_sum(kda, N, T, dtype, interleaved):  # noqa: F811
    """Keys are what separate products and sums in fp32 make of them, in every bit: the scales do not hang on a compiler."""
    gen, size, H, K = _gen(6), 16, 4, 128
    x = torch.randn(N * T, H, K, generator=gen).to(DT[dtype])
    rope = rope_table(T + 9, K)
    lens = torch.randint(0, 9, (N,), generator=gen).to(torch.int32)
    width = -(-(T + 9) // size)
    table = torch.randperm(N * width, generator=gen).to(torch.int32).view(N, width)
    kc, vc, ks, vs = kda.new_cache(N * width, size, H, K, K, dtype=E4M3, scale_block=1)
    q = kda.cache_append(x.cuda(), x.cuda(), kc, vc, table.cuda(), lens.cuda(), q=x.cuda(), rope=rope.cuda(),
                         interleaved=interleaved, k_scale=ks, v_scale=vs)
    n = torch.arange(N).repeat_interleave(T)
    pos = lens.long()[n] + torch.arange(T).repeat(N)
    c, s = (t[:, None] for t in rope[pos].chunk(2, 1))
    f = x.float()
    a, b = (f[..., ::2], f[..., 1::2]) if interleaved else f.chunk(2, -1)
    ac, bs, bc, as_ = a * c, b * s, b * c, a * s
    u, v = ac - bs, bc + as_
    want = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    assert torch.equal(q.cpu(), want.to(DT[dtype]))
    at, row = table[n, pos // size].long(), pos % size
    scale = torch.tensor([least(float(t)) for t in want.abs().amax(-1).flatten()]).view(N * T, H)
    assert torch.equal(ks.cpu()[at, row], scale)
    assert torch.equal(kc.float().cpu()[at, row], (want / scale[..., None]).to(E4M3).float())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [4, 16, 64])
def test_append8_values(kda, block, dtype):  # noqa: F811
    """Zeros, the smallest and largest values, infinities and NaN, values at the border of a scale; then rows that are
    larger, smaller or not finite, one by one."""
    dt, size, D = DT[dtype], 64, 64
    tiny, huge = (2.0 ** -133, 3.38e38) if dtype == "bf16" else (2.0 ** -149, 3.4e38)
    levels = [0.0, tiny, 2.0 ** -126, 448 * 2.0 ** -126, 450 * 2.0 ** -126, 1e-30, 1.0, 3.5, 3.515625, 448.0, 1e30, huge, 0.0, 2.0]
    gen = _gen(3)
    new = torch.stack([torch.rand(1, D, generator=gen) * 2 - 1 for _ in levels]).double() * torch.tensor(levels).double()[:, None, None]
    new[:, 0, 0] = torch.tensor(levels).double()  # the largest of each row
    new[6, 0, 5], new[6, 0, 6], new[7, 0, 7] = math.inf, -math.inf, math.nan
    new = new.to(dt).double()
    new[12] = math.inf
    cache = make_cache8(gen, 2, size, 1, D, D, block)
    table = torch.tensor([[1]], dtype=torch.int32)
    R = len(levels)
    for together in (True, False):
        kc, vc, ks, vs = (gpu8(t) for t in cache)
        x = new.to(dt).cuda()
        for a, b in ([(0, R)] if together else [(i, i + 1) for i in range(R)]):
            was = [t.cpu().clone() for t in (kc, ks, vc, vs)]
            kda.cache_append(x[a:b], x[a:b], kc, vc, table.cuda(), torch.tensor([a], dtype=torch.int32).cuda(), k_scale=ks,
                             v_scale=vs)
            pos, n = torch.arange(a, b), torch.zeros(b - a, dtype=torch.int64)
            for c, s, c0, s0 in ((kc, ks, *was[:2]), (vc, vs, *was[2:])):
                check_append8(new[a:b], 0 * new[a:b].nan_to_num(0, 0, 0), pos, n, [a], table, size, block, (c0, s0),
                              (c.cpu(), s.cpu()))


def test_append8_onto_scales_of_other_kinds(kda):  # noqa: F811
    """Old scales that are not powers of two, negative, 0, infinite or NaN: the rows stand for what they stood for."""
    gen, size, D = _gen(4), 16, 64
    old = [0.3, -0.3, 0.0, math.inf, math.nan, -2.0, 2.0 ** -126, float(torch.tensor(3e38))]
    kc, vc, ks, vs = make_cache8(gen, len(old), size, 1, D, D, size)
    ks[:, 0, 0], vs[:, 0, 0] = torch.tensor(old), torch.tensor(old)
    table, lens = torch.arange(len(old), dtype=torch.int32)[:, None], torch.full((len(old),), 9, dtype=torch.int32)
    x = torch.randn(len(old), 1, D, generator=gen).bfloat16()
    g = [gpu8(t) for t in (kc, vc, ks, vs)]
    kda.cache_append(x.cuda(), x.cuda(), g[0], g[1], table.cuda(), lens.cuda(), k_scale=g[2], v_scale=g[3])
    for c0, s0, c1, s1 in ((kc, ks, g[0].cpu(), g[2].cpu()), (vc, vs, g[1].cpu(), g[3].cpu())):
        for n, s in enumerate(old):
            now, top = float(s1[n, 0, 0]), float(x[n].abs().max())
            assert now == max(least(top), held(s))
            assert torch.equal(c1[n, 9].double(), (x[n].float() / now).to(E4M3).double())
            stood = c0[n, :9].double() * s
            stands = c1[n, :9].double() * now
            fits = torch.isfinite(stood) & (stood.abs() <= 448 * now)  # (3e38 lies above the largest scale, 2^126)
            assert torch.equal(torch.isnan(stands), ~fits) and (fits.all() or not 0 < abs(s) < 1e38)
            err = torch.maximum(2.0 ** -4 * stood.abs(), torch.tensor(2.0 ** -10 * now))
            assert ((stands - stood).abs() <= err)[fits].all()


def test_append8_drops_what_has_no_place(kda):  # noqa: F811
    """As a cache in 16 bits does: inactive sequences silently, what does not exist flagged; scales stay with their rows."""
    gen, size, HKV, K = _gen(2), 8, 2, 64
    k, v, q = (torch.randn(6, HKV, K, generator=gen).bfloat16().cuda() for _ in range(3))
    table = torch.tensor([[0, 1], [2, -1], [3, 9], [4, 5], [6, 7], [1, 2]], dtype=torch.int32).cuda()
    lens = torch.tensor([-1, 8, 9, 16, 12, 3], dtype=torch.int32).cuda()  # row 5 alone has a place
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rope = rope_table(12, 32).cuda()
    before = [gpu8(t) for t in make_cache8(gen, 9, size, HKV, K, K, 4)]
    for who, flag in (([0], 0), ([1], 1), ([2], 1), ([3], 1), ([4], 1), ([5], 0), ([0, 1, 2, 3, 4, 5], 1)):
        for with_q in (True, False):
            kc, vc, ks, vs = (t.clone() for t in before)
            status.zero_()
            out = kda.cache_append(k[who], v[who], kc, vc, table[who], lens[who], q=q[who] if with_q else None, rope=rope,
                                   status=status, k_scale=ks, v_scale=vs)
            assert int(status) == flag
            if with_q:
                for i, n in enumerate(who):
                    assert bool(out[i].any()) == (n == 5)
            for a, b in zip((kc, vc, ks, vs), before):
                rows = (bits(a) != bits(b)).flatten(2).any(2).nonzero().tolist()
                assert set(map(tuple, rows)) <= ({(1, r) for r in range(4)} if 5 in who else set())
            assert bool((bits(vc) != bits(before[1])).any()) == (5 in who)


def test_append8_rows_of_no_sequence(kda):  # noqa: F811
    """cu_seqlens that leave rows out, or do not rise: flagged, and nothing is written for those rows."""
    gen = _gen(5)
    x = torch.randn(20, 1, 64, generator=gen).bfloat16().cuda()
    table = torch.arange(6, dtype=torch.int32).view(3, 2).cuda()
    lens = torch.tensor([3, 0, 5], dtype=torch.int32).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for cu, flag in (([0, 4, 9, 20], 0), ([0, 4, 9, 15], 1), ([2, 4, 9, 20], 1), ([0, 4, 4, 20], 0), ([0, 9, 4, 20], 1),
                     ([0, 4, 9, 25], 1), ([-5, 4, 9, 20], 1), ([0, 4, 2 ** 40, 20], 1)):
        kc, vc, ks, vs = kda.new_cache(6, 16, 1, 64, 64, dtype=E4M3)
        status.zero_()
        q = kda.cache_append(x, x, kc, vc, table, lens, q=x, cu_seqlens=torch.tensor(cu).cuda(), status=status, k_scale=ks,
                             v_scale=vs)
        assert int(status) == flag, cu
        if cu == [0, 4, 9, 15]:
            assert not q[15:].any() and q[:15].flatten(1).any(1).all()
            assert int((kc.float() != 0).flatten(2).any(2).sum()) == 15


# ------------------------------------------------------------------ attention


def attend8_ref(q, kc, vc, ks, vs, table, lens, scale, window, sinks):
    """Row by row in 64 bits: o, lse, and the bounds of their errors (that of o before its rounding)."""
    more = 2.0 ** -23 if q.dtype == torch.float32 else 0.0
    N, HQ, K = q.shape
    pages, size, HKV, V = vc.shape
    block = size // ks.shape[1]
    kc, vc = kc.float(), vc.float()
    o, lse = torch.zeros(N, HQ, V, dtype=torch.float64), torch.full((N, HQ), -math.inf, dtype=torch.float64)
    err, err_lse = torch.zeros(N, HQ, V, dtype=torch.float64), torch.zeros(N, HQ, dtype=torch.float64)
    for n in range(N):
        pos = visible(int(lens[n]), window, sinks)
        pos = pos[pos < table.shape[1] * size]
        page = table[n, pos // size].long()
        pos, page = pos[(page >= 0) & (page < pages)], page[(page >= 0) & (page < pages)]
        if not len(pos):
            continue
        for j in range(HKV):
            kk = kc[page, pos % size, j].double() * ks[page, pos % size // block, j].double()[:, None]
            v8, sv = vc[page, pos % size, j].double(), vs[page, pos % size // block, j].double()
            vv = v8 * sv[:, None]
            for h in range(j * HQ // HKV, (j + 1) * HQ // HKV):
                qq = q[n, h].double()
                s = scale * (kk @ qq)
                p = torch.softmax(s, 0)
                o[n, h], lse[n, h] = p @ vv, torch.logsumexp(s, 0)
                ds = float((scale * (kk.abs() @ qq.abs())).max()) * ((K + 4) * 2 * U + more) + 4 * U * float(s.abs().max())
                w = 2 * ds + 2.0 ** -20 + 2.0 ** -22 + 2 * U + 2 * (len(pos) + 16) * U
                err[n, h] = w * (p @ vv.abs()) + 2.0 ** -35 * float((p * sv.abs()).max()) * v8.abs().sum(0)
                err_lse[n, h] = w + 4 * U * (abs(float(lse[n, h])) + 1)
    return o, lse, err, err_lse


def run8(kda, q, cache, table, lens, **kw):  # noqa: F811
    kc, vc, ks, vs = (t if t.is_cuda else gpu8(t) for t in cache)
    o, lse = kda.cache_attend(q.cuda(), kc, vc, table.cuda(), torch.as_tensor(lens, dtype=torch.int32).cuda(), k_scale=ks,
                              v_scale=vs, **kw)
    torch.cuda.synchronize()
    return o, lse


def check8(dtype, got, ref):
    (o, lse), (ro, rl, err, err_lse) = got, ref
    assert o.dtype == DT[dtype]
    assert ((o.double().cpu() - ro).abs() <= 1.01 * (err + ROUND[dtype] * ro.abs())).all()
    some = rl > -math.inf
    assert ((lse.double().cpu() - rl).abs()[some] <= err_lse[some]).all()
    assert (lse.cpu()[~some] == -math.inf).all() and not o.cpu()[~some].any()


ATTENDS = [
    # lens, HQ, HKV, K, V, page, block, window, sinks, layout
    ([1], 1, 1, 64, 64, 1, 1, 0, 0, "heads first"),
    ([0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65], 4, 2, 128, 128, 16, 4, 0, 0, "heads first"),
    ([300, 0, 1, 129], 5, 1, 128, 64, 27, 9, 0, 0, "rows first"),
    ([700, 33], 16, 2, 64, 128, 64, 64, 0, 0, "shared pool"),
    ([513, 1025, 7], 12, 4, 128, 128, 100, 20, 0, 0, "rows first"),
    ([900, 100, 0, 40], 8, 8, 64, 64, 20, 1, 129, 6, "shared pool"),
    ([70, 2, 1], 3, 3, 128, 128, 5, 5, 1, 0, "heads first"),
    ([400, 250], 20, 1, 128, 128, 32, 16, 250, 33, "heads first"),
    ([5000], 32, 1, 64, 64, 16, 16, 0, 0, "rows first"),
    ([9000], 16, 1, 128, 128, 64, 64, 0, 0, "heads first"),
    ([6000], 2, 1, 128, 128, 64, 8, 0, 0, "heads first"),
    ([40] * 90, 4, 4, 64, 128, 16, 16, 0, 0, "heads first"),
    ([3000, 1, 2999], 6, 2, 128, 64, 128, 32, 2000, 100, "shared pool"),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(ATTENDS)))
def test_attend8(kda, case, dtype):  # noqa: F811
    lens, HQ, HKV, K, V, size, block, window, sinks, layout = ATTENDS[case]
    gen = _gen(case)
    pages = sum(-(-x // size) for x in lens) + 2
    kc, vc, ks, vs = make_cache8(gen, pages, size, HKV, K, V, block, layout)
    table = make_table(gen, lens, size, pages)
    # whatever is not visible holds NaN: rows, and scales of blocks without a visible row
    own, alive = torch.zeros(pages, size, dtype=torch.bool), torch.zeros(ks.shape[:2], dtype=torch.bool)
    for n, m in enumerate(lens):
        pos = visible(m, window, sinks)
        own[table[n, pos // size].long(), pos % size] = True
        alive[table[n, pos // size].long(), pos % size // block] = True
    for c in (kc, vc):
        c.view(torch.uint8)[~own] = 0x7F
    ks[~alive], vs[~alive] = math.nan, math.nan
    q = (2 * torch.randn(len(lens), HQ + 3, K, generator=gen)).to(DT[dtype])[:, 2:-1]  # rows apart
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run8(kda, q, (kc, vc, ks, vs), table, lens, window=window, sinks=sinks, status=status)
    assert int(status) == 0
    check8(dtype, got, attend8_ref(q, kc, vc, ks, vs, table, lens, K ** -0.5, window, sinks))
    again = run8(kda, q, (kc, vc, ks, vs), table, lens, window=window, sinks=sinks)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("split, N, L, heads, group", [
    ("cache8_attend", 300, 100, 2, 2), ("cache8_attend_cluster", 2, 2000, 2, 2), ("cache8_attend_parts", 1, 30000, 2, 2),
    # shares of all heads of a sequence together, and of some; of tiles of query heads; of one alone
    ("cache8_attend_shares", 48, 6000, 8, 2), ("cache8_attend_shares", 90, 3000, 5, 1), ("cache8_attend_shares", 70, 3000, 7, 12),
    ("cache8_attend_shares", 40, 3000, 3, 40), ("cache8_attend_shares", 12, 5000, 50, 1), ("cache8_attend_shares", 450, 5000, 1, 3)])
def test_attend8_of_each_split(kda, split, N, L, heads, group, dtype):  # noqa: F811
    gen, size, D, some = _gen(7), 20, 64, 4
    width = -(-L // size)
    cache = make_cache8(gen, some * width, size, heads, D, D, 10)
    table = (torch.arange(N)[:, None] % some * width + torch.arange(width)).to(torch.int32)
    lens = [(L, 0, L // 2 + 1, L - 7)[n % 4] for n in range(N)]
    q = torch.randn(some, group * heads, D, generator=gen).to(DT[dtype])
    got = run8(kda, q[torch.arange(N) % some], cache, table, lens)
    assert kda.load().kda_launch_name(0).decode() == split
    few = list(range(min(N, some)))
    ref = attend8_ref(q[few], *cache, table[few], lens, D ** -0.5, 0, 0)
    check8(dtype, (got[0][few], got[1][few]), ref)
    for n in range(N):  # (the others differ in how their rows were shared out alone)
        i = n % some
        assert ((got[0][n].double().cpu() - ref[0][i]).abs() <= 1.01 * (ref[2][i] + ROUND[dtype] * ref[0][i].abs())).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("split, N, L, heads, window, sinks", [
    ("cache8_attend", 300, 300, 2, 70, 20), ("cache8_attend_cluster", 2, 4000, 2, 1500, 100),
    ("cache8_attend_parts", 1, 60000, 2, 25000, 1001), ("cache8_attend_shares", 60, 9000, 8, 5000, 70)])
def test_attend8_sinks_of_each_split(kda, split, N, L, heads, window, sinks, dtype):  # noqa: F811
    """First rows that end inside a tile, a turn, a block and a page; lengths at which they and the window meet."""
    gen, size, D, some = _gen(13), 27, 64, 4
    width = -(-L // size)
    cache = make_cache8(gen, some * width, size, heads, D, D, 9)
    table = (torch.arange(N)[:, None] % some * width + torch.arange(width)).to(torch.int32)
    lens = [(L, window + sinks, window + sinks // 2, L - 77)[n % 4] for n in range(N)]
    q = torch.randn(some, 2 * heads, D, generator=gen).to(DT[dtype])
    got = run8(kda, q[torch.arange(N) % some], cache, table, lens, window=window, sinks=sinks)
    assert kda.load().kda_launch_name(0).decode() == split
    few = list(range(min(N, some)))
    ref = attend8_ref(q[few], *cache, table[few], lens, D ** -0.5, window, sinks)
    check8(dtype, (got[0][few], got[1][few]), ref)
    for n in range(N):
        i = n % some
        assert ((got[0][n].double().cpu() - ref[0][i]).abs() <= 1.01 * (ref[2][i] + ROUND[dtype] * ref[0][i].abs())).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend8_scales(kda, dtype):  # noqa: F811
    """Scales of V that differ by many powers of two and signs, in an order that makes the greatest come last or first;
    zero blocks of the smallest scale; scales of K that take scores far from 0; large and small queries."""
    gen, size, D, blocks = _gen(8), 16, 64, 24
    table, lens = torch.arange(blocks, dtype=torch.int32)[None], [size * blocks - 3]
    kc, vc, ks, vs = make_cache8(gen, blocks, size, 1, D, D, size)
    q = torch.randn(1, 3, D, generator=gen).to(DT[dtype])
    up = torch.arange(blocks).double()[:, None, None]
    for powers in (3 * up - 40, 40 - 3 * up, 0 * up - 126, 0 * up + 100, 5 * (up % 7) - 126, 4 * up, 0 * up - 60):
        vd = torch.exp2(powers).float() * torch.where(up % 3 == 1, -1.0, 1.0)
        check8(dtype, run8(kda, q, (kc, vc, ks, vd.float()), table, lens),
               attend8_ref(q, kc, vc, ks, vd.float(), table, lens, 0.125, 0, 0))
    zero = vc.clone()
    zero.view(torch.uint8)[::2] = 0
    vd = torch.where(up % 2 == 0, 2.0 ** -126, 0.01).float()
    check8(dtype, run8(kda, q, (kc, zero, ks, vd), table, lens), attend8_ref(q, kc, zero, ks, vd, table, lens, 0.125, 0, 0))
    for factor in (30.0, -30.0, 1e-12, 1e12, 1e-30):
        kd, qd = (ks * factor).float(), q
        if factor in (1e-12, 1e12, 1e-30):
            qd = (q.double() / factor).to(DT[dtype])  # the same scores, of another query
        check8(dtype, run8(kda, qd, (kc, vc, kd, vs), table, lens), attend8_ref(qd, kc, vc, kd, vs, table, lens, 0.125, 0, 0))
    # scores that are all below the least exponent of fp32, the greatest of them at the end
    kd, q1 = torch.full_like(ks, -1.0), torch.zeros_like(q)
    q1[..., 0] = 1.0
    k1 = kc.clone()
    k1.view(torch.uint8)[..., 0] = torch.linspace(448, 200, blocks)[:, None, None].to(E4M3).view(torch.uint8)
    check8(dtype, run8(kda, q1, (k1, vc, kd, vs), table, lens, scale=1.0), attend8_ref(q1, k1, vc, kd, vs, table, lens, 1.0, 0, 0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend8_that_is_not_finite(kda, dtype):  # noqa: F811
    """A NaN value of V makes its channel NaN, one of K, or a NaN scale in the range, its heads; an infinite query does
    what the sum says."""
    gen, size, D = _gen(9), 16, 64
    table = torch.arange(8, dtype=torch.int32)[None]
    kc, vc, ks, vs = make_cache8(gen, 8, size, 2, D, D, 4)
    q = torch.randn(1, 4, D, generator=gen).to(DT[dtype])
    vd = vc.clone()
    vd.view(torch.uint8)[3, 5, 1, 7], vd.view(torch.uint8)[0, 0, 0, 63] = 0x7F, 0xFF
    o, lse = run8(kda, q, (kc, vd, ks, vs), table, [120])
    bad = torch.zeros(1, 4, D, dtype=torch.bool)
    bad[0, 2:, 7], bad[0, :2, 63] = True, True
    assert torch.equal(torch.isnan(o).cpu(), bad) and torch.isfinite(lse).all()
    whole = run8(kda, q, (kc, vc, ks, vs), table, [120])
    assert torch.equal(o.cpu()[~bad], whole[0].cpu()[~bad])
    kd = kc.clone()
    kd.view(torch.uint8)[3, 5, 1, 7] = 0x7F
    o, lse = run8(kda, q, (kd, vc, ks, vs), table, [120])
    assert torch.isnan(o[:, 2:]).all() and torch.isnan(lse[:, 2:]).all()
    assert torch.equal(o[:, :2], whole[0][:, :2]) and torch.equal(lse[:, :2], whole[1][:, :2])
    for which in (0, 1):
        sd = [ks.clone(), vs.clone()]
        sd[which][7, 1, 0] = math.nan
        o, lse = run8(kda, q, (kc, vc, *sd), table, [120])
        assert torch.isnan(o[:, :2]).all() and torch.equal(o[:, 2:], whole[0][:, 2:])
        assert torch.isnan(lse[:, :2]).all() == (which == 0)
    qd = q.clone()
    qd[0, 0, 3], qd[0, 1, 4] = math.inf, math.nan
    o, lse = run8(kda, qd, (kc, vc, ks, vs), table, [120])
    assert torch.isnan(o[:, :2]).all() and torch.equal(o[:, 2:], whole[0][:, 2:])
    one = kc.clone()
    one.view(torch.uint8)[..., 3] = torch.tensor(-2.0).to(E4M3).view(torch.uint8)
    o, lse = run8(kda, qd[:, :1].expand(1, 2, D).contiguous(), (one[:, :, :1], vc[:, :, :1], ks[:, :, :1].abs(), vs[:, :, :1]), table, [120])
    assert not o.any() and (lse == -math.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend8_leaves_out_what_does_not_exist(kda, dtype):  # noqa: F811
    gen, size = _gen(10), 16
    cache = make_cache8(gen, 6, size, 2, 64, 64, 8)
    q = torch.randn(3, 4, 64, generator=gen).to(DT[dtype])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, 6, 1], [2, 3, 4], [5, -7, 0]], dtype=torch.int32)
    for lens, flag in (([16, 48, 16], 0), ([48, 48, 16], 1), ([0, 49, 0], 1), ([16, 2 ** 31 - 1, 40], 1), ([-3, -1, 5], 0)):
        status.zero_()
        got = run8(kda, q, cache, table, lens, status=status)
        assert int(status) == flag
        check8(dtype, got, attend8_ref(q, *cache, table, lens, 0.125, 0, 0))


def test_cache8_beyond_32_bits(kda):  # noqa: F811
    """Pages whose offset in the pool passes 2^32 bytes."""
    gen, K, size, stride = _gen(11), 128, 64, 1 << 26
    pool = torch.empty(66 * stride, dtype=torch.uint8, device="cuda")
    kc = pool.as_strided((66, size, 1, K), (stride, K, K, 1)).view(E4M3)
    vc = pool.as_strided((66, size, 1, K), (stride, K, K, 1), 2 * size * K).view(E4M3)
    ks, vs = (torch.zeros(66, 4, 1, device="cuda") for _ in range(2))
    table = torch.tensor([[65, 0, 64]], dtype=torch.int32)
    k, v = (torch.randn(150, 1, K, generator=gen).bfloat16() for _ in range(2))
    kda.cache_append(k.cuda(), v.cuda(), kc, vc, table.cuda(), torch.zeros(1, dtype=torch.int32).cuda(), k_scale=ks, v_scale=vs)
    q = torch.randn(1, 4, K, generator=gen).bfloat16()
    got = run8(kda, q, (kc, vc, ks, vs), table, [150])
    order = table[0].long().cuda()
    rows = lambda c: c.view(torch.uint8)[order].cpu().view(E4M3).float()  # noqa: E731
    ref = attend8_ref(q, rows(kc), rows(vc), ks[order].cpu(), vs[order].cpu(), torch.tensor([[0, 1, 2]]), [150], K ** -0.5, 0, 0)
    check8("bf16", got, ref)
    flat = lambda c, s: (rows(c).double() * s[order].cpu().double().repeat_interleave(16, 1)[..., None]).flatten(0, 1)[:150]  # noqa: E731
    for x, c, s in ((k, kc, ks), (v, vc, vs)):
        assert ((flat(c, s) - x.double()).abs() <= 2.0 ** -4 * x.double().abs() + 2.0 ** -10 * s.max().item()).all()


def test_cache8_calls_refuse(kda):  # noqa: F811
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    kc, vc, ks, vs = kda.new_cache(6, 16, 2, 64, 128, dtype=E4M3, scale_block=4)
    assert ks.shape == vs.shape == (6, 4, 2) and kc.dtype == E4M3
    assert kda.new_cache(2, 27, 1, 64, 64, dtype=E4M3)[2].shape == (2, 1, 1)
    table, lens = z(3, 2, dt=torch.int32), z(3, dt=torch.int32)
    append = lambda **c: kda.cache_append(**{**dict(k=z(3, 2, 64), v=z(3, 2, 128), k_cache=kc, v_cache=vc,  # noqa: E731
                                                    page_table=table, kv_lens=lens, k_scale=ks, v_scale=vs), **c})
    attend = lambda **c: kda.cache_attend(**{**dict(q=z(3, 4, 64), k_cache=kc, v_cache=vc, page_table=table,  # noqa: E731
                                                    kv_lens=lens, k_scale=ks, v_scale=vs), **c})
    assert append() is None and attend()[0].shape == (3, 4, 128)
    f = torch.float32
    both = [dict(v_cache=z(6, 16, 2, 128)), dict(k_scale=z(6, 4, 2)), dict(k_scale=z(6, 3, 2, dt=f)), dict(v_scale=z(5, 4, 2, dt=f)),
            dict(v_scale=z(6, 4, 1, dt=f)), dict(v_scale=z(6, 2, 2, dt=f)), dict(k_scale=ks.cpu()), dict(k_scale=z(6, 4, dt=f)),
            dict(k_scale=z(6, 0, 2, dt=f))]
    for bad in both + [dict(k=z(3, 2, 64, dt=f)), dict(q=z(3, 4, 64, dt=f)), dict(q=z(3, 4, 64), q_out=z(3, 4, 64, dt=f))]:
        with pytest.raises(ValueError):
            append(**bad)
    for bad in both + [dict(q=z(2, 4, 64)), dict(out=z(3, 4, 128, dt=f))]:
        with pytest.raises(ValueError):
            attend(**bad)
    for call in (append, attend):
        for bad in (dict(k_scale=None), dict(v_scale=None)):
            with pytest.raises(TypeError):
                call(**bad)
    with pytest.raises(TypeError):
        attend(q=z(3, 4, 64, dt=torch.float16))
    with pytest.raises(TypeError):
        attend(q=z(3, 4, 64).to(E4M3))
    with pytest.raises(ValueError, match="float8"):
        k16, v16 = kda.new_cache(6, 16, 2, 64, 128)
        attend(k_cache=k16, v_cache=v16)
    for bad in (dict(k_scale=z(6, 1, 1, dt=f).expand(6, 4, 2)), dict(v_scale=z(1, 4, 2, dt=f).expand(6, 4, 2))):
        with pytest.raises(kda.KdaError, match="KDA_ERR_INVALID_ARG"):  # blocks that share a scale
            append(**bad)
        attend(**bad)
    with pytest.raises(kda.KdaError, match="KDA_ERR_INVALID_ARG"):
        attend(sinks=-1)
    for bad in (dict(scale_block=5), dict(scale_block=-4), dict(dtype=torch.bfloat16, scale_block=4)):
        with pytest.raises(ValueError):
            kda.new_cache(**{**dict(num_pages=2, page_size=16, heads=1, K=64, V=64, dtype=E4M3), **bad})
    need = kda.cache_attend_workspace_bytes(z(3, 4, 64), kc, vc, table)
    out, ws = z(3, 4, 128), z(need, dt=torch.uint8)
    assert attend(out=out, ws=ws)[0] is out


def test_cache8_in_a_graph(kda):  # noqa: F811
    """A captured token's append and attention replay on new contents of the same buffers, while blocks fill up and their
    scales grow."""
    gen = _gen(12)
    kc, vc, ks, vs = kda.new_cache(8, 16, 2, 64, 64, dtype=E4M3, scale_block=8)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    rope = rope_table(64, 64).cuda()
    rows = [[torch.randn(2, 2, 64, generator=gen).bfloat16().cuda() * 2.0 ** (t % 5) for _ in range(3)] for t in range(40)]
    buf = [torch.zeros_like(x) for x in rows[0]]

    def token():
        turned = kda.cache_append(buf[1], buf[2], kc, vc, table, lens, q=buf[0], rope=rope, k_scale=ks, v_scale=vs)
        lens.add_(1)
        return kda.cache_attend(turned, kc, vc, table, lens, k_scale=ks, v_scale=vs, window=20, sinks=3)[0]

    def run(step):
        lens.zero_()
        out = []
        for r in rows:
            for b, x in zip(buf, r):
                b.copy_(x)
            out.append(step().clone())
        return out

    want = run(token)
    state = [bits(t).clone() for t in (kc, vc, ks, vs)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        o = token()

    def replay():
        graph.replay()
        return o

    for a, b in zip(want, run(replay)):
        assert torch.equal(a, b)
    for a, t in zip(state, (kc, vc, ks, vs)):
        assert torch.equal(a, bits(t))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("where", ["all", "first", "every other", "some heads", "keys"])
@pytest.mark.parametrize("split, N, L, heads, group", [
    ("cache8_attend", 300, 600, 2, 2), ("cache8_attend_cluster", 3, 3000, 4, 2), ("cache8_attend_parts", 1, 60000, 2, 2),
    ("cache8_attend_shares", 48, 6000, 8, 2), ("cache8_attend", 300, 600, 2, 12)])
def test_attend8_scales_of_zero(kda, split, N, L, heads, group, where, dtype):  # noqa: F811
    """Blocks whose scale is 0, as of values that are all 0: of V for all rows, the first ones, every other block or one
    head, and of K. Scores are whole multiples of 2.5 (log2 units) that go up and down from 32 rows to the next, so that
    some rows weigh four to eight times the largest before them."""
    gen, size, D, some, block = _gen(14), 20, 64, 2, 10
    width = -(-L // size)
    kc, vc, ks, vs = make_cache8(gen, some * width, size, heads, D, D, block)
    kc.view(torch.uint8)[:] = 0
    at = (torch.arange(some * width)[:, None] % width * size + torch.arange(size)) // 32  # the 32 rows of a row
    steps = torch.randint(0, 2, (some * width, heads), generator=gen)[at].float()  # [pages, rows, heads]
    kc.view(torch.uint8)[..., 0] = steps.to(E4M3).view(torch.uint8)
    ks.fill_(1.0)
    number = torch.arange(some * width)[:, None] % width * (size // block) + torch.arange(size // block)  # of a block
    if where == "all":
        vs.zero_()
    elif where == "first":
        vs[number < width * (size // block) // 2] = 0.0
    elif where == "every other":
        vs[number % 2 == 0] = 0.0
    elif where == "some heads":
        vs[..., ::2] = 0.0
    else:
        ks[number % 3 > 0] = 0.0
        vs[number % 2 == 0] = 0.0
    table = (torch.arange(N)[:, None] % some * width + torch.arange(width)).to(torch.int32)
    q = torch.zeros(some, group * heads, D)
    q[..., 0] = 1.0
    q[..., 1:] = torch.randn(some, group * heads, D - 1, generator=gen)  # (of keys that are 0)
    q, scale, lens = q.to(DT[dtype]), 2.5 * math.log(2), [L if n % some == 0 else L - 45 for n in range(N)]
    got = run8(kda, q[torch.arange(N) % some], (kc, vc, ks, vs), table, lens, scale=scale)
    assert kda.load().kda_launch_name(0).decode() == split
    few = list(range(min(N, some)))
    ref = attend8_ref(q[few], kc, vc, ks, vs, table[few], lens, scale, 0, 0)
    check8(dtype, (got[0][few], got[1][few]), ref)
    for n in range(N):
        assert ((got[0][n].double().cpu() - ref[0][n % some]).abs() <= 1.01 * (ref[2][n % some] + ROUND[dtype] * ref[0][n % some].abs())).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("split, N, L, heads, group", [
    ("cache8_attend", 300, 600, 2, 2), ("cache8_attend_cluster", 3, 3000, 4, 2), ("cache8_attend_parts", 1, 30000, 2, 2),
    ("cache8_attend_shares", 48, 6000, 8, 2), ("cache8_attend", 300, 600, 2, 12)])
def test_attend8_infinite_scales(kda, split, N, L, heads, group, dtype):  # noqa: F811
    """A block of V whose scale is infinite makes its head's channels infinite, of the sign of its values (NaN where one of
    them is 0, or where they have both signs); the other heads are as without it."""
    gen, size, D, some, block = _gen(15), 20, 64, 2, 10
    width = -(-L // size)
    kc, vc, ks, vs = make_cache8(gen, some * width, size, heads, D, D, block, spread=0)
    table = (torch.arange(N)[:, None] % some * width + torch.arange(width)).to(torch.int32)
    lens = [L - 45 * (n % some) for n in range(N)]
    q = torch.randn(some, group * heads, D, generator=gen).to(DT[dtype])
    every = torch.arange(N) % some
    whole = run8(kda, q[every], (kc, vc, ks, vs), table, lens)
    at = [n * width + width // 3 for n in range(some)]
    vc, vs = vc.clone(), vs.clone()
    for n, p in enumerate(at):
        rows = vc[p, :block, 1].float().abs().clamp_min(1.0) * torch.where(torch.arange(D) % 3 == n, -1.0, 1.0)
        rows[2, 5], rows[3, 6] = 0.0, -rows[4, 6]
        vc.view(torch.uint8)[p, :block, 1] = rows.to(E4M3).view(torch.uint8)
        vs[p, 0, 1] = math.inf if n == 0 else -math.inf
    o, lse = run8(kda, q[every], (kc, vc, ks, vs), table, lens)
    assert kda.load().kda_launch_name(0).decode() == split
    sign = torch.stack([torch.where(torch.arange(D) % 3 == n, -math.inf, math.inf) * (1 - 2 * n) for n in range(some)])
    sign[:, 5:7] = math.nan
    mine = slice(group, 2 * group)
    want = sign[every][:, None, :].expand(N, group, D)
    assert torch.equal(o[:, mine].float().cpu().nan_to_num(9.0, 1.0, -1.0), want.nan_to_num(9.0, 1.0, -1.0))
    assert torch.equal(lse, whole[1])
    for others in (slice(0, group), slice(2 * group, None)):
        assert torch.equal(o[:, others], whole[0][:, others])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("power", [20, 24, 26, 40, 100, -40])
def test_attend8_far_scores_and_large_scales(kda, power, dtype):  # noqa: F811
    """Scores so far from 0 that fp32 holds them in steps of more than one, of which one row's is above all others, and
    scales of V that are large or small: o is that row's value, in an order of rows that has it come last, or that raises
    the maximum with every 32 rows before it."""
    gen, size, D, rows = _gen(17), 16, 64, 1280
    table = torch.arange(rows // size, dtype=torch.int32)[None]
    kc, vc, ks, vs = make_cache8(gen, rows // size, size, 1, D, D, size, spread=0)
    q = torch.zeros(1, 3, D)
    q[..., 0] = 1.0
    q = q.to(DT[dtype])
    for order in (torch.zeros(rows // 32), torch.arange(rows // 32) / 8, torch.linspace(-7, -1, rows // 32)):
        for best in (5, rows - 7):
            k = kc.clone()
            k.view(torch.uint8)[:] = 0
            x = order.repeat_interleave(32).clamp(max=7)
            x[best] = 16.0
            k.view(torch.uint8)[..., 0, 0] = x.to(E4M3).view(torch.uint8).view(rows // size, size)
            for scale_of_v in (1.0, 2.0 ** 20, -(2.0 ** 90), 2.0 ** -60):
                sv = torch.full_like(vs, scale_of_v)
                kd = torch.full_like(ks, 2.0 ** power)
                o, lse = run8(kda, q, (k, vc, kd, sv), table, [rows], scale=1.0)
                ref = attend8_ref(q, k, vc, kd, sv, table, [rows], 1.0, 0, 0)
                if power > 0:  # (the other rows weigh nothing: e to the power of -2^20 and less)
                    want = vc.float().flatten(0, 1)[best, 0].double() * scale_of_v
                    assert torch.equal(ref[0][0, 0], want)
                    err = (2.0 ** -21 + ROUND[dtype]) * want.abs() + 2.0 ** -34 * abs(scale_of_v) * 448
                    assert ((o.double().cpu() - want).abs() <= err).all(), (order[-1], best, scale_of_v)
                    assert ((lse.double().cpu() - ref[1]).abs() <= 4 * U * ref[1].abs()).all()
                else:
                    check8(dtype, (o, lse), ref)


@pytest.mark.parametrize("times, block", [(1, 4), (1, 16), (5, 4), (5, 16)])
def test_append8_offsets_and_queries_agree(kda, times, block):  # noqa: F811
    """Whatever cu_seqlens holds, a row's queries are 0 where the row is not appended, and there alone; where offsets end
    beyond the rows, those that there are are appended, as to a cache in 16 bits."""
    gen, R, pages = _gen(16), 20 * times, 8 * times
    x = torch.randn(R, 1, 64, generator=gen).bfloat16().cuda()
    table = torch.arange(3 * pages, dtype=torch.int32).view(3, pages).cuda()
    lens = torch.tensor([3, 0, 5], dtype=torch.int32).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    far = 2 ** 40
    for cu in ([0, 4, 9, 20], [0, 4, 9, 15], [2, 4, 9, 20], [0, 4, 4, 20], [0, 4, 9, 25], [-5, 4, 9, 20], [0, 4, far, 20],
               [0, 4, far, far], [-far, 4, 9, far], [-9, -5, 9, 20], [20, 20, 20, 20], [0, 0, 0, 0], [5, 5, 25, 30], [-4, -3, -2, -1],
               [22, 25, 25, 30]):
        cu = torch.tensor([c if abs(c) == far else c * times for c in cu])
        kc, vc, ks, vs = kda.new_cache(3 * pages, 16, 1, 64, 64, dtype=E4M3, scale_block=block)
        status.zero_()
        q = kda.cache_append(x, x, kc, vc, table, lens, q=x, cu_seqlens=cu.cuda(), status=status, k_scale=ks, v_scale=vs)
        good = cu[0] == 0 and cu[-1] == R and bool((cu[1:] >= cu[:-1]).all())
        assert bool(int(status)) != good, cu
        stands = (vc.float() * vs.repeat_interleave(block, 1)[..., None])[..., 0, :].flatten(0, 1).cpu()
        held = stands[stands.any(1)]
        there = [bool((held - row).abs().le(2.0 ** -4 * row.abs() + 2.0 ** -10 * vs.max().item()).all(1).any()) for row in x[:, 0].float().cpu()]
        assert [bool(y) for y in q.flatten(1).any(1)] == there, cu
        assert len(held) == sum(there), cu
        if cu.min() >= 0:
            k16, v16 = kda.new_cache(3 * pages, 16, 1, 64, 64)
            as16 = kda.cache_append(x, x, k16, v16, table, lens, q=x, cu_seqlens=cu.cuda())
            assert torch.equal(as16, q) and torch.equal(v16.float().any(-1), stands.view(3 * pages, 16, 1, 64).cuda().any(-1)), cu
