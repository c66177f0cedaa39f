"""Pages, appends and attention together, as a server calls them: sequences that come, grow and go, on one pool of pages."""
import importlib.util
import os

import pytest
import torch

from tests.test_gpu_serve import DT, _gen, attend_ref, check_attend, kda, rope_table  # noqa: F401
from tests.test_gpu_serve8 import E4M3, attend8_ref, bits, check8
from tests.test_gpu_serve_resize import resize_ref
from tests.test_gpu_serve_sinks import sinks_ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("pool", [60, 14, 8])
@pytest.mark.parametrize("window, sinks", [(0, 0), (20, 5)])
@pytest.mark.parametrize("kind, dtype", [("8", "bf16"), ("8", "f32"), ("16", "bf16"), ("32", "f32")])
def test_sequences_come_and_go(kda, kind, dtype, window, sinks, pool):  # noqa: F811
    """Every round some sequences end, others begin with a prompt or have one more token. Tables, lists and slots are those
    of the rules; each new row lies where its slot says; attention is that of the rows that the sequences hold. With few
    pages some sequences are not served in some rounds, and are tried again."""
    gen, dt, N, size, H, HQ, D, width = _gen(pool), DT[dtype], 5, 16, 2, 4, 64, 5
    cache = kda.new_cache(pool, size, H, D, D, dtype=E4M3 if kind == "8" else dt, **(dict(scale_block=8) if kind == "8" else {}))
    scales = dict(zip(("k_scale", "v_scale"), cache[2:]))
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    table, lens, new = i32(N, width) - 1, i32(N), i32(N)
    free, count, status = torch.randperm(pool, generator=gen).to(torch.int32).cuda(), i32(1) + pool, i32(1)
    rope = rope_table(width * size, D).cuda()
    held = [0] * N
    short = False
    for turn in range(25):
        wanted = []
        for n in held:
            what = int(torch.randint(0, 8, (1,), generator=gen))
            wanted.append(0 if n > 0 and what == 0 or n >= width * size else n + 1 if n else int(
                torch.randint(1, 50, (1,), generator=gen)) if what > 2 else -1)
        before = table.tolist(), free.tolist(), int(count)
        rows = sum(max(0, max(b, 0) - a) for a, b in zip(held, wanted))
        new.copy_(torch.tensor(wanted))
        cu, slots, granted = kda.cache_resize(table, lens, new, free, count, size, rows=rows, status=status)
        ref = resize_ref(before[0], held, wanted, before[1], before[2], size, rows)
        assert table.tolist() == ref[0] and slots.tolist() == ref[4] and granted.tolist() == ref[5] and int(count) == ref[2]
        assert bool(int(status)) == ref[6]
        short |= ref[6]
        used = [x for r in ref[0] for x in r if x >= 0] + ref[1][: ref[2]]
        assert sorted(used) == list(range(pool))  # every page has one place
        status.zero_()
        if rows:
            x = [torch.randn(rows, h, D, generator=gen).to(dt).cuda() * 2.0 ** float(torch.randn(1, generator=gen)) for h in (HQ, H, H)]
            q = kda.cache_append(x[1], x[2], *cache[:2], table, lens, q=x[0], rope=rope, cu_seqlens=cu, status=status, **scales)
            at = slots.long()
            there = at >= 0
            assert torch.equal(q.flatten(1).any(1), there) and bool(int(status)) == bool((~there).any())
            v = cache[1].float()[at[there] // size, at[there] % size]
            if kind == "8":
                s = cache[3][at[there] // size, at[there] % size // 8]
                v = v * s[..., None]
                w = x[2][there].float()
                assert ((v - w).abs() <= torch.maximum(2.0 ** -4 * w.abs(), 2.0 ** -10 * s[..., None])).all()
            else:
                assert torch.equal(v, x[2][there].float())
            status.zero_()
        lens.copy_(granted)
        held = [max(x, 0) for x in granted.tolist()]
        lens.clamp_(min=0)
        one = torch.randn(N, HQ, D, generator=gen).to(dt)
        got = kda.cache_attend(one.cuda(), *cache[:2], table, lens, window=window, sinks=sinks, status=status, **scales)
        assert int(status) == 0
        if kind == "8":
            back = [bits(t).cpu().view(t.dtype) for t in cache]
            check8(dtype, got, attend8_ref(one, *back, table.cpu(), held, D ** -0.5, window, sinks))
        else:
            check_attend(dtype, got, sinks_ref(one, cache[0].cpu(), cache[1].cpu(), table.cpu(), held, D ** -0.5, window, sinks, size))
    assert pool == 14 or short == (pool == 8)


@pytest.mark.parametrize("rows, block", [(1, 8), (13, 8), (27, 8), (300, 8), (300, 16), (27, 1)])
@pytest.mark.parametrize("kind, dtype", [("8", "bf16"), ("8", "f32"), ("16", "bf16"), ("32", "f32")])
def test_sequences_that_are_not_served_keep_their_cache(kda, kind, dtype, rows, block):  # noqa: F811
    """Sequences in the middle of a page that want more rows than there are pages for: with what was granted, an append of
    all rows changes nothing of theirs, though their last page has room, and its queries are 0 where slots are -1."""
    gen, dt, size, H, HQ, D, width = _gen(rows), DT[dtype], 16, 2, 4, 64, 40
    held, pool = [3, 19, 0, 40, 16, 8], 30
    cache = kda.new_cache(pool, size, H, D, D, dtype=E4M3 if kind == "8" else dt, **(dict(scale_block=block) if kind == "8" else {}))
    scales = dict(zip(("k_scale", "v_scale"), cache[2:]))
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    N = len(held)
    table, lens, new = i32(N, width) - 1, i32(N), i32(N)
    free, count, status = torch.randperm(pool, generator=gen).to(torch.int32).cuda(), i32(1) + pool, i32(1)
    rope = rope_table(width * size, D).cuda()
    draw = lambda n, h, big: (big * torch.randn(n, h, D, generator=gen)).to(dt).cuda()  # noqa: E731
    new.copy_(torch.tensor(held))
    cu, _, granted = kda.cache_resize(table, lens, new, free, count, size, status=status)
    kda.cache_append(draw(sum(held), H, 0.01), draw(sum(held), H, 0.01), *cache[:2], table, lens, cu_seqlens=cu, rope=rope,
                     granted=granted, status=status, **scales)
    lens.copy_(granted)
    assert int(status) == 0 and lens.tolist() == held
    # the first has its rows, the third nothing, the fourth one, the fifth has its own; the second and last want all
    wants = [held[0] + 2, held[1] + rows + 400, 0, held[3] + 1, held[4], held[5] + rows + 400]
    new.copy_(torch.tensor(wants))
    R = sum(b - a for a, b in zip(held, wants))
    before = [t.clone() for t in cache]
    cu, slots, granted = kda.cache_resize(table, lens, new, free, count, size, rows=R, status=status)
    assert granted.tolist() == [held[0] + 2, held[1], 0, held[3] + 1, held[4], held[5]] and int(status) != 0
    status.zero_()
    q = kda.cache_append(draw(R, H, 1000.0), draw(R, H, 1000.0), *cache[:2], table, lens, q=draw(R, HQ, 1.0), rope=rope, cu_seqlens=cu,
                         granted=granted, status=status, **scales)
    assert int(status) == 0
    assert torch.equal(q.flatten(1).any(1), slots >= 0) and int((slots >= 0).sum()) == 3
    for n in (1, 4, 5):
        for p in table[n][: -(-held[n] // size)].tolist():
            for a, b in zip(before, cache):
                assert torch.equal(bits(a[p]), bits(b[p])), n
    at = slots[slots >= 0]
    assert cache[1].float()[at // size, at % size].flatten(1).any(1).all()


@pytest.mark.parametrize("lengths", [[0, 5, 20, 7], [3, -4, 9, 70], [2 ** 31 - 1] * 4])
@pytest.mark.parametrize("T", [1, 6, 40])
@pytest.mark.parametrize("kind", ["8", "16"])
def test_rows_up_to_a_length(kda, kind, T, lengths):  # noqa: F811
    """Any granted lengths: rows below them lie in the cache as an append of those rows alone leaves them."""
    gen, N, size, H, D, width = _gen(T), 4, 16, 2, 64, 5
    held = [3, 0, 9, 7]
    cache = kda.new_cache(N * width, size, H, D, D, **(dict(dtype=E4M3, scale_block=4) if kind == "8" else {}))
    scales = dict(zip(("k_scale", "v_scale"), cache[2:]))
    table = torch.randperm(N * width, generator=gen).to(torch.int32).view(N, width).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    first = torch.randn(N * 9, H, D, generator=gen).bfloat16().cuda()
    kda.cache_append(first, first, *cache[:2], table, i32([0] * N), **scales)
    k, v, q = (4 * torch.randn(N * T, H, D, generator=gen).bfloat16().cuda() for _ in range(3))
    rope = rope_table(60, D).cuda()
    copies = [[t.clone() for t in cache] for _ in range(3)]
    outs = []
    for c, cu in zip(copies, (None, torch.arange(N + 1).cuda() * T)):
        s = dict(zip(("k_scale", "v_scale"), c[2:]))
        outs.append(kda.cache_append(k, v, *c[:2], table, i32(held), q=q, rope=rope, cu_seqlens=cu, granted=i32(lengths), **s))
    few = [min(T, max(0, b - a)) for a, b in zip(held, lengths)]
    which = torch.cat([n * T + torch.arange(m) for n, m in enumerate(few)]).cuda()
    want = torch.zeros_like(q)
    if sum(few):
        s = dict(zip(("k_scale", "v_scale"), copies[2][2:]))
        cu = torch.tensor([0] + few).cumsum(0).cuda()
        want[which] = kda.cache_append(k[which], v[which], *copies[2][:2], table, i32(held), q=q[which], rope=rope, cu_seqlens=cu, **s)
    for out, c in zip(outs, copies):
        assert torch.equal(out, want)
        for a, b in zip(c, copies[2]):
            assert torch.equal(bits(a), bits(b))


def test_granted_refuses(kda):  # noqa: F811
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    x, (kc, vc) = torch.zeros(3, 1, 64, dtype=torch.bfloat16, device="cuda"), kda.new_cache(3, 16, 1, 64, 64)
    call = lambda g: kda.cache_append(x, x, kc, vc, i32(3, 1), i32(3), granted=g)  # noqa: E731
    assert call(i32(3)) is None and call(None) is None
    for bad in (i32(2), i32(3, 1), i32(3).long(), i32(3).cpu(), i32(6)[::2]):
        with pytest.raises(ValueError, match="granted"):
            call(bad)
    with pytest.raises(TypeError, match="granted"):
        call([1, 2, 3])


@pytest.mark.parametrize("args", [["--eight-bit"], ["--eight-bit", "--window", "40", "--sinks", "3"], ["--window", "33", "--sinks", "4"],
                                  ["--no-graph", "--eight-bit", "--batch", "3", "--prompt", "70"]])
def test_example_runs(args):
    """The example with caches in 8 bits, and with a window: it runs, finds its pages, and is content with itself."""
    spec = importlib.util.spec_from_file_location("serve_hybrid", os.path.join(ROOT, "examples", "serve_hybrid.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main(args + ["--tokens", "20"]) <= 0.05  # what it asks when run as a script


def test_on_another_stream(kda):  # noqa: F811
    """The kernels run on the current stream: work queued there before and after them is in order with them."""
    gen, N, size, pool = _gen(3), 3, 16, 64
    side = torch.cuda.Stream()
    cache = kda.new_cache(pool, size, 2, 128, 128, dtype=E4M3)
    scales = dict(k_scale=cache[2], v_scale=cache[3])
    rows = [300, 1, 200]
    x = [torch.randn(sum(rows), 2, 128, generator=gen).bfloat16().pin_memory() for _ in range(2)]
    q = torch.randn(N, 8, 128, generator=gen).bfloat16()
    new = torch.tensor(rows, dtype=torch.int32).pin_memory()
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    table, lens, wanted, count, free = i32(N, 20) - 1, i32(N), i32(N), i32(1), torch.arange(pool, dtype=torch.int32, device="cuda")
    gq = q.cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        wanted.copy_(new, non_blocking=True)
        count.fill_(pool)
        k, v = (t.cuda(non_blocking=True) for t in x)
        cu, _, granted = kda.cache_resize(table, lens, wanted, free, count, size)
        kda.cache_append(k, v, *cache[:2], table, lens, cu_seqlens=cu, **scales)
        o, lse = kda.cache_attend(gq, *cache[:2], table, granted, **scales)
        o, lse = o + 0, lse + 0
    side.synchronize()
    back = [bits(t).cpu().view(t.dtype) for t in cache]
    check8("bf16", (o, lse), attend8_ref(q, *back, table.cpu(), rows, 128 ** -0.5, 0, 0))
    at = torch.cat([torch.arange(n) for n in rows])
    page = table.cpu()[torch.repeat_interleave(torch.arange(N), torch.tensor(rows)), at // size].long()
    stands = back[1].float()[page, at % size] * back[3][page, at % size // 16][..., None]
    assert ((stands - x[1].float()).abs() <= 2.0 ** -4 * x[1].float().abs() + 2.0 ** -10 * back[3].max()).all()
