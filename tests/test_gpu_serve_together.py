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
