"""Page tables, offsets and slots from lengths on the GPU, against the rules as they are written, one page at a time."""
import pytest
import torch

from tests.test_gpu_serve import _gen, kda  # noqa: F401

pytestmark = pytest.mark.gpu


def resize_ref(table, lens, wanted, free, count, size, rows):
    """Lists in, lists out; says whether something was not as it should be."""
    table, free, bad = [list(x) for x in table], list(free), False
    pool, width = len(free), len(table[0]) if table else 0
    pages = lambda n: -(-max(n, 0) // size)  # noqa: E731
    if not 0 <= count <= pool:
        bad, count = True, min(max(count, 0), pool)
    for n, (a, b) in enumerate(zip(lens, wanted)):
        bad |= pages(b) <= pages(a) and pages(a) > width
        for j in range(pages(b), min(pages(a), width)):
            bad |= not 0 <= table[n][j] < pool
            if count < pool:
                free[count] = table[n][j]
                count += 1
            else:
                bad = True
            table[n][j] = -1
    room, asked, granted = count, 0, []
    for n, (a, b) in enumerate(zip(lens, wanted)):
        fits, take = pages(b) <= width, max(0, pages(b) - pages(a))
        asked += take if fits else 0
        served = fits and (take == 0 or asked <= room)
        granted.append(b if served else a)
        bad |= not served
        for j in range(pages(a), pages(b)) if served else ():
            count -= 1
            page = free[count]
            bad |= not 0 <= page < pool
            table[n][j] = page if 0 <= page < pool else -1
    cu, slots = [0], []
    for n, (a, b) in enumerate(zip(lens, wanted)):
        new = range(max(a, 0), max(b, 0))
        cu.append(cu[-1] + len(new))
        for t in new:
            page = table[n][t // size] if granted[n] == b and t // size < width else -1
            slots.append(page * size + t % size if 0 <= page < pool else -1)
            bad |= rows > len(slots) - 1 and granted[n] == b and not 0 <= page < pool
    bad |= rows > 0 and len(slots) > rows
    return table, free, count, cu, (slots + [-1] * rows)[:rows], granted, bad


def check(kda, table, lens, wanted, free, count, size, rows):  # noqa: F811
    i32 = lambda x, *s: torch.tensor(x, dtype=torch.int32).reshape(*s).cuda()  # noqa: E731
    N, width = len(lens), len(table[0]) if table else 3
    t = torch.full((N, width + 2), 77, dtype=torch.int32, device="cuda")  # rows apart
    if N:
        t[:, :width] = i32(table, N, width)
    f, c, status = i32(free, -1), i32([count], 1), i32([0], 1)
    cu, slots, granted = kda.cache_resize(t[:, :width], i32(lens, -1), i32(wanted, -1), f, c, size, rows=rows, status=status)
    ref = resize_ref(table, lens, wanted, free, count, size, rows)
    assert t[:, :width].tolist() == ref[0] and (t[:, width:] == 77).all()
    assert f.tolist() == ref[1] and int(c) == ref[2]
    assert cu.tolist() == ref[3] and slots.tolist() == ref[4] and granted.tolist() == ref[5]
    assert bool(int(status)) == ref[6]
    assert cu.dtype == slots.dtype == torch.int64 and granted.dtype == torch.int32
    return ref


def pool_of(gen, lens, size, width, spare, capacity=None):
    """A table of scattered pages for these lengths and the list of the others, with room for all."""
    need = [-(-max(x, 0) // size) for x in lens]
    pool = capacity or sum(need) + spare
    order = torch.randperm(pool, generator=gen).tolist()
    table = [[order.pop() if j < m else -1 for j in range(width)] for m in need]
    return table, order[:spare] + [-5] * (pool - len(order[:spare])), len(order[:spare])


CASES = [
    # N, longest, page, rows beyond the new ones
    (1, 1, 1, 0), (1, 100, 16, 5), (3, 40, 5, 0), (7, 1000, 64, 1), (33, 300, 16, 0), (256, 200, 16, 7), (1000, 60, 4, 0),
    (1024, 30, 1, 100), (1025, 30, 16, 0), (2500, 90, 7, 3), (40, 9000, 16, 0), (2, 70000, 8, 0),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_resize(kda, case):  # noqa: F811
    """Sequences that grow, shrink, end, begin, stay or are inactive, with pages enough: there, and on to other lengths."""
    N, longest, size, more = CASES[case]
    gen = _gen(case)
    draw = lambda: torch.randint(0, longest + 1, (N,), generator=gen)  # noqa: E731
    kind = lambda: torch.randint(0, 6, (N,), generator=gen)  # noqa: E731
    lens = torch.where(kind() == 0, -1, draw()).tolist()
    width = -(-longest // size)
    table, free, count = pool_of(gen, lens, size, width, N * width)
    for turn in range(3):
        k = kind()
        wanted = torch.where(k == 0, -1, torch.where(k == 1, 0, torch.where(k == 2, torch.tensor(lens), torch.where(
            k == 3, (torch.tensor(lens) + 1).clamp(max=longest), draw())))).tolist()
        rows = sum(max(0, max(b, 0) - max(a, 0)) for a, b in zip(lens, wanted)) + more
        table, free, count, cu, slots, granted, bad = check(kda, table, lens, wanted, free, count, size, rows)
        assert not bad and granted == wanted
        used = [x for r in table for x in r if x >= 0]
        assert len(set(used + free[:count])) == len(free) == len(used) + count  # every page has one place
        lens = wanted


@pytest.mark.parametrize("N, longest, size", [(5, 64, 16), (300, 64, 16), (1500, 40, 4)])
def test_resize_runs_out_of_pages(kda, N, longest, size):  # noqa: F811
    """Pages for some of the sequences alone: those in front are served, the others keep what they have; what comes back is
    there for others in the same call."""
    gen = _gen(N)
    lens = torch.randint(1, longest + 1, (N,), generator=gen).tolist()
    width = -(-longest // size) + 1
    for spare in (0, 1, N // 2, 2 * N):
        table, free, count = pool_of(gen, lens, size, width, spare)
        wanted = torch.randint(0, longest + size + 1, (N,), generator=gen).tolist()
        check(kda, table, lens, wanted, free, count, size, 0)
        check(kda, table, lens, [x + size for x in lens], free, count, size, 3 * N)
    # one that wants more than its row of the table holds is left out, and the others are served
    wanted = list(lens)
    wanted[N // 2], wanted[-1] = width * size + 1, lens[-1] + 1
    table, free, count = pool_of(gen, lens, size, width, 2 * N)
    ref = check(kda, table, lens, wanted, free, count, size, 0)
    assert ref[5][N // 2] == lens[N // 2] and ref[5][-1] == wanted[-1]


@pytest.mark.parametrize("alone", [True, False])
def test_resize_with_what_should_not_be(kda, alone):  # noqa: F811
    """Entries that are no pages, a list without room, a count beyond the list, lengths beyond the table, too few rows."""
    rows = 10 if alone else 6000
    table = [[3, 9, -1, -1], [1, -7, 2, -1], [0, -1, -1, -1], [4, -1, -1, -1]]
    lens, free = [8, 12, 3, 4], [5, 6, 99, 7, -1, -1, -1, -1]
    check(kda, table, lens, [4, 4, 4, 4], free, 4, 4, rows)       # what goes back is no page
    check(kda, table, lens, [8, 12, 12, 8], free, 4, 4, rows)     # nor what is taken
    check(kda, table, lens, [9, 13, 5, 5], free, 2, 4, rows)
    check(kda, table, lens, [0, 0, 0, 0], free, 6, 4, rows)       # no room for all
    check(kda, table, lens, [0, 4, 3, 4], free, 8, 4, rows)
    check(kda, table, lens, [9, 12, 3, 4], free, 9, 4, rows)      # a count beyond the list
    check(kda, table, lens, [9, 12, 3, 4], free, -1, 4, rows)
    check(kda, table, [8, 40, 3, 4], [8, 4, 3, 4], free, 2, 4, rows)  # a length beyond the table
    check(kda, table, [8, 40, 3, 4], [8, 30, 3, 5], free, 2, 4, rows)
    check(kda, table, [8, 12, 3, 2 ** 31 - 1], [8, 12, 3, 2 ** 31 - 1], free, 2, 4, rows)
    check(kda, table, [7, 11, 3, 3], [8, 12, 4, 4], free, 2, 4, 0 if alone else 5000)
    check(kda, table, [7, 11, 3, 3], [8, 12, 4, 4], free, 2, 4, 2)    # fewer rows than there are
    check(kda, table, [-9, -1, -2 ** 31, 4], [-1, -2 ** 31, 4, -3], free, 2, 4, rows)


def test_resize_of_nothing(kda):  # noqa: F811
    for rows in (0, 5, 9000):
        check(kda, [], [], [], [1, 2, -1], 2, 16, rows)
    check(kda, [[], []], [0, 0], [0, 5], [1, 2, -1], 2, 16, 4)


def test_resize_refuses(kda):  # noqa: F811
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    call = lambda **c: kda.cache_resize(**{**dict(page_table=i32(3, 4), kv_lens=i32(3), new_lens=i32(3),  # noqa: E731
                                                  free_pages=i32(12), free_count=i32(1), page_size=16), **c})
    assert [x.shape for x in call(rows=7)] == [(4,), (7,), (3,)]
    for bad in (dict(page_table=i32(3, 4).long()), dict(page_table=i32(4, 3).t()), dict(page_table=i32(12)), dict(kv_lens=i32(2)),
                dict(new_lens=i32(3).long()), dict(new_lens=i32(3).cpu()), dict(free_pages=i32(3, 4)), dict(free_pages=i32(12).float()),
                dict(free_count=i32(2)), dict(status=i32(2)), dict(rows=-1), dict(page_size=2 ** 31), dict(page_table=i32(3, 4).cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(page_size=0), dict(page_size=-4), dict(page_table=i32(4).expand(3, 4))):
        with pytest.raises(kda.KdaError, match="KDA_ERR_INVALID_ARG"):
            call(**bad)
    n = 65536
    with pytest.raises(kda.KdaError, match="KDA_ERR_UNSUPPORTED"):
        call(page_table=i32(n, 1), kv_lens=i32(n), new_lens=i32(n))


@pytest.mark.parametrize("N, width", [(4, 8), (1200, 3)])
def test_resize_in_a_graph(kda, N, width):  # noqa: F811
    """A captured call that gives every sequence one more row at each replay, until the pages run out."""
    size, pool = 4, N * width
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    table, lens, free = i32(N, width).fill_(-1), i32(N), torch.arange(pool, dtype=torch.int32, device="cuda")
    count, status = i32(1).fill_(pool), i32(1)

    def step():
        _, slots, granted = kda.cache_resize(table, lens, lens + 1, free, count, size, rows=N, status=status)
        lens.copy_(granted)
        return slots

    step()  # outside of the capture
    state = [table.tolist(), lens.tolist(), free.tolist(), int(count)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        slots = step()
    for _ in range(width * size + 1):
        graph.replay()
        ref = resize_ref(state[0], state[1], [x + 1 for x in state[1]], state[2], state[3], size, N)
        assert slots.tolist() == ref[4] and table.tolist() == ref[0] and lens.tolist() == ref[5] and int(count) == ref[2]
        state = [ref[0], ref[5], ref[1], ref[2]]
    assert lens.tolist() == [width * size] * N and int(status)
