"""Attention of one token with a window and a few first rows that stay visible, against 64 bits.

The bounds are those of attention without first rows: only which rows are summed is different."""
import math

import pytest
import torch

from tests.test_gpu_serve import DT, ROUND, U, _gen, check_attend, kda, make_cache, make_table, run_attend  # noqa: F401

pytestmark = pytest.mark.gpu


def visible(end, window, sinks):
    begin = max(0, end - window) if window else 0
    return torch.cat([torch.arange(min(sinks, begin)), torch.arange(begin, max(begin, end))])


def sinks_ref(q, kc, vc, table, lens, scale, window, sinks, size):
    """Row by row in 64 bits: o, lse, and the bounds of their errors (that of o before its rounding)."""
    pair = 2.0 ** -16 if kc.dtype == torch.bfloat16 else 0.0
    N, HQ, K = q.shape
    HKV, V, pages = kc.shape[2], vc.shape[3], kc.shape[0]
    o, lse = torch.zeros(N, HQ, V, dtype=torch.float64), torch.full((N, HQ), -math.inf, dtype=torch.float64)
    err, err_lse = torch.zeros(N, HQ, V, dtype=torch.float64), torch.zeros(N, HQ, dtype=torch.float64)
    for n in range(N):
        pos = visible(int(lens[n]), window, sinks)
        pos = pos[pos < table.shape[1] * size]
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


CASES = [
    # lens, HQ, HKV, K, V, page, window, sinks, layout
    ([0, 1, 2, 5, 6, 7, 8, 9, 40, 100], 4, 2, 128, 128, 16, 5, 2, "heads first"),
    ([300, 0, 1, 129], 5, 1, 128, 64, 27, 30, 1, "rows first"),
    ([700, 33, 64, 65], 16, 2, 64, 128, 64, 64, 64, "shared pool"),
    ([513, 1025, 7], 12, 4, 128, 128, 100, 1, 300, "rows first"),
    ([900, 100, 0, 40], 8, 8, 64, 64, 20, 129, 17, "shared pool"),
    ([70, 2, 1, 33], 3, 3, 128, 128, 5, 1, 31, "heads first"),
    ([400, 250], 20, 1, 128, 128, 32, 250, 4, "heads first"),
    ([9000], 32, 1, 64, 64, 16, 6000, 333, "rows first"),
    ([20000], 2, 1, 128, 128, 64, 17000, 2000, "heads first"),
    ([90] * 90, 4, 4, 64, 128, 16, 30, 10, "heads first"),
    ([3000, 1, 2999, 2005], 6, 2, 128, 128, 128, 2000, 5, "shared pool"),
    ([3000, 10, 2000, 700] * 12, 16, 8, 128, 64, 16, 1500, 100, "heads first"),
    ([100, 2], 2, 2, 64, 64, 16, 2 ** 31 - 1, 2 ** 31 - 1, "heads first"),
    ([100, 2], 2, 2, 64, 64, 16, 3, 2 ** 31 - 1, "heads first"),
    ([100, 2], 2, 2, 64, 64, 16, 0, 7, "heads first"),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_sinks(kda, case, dtype):  # noqa: F811
    lens, HQ, HKV, K, V, size, window, sinks, layout = CASES[case]
    gen = _gen(100 + case)
    pages = sum(-(-x // size) for x in lens) + 2
    kc, vc = make_cache(gen, pages, size, HKV, K, V, dtype, layout)
    table = make_table(gen, lens, size, pages)
    own = torch.zeros(pages, size, dtype=torch.bool)  # whatever is not visible holds NaN
    for n, m in enumerate(lens):
        pos = visible(m, window, sinks)
        own[table[n, pos // size].long(), pos % size] = True
    kc[~own], vc[~own] = math.nan, math.nan
    q = (2 * torch.randn(len(lens), HQ + 3, K, generator=gen)).to(DT[dtype])[:, 2:-1]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_attend(kda, q, kc, vc, table, lens, window=window, sinks=sinks, status=status)
    assert int(status) == 0
    check_attend(dtype, got, sinks_ref(q, kc, vc, table, lens, K ** -0.5, window, sinks, size))
    again = run_attend(kda, q, kc, vc, table, lens, window=window, sinks=sinks)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("split, N, L, window, sinks", [
    ("cache_attend", 300, 100, 40, 20), ("cache_attend_cluster", 2, 2000, 800, 100),
    ("cache_attend_parts", 1, 30000, 9000, 1001), ("cache_attend_shares", 48, 5000, 3000, 70)])
def test_sinks_of_each_split(kda, split, N, L, window, sinks, dtype):  # noqa: F811
    """First rows that end inside a tile, a turn and a page, in every way that rows are given to CTAs; lengths that differ,
    among them ones where first rows and window touch or overlap."""
    gen, size, heads, D = _gen(7), 27, 8 if N == 48 else 2, 64
    width = -(-L // size)
    some = 4
    kc, vc = make_cache(gen, some * width, size, heads, D, D, dtype, "heads first")
    table = (torch.arange(N)[:, None] % some * width + torch.arange(width)).to(torch.int32)
    lens = [(L, window + sinks, window + sinks // 2, L - 77)[n % 4] for n in range(N)]
    q = torch.randn(some, 2 * heads, D, generator=gen).to(DT[dtype])
    got = run_attend(kda, q[torch.arange(N) % some], kc, vc, table, lens, window=window, sinks=sinks)
    if dtype == "bf16":
        assert kda.load().kda_launch_name(0).decode() == split
    few = list(range(min(N, some)))
    ref = sinks_ref(q[few], kc, vc, table[few], lens, D ** -0.5, window, sinks, size)
    check_attend(dtype, (got[0][few], got[1][few]), ref)
    for n in range(N):
        assert torch.allclose(got[0][n].float(), got[0][n % some].float(), rtol=2 * ROUND[dtype], atol=2.0 ** -18)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sinks_leave_out_what_does_not_exist(kda, dtype):  # noqa: F811
    """A first page that does not exist, and lengths beyond the table: flagged, and what exists is attended."""
    gen, size = _gen(9), 16
    kc, vc = make_cache(gen, 6, size, 2, 64, 64, dtype, "heads first")
    q = torch.randn(3, 4, 64, generator=gen).to(DT[dtype])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.tensor([[6, 0, 1], [2, 3, 4], [5, -7, 0]], dtype=torch.int32)
    for lens, flag in (([20, 48, 16], 1), ([0, 47, 16], 0), ([0, 50, 0], 1), ([0, 2 ** 31 - 1, 0], 1), ([0, 0, 30], 1),
                       ([-3, -1, 5], 0)):
        status.zero_()
        got = run_attend(kda, q, kc, vc, table, lens, window=6, sinks=9, status=status)
        assert int(status) == flag
        check_attend(dtype, got, sinks_ref(q, kc, vc, table, lens, 0.125, 6, 9, size))


def test_sinks_refused_and_workspace(kda):  # noqa: F811
    kc, vc = kda.new_cache(400, 16, 2, 64, 64)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    table, lens = torch.zeros(1, 400, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(kda.KdaError, match="KDA_ERR_INVALID_ARG"):
        kda.cache_attend(q, kc, vc, table, lens, window=4, sinks=-1)
    with pytest.raises(ValueError):
        kda.cache_attend(q, kc, vc, table, lens, window=4, sinks=2 ** 31)
    need = [kda.cache_attend_workspace_bytes(q, kc, vc, table, window=w, sinks=s) for w, s in ((20, 0), (20, 6000), (0, 9))]
    assert need[0] < need[1] and need[2] == kda.cache_attend_workspace_bytes(q, kc, vc, table)
    ws = torch.empty(need[1], dtype=torch.uint8, device="cuda")
    lens.fill_(6400)
    one = kda.cache_attend(q, kc, vc, table, lens, window=20, sinks=6000, ws=ws)
    assert torch.equal(one[0], kda.cache_attend(q, kc, vc, table, lens, window=20, sinks=6000)[0])


def test_sinks_in_a_graph(kda):  # noqa: F811
    """A captured call while the sequence grows past its window."""
    gen, size = _gen(12), 16
    kc, vc = make_cache(gen, 16, size, 2, 64, 64, "bf16", "heads first")
    table, q = torch.arange(16, dtype=torch.int32)[None], torch.randn(1, 4, 64, generator=gen).bfloat16()
    gk, gv, gq, gt, lens = kc.cuda(), vc.cuda(), q.cuda(), table.cuda(), torch.ones(1, dtype=torch.int32, device="cuda")
    kda.cache_attend(gq, gk, gv, gt, lens, window=10, sinks=3)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        o, lse = kda.cache_attend(gq, gk, gv, gt, lens, window=10, sinks=3)
    for now in (1, 10, 11, 12, 13, 14, 200, 256):
        lens.fill_(now)
        graph.replay()
        torch.cuda.synchronize()
        check_attend("bf16", (o, lse), sinks_ref(q, kc, vc, table, [now], 0.125, 10, 3, size))


def test_workspace_bytes_go_by_sizes(kda):  # noqa: F811
    """Of a cache in 16 or 32 bits q's sizes count, and not its type; of one in 8 bits the type is that of a call."""
    table = torch.zeros(3, 200, dtype=torch.int32, device="cuda")
    for dt in (torch.bfloat16, torch.float32):
        kc, vc = kda.new_cache(4, 16, 2, 64, 128, dtype=dt)
        need = {kda.cache_attend_workspace_bytes(torch.zeros(3, 4, 64, dtype=t, device="cuda"), kc, vc, table)
                for t in (torch.bfloat16, torch.float32, torch.float16, torch.int8)}
        assert len(need) == 1 and need.pop() > 0
    kc, vc = kda.new_cache(4, 16, 2, 64, 128, dtype=torch.float8_e4m3fn)[:2]
    with pytest.raises(TypeError, match="q"):
        kda.cache_attend_workspace_bytes(torch.zeros(3, 4, 64, dtype=torch.float16, device="cuda"), kc, vc, table)
